"""The block-sparse step's operators from their definitions, in float64 (numpy)."""
import numpy as np
import torch


def f64(t):
    """A tensor's values; uint8 tensors are E4M3 codes."""
    t = t.detach().cpu()
    return (t.view(torch.float8_e4m3fn) if t.dtype == torch.uint8 else t).to(torch.float64).numpy()


def step_tables(ctx, new, table, bs, free, head, T):
    """(table, head, qsl, seq, positions, slots); the caller checks that the step fits."""
    table = table.copy()
    qsl, seq, pos, slots = [0], [], [], []
    for r, (c, n) in enumerate(zip(ctx, new)):
        for page in range(-(-c // bs), -(-(c + n) // bs)):
            table[r, page] = free[head]
            head += 1
        for p in range(c, c + n):
            pos.append(p)
            slots.append(int(table[r, p // bs]) * bs + p % bs if table[r, p // bs] >= 0 else -1)
        qsl.append(qsl[-1] + n)
        seq.append(c + n)
    pad = T - len(pos)
    return table, head, qsl, seq, pos + [-1] * pad, slots + [-1] * pad


def rope(x, weight, eps, cos_sin, pos, interleaved):
    """x [T, H, d] -> (rotated values, |a| + |b| of each element's pair: what an error of the parts scales with)."""
    x = x.copy()
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight
    size = np.abs(x)
    if cos_sin is None or cos_sin.shape[1] == 0:
        return x, size
    half = cos_sin.shape[1] // 2
    c, s = cos_sin[pos, None, :half], cos_sin[pos, None, half:]
    ia = np.arange(half) * 2 if interleaved else np.arange(half)
    ib = ia + 1 if interleaved else ia + half
    a, b = x[..., ia], x[..., ib]
    size[..., ia] = size[..., ib] = np.abs(a) + np.abs(b)
    x[..., ia], x[..., ib] = a * c - b * s, b * c + a * s
    return x, size


def unit_exponent(a):
    """The least e >= -60 with a <= 127 * 2^e."""
    e = -60
    while a > 127 * 2.0 ** e:
        e += 1
    return e


def page_bounds(keys):
    """keys [bs, d] -> (lo codes, hi codes, scale)."""
    if not np.isfinite(keys).all():
        return np.zeros(keys.shape[1]), np.zeros(keys.shape[1]), np.inf
    unit = 2.0 ** unit_exponent(np.abs(keys).max())
    return np.floor(keys.min(0) / unit), np.ceil(keys.max(0) / unit), unit


def query_codes(q):
    """q [d] -> (codes, unit)."""
    if not np.isfinite(q).all():
        return np.zeros_like(q), 1.0
    unit = 2.0 ** unit_exponent(np.abs(q).max())
    return np.rint(q / unit), unit


def positions(qsl, seq):
    """[(token, request, position)] of a batch."""
    return [(t, r, seq[r] - qsl[r + 1] + t) for r in range(len(seq)) for t in range(qsl[r], qsl[r + 1])]


def select_pages(q, bounds, scales, table, qsl, seq, bs, first, last, K, selected):
    """selected [T, Hkv, K] as pka_select_pages leaves it (float64 q, bounds; int table)."""
    out = selected.copy()
    Hkv, G = bounds.shape[1], q.shape[1] // bounds.shape[1]
    for t, r, p in positions(qsl, seq):
        n = p // bs + 1
        for g in range(Hkv):
            chosen = list(range(n))
            if n > K:
                blk = table[r, :n]
                score = np.full(n, -np.inf)
                for h in range(g * G, (g + 1) * G):
                    c, unit = query_codes(q[t, h])
                    dots = np.maximum(c * bounds[blk, g, 0], c * bounds[blk, g, 1]).sum(-1)
                    with np.errstate(invalid="ignore"):
                        score = np.maximum(score, dots * scales[blk, g] * unit)
                score = np.where(np.isinf(scales[blk, g]), np.inf, score)
                rest = sorted(range(first, n - last), key=lambda i: (-score[i], i))[:K - first - last]
                chosen = sorted(list(range(first)) + rest + list(range(n - last, n)))
            out[t, g] = chosen + [-1] * (K - len(chosen))
    return out


def sparse_attn(q, k_cache, v_cache, table, qsl, seq, selected, scale, unit=(1.0, 1.0)):
    """out [T, Hq, d], lse [T, Hq], sum_j softmax_j |V_j| (rows of no request: NaN)."""
    T, Hq, d = q.shape
    Hkv, bs = k_cache.shape[1], k_cache.shape[2]
    out, lse, size = np.full((T, Hq, d), np.nan), np.full((T, Hq), np.nan), np.full((T, Hq, d), np.nan)
    for t, r, p in positions(qsl, seq):
        for h in range(Hq):
            g = h // (Hq // Hkv)
            keys = [(e, j) for e in selected[t, g] if e >= 0 for j in range(bs) if e * bs + j <= p]
            if not keys:
                out[t, h], size[t, h], lse[t, h] = 0, 0, -np.inf
                continue
            blk, off = table[r, [e for e, _ in keys]], [j for _, j in keys]
            s = k_cache[blk, g, off] @ q[t, h] * (scale * unit[0])
            m = s.max()
            w = np.exp(s - m)
            lse[t, h] = m + np.log(w.sum())
            v = v_cache[blk, g, off] * unit[1]
            out[t, h], size[t, h] = w @ v / w.sum(), w @ np.abs(v) / w.sum()
    return out, lse, size
