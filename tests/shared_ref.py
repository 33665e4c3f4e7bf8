"""The definitions of the calls over shared pages in float64 and plain Python, for the tests."""
import numpy as np


def beam_select(logits, scores, finished, end_token, keep):
    """logits [G * W, V], scores [G, W], finished [G, W] or None -> (scores [G, keep] float64, parents, tokens, finished,
    whether a row was refused)."""
    x = np.asarray(logits, np.float64)
    G, W = np.shape(scores)
    out = (np.full((G, keep), -np.inf), np.full((G, keep), -1), np.full((G, keep), -1), np.zeros((G, keep), int))
    bad = False
    for g in range(G):
        cand = []
        for i in range(W):
            s, row = float(scores[g][i]), x[g * W + i]
            if np.isnan(s) or s == np.inf:
                bad = True
            elif s == -np.inf:
                continue
            elif finished is not None and finished[g][i]:
                cand.append((-s, i, 0.0, end_token, 1))
            elif np.isnan(row).any() or (row == np.inf).any():
                bad = True
            elif (row > -np.inf).any():
                m = row.max()
                lse = m + np.log(np.exp(row - m).sum())
                best = np.lexsort((np.arange(row.size), -row))[:keep]
                cand += [(-(s + (row[v] - lse)), i, -row[v], int(v), int(v == end_token)) for v in best if row[v] > -np.inf]
        for k, (s, i, _, v, f) in enumerate(sorted(cand)[:keep]):
            out[0][g, k], out[1][g, k], out[2][g, k], out[3][g, k] = -s, g * W + i, v, f
    return (*out, bad)


def fork_pages(parents, ctx, table, bs, counts, free, head, num_blocks, table_out):
    """-> (ctx_out, table_out, counts, free, head, copy_src, copy_dst): the definition, place by place."""
    table, table_out = np.array(table), np.array(table_out)
    counts, free = list(counts), list(free)
    held = [-(-c // bs) for c in ctx]
    children = [[i for i, p in enumerate(parents) if p == r] for r in range(len(ctx))]
    ctx_out, src, dst, taken = [], [], [], 0
    for i, p in enumerate(parents):
        if p < 0:
            ctx_out.append(0), src.append(-1), dst.append(-1)
            continue
        ctx_out.append(ctx[p])
        table_out[i, :held[p]] = table[p, :held[p]]
        if ctx[p] % bs and children[p][0] != i:
            page = free[head + taken]
            taken += 1
            src.append(int(table[p, held[p] - 1])), dst.append(page)
            table_out[i, held[p] - 1] = page
        else:
            src.append(-1), dst.append(-1)
    gone = []
    for r, kids in enumerate(children):
        for c in range(held[r]):
            page, n = int(table[r, c]), len(kids)
            if 0 <= page < num_blocks:
                counts[page] += (min(n, 1) if ctx[r] % bs and c == held[r] - 1 else n) - 1
    for r in range(len(ctx)):
        for c in range(held[r]):
            page = int(table[r, c])
            if 0 <= page < num_blocks and counts[page] < 0:
                counts[page] = 0
                gone.append(page)
    head = head + taken - len(gone)
    free[head:head + len(gone)] = gone
    return ctx_out, table_out, counts, free, head, src, dst


def prefix_attention(q, k_cache, v_cache, table, qsl, seq, starts, prefix, scale, v_scale=1.0):
    """q [T, Hq, d], caches [nb, Hkv, bs, d] float64 -> out, lse, and for each output the sum of the weights times the
    values' magnitudes, and the largest sum of |q_i k_i| * scale (for tolerances)."""
    T, Hq, d = q.shape
    _, Hkv, bs, _ = k_cache.shape
    G = Hq // Hkv
    out, mag = np.full(q.shape, np.nan), np.full(q.shape, np.nan)
    lse, reach = np.full((T, Hq), np.nan), np.full((T, Hq), np.nan)
    for g in range(len(prefix)):
        reqs = [r for r in range(starts[g], starts[g + 1]) if qsl[r + 1] > qsl[r]]
        for r in reqs:
            n = seq[r]
            pos = np.arange(n)
            row = np.where(pos < prefix[g], table[reqs[0]][pos // bs], table[r][pos // bs]) if len(
                range(starts[g], starts[g + 1])) > 1 else table[r][pos // bs]
            K, V = k_cache[row, :, pos % bs], v_cache[row, :, pos % bs]  # [n, Hkv, d]
            for t in range(qsl[r], qsl[r + 1]):
                p = n - (qsl[r + 1] - t)
                for h in range(Hq):
                    k, v = K[:p + 1, h // G], V[:p + 1, h // G]
                    s = scale * (k @ q[t, h])
                    m = s.max()
                    w = np.exp(s - m)
                    z = w.sum()
                    out[t, h] = v_scale * (w / z) @ v
                    mag[t, h] = v_scale * (w / z) @ np.abs(v)
                    lse[t, h] = m + np.log(z)
                    reach[t, h] = scale * (np.abs(k) @ np.abs(q[t, h])).max()
    return out, lse, mag, reach
