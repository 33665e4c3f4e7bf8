"""The block-sparse step on the GPU against its definitions in float64.

Tolerances, from the arithmetic: a rounding to bf16 is off by at most 2^-8 of the value
(torch.finfo(bf16).eps / 2), to E4M3 by 2^-4 of it or half the least code; whole numbers
(tables, codes, page lists) are equal."""
import threading

import numpy as np
import pytest
import torch

from oracle import fp8
from paged_kv_attention_07_gb300 import pka
from tests import sparse_ref as ref

pytestmark = pytest.mark.gpu

BF16, I32, I64 = torch.bfloat16, torch.int32, torch.int64
E = pka.DEVERR


def dev(x, dtype):
    return torch.tensor(np.asarray(x), dtype=dtype, device="cuda")


def word():
    return torch.zeros(1, dtype=I32, device="cuda")


def randn(rng, *shape):
    return torch.from_numpy(rng.standard_normal(shape)).to(BF16).cuda()


# ---------------------------------------------------------------- step tables


def tables_case(ctx, new, bs, T, free, head, width=None, seed=0, in_place=False, positions=True):
    rng = np.random.default_rng(seed)
    B = len(ctx)
    width = width or max(-(-(c + n) // bs) for c, n in zip(ctx, new)) + 2
    table0 = rng.integers(0, 10000, (B, width))
    s = dict(ctx=dev(ctx, I32), new=dev(new, I32), table=dev(table0, I32), free=dev(free, I32), head=dev([head], I32),
             qsl=dev([-7] * (B + 1), I32), seq=dev([-7] * B, I32), pos=dev([-7] * T, I32) if positions else None,
             slots=dev([-7] * T, I64), err=word())
    s["head_out"] = s["head"] if in_place else dev([-7], I32)
    pka.pka_step_tables(s["ctx"], s["new"], s["table"], bs, s["free"], s["head"], s["head_out"], s["qsl"], s["seq"],
                        s["pos"], s["slots"], error_word=s["err"])
    return s, table0


@pytest.mark.parametrize("B,bs,longest,most,pad", [
    (1, 16, 0, 1, 0), (1, 16, 100, 1, 3), (7, 1, 20, 5, 2), (33, 24, 300, 70, 0), (64, 64, 5000, 1, 11),
    (1500, 16, 200, 3, 1), (4096, 32, 64, 2, 0), (5, 128, 3000, 2000, 17), (40, 64, 0, 900, 64),
])
@pytest.mark.parametrize("in_place", [False, True])
def test_step_tables(B, bs, longest, most, pad, in_place):
    rng = np.random.default_rng(B + bs)
    ctx, new = rng.integers(0, longest + 1, B).tolist(), rng.integers(0 if B > 1 else 1, most + 1, B).tolist()
    need = sum(-(-(c + n) // bs) - -(-c // bs) for c, n in zip(ctx, new))
    head = 5
    free = rng.permutation(need + head)  # exactly as many as the step takes
    T = sum(new) + pad
    s, table0 = tables_case(ctx, new, bs, T, free, head, in_place=in_place)
    want = ref.step_tables(ctx, new, table0, bs, free.tolist(), head, T)
    assert int(s["err"]) == 0
    for name, w in zip(("table", "head_out", "qsl", "seq", "pos", "slots"), want):
        assert np.array_equal(s[name].cpu().numpy().reshape(np.shape(w)), np.asarray(w)), name
    if not in_place:
        assert int(s["head"]) == head


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,most,pad", [
    (255, 1, 0), (256, 1, 0), (256, 6, 5), (257, 1, 0), (31, 50, 0), (256, 8, 0), (2, 511, 3)])
def test_step_tables_at_the_sizes_of_a_cta(B, most, pad, in_place):
    test_step_tables(B, 16, 100, most, pad, in_place)


def test_step_tables_negative_page_ids_have_no_slots():
    ctx, new, bs = [5, 8], [4, 2], 4
    s, table0 = tables_case(ctx, new, bs, 6, [-3, 11, 12], 0, positions=False)
    want = ref.step_tables(ctx, new, table0, bs, [-3, 11, 12], 0, 6)
    assert s["slots"].tolist() == want[5] and -1 in want[5] and int(s["err"]) == 0


@pytest.mark.parametrize("change,bit", [
    (dict(new=[3, -1, 2]), "QUERY_LEN"), (dict(ctx=[4, -5, 2]), "SEQ_LEN"), (dict(width=1), "BLOCK_TABLE"),
    (dict(T=5), "QUERY_START_LOC"), (dict(free=[1]), "CAPACITY"), (dict(head=-1), "CAPACITY"),
    (dict(head=3), "CAPACITY"), (dict(new=[2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1], width=9), "BLOCK_TABLE"),
])
def test_step_tables_takes_all_or_nothing(change, bit):
    a = dict(ctx=[4, 5, 2], new=[3, 1, 2], bs=4, T=7, free=[20, 21, 22], head=1)
    a.update(change)
    a.setdefault("width", 3)
    s, table0 = tables_case(**a)
    assert int(s["err"]) & E[bit]
    assert np.array_equal(s["table"].cpu().numpy(), table0) and int(s["head_out"]) == a["head"]
    assert not s["qsl"].any() and not s["seq"].any() and (s["slots"] == -1).all() and (s["pos"] == -1).all()


@pytest.mark.parametrize("in_place", [False, True])
def test_step_tables_takes_nothing_on_many_ctas(in_place):
    ctx, new = [700] * 30, [400] * 30
    s, table0 = tables_case(ctx, new, 16, 12100, list(range(100)), 3, in_place=in_place)  # needs 750 pages
    assert int(s["err"]) == E["CAPACITY"] and int(s["head_out"]) == 3
    assert np.array_equal(s["table"].cpu().numpy(), table0)
    assert not s["qsl"].any() and not s["seq"].any() and (s["slots"] == -1).all() and (s["pos"] == -1).all()


# ---------------------------------------------------------------- norm, rotation, cache write


def rope_case(T, Hq, Hkv, d, rotary, interleaved, norm, fp8, packed, bs=16, keep=True, seed=0, nb=None):
    rng = np.random.default_rng(seed)
    heads = Hq + 2 * Hkv
    if packed:
        qkv = randn(rng, T, heads, d) * torch.exp(randn(rng, heads, 1))
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    else:
        q, k, v = (randn(rng, T, h, d) for h in (Hq, Hkv, Hkv))
    nb = nb or -(-T // bs) + 3
    maxp = 500
    angle = rng.uniform(0, 6.28, (maxp, rotary // 2))
    table = torch.from_numpy(np.concatenate([np.cos(angle), np.sin(angle)], 1)).float().cuda() if rotary else None
    cache = lambda: torch.from_numpy(rng.integers(0, 120, (nb, Hkv, bs, d))).to(torch.uint8).cuda() if fp8 \
        else randn(rng, nb, Hkv, bs, d)
    return dict(q=q, k=k, v=v, qw=1 + 0.1 * randn(rng, d) if norm else None, kw=1 + 0.1 * randn(rng, d) if norm else None,
                eps=1e-5, table=table, interleaved=interleaved, pos=dev(rng.integers(0, maxp, T), I32),
                slots=dev(rng.permutation(nb * bs)[:T], I64), q_out=torch.full((T, Hq, d), 7.0, dtype=BF16, device="cuda"),
                k_out=torch.full((T, Hkv, d), 7.0, dtype=BF16, device="cuda") if keep else None,
                v_out=torch.full((T, Hkv, d), 7.0, dtype=BF16, device="cuda") if keep else None, k_cache=cache(),
                v_cache=cache(), scales=(0.03, 0.02) if fp8 else None, err=word())


def rope_call(s, **kw):
    pka.pka_qk_rope_cache_write(s["q"], s["k"], s["v"], s["qw"], s["kw"], s["eps"], s["table"], s["interleaved"],
                                s["pos"], s["slots"], s["q_out"], s["k_out"], s["v_out"], s["k_cache"], s["v_cache"],
                                kv_scales=s["scales"], error_word=s["err"], **kw)


# float32 up to the rounding: the mean of at most 256 squares is off by 256 * 2^-24 at most, its root by
# half of that, and about six more roundings of 2^-24: below 2^-16 of the magnitudes that are combined.
F32 = 2.0 ** -16


def near_bf16(got, want, size):
    return (np.abs(ref.f64(got) - want) <= 2.0 ** -8 * (np.abs(want) + F32 * size) + F32 * size).all()


def near_code(got, want, size, unit):
    """Values of codes (in units) against the value / unit, saturated; half the least code is 2^-10."""
    w, z = want / unit, F32 * size / unit
    w = np.clip(w, -448, 448)
    return (np.abs(ref.f64(got) - w) <= np.maximum(2.0 ** -4 * (np.abs(w) + z), 2.0 ** -10) + z).all()


def rope_check(s, before, rows=None):
    """Every output against the definition for the tokens `rows`; all other elements as they were."""
    table = None if s["table"] is None else ref.f64(s["table"])
    pos = s["pos"].cpu().numpy()
    T, bs = len(pos), s["k_cache"].shape[2]
    rows = np.arange(T) if rows is None else np.asarray(rows, dtype=np.int64)
    w = {n: None if s[n] is None else ref.f64(s[n]) for n in ("qw", "kw")}
    q, qsize = ref.rope(ref.f64(before["q"])[rows], w["qw"], s["eps"], table, pos[rows], s["interleaved"])
    k, ksize = ref.rope(ref.f64(before["k"])[rows], w["kw"], s["eps"], table, pos[rows], s["interleaved"])
    v = ref.f64(before["v"])[rows]
    idx = torch.from_numpy(rows).cuda()
    assert near_bf16(s["q_out"][idx], q, qsize)
    rest = torch.ones(T, dtype=torch.bool)
    rest[rows] = False
    assert torch.equal(s["q_out"].cpu()[rest], before["q_out"].cpu()[rest])
    if s["k_out"] is not None:
        assert near_bf16(s["k_out"][idx], k, ksize)
        assert np.array_equal(ref.f64(s["v_out"][idx]), v)
        assert torch.equal(s["k_out"].cpu()[rest], before["k_out"].cpu()[rest])
    slots = s["slots"].cpu().numpy()[rows]
    limit = s["k_cache"].shape[0] * bs
    on = (slots >= 0) & (slots < limit)
    blk, off = slots[on] // bs, slots[on] % bs
    for name, x, size, n in (("k_cache", k, ksize, 0), ("v_cache", v, np.abs(v), 1)):
        got = s[name].cpu()[blk, :, off]
        if s["scales"]:
            assert near_code(got, x[on], size[on], np.float32(s["scales"][n]))
        elif n == 0:
            assert near_bf16(got, x[on], size[on])
        else:
            assert np.array_equal(ref.f64(got), x[on])
        untouched = torch.ones(s[name].shape[0], bs, dtype=torch.bool)
        untouched[blk, off] = False
        view = lambda t: t.cpu().view(torch.uint8 if s["scales"] else torch.int16).transpose(1, 2)[untouched]
        assert torch.equal(view(s[name]), view(before[name]))


def copies(s):
    return {n: x.clone() if isinstance(x, torch.Tensor) else x for n, x in s.items()}


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,Hq,Hkv,d,rotary,interleaved,norm,packed,bs", [
    (1, 8, 2, 128, 128, False, True, True, 16),
    (1, 1, 1, 8, 0, False, True, False, 1),
    (37, 6, 2, 64, 64, True, True, True, 16),
    (130, 32, 4, 128, 64, False, True, True, 64),
    (65, 5, 5, 80, 32, False, False, False, 16),
    (19, 3, 1, 192, 192, True, True, True, 24),
    (23, 7, 7, 256, 256, False, True, True, 128),
    (40, 2, 1, 256, 16, True, True, False, 8),
    (300, 9, 3, 96, 96, False, True, True, 16),
    (33, 4, 2, 16, 16, False, True, True, 16),
    (50, 4, 4, 128, 0, False, False, True, 32),
])
def test_rope(T, Hq, Hkv, d, rotary, interleaved, norm, packed, bs, fp8):
    s = rope_case(T, Hq, Hkv, d, rotary, interleaved, norm, fp8, packed, bs=bs, seed=T + d, keep=T % 2 == 1)
    before = copies(s)
    rope_call(s)
    assert int(s["err"]) == 0
    rope_check(s, before)


@pytest.mark.parametrize("k_scale,v_scale", [(0.05, 0.03125), (0.75, 0.0371), (1.0, 3.3e4), (1e-3, 448.0),
                                             (1e-40, 3e38), (2.0 ** -120, 2.0 ** 90), (1.1754944e-38, 2e-30),
                                             (2.0 - 2.0 ** -23, 1.0 - 2.0 ** -24), (1.0 + 2.0 ** -23, 1.4e-45)])
def test_rope_codes_are_those_of_the_cache_write(k_scale, v_scale):
    # every bf16 pattern, NaN and infinities among them: without norms and rotation both calls store the same codes
    x = torch.arange(65536, dtype=I32, device="cuda").to(torch.int16).view(BF16).view(128, 4, 128)
    slots = dev(np.arange(128), I64)
    caches = [torch.zeros(8, 4, 16, 128, dtype=torch.uint8, device="cuda") for _ in range(4)]
    pka.pka_qk_rope_cache_write(x, x, x, None, None, 0.0, None, False, dev(np.zeros(128), I32), slots,
                                torch.empty_like(x), None, None, caches[0], caches[1], kv_scales=(k_scale, v_scale))
    pka.pka_cache_write_fp8(x, x, slots, caches[2], caches[3], k_scale, v_scale)
    assert torch.equal(caches[0], caches[2]) and torch.equal(caches[1], caches[3])


@pytest.mark.parametrize("scale", [0.05, 0.75, 2.0 ** -5])
def test_rope_codes_at_the_borders(scale):
    # rotated keys are float32: products of small integers put quotients on and next to every border of two codes
    n = 512
    k = torch.zeros(n, 1, 64, dtype=BF16, device="cuda")
    k[:, 0, 0::2] = (torch.arange(32, device="cuda") * 8 + 1).to(BF16)
    border = torch.arange(n, device="cuda", dtype=torch.float64) / 32
    border[0] = 2.0 ** -10  # half the least code
    table = torch.zeros(n, 64, dtype=torch.float64, device="cuda")
    u32 = np.float32(scale).astype(np.float64)
    table[:, :32] = border[:, None] * u32 / k[0, 0, 0::2].double()
    step = torch.arange(n, device="cuda") % 5 - 2  # the float32 numbers around them
    table = (table.float().view(I32) + torch.where(table != 0, step[:, None].int(), 0)).view(torch.float32)
    caches = [torch.zeros(n // 16, 1, 16, 64, dtype=torch.uint8, device="cuda") for _ in range(2)]
    pka.pka_qk_rope_cache_write(k, k, k, None, None, 0.0, table, True, dev(np.arange(n), I32), dev(np.arange(n), I64),
                                torch.empty_like(k), None, None, *caches, kv_scales=(scale, 1.0))
    # (a c - 0 s) and (0 c + a s) with s = 0: one rounding, of a c
    a = (k[:, 0].float()[:, 0::2] * table[:, :32]).cpu().numpy()
    got = caches[0].view(n, 64).cpu().numpy()
    assert np.array_equal(got[:, 0::2], fp8.quantize_f32(a, scale)) and not got[:, 1::2].any()


@pytest.mark.parametrize("fp8", [False, True])
def test_rope_skips_padding_and_bad_rows(fp8):
    s = rope_case(24, 4, 2, 128, 128, False, True, fp8, True, seed=3)
    s["pos"][[2, 20]] = -1     # rows behind the last sequence
    s["pos"][7] = 500          # past the rotation table
    s["slots"][[3, 20]] = -1   # no slot: rotated, not written to the cache
    s["slots"][9] = s["k_cache"].shape[0] * 16
    before = copies(s)
    rope_call(s)
    assert int(s["err"]) == E["INDEX"] | E["SLOT"]
    rope_check(s, before, [t for t in range(24) if t not in (2, 7, 20)])


def test_rope_in_place_is_the_same():
    s = rope_case(41, 8, 2, 128, 64, False, True, False, False, seed=4)
    other = copies(s)
    rope_call(s)
    other["q_out"], other["k_out"], other["v_out"] = other["q"], other["k"], other["v"]
    rope_call(other)
    for a, b in (("q_out", "q"), ("k_out", "k"), ("v_out", "v"), ("k_cache", "k_cache")):
        assert torch.equal(s[a], other[b])


def test_rope_extreme_values():
    """Zero heads, the largest and the smallest values, NaN and infinity stay in their own head."""
    s = rope_case(6, 4, 2, 128, 128, False, True, False, True, seed=5)
    s["q"][0, 0] = 0
    s["q"][1, 1] *= 2.0 ** 50     # the squares' sum stays finite
    s["q"][2, 2] *= 2.0 ** -50
    before = copies(s)
    s["q"][3, 3, 5] = float("nan")
    s["q"][4, 0, 5] = float("inf")
    rope_call(s)
    out = s["q_out"].float()
    assert (out[0, 0] == 0).all() and torch.isnan(out[3, 3]).all() and torch.isnan(out[4, 0]).any()
    good = torch.ones(6, 4, dtype=torch.bool, device="cuda")
    good[3, 3] = good[4, 0] = False
    assert torch.isfinite(out[good]).all()
    rope_check(dict(s, q_out=torch.where(good[..., None], s["q_out"], before["q_out"])[:3],
                    q=s["q"][:3], k=s["k"][:3], v=s["v"][:3], pos=s["pos"][:3], slots=s["slots"][:3], k_out=None),
               dict(before, q=before["q"][:3], k=before["k"][:3], v=before["v"][:3], q_out=before["q_out"][:3],
                    k_cache=s["k_cache"], v_cache=s["v_cache"]))


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_keeps_infinities_to_their_pair(interleaved):
    """An infinity spoils its own pair alone; behind the rotated part only its own element."""
    s = rope_case(3, 4, 2, 128, 64, interleaved, False, False, True, seed=7)
    s["q"][0, 0, 70], s["q"][1, 2, 5], s["k"][2, 1, 127] = float("inf"), float("-inf"), float("inf")
    rope_call(s)
    bad = {n: ~torch.isfinite(s[n].float()).cpu() for n in ("q_out", "k_out")}
    pair = [4, 5] if interleaved else [5, 37]
    assert bad["q_out"].nonzero().tolist() == [[0, 0, 70]] + [[1, 2, i] for i in pair]
    assert bad["k_out"].nonzero().tolist() == [[2, 1, 127]]
    assert s["q_out"][0, 0, 70] == float("inf") and s["k_out"][2, 1, 127] == float("inf")


def test_rope_then_cache_write_is_the_same_cache():
    """k_out and v_out through pka_cache_write give the bits that the one pass wrote."""
    s = rope_case(77, 4, 2, 128, 128, True, True, False, True, seed=6)
    k2, v2 = s["k_cache"].clone(), s["v_cache"].clone()
    rope_call(s)
    pka.pka_cache_write(s["k_out"], s["v_out"], s["slots"], k2, v2)
    assert torch.equal(k2, s["k_cache"]) and torch.equal(v2, s["v_cache"])


# ---------------------------------------------------------------- page bounds


def bounds_case(rng, nb, Hkv, bs, d, fp8):
    keys = rng.standard_normal((nb, Hkv, bs, d)) * rng.lognormal(0, 2, (nb, Hkv, 1, d))
    if fp8:
        keys = torch.from_numpy(np.clip(keys * 8, -448, 448)).float().to(torch.float8_e4m3fn).view(torch.uint8).cuda()
    else:
        keys = torch.from_numpy(keys).to(BF16).cuda()
    codes = torch.from_numpy(rng.integers(-127, 128, (nb, Hkv, 2, d))).to(torch.int8).cuda()
    return keys, codes, torch.from_numpy(rng.random((nb, Hkv))).float().cuda()


def bounds_check(keys, slots, codes0, scales0, codes, scales):
    nb, Hkv, bs, d = keys.shape
    values, want, unit = ref.f64(keys), ref.f64(codes0.float()), ref.f64(scales0)
    for s in slots:
        if 0 <= s < nb * bs and s % bs == bs - 1:
            for h in range(Hkv):
                want[s // bs, h, 0], want[s // bs, h, 1], unit[s // bs, h] = ref.page_bounds(values[s // bs, h])
    assert np.array_equal(ref.f64(codes.float()), want) and np.array_equal(ref.f64(scales), unit)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,nb,Hkv,bs,d", [(1, 3, 1, 1, 64), (1, 3, 2, 128, 128), (50, 9, 3, 16, 128), (9, 12, 2, 8, 64),
                                           (700, 16, 4, 64, 128), (333, 20, 2, 24, 64), (40, 5, 1, 200, 128)])
def test_page_bounds(T, nb, Hkv, bs, d, fp8):
    rng = np.random.default_rng(T + bs)
    keys, codes, scales = bounds_case(rng, nb, Hkv, bs, d, fp8)
    slots = rng.permutation(nb * bs)[:T]
    slots[::7] = slots[::7] // bs * bs + bs - 1  # pages that are filled, some of them twice
    slots[1::9] = -1
    c0, s0, err = codes.clone(), scales.clone(), word()
    pka.pka_page_bounds(keys, dev(slots, I64), codes, scales, error_word=err)
    assert int(err) == 0
    bounds_check(keys, slots, c0, s0, codes, scales)


@pytest.mark.parametrize("fp8", [False, True])
def test_page_bounds_special_pages(fp8):
    rng = np.random.default_rng(8)
    keys, codes, scales = bounds_case(rng, 12, 2, 16, 128, fp8)
    if fp8:
        keys[0] = 0
        keys[1, 0, 3, 7] = 0x7F        # a NaN code
        keys[2, 1] = 0x7E              # 448 everywhere
        keys[3, 1] = 0x81              # the least negative value
    else:
        keys[0] = 0
        keys[1, 0, 3, 7] = float("nan")
        keys[2, 1, 15, 127] = float("-inf")
        keys[3] = 2.0 ** -130          # subnormal
        keys[4] *= 2.0 ** -58
        keys[5, 0] = torch.finfo(BF16).max
        keys[6, 1] = 127.5             # just past 127 units of one
        keys[7, 1] = 127.0
        keys[8] = -2.0 ** -62
    slots = [b * 16 + 15 for b in range(12)] + [12 * 16 + 15]
    c0, s0, err = codes.clone(), scales.clone(), word()
    pka.pka_page_bounds(keys, dev(slots, I64), codes, scales, error_word=err)
    assert int(err) == E["SLOT"]
    bounds_check(keys, slots, c0, s0, codes, scales)


# ---------------------------------------------------------------- page selection


def batch(rng, ctx, new, bs, extra_rows=0, extra_pages=2):
    """Tables of a batch whose requests have ctx cached and new tokens each."""
    seq = [c + n for c, n in zip(ctx, new)]
    qsl = np.concatenate([[0], np.cumsum(new)]).tolist()
    pages = [-(-s // bs) for s in seq]
    nb = sum(pages) + 3
    width = max(max(pages), 1) + extra_pages
    table = np.full((len(ctx), width), 10 ** 8)  # entries behind a request's pages are never looked at
    perm, at = rng.permutation(nb), 0
    for r, n in enumerate(pages):
        table[r, :n] = perm[at:at + n]
        at += n
    return dict(table=table, qsl=qsl, seq=seq, bs=bs, nb=nb, T=qsl[-1] + extra_rows, longest=max(max(seq), 1))


def select_case(rng, b, Hq, Hkv, d, levels=None):
    lo = rng.integers(-127, 100, (b["nb"], Hkv, 1, d))
    hi = np.minimum(lo + rng.integers(0, 100, lo.shape), 127)
    bounds = np.concatenate([lo, hi], 2)
    scales = 2.0 ** rng.integers(-6, -3, (b["nb"], Hkv))
    if levels:  # few different pages: ties everywhere
        pick = rng.integers(0, levels, b["nb"])
        bounds, scales = bounds[pick], scales[pick]
    q = randn(rng, b["T"], Hq, d) * torch.exp(randn(rng, b["T"], Hq, 1))
    return q, bounds, scales


def select_run(b, q, bounds, scales, first, last, K, **kw):
    sel = torch.full((b["T"], bounds.shape[1], K), -9, dtype=I32, device="cuda")
    err = word()
    pka.pka_select_pages(q, dev(bounds, torch.int8), dev(scales, torch.float32), dev(b["table"], I32),
                         dev(b["qsl"], I32), dev(b["seq"], I32), b["bs"], first, last, b["longest"], sel,
                         error_word=err, **kw)
    return sel.cpu().numpy(), int(err)


def select_check(b, q, bounds, scales, first, last, K):
    sel, err = select_run(b, q, bounds, scales, first, last, K)
    assert err == 0
    want = ref.select_pages(ref.f64(q), bounds.astype(np.float64), scales, b["table"], b["qsl"], b["seq"], b["bs"],
                            first, last, K, np.full(sel.shape, -9))
    assert np.array_equal(sel, want)


@pytest.mark.parametrize("Hq,Hkv,d", [(8, 8, 128), (6, 2, 64), (32, 4, 128), (16, 1, 128), (13, 1, 64), (9, 1, 128)])
@pytest.mark.parametrize("first,last,K", [(1, 2, 8), (0, 1, 1), (0, 1, 5), (4, 4, 8), (2, 1, 33)])
def test_select_pages(Hq, Hkv, d, first, last, K):
    rng = np.random.default_rng(Hq + K)
    # no context, one page, exactly K pages, a page boundary, many; several new tokens; none
    b = batch(rng, [0, 15, 16 * K - 1, 16 * K, 700, 300, 1000], [1, 1, 1, 3, 1, 0, 5], 16, extra_rows=2)
    select_check(b, *select_case(rng, b, Hq, Hkv, d), first, last, K)


@pytest.mark.parametrize("levels", [1, 2, 5])
def test_select_pages_ties_go_to_the_lowest_page(levels):
    rng = np.random.default_rng(levels)
    b = batch(rng, [900, 3000, 50], [1, 1, 1], 8)
    select_check(b, *select_case(rng, b, 8, 2, 64, levels=levels), 1, 2, 20)


@pytest.mark.parametrize("ctx,bs,Hkv", [(20000, 8, 1), (32767 * 2, 2, 2), (9000, 1, 1)])
def test_select_pages_long_context_over_a_cluster(ctx, bs, Hkv):
    rng = np.random.default_rng(bs)
    b = batch(rng, [ctx], [1], bs)
    q, bounds, scales = select_case(rng, b, 4 * Hkv, Hkv, 128)
    sel, err = select_run(b, q, bounds, scales, 1, 2, 64)
    table = b["table"][0]
    n = ctx // bs + 1
    for g in range(Hkv):  # the definition, a page at a time no more
        score = np.full(n, -np.inf)
        for h in range(4 * g, 4 * g + 4):
            c, unit = ref.query_codes(ref.f64(q)[0, h])
            x = bounds[table[:n], g].astype(np.float64)
            score = np.maximum(score, np.maximum(c * x[:, 0], c * x[:, 1]).sum(-1) * scales[table[:n], g] * unit)
        rest = sorted(range(1, n - 2), key=lambda i: (-score[i], i))[:61]
        assert sel[0, g].tolist() == sorted([0] + rest + [n - 2, n - 1])
    assert err == 0


@pytest.mark.parametrize("B,Hkv,group", [(3, 2, 3), (20, 8, 1), (20, 8, 9), (45, 8, 1), (45, 8, 9), (60, 8, 2)])
def test_select_pages_shares_of_a_cluster(B, Hkv, group):
    # few units in clusters of wide CTAs, more in pairs, many alone; contexts from one page to all CTAs' worth
    rng = np.random.default_rng(B + group)
    ctx = np.exp(rng.uniform(0, np.log(5000), B)).astype(int)
    ctx[:3] = 8 * 590, 8 * (64 + 3) - 1, 8 * (128 + 3)  # all CTAs; a page less than one CTA's share, two CTAs' share
    b = batch(rng, ctx.tolist(), [1] * B, 8)
    select_check(b, *select_case(rng, b, group * Hkv, Hkv, 64), 1, 2, 12)


@pytest.mark.parametrize("d,Hq", [(64, 4), (128, 8), (128, 16)])
def test_select_pages_sums_at_the_end_of_their_range(d, Hq):
    """Codes of 127 throughout but for single units: scores of 127 * 127 * d that differ by one are told apart."""
    rng = np.random.default_rng(d)
    b = batch(rng, [4000], [1], 16)
    for sign in (1, -1):
        bounds = np.full((b["nb"], 1, 2, d), 127.0) - (rng.random((b["nb"], 1, 2, d)) < 0.01)
        bounds = np.sort(sign * bounds, axis=2)  # low before high
        q = sign * torch.full((1, Hq, d), 127.0)
        q[..., rng.permutation(d)[:d // 4]] = sign  # the codes are the values: units of these elements count one
        select_check(b, q.to(BF16).cuda(), bounds, np.ones((b["nb"], 1)), 1, 2, 50)


def test_select_pages_values_without_an_order():
    """Pages that bound nothing come first; query heads with NaN or infinity count as zero scores."""
    rng = np.random.default_rng(9)
    b = batch(rng, [800, 640], [1, 2], 16)
    q, bounds, scales = select_case(rng, b, 8, 2, 128)
    blk = b["table"][0, [7, 20]]
    scales[blk, 0] = np.inf
    bounds[blk, 0] = 0
    q[0, 1, 3], q[1, 5, 0] = float("nan"), float("inf")
    q[2, :4] = 0
    q[2, 5] *= 2.0 ** -70
    select_check(b, q, bounds, scales, 1, 1, 9)


def test_select_pages_reports_bad_tables():
    rng = np.random.default_rng(10)
    b = batch(rng, [400], [1], 16)
    args = select_case(rng, b, 4, 1, 64)
    for change, bit in ((dict(seq=[0]), "SEQ_LEN"), (dict(longest=399), "SEQ_LEN"),
                        (dict(table=np.where(np.arange(b["table"].shape[1]) == 5, -1, b["table"])), "BLOCK_ID"),
                        (dict(table=np.where(np.arange(b["table"].shape[1]) == 5, b["nb"], b["table"])), "BLOCK_ID")):
        sel, err = select_run(dict(b, **change), *args, 1, 1, 4)
        assert err == E[bit], change
        if bit == "SEQ_LEN":
            assert (sel == -9).all()


# ---------------------------------------------------------------- attention over selected pages


def attn_case(rng, b, Hq, Hkv, d, K, fp8=False, own=True):
    """Caches whose unused pages and unwritten places hold NaN, and random ascending lists."""
    nb, bs = b["nb"], b["bs"]
    values = [rng.standard_normal((nb, Hkv, bs, d)) for _ in range(2)]
    used = np.zeros((nb, bs), bool)
    for r, s in enumerate(b["seq"]):
        for p in range(s):
            used[b["table"][r, p // bs], p % bs] = True
    caches = []
    for x in values:
        t = torch.from_numpy(x * (8 if fp8 else 1)).float().to(torch.float8_e4m3fn if fp8 else BF16)
        t = t.view(torch.uint8) if fp8 else t
        t = t.permute(0, 2, 1, 3).contiguous()
        t[torch.from_numpy(~used)] = 0x7F if fp8 else float("nan")
        caches.append(t.permute(0, 2, 1, 3).contiguous().cuda())
    sel = np.full((b["T"], Hkv, K), -1)
    for t, r, p in ref.positions(b["qsl"], b["seq"]):
        for g in range(Hkv):
            n = p // bs + 1
            k = min(K, int(rng.integers(1, n + 1)))
            pages = sorted(rng.permutation(n)[:k].tolist())
            if own and n - 1 not in pages:
                pages[-1] = n - 1
            sel[t, g, :k] = pages
    q = randn(rng, b["T"], Hq, d)
    return q, caches, sel


def attn_run(b, q, caches, sel, scale, units=None, lse=True, **kw):
    out = torch.full(q.shape, 5.0, dtype=BF16, device="cuda")
    l = torch.full(q.shape[:2], 5.0, device="cuda") if lse else None
    err = word()
    pka.pka_sparse_attn_forward(q, *caches, dev(b["table"], I32), dev(b["qsl"], I32), dev(b["seq"], I32),
                                dev(sel, I32), scale, b["longest"], out, l, kv_scales=units, error_word=err, **kw)
    return out, l, int(err)


def attn_near(out, lse, want):
    """P is rounded to bf16 (or f16) before the product and the result to bf16, 2^-8 each: of the sum of
    the weighted magnitudes, and of the value. Scores of up to 2^5 with a relative error of a few 2^-23
    (products of at most 128 terms, the scale, the exponential): 2^-14 more of that sum."""
    o, l, size = want
    real = ~np.isnan(size)
    assert (np.abs(ref.f64(out) - o) <= 2.0 ** -8 * np.abs(o) + (2.0 ** -8 + 2.0 ** -14) * size)[real].all()
    assert (ref.f64(out)[~real] == 5.0).all()  # rows of no request
    if lse is not None:
        got, none = ref.f64(lse), np.isneginf(l)
        ok = ~np.isnan(l) & ~none
        assert (np.abs(got - l)[ok] <= 2.0 ** -14 * (1 + np.abs(l[ok]))).all()
        assert np.isneginf(got[none]).all() and (got[np.isnan(l)] == 5.0).all()


@pytest.mark.parametrize("Hq,Hkv,d,bs", [(8, 8, 128, 16), (6, 2, 64, 8), (32, 4, 128, 64), (16, 1, 128, 8),
                                         (13, 1, 64, 128), (9, 1, 128, 32), (2, 1, 64, 16), (8, 1, 128, 128)])
@pytest.mark.parametrize("K", [1, 5, 40])
@pytest.mark.parametrize("own", [True, False])
def test_sparse_attn(Hq, Hkv, d, bs, K, own):
    rng = np.random.default_rng(Hq + K + bs)
    b = batch(rng, [0, 1, bs - 1, bs, 15 * bs + 3, 700, 20], [1, 1, 1, 3, 1, 1, 0], bs, extra_rows=2)
    q, caches, sel = attn_case(rng, b, Hq, Hkv, d, K, own=own)
    sel[2] = -1  # a token that reads nothing
    out, lse, err = attn_run(b, q, caches, sel, d ** -0.5)
    assert err == 0
    attn_near(out, lse, ref.sparse_attn(ref.f64(q), *map(ref.f64, caches), b["table"], b["qsl"], b["seq"], sel, d ** -0.5))


@pytest.mark.parametrize("Hq,Hkv,bs", [(8, 2, 16), (16, 1, 64), (3, 3, 8), (12, 1, 32)])
@pytest.mark.parametrize("K", [1, 7, 50])
def test_sparse_attn_8_bit(Hq, Hkv, bs, K):
    rng = np.random.default_rng(Hq + K + bs)
    b = batch(rng, [0, bs - 1, 10 * bs + 3, 900], [1, 1, 4, 1], bs, extra_rows=1)
    q, caches, sel = attn_case(rng, b, Hq, Hkv, 128, K, fp8=True)
    units = (0.125, 0.11)
    out, lse, err = attn_run(b, q, caches, sel, 128 ** -0.5, units)
    assert err == 0
    want = ref.sparse_attn(ref.f64(q), *map(ref.f64, caches), b["table"], b["qsl"], b["seq"], sel, 128 ** -0.5,
                           [float(np.float32(u)) for u in units])
    attn_near(out, lse, want)


@pytest.mark.parametrize("fp8,d,group,bs,K", [
    (False, 128, 4, 16, 20), (False, 128, 12, 64, 40), (False, 64, 2, 64, 40), (False, 64, 16, 16, 20),
    (True, 128, 4, 16, 40), (True, 128, 11, 64, 30)])
def test_sparse_attn_of_more_tokens_than_sms(fp8, d, group, bs, K):
    rng = np.random.default_rng(K + group)
    ctx = np.exp(rng.uniform(0, np.log(4000), 90)).astype(int).tolist()
    b = batch(rng, ctx, [1] * 90, bs)
    q, caches, sel = attn_case(rng, b, 2 * group, 2, d, K, fp8=fp8)
    units = (0.125, 0.11) if fp8 else None
    out, lse, err = attn_run(b, q, caches, sel, d ** -0.5, units)
    assert err == 0
    attn_near(out, lse, ref.sparse_attn(ref.f64(q), *map(ref.f64, caches), b["table"], b["qsl"], b["seq"], sel, d ** -0.5,
                                        [float(np.float32(u)) for u in units] if fp8 else (1.0, 1.0)))


@pytest.mark.parametrize("power", [-60, -12, 0, 17, 90])
def test_sparse_attn_8_bit_takes_queries_of_any_magnitude(power):
    """Queries of a head far from one, elements of a head far apart: q is held in units of a power of two of
    its own head, off by at most 2^-22 of the head's largest element."""
    rng = np.random.default_rng(power + 100)
    b = batch(rng, [300, 77], [1, 2], 16)
    q, caches, sel = attn_case(rng, b, 4, 2, 128, 9, fp8=True)
    q = q * torch.exp2(torch.from_numpy(rng.integers(-9, 1, (b["T"], 4, 128))).float().cuda()).to(BF16)
    scale = 128 ** -0.5 * 2.0 ** -power
    q = (q.double() * 2.0 ** power).to(BF16)
    out, lse, err = attn_run(b, q, caches, sel, scale, (0.125, 0.11))
    assert err == 0
    attn_near(out, lse, ref.sparse_attn(ref.f64(q), *map(ref.f64, caches), b["table"], b["qsl"], b["seq"], sel, scale,
                                        [float(np.float32(u)) for u in (0.125, 0.11)]))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("bs", [8, 64])
def test_sparse_attn_long_lists_over_clusters(bs, fp8):
    """Enough tiles that every warp of a cluster looks its pages up several times."""
    rng = np.random.default_rng(bs)
    b = batch(rng, [40000, 12345], [1, 1], bs)
    n = -(-40001 // bs)
    q, caches, sel = attn_case(rng, b, 2, 1, 128, n, fp8=fp8)
    for t, r, p in ref.positions(b["qsl"], b["seq"]):
        sel[t] = -1
        sel[t, 0, :p // bs + 1] = np.arange(p // bs + 1)
    sel[1, 0, 1:] = np.append(sel[1, 0, 2:], -1)  # one page left out
    out, lse, err = attn_run(b, q, caches, sel, 0.05, (1.0, 1.0) if fp8 else None)
    assert err == 0
    attn_near(out, lse, ref.sparse_attn(ref.f64(q), *map(ref.f64, caches), b["table"], b["qsl"], b["seq"], sel, 0.05))


def grouped_case(Hq, Hkv, d, bs, K, new, fp8, alike, seed=0):
    """Requests with several new tokens, whose lists share most pages (alike) or are drawn apart."""
    rng = np.random.default_rng(seed + Hq + K + bs)
    b = batch(rng, [0, 2 * bs - 3, 500, 40, 7, 333], new, bs, extra_rows=2)
    q, caches, sel = attn_case(rng, b, Hq, Hkv, d, K, fp8=fp8)
    if alike:
        for t, r, p in ref.positions(b["qsl"], b["seq"]):
            first = b["qsl"][r]
            if t > first:
                for g in range(Hkv):
                    own = p // bs
                    pages = sorted({e for e in sel[first, g] if e >= 0} | {own})[-K:]
                    sel[t, g] = pages + [-1] * (K - len(pages))
    return b, q, caches, sel


GROUPS = [(8, 2, 128, 16, 6, [4, 4, 4, 4, 4, 4]), (6, 2, 64, 8, 9, [9, 1, 17, 3, 8, 2]), (16, 1, 128, 64, 3, [2, 3, 5, 1, 4, 2]),
          (4, 4, 64, 16, 12, [33, 1, 0, 20, 7, 50]), (24, 2, 128, 32, 5, [3, 3, 3, 3, 3, 3]), (32, 4, 128, 8, 20, [4, 1, 6, 2, 5, 3]),
          (8, 1, 128, 128, 2, [5, 5, 5, 5, 5, 5]), (2, 1, 64, 64, 4, [16, 16, 16, 0, 0, 16])]


@pytest.mark.parametrize("Hq,Hkv,d,bs,K,new", GROUPS)
@pytest.mark.parametrize("alike", [False, True])
@pytest.mark.parametrize("fp8", [False, True])
def test_sparse_attn_of_several_tokens(Hq, Hkv, d, bs, K, new, alike, fp8):
    if fp8 and d == 64:
        pytest.skip("the 8-bit cache's attention has head dim 128")
    b, q, caches, sel = grouped_case(Hq, Hkv, d, bs, K, new, fp8, alike)
    sel[b["qsl"][1] - 1] = -1                    # the last token of a request reads nothing
    sel[b["qsl"][3] - 2, :, 1:] = -1             # another one page only
    units = (0.125, 0.11) if fp8 else None
    out, lse, err = attn_run(b, q, caches, sel, d ** -0.5, units)
    assert err == 0
    attn_near(out, lse, ref.sparse_attn(ref.f64(q), *map(ref.f64, caches), b["table"], b["qsl"], b["seq"], sel, d ** -0.5,
                                        [float(np.float32(u)) for u in units] if fp8 else (1.0, 1.0)))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("bs", [8, 16, 64])
def test_sparse_attn_values_of_other_tokens_stay_hidden(bs, fp8):
    """NaN and infinities in the values and keys of pages that a token does not list, and of the tokens after
    it, do not reach it, whoever else in its request reads them; who lists them gets them."""
    b, q, caches, sel = grouped_case(8, 2, 128, bs, 6, [4, 4, 4, 4, 4, 4], fp8, False, seed=1)
    spoil = 0x7F if fp8 else float("nan")
    reads = {}
    for r in (2, 5):  # one page of the request, listed by its second token only
        t0 = b["qsl"][r]
        page = 1
        pages = sorted([page] + [e for e in sel[t0 + 1, 0] if e >= 0 and e != page][-5:])
        sel[t0 + 1, 0] = pages + [-1] * (6 - len(pages))
        for t in range(t0, t0 + 4):
            for g in range(2):
                if t != t0 + 1 or g:
                    kept = [e for e in sel[t, g] if e >= 0 and e != page]
                    sel[t, g] = kept + [-1] * (6 - len(kept))
        caches[1][b["table"][r, page], 0, 3] = spoil
        reads[t0 + 1] = True
        if r == 5:
            caches[0][b["table"][r, page], 0, 2] = spoil
    # the newest token of request 3: infinite values that its earlier ones stand before
    p = b["seq"][3] - 1
    caches[1][b["table"][3, p // bs], :, p % bs] = spoil if fp8 else float("inf")
    for t in range(b["qsl"][3], b["qsl"][4]):
        own = (p - (b["qsl"][4] - 1 - t)) // bs
        for g in range(2):
            pages = sorted({e for e in sel[t, g] if 0 <= e < own} | {own})[-6:]
            sel[t, g] = pages + [-1] * (6 - len(pages))
    reads[b["qsl"][4] - 1] = True
    units = (0.125, 0.11) if fp8 else None
    out, lse, err = attn_run(b, q, caches, sel, 0.1, units)
    assert err == 0
    hit = ~torch.isfinite(out.float()).all(-1)
    for t in range(b["qsl"][-1]):
        heads = hit[t].cpu().numpy()
        if t in reads and t == b["qsl"][4] - 1:
            assert heads.all()
        elif t in reads:
            assert heads[:4].all() and not heads[4:].any()
        else:
            assert not heads.any(), t
    want = ref.sparse_attn(ref.f64(q), *map(ref.f64, caches), b["table"], b["qsl"], b["seq"], sel, 0.1,
                           [float(np.float32(u)) for u in units] if fp8 else (1.0, 1.0))
    for t in reads:  # (compared above)
        want[2][t] = 1e9
        want[0][t] = 0
        want[1][t] = lse[t].cpu().numpy()
        out[t] = 0
    out, lse = out.nan_to_num(0, 0, 0), lse.nan_to_num(0, 0, 0)
    want = (want[0], np.nan_to_num(want[1], nan=np.nan), want[2])
    ok = ~np.isnan(want[1])
    assert (np.abs(ref.f64(lse) - want[1])[ok] <= 2.0 ** -14 * (1 + np.abs(want[1][ok]))).all()
    attn_near(out, None, want)


def test_sparse_attn_of_several_tokens_reports_bad_lists():
    b, q, caches, sel = grouped_case(8, 2, 128, 16, 6, [4, 4, 4, 4, 4, 4], False, False, seed=2)
    t = b["qsl"][2] + 1
    sel[t, 1] = [3, 9, 9, 12, -1, -1]            # twice the same page: the list ends there
    sel[t + 1, 0] = [1, 4, 5, 600, -1, -1]       # past the token's page
    out, lse, err = attn_run(b, q, caches, sel, 0.1)
    assert err == E["INDEX"]
    sel[t, 1], sel[t + 1, 0] = [3, 9, -1, -1, -1, -1], [1, 4, 5, -1, -1, -1]
    attn_near(out, lse, ref.sparse_attn(ref.f64(q), *map(ref.f64, caches), b["table"], b["qsl"], b["seq"], sel, 0.1))


def test_sparse_attn_with_every_page_is_the_dense_decode():
    rng = np.random.default_rng(11)
    b = batch(rng, [5, 100, 1000, 333], [1, 1, 1, 1], 16)
    q, caches, sel = attn_case(rng, b, 8, 2, 128, 64)
    for t, r, p in ref.positions(b["qsl"], b["seq"]):
        sel[t] = -1
        sel[t, :, :p // 16 + 1] = np.arange(p // 16 + 1)
    out, lse, _ = attn_run(b, q, caches, sel, 0.1)
    ws = torch.empty(pka.pka_workspace_size(4, 0, 0, 4, 8, 2, 128, 128, 1, 1001, 1024), dtype=torch.uint8, device="cuda")
    dense, dl = torch.empty_like(out), torch.empty_like(lse)
    pka.pka_paged_attn_forward(q, None, None, *caches, dev(b["table"], I32), dev(b["qsl"], I32), dev(b["seq"], I32),
                               4, 0, 0, 0.1, 1024, 1, 1001, dense, dl, ws)
    assert pka.pka_get_error(ws) == 0
    want = ref.sparse_attn(ref.f64(q), *map(ref.f64, caches), b["table"], b["qsl"], b["seq"], sel, 0.1)
    attn_near(out, lse, want)
    attn_near(dense, dl, want)


def test_sparse_attn_reports_bad_lists():
    rng = np.random.default_rng(12)
    b = batch(rng, [200], [1], 16)
    q, caches, _ = attn_case(rng, b, 4, 1, 64, 4)
    good = dict(b, T=1)
    for entries, kept, bit in (([3, 3, 5, -1], [3], "INDEX"), ([3, 2, 5, 7], [3], "INDEX"), ([2, 13, -1, -1], [2], "INDEX"),
                               ([13, 1, 2, 3], [], "INDEX"), ([2, -1, 5, 6], [2], None), ([-5, 1, 2, 3], [], None)):
        out, lse, err = attn_run(good, q, caches, np.array([[entries]]), 0.1)
        assert err == (E[bit] if bit else 0), entries
        sel = np.array([[kept + [-1] * (4 - len(kept))]])
        attn_near(out, lse, ref.sparse_attn(ref.f64(q), *map(ref.f64, caches), b["table"], b["qsl"], b["seq"], sel, 0.1))
    for change, bit in ((dict(seq=[0]), "SEQ_LEN"), (dict(longest=200), "SEQ_LEN"),
                        (dict(table=np.where(b["table"] == b["table"][0, 2], -4, b["table"])), "BLOCK_ID")):
        out, _, err = attn_run(dict(b, **change), q, caches, np.array([[[1, 2, 4, -1]]]), 0.1, lse=False)
        assert err == E[bit]


@pytest.mark.parametrize("fp8", [False, True])
def test_caches_past_32_bits(fp8):
    """The last pages of caches of more than 2^32 bytes: written, bounded and read where they lie."""
    d, bs, Hkv = 128, 128, 2
    nb = (1 << 32) // (bs * Hkv * d * (1 if fp8 else 2)) + 40
    rng = np.random.default_rng(13)
    T = 300
    s = rope_case(T, 4, Hkv, d, d, False, True, fp8, True, bs=bs, nb=8, seed=13)
    kind = torch.uint8 if fp8 else BF16
    for name in ("k_cache", "v_cache"):
        s[name] = torch.zeros((nb, Hkv, bs, d), dtype=kind, device="cuda")
    table = np.array([[nb - 1, nb - 7, nb - 2]])
    p = np.arange(T)
    s["slots"] = dev(table[0, p // bs] * bs + p % bs, I64)
    tail = slice(nb - 8, nb)
    before = copies({n: x for n, x in s.items() if n not in ("k_cache", "v_cache")})
    rope_call(s)
    assert int(s["err"]) == 0
    small = dict(s, slots=s["slots"] - (nb - 8) * bs, k_cache=s["k_cache"][tail], v_cache=s["v_cache"][tail])
    rope_check(small, dict(before, k_cache=torch.zeros_like(small["k_cache"]), v_cache=torch.zeros_like(small["v_cache"])))
    assert not any(s[n][:8].any() for n in ("k_cache", "v_cache"))
    codes, scales = torch.zeros(nb, Hkv, 2, d, dtype=torch.int8, device="cuda"), torch.zeros(nb, Hkv, device="cuda")
    pka.pka_page_bounds(s["k_cache"], s["slots"], codes, scales, error_word=s["err"])
    bounds_check(small["k_cache"], small["slots"].tolist(), codes[tail] * 0, scales[tail] * 0, codes[tail], scales[tail])
    out, lse = torch.empty(1, 4, d, dtype=BF16, device="cuda"), torch.empty(1, 4, device="cuda")
    q, sel = s["q_out"][-1:].contiguous(), np.array([[[0, 1, 2], [0, 2, -1]]])
    pka.pka_sparse_attn_forward(q, s["k_cache"], s["v_cache"], dev(table, I32), dev([0, 1], I32), dev([T], I32),
                                dev(sel, I32), 0.1, T, out, lse, kv_scales=s["scales"], error_word=s["err"])
    assert int(s["err"]) == 0
    attn_near(out, lse, ref.sparse_attn(ref.f64(q), ref.f64(small["k_cache"]), ref.f64(small["v_cache"]),
                                        table - (nb - 8), [0, 1], [T], sel, 0.1,
                                        [float(np.float32(u)) for u in s["scales"]] if fp8 else (1.0, 1.0)))


# ---------------------------------------------------------------- the step as a whole


class Server:
    """A small server's state: caches, bounds, tables of B requests, and one step over them."""

    def __init__(self, rng, B, Hq, Hkv, d, bs, width, K, fp8, rows):
        self.nb, self.bs, self.K, self.Hq, self.Hkv, self.d = B * width + 4, bs, K, Hq, Hkv, d
        self.rng, self.fp8, self.longest = rng, fp8, width * bs
        self.units = (0.02, 0.02) if fp8 else None
        z = lambda *s, dtype=I32: torch.zeros(s, dtype=dtype, device="cuda")
        cache = lambda: torch.full((self.nb, Hkv, bs, d), 0x7F if fp8 else float("nan"),
                                   dtype=torch.uint8 if fp8 else BF16, device="cuda")
        self.k_cache, self.v_cache = cache(), cache()
        self.bounds, self.scales = z(self.nb, Hkv, 2, d, dtype=torch.int8), z(self.nb, Hkv, dtype=torch.float32)
        self.free, self.head = dev(rng.permutation(self.nb), I32), z(1)
        self.table, self.ctx, self.new, self.seq, self.qsl = z(B, width) - 1, z(B), z(B), z(B), z(B + 1)
        self.err = z(1)
        angle = rng.uniform(0, 6.28, (self.longest, d // 2))
        self.cos_sin = torch.from_numpy(np.concatenate([np.cos(angle), np.sin(angle)], 1)).float().cuda()
        self.qw, self.kw = 1 + 0.1 * randn(rng, d), 1 + 0.1 * randn(rng, d)
        self.rows(rows)

    def rows(self, T):
        self.T = T
        e = lambda *s, dtype=BF16: torch.full(s, 3, dtype=dtype, device="cuda")
        self.qkv = e(T, self.Hq + 2 * self.Hkv, self.d)
        self.q, self.pos, self.slots = e(T, self.Hq, self.d), e(T, dtype=I32), e(T, dtype=I64)
        self.sel, self.out = e(T, self.Hkv, self.K, dtype=I32), e(T, self.Hq, self.d)
        self.lse = e(T, self.Hq, dtype=torch.float32)

    def step(self, stream=None):
        Hq, Hkv, w = self.Hq, self.Hkv, dict(error_word=self.err, stream=stream)
        pka.pka_step_tables(self.ctx, self.new, self.table, self.bs, self.free, self.head, self.head, self.qsl,
                            self.seq, self.pos, self.slots, **w)
        pka.pka_qk_rope_cache_write(self.qkv[:, :Hq], self.qkv[:, Hq:Hq + Hkv], self.qkv[:, Hq + Hkv:], self.qw,
                                    self.kw, 1e-6, self.cos_sin, False, self.pos, self.slots, self.q, None, None,
                                    self.k_cache, self.v_cache, kv_scales=self.units, **w)
        pka.pka_page_bounds(self.k_cache, self.slots, self.bounds, self.scales, **w)
        pka.pka_select_pages(self.q, self.bounds, self.scales, self.table, self.qsl, self.seq, self.bs, 1, 2,
                             self.longest, self.sel, **w)
        pka.pka_sparse_attn_forward(self.q, self.k_cache, self.v_cache, self.table, self.qsl, self.seq, self.sel,
                                    self.d ** -0.5, self.longest, self.out, self.lse, kv_scales=self.units, **w)

    def feed(self, ctx, new, history):
        """The next step's inputs; every request's rotated keys and values so far go to `history`."""
        self.ctx.copy_(dev(ctx, I32))
        self.new.copy_(dev(new, I32))
        self.qkv.copy_(randn(self.rng, *self.qkv.shape))
        x, table, at = ref.f64(self.qkv), ref.f64(self.cos_sin), 0
        for r, (c, n) in enumerate(zip(ctx, new)):
            pos = np.arange(c, c + n)
            k, _ = ref.rope(x[at:at + n, self.Hq:self.Hq + self.Hkv], ref.f64(self.kw), 1e-6, table, pos, False)
            history[r] = (np.concatenate([history[r][0], k]),
                          np.concatenate([history[r][1], x[at:at + n, self.Hq + self.Hkv:]]))
            at += n

    def check(self, ctx, new, history):
        assert int(self.err) == 0
        qsl = np.concatenate([[0], np.cumsum(new)]).tolist()
        seq = [c + n for c, n in zip(ctx, new)]
        table = self.table.cpu().numpy()
        total = qsl[-1]
        # the cache holds every token of every request
        kc, vc = ref.f64(self.k_cache), ref.f64(self.v_cache)
        for r, s in enumerate(seq):
            p = np.arange(s)
            for got, want, i in ((kc, history[r][0], 0), (vc, history[r][1], 1)):
                got = got[table[r, p // self.bs], :, p % self.bs] * (np.float32(self.units[i]) if self.fp8 else 1)
                assert (np.abs(got - want) <= (2.0 ** -4 if self.fp8 else 2.0 ** -7) * (np.abs(want) + 0.05)).all()
        # the pages and the attention, from the queries, caches and bounds the step left
        q = ref.f64(self.q)
        bounds, scales = ref.f64(self.bounds.float()), ref.f64(self.scales)
        for r, s in enumerate(seq):
            for blk in table[r, :s // self.bs]:
                for h in range(self.Hkv):
                    lo, hi, unit = ref.page_bounds(kc[blk, h])
                    assert (bounds[blk, h] == [lo, hi]).all() and scales[blk, h] == unit
        sel = self.sel.cpu().numpy()
        want = ref.select_pages(q, bounds, scales, table, qsl, seq, self.bs, 1, 2, self.K, np.full(sel.shape, 3))
        assert np.array_equal(sel, want)
        unit = [float(np.float32(u)) for u in self.units] if self.fp8 else (1.0, 1.0)
        o, l, size = ref.sparse_attn(q, kc, vc, table, qsl, seq, sel, self.d ** -0.5, unit)
        out = self.out.clone()
        assert (out[total:] == 3).all() and (self.lse[total:] == 3).all() and (self.q[total:] == 3).all()
        out[total:] = 5.0
        lse = self.lse.clone()
        lse[total:] = 5.0
        attn_near(out, lse, (o, l, size))


def plan(rng, B, steps, rows):
    """(ctx, new) of each step: prompts first, then mostly single tokens, some requests idle."""
    ctx, out = [0] * B, []
    for i in range(steps):
        new = rng.integers(20, 90, B).tolist() if i == 0 else [int(rng.choice([0, 1, 1, 1, 3])) for _ in range(B)]
        new[0] = max(new[0], 1)
        assert sum(new) <= rows
        out.append((list(ctx), new))
        ctx = [c + n for c, n in zip(ctx, new)]
    return out


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("bs,d", [(8, 128), (16, 128), (16, 64)])
def test_steps_of_a_server(bs, d, fp8):
    if fp8 and d == 64:
        pytest.skip("the 8-bit cache's attention has head dim 128")
    rng = np.random.default_rng(bs + d)
    B, rows = 4, 400
    server = Server(rng, B, 8, 2, d, bs, -(-120 // bs), 5, fp8, rows)
    history = [(np.zeros((0, 2, d)), np.zeros((0, 2, d))) for _ in range(B)]
    for ctx, new in plan(rng, B, 6, rows):
        server.rows(sum(new) + 3)
        server.feed(ctx, new, history)
        server.step()
        server.check(ctx, new, history)


def test_step_captured_once_and_replayed():
    """One graph of a padded step, replayed for steps of other lengths, with an eager step between."""
    rng = np.random.default_rng(21)
    B, rows = 5, 24
    server = Server(rng, B, 8, 2, 128, 16, 8, 4, False, 500)
    history = [(np.zeros((0, 2, 128)), np.zeros((0, 2, 128))) for _ in range(B)]
    steps = plan(rng, B, 8, 500)
    server.feed(*steps[0], history)
    server.step()
    server.check(*steps[0], history)
    server.rows(rows)
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    server.new.zero_()  # the capture's warm-up step has no tokens
    server.ctx.copy_(server.seq)
    with torch.cuda.stream(stream):
        server.step()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        server.step()
    for i, (ctx, new) in enumerate(steps[1:]):
        for t in (server.out, server.lse, server.q, server.sel):
            t.fill_(3)
        server.feed(ctx, new, history)
        if i == 3:
            server.step()
        else:
            graph.replay()
        torch.cuda.synchronize()
        server.check(ctx, new, history)


def test_two_servers_on_two_streams():
    """Steps of two servers that overlap give what each gives alone, bit for bit."""
    results = []
    for together in (False, True):
        servers = [Server(np.random.default_rng(30 + i), 3, 8, 2, 128, 16, 30, 6, False, 1300) for i in range(2)]
        streams = [torch.cuda.Stream() for _ in servers]
        for s in servers:
            s.feed([0, 0, 0], [400, 300, 470], [(np.zeros((0, 2, 128)),) * 2] * 3)
        torch.cuda.synchronize()
        for _ in range(6):  # the same step again and again
            for s, stream in zip(servers, streams):
                with torch.cuda.stream(stream if together else torch.cuda.current_stream()):
                    s.head.zero_()
                    s.step()
        torch.cuda.synchronize()
        assert all(int(s.err) == 0 for s in servers)
        results.append([[t.clone() for t in (s.out, s.lse, s.sel, s.table, s.bounds, s.k_cache.view(torch.int16))]
                        for s in servers])
    for alone, both in zip(*results):
        assert all(torch.equal(x, y) for x, y in zip(alone, both))


def test_repeats_are_bit_for_bit():
    rng = np.random.default_rng(31)
    b = batch(rng, [3000, 5000, 77], [1, 2, 1], 16)
    q, caches, _ = attn_case(rng, b, 16, 2, 128, 32)
    q2, bounds, scales = select_case(rng, b, 16, 2, 128)
    first, _ = select_run(b, q2, bounds, scales, 1, 2, 32)
    out, lse, _ = attn_run(b, q, caches, first, 0.1)
    for _ in range(5):
        sel, _ = select_run(b, q2, bounds, scales, 1, 2, 32)
        o, l, _ = attn_run(b, q, caches, sel, 0.1)
        assert np.array_equal(sel, first) and torch.equal(o, out) and torch.equal(l, lse)


def test_bindings_refuse_wrong_tensors():
    rng = np.random.default_rng(32)
    b = batch(rng, [100], [1], 16)
    q, caches, sel = attn_case(rng, b, 4, 1, 64, 4)
    args = [q, *caches, dev(b["table"], I32), dev(b["qsl"], I32), dev(b["seq"], I32), dev(sel, I32), 0.1, b["longest"],
            torch.empty_like(q), None]
    for i, bad in ((0, q.float()), (0, q.cpu()), (1, caches[0].transpose(1, 2)), (2, caches[1][:-1]), (4, dev([0], I32)),
                   (5, dev(b["seq"], I64)), (6, dev(sel, I64)), (9, torch.empty_like(q)[:, :2])):
        with pytest.raises(ValueError):
            pka.pka_sparse_attn_forward(*args[:i], bad, *args[i + 1:])
    s = rope_case(4, 4, 2, 64, 64, False, True, False, True)
    for n, bad in (("q", s["q"].transpose(1, 2)), ("k", s["k"][..., ::2]), ("table", s["table"].double()), ("qw", s["qw"][:8]),
                   ("pos", s["pos"].long()), ("v", s["v"][:2]), ("q_out", s["q_out"][:, :2]), ("v_cache", s["v_cache"].float())):
        with pytest.raises(ValueError):
            rope_call(dict(s, **{n: bad}))
    with pytest.raises(pka.PkaError):
        rope_call(dict(s, kw=None))
    for bad in (dict(scales=(0.1,)), dict(scales=3.0), dict(eps="small")):
        with pytest.raises((ValueError, TypeError)):
            rope_call(dict(s, k_cache=s["k_cache"].view(torch.uint8)[..., :64].contiguous(),
                           v_cache=s["v_cache"].view(torch.uint8)[..., :64].contiguous(), **bad))
    with pytest.raises(TypeError):
        pka.pka_sparse_attn_forward(None, *args[1:])
    with pytest.raises((TypeError, AttributeError)):
        pka.pka_sparse_attn_forward(*args, stream="main")


def test_steps_without_tokens():
    s, table0 = tables_case([37, 0], [0, 0], 16, 0, [], 0)
    assert int(s["err"]) == 0 and s["qsl"].tolist() == [0, 0, 0] and s["seq"].tolist() == [37, 0]
    assert int(s["head_out"]) == 0 and np.array_equal(s["table"].cpu().numpy(), table0)
    r = rope_case(0, 4, 2, 64, 64, False, True, False, False, nb=2)
    before = copies(r)
    rope_call(r)
    assert torch.equal(r["k_cache"], before["k_cache"]) and int(r["err"]) == 0
    rng = np.random.default_rng(33)
    b = batch(rng, [100, 20], [0, 0], 16)
    q, bounds, scales = select_case(rng, b, 4, 2, 64)
    sel, err = select_run(b, q, bounds, scales, 1, 1, 5)
    assert sel.shape == (0, 2, 5) and err == 0
    cache = torch.zeros(b["nb"], 2, 16, 64, dtype=BF16, device="cuda")
    assert attn_run(b, q, (cache, cache), sel, 0.1)[2] == 0
    codes = torch.ones(b["nb"], 2, 2, 64, dtype=torch.int8, device="cuda")
    units = torch.ones(b["nb"], 2, device="cuda")
    pka.pka_page_bounds(cache, dev(np.zeros(0), I64), codes, units)
    assert (codes == 1).all() and (units == 1).all()


def test_lists_longer_than_the_pages():
    rng = np.random.default_rng(34)
    b = batch(rng, [300, 5], [1, 2], 16)
    q, bounds, scales = select_case(rng, b, 8, 2, 128)
    sel, err = select_run(b, q, bounds, scales, 3, 2, 3000)
    assert err == 0
    for t, n in enumerate([19, 1, 1]):
        assert (sel[t] == np.concatenate([np.arange(n), np.full(3000 - n, -1)])).all()
    q, caches, _ = attn_case(rng, b, 8, 2, 128, 4)
    out, lse, err = attn_run(b, q, caches, sel, 0.1)
    assert err == 0
    attn_near(out, lse, ref.sparse_attn(ref.f64(q), *map(ref.f64, caches), b["table"], b["qsl"], b["seq"], sel, 0.1))


def test_streams_and_threads():
    rng = np.random.default_rng(35)
    b = batch(rng, [3000, 5000, 77], [1, 2, 1], 16)
    q, caches, sel = attn_case(rng, b, 16, 2, 128, 32)
    want = attn_run(b, q, caches, sel, 0.1)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # made there, run there by the three ways to name a stream
        for stream in (None, side, side.cuda_stream):
            got = attn_run(b, q, caches, sel, 0.1, stream=stream)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and got[2] == 0
    torch.cuda.synchronize()
    wrong = []

    def serve():
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(20):
                out, lse, err = attn_run(b, q, caches, sel, 0.1)
                if err or not torch.equal(out, want[0]) or not torch.equal(lse, want[1]):
                    wrong.append(err)

    threads = [threading.Thread(target=serve) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
