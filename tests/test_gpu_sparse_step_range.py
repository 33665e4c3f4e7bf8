"""The block-sparse step at the far ends of the ranges its header names: magnitudes up to a type's own limits, weights
far below the largest, lists of many turns, batches of many requests. Against float64; a tolerance's parts stand at
its test."""
import numpy as np
import pytest
import torch

from paged_kv_attention_07_gb300 import pka
from tests import sparse_ref as ref
from tests.test_gpu_sparse_step import (BF16, I32, I64, attn_case, attn_near, attn_run, batch, bounds_check, dev, randn,
                                        select_case, select_check, word)

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- page bounds


def keys_far_apart(rng, nb, Hkv, bs, d):
    """Each element of a page of one sign and magnitude, from the least subnormal to beyond 2^120."""
    e = rng.integers(-133, 121, (nb, Hkv, 1, d)).astype(np.float64)
    e[..., rng.integers(0, d)] = 120
    sign = rng.choice([-1.0, 1.0], e.shape)
    return torch.from_numpy(sign * np.exp2(e) * rng.uniform(1, 2, (nb, Hkv, bs, d))).float().to(BF16)


@pytest.mark.parametrize("bs,d", [(1, 64), (8, 64), (16, 128), (64, 64), (64, 128), (200, 128)])
def test_page_bounds_enclose_elements_far_below_the_largest(bs, d):
    rng = np.random.default_rng(bs + d)
    nb, Hkv = 6, 2
    keys = keys_far_apart(rng, nb, Hkv, bs, d)
    keys[0, 0], keys[0, 0, 0, 3] = -2.0 ** -40, 2.0 ** 120  # the low code -1, not 0
    keys[1, 1], keys[1, 1, bs - 1, d - 1] = 2.0 ** -133, torch.finfo(BF16).max  # the high code 1
    keys[2, 0], keys[2, 0, 0, 0] = 0, -torch.finfo(BF16).max  # and zeros have both 0
    keys = keys.cuda()
    codes = torch.zeros(nb, Hkv, 2, d, dtype=torch.int8, device="cuda")
    scales, err = torch.zeros(nb, Hkv, device="cuda"), word()
    slots = [b * bs + bs - 1 for b in range(nb)]
    c0, s0 = codes.clone(), scales.clone()
    pka.pka_page_bounds(keys, dev(slots, I64), codes, scales, error_word=err)
    assert int(err) == 0
    bounds_check(keys, slots, c0, s0, codes, scales)
    assert codes[0, 0, 0, 5] == -1 and codes[1, 1, 1, 5] == 1 and codes[2, 0, :, 5].tolist() == [0, 0]


# ---------------------------------------------------------------- page selection


def far_select_case(rng, b, Hq, Hkv, d, q_power, page_power):
    """Queries and pages whose units are powers of two from the given ranges; bounds of both signs and of one."""
    lo = rng.integers(-127, 100, (b["nb"], Hkv, 1, d))
    hi = np.minimum(lo + rng.integers(0, 100, lo.shape), 127)
    sign = rng.choice([-1, 0, 1], (b["nb"], Hkv, 1, 1))
    bounds = np.where(sign == 0, np.concatenate([lo, hi], 2), sign * np.abs(np.concatenate([lo, hi], 2)))
    bounds = np.sort(bounds, axis=2)  # low before high
    scales = 2.0 ** rng.integers(*page_power, (b["nb"], Hkv))
    q = ref.f64(randn(rng, b["T"], Hq, d)) * 2.0 ** rng.integers(*q_power, (b["T"], Hq, 1))
    q = np.where(rng.random((b["T"], Hq, 1)) < 0.5, np.abs(q), q)  # scores below zero, with bounds of one sign
    q = np.clip(q, -3e38, 3e38)
    return torch.from_numpy(q).to(BF16).cuda(), bounds, scales


@pytest.mark.parametrize("q_power,page_power", [
    ((-3, 3), (107, 123)),     # one factor takes the sum past float32, the other brings it back
    ((100, 126), (-60, -50)), ((-80, 126), (-60, 123)), ((110, 126), (110, 123)), ((-80, -60), (-60, -55)),
    ((60, 64), (60, 64)),      # about the largest float32
])
@pytest.mark.parametrize("Hq,Hkv,d", [(8, 2, 128), (9, 1, 64), (6, 6, 128)])
def test_select_pages_scores_are_exact_at_any_magnitude(q_power, page_power, Hq, Hkv, d):
    rng = np.random.default_rng(Hq + q_power[0] + 1000)
    b = batch(rng, [900, 300, 3000], [1, 2, 1], 8)
    q, bounds, scales = far_select_case(rng, b, Hq, Hkv, d, q_power, page_power)
    # pages that bound nothing stand before the largest scores
    for blk in b["table"][0, [5, 60]]:
        scales[blk], bounds[blk] = np.inf, 0
    for K in (4, 20):
        select_check(b, q, bounds, scales, 1, 2, K)


def test_select_pages_large_units_keep_their_order():
    """127 codes of 127 in units of 2^110 against a query of ones: scores of about 2e37, of which the last page's
    is the best."""
    rng = np.random.default_rng(3)
    b = batch(rng, [640], [1], 16)
    n = 640 // 16
    bounds = np.full((b["nb"], 1, 2, 128), 127.0)
    for i in range(n):
        bounds[b["table"][0, i], 0, :, 0] = i
    q = torch.ones(1, 4, 128, dtype=BF16, device="cuda")
    select_check(b, q, bounds, np.full((b["nb"], 1), 2.0 ** 110), 0, 1, 6)


def test_select_pages_large_units_over_a_cluster():
    rng = np.random.default_rng(4)
    b = batch(rng, [20000], [1], 8)
    q, bounds, scales = far_select_case(rng, b, 4, 1, 128, (-3, 126), (90, 123))
    select_check(b, q, bounds, scales, 1, 2, 64)


# ---------------------------------------------------------------- attention over selected pages


def attn(b, q, caches, sel, scale, units=None):
    out, lse, err = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda"), word()
    pka.pka_sparse_attn_forward(q, *caches, dev(b["table"], I32), dev(b["qsl"], I32), dev(b["seq"], I32), dev(sel, I32),
                                scale, b["longest"], out, lse, kv_scales=units, error_word=err)
    assert int(err) == 0
    return ref.f64(out), ref.f64(lse)


def attn64(b, q, caches, sel, scale, units=(1.0, 1.0)):
    return ref.sparse_attn(ref.f64(q), *map(ref.f64, caches), b["table"], b["qsl"], b["seq"], sel, scale, units)


def lists(rng, b, Hkv, K, every=False):
    sel = np.full((b["T"], Hkv, K), -1)
    for t, r, p in ref.positions(b["qsl"], b["seq"]):
        for g in range(Hkv):
            n = p // b["bs"] + 1
            pages = np.sort(rng.permutation(n)[:n if every else min(n, K)])
            sel[t, g, :len(pages)] = pages
    return sel


@pytest.mark.parametrize("power", [20, 26, 29])
@pytest.mark.parametrize("pages,bs", [(33, 8), (2000, 8), (40, 64)])
def test_sparse_attn_8_bit_keeps_small_weights(power, pages, bs):
    """Every eighth key has the largest score and a value of zero: the result is what keys with weights of 2^-power
    of it add up to. A weight is off by 2^-11 of itself or by 2^-40 of the largest."""
    rng = np.random.default_rng(power + pages)
    b = batch(rng, [pages * bs - 3], [1], bs)
    k, v = np.zeros((b["nb"], 1, bs, 128)), np.abs(rng.standard_normal((b["nb"], 1, bs, 128))) * 8
    k[:, :, ::8, 0], v[:, :, ::8] = 1, 0
    caches = [torch.from_numpy(x).float().to(torch.float8_e4m3fn).view(torch.uint8).cuda() for x in (k, v)]
    q = torch.zeros(1, 2, 128, dtype=BF16, device="cuda")
    q[0, 0, 0], q[0, 1, 0] = 1, 1.0625
    sel = lists(rng, b, 1, pages + 1, every=True)
    scale = float(np.float32(power * np.log(2)))
    out, lse = attn(b, q, caches, sel, scale, (1.0, 1.0))
    o, l, size = attn64(b, q, caches, sel, scale)
    largest = 8 * 2.0 ** -40 * ref.f64(caches[1]).max()  # (of the seven keys beside each largest one)
    assert (np.abs(out - o) <= 2.0 ** -8 * np.abs(o) + (2.0 ** -14 + 2.0 ** -11) * size + largest).all()
    assert (np.abs(lse - l) <= 2.0 ** -14 * (1 + np.abs(l))).all()


@pytest.mark.parametrize("Hq,Hkv,d,bs,K", [(8, 2, 128, 16, 6), (6, 2, 64, 8, 9), (16, 1, 128, 64, 3), (9, 1, 64, 16, 40),
                                           (32, 4, 128, 64, 16), (2, 2, 128, 8, 80)])
@pytest.mark.parametrize("new", [1, 4])
def test_sparse_attn_is_off_by_its_results_rounding(Hq, Hkv, d, bs, K, new):
    """That rounding: 2^-8 of the value. Scores of up to 2^5 with a relative error of a few 2^-23: 2^-14 of the sum of
    the weighted magnitudes. A weight as two bf16 numbers, the first cut off, the second rounded: 2^-8 of 2^-7 of
    it, 2^-15 of that sum."""
    rng = np.random.default_rng(Hq + K + new)
    b = batch(rng, [0, 2 * bs - 3, 500, 40, 7, 1200], [new] * 6, bs)
    caches = [randn(rng, b["nb"], Hkv, bs, d) for _ in range(2)]
    q, sel = randn(rng, b["T"], Hq, d), lists(rng, b, Hkv, K)
    out, lse = attn(b, q, caches, sel, d ** -0.5)
    o, l, size = attn64(b, q, caches, sel, d ** -0.5)
    assert (np.abs(out - o) <= 2.0 ** -8 * np.abs(o) + (2.0 ** -14 + 2.0 ** -15) * size).all()
    assert (np.abs(lse - l) <= 2.0 ** -14 * (1 + np.abs(l))).all()


@pytest.mark.parametrize("d,bs", [(128, 16), (64, 8)])
def test_sparse_attn_infinite_values_are_infinite_results(d, bs):
    """Also where the key's weight is a power of two, the largest one, or has all its bits."""
    rng = np.random.default_rng(d)
    b = batch(rng, [37 * bs - 1], [1], bs)
    caches = [randn(rng, b["nb"], 1, bs, d) for _ in range(2)]
    q, sel = randn(rng, 1, 4, d), lists(rng, b, 1, 40, every=True)
    q[0, 1] = 0                                   # all weights one
    caches[0][b["table"][0, 5], 0, 1] = q[0, 2]  # the largest weight of its head
    caches[1][b["table"][0, 5], 0, 1, 3] = float("inf")
    caches[1][b["table"][0, 36], 0, 0, 4] = float("-inf")
    caches[1][b["table"][0, 8], 0, 2, 5] = float("inf")
    caches[1][b["table"][0, 9], 0, 2, 5] = float("-inf")
    out, lse = attn(b, q, caches, sel, d ** -0.5)
    assert (out[..., 3] == np.inf).all() and (out[..., 4] == -np.inf).all() and np.isnan(out[..., 5]).all()
    assert np.isfinite(np.delete(out, [3, 4, 5], -1)).all() and np.isfinite(lse).all()


def page_for_each_head(rng, B, bs, keys, d, fp8):
    """B requests that share one block table, a token each, whose heads look for a page each: keys of a page are
    its own signs, values its own numbers, so a page that is lost, doubled or another's shows in its head's row."""
    b = batch(rng, [keys - 1], [1], bs)
    n = -(-keys // bs)
    sign = torch.from_numpy(rng.choice([-1.0, 1.0], (b["nb"], d)))
    values = torch.from_numpy(rng.standard_normal((b["nb"], d)) * (8 if fp8 else 1))
    kind = torch.float8_e4m3fn if fp8 else BF16
    caches = [x.float().to(kind).view(torch.uint8 if fp8 else BF16)[:, None, None].expand(-1, 1, bs, -1).contiguous()
              for x in (sign, values)]
    b = dict(b, table=np.repeat(b["table"], B, 0), qsl=list(range(B + 1)), seq=[keys] * B, T=B)
    return b, caches, n, sign


def targets_of(rng, n, count):
    """Pages about every 32nd of each of 16 runs of the list, then any."""
    near = [run * n // 16 + i + j for run in range(16) for i in range(0, n // 16 + 1, 32) for j in (-1, 0, 1)]
    near = list(dict.fromkeys(x for x in near if 0 <= x < n))[:count]
    rest = [x for x in rng.permutation(n).tolist() if x not in set(near)]
    return np.array((near + rest * -(-count // max(len(rest), 1)))[:count])


def each_page_case(bs, fp8):
    rng = np.random.default_rng(bs)
    B, G, d, keys = 40, 16, 128, 40001
    b, caches, n, sign = page_for_each_head(rng, B, bs, keys, d, fp8)
    look = targets_of(rng, n, B * G)
    q = sign[torch.from_numpy(b["table"][0][look])].view(B, G, d).to(BF16)
    return b, caches, q, np.arange(n), look.reshape(B, G)


def attn_of_list(b, q, caches, pages, scale):
    """Of every head over the listed pages (some twice, perhaps), all keys up to the last: out, lse, the sum of the
    weighted magnitudes, and what the magnitudes add up to with 2^-40 of the largest weight each."""
    bs, keys = b["bs"], b["seq"][0]
    blk = torch.from_numpy(b["table"][0][pages])
    there = (torch.from_numpy(pages)[:, None] * bs + torch.arange(bs) < keys).flatten()
    k, v = (torch.from_numpy(ref.f64(c[:, 0]))[blk].flatten(0, 1)[there] for c in caches)
    s = q.double().flatten(0, 1) @ k.T * scale
    w = s.softmax(-1)
    least = 2.0 ** -40 * w.amax(-1, keepdim=True) * v.abs().sum(0)
    return tuple(x.unflatten(0, q.shape[:2]).numpy() for x in (w @ v, s.logsumexp(-1), w @ v.abs(), least))


def each_page_near(out, lse, want, fp8):
    """The result's rounding to bf16, 2^-8 of the value. Scores of up to 2^5 with a relative error of a few 2^-23: 2^-14
    of the sum of the weighted magnitudes. A weight as two bf16 numbers is off by 2^-15 of itself, as one of f16 by
    2^-11 of itself or by 2^-40 of the largest."""
    o, l, size, least = want
    near = np.abs(out - o) <= 2.0 ** -8 * np.abs(o) + (2.0 ** -14 + (2.0 ** -11 if fp8 else 2.0 ** -15)) * size + \
        (least if fp8 else 0)
    return near.all(-1) & (np.abs(lse - l) <= 2.0 ** -14 * (1 + np.abs(l)))


SCALE = 0.2


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("bs", [8, 64])
def test_sparse_attn_long_lists_page_by_page(bs, fp8):
    b, caches, q, pages, _ = each_page_case(bs, fp8)
    sel = np.broadcast_to(pages, (b["T"], 1, len(pages)))
    out, lse = attn(b, q.cuda(), [c.cuda() for c in caches], sel, SCALE, (1.0, 1.0) if fp8 else None)
    assert each_page_near(out, lse, attn_of_list(b, q, caches, pages, SCALE), fp8).all()
    if bs == 8:  # and without every third page
        pages = pages[pages % 3 != 1]
        sel = np.broadcast_to(pages, (b["T"], 1, len(pages)))
        out, lse = attn(b, q.cuda(), [c.cuda() for c in caches], sel, SCALE, (1.0, 1.0) if fp8 else None)
        assert each_page_near(out, lse, attn_of_list(b, q, caches, pages, SCALE), fp8).all()


# ---------------------------------------------------------------- batches of many requests


def many_requests(B, bs):
    """Requests of 0, 1, 2 and 5 new tokens in any order, runs of idle ones at both ends and within."""
    rng = np.random.default_rng(B + bs)
    new = rng.choice([0, 1, 1, 2, 5], B)
    new[:3] = new[-2:] = 0
    new[B // 2:B // 2 + min(B // 3, 70)] = 0
    new[B // 4] = 5
    ctx = rng.integers(0, 60, B)
    return rng, batch(rng, ctx.tolist(), new.tolist(), bs, extra_rows=3)


@pytest.mark.parametrize("B", [33, 64, 65, 1024, 1025, 3000])
def test_select_pages_of_many_requests(B):
    rng, b = many_requests(B, 4)
    select_check(b, *select_case(rng, b, 2, 1, 64), 1, 1, 5)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("B", [33, 64, 65, 1024, 1025, 3000])
def test_sparse_attn_of_many_requests(B, fp8):
    rng, b = many_requests(B, 8)
    q, caches, sel = attn_case(rng, b, 2, 1, 128, 3, fp8=fp8)
    units = (0.125, 0.25) if fp8 else None  # (float32 numbers)
    out, lse, err = attn_run(b, q, caches, sel, 0.09, units)
    assert err == 0
    attn_near(out, lse, ref.sparse_attn(ref.f64(q), *map(ref.f64, caches), b["table"], b["qsl"], b["seq"], sel, 0.09,
                                        units or (1.0, 1.0)))
