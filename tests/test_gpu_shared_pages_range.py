"""The calls over shared pages at the borders of what they promise: bad page ids wherever they are passed on, the error of
attention's results, infinite values, the size of its workspace."""
import math

import numpy as np
import pytest
import torch

from paged_kv_attention_07_gb300 import pka
from tests import shared_ref as ref
from tests.test_gpu_shared_pages import E, SHAPES, dev, f64, fork_case, one, prefix_call, prefix_case, prefix_check, word

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,width,bs", [(1, 1, 16), (3, 5, 4), (16, 200, 16), (17, 6, 16), (40, 700, 1), (64, 2500, 16)])
@pytest.mark.parametrize("bad", [0, 2 ** 31 - 1])
def test_fork_pages_bad_ids_of_rows_that_go_on_as_one(B, width, bs, bad):
    """A row with one child passes its pages on without looking at their counts: an id past the cache is an error all the
    same, in each size of launch (one CTA, a cluster, further ones for the copies), in whole pages and in the last one."""
    rng = np.random.default_rng(B * width)
    blocks = B * width + 5
    bad = bad or blocks
    parents = rng.permutation(B).tolist()
    for at in {(0, 0), (B - 1, width - 1), (B // 2, width // 3)}:
        for last in (0, bs - 1):  # tokens that its last page lacks
            table = rng.permutation(blocks)[:B * width].reshape(B, width)
            ctx = [width * bs] * B
            ctx[at[0]] = (at[1] + 1) * bs - last
            table[at] = bad
            s = fork_case(parents, ctx, table, bs, [0] * blocks, list(range(8)), 4)
            assert int(s["err"]) == E["BLOCK_ID"]
            want = np.full((B, width), -5)
            for i, p in enumerate(parents):
                held = -(-ctx[p] // bs)
                want[i, :held] = table[p, :held]
            assert np.array_equal(s["table_out"].cpu().numpy(), want) and s["ctx_out"].tolist() == [ctx[p] for p in parents]
            assert not s["counts"].any() and s["head_out"].tolist() == [4] and s["free"].tolist() == list(range(8))
            # behind the row's pages, and as a place that is no page, it is none
            if at[1] > 0:
                ctx[at[0]] = at[1] * bs
                assert int(fork_case(parents, ctx, table, bs, [0] * blocks, list(range(8)), 4)["err"]) == 0
            table[at] = -1
            ctx[at[0]] = (at[1] + 1) * bs
            assert int(fork_case(parents, ctx, table, bs, [0] * blocks, list(range(8)), 4)["err"]) == 0


@pytest.mark.parametrize("groups,Hq,Hkv,d,bs", SHAPES)
def test_prefix_attention_is_off_by_its_results_rounding(groups, Hq, Hkv, d, bs):
    """That rounding: 2^-8 of the value. A score of d products in 32 bits: (d + 8) 2^-24 of the largest sum of their
    magnitudes, exponentials and sums 2^-20, three times for weight, sum and their quotient. A weight as two bf16 numbers,
    the first cut off, the second rounded: half a step of the eighth bit behind the first's eight, 2^-16 of it, and 2^-17 that
    keeps the second above zero, below 2^-15 together."""
    rng = np.random.default_rng(Hq * d + bs)
    s = prefix_case(rng, groups, Hq, Hkv, d, bs)
    prefix_call(s)
    (k, v), table, qsl, seq, starts, prefix = s["host"]
    out, lse, mag, reach = ref.prefix_attention(f64(s["q"]), k, v, table, qsl, seq, starts, prefix, s["scale"])
    delta = (d + 8) * 2.0 ** -24 * reach + 2.0 ** -20
    limit = 2.0 ** -8 * np.abs(out) + (2.0 ** -15 + 3 * delta[..., None]) * mag * (1 + 2.0 ** -6) + 1e-30
    worst = np.abs(f64(s["out"]) - out) / limit
    assert int(s["err"]) == 0 and (worst <= 1).all(), (worst.max(), np.unravel_index(worst.argmax(), worst.shape))


@pytest.mark.parametrize("d,bs", [(128, 16), (64, 8)])
@pytest.mark.parametrize("groups", [one(0, [300, 20]), one(384, [1, 1, 200]), one(512, [40] * 40), one(129, [1]), one(256, [7, 30], 3)])
def test_prefix_attention_infinite_values_are_infinite_results(groups, d, bs):
    """Also where the key's weight is a power of two, the largest one, or has all its bits."""
    rng = np.random.default_rng(d + len(groups[0][1]))
    s = prefix_case(rng, groups, 8, 2, d, bs)
    (k, v), table, qsl, seq, starts, prefix = s["host"]
    reqs = [r for r in range(len(seq)) if qsl[r + 1] > qsl[r]]
    first = min(seq[r] - (qsl[r + 1] - qsl[r]) for r in reqs)  # keys that every token sees
    q = s["q"]
    q[:, 1] = 0  # all weights one
    many = len(seq) > 1
    for r in reqs:
        row = [table[reqs[0]][p // bs] if many and p < prefix[0] else table[r][p // bs] for p in range(first + 1)]
        at = lambda p: (int(row[p]), slice(None), p % bs)  # noqa: E731
        if r == reqs[0]:
            q[qsl[r], 2] = s["k"][int(row[first // 2]), 0, first // 2 % bs] * 4  # the largest weight of its head
        s["v"][at(first // 2)][:, 3] = math.inf
        s["v"][at(first)][:, 4] = -math.inf
        s["v"][at(first // 3)][:, 5] = math.inf
        s["v"][at(first - 1 if first else 0)][:, 5] = -math.inf
    prefix_call(s)
    got = f64(s["out"])
    assert int(s["err"]) == 0 and (got[..., 3] == np.inf).all() and (got[..., 4] == -np.inf).all() and np.isnan(got[..., 5]).all()
    assert np.isfinite(np.delete(got, [3, 4, 5], -1)).all() and torch.isfinite(s["lse"]).all()


@pytest.mark.parametrize("reqs,groups,tokens,Hq,Hkv,d,new", [
    (1024, 1024, 1024, 32, 8, 128, 1), (4096, 4096, 4096, 32, 16, 64, 1), (256, 256, 287, 32, 8, 128, 32),
    (192, 24, 192, 32, 8, 128, 1), (1, 1, 1, 8, 8, 128, 1), (64, 64, 8192, 64, 4, 128, 300), (40, 3, 120, 14, 2, 64, 3)])
def test_prefix_workspace_holds_what_can_be_written(reqs, groups, tokens, Hq, Hkv, d, new):
    """Of each token and head, for common and own keys, two partial results of d + 1 numbers, and those of one unit (up to
    two tiles of 128 rows) more per CTA; some words per request. Not more for groups that have nothing in common."""
    size = pka.pka_prefix_workspace_size(reqs, groups, tokens, Hq, Hkv, d, new)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    per_row = 2 * 4 * (d + 1)
    least = 2 * tokens * Hq * per_row if reqs > 1 else tokens * Hq * per_row
    assert least <= size <= least + 2 * sms * 256 * per_row + 16 * (reqs + groups + 64) + 8 * 256


@pytest.mark.parametrize("scales", [None, (0.02, 0.03)])
@pytest.mark.parametrize("groups,Hq,Hkv,bs", [(g, hq, hkv, bs) for g, hq, hkv, d, bs in SHAPES if d == 128])
def test_prefix_attention_stays_in_its_workspace(groups, Hq, Hkv, bs, scales):
    s = prefix_case(np.random.default_rng(Hq + bs), groups, Hq, Hkv, 128, bs, fp8_scales=scales)
    size = s["work"].numel()
    store = torch.full((size + (1 << 20),), 0x5a, dtype=torch.uint8, device="cuda")
    prefix_call(s, work=store[:size])
    prefix_check(s)
    assert (store[size:] == 0x5a).all()


def test_prefix_attention_workspace_past_32_bits():
    """Partial results whose offsets pass 32 bits: 4096 requests in pairs, 32 new tokens each, within the bound above."""
    rng = np.random.default_rng(50)
    B, new, common, bs, Hq, Hkv, d = 4096, 32, 16, 16, 32, 8, 128
    T, own = B * new, new // bs
    pages = torch.from_numpy(rng.permutation(B // 2 + B * own)).int().cuda()
    table = torch.cat([pages[:B // 2].repeat_interleave(2)[:, None], pages[B // 2:].view(B, own)], 1).contiguous()
    gen = torch.Generator(device="cuda")
    gen.manual_seed(50)
    normal = lambda *s: torch.randn(s, generator=gen, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    q, k, v = normal(T, Hq, d), normal(len(pages), Hkv, bs, d), normal(len(pages), Hkv, bs, d)
    size = pka.pka_prefix_workspace_size(B, B // 2, T, Hq, Hkv, d, new)
    assert size > 2 ** 33
    s = dict(q=q, k=k, v=v, table=table, qsl=dev(np.arange(B + 1) * new), seq=dev([common + new] * B), starts=dev(np.arange(0, B + 1, 2)),
             prefix=dev([common] * (B // 2)), scale=d ** -0.5, new=new, longest=common + new, out=torch.empty_like(q),
             lse=torch.empty(T, Hq, device="cuda"), scales=None, err=word(), work=torch.empty(size, dtype=torch.uint8, device="cuda"))
    prefix_call(s)
    assert int(s["err"]) == 0
    hidden = torch.ones(new, common + new, dtype=torch.bool, device="cuda").triu(common + 1)[None, :, None, None]
    for r in range(0, B, 256):
        at = table[r:r + 256].long()
        K, V = (x[at].double().transpose(2, 3).reshape(256, -1, Hkv, d) for x in (k, v))
        Q = q[r * new:(r + 256) * new].double().view(256, new, Hkv, Hq // Hkv, d)
        score = torch.einsum("rthgd,rnhd->rthgn", Q, K).mul_(s["scale"]).masked_fill_(hidden, -math.inf)
        reach = torch.einsum("rthgd,rnhd->rthgn", Q.abs(), K.abs()).amax(-1, keepdim=True) * s["scale"]
        weight, lse = score.softmax(-1), score.logsumexp(-1)
        want, mag = (torch.einsum("rthgn,rnhd->rthgd", weight, x) for x in (V, V.abs()))
        delta = (d + 8) * 2.0 ** -24 * reach + 2.0 ** -20
        limit = 2.0 ** -8 * want.abs() + (2.0 ** -15 + 3 * delta) * mag * (1 + 2.0 ** -6) + 1e-30
        got = s["out"][r * new:(r + 256) * new].double().view_as(want)
        assert ((got - want).abs() <= limit).all(), r
        assert ((s["lse"][r * new:(r + 256) * new].view_as(lse) - lse).abs() <= 2 * delta[..., 0] + 2.0 ** -22 * lse.abs()).all()


@pytest.mark.parametrize("scales", [None, (0.02, 0.03)])
@pytest.mark.parametrize("width,new", [(1, 1), (1, 3), (2, 1), (4, 2)])
def test_prefix_attention_lists_that_follow_one_another(width, new, scales):
    """More pieces in a CTA's share than it lists at a time, over either cache, of common keys too, with one new token and
    with several: roles and their barriers go on from list to list."""
    rng = np.random.default_rng(60 + width + new)
    B, Hkv, d, bs, common = 4096, 16, 128, 16, 16 if width > 1 else 0
    lens = rng.integers(new, bs + 1, B)
    own = torch.from_numpy(rng.permutation(B + B // width)).int().cuda()
    table = own[:B, None]
    if common:
        table = torch.cat([own[B:].repeat_interleave(width)[:, None], table], 1)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(width)
    normal = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    q = normal(B * new, Hkv, d).bfloat16()
    k, v = (normal(len(own), Hkv, bs, d) for _ in range(2))
    if scales:
        k, v = ((x / u).to(torch.float8_e4m3fn) for x, u in zip((k, v), scales))
        K, V = (x.double() * float(np.float32(u)) for x, u in zip((k, v), scales))
        k, v = k.view(torch.uint8), v.view(torch.uint8)
    else:
        k, v = k.bfloat16(), v.bfloat16()
        K, V = k.double(), v.double()
    size = pka.pka_prefix_workspace_size(B, B // width, B * new, Hkv, Hkv, d, new)
    s = dict(q=q, k=k, v=v, table=table.contiguous(), qsl=dev(np.arange(B + 1) * new), seq=dev(lens + common), starts=dev(np.arange(0, B + 1, width)),
             prefix=dev([common] * (B // width)), scale=d ** -0.5, new=new, longest=common + bs, out=torch.empty_like(q),
             lse=torch.empty(B * new, Hkv, device="cuda"), scales=scales, err=word(),
             work=torch.full((size,), 0xff, dtype=torch.uint8, device="cuda"))
    prefix_call(s)
    assert int(s["err"]) == 0
    seen = dev(lens + common)[:, None] - new + torch.arange(1, new + 1, device="cuda")  # [B, new] keys of each token
    for r in range(0, B, 512):
        rows = slice(r * new, (r + 512) * new)
        Kr, Vr = (x[table[r:r + 512].long()].transpose(2, 3).reshape(512, -1, Hkv, d) for x in (K, V))
        Q = q[rows].double().view(512, new, Hkv, d)
        hidden = (torch.arange(Kr.shape[1], device="cuda") >= seen[r:r + 512, :, None])[:, :, None]
        score = torch.einsum("rthd,rnhd->rthn", Q, Kr).mul_(s["scale"]).masked_fill_(hidden, -math.inf)
        delta = (d + 8) * 2.0 ** -24 * torch.einsum("rthd,rnhd->rthn", Q.abs(), Kr.abs()).amax(-1, keepdim=True) * s["scale"] + 2.0 ** -20
        if scales:  # the queries' split, as beside the other tests of this cache; weights in f16
            delta = delta + 2.0 ** -17 * Q.abs().amax(-1, keepdim=True) * Kr.abs().sum(-1).amax() * s["scale"]
        weight = score.softmax(-1)
        want, mag = (torch.einsum("rthn,rnhd->rthd", weight, x) for x in (Vr, Vr.abs()))
        limit = 2.0 ** -8 * want.abs() + ((2.0 ** -11 if scales else 2.0 ** -15) + 3 * delta) * mag * (1 + 2.0 ** -6) + 1e-30
        assert ((s["out"][rows].double().view_as(want) - want).abs() <= limit).all(), r
        lse = score.logsumexp(-1)
        assert ((s["lse"][rows].view_as(lse) - lse).abs() <= 2 * delta[..., 0] + 2.0 ** -22 * lse.abs()).all()
