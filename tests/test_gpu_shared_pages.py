"""The calls over shared pages on the GPU against their definitions in float64.

Tolerances, from the arithmetic. Whole numbers are equal. Attention: the result's and the weights' rounding to bf16 are
off by at most 2^-8 of the value and of each weight; a score of d products in 32 bits by (d + 8) 2^-24 of the sum of
their magnitudes, which moves a weight by as much of itself; exponentials and logarithms by a few 2^-22. Over an 8-bit
cache a query is two E4M3 numbers in units that bring its largest element to 224 at least: off by half of 2^-9, 2^-17 of
the largest, per element; the weights there are f16 (2^-11), within the bf16 bound."""
import math
import threading

import numpy as np
import pytest
import torch

from oracle import fp8
from paged_kv_attention_07_gb300 import pka
from tests import shared_ref as ref

pytestmark = pytest.mark.gpu

BF16, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
E = pka.DEVERR


def dev(x, dtype=I32):
    return torch.tensor(np.asarray(x), dtype=dtype, device="cuda")


def word():
    return torch.zeros(1, dtype=I32, device="cuda")


def f64(t):
    return t.double().cpu().numpy()


# ---------------------------------------------------------------- selection


def select_case(logits, scores, keep, finished=None, end=-1, ended=True):
    G, W = scores.shape
    s = dict(scores=torch.full((G, keep), 7.0, device="cuda"), parents=dev(np.full((G, keep), -9)),
             tokens=dev(np.full((G, keep), -9)), finished=dev(np.full((G, keep), 9), U8) if ended else None, err=word())
    pka.pka_beam_select(logits, scores, s["scores"], s["parents"], s["tokens"], end, finished, s["finished"],
                        error_word=s["err"])
    return s


def check_select(logits, scores, keep, finished=None, end=-1):
    s = select_case(logits, scores, keep, finished, end)
    want = ref.beam_select(f64(logits), f64(scores), None if finished is None else finished.cpu().numpy(), end, keep)
    assert np.array_equal(s["parents"].cpu().numpy(), want[1])
    assert np.array_equal(s["tokens"].cpu().numpy(), want[2])
    assert np.array_equal(s["finished"].cpu().numpy(), want[3])
    got, w = f64(s["scores"]), want[0]
    ok = np.isfinite(w)
    assert np.array_equal(np.isfinite(got), ok) and (got[~ok] == -np.inf).all()
    # the sum of exponentials in 32 bits (2^-20 of it, with room), the rounding to 32 bits
    assert (np.abs(got[ok] - w[ok]) <= 2.0 ** -20 + 2.0 ** -24 * np.abs(w[ok])).all()
    assert int(s["err"]) == (E["LOGITS"] if want[4] else 0)
    return s


def rows(rng, n, vocab, dtype, pad=0, offset=0):
    x = torch.from_numpy(rng.standard_normal((n, vocab)) * 3).to(dtype).cuda()
    store = torch.full((n * (vocab + pad) + offset,), math.nan, dtype=dtype, device="cuda")
    view = store[offset:].view(n, vocab + pad)[:, :vocab]
    view.copy_(x)
    return view


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("G,W,V,K,pad,offset", [
    (1, 1, 1, 1, 0, 0), (1, 4, 32000, 4, 0, 0), (3, 5, 50001, 5, 0, 0), (2, 3, 8191, 6, 1, 3), (2, 2, 8193, 64, 7, 0),
    (40, 8, 1000, 16, 24, 8), (1, 64, 777, 64, 0, 0), (1, 1, 200000, 64, 0, 0), (300, 2, 100, 4, 0, 0),
    (5, 7, 3, 10, 0, 0), (1, 63, 9000, 20, 0, 0), (2, 16, 70000, 33, 8, 0), (1, 2, 65536, 2, 0, 1)])
def test_beam_select(G, W, V, K, pad, offset, dtype):
    rng = np.random.default_rng(G * W + V + K)
    logits = rows(rng, G * W, V, dtype, pad, offset)
    scores = dev(-20 * rng.random((G, W)), F32)
    end = int(rng.integers(0, V))
    check_select(logits, scores, K)
    check_select(logits, scores, K, dev(rng.random((G, W)) < 0.3, U8), end)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("G,W,V,K", [(30, 16, 900, 16), (25, 13, 5001, 7), (160, 8, 1029, 8), (9, 40, 3001, 40), (200, 3, 2500, 3)])
def test_beam_select_many_groups(G, W, V, K, dtype):
    """More clusters than run at once, parts that follow one another in a CTA, odd rows."""
    rng = np.random.default_rng(G)
    check_select(rows(rng, G * W, V, dtype, offset=int(dtype == BF16)), torch.from_numpy(-rng.random((G, W)) * 9).float().cuda(), K)


@pytest.mark.parametrize("W,K", [(10, 48), (13, 40), (20, 26), (20, 30), (17, 40), (20, 37), (26, 32), (41, 21)])
def test_beam_select_lists_of_every_size(W, K):
    """Lists about as large as the shared memory that needs no leave."""
    rng = np.random.default_rng(W)
    check_select(rows(rng, 3 * W, 2000, F32), torch.from_numpy(-rng.random((3, W)) * 9).float().cuda(), K)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [40, 8192, 30001, 100000])
def test_beam_select_ties(V, dtype):
    """Few values, constant rows, equal rows with equal scores: the lower beam and the lower token."""
    rng = np.random.default_rng(V)
    G, W, K = 2, 4, 12
    x = torch.from_numpy(rng.integers(-2, 3, (G * W, V)).astype(np.float64)).to(dtype).cuda()
    x[1] = 0.5
    x[2] = x[0]
    x[3] = x[0]
    x[5] = torch.where(torch.arange(V, device="cuda") % 2 == 0, 0.0, -0.0)
    x[6] = torch.finfo(dtype).min
    x[7] = torch.arange(V, device="cuda").to(dtype) / V
    scores = dev([[-1.0, -1.0, -1.0, -1.0], [-3.0, -0.25, -0.5, 0.0]], F32)
    check_select(x, scores, K)
    check_select(x[:, :V - 3], scores, 64)  # rows that are not aligned to 16 bytes


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_beam_select_masks(dtype):
    """-infinity and the type's lowest value as masks, rows with few tokens or none, beams that are not alive."""
    rng = np.random.default_rng(5)
    G, W, V, K = 3, 4, 20011, 9
    x = rows(rng, G * W, V, dtype)
    x[0, 3:] = -math.inf
    x[1, :] = -math.inf
    x[2, 10:] = torch.finfo(dtype).min
    x[3, :V - 1] = -math.inf
    x[4:8] = -math.inf
    x[9, 5000:] = -math.inf
    scores = dev([[-1, -2, -3, -0.5], [-1, -1, -1, -1], [0, -math.inf, -math.inf, -math.inf]], F32)
    s = check_select(x, scores, K)
    assert (s["parents"][1] == -1).all() and (s["tokens"][1] == -1).all()
    check_select(x, scores, K, dev([[0, 1, 0, 0], [0, 1, 0, 1], [0, 1, 0, 0]], U8), 7)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_beam_select_refused_rows(dtype):
    rng = np.random.default_rng(6)
    G, W, V, K = 4, 3, 9001, 5
    x = rows(rng, G * W, V, dtype)
    x[1, 8999] = math.nan
    x[5, 0] = math.inf
    x[6] = math.nan
    x[7] = -math.inf
    x[7, 9] = math.nan
    x[10] = math.nan  # of a beam that is finished, and of one that is not alive
    x[11] = math.inf
    scores = dev([[-1, -2, -3], [-1, -1, -1], [-1, -2, -2.5], [-1, -1.5, -math.inf]], F32)
    done = dev([[0] * 3, [0] * 3, [0] * 3, [0, 1, 0]], U8)
    check_select(x, scores, K, done, 4)
    scores[0, 0], scores[1, 1], scores[3, 1] = math.nan, math.inf, math.nan
    check_select(x, scores, K, done, 4)


def test_beam_select_magnitudes():
    """Logits of 1e38 and sums that only the difference from the largest keeps finite."""
    x = torch.zeros(4, 10000, device="cuda")
    x[0, :5000] = 3e38
    x[0, 5000:] = -3e38
    x[1] = torch.linspace(-1e30, 1e30, 10000, device="cuda")
    x[2] = torch.linspace(1e4, 1e4 + 1, 10000, device="cuda")
    x[3] = -3.4e38
    check_select(x, dev([[0, 0, 0, 0]], F32), 8)
    check_select(x, dev([[-1e30, 2.0, -5.0, 0.25]], F32), 8)


def test_beam_select_in_place_repeated_captured_and_on_another_stream():
    rng = np.random.default_rng(7)
    G, W, V = 6, 4, 33000
    x = rows(rng, G * W, V, BF16)
    first = dev(-5 * rng.random((G, W)), F32)
    done = dev(rng.random((G, W)) < 0.2, U8)
    want = check_select(x, first, W, done, 11)
    scores, ended = first.clone(), done.clone()
    parents, tokens, err = dev(np.zeros((G, W))), dev(np.zeros((G, W))), word()

    def call():
        pka.pka_beam_select(x, scores, scores, parents, tokens, 11, ended, ended, error_word=err)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    for a, b in ((scores, "scores"), (parents, "parents"), (tokens, "tokens"), (ended, "finished")):
        assert torch.equal(a, want[b])
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        scores.copy_(first), ended.copy_(done), parents.zero_(), tokens.zero_()
        graph.replay()
        assert torch.equal(scores, want["scores"]) and torch.equal(parents, want["parents"])
        assert torch.equal(tokens, want["tokens"]) and torch.equal(ended, want["finished"])


def test_beam_select_of_nothing():
    e = lambda *s, t=I32: torch.empty(s, dtype=t, device="cuda")  # noqa: E731
    pka.pka_beam_select(e(0, 10, t=BF16), e(0, 4, t=F32), e(0, 4, t=F32), e(0, 4), e(0, 4))


# ---------------------------------------------------------------- forks


def pool(rng, B, width, ctx, bs, share=True):
    """A table whose rows share leading whole pages with an earlier row, its counts, and a free list."""
    held = [-(-c // bs) for c in ctx]
    blocks = sum(held) + 2 * B + 9
    perm = rng.permutation(blocks).tolist()
    table = rng.integers(0, blocks, (B, width))
    used = 0
    counts = [0] * blocks
    for r in range(B):
        own = int(rng.integers(0, r)) if share and r and rng.random() < 0.7 else -1
        whole = min(ctx[r] // bs, ctx[own] // bs) if own >= 0 else 0
        same = int(rng.integers(0, whole + 1)) if whole else 0
        for c in range(held[r]):
            if c < same:
                table[r, c] = table[own, c]
                counts[table[r, c]] += 1
            else:
                table[r, c] = perm[used]
                used += 1
    return table, counts, perm, used


def fork_case(parents, ctx, table, bs, counts, free, head, in_place=False, out_rows=None):
    N, width = len(parents), table.shape[1]
    s = dict(parents=dev(parents), ctx=dev(ctx), table=dev(table), counts=dev(counts), free=dev(free), head=dev([head]),
             ctx_out=dev([-7] * N), table_out=dev(np.full((N, width), -5)), src=dev([-7] * N), dst=dev([-7] * N), err=word())
    s["head_out"] = s["head"] if in_place else dev([-7])
    pka.pka_fork_pages(s["parents"], s["ctx"], s["table"], bs, s["counts"], s["free"], s["head"], s["head_out"],
                       s["ctx_out"], s["table_out"], s["src"], s["dst"], error_word=s["err"])
    return s


def check_fork(parents, ctx, table, bs, counts, free, head, in_place=False):
    s = fork_case(parents, ctx, table, bs, counts, free, head, in_place)
    want = ref.fork_pages(parents, ctx, table, bs, counts, free, head, len(counts), np.full((len(parents), table.shape[1]), -5))
    assert int(s["err"]) == 0
    for name, w in zip(("ctx_out", "table_out", "counts", "free", "head_out", "src", "dst"), want):
        assert np.array_equal(s[name].cpu().numpy().reshape(np.shape(w)), np.asarray(w)), name
    assert np.array_equal(s["table"].cpu().numpy(), table)
    return want


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,N,bs,longest,lost", [
    (1, 1, 16, 0, 0.0), (1, 8, 16, 100, 0.0), (4, 4, 16, 90, 0.3), (8, 3, 1, 40, 0.5), (33, 40, 24, 700, 0.4),
    (64, 64, 64, 5000, 0.5), (300, 512, 16, 900, 0.2), (4096, 4096, 32, 64, 0.5), (40, 0, 16, 300, 1.0),
    (5, 1200, 16, 333, 0.1), (16, 16, 1, 3000, 0.5), (31, 32, 4, 37, 1.0)])
def test_fork_pages(B, N, bs, longest, lost, in_place):
    rng = np.random.default_rng(B + N + bs)
    ctx = rng.integers(0, longest + 1, B).tolist()
    table, counts, free, head = pool(rng, B, max(-(-c // bs) for c in ctx) + 2, ctx, bs)
    free = free + rng.integers(0, len(counts), max(0, N - (len(free) - head))).tolist()
    alive = np.flatnonzero(rng.random(B) >= lost)
    parents = rng.choice(alive, N).tolist() if len(alive) else [-1] * N
    parents = [-1 if rng.random() < 0.1 else int(x) for x in parents]
    check_fork(parents, ctx, table, bs, counts, free, head, in_place)


def test_fork_pages_step_after_step():
    """Forks and ends over many steps: the pages held and the free ones are always the whole pool."""
    rng = np.random.default_rng(3)
    B, bs, width = 12, 8, 40
    blocks = 500
    free, head = rng.permutation(blocks).tolist(), 0
    counts, ctx = [0] * blocks, [0] * B
    table = np.full((B, width), -5)
    for step in range(60):
        new = [int(rng.integers(0, 9)) if c < bs * (width - 2) else 0 for c in ctx]
        for r in range(B):  # pages of the new tokens, as pka_step_tables takes them
            for c in range(-(-ctx[r] // bs), -(-(ctx[r] + new[r]) // bs)):
                table[r, c] = free[head]
                head += 1
            ctx[r] += new[r]
        parents = [int(rng.integers(0, B)) if rng.random() < 0.5 else i for i in range(B)]
        if step % 7 == 6:
            parents[int(rng.integers(0, B))] = -1
        s = fork_case(parents, ctx, table, bs, counts, free, head, in_place=True)
        ctx, full, counts, free, head, src, dst = ref.fork_pages(parents, ctx, table, bs, counts, free, head, blocks,
                                                                 np.full((B, width), -5))
        for name, w in (("ctx_out", ctx), ("table_out", full), ("counts", counts), ("free", free), ("head", [head]),
                        ("src", src), ("dst", dst)):
            assert np.array_equal(s[name].cpu().numpy(), np.asarray(w)), (step, name)
        table = full
        held = [table[r, :-(-ctx[r] // bs)] for r in range(B)]
        ids, times = np.unique(np.concatenate(held), return_counts=True)
        assert np.array_equal(np.asarray(counts)[ids], times - 1) and sum(counts) == (times - 1).sum()
        assert sorted(ids.tolist() + free[head:]) == list(range(blocks))
    want = check_fork([-1] * B, ctx, table, bs, counts, free, head)
    assert want[4] == 0 and sorted(want[3]) == list(range(blocks))


@pytest.mark.parametrize("change,bit", [
    (dict(parents=[0, 3, 1]), "INDEX"), (dict(ctx=[5, -1, 3]), "SEQ_LEN"), (dict(ctx=[5, 1000, 3]), "BLOCK_TABLE"),
    (dict(head=8), "CAPACITY"), (dict(head=-1), "CAPACITY"), (dict(free=[1, 2, 3]), "CAPACITY")])
@pytest.mark.parametrize("in_place", [False, True])
def test_fork_pages_refused_on_the_device(change, bit, in_place):
    a = dict(parents=[0, 0, 1], ctx=[5, 6, 3], table=np.arange(12).reshape(3, 4), bs=4, counts=[0] * 20,
             free=[12, 13, 14, 15, 16, 17, 18, 19], head=3)
    a.update(change)
    s = fork_case(**a, in_place=in_place)
    assert int(s["err"]) & E[bit]
    assert s["ctx_out"].tolist() == [0] * 3 and s["src"].tolist() == s["dst"].tolist() == [-1] * 3
    assert s["counts"].tolist() == a["counts"] and s["free"].tolist() == a["free"] and s["head_out"].tolist() == [a["head"]]


def test_fork_pages_ids_that_are_no_pages():
    table = np.array([[3, -1, 4, 7], [3, 99, 5, 8]])
    s = fork_case([0, 0], [16, 11], table, 4, [0, 0, 0, 1, 0, 0, 0, 0, 0, 0], [3, 4, 7, 5, 8, 9, 6], 5)
    assert int(s["err"]) == E["BLOCK_ID"]
    assert s["table_out"].tolist() == [[3, -1, 4, 7]] * 2 and s["ctx_out"].tolist() == [16, 16]
    assert s["counts"].tolist() == [0, 0, 0, 1, 1, 0, 0, 1, 0, 0]
    assert s["head_out"].tolist() == [4] and s["free"].tolist() == [3, 4, 7, 5, 5, 9, 6]


def test_fork_pages_without_room_in_front():
    s = fork_case([-1], [8], np.array([[1, 2]]), 4, [0] * 4, [3, 0], 1)
    assert int(s["err"]) == E["CAPACITY"] and s["head_out"].tolist() == [0] and s["free"].tolist() == [2, 0]


def test_fork_pages_captured():
    rng = np.random.default_rng(9)
    ctx = rng.integers(0, 300, 20).tolist()
    table, counts, free, head = pool(rng, 20, 25, ctx, 16)
    parents = rng.integers(-1, 20, 20).tolist()
    s = fork_case(parents, ctx, table, 16, counts, free, head)
    c, f, out = dev(counts), dev(free), dev(np.full((20, 25), -5))
    h, lens, src, dst, err = dev([head]), dev([0] * 20), dev([0] * 20), dev([0] * 20), word()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        pka.pka_fork_pages(s["parents"], s["ctx"], s["table"], 16, c, f, h, h, lens, out, src, dst, error_word=err)
    for _ in range(3):
        c.copy_(dev(counts)), f.copy_(dev(free)), h.copy_(dev([head]))
        graph.replay()
        for a, b in ((c, "counts"), (f, "free"), (h, "head_out"), (lens, "ctx_out"), (out, "table_out"), (src, "src"), (dst, "dst")):
            assert torch.equal(a, s[b]), b


# ---------------------------------------------------------------- copies


@pytest.mark.parametrize("caches,blocks,shape,dtype,pairs", [
    (1, 2, (8,), BF16, 1), (2, 9, (3, 16, 64), BF16, 4), (7, 30, (4, 16, 128), U8, 13), (256, 11, (1, 1, 16), U8, 5),
    (3, 6, (8, 128, 128), BF16, 2), (2, 4000, (1, 8, 64), BF16, 1900), (0, 2, (8,), BF16, 1), (2, 5, (5, 3, 8), F32, 0)])
def test_copy_pages(caches, blocks, shape, dtype, pairs):
    rng = np.random.default_rng(blocks)
    new = lambda: torch.randint(0, 256, (blocks, *shape, dtype.itemsize), device="cuda").to(U8).flatten(-2).view(dtype)  # noqa: E731
    have = [new() for _ in range(caches)]
    perm = rng.permutation(blocks)[:2 * pairs]
    src, dst = perm[:pairs].copy(), perm[pairs:].copy()
    skip = rng.random(pairs) < 0.3
    src[skip], dst[rng.random(pairs) < 0.1] = -1, -1
    want = [c.clone() for c in have]
    ok = (src >= 0) & (dst >= 0)
    for c in want:
        c[dev(dst[ok], torch.long)] = c[dev(src[ok], torch.long)]
    err = word()
    pka.pka_copy_pages(have, dev(src), dev(dst), error_word=err)
    for a, b in zip(have, want):
        assert torch.equal(a.view(U8), b.view(U8))
    assert int(err) == 0


def test_copy_pages_ids_past_the_cache_and_past_32_bits():
    c = torch.arange(6 * 8, device="cuda", dtype=F32).view(6, 8)
    want = c.clone()
    want[2] = want[1]
    err = word()
    pka.pka_copy_pages([c], dev([1, 6, 3]), dev([2, 4, 2 ** 31 - 1]), error_word=err)
    assert torch.equal(c, want) and int(err) == E["BLOCK_ID"]
    big = torch.empty(70000, 65536, dtype=U8, device="cuda")  # 4.6 GB
    big[69999] = 5
    big[3] = 1
    pka.pka_copy_pages([big], dev([69999, 3]), dev([1, 69998]), error_word=err)
    assert (big[1] == 5).all() and (big[69998] == 1).all()


# ---------------------------------------------------------------- attention


def prefix_batch(rng, groups, Hkv, d, bs, kv=None, extra=3, poison=True):
    """groups: a list of (prefix, [(own tokens, new tokens), ...]). Pages of common tokens are shared."""
    starts, prefix, seq, new = [0], [], [], []
    for p, members in groups:
        prefix.append(p)
        starts.append(starts[-1] + len(members))
        seq += [p + own for own, _ in members]
        new += [n for _, n in members]
    B = len(seq)
    width = max(1, max(-(-s // bs) for s in seq)) + 1
    total = sum(-(-s // bs) for s in seq) + extra
    perm = rng.permutation(total).tolist()
    table = np.full((B, width), 10 ** 8)
    for g, (p, members) in enumerate(groups):
        shared = [perm.pop() for _ in range(p // bs)]
        for i, r in enumerate(range(starts[g], starts[g + 1])):
            for c in range(-(-seq[r] // bs)):
                table[r, c] = shared[c] if c < len(shared) else perm.pop()
        # only the row of the first request with new tokens is read for the common ones
        read = next((r for r in range(starts[g], starts[g + 1]) if new[r]), -1)
        for r in range(starts[g], starts[g + 1]):
            if poison and r != read and len(members) > 1:
                table[r, :p // bs] = 10 ** 8
    qsl = [0]
    for n in new:
        qsl.append(qsl[-1] + n)
    return starts, prefix, seq, qsl, table, total


def prefix_case(rng, groups, Hq, Hkv, d, bs, fp8_scales=None, pad=0, q=None, caches=None, lse=True, scale=None, width=None):
    starts, prefix, seq, qsl, table, total = prefix_batch(rng, groups, Hkv, d, bs)
    T = qsl[-1] + pad
    q = torch.from_numpy(rng.standard_normal((T, Hq, d)) * 1.5).to(BF16).cuda() if q is None else q
    if caches is None:
        caches = [torch.from_numpy(rng.standard_normal((total, Hkv, bs, d))).to(BF16).cuda() for _ in range(2)]
    scale = scale or 1 / math.sqrt(d)
    # what no request holds is NaN
    held = np.zeros((total, bs), bool)
    for g in range(len(prefix)):
        reqs = [r for r in range(starts[g], starts[g + 1]) if qsl[r + 1] > qsl[r]]
        for r in reqs:
            many = starts[g + 1] - starts[g] > 1
            for pos in range(seq[r]):
                row = reqs[0] if many and pos < prefix[g] else r
                held[table[row, pos // bs], pos % bs] = True
    gap = torch.from_numpy(~held).cuda()[:, None, :, None]
    caches = [c.masked_fill(gap, math.nan) for c in caches]
    if fp8_scales:
        stored = [torch.from_numpy(fp8.quantize_f32(c.float().cpu().numpy(), s)).cuda() for c, s in zip(caches, fp8_scales)]
        stored = [s.masked_fill(gap, 0x7f) for s in stored]
        values = [np.nan_to_num(fp8.decode(s.cpu().numpy()).astype(np.float64)) for s in stored]
    else:
        stored, values = caches, [np.nan_to_num(f64(c), nan=0.0) for c in caches]
    new = max([b - a for a, b in zip(qsl, qsl[1:])] + [1])
    size = pka.pka_prefix_workspace_size(len(seq), len(prefix), T, Hq, Hkv, d, new)
    s = dict(q=q, k=stored[0], v=stored[1], table=dev(np.minimum(table, 2 ** 31 - 1)), qsl=dev(qsl), seq=dev(seq),
             starts=dev(starts), prefix=dev(prefix), scale=scale, new=new, longest=max(seq + [1]),
             out=torch.full((T, Hq, d), 7.0, dtype=BF16, device="cuda"),
             lse=torch.full((T, Hq), 7.0, device="cuda") if lse else None,
             work=torch.full((size,), 0xff, dtype=U8, device="cuda"), scales=fp8_scales, err=word())
    s["host"] = (values, table, qsl, seq, starts, prefix)
    return s


def prefix_call(s, **kw):
    a = dict(s, **kw)
    pka.pka_prefix_attn_forward(a["q"], a["k"], a["v"], a["table"], a["qsl"], a["seq"], a["starts"], a["prefix"],
                                a["scale"], a["new"], a["longest"], a["out"], a["lse"], a["work"], kv_scales=a["scales"],
                                error_word=a["err"])


def prefix_check(s):
    (k, v), table, qsl, seq, starts, prefix = s["host"]
    ks, vs = s["scales"] or (1.0, 1.0)
    ks, vs = float(np.float32(ks)), float(np.float32(vs))
    out, lse, mag, reach = ref.prefix_attention(f64(s["q"]), k, v, table, qsl, seq, starts, prefix, s["scale"] * ks, vs)
    assert int(s["err"]) == 0
    n, d = qsl[-1], s["q"].shape[2]
    got = f64(s["out"])
    delta = (d + 8) * 2.0 ** -24 * reach[:n] + 2.0 ** -20
    if s["scales"]:  # the queries' split
        largest = np.abs(f64(s["q"])[:n]).max(-1)
        delta += 2.0 ** -17 * largest * np.abs(k).sum(-1).max() * s["scale"] * ks
    limit = 2.0 ** -8 * np.abs(out[:n]) + (2.0 ** -8 + 3 * delta[..., None]) * mag[:n] * (1 + 2.0 ** -6) + 1e-30
    worst = np.abs(got[:n] - out[:n]) / limit
    assert np.isfinite(got[:n]).all() and (worst <= 1).all(), (worst.max(), np.unravel_index(worst.argmax(), worst.shape))
    assert (got[n:] == 7.0).all()
    if s["lse"] is not None:
        g = f64(s["lse"])
        assert (np.abs(g[:n] - lse[:n]) <= 2 * delta + 2.0 ** -22 * np.abs(lse[:n])).all()
        assert (g[n:] == 7.0).all()


def one(prefix, own, new=1):
    return [(prefix, [(o, new) for o in own])]


SHAPES = [
    # groups, Hq, Hkv, d, bs
    (one(0, [1]), 1, 1, 64, 16), (one(1, [1, 1]), 8, 8, 128, 16), (one(64, [3, 70, 129, 1]), 32, 8, 128, 16),
    (one(300, [5, 1, 40]), 32, 4, 128, 16), (one(127, [2, 2, 2, 2, 2]), 12, 4, 64, 32), (one(513, [9] * 20), 16, 2, 128, 64),
    (one(200, [30, 4, 2, 90], 2), 14, 2, 128, 8), (one(1000, [600, 3, 1]), 3, 3, 64, 128), (one(37, [40] * 9, 3), 16, 1, 64, 1),
    (one(90, [20, 21, 22], 5), 10, 2, 128, 2), (one(40, [300, 310], 260), 8, 2, 128, 16), (one(2000, [100]), 32, 8, 128, 16),
    ([(0, [(50, 1), (3, 1)]), (128, [(1, 1)]), (77, [(5, 2), (9, 1), (200, 4)]), (640, [(1, 1)] * 33)], 32, 8, 128, 16),
    ([(p, [(1 + i, 1) for i in range(1 + p % 4)]) for p in range(0, 900, 19)], 8, 2, 64, 16),
    ([(96, [(17, 16), (33, 1)]), (0, [(130, 130)]), (256, [(1, 1), (64, 64)])], 40, 8, 128, 32),
]


@pytest.mark.parametrize("groups,Hq,Hkv,d,bs", SHAPES)
def test_prefix_attention(groups, Hq, Hkv, d, bs):
    rng = np.random.default_rng(Hq + d + bs)
    s = prefix_case(rng, groups, Hq, Hkv, d, bs)
    prefix_call(s)
    prefix_check(s)
    first = s["out"].clone(), s["lse"].clone()
    s["work"].fill_(0x7f)
    prefix_call(s)
    assert torch.equal(first[0], s["out"]) and torch.equal(first[1], s["lse"])


@pytest.mark.parametrize("scales", [(0.0125, 0.02), (0.5, 3.0)])
@pytest.mark.parametrize("groups,Hq,Hkv,bs", [(g, hq, hkv, bs) for g, hq, hkv, d, bs in SHAPES if d == 128] + [
    (one(300, [5, 1, 40], 1), 12, 4, 128), (one(77, [20, 21], 7), 10, 2, 1), (one(130, [3] * 50), 16, 2, 4)])
def test_prefix_attention_fp8(groups, Hq, Hkv, bs, scales):
    rng = np.random.default_rng(Hq + bs)
    s = prefix_case(rng, groups, Hq, Hkv, 128, bs, fp8_scales=scales)
    prefix_call(s)
    prefix_check(s)
    first = s["out"].clone()
    s["work"].fill_(0x7f)
    prefix_call(s)
    assert torch.equal(first, s["out"])


def test_prefix_attention_idle_requests_padded_rows_empty_groups():
    rng = np.random.default_rng(1)
    groups = [(50, [(10, 0), (20, 1), (5, 0), (7, 2)]), (30, []), (0, [(4, 0)]), (16, [(9, 0), (8, 0)]), (64, [(0 + 1, 1), (64, 3)])]
    s = prefix_case(rng, groups, 8, 2, 64, 16, pad=5)
    s["seq"][0] = -3  # lengths of idle requests are not looked at
    prefix_call(s)
    prefix_check(s)
    s = prefix_case(rng, [(50, [(10, 0), (20, 0)])], 8, 2, 64, 16, pad=3, lse=False)
    prefix_call(s)
    prefix_check(s)


def test_prefix_attention_is_that_of_plain_groups():
    """The same batch as groups, as groups of one, and through the dense decode: the same within roundings."""
    rng = np.random.default_rng(2)
    starts, prefix, seq, qsl, table, total = prefix_batch(rng, one(896, [40, 1, 300, 77]), 4, 128, 16, poison=False)
    q = torch.from_numpy(rng.standard_normal((4, 16, 128))).to(BF16).cuda()
    k, v = (torch.from_numpy(rng.standard_normal((total, 4, 16, 128))).to(BF16).cuda() for _ in range(2))
    out, lse = [], []
    for st, pf in ((starts, prefix), ([0, 1, 2, 3, 4], [896, 0, 3, 896]), ([0, 4], [0])):
        size = pka.pka_prefix_workspace_size(4, len(pf), 4, 16, 4, 128, 1)
        o, l, err = torch.empty_like(q), torch.empty(4, 16, device="cuda"), word()
        pka.pka_prefix_attn_forward(q, k, v, dev(table), dev(qsl), dev(seq), dev(st), dev(pf), 0.1, 1, max(seq), o, l,
                                    torch.empty(size, dtype=U8, device="cuda"), error_word=err)
        assert int(err) == 0
        out.append(o.float())
        lse.append(l)
    work = torch.empty(pka.pka_workspace_size(4, 0, 0, 4, 16, 4, 128, 128, 1, max(seq), 32768), dtype=U8, device="cuda")
    o, l = torch.empty_like(q), torch.empty(4, 16, device="cuda")
    pka.pka_paged_attn_forward(q, None, None, k, v, dev(np.minimum(table, 2 ** 31 - 1)), dev(qsl), dev(seq), 4, 0, 0, 0.1, 32768, 1, max(seq), o, l, work)
    out.append(o.float())
    lse.append(l)
    for a, b in zip(out[1:], lse[1:]):
        assert (a - out[0]).abs().max() <= 2 ** -6 * 4 and (b - lse[0]).abs().max() <= 1e-4


def test_prefix_attention_many_small_units():
    """More pieces in a CTA's share than it lists at a time."""
    rng = np.random.default_rng(4)
    B, Hkv, bs = 4096, 16, 16
    table = dev(np.arange(B)[:, None])
    q = torch.from_numpy(rng.standard_normal((B, 16, 64))).to(BF16).cuda()
    k, v = (torch.from_numpy(rng.standard_normal((B, Hkv, bs, 64))).to(BF16).cuda() for _ in range(2))
    seq = rng.integers(1, bs + 1, B)
    s = dict(q=q, k=k, v=v, table=table, qsl=dev(np.arange(B + 1)), seq=dev(seq), starts=dev(np.arange(B + 1)),
             prefix=dev([0] * B), scale=0.125, new=1, longest=bs, out=torch.empty_like(q),
             lse=torch.empty(B, 16, device="cuda"), scales=None, err=word(),
             work=torch.empty(pka.pka_prefix_workspace_size(B, B, B, 16, Hkv, 64, 1), dtype=U8, device="cuda"))
    prefix_call(s)
    score = torch.einsum("bhd,bhnd->bhn", q.double(), k.double()) * 0.125
    score = score.masked_fill(torch.arange(bs, device="cuda") >= dev(seq)[:, None, None], -math.inf)
    want = torch.einsum("bhn,bhnd->bhd", score.softmax(-1), v.double())
    assert (s["out"].double() - want).abs().max() <= 2 ** -8 * 2 * v.abs().max().item() and int(s["err"]) == 0
    assert (s["lse"].double() - score.logsumexp(-1)).abs().max() <= 1e-5


@pytest.mark.parametrize("change,bit", [
    (dict(starts=[1, 2, 4]), "INDEX"), (dict(starts=[0, 3, 2]), "INDEX"), (dict(starts=[0, 2, 3]), "INDEX"),
    (dict(starts=[0, 9, 4]), "INDEX"), (dict(starts=[0, -5, 4]), "INDEX"), (dict(prefix=[40, -1]), "SEQ_LEN"),
    (dict(prefix=[41, 10]), "SEQ_LEN"), (dict(seq=[41, 50, 30, 2 ** 31 - 1]), "SEQ_LEN"), (dict(seq=[41, 0, 30, 11]), "SEQ_LEN"),
    (dict(seq=[41, -7, 30, 11]), "SEQ_LEN"), (dict(qsl=[0, 1, 3, 4, 9]), "QUERY_START_LOC"), (dict(qsl=[0, 2, 1, 4, 5]), "QUERY_START_LOC"),
    (dict(qsl=[1, 2, 3, 4, 5]), "QUERY_START_LOC"), (dict(qsl=[0, 1, 4, 5, 5]), "QUERY_LEN"), (dict(qsl=[-2, 1, 3, 4, 5]), "QUERY_START_LOC")])
def test_prefix_attention_refused_on_the_device(change, bit):
    rng = np.random.default_rng(8)
    s = prefix_case(rng, [(40, [(1, 1), (10, 2)]), (10, [(20, 1), (1, 1)])], 8, 2, 64, 16)
    prefix_call(s, **{k: dev(v) for k, v in change.items()})
    assert int(s["err"]) & E[bit]
    assert (s["out"] == 7.0).all() and (s["lse"] == 7.0).all()


def test_prefix_attention_block_ids_outside_the_cache():
    rng = np.random.default_rng(8)
    s = prefix_case(rng, one(40, [20, 1]), 8, 2, 64, 16)
    for bad in (-1, 10 ** 8):
        table = s["table"].clone()
        table[0, 1] = bad
        s["err"].zero_()
        prefix_call(s, table=table)
        assert int(s["err"]) == E["BLOCK_ID"]


def test_prefix_attention_captured_on_a_stream_and_from_threads():
    rng = np.random.default_rng(10)
    s = prefix_case(rng, SHAPES[12][0], 32, 8, 128, 16)
    prefix_call(s)
    want = s["out"].clone()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        prefix_call(s)
    for _ in range(3):
        s["out"].zero_()
        graph.replay()
        assert torch.equal(s["out"], want)
    outs = [torch.empty_like(want) for _ in range(3)]
    torch.cuda.synchronize()

    def go(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            work = torch.empty_like(s["work"])
            for _ in range(10):
                prefix_call(s, out=outs[i], lse=None, work=work)
            torch.cuda.current_stream().synchronize()

    threads = [threading.Thread(target=go, args=(i,)) for i in range(3)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert all(torch.equal(o, want) for o in outs)


# groups of requests with several new tokens; what is not finite lies in the last `late` of them
LATE = [(one(40, [20, 30], 3), 1), (one(200, [64, 65, 90], 5), 2), (one(3, [260, 300], 200), 70), (one(16, [9] * 12, 2), 1),
        ([(0, [(130, 130)]), (50, [(129, 2), (3, 3)])], 1)]


@pytest.mark.parametrize("scales", [None, (0.02, 0.03)])
@pytest.mark.parametrize("d,bs", [(64, 16), (128, 16), (128, 2)])
@pytest.mark.parametrize("groups,late", LATE)
def test_prefix_attention_values_that_are_not_finite(groups, late, d, bs, scales):
    """Infinities and NaN among the values of later tokens reach the tokens that see them, in their dims, and no other."""
    if scales and d != 128:
        d, bs = 128, 1
    rng = np.random.default_rng(late + d + bs)
    Hq, Hkv = 8, 2
    s = prefix_case(rng, groups, Hq, Hkv, d, bs, fp8_scales=scales)
    (k, v), table, qsl, seq, starts, prefix = s["host"]
    seen = np.zeros(s["q"].shape)  # the sum of what a token sees: 0, an infinity or NaN
    for r in range(len(seq)):
        n = qsl[r + 1] - qsl[r]
        for j in range(max(0, n - late), n):
            pos = seq[r] - n + j
            page, at = int(table[r, pos // bs]), pos % bs
            for h in range(Hkv):
                for dim in rng.choice(d, 5, replace=False):
                    x = float(rng.choice([np.inf, -np.inf, np.nan]))
                    if scales:
                        x = np.nan
                        s["v"][page, h, at, dim] = int(rng.choice([0x7f, 0xff]))
                    else:
                        s["v"][page, h, at, dim] = x
                    v[page, h, at, dim] = 0
                    seen[qsl[r] + j:qsl[r + 1], h * (Hq // Hkv):(h + 1) * (Hq // Hkv), dim] += x
    prefix_call(s)
    got = f64(s["out"])
    odd = seen != 0
    assert odd.any() and np.array_equal(np.isnan(got), np.isnan(seen)) and np.array_equal(got[np.isinf(seen)], seen[np.isinf(seen)])
    want = ref.prefix_attention(f64(s["q"]), k, v, table, qsl, seq, starts, prefix, s["scale"] * (scales or [1])[0],
                                (scales or [1, 1])[1])[0]
    s["out"] = torch.where(torch.from_numpy(odd).cuda(), torch.from_numpy(want).to(BF16).cuda(), s["out"])
    prefix_check(s)


def test_prefix_attention_keys_and_queries_that_are_not_finite():
    rng = np.random.default_rng(30)
    for scales in (None, (0.02, 0.03)):
        s = prefix_case(rng, [(64, [(20, 1), (30, 2), (1, 1)]), (0, [(200, 3)])], 8, 2, 128, 16, fp8_scales=scales)
        table, qsl, seq = s["host"][1:4]
        want = ref.prefix_attention(f64(s["q"]), *s["host"][0], *s["host"][1:], s["scale"] * (scales or [1])[0], (scales or [1, 1])[1])[0]
        bad = np.zeros(s["q"].shape[:2], bool)
        # a key of the last new token of requests 1 and 3, head 1, and queries
        for r in (1, 3):
            pos = seq[r] - 1
            s["k"][int(table[r, pos // 16]), 1, pos % 16, 3] = 0x7f if scales else math.nan
            bad[qsl[r + 1] - 1, 4:] = True
        for t, h, x in ((0, 2, math.inf), (3, 6, math.nan), (4, 0, -math.inf)):
            s["q"][t, h, 9] = x
            bad[t, h] = True
        prefix_call(s)
        got = f64(s["out"])
        assert np.isnan(got[bad]).all() and np.isnan(f64(s["lse"])[bad]).all()
        s["q"][torch.from_numpy(bad).cuda()] = 0
        s["out"] = torch.where(torch.from_numpy(bad).cuda()[..., None], torch.from_numpy(want).to(BF16).cuda(), s["out"])
        fixed = ref.prefix_attention(f64(s["q"]), *s["host"][0], *s["host"][1:], s["scale"] * (scales or [1])[0], (scales or [1, 1])[1])
        s["out"] = torch.where(torch.from_numpy(bad).cuda()[..., None], torch.from_numpy(fixed[0]).to(BF16).cuda(), s["out"])
        s["lse"] = torch.where(torch.from_numpy(bad).cuda(), torch.from_numpy(fixed[1]).float().cuda(), s["lse"])
        prefix_check(s)


@pytest.mark.parametrize("power", [-90, -30, 0, 30, 90])
def test_prefix_attention_fp8_magnitudes_of_queries(power):
    """Queries of any magnitude are split alike: with the scale that brings the scores back the results are the same."""
    rng = np.random.default_rng(31)
    q = torch.from_numpy(rng.standard_normal((4, 8, 128)) * np.exp2(rng.integers(-12, 1, (4, 8, 128)))).to(BF16).cuda()
    q[1, 3] = 0
    s = prefix_case(rng, one(100, [20, 3, 40, 1]), 8, 2, 128, 16, fp8_scales=(0.02, 0.03), q=q * 2.0 ** power, scale=0.1 * 2.0 ** -power)
    prefix_call(s)
    prefix_check(s)


@pytest.mark.parametrize("bs", [4, 128])
def test_prefix_attention_pages_past_32_bits(bs):
    """Pages whose offsets pass 32 bits in bytes and in elements."""
    rng = np.random.default_rng(32)
    Hkv, d = 2, 128
    nb = 2 ** 32 // (Hkv * bs * d) + 64
    cache = torch.empty(nb, Hkv, bs, d, dtype=BF16, device="cuda")
    groups, Hq = one(300, [5, 140, 40], 2), 8
    s = prefix_case(rng, groups, Hq, Hkv, d, bs)
    used = torch.unique(s["table"][(s["table"] >= 0) & (s["table"] < s["k"].shape[0])]).long()
    to = torch.arange(nb - 1, -1, -1, device="cuda")[:s["k"].shape[0]].clone()
    to[::3] = torch.arange(s["k"].shape[0], device="cuda")[::3]  # some of them in front
    big = s["table"].clone()
    inside = (big >= 0) & (big < s["k"].shape[0])
    big[inside] = to[big[inside].long()].to(I32)
    want = s["out"].clone()
    prefix_call(s, out=want, lse=None)
    # (keys and values in one tensor: a cache of one is enough to pass the limit)
    cache[to[used]] = s["k"][used]
    same = want.clone()
    prefix_call(s, v=s["k"], out=want, lse=None)
    prefix_call(s, k=cache, v=cache, table=big, out=same, lse=None)
    assert torch.equal(want.view(torch.int16), same.view(torch.int16)) and int(s["err"]) == 0


def test_prefix_attention_graphs_that_share_a_workspace():
    rng = np.random.default_rng(33)
    cases = [prefix_case(rng, g, 8, 2, 128, 16) for g in (one(300, [5, 1, 40]), one(64, [200, 3] * 5, 2))]
    work = torch.empty(max(c["work"].numel() for c in cases), dtype=U8, device="cuda")
    graphs, want = [], []
    for c in cases:
        prefix_call(c)
        want.append(c["out"].clone())
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            prefix_call(c, work=work)
    for c in cases:
        c["out"].fill_(7.0)
    for _ in range(5):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(c["out"], w) for c, w in zip(cases, want))


def test_arguments_that_are_refused():
    x = torch.zeros(4, 64, device="cuda")
    row = torch.zeros(1, 4, device="cuda")
    ids = torch.zeros(1, 4, dtype=I32, device="cuda")
    for change in (dict(logits=x.half()), dict(logits=x.cpu()), dict(logits=x.t()), dict(scores=row.double()),
                   dict(scores=torch.zeros(1, 3, device="cuda")), dict(parents=ids.long()), dict(tokens=ids[:, :3]),
                   dict(out_scores=torch.zeros(4, 1, device="cuda")), dict(finished=ids), dict(error_word=row)):
        a = dict(logits=x, scores=row, out_scores=row.clone(), parents=ids, tokens=ids.clone(), end_token=1, finished=None,
                 out_finished=None, error_word=None)
        with pytest.raises(ValueError):
            pka.pka_beam_select(**dict(a, **change))
    caches = [torch.zeros(4, 2, 16, device="cuda") for _ in range(2)]
    pka.pka_copy_pages([], ids[0], ids[0].clone())  # (nothing to copy)
    for bad in ([caches[0], caches[1][:, :1]], [caches[0].cpu()], [caches[0].transpose(1, 2)]):
        with pytest.raises(ValueError):
            pka.pka_copy_pages(bad, ids[0], ids[0].clone())
    with pytest.raises(ValueError):
        pka.pka_copy_pages(caches, ids[0], ids[0, :2].clone())
    with pytest.raises(ValueError):
        pka.pka_copy_pages(caches, ids[0].long(), ids[0].long())


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_beam_select_rows_far_apart(dtype):
    """Rows whose offsets pass 32 bits in bytes and in elements."""
    rng = np.random.default_rng(40)
    W, V, stride = 40, 1000, 2 ** 27 - 8 if dtype == BF16 else 2 ** 26 + 4
    store = torch.empty((W - 1) * stride + V, dtype=dtype, device="cuda")
    view = store.as_strided((W, V), (stride, 1))
    view.copy_(torch.from_numpy(rng.standard_normal((W, V)) * 3).to(dtype))
    check_select(view, torch.from_numpy(-rng.random((1, W))).float().cuda(), 20)


def test_beam_select_of_the_largest_vocabulary():
    V = 2 ** 26
    logits = torch.zeros(2, V, dtype=BF16, device="cuda")
    logits[0, V - 1], logits[0, 12345], logits[1, V - 2], logits[1, 0] = 9, 8, 10, 8
    s = select_case(logits, torch.tensor([[0.0, -1.5]], device="cuda"), 5)
    # of equal scores the lower beam's; of a row's equal logits the lower tokens
    assert s["parents"].tolist() == [[0, 1, 0, 1, 0]] and s["tokens"].tolist() == [[V - 1, V - 2, 12345, 0, 0]]
    lse = [math.log(V - 2 + sum(math.exp(x) for x in xs)) for xs in ((9, 8), (10, 8))]
    want = [9 - lse[0], 8.5 - lse[1], 8 - lse[0], 6.5 - lse[1], -lse[0]]
    assert np.abs(f64(s["scores"])[0] - want).max() <= 2.0 ** -20 + 2.0 ** -24 * 20 and int(s["err"]) == 0


def test_calls_without_an_error_word():
    rng = np.random.default_rng(42)
    s = prefix_case(rng, one(40, [20, 3]), 8, 2, 64, 16)
    prefix_call(s)
    want = s["out"].clone()
    prefix_call(s, err=None)
    assert torch.equal(s["out"], want)
    bad = s["table"].clone()
    bad[0, 0] = -1  # (set nowhere, read nowhere)
    prefix_call(s, table=bad, err=None)
    prefix_call(s, prefix=dev([50]), err=None)  # refused
    x = torch.full((1, 8), math.nan, device="cuda")
    out = torch.empty(1, 1, device="cuda")
    ids = dev([[7]]), dev([[7]])
    pka.pka_beam_select(x, torch.zeros(1, 1, device="cuda"), out, *ids)
    assert out.tolist() == [[-math.inf]] and ids[0].tolist() == [[-1]]
    cache = torch.zeros(4, 16, device="cuda")
    pka.pka_copy_pages([cache], dev([9]), dev([0]))
    args = dev([0]), dev([5]), dev([[0]]), 4, dev([0] * 4), dev([0, 1]), dev([1]), dev([7]), dev([7]), dev([[7]]), dev([7]), dev([7])
    pka.pka_fork_pages(*args)  # too long for the table: refused
    assert args[7].tolist() == [1] and args[8].tolist() == [0] and args[10].tolist() == [-1]
    torch.cuda.synchronize()
