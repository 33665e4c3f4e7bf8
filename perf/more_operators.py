"""The operators of a step of beam search and parallel sampling over shared pages, as a program that serves a model calls them.

The requests of a group (the beams of one prompt, the samples of one prompt, the users of one system prompt) hold the
same pages for what they have in common:

  select  the best continuations of each group's beams over the whole vocabulary
  fork    block tables of the chosen beams: pages shared, counted and freed, half-filled last pages copied on write
  copy    the copies of those pages, in the caches of all layers
  prefix  attention of each new token where a group's common tokens are read once for all its requests

Each has a plain form (torch, `own` false) and the framework's calls (`own` true). Sizes follow the repository's
serving workloads: 32 query heads over 4 or 8 key-value heads of 64 or 128 elements, pages of 16 or 64 tokens; the
vocabularies are generic.
"""
import math

import torch

own = False

GOLDEN = 0.6180339887498949
Q_HEADS = 32
END_TOKEN = 2


def listed():
    return [
        # one conversation's four beams
        dict(name="select, 4 beams of one", op="select", groups=1, beams=4, vocab=32000, keep=4, dtype="bf16"),
        # a server's batch of groups, twice the beams kept so that ended ones can be set aside
        dict(name="select, 64 x 4 beams", op="select", groups=64, beams=4, vocab=131072, keep=8, dtype="bf16"),
        # an odd vocabulary, its logits in 32 bits
        dict(name="select, 17 x 5 beams float32", op="select", groups=17, beams=5, vocab=50001, keep=5, dtype="f32"),
        # one conversation's four beams
        dict(name="fork, 4 beams of one", op="fork", groups=1, beams=4, ctx_from=2000, ctx_to=2000, block=16),
        # a server's batch of groups with contexts of all lengths
        dict(name="fork, 64 x 8 beams", op="fork", groups=64, beams=8, ctx_from=500, ctx_to=16384, block=16),
        # the last pages of a few beams
        dict(name="copy, 4 beams, 16 caches", op="copy", rows=4, caches=16, kv_heads=8, dim=128, block=16, fp8=False),
        # those of a batch of groups
        dict(name="copy, 512 beams, 32 caches", op="copy", rows=512, caches=32, kv_heads=4, dim=128, block=16, fp8=False),
        # one conversation's four beams after a long prompt
        dict(name="prefix, 4 beams of one", op="prefix", groups=1, width=4, prefix_from=8192, prefix_to=8192, own_from=1,
             own_to=200, new=1, kv_heads=8, dim=128, block=16, fp8=False),
        # a full batch of users behind one system prompt
        dict(name="prefix, 64 requests of one", op="prefix", groups=1, width=64, prefix_from=16384, prefix_to=16384,
             own_from=16, own_to=2048, new=1, kv_heads=4, dim=128, block=16, fp8=False),
        # a batch of prompts with eight beams each
        dict(name="prefix, 24 x 8 beams", op="prefix", groups=24, width=8, prefix_from=1000, prefix_to=8192, own_from=1,
             own_to=512, new=1, kv_heads=8, dim=128, block=64, fp8=False),
        # drafted tokens of a few samples checked together, heads of 64
        dict(name="prefix, 5 x 7, 3 tokens", op="prefix", groups=5, width=7, prefix_from=300, prefix_to=5000, own_from=3,
             own_to=700, new=3, kv_heads=8, dim=64, block=16, fp8=False),
        # a batch of prompts with four samples each over an 8-bit cache
        dict(name="prefix, 32 x 4 8-bit", op="prefix", groups=32, width=4, prefix_from=2048, prefix_to=16384, own_from=1,
             own_to=1024, new=1, kv_heads=4, dim=128, block=16, fp8=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["select", "fork", "copy", "prefix", "prefix"])
    if op == "select":
        beams = rng.choice([1, 2, 3, 4, 5, 8, 16])
        vocab = _log(rng, 1000, 200000)
        groups = _log(rng, 1, min(200, max(1, 32000000 // (beams * vocab))))
        return dict(op=op, groups=groups, beams=beams, vocab=vocab, keep=rng.choice([1, beams, beams, 2 * beams]),
                    dtype=rng.choice(["bf16", "f32"]))
    if op == "fork":
        beams = rng.choice([2, 3, 4, 8, 16])
        lo = _log(rng, 1, 4000)
        return dict(op=op, groups=_log(rng, 1, 512 // beams), beams=beams, ctx_from=lo, ctx_to=lo + _log(rng, 1, 12000),
                    block=rng.choice([16, 32, 64]))
    if op == "copy":
        return dict(op=op, rows=_log(rng, 2, 400), caches=rng.choice([2, 6, 16, 32]), kv_heads=rng.choice([1, 2, 4]),
                    dim=rng.choice([64, 128]), block=rng.choice([8, 16]), fp8=rng.random() < 0.4)
    fp8 = rng.random() < 0.35
    width = _log(rng, 1, 48)
    groups = _log(rng, 1, max(1, 96 // width))
    longest = min(16384, 400000 // (groups * width))
    lo = _log(rng, 1, longest // 2)
    return dict(op=op, groups=groups, width=width, prefix_from=lo - 1, prefix_to=lo + _log(rng, 1, longest // 2),
                own_from=rng.choice([1, 5, 40]), own_to=40 + _log(rng, 1, 1000), new=rng.choice([1, 1, 1, 2, 5]),
                kv_heads=rng.choice([2, 4, 8, 16]), dim=128 if fp8 else rng.choice([64, 128]),
                block=rng.choice([16, 32, 64, 128]), fp8=fp8)


def _spread(n, lo, hi):
    """n lengths between two bounds, even over their logarithm, the same for every seed."""
    return [min(hi, max(lo, int(round(math.exp(math.log(lo + 1) + ((i + 0.5) * GOLDEN % 1.0)
                                               * (math.log(hi + 1) - math.log(lo + 1))) - 1)))) for i in range(n)]


def _pages(tokens, block):
    return -(-tokens // block)


# ---------------------------------------------------------------- inputs


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return {"select": _prepare_select, "fork": _prepare_fork, "copy": _prepare_copy,
            "prefix": _prepare_prefix}[case["op"]](case, gen)


def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device="cuda")


def _empty(*shape, dtype=torch.int32):
    return torch.zeros(shape, dtype=dtype, device="cuda")


def _normal(gen, *shape, dtype=torch.float32):
    return torch.randn(shape, generator=gen, device="cuda", dtype=dtype)


def _permutation(gen, n):
    return torch.randperm(n, generator=gen, device="cuda").to(torch.int32)


def _cache(gen, fp8, *shape):
    x = _normal(gen, *shape, dtype=torch.bfloat16)
    return (x.float() * 40).to(torch.float8_e4m3fn).view(torch.uint8) if fp8 else x


def _prepare_select(case, gen):
    groups, beams, vocab = case["groups"], case["beams"], case["vocab"]
    # logits of a model: a broad middle and a tail of likely tokens, the same ones for the beams of a group more often
    # than not; ended beams now and then
    logits = _normal(gen, groups, beams, vocab).mul_(1.5)
    logits += _normal(gen, groups, 1, vocab)
    logits[..., :vocab // 50] *= 2
    scores = -(2 + 20 * torch.rand(groups, 1, generator=gen, device="cuda")) - 2 * torch.rand(
        groups, beams, generator=gen, device="cuda")
    finished = (torch.rand(groups, beams, generator=gen, device="cuda") < 0.1).to(torch.uint8)
    kind = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    keep = case["keep"]
    return dict(op="select", logits=logits.view(groups * beams, vocab).to(kind), scores=scores.sort(1, True).values,
                finished=finished, out_scores=_empty(groups, keep, dtype=torch.float32), parents=_empty(groups, keep),
                tokens=_empty(groups, keep), out_finished=_empty(groups, keep, dtype=torch.uint8), error=_empty(1))


def _prepare_fork(case, gen):
    groups, beams, block = case["groups"], case["beams"], case["block"]
    rows = groups * beams
    ctx = _spread(groups, case["ctx_from"], case["ctx_to"])
    held = _ints([_pages(c, block) for c in ctx], torch.int64)
    width = int(held.max()) + 2
    # about half of a group's beams go on, in an order of their own, some of them as several beams
    order = torch.rand(groups, beams, generator=gen, device="cuda").argsort(1)  # the first `stay` of these go on
    stay = max(1, (beams + 1) // 2)
    place = torch.arange(beams, device="cuda").expand(groups, beams)
    chosen = torch.randint(0, stay, (groups, beams), generator=gen, device="cuda")
    rank = torch.where(place < stay, (place + 1) % stay, chosen)
    parent = torch.empty_like(order).scatter_(1, order, order.gather(1, rank))
    # the table that such steps lead to: a beam shares the pages of the one that it comes from, up to its last few
    source = torch.empty_like(order).scatter_(1, order, order.gather(1, torch.where(place < stay, place, (chosen - 1) % stay)))
    row = torch.arange(groups, device="cuda")[:, None] * beams
    column = torch.arange(width, device="cuda")
    ids = torch.arange(rows, device="cuda")[:, None] * width + column
    shared = (row + source).view(rows, 1) * width + column
    lens = held.repeat_interleave(beams)[:, None]
    apart = torch.randint(1, 4, (rows, 1), generator=gen, device="cuda")
    ids = torch.where(column < lens - apart, shared, ids)
    valid = column < lens
    flat = ids[valid]
    found, back = flat.unique(return_inverse=True)
    blocks = beams * sum(_pages(c, block) for c in ctx) + rows + 64  # of which sharing leaves many free
    perm = _permutation(gen, blocks)
    table = perm[torch.arange(rows * width, device="cuda").view(rows, width) % blocks].contiguous()
    table[valid] = perm[back]
    counts = torch.zeros(blocks, dtype=torch.int32, device="cuda")
    counts[perm[:found.numel()].long()] = (torch.bincount(back) - 1).to(torch.int32)
    return dict(op="fork", block=block, parents=(row + parent).view(-1).to(torch.int32).contiguous(),
                lens=(_ints(ctx).repeat_interleave(beams), _empty(rows)), tables=(table, table.clone()), counts=counts,
                free=perm, head=_ints([found.numel()]), src=_empty(rows), dst=_empty(rows), error=_empty(1))


def _prepare_copy(case, gen):
    rows, blocks = case["rows"], 2 * case["rows"] + 5
    # the keys' and the values' caches of all layers, from one allocation
    pool = _cache(gen, case["fp8"], case["caches"], blocks, case["kv_heads"], case["block"], case["dim"])
    perm = _permutation(gen, blocks)
    # half of the rows go on in their own pages
    kept = torch.rand(rows, generator=gen, device="cuda") < 0.5
    return dict(op="copy", pool=pool, caches=list(pool.unbind(0)), src=perm[:rows].masked_fill(kept, -1),
                dst=perm[rows:2 * rows].masked_fill(kept, -1), fp8=case["fp8"], error=_empty(1))


def _lengths(case):
    """Each group's common tokens, and each request's own ones (the new ones among them)."""
    prefix = _spread(case["groups"], case["prefix_from"], case["prefix_to"])
    mine = _spread(case["groups"] * case["width"], case["own_from"], case["own_to"])
    return prefix, [max(m, case["new"]) for m in mine]


def _prepare_prefix(case, gen):
    groups, width, block, new = case["groups"], case["width"], case["block"], case["new"]
    hkv, dim, reqs = case["kv_heads"], case["dim"], groups * width
    prefix, mine = _lengths(case)
    seq = [prefix[i // width] + m for i, m in enumerate(mine)]
    columns = _pages(max(seq), block)
    # whole pages of the common tokens are held by all of a group's requests, the rest by each its own
    column = torch.arange(columns, device="cuda")
    common = _ints([p // block for p in prefix], torch.int64).repeat_interleave(width)[:, None]
    first = torch.arange(reqs, device="cuda")[:, None] // width * width
    ids = torch.where(column < common, first, torch.arange(reqs, device="cuda")[:, None]) * columns + column
    valid = column < _ints([_pages(s, block) for s in seq], torch.int64)[:, None]
    found, back = ids[valid].unique(return_inverse=True)
    blocks = found.numel() + 3
    perm = _permutation(gen, blocks)
    table = _empty(reqs, columns)
    table[valid] = perm[back]
    k_cache, v_cache = (_cache(gen, case["fp8"], blocks, hkv, block, dim) for _ in range(2))
    # a common token in a page that is not whole: each request holds a copy
    rest = _ints(prefix, torch.int64) % block
    page = torch.arange(groups, device="cuda") * width
    where = _ints(prefix, torch.int64) // block
    lead = table[page, where.clamp(max=columns - 1)].long().repeat_interleave(width)
    copy = table[torch.arange(reqs, device="cuda"), where.clamp(max=columns - 1).repeat_interleave(width)].long()
    mask = (torch.arange(block, device="cuda") < rest.repeat_interleave(width)[:, None])[:, None, :, None]
    for cache in (k_cache, v_cache):
        cache[copy] = torch.where(mask, cache[lead], cache[copy])
    tokens = reqs * new
    q = (_normal(gen, tokens, Q_HEADS, dim) * (1 + torch.rand(Q_HEADS, 1, generator=gen, device="cuda"))).to(torch.bfloat16)
    return dict(op="prefix", q=q, k_cache=k_cache, v_cache=v_cache, table=table, seq=_ints(seq),
                qsl=_ints([i * new for i in range(reqs + 1)]), starts=_ints([i * width for i in range(groups + 1)]),
                prefix=_ints(prefix), new=new, block=block, longest=max(seq), scale=1 / math.sqrt(dim),
                scales=(1 / 40, 1 / 40) if case["fp8"] else None, out=torch.empty_like(q),
                lse=_empty(tokens, Q_HEADS, dtype=torch.float32), error=_empty(1),
                work=torch.empty(0, dtype=torch.uint8, device="cuda"))  # scratch, of the size that the call asks for


# ---------------------------------------------------------------- one pass


def run(state):
    return {"select": _run_select, "fork": _run_fork, "copy": _run_copy, "prefix": _run_prefix}[state["op"]](state)


def _run_select(s):
    names = ("out_scores", "parents", "tokens", "out_finished")
    if own:
        from paged_kv_attention_07_gb300 import pka
        pka.pka_beam_select(s["logits"], s["scores"], s["out_scores"], s["parents"], s["tokens"], END_TOKEN,
                            s["finished"], s["out_finished"], error_word=s["error"])
        return {n: s[n] for n in names}
    groups, beams = s["scores"].shape
    keep, vocab = s["tokens"].shape[1], s["logits"].shape[1]
    # 64 bits: what is kept hangs on differences that 32 bits would lose
    x = s["logits"].double().view(groups, beams, vocab)
    largest = x.amax(2, keepdim=True)
    total = (x - largest).exp().sum(2, keepdim=True)
    score = s["scores"].double()[..., None] + (x - (largest + total.log()))
    ended = s["finished"].bool()[..., None]
    only = torch.where(torch.arange(vocab, device="cuda") == END_TOKEN, s["scores"].double()[..., None], -math.inf)
    score = torch.where(ended, only, score)
    best = score.view(groups, -1).sort(dim=1, descending=True, stable=True)
    value, index = best.values[:, :keep], best.indices[:, :keep]
    beam, token = index // vocab, index % vocab
    over = s["finished"].bool().gather(1, beam) | (token == END_TOKEN)
    row = torch.arange(groups, device="cuda")[:, None] * beams + beam
    none = value == -math.inf
    return dict(out_scores=value.float(), parents=row.masked_fill(none, -1).to(torch.int32),
                tokens=token.masked_fill(none, -1).to(torch.int32), out_finished=(over & ~none).to(torch.uint8))


def _run_fork(s):
    # the step's tables are read, the next step's written; the next step reads those
    (lens, lens_out), (table, table_out) = s["lens"], s["tables"]
    s["lens"], s["tables"] = (lens_out, lens), (table_out, table)
    if own:
        from paged_kv_attention_07_gb300 import pka
        pka.pka_fork_pages(s["parents"], lens, table, s["block"], s["counts"], s["free"], s["head"], s["head"], lens_out,
                           table_out, s["src"], s["dst"], error_word=s["error"])
    else:
        rows, width, block = table.shape[0], table.shape[1], s["block"]
        parent = s["parents"].long()
        children = torch.bincount(parent, minlength=rows)
        child = torch.arange(rows, device="cuda")
        first = torch.full((rows,), rows, device="cuda").scatter_reduce_(0, parent, child, "amin")
        held = (lens.long() + block - 1) // block
        partial = lens % block != 0
        column = torch.arange(width, device="cuda")
        # children after a parent's first take a page each for its half-filled last page
        fresh = partial[parent] & (first[parent] != child)
        head = s["head"].long()
        page = s["free"][(head + fresh.cumsum(0) - 1).clamp(0, s["free"].numel() - 1)]
        mine = table[parent]
        tail = (column == held[parent][:, None] - 1) & fresh[:, None]
        s["src"].copy_(torch.where(fresh, mine.gather(1, (held[parent] - 1).clamp(min=0)[:, None]).squeeze(1), -1))
        s["dst"].copy_(torch.where(fresh, page, -1))
        lens_out.copy_(lens[parent])
        table_out.copy_(torch.where(column < held[parent][:, None], torch.where(tail, page[:, None], mine), table_out))
        # who holds each page now
        last = (column == held[:, None] - 1) & partial[:, None]
        more = torch.where(last, children[:, None].clamp(max=1), children[:, None]) - 1
        inside = column < held[:, None]
        at = table[inside].long()
        s["counts"].index_add_(0, at, more[inside].to(torch.int32))
        # pages that nobody holds go back, in the order of their first places in the table
        place = torch.arange(at.numel(), device="cuda")
        earliest = torch.full_like(s["counts"], at.numel(), dtype=torch.int64).scatter_reduce_(0, at, place, "amin")
        back = at[(s["counts"][at] < 0) & (earliest[at] == place)]
        s["counts"].clamp_(min=0)
        end = head + fresh.sum()
        s["free"][end - back.numel() + torch.arange(back.numel(), device="cuda")] = back.to(torch.int32)
        s["head"].copy_(end - back.numel())
    return dict(lens=lens_out, table=table_out, counts=s["counts"], free=s["free"], head=s["head"], src=s["src"],
                dst=s["dst"])


def _run_copy(s):
    if own:
        from paged_kv_attention_07_gb300 import pka
        pka.pka_copy_pages(s["caches"], s["src"], s["dst"], error_word=s["error"])
    else:
        wanted = s["src"] >= 0
        src, dst = s["src"][wanted].long(), s["dst"][wanted].long()
        s["pool"][:, dst] = s["pool"][:, src]
    return s["pool"].view(torch.float8_e4m3fn) if s["fp8"] else s["pool"]


def _run_prefix(s):
    if own:
        from paged_kv_attention_07_gb300 import pka
        if not s["work"].numel():  # once, for the largest step
            tokens, heads, dim = s["q"].shape
            size = pka.pka_prefix_workspace_size(s["seq"].numel(), s["prefix"].numel(), tokens, heads,
                                                 s["k_cache"].shape[1], dim, s["new"])
            s["work"] = torch.empty(size, dtype=torch.uint8, device="cuda")
        pka.pka_prefix_attn_forward(s["q"], s["k_cache"], s["v_cache"], s["table"], s["qsl"], s["seq"], s["starts"],
                                    s["prefix"], s["scale"], s["new"], s["longest"], s["out"], s["lse"], s["work"],
                                    kv_scales=s["scales"], error_word=s["error"])
        return dict(out=s["out"], lse=s["lse"])
    tokens, heads, dim = s["q"].shape
    reqs, columns = s["table"].shape
    hkv, block, new = s["k_cache"].shape[1], s["block"], s["new"]

    def rows(cache):
        x = cache.view(torch.float8_e4m3fn) if s["scales"] else cache
        x = x.view(torch.uint8 if s["scales"] else torch.bfloat16)[s["table"].long()].view(x.dtype)
        return x.float().transpose(1, 2).reshape(reqs, hkv, columns * block, dim)

    keys, values = rows(s["k_cache"]), rows(s["v_cache"])
    # a request's new tokens, each with the heads of a key-value head
    q = s["q"].float().view(reqs, new, hkv, heads // hkv, dim).permute(0, 2, 1, 3, 4)
    score = torch.matmul(q.reshape(reqs, hkv, -1, dim), keys.transpose(2, 3))
    score = score.view(reqs, hkv, new, heads // hkv, -1) * (s["scale"] * (s["scales"][0] if s["scales"] else 1.0))
    position = (s["seq"] - new)[:, None] + torch.arange(new, device="cuda")
    key = torch.arange(columns * block, device="cuda")
    score = score.masked_fill((key > position[..., None])[:, None, :, None], -math.inf)
    largest = score.amax(-1, keepdim=True)
    weight = (score - largest).exp()
    total = weight.sum(-1, keepdim=True)
    values = values.masked_fill((key >= s["seq"][:, None])[:, None, :, None], 0)
    out = torch.matmul(weight.flatten(2, 3), values).view(reqs, hkv, new, heads // hkv, dim) / total
    out = out * (s["scales"][1] if s["scales"] else 1.0)
    lse = (total.log() + largest).squeeze(-1)
    return dict(out=out.permute(0, 2, 1, 3, 4).reshape(tokens, heads, dim).to(torch.bfloat16),
                lse=lse.permute(0, 2, 1, 3).reshape(tokens, heads))


# ---------------------------------------------------------------- what a pass cannot do without


def work(case):
    op = case["op"]
    if op == "select":
        rows = case["groups"] * case["beams"]
        size = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": rows * (case["vocab"] * size + 5) + case["groups"] * case["keep"] * 13,
                "flops": rows * case["vocab"] * 4}
    if op == "fork":
        held = [_pages(c, case["block"]) for c in _spread(case["groups"], case["ctx_from"], case["ctx_to"])]
        rows = case["groups"] * case["beams"]
        return {"bytes": 8 * case["beams"] * sum(held) + 20 * rows, "flops": case["beams"] * sum(held)}
    if op == "copy":
        page = case["kv_heads"] * case["block"] * case["dim"] * (1 if case["fp8"] else 2)
        return {"bytes": case["rows"] / 2 * case["caches"] * page * 2 + 8 * case["rows"], "flops": 0}
    prefix, mine = _lengths(case)
    hkv, dim, new = case["kv_heads"], case["dim"], case["new"]
    tokens = new * case["groups"] * case["width"]
    seen = sum((prefix[i // case["width"]] + m) * new - new * (new - 1) // 2 for i, m in enumerate(mine))
    size = 2 * hkv * dim * (1 if case["fp8"] else 2)
    return {"bytes": (sum(prefix) + sum(mine)) * size + tokens * (4 * Q_HEADS * dim + 4 * Q_HEADS),
            "flops": 4 * seen * Q_HEADS * dim}


# ---------------------------------------------------------------- the definitions, in 64 bits


def exact(case, seed):
    if case["op"] == "select":
        return _exact_select(prepare(case, seed))
    if case["op"] == "prefix":
        return _exact_prefix(prepare(case, seed))
    if case["op"] == "copy":
        return _exact_copy(prepare(case, seed))
    return None  # tables, counts and lists of pages are whole numbers, equal or wrong


def _exact_select(s):
    logp = s["logits"].double().log_softmax(1) + s["scores"].double().view(-1, 1)
    done = s["finished"].view(-1) != 0
    logp[done] = -math.inf
    logp[done, END_TOKEN] = s["scores"].double().view(-1)[done]
    groups, keep = s["tokens"].shape
    return dict(out_scores=logp.view(groups, -1).topk(keep, 1).values, parents=None, tokens=None, out_finished=None)


def _exact_copy(s):
    pool = s["pool"].view(torch.float8_e4m3fn) if s["fp8"] else s["pool"]
    source = torch.arange(pool.shape[1], device="cuda")
    source[s["dst"][s["dst"] >= 0].long()] = s["src"][s["src"] >= 0].long()
    return pool.double().index_select(1, source)


def _exact_prefix(s):
    tokens, heads, dim = s["q"].shape
    hkv, block = s["k_cache"].shape[1], s["block"]
    unit = s["scales"] or (1.0, 1.0)
    out = torch.empty(tokens, heads, dim, dtype=torch.float64, device="cuda")
    lse = torch.empty(tokens, heads, dtype=torch.float64, device="cuda")
    for r, (n, t) in enumerate(zip(s["seq"].tolist(), s["qsl"].tolist())):
        pages = s["table"][r, :_pages(n, block)].long()

        def of(cache):
            x = cache.index_select(0, pages)
            x = x.view(torch.float8_e4m3fn) if s["scales"] else x
            return x.double().permute(1, 0, 2, 3).flatten(1, 2)[:, :n]

        q = s["q"][t:t + s["new"]].double().unflatten(1, (hkv, -1))
        logit = torch.einsum("thgd,hnd->thgn", q, of(s["k_cache"])) * (s["scale"] * unit[0])
        hidden = torch.ones(s["new"], n, dtype=torch.bool, device="cuda").triu(n - s["new"] + 1)
        logit[hidden[:, None, None].expand_as(logit)] = -math.inf
        out[t:t + s["new"]] = (torch.einsum("thgn,hnd->thgd", logit.softmax(-1), of(s["v_cache"])) * unit[1]).flatten(1, 2)
        lse[t:t + s["new"]] = logit.logsumexp(-1).flatten(1, 2)
    return dict(out=out, lse=lse)
