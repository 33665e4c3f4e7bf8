"""The operators of the block-sparse serving step, as a program that serves a model calls them.

One step over a paged cache whose contexts are too long to read in full:

  tables   the step's block tables, slot map and positions, made on the GPU from the requests' lengths
  rope     norms of each query and key head, the position rotation and the cache write, in one pass
  bounds   element-wise bounds of the keys of each page that the step filled, as 8-bit codes
  select   the pages that each new token reads, by an upper bound of its scores over each page
  attn     attention of each new token over the pages that were selected for it

Each has a plain form (torch, `own` false) and the framework's calls (`own` true). Sizes follow the
repository's serving workloads: 32 query heads over 4 or 8 key-value heads of 64 or 128 elements, pages
of 16 or 64 tokens, contexts of a thousand to some hundred thousand tokens.
"""
import math

import torch

own = False

GOLDEN = 0.6180339887498949
Q_HEADS = 32
MAX_POSITION = 131072
FIRST, LAST = 1, 2  # pages that are always read: where attention sinks lie, and the newest


def listed():
    return [
        # every decode step of a small server: one new token per request
        dict(name="tables, 48 decodes", op="tables", reqs=48, ctx_from=500, ctx_to=8192, new_from=1, new_to=1, block=16),
        # a step that also takes in long prompts: 300 requests, some of them with hundreds of new tokens
        dict(name="tables, 300 requests", op="tables", reqs=300, ctx_from=0, ctx_to=65536, new_from=1, new_to=1500, block=64),
        # a decode step: the new token of each of 64 requests
        dict(name="rope, 64 decodes", op="rope", tokens=64, kv_heads=4, dim=128, block=16, rotary=128,
             interleaved=False, norm=True, fp8=False, decode=True),
        # a long prompt's chunk, its keys and values also kept for the attention among themselves
        dict(name="rope, 8192 tokens", op="rope", tokens=8192, kv_heads=8, dim=128, block=64, rotary=128,
             interleaved=False, norm=True, fp8=False, decode=False),
        # an odd chunk into an 8-bit cache, half of each head rotated in neighbouring pairs, no norms
        dict(name="rope, 5003 tokens 8-bit", op="rope", tokens=5003, kv_heads=4, dim=128, block=16, rotary=64,
             interleaved=True, norm=False, fp8=True, decode=False),
        # a prompt's chunk fills whole pages
        dict(name="bounds, 16384 tokens", op="bounds", tokens=16384, kv_heads=4, dim=128, block=64, fp8=False,
             decode=False),
        # a decode step over an 8-bit cache: one request in sixteen fills a page
        dict(name="bounds, 256 decodes 8-bit", op="bounds", tokens=256, kv_heads=4, dim=128, block=16, fp8=True,
             decode=True),
        # one long conversation
        dict(name="select, 131072 of one", op="select", reqs=1, ctx_from=131071, ctx_to=131071, new=1, kv_heads=8, dim=128,
             block=64, pages=64),
        # a full batch of contexts of all lengths
        dict(name="select, 96 requests", op="select", reqs=96, ctx_from=4096, ctx_to=65536, new=1, kv_heads=8, dim=128,
             block=64, pages=64),
        # one long conversation
        dict(name="attn, 131072 of one", op="attn", reqs=1, ctx_from=131071, ctx_to=131071, new=1, kv_heads=8, dim=128,
             block=64, pages=64, fp8=False),
        # a full batch
        dict(name="attn, 96 requests", op="attn", reqs=96, ctx_from=4096, ctx_to=65536, new=1, kv_heads=4, dim=128, block=64,
             pages=64, fp8=False),
        # four drafted tokens of each request checked together, small pages of an 8-bit cache
        dict(name="attn, 24 x 4 tokens 8-bit", op="attn", reqs=24, ctx_from=2048, ctx_to=32768, new=4, kv_heads=4, dim=128,
             block=16, pages=128, fp8=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "rope", "bounds", "select", "attn"])
    block = rng.choice([16, 32, 64, 128])
    kv_heads = rng.choice([2, 4, 8, 16])
    dim = rng.choice([64, 128])
    if op == "tables":
        hi = _log(rng, 1, 1500)
        return dict(op=op, reqs=_log(rng, 1, 300), ctx_from=rng.choice([0, 1, 37]), ctx_to=_log(rng, 100, 65536),
                    new_from=1, new_to=hi, block=block)
    if op == "rope":
        interleaved = rng.random() < 0.5
        return dict(op=op, tokens=_log(rng, 1, 8192), kv_heads=rng.choice([2, 4, 8]), dim=dim, block=block,
                    rotary=rng.choice([dim, dim // 2, dim // 4]), interleaved=interleaved, norm=rng.random() < 0.7,
                    fp8=rng.random() < 0.4, decode=rng.random() < 0.4)
    if op == "bounds":
        decode = rng.random() < 0.4
        return dict(op=op, tokens=_log(rng, 1, 512) if decode else _log(rng, block, 16384),
                    kv_heads=rng.choice([2, 4]), dim=dim, block=block, fp8=rng.random() < 0.4, decode=decode)
    block = rng.choice([16, 32, 64])
    reqs = _log(rng, 1, 64)
    top = 262144 if reqs < 5 else 32768
    pages = rng.choice([8, 16, 31, 48, 64])
    lo = _log(rng, 1, 2000)
    hi = lo + _log(rng, 1, top * block // 64)
    if op == "select":  # contexts that are longer than the pages read of them, at least some
        lo = lo if reqs > 3 else 2 * pages * block + lo
        hi = max(hi, lo + 3 * pages * block)
        return dict(op=op, reqs=reqs, ctx_from=lo, ctx_to=hi, new=rng.choice([1, 1, 2, 3]), kv_heads=kv_heads,
                    dim=dim, block=block, pages=pages)
    fp8 = rng.random() < 0.4
    return dict(op=op, reqs=reqs, ctx_from=lo, ctx_to=hi, new=rng.choice([1, 1, 2, 4]), kv_heads=rng.choice([2, 4]),
                dim=128 if fp8 else dim, block=block, pages=pages, fp8=fp8)


def _spread(n, lo, hi):
    """n lengths between two bounds, even over their logarithm, the same for every seed."""
    return [min(hi, max(lo, int(round(math.exp(math.log(lo + 1) + ((i + 0.5) * GOLDEN % 1.0)
                                               * (math.log(hi + 1) - math.log(lo + 1))) - 1)))) for i in range(n)]


def _contexts(case):
    return _spread(case["reqs"], case["ctx_from"], case["ctx_to"])


def _news(case):
    return _spread(case["reqs"], case["new_from"], case["new_to"])[::-1]


def _pages(tokens, block):
    return -(-tokens // block)


# ---------------------------------------------------------------- inputs


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return {"tables": _prepare_tables, "rope": _prepare_rope, "bounds": _prepare_bounds, "select": _prepare_select,
            "attn": _prepare_attn}[case["op"]](case, gen)


def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device="cuda")


def _normal(gen, *shape, dtype=torch.float32):
    return torch.randn(shape, generator=gen, device="cuda", dtype=dtype)


def _permutation(gen, n):
    return torch.randperm(n, generator=gen, device="cuda").to(torch.int32)


def _prepare_tables(case, gen):
    ctx = _contexts(case)
    new = _news(case)
    block, reqs = case["block"], case["reqs"]
    width = max(_pages(c + n, block) for c, n in zip(ctx, new)) + 3
    held = [_pages(c, block) for c in ctx]
    taken = sum(_pages(c + n, block) - h for c, n, h in zip(ctx, new, held))
    perm = _permutation(gen, sum(held) + taken + 100)
    # the pages that the requests hold already, the rest of each row as an earlier request left it
    index = torch.arange(reqs * width, device="cuda").view(reqs, width) % perm.numel()
    table = perm[index].contiguous()
    tokens = -(-sum(new) // 64) * 64  # a captured step is padded to a whole number of rows
    empty = lambda *s, dtype=torch.int32: torch.zeros(s, dtype=dtype, device="cuda")  # noqa: E731
    return dict(op="tables", block=block, tokens=tokens, ctx=_ints(ctx), new=_ints(new), table=table, free=perm,
                head=_ints([sum(held)]), head_out=empty(1), qsl=empty(reqs + 1), seq=empty(reqs),
                positions=empty(tokens), slots=empty(tokens, dtype=torch.int64), error=empty(1))


def _rotation(rotary):
    """Cosines and sines of every position, the angles formed in 64 bits."""
    inv = 500000.0 ** (-torch.arange(0, rotary, 2, device="cuda", dtype=torch.float64) / rotary)
    angle = torch.arange(MAX_POSITION, device="cuda", dtype=torch.float64)[:, None] * inv
    return torch.cat([angle.cos(), angle.sin()], 1).to(torch.float32)


def _slots(case, gen, blocks):
    """Where the new tokens go: whole runs of pages for a prompt, one place in a page of its own for a decode."""
    t = torch.arange(case["tokens"], device="cuda")
    perm = _permutation(gen, blocks).long()
    if case["decode"]:
        offset = torch.randint(0, case["block"], (case["tokens"],), generator=gen, device="cuda")
        return perm[t] * case["block"] + offset
    return perm[t // case["block"]] * case["block"] + t % case["block"]


def _blocks(case):
    return case["tokens"] + 7 if case["decode"] else _pages(case["tokens"], case["block"]) + 7


def _cache(gen, fp8, *shape):
    x = _normal(gen, *shape, dtype=torch.bfloat16)
    return (x.float() * 40).to(torch.float8_e4m3fn).view(torch.uint8) if fp8 else x


def _prepare_rope(case, gen):
    tokens, hkv, dim, block = case["tokens"], case["kv_heads"], case["dim"], case["block"]
    channel = (0.5 * _normal(gen, Q_HEADS + 2 * hkv, dim)).exp()
    qkv = (_normal(gen, tokens, Q_HEADS + 2 * hkv, dim) * channel).to(torch.bfloat16)
    q, k, v = qkv[:, :Q_HEADS], qkv[:, Q_HEADS:Q_HEADS + hkv], qkv[:, Q_HEADS + hkv:]
    weight = lambda: (1 + 0.2 * _normal(gen, dim)).to(torch.bfloat16) if case["norm"] else None  # noqa: E731
    start = int(torch.randint(0, MAX_POSITION - tokens, (1,), generator=gen, device="cuda"))
    positions = torch.arange(start, start + tokens, device="cuda", dtype=torch.int32)
    if case["decode"]:
        positions = torch.randint(0, MAX_POSITION, (tokens,), generator=gen, device="cuda", dtype=torch.int32)
    blocks = _blocks(case)
    out = lambda h: torch.empty(tokens, h, dim, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    keep = not case["decode"]
    return dict(op="rope", q=q, k=k, v=v, q_weight=weight(), k_weight=weight(), eps=1e-6,
                cos_sin=_rotation(case["rotary"]), interleaved=case["interleaved"], positions=positions,
                slots=_slots(case, gen, blocks), q_out=out(Q_HEADS), k_out=out(hkv) if keep else None,
                v_out=out(hkv) if keep else None, k_cache=_cache(gen, case["fp8"], blocks, hkv, block, dim),
                v_cache=_cache(gen, case["fp8"], blocks, hkv, block, dim),
                scales=(0.03125, 0.05) if case["fp8"] else None, error=torch.zeros(1, dtype=torch.int32, device="cuda"))


def _prepare_bounds(case, gen):
    hkv, dim, block, blocks = case["kv_heads"], case["dim"], case["block"], _blocks(case)
    # keys of a page lie around a common point, some channels far larger than others
    shape = (blocks, hkv, block, dim)
    keys = _normal(gen, *shape, dtype=torch.bfloat16)
    keys += 2 * _normal(gen, blocks, hkv, 1, dim, dtype=torch.bfloat16)
    keys *= (0.7 * _normal(gen, hkv, 1, dim)).exp().to(torch.bfloat16)
    if case["fp8"]:
        keys = (keys.float() * 10).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return dict(op="bounds", keys=keys, slots=_slots(case, gen, blocks),
                codes=torch.randint(-127, 128, (blocks, hkv, 2, dim), generator=gen, device="cuda", dtype=torch.int8),
                scales=torch.ones(blocks, hkv, device="cuda"), error=torch.zeros(1, dtype=torch.int32, device="cuda"))


def _batch(case, gen):
    """Requests of one step: their lengths, the pages of each, and its new tokens."""
    ctx, new, block = _contexts(case), case["new"], case["block"]
    seq = [c + new for c in ctx]
    width = _pages(max(seq), block)
    count = [_pages(s, block) for s in seq]
    blocks = sum(count) + 3
    first = [sum(count[:i]) for i in range(len(count))]
    perm = _permutation(gen, blocks)
    index = _ints(first, torch.int64)[:, None] + torch.arange(width, device="cuda")
    table = perm[index.clamp(max=blocks - 1)].contiguous()
    return dict(table=table, seq=_ints(seq), qsl=_ints([i * new for i in range(len(seq) + 1)]), blocks=blocks,
                block=block, longest=max(seq), tokens=len(seq) * new,
                error=torch.zeros(1, dtype=torch.int32, device="cuda"))


def _prepare_select(case, gen):
    s = _batch(case, gen)
    hkv, dim, tokens = case["kv_heads"], case["dim"], s["tokens"]
    middle = 35 * _normal(gen, s["blocks"], hkv, 1, dim, dtype=torch.bfloat16).float()
    width = (25 + 8 * _normal(gen, s["blocks"], hkv, 1, dim, dtype=torch.bfloat16).float()).abs()
    codes = torch.cat([middle - width, middle + width], 2).round_().clamp_(-127, 127).to(torch.int8)
    power = torch.randint(-6, -3, (s["blocks"], hkv), generator=gen, device="cuda").float()
    q = (_normal(gen, tokens, Q_HEADS, dim) * (0.5 * _normal(gen, Q_HEADS, 1)).exp()).to(torch.bfloat16)
    return dict(s, op="select", q=q, codes=codes, scales=power.exp2(), pages=case["pages"],
                selected=torch.full((tokens, hkv, case["pages"]), -1, dtype=torch.int32, device="cuda"))


def _prepare_attn(case, gen):
    s = _batch(case, gen)
    hkv, dim, tokens, block = case["kv_heads"], case["dim"], s["tokens"], s["block"]
    cache = lambda: _cache(gen, case["fp8"], s["blocks"], hkv, block, dim)  # noqa: E731
    # the tokens of one request read the same older pages, and each its own newest page
    row = torch.arange(tokens, device="cuda")
    req = row // case["new"]
    newest = (s["seq"].long()[req] - case["new"] + row % case["new"]) // block
    oldest_newest = (s["seq"].long() - case["new"]) // block
    weight = torch.rand(len(s["seq"]), hkv, s["table"].shape[1], generator=gen, device="cuda")
    weight = weight.masked_fill(torch.arange(weight.shape[2], device="cuda") >= oldest_newest[:, None, None], -1.0)
    top = weight.topk(min(case["pages"] - 1, weight.shape[2]), 2)
    older = top.indices.masked_fill(top.values < 0, 1 << 30)[req]
    chosen = torch.cat([older, newest[:, None, None].expand(tokens, hkv, 1)], 2).sort(2).values
    chosen = torch.nn.functional.pad(chosen.masked_fill(chosen >= 1 << 30, -1), (0, case["pages"] - chosen.shape[2]),
                                     value=-1)
    q = _normal(gen, tokens, Q_HEADS, dim, dtype=torch.bfloat16)
    return dict(s, op="attn", q=q, k_cache=cache(), v_cache=cache(), selected=chosen.to(torch.int32).contiguous(),
                scale=1 / math.sqrt(dim), scales=(1 / 40, 1 / 40) if case["fp8"] else None,
                out=torch.empty(tokens, Q_HEADS, dim, dtype=torch.bfloat16, device="cuda"),
                lse=torch.empty(tokens, Q_HEADS, device="cuda"))


# ---------------------------------------------------------------- one pass


def run(state):
    return {"tables": _run_tables, "rope": _run_rope, "bounds": _run_bounds, "select": _run_select,
            "attn": _run_attn}[state["op"]](state)


def _run_tables(s):
    if own:
        from paged_kv_attention_07_gb300 import pka
        pka.pka_step_tables(s["ctx"], s["new"], s["table"], s["block"], s["free"], s["head"], s["head_out"], s["qsl"],
                            s["seq"], s["positions"], s["slots"], error_word=s["error"])
        return dict(table=s["table"], head=s["head_out"], qsl=s["qsl"], seq=s["seq"], positions=s["positions"],
                    slots=s["slots"])
    ctx, new, block = s["ctx"].long(), s["new"].long(), s["block"]
    seq = ctx + new
    held, pages = (ctx + block - 1) // block, (seq + block - 1) // block
    need = pages - held
    first = need.cumsum(0) - need
    column = torch.arange(s["table"].shape[1], device="cuda")
    fresh = (column >= held[:, None]) & (column < pages[:, None])
    source = s["head"].long() + first[:, None] + column - held[:, None]
    table = torch.where(fresh, s["free"][source.clamp(0, s["free"].numel() - 1)], s["table"])
    ends = new.cumsum(0)
    token = torch.arange(s["tokens"], device="cuda")
    req = torch.searchsorted(ends, token, right=True).clamp(max=new.numel() - 1)
    position = ctx[req] + token - (ends - new)[req]
    real = token < ends[-1]
    position = torch.where(real, position, -1)
    slot = table[req, position.clamp(min=0) // block].long() * block + position % block
    return dict(table=table, head=(s["head"] + need.sum()).to(torch.int32),
                qsl=torch.cat([torch.zeros_like(ends[:1]), ends]).to(torch.int32), seq=seq.to(torch.int32),
                positions=position.to(torch.int32), slots=torch.where(real, slot, -1))


def _rotate(x, c, s, interleaved):
    half = c.shape[-1]
    turned, rest = x[..., :2 * half], x[..., 2 * half:]
    a, b = (turned[..., 0::2], turned[..., 1::2]) if interleaved else (turned[..., :half], turned[..., half:])
    p, q = a * c - b * s, b * c + a * s
    return torch.cat([torch.stack([p, q], -1).flatten(-2) if interleaved else torch.cat([p, q], -1), rest], -1)


def _run_rope(s):
    if own:
        from paged_kv_attention_07_gb300 import pka
        pka.pka_qk_rope_cache_write(s["q"], s["k"], s["v"], s["q_weight"], s["k_weight"], s["eps"], s["cos_sin"],
                                    s["interleaved"], s["positions"], s["slots"], s["q_out"], s["k_out"], s["v_out"],
                                    s["k_cache"], s["v_cache"], kv_scales=s["scales"], error_word=s["error"])
        return _rope_outputs(s, s["q_out"], s["k_out"], s["v_out"])
    angles = s["cos_sin"][s["positions"].long()][:, None]
    cos, sin = angles.chunk(2, -1)

    def head(x, weight):
        x = x.float()
        if weight is not None:
            x = x / (x.square().mean(-1, keepdim=True) + s["eps"]).sqrt() * weight.float()
        return _rotate(x, cos, sin, s["interleaved"])

    q, k, v = head(s["q"], s["q_weight"]), head(s["k"], s["k_weight"]), s["v"].float()
    block = s["k_cache"].shape[2]
    page, offset = s["slots"] // block, s["slots"] % block
    for cache, x, n in ((s["k_cache"], k, 0), (s["v_cache"], v, 1)):
        if s["scales"]:
            code = (x / torch.full_like(x, s["scales"][n])).clamp(-448, 448).to(torch.float8_e4m3fn)
            cache[page, :, offset] = code.view(torch.uint8)
        else:
            cache[page, :, offset] = x.to(torch.bfloat16)
    keep = s["k_out"] is not None
    return _rope_outputs(s, q.to(torch.bfloat16), k.to(torch.bfloat16) if keep else None,
                         s["v"].contiguous() if keep else None)


def _rope_outputs(s, q, k, v):
    kind = torch.float8_e4m3fn if s["scales"] else torch.bfloat16
    return dict(q=q, k=k, v=v, k_cache=s["k_cache"].view(kind), v_cache=s["v_cache"].view(kind))


def _run_bounds(s):
    if own:
        from paged_kv_attention_07_gb300 import pka
        pka.pka_page_bounds(s["keys"], s["slots"], s["codes"], s["scales"], error_word=s["error"])
        return dict(codes=s["codes"], scales=s["scales"])
    block = s["keys"].shape[2]
    page = s["slots"][s["slots"] % block == block - 1] // block  # the pages whose last place was just written
    keys = s["keys"][page]
    keys = (keys.view(torch.float8_e4m3fn) if keys.dtype == torch.uint8 else keys).float()
    low, high = keys.amin(2), keys.amax(2)
    largest = torch.maximum(-low, high).amax(-1)
    # the least power of two that brings the largest magnitude to 127 at most
    power = torch.frexp(largest)[1] - 7
    power = torch.where(torch.ldexp(largest, -power) > 127, power + 1, power).clamp(min=-60)
    power = torch.where(largest == 0, -60, power)
    scale = torch.ldexp(torch.ones_like(largest), power)
    unit = scale[..., None]
    s["codes"][page] = torch.stack([(low / unit).floor(), (high / unit).ceil()], 2).to(torch.int8)
    s["scales"][page] = scale
    return dict(codes=s["codes"], scales=s["scales"])


def _positions(s):
    """The request and the position of each new token."""
    row = torch.arange(s["tokens"], device="cuda")
    req = torch.searchsorted(s["qsl"][1:].long(), row, right=True)
    return req, s["seq"].long()[req] - s["qsl"].long()[req + 1] + row


def _run_select(s):
    if own:
        from paged_kv_attention_07_gb300 import pka
        pka.pka_select_pages(s["q"], s["codes"], s["scales"], s["table"], s["qsl"], s["seq"], s["block"], FIRST, LAST,
                             s["longest"], s["selected"], error_word=s["error"])
        return s["selected"]
    tokens, heads, dim = s["q"].shape
    hkv = s["codes"].shape[1]
    req, position = _positions(s)
    count = position // s["block"] + 1
    # 8-bit queries: the power of two that brings each head's largest magnitude to 127 at most
    q = s["q"].float().view(tokens, hkv, heads // hkv, dim)
    largest = q.abs().amax(-1)
    power = torch.frexp(largest)[1] - 7
    power = torch.where(torch.ldexp(largest, -power) > 127, power + 1, power).clamp(min=-60)
    unit = torch.ldexp(torch.ones_like(largest), torch.where(largest == 0, -60, power))
    q = (q / unit[..., None]).round()
    table = s["table"].long()[req]
    codes = s["codes"][table].float()  # tokens, pages, key-value heads, low and high, elements
    bound = torch.einsum("thgd,tnhd->thgn", q.clamp(min=0), codes[:, :, :, 1])
    bound = bound + torch.einsum("thgd,tnhd->thgn", q.clamp(max=0), codes[:, :, :, 0])
    score = (bound * s["scales"][table].transpose(1, 2)[:, :, None] * unit[..., None]).amax(2)
    page = torch.arange(table.shape[1], device="cuda")
    count = count[:, None, None]
    score = score.masked_fill((page < FIRST) | (page >= count - LAST), math.inf).masked_fill(page >= count, -math.inf)
    order = score.sort(dim=-1, descending=True, stable=True).indices[..., :s["selected"].shape[2]]
    order = order.masked_fill(order >= count, 1 << 30).sort(-1).values
    order = torch.nn.functional.pad(order, (0, s["selected"].shape[2] - order.shape[2]), value=1 << 30)
    return order.masked_fill(order == 1 << 30, -1).to(torch.int32)


def _run_attn(s):
    if own:
        from paged_kv_attention_07_gb300 import pka
        pka.pka_sparse_attn_forward(s["q"], s["k_cache"], s["v_cache"], s["table"], s["qsl"], s["seq"], s["selected"],
                                    s["scale"], s["longest"], s["out"], s["lse"], kv_scales=s["scales"],
                                    error_word=s["error"])
        return dict(out=s["out"], lse=s["lse"])
    tokens, heads, dim = s["q"].shape
    hkv = s["k_cache"].shape[1]
    req, position = _positions(s)
    seen, block = s["selected"].long(), s["block"]
    page = s["table"].long()[req[:, None, None], seen.clamp(min=0)]
    head = torch.arange(hkv, device="cuda")[:, None]

    def rows(cache):
        x = cache.view(torch.float8_e4m3fn) if s["scales"] else cache
        return x.view(torch.uint8 if s["scales"] else torch.bfloat16)[page, head].view(x.dtype).float().flatten(2, 3)

    keys, values = rows(s["k_cache"]), rows(s["v_cache"])
    key = seen[..., None] * block + torch.arange(block, device="cuda")
    hidden = ((seen < 0)[..., None] | (key > position[:, None, None, None])).flatten(2)[:, :, None]
    factor = s["scale"] * (s["scales"][0] if s["scales"] else 1.0)
    score = torch.matmul(s["q"].float().view(tokens, hkv, heads // hkv, dim), keys.transpose(2, 3)) * factor
    score = score.masked_fill(hidden, -math.inf)
    largest = score.amax(-1, keepdim=True)
    weight = (score - largest).exp()
    total = weight.sum(-1, keepdim=True)
    out = torch.matmul(weight, values.masked_fill(hidden.squeeze(2)[..., None], 0)) / total
    out = out * (s["scales"][1] if s["scales"] else 1.0)
    lse = (total.log() + largest).squeeze(-1)
    return dict(out=out.view(tokens, heads, dim).to(torch.bfloat16), lse=lse.view(tokens, heads))


# ---------------------------------------------------------------- what a pass cannot do without


def work(case):
    op = case["op"]
    if op == "tables":
        ctx, new = _contexts(case), _news(case)
        taken = sum(_pages(c + n, case["block"]) - _pages(c, case["block"]) for c, n in zip(ctx, new))
        return {"bytes": 20 * case["reqs"] + 8 * taken + 12 * sum(new), "flops": 2 * sum(new)}
    hkv, dim, block = case["kv_heads"], case["dim"], case["block"]
    if op == "rope":
        width = 1 if case["fp8"] else 2
        rows = case["tokens"] * dim
        read = 2 * rows * (Q_HEADS + 2 * hkv) + case["tokens"] * (12 + 4 * case["rotary"])
        wrote = 2 * rows * Q_HEADS + 2 * width * rows * hkv + (0 if case["decode"] else 4 * rows * hkv)
        return {"bytes": read + wrote, "flops": rows * (Q_HEADS + hkv) * 8}
    if op == "bounds":
        filled = case["tokens"] / block if case["decode"] else case["tokens"] // block
        size = hkv * block * dim * (1 if case["fp8"] else 2)
        return {"bytes": int(8 * case["tokens"] + filled * (size + hkv * (2 * dim + 4))),
                "flops": int(filled * 2 * hkv * block * dim)}
    ctx, new = _contexts(case), case["new"]
    tokens = new * case["reqs"]
    if op == "select":
        pages = [_pages(c + new, block) - 1 for c in ctx]
        return {"bytes": sum(pages) * (4 + hkv * (2 * dim + 4)) + tokens * (2 * Q_HEADS * dim + 4 * hkv * case["pages"]),
                "flops": 2 * dim * Q_HEADS * new * sum(pages)}
    read, seen = 0, 0
    for c in ctx:
        at = [c + i for i in range(new)]
        older = min(case["pages"] - 1, c // block) * block
        read += older + sum(min(block, at[-1] + 1 - p * block) for p in {a // block for a in at})
        seen += sum(older + a % block + 1 for a in at)
    size = 2 * hkv * dim * (1 if case["fp8"] else 2)
    return {"bytes": read * size + tokens * (4 * Q_HEADS * dim + 4 * Q_HEADS + 4 * hkv * case["pages"]),
            "flops": 4 * seen * Q_HEADS * dim}


# ---------------------------------------------------------------- the definitions, in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(s)
    if case["op"] == "bounds":
        return _exact_bounds(s)
    if case["op"] == "attn":
        return _exact_attn(s)
    return None  # tables and page lists are whole numbers, equal or wrong


def _exact_rope(s):
    c_s = s["cos_sin"].double().index_select(0, s["positions"].long())
    half = c_s.shape[1] // 2
    turn = torch.polar(torch.ones_like(c_s[:, :half]), torch.zeros_like(c_s[:, :half]))
    turn = torch.complex(c_s[:, :half], c_s[:, half:]) * turn

    def head(x, w):
        y = x.double()
        if w is not None:
            y = y * (y.pow(2).sum(2, keepdim=True) / y.shape[2] + s["eps"]).rsqrt() * w.double()
        pairs = y[:, :, :2 * half].reshape(y.shape[0], y.shape[1], *((half, 2) if s["interleaved"] else (2, half)))
        if not s["interleaved"]:
            pairs = pairs.transpose(2, 3)
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn[:, None, :])
        if not s["interleaved"]:
            z = z.transpose(2, 3)
        return torch.cat((z.reshape(y.shape[0], y.shape[1], 2 * half), y[:, :, 2 * half:]), 2)

    q, k, v = head(s["q"], s["q_weight"]), head(s["k"], s["k_weight"]), s["v"].double()

    def written(cache, x, unit):
        n, hkv, block, dim = cache.shape
        flat = (cache if unit is None else cache.view(torch.float8_e4m3fn)).double().transpose(1, 2).reshape(-1, hkv, dim)
        flat[s["slots"]] = x if unit is None else (x / torch.tensor(unit).double().item()).clamp(-448, 448)
        return flat.view(n, block, hkv, dim).transpose(1, 2)

    units = s["scales"] or (None, None)
    keep = s["k_out"] is not None
    return dict(q=q, k=k if keep else None, v=v if keep else None, k_cache=written(s["k_cache"], k, units[0]),
                v_cache=written(s["v_cache"], v, units[1]))


def _exact_bounds(s):
    n, hkv, block, dim = s["keys"].shape
    filled = torch.zeros(n * block, dtype=torch.bool, device="cuda")
    filled[s["slots"]] = True
    filled = filled.view(n, block)[:, -1]
    keys = (s["keys"].view(torch.float8_e4m3fn) if s["keys"].dtype == torch.uint8 else s["keys"]).double()
    reach = keys.abs().flatten(2).unflatten(2, (block, dim)).amax((2, 3))
    # magnitudes are at least 0.005 of a power of two apart: a slip of the logarithm at a whole one does not count
    scale = torch.exp2(((reach / 127).log2() - 1e-6).ceil().clamp(min=-60))
    codes = torch.stack(((keys.min(2).values / scale[:, :, None]).floor(),
                         (keys.max(2).values / scale[:, :, None]).ceil()), 2)
    return dict(codes=torch.where(filled[:, None, None, None], codes.to(torch.int8), s["codes"]),
                scales=torch.where(filled[:, None], scale, s["scales"].double()))


def _exact_attn(s):
    tokens, heads, dim = s["q"].shape
    hkv, block = s["k_cache"].shape[1], s["block"]
    width = s["selected"].shape[2]
    row = torch.arange(tokens, device="cuda")
    req = (row[:, None] >= s["qsl"][None, 1:]).sum(1)
    last = s["seq"][req] - (s["qsl"][req + 1] - row)
    # every slot of the cache by its row, and the rows of each selected key
    key = (s["selected"].long().unsqueeze(3) * block + torch.arange(block, device="cuda")).view(tokens, hkv, -1)
    good = (s["selected"] >= 0).repeat_interleave(block, 2) & (key <= last[:, None, None])
    page = s["table"].long()[req[:, None, None], torch.div(key.clamp(min=0), block, rounding_mode="floor")]
    place = (page * hkv + torch.arange(hkv, device="cuda")[:, None]) * block + key % block
    unit = s["scales"] or (1.0, 1.0)

    def of(cache):
        x = cache.view(-1, dim)[place.clamp(min=0).view(-1)]
        return (x.view(torch.float8_e4m3fn) if s["scales"] else x).double().view(tokens, hkv, width * block, dim)

    q = s["q"].double().view(tokens, hkv, heads // hkv, dim)
    logit = torch.einsum("thgd,thnd->thgn", q, of(s["k_cache"])) * (s["scale"] * unit[0])
    logit = torch.where(good[:, :, None], logit, -math.inf)
    out = torch.einsum("thgn,thnd->thgd", logit.softmax(-1), of(s["v_cache"])) * unit[1]
    return dict(out=out.reshape(tokens, heads, dim), lse=logit.logsumexp(-1).reshape(tokens, heads))
