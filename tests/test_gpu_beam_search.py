"""Beam search over shared pages, every call of a step together: tables, cache writes of two layers, attention that reads
each prompt once, logits, selection, forked tables, copied pages. Beside it each beam's keys and values are kept densely and
reordered by the parents; pages must hold them bit for bit, the attention must be that over them, the selection that of the
logits, and the counts and the free list those of the tables. Prompts are forked into beams by the same call."""
import math

import numpy as np
import pytest
import torch

from oracle import fp8
from paged_kv_attention_07_gb300 import pka
from tests import shared_ref as ref

pytestmark = pytest.mark.gpu

BF16, I32, U8 = torch.bfloat16, torch.int32, torch.uint8
LAYERS, HQ, HKV, D, VOCAB = 2, 8, 2, 128, 500
END = 7


class Search:
    def __init__(self, prompts, beams, bs, kv_scales=None, seed=0, spare=4, longest=64):
        self.rng = np.random.default_rng(seed)
        self.prompts, self.groups, self.beams, self.bs, self.scales = prompts, len(prompts), beams, bs, kv_scales
        self.B = self.groups * beams
        self.width = -(-(max(prompts) + longest) // bs)
        self.blocks = sum(-(-p // bs) for p in prompts) + self.B * (-(-longest // bs) + 1) + spare
        kind = U8 if kv_scales else BF16
        self.caches = [torch.full((self.blocks, HKV, bs, D), 0x7f if kv_scales else math.nan, dtype=kind, device="cuda")
                       for _ in range(2 * LAYERS)]
        gen = torch.Generator("cuda").manual_seed(seed)

        def rand(*shape):
            return torch.randn(shape, generator=gen, device="cuda", dtype=BF16)

        self.embed = [[rand(VOCAB, h, D) for h in (HQ, HKV, HKV)] for _ in range(LAYERS)]
        self.head = torch.randn(HQ * D, VOCAB, generator=gen, device="cuda") * 0.2
        angle = torch.rand(4096, 32, generator=gen, device="cuda") * 6
        self.cos_sin = torch.cat([angle.cos(), angle.sin()], 1)
        self.table = self.ints(self.B, self.width)
        self.spare_table = self.ints(self.B, self.width)
        self.counts, self.free = self.ints(self.blocks), torch.randperm(self.blocks, generator=gen, device="cuda").to(I32)
        self.free_head, self.err = self.ints(1), self.ints(1)
        self.starts = torch.arange(self.groups + 1, device="cuda", dtype=I32) * beams
        self.prefix = torch.tensor(prompts, dtype=I32, device="cuda")
        self.history = None  # [row][cache]: [tokens, HKV, D]

    @staticmethod
    def ints(*shape, dtype=I32):
        return torch.zeros(shape, dtype=dtype, device="cuda")

    def write(self, rows, table, ctx, new, tokens, history):
        """New tokens of `rows` requests into the caches of all layers -> the queries of each layer and the step's tables."""
        T = tokens.numel()
        qsl, seq, pos, slots = self.ints(rows + 1), self.ints(rows), self.ints(T), self.ints(T, dtype=torch.int64)
        pka.pka_step_tables(ctx, new, table, self.bs, self.free, self.free_head, self.free_head, qsl, seq, pos, slots,
                            error_word=self.err)
        queries = []
        for layer in range(LAYERS):
            q, k, v = (e[tokens.long().clamp(min=0)] for e in self.embed[layer])
            out = torch.empty_like(q)
            kc, vc = self.caches[2 * layer:2 * layer + 2]
            pka.pka_qk_rope_cache_write(q, k, v, None, None, 1e-6, self.cos_sin, False, pos, slots, out, None, None, kc, vc,
                                        kv_scales=self.scales, error_word=self.err)
            queries.append(out)
        # the dense copy, read back slot by slot
        at, n = slots.cpu().tolist(), qsl.cpu().tolist()
        for r in range(rows):
            for t in range(n[r], n[r + 1]):
                for c, cache in enumerate(self.caches):
                    history[r][c].append(cache[at[t] // self.bs, :, at[t] % self.bs].clone())
        return queries, qsl, seq

    def fork(self, parents, ctx, table, out_table):
        n = parents.numel()
        ctx_out, src, dst = self.ints(n), self.ints(n), self.ints(n)
        pka.pka_fork_pages(parents, ctx, table, self.bs, self.counts, self.free, self.free_head, self.free_head, ctx_out,
                           out_table, src, dst, error_word=self.err)
        pka.pka_copy_pages(self.caches, src, dst, error_word=self.err)
        return ctx_out

    def start(self):
        """The prompts, each once, then a row per beam."""
        rows = self.groups
        table, ctx = self.ints(rows, self.width), self.ints(rows)
        tokens = torch.from_numpy(self.rng.integers(0, VOCAB, sum(self.prompts))).to(I32).cuda()
        history = [[[] for _ in self.caches] for _ in range(rows)]
        _, _, seq = self.write(rows, table, ctx, self.prefix.clone(), tokens, history)
        parents = torch.arange(rows, device="cuda", dtype=I32).repeat_interleave(self.beams)
        self.ctx = self.fork(parents, seq, table, self.table)
        self.history = [[list(c) for c in history[p]] for p in parents.tolist()]
        self.scores = torch.full((self.groups, self.beams), -math.inf, device="cuda")
        self.scores[:, 0] = 0  # (the beams are equal: one counts)
        self.finished = self.ints(self.groups, self.beams, dtype=U8)
        self.tokens = torch.from_numpy(self.rng.integers(0, VOCAB, self.groups)).to(I32).cuda().repeat_interleave(self.beams)
        self.check_pages()

    def step(self):
        B = self.B
        live = (self.finished.flatten() == 0) & (self.tokens >= 0)
        new = live.to(I32)
        T = B  # (rows behind the last request's new token are padding)
        order = torch.argsort(~live, stable=True)
        tokens = torch.where(torch.arange(B, device="cuda") < live.sum(), self.tokens[order], 0)
        queries, qsl, seq = self.write(B, self.table, self.ctx, new, tokens, self.history)
        longest = int(seq.max())
        work = torch.empty(pka.pka_prefix_workspace_size(B, self.groups, T, HQ, HKV, D, 1), dtype=U8, device="cuda")
        hidden = torch.zeros(T, HQ * D, device="cuda")
        host = dict(qsl=qsl.tolist(), seq=seq.tolist())
        for layer in range(LAYERS):
            out, lse = torch.zeros_like(queries[layer]), torch.zeros(T, HQ, device="cuda")
            kc, vc = self.caches[2 * layer:2 * layer + 2]
            pka.pka_prefix_attn_forward(queries[layer], kc, vc, self.table, qsl, seq, self.starts, self.prefix, 0.09, 1,
                                        longest, out, lse, work, kv_scales=self.scales, error_word=self.err)
            self.check_attention(layer, queries[layer], out, lse, host)
            hidden += out.float().flatten(1)
        logits = torch.zeros(B, VOCAB, device="cuda")
        logits[order] = hidden @ self.head  # (rows of beams that are finished or empty are not read)
        logits[~live] = math.nan
        chosen = torch.empty_like(self.scores)
        parents, picked = self.ints(self.groups, self.beams), self.ints(self.groups, self.beams)
        ended = self.ints(self.groups, self.beams, dtype=U8)
        pka.pka_beam_select(logits, self.scores, chosen, parents, picked, END, self.finished, ended, error_word=self.err)
        self.check_select(logits, chosen, parents, picked, ended)
        # what is kept of this step: a beam's tokens so far have been written, its new one has not
        ctx = self.ctx + new
        self.ctx = self.fork(parents.flatten(), ctx, self.table, self.spare_table)
        self.table, self.spare_table = self.spare_table, self.table
        self.history = [[list(c) for c in self.history[p]] if p >= 0 else [[] for _ in self.caches]
                        for p in parents.flatten().tolist()]
        self.scores, self.finished, self.tokens = chosen, ended, picked.flatten()
        self.check_pages()

    # ---------------------------------------------------------------- checks

    def check_pages(self):
        assert int(self.err) == 0
        table, ctx = self.table.cpu().numpy(), self.ctx.tolist()
        holders = np.zeros(self.blocks, int)
        for r in range(self.B):
            pages = table[r, :-(-ctx[r] // self.bs)]
            holders[pages] += 1
            assert len(self.history[r][0]) == ctx[r]
            if ctx[r] == 0:
                continue
            at = torch.from_numpy(pages).long().cuda()
            for c, cache in enumerate(self.caches):
                held = cache[at].transpose(1, 2).reshape(-1, HKV, D)[:ctx[r]]
                want = torch.stack(self.history[r][c])
                assert torch.equal(held.view(U8), want.view(U8))
        assert np.array_equal(self.counts.cpu().numpy(), np.maximum(holders - 1, 0))
        free = self.free.cpu().numpy()[int(self.free_head):]
        assert sorted(free) == np.flatnonzero(holders == 0).tolist()

    def check_attention(self, layer, q, out, lse, host):
        ks, vs = self.scales or (1.0, 1.0)
        for r in range(self.B):
            for t in range(host["qsl"][r], host["qsl"][r + 1]):
                k, v = (torch.stack(self.history[r][2 * layer + i]).cpu() for i in range(2))
                if self.scales:
                    k, v = (torch.from_numpy(fp8.decode(x.numpy()).astype(np.float64)) for x in (k, v))
                k, v = k.double() * ks, v.double() * vs
                x = q[t].double().cpu().view(HKV, HQ // HKV, D)
                s = torch.einsum("hgd,nhd->hgn", x, k) * 0.09
                w = s.softmax(-1)
                want, mag = (torch.einsum("hgn,nhd->hgd", w, y).reshape(HQ, D) for y in (v, v.abs()))
                # roundings of the weights and of the result to bf16; scores in 32 bits, of 8-bit codes the query's split
                delta = (D + 8) * 2.0 ** -24 * 0.09 * torch.einsum("hgd,nhd->hgn", x.abs(), k.abs()).max() + 2.0 ** -20
                if self.scales:
                    delta += 2.0 ** -17 * x.abs().max() * k.abs().sum(-1).max() * 0.09
                got = out[t].double().cpu()
                assert ((got - want).abs() <= 2.0 ** -8 * want.abs() + (2.0 ** -8 + 3 * delta) * mag * (1 + 2.0 ** -6)).all()
                l = torch.logsumexp(s, -1).reshape(HQ)
                assert ((lse[t].double().cpu() - l).abs() <= 2 * delta + 2.0 ** -22 * l.abs()).all()
        assert (out[host["qsl"][-1]:] == 0).all() and (lse[host["qsl"][-1]:] == 0).all()

    def check_select(self, logits, scores, parents, tokens, finished):
        want = ref.beam_select(logits.double().cpu().numpy(), self.scores.double().cpu().numpy(), self.finished.cpu().numpy(),
                               END, self.beams)
        assert np.array_equal(parents.cpu().numpy(), want[1]) and np.array_equal(tokens.cpu().numpy(), want[2])
        assert np.array_equal(finished.cpu().numpy(), want[3]) and not want[4]
        got, ok = scores.double().cpu().numpy(), np.isfinite(want[0])
        assert (np.abs(got[ok] - want[0][ok]) <= 2.0 ** -20 + 2.0 ** -24 * np.abs(want[0][ok])).all() and (got[~ok] == -np.inf).all()


@pytest.mark.parametrize("prompts,beams,bs,scales", [
    ([21], 4, 16, None), ([1, 40, 64, 17], 3, 16, None), ([300, 5], 5, 8, None), ([33, 128], 4, 32, (0.02, 0.03)),
    ([9, 2, 30], 2, 1, None), ([70, 3], 8, 4, (0.02, 0.03))])
def test_beam_search(prompts, beams, bs, scales):
    s = Search(prompts, beams, bs, scales, seed=beams + bs)
    s.start()
    for _ in range(12):
        s.step()
    ended = int(s.finished.sum())
    assert ended < s.B  # (what was tested to the end is a search that goes on)
    # the end: all rows gone, every page is free
    s.ctx = s.fork(torch.full((s.B,), -1, dtype=I32, device="cuda"), s.ctx, s.table, s.spare_table)
    assert int(s.err) == 0 and int(s.free_head) == 0 and not s.counts.any() and not s.ctx.any()
    assert sorted(s.free.tolist()) == list(range(s.blocks))
