"""The calls over shared pages without a GPU: what the entry points refuse, and the float64 definitions against simple cases."""
import ctypes

import numpy as np
import pytest
import torch

from paged_kv_attention_07_gb300 import build as B
from paged_kv_attention_07_gb300 import pka
from tests import shared_ref as ref

P, F = ctypes.c_void_p, ctypes.c_float
FAKE, OTHER = P(0x10000), P(0x20000)  # never dereferenced: every case below fails validation first
INVALID, UNSUPPORTED, SMALL = 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    B.build()
    return pka.load()


def select(lib, **kw):
    a = dict(x=FAKE, io=1, stride=100, s=FAKE, f=None, G=2, W=4, V=100, end=-1, K=4, os=OTHER, p=FAKE, t=FAKE, of=None, e=None)
    a.update(kw)
    return lib.pka_beam_select(a["x"], a["io"], a["stride"], a["s"], a["f"], a["G"], a["W"], a["V"], a["end"], a["K"],
                               a["os"], a["p"], a["t"], a["of"], a["e"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), INVALID), (dict(s=None), INVALID), (dict(os=None), INVALID), (dict(p=None), INVALID),
    (dict(t=None), INVALID), (dict(io=2), INVALID), (dict(G=-1), INVALID), (dict(W=0), INVALID), (dict(V=0), INVALID),
    (dict(K=0), INVALID), (dict(stride=99), INVALID), (dict(end=100), INVALID), (dict(end=-2), INVALID),
    (dict(f=FAKE), INVALID), (dict(x=P(0x10001)), INVALID), (dict(x=P(0x10002), io=0), INVALID), (dict(s=P(0x10002)), INVALID),
    (dict(K=5, os=FAKE), INVALID), (dict(K=5, f=FAKE, of=FAKE, end=1), INVALID), (dict(W=65), UNSUPPORTED),
    (dict(K=65), UNSUPPORTED), (dict(V=2 ** 26 + 1, stride=2 ** 27), UNSUPPORTED), (dict(G=2 ** 23), UNSUPPORTED),
    (dict(e=P(0x10002)), INVALID), (dict(G=0, x=None), 0)])
def test_beam_select_refuses(lib, kw, status):
    assert select(lib, **kw) == status


def fork(lib, **kw):
    a = dict(p=FAKE, N=4, c=FAKE, t=FAKE, R=4, mb=8, bs=16, sc=FAKE, nb=64, f=FAKE, nf=64, h=FAKE, ho=FAKE, co=OTHER,
             to=OTHER, s=FAKE, d=FAKE, e=None)
    a.update(kw)
    return lib.pka_fork_pages(a["p"], a["N"], a["c"], a["t"], a["R"], a["mb"], a["bs"], a["sc"], a["nb"], a["f"], a["nf"],
                              a["h"], a["ho"], a["co"], a["to"], a["s"], a["d"], a["e"], None)


@pytest.mark.parametrize("kw,status", [
    *[({k: None}, INVALID) for k in ("p", "c", "t", "sc", "f", "h", "ho", "co", "to", "s", "d")],
    (dict(R=0), INVALID), (dict(N=-1), INVALID), (dict(mb=0), INVALID), (dict(bs=0), INVALID), (dict(nb=0), INVALID),
    (dict(nf=-1), INVALID), (dict(co=FAKE), INVALID), (dict(to=FAKE), INVALID), (dict(s=P(0x10002)), INVALID),
    (dict(R=4097), UNSUPPORTED), (dict(N=4097), UNSUPPORTED), (dict(mb=2 ** 27), UNSUPPORTED),
    (dict(mb=2 ** 19, R=4096), UNSUPPORTED), (dict(nb=2 ** 31), UNSUPPORTED)])
def test_fork_pages_refuses(lib, kw, status):
    assert fork(lib, **kw) == status


def copy(lib, caches, n=None, nb=8, size=64, src=FAKE, dst=FAKE, pairs=2, e=None):
    arr = (P * max(1, len(caches)))(*caches) if caches is not None else None
    return lib.pka_copy_pages(arr, len(caches) if n is None else n, nb, size, src, dst, pairs, e, None)


@pytest.mark.parametrize("kw,status", [
    (dict(caches=[FAKE, None]), INVALID), (dict(caches=[P(0x10008)]), INVALID), (dict(caches=None, n=1), INVALID),
    (dict(caches=[FAKE], nb=0), INVALID), (dict(caches=[FAKE], size=0), INVALID), (dict(caches=[FAKE], size=24), INVALID),
    (dict(caches=[FAKE], pairs=-1), INVALID), (dict(caches=[FAKE], src=None), INVALID), (dict(caches=[FAKE], dst=None), INVALID),
    (dict(caches=[], n=-1), INVALID), (dict(caches=[FAKE] * 257), UNSUPPORTED), (dict(caches=[FAKE], size=2 ** 30 + 16), UNSUPPORTED),
    (dict(caches=[FAKE], nb=2 ** 31), UNSUPPORTED), (dict(caches=[FAKE], pairs=2 ** 24 + 1), UNSUPPORTED),
    (dict(caches=[], src=None), 0), (dict(caches=[FAKE], pairs=0, src=None), 0)])
def test_copy_pages_refuses(lib, kw, status):
    assert copy(lib, **kw) == status


def prefix(lib, fp8=False, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, bt=FAKE, mb=8, qsl=FAKE, sl=FAKE, B=4, gs=FAKE, pl=FAKE, g=2, T=4, Hq=8, Hkv=2, d=128,
             nb=64, bs=16, scale=0.1, ks=0.5, vs=0.5, maxq=1, maxs=100, out=FAKE, lse=None, ws=FAKE, size=1 << 40, e=None)
    a.update(kw)
    return (lib.pka_prefix_attn_forward_fp8 if fp8 else lib.pka_prefix_attn_forward)(
        a["q"], a["k"], a["v"], a["bt"], a["mb"], a["qsl"], a["sl"], a["B"], a["gs"], a["pl"], a["g"], a["T"], a["Hq"],
        a["Hkv"], a["d"], a["nb"], a["bs"], F(a["scale"]), *((F(a["ks"]), F(a["vs"])) if fp8 else ()), a["maxq"], a["maxs"],
        a["out"], a["lse"], a["ws"], a["size"], a["e"], None)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kw,status", [
    *[({k: None}, INVALID) for k in ("q", "k", "v", "bt", "qsl", "sl", "gs", "pl", "out", "ws")],
    *[({k: 0}, INVALID) for k in ("mb", "B", "g", "Hq", "Hkv", "nb", "bs", "maxq", "maxs")],
    (dict(T=-1), INVALID), (dict(g=5), INVALID), (dict(Hq=7), INVALID), (dict(scale=0.0), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(maxs=129), INVALID), (dict(ws=P(0x10010)), INVALID),
    (dict(q=P(0x10008)), INVALID), (dict(lse=P(0x10002)), INVALID), (dict(d=96), UNSUPPORTED), (dict(Hq=34), UNSUPPORTED),
    (dict(bs=24), UNSUPPORTED), (dict(bs=256), UNSUPPORTED), (dict(B=4097, g=1), UNSUPPORTED),
    (dict(nb=2 ** 28), UNSUPPORTED), (dict(T=2 ** 25), UNSUPPORTED), (dict(mb=2 ** 28, maxs=2 ** 30 + 1), UNSUPPORTED),
    (dict(T=0, q=None), 0)])
def test_prefix_attention_refuses(lib, kw, status, fp8):
    assert prefix(lib, fp8, **kw) == status


def test_prefix_attention_fp8_refuses(lib):
    for bad in (0.0, -1.0, float("inf"), float("nan")):
        assert prefix(lib, True, ks=bad) == INVALID and prefix(lib, True, vs=bad) == INVALID
    assert prefix(lib, True, d=64) == UNSUPPORTED


def test_prefix_workspace_size_refuses(lib):
    for bad in ((0, 1, 1, 8, 2, 128, 1), (4, 5, 4, 8, 2, 128, 1), (4, 1, 4, 8, 3, 128, 1), (4, 1, 4, 8, 2, 96, 1),
                (4, 1, 4, 64, 2, 128, 1), (4, 1, 4, 8, 2, 128, 0), (4, 1, -1, 8, 2, 128, 1)):
        assert lib.pka_prefix_workspace_size(*bad) == 0


# ---------------------------------------------------------------- the definitions


def test_selection_is_that_of_log_softmax():
    rng = np.random.default_rng(0)
    x, s = rng.standard_normal((6, 50)), -rng.random((2, 3))
    got = ref.beam_select(x, s, None, 7, 5)
    full = torch.from_numpy(x).log_softmax(1).view(2, -1) + torch.from_numpy(s).repeat_interleave(50, 1)
    top = full.topk(5, 1)
    assert np.allclose(got[0], top.values.numpy(), atol=1e-12)
    assert np.array_equal(got[1], top.indices.numpy() // 50 + [[0], [3]]) and np.array_equal(got[2], top.indices.numpy() % 50)
    done = np.array([[1, 0, 0], [1, 1, 1]])
    got = ref.beam_select(x, s, done, 7, 4)
    assert (got[2][1] == [7, 7, 7, -1]).all() and (got[3][1] == [1, 1, 1, 0]).all()
    assert sorted(got[0][1][:3], reverse=True) == list(got[0][1][:3]) and got[0][1][3] == -np.inf


def test_a_fork_and_an_end():
    # row 0 holds pages 5, 6 and half of 7; row 1 shares 5 and has half of 9
    table = np.array([[5, 6, 7, 0], [5, 9, 0, 0]])
    counts = [0] * 10
    counts[5] = 1
    free = [5, 6, 7, 9, 1, 2, 3, 4, 8, 0]
    got = ref.fork_pages([0, 0], [10, 6], table, 4, counts, free, 4, 10, np.full((2, 4), -5))
    assert got[0] == [10, 10] and got[1].tolist() == [[5, 6, 7, -5], [5, 6, 1, -5]]
    assert got[2] == [0, 0, 0, 0, 0, 1, 1, 0, 0, 0] and got[5:] == ([-1, 7], [-1, 1])
    assert got[4] == 4 and got[3][4:] == [9, 2, 3, 4, 8, 0]


def test_attention_with_and_without_groups():
    rng = np.random.default_rng(1)
    k, v = rng.standard_normal((9, 2, 4, 8)), rng.standard_normal((9, 2, 4, 8))
    q = rng.standard_normal((3, 4, 8))
    table, seq, qsl = np.array([[3, 1, 7], [3, 5, 2]]), [10, 9], [0, 1, 3]
    a = ref.prefix_attention(q, k, v, table, qsl, seq, [0, 2], [4], 0.5)
    b = ref.prefix_attention(q, k, v, table, qsl, seq, [0, 1, 2], [4, 0], 0.5)
    for x, y in zip(a, b):
        assert np.array_equal(x, y)
    keys = torch.from_numpy(np.concatenate([k[p].transpose(1, 0, 2) for p in table[1]])[:9])
    vals = torch.from_numpy(np.concatenate([v[p].transpose(1, 0, 2) for p in table[1]])[:9])
    mask = torch.arange(9)[None] <= torch.tensor([7, 8])[:, None]
    want = torch.nn.functional.scaled_dot_product_attention(
        torch.from_numpy(q[1:]).transpose(0, 1), keys.transpose(0, 1).repeat_interleave(2, 0),
        vals.transpose(0, 1).repeat_interleave(2, 0), attn_mask=mask, scale=0.5).transpose(0, 1)
    assert np.allclose(a[0][1:], want.numpy(), atol=1e-12)
