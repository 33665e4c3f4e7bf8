"""The block-sparse step's entry points refuse bad arguments on the host, before any launch
(no GPU), and the float64 definitions the GPU tests compare with agree with simple cases."""
import ctypes

import numpy as np
import pytest
import torch

from paged_kv_attention_07_gb300 import build as B
from paged_kv_attention_07_gb300 import pka
from tests import sparse_ref as ref

P = ctypes.c_void_p
FAKE, OTHER, ODD = P(0x10000), P(0x20000), P(0x10002)  # never dereferenced
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def lib():
    B.build()
    return pka.load()


def _call(fn, order, defaults, kw):
    assert set(kw) <= set(defaults)
    a = {**defaults, **kw}
    return fn(*[a[n] for n in order.split()])


TABLES = ("ctx new B T table width bs free nfree head head_out qsl seq pos slots err stream",
          dict(ctx=FAKE, new=FAKE, B=4, T=9, table=FAKE, width=8, bs=16, free=FAKE, nfree=50, head=FAKE, head_out=FAKE,
               qsl=OTHER, seq=OTHER, pos=FAKE, slots=FAKE, err=None, stream=None))


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), 1), (dict(T=-1), 1), (dict(width=0), 1), (dict(bs=0), 1), (dict(nfree=-1), 1),
    (dict(ctx=None), 1), (dict(new=None), 1), (dict(table=None), 1), (dict(free=None), 1), (dict(head=None), 1),
    (dict(head_out=None), 1), (dict(qsl=None), 1), (dict(seq=None), 1), (dict(slots=None), 1),
    (dict(seq=FAKE), 1),               # seq_lens may not be ctx_lens
    (dict(qsl=FAKE), 1),
    (dict(slots=P(0x10004)), 1), (dict(ctx=ODD), 1), (dict(err=ODD), 1),
    (dict(B=4097), 2), (dict(width=1 << 28), 2), (dict(T=1 << 31), 2),
])
def test_step_tables_refuses(lib, kw, status):
    assert _call(lib.pka_step_tables, *TABLES, kw) == status


ROPE_ORDER = ("q k v qs ks vs qw kw eps cs rot maxp inter pos slots T Hq Hkv d qo ko vo kc vc nb bs")
ROPE = dict(q=FAKE, k=FAKE, v=FAKE, qs=512, ks=256, vs=256, qw=FAKE, kw=FAKE, eps=1e-6, cs=FAKE, rot=64, maxp=100,
            inter=0, pos=FAKE, slots=FAKE, T=3, Hq=4, Hkv=2, d=128, qo=FAKE, ko=None, vo=None, kc=FAKE, vc=FAKE, nb=8,
            bs=16, err=None, stream=None, k_scale=1.0, v_scale=1.0)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(qo=None), 1), (dict(kc=None), 1),
    (dict(vc=None), 1), (dict(pos=None), 1), (dict(slots=None), 1),
    (dict(T=-1), 1), (dict(Hq=0), 1), (dict(Hkv=0), 1), (dict(d=0), 1), (dict(nb=0), 1), (dict(bs=0), 1),
    (dict(qw=None), 1), (dict(kw=None), 1),            # one weight without the other
    (dict(eps=-1e-6), 1), (dict(eps=NAN), 1), (dict(eps=INF), 1),
    (dict(rot=144), 1),                                # more than the head
    (dict(rot=-16), 1), (dict(cs=None), 1), (dict(maxp=0), 1), (dict(inter=2), 1),
    (dict(qs=504), 1), (dict(ks=248), 1), (dict(vs=128), 1),   # rows that overlap
    (dict(q=P(0x10008)), 1), (dict(cs=P(0x10004)), 1), (dict(kw=P(0x10008)), 1), (dict(ko=P(0x10008)), 1),
    (dict(slots=P(0x10004)), 1), (dict(pos=ODD), 1), (dict(err=ODD), 1),
    (dict(nb=1 << 62), 1),
    (dict(qs=516), 2), (dict(rot=24), 2), (dict(d=260, qs=1040, ks=520, vs=520), 2),
    (dict(d=264, qs=1056, ks=528, vs=528), 2),
    (dict(T=0, q=None), 0),
])
def test_qk_rope_cache_write_refuses(lib, kw, status):
    assert _call(lib.pka_qk_rope_cache_write, ROPE_ORDER + " err stream", ROPE, kw) == status
    order = ROPE_ORDER + " k_scale v_scale err stream"
    assert _call(lib.pka_qk_rope_cache_write_fp8, order, ROPE, kw) == status


@pytest.mark.parametrize("kw", [dict(k_scale=0.0), dict(k_scale=INF), dict(v_scale=-1.0), dict(v_scale=NAN)])
def test_qk_rope_cache_write_fp8_refuses_scales(lib, kw):
    order = ROPE_ORDER + " k_scale v_scale err stream"
    assert _call(lib.pka_qk_rope_cache_write_fp8, order, ROPE, kw) == 1


BOUNDS = ("kc dtype slots T Hkv d nb bs bounds scales err stream",
          dict(kc=FAKE, dtype=1, slots=FAKE, T=5, Hkv=2, d=128, nb=8, bs=16, bounds=FAKE, scales=FAKE, err=None,
               stream=None))


@pytest.mark.parametrize("kw,status", [
    (dict(kc=None), 1), (dict(slots=None), 1), (dict(bounds=None), 1), (dict(scales=None), 1),
    (dict(dtype=0), 1), (dict(dtype=3), 1), (dict(T=-1), 1), (dict(Hkv=0), 1), (dict(d=0), 1), (dict(nb=0), 1),
    (dict(bs=0), 1), (dict(kc=P(0x10008)), 1), (dict(bounds=P(0x10008)), 1), (dict(scales=ODD), 1),
    (dict(slots=P(0x10004)), 1), (dict(err=ODD), 1), (dict(nb=1 << 62), 1),
    (dict(d=96), 2), (dict(d=256), 2), (dict(Hkv=70000), 2), (dict(T=0, kc=None), 0),
])
def test_page_bounds_refuses(lib, kw, status):
    assert _call(lib.pka_page_bounds, *BOUNDS, kw) == status


SELECT = ("q bounds scales bt width qsl seq B T Hq Hkv d nb bs first last maxs K sel err stream",
          dict(q=FAKE, bounds=FAKE, scales=FAKE, bt=FAKE, width=64, qsl=FAKE, seq=FAKE, B=2, T=3, Hq=8, Hkv=2, d=128,
               nb=100, bs=16, first=1, last=2, maxs=1024, K=8, sel=FAKE, err=None, stream=None))


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), 1), (dict(bounds=None), 1), (dict(scales=None), 1), (dict(bt=None), 1), (dict(qsl=None), 1),
    (dict(seq=None), 1), (dict(sel=None), 1), (dict(B=0), 1), (dict(T=-1), 1), (dict(Hq=7), 1), (dict(Hkv=0), 1),
    (dict(nb=0), 1), (dict(bs=0), 1), (dict(width=0), 1), (dict(maxs=0), 1), (dict(K=0), 1),
    (dict(maxs=1025), 1),                          # the table is narrower than max_seq_len needs
    (dict(first=-1), 1), (dict(last=0), 1), (dict(first=7), 1), (dict(last=9, first=0), 1),
    (dict(q=P(0x10008)), 1), (dict(bounds=P(0x10008)), 1), (dict(sel=ODD), 1), (dict(err=ODD), 1),
    (dict(d=96), 2), (dict(Hq=34), 2), (dict(Hkv=70000, Hq=70000), 2), (dict(T=(1 << 26) + 1), 2),
    (dict(maxs=32769, width=32769, bs=1), 2),      # more pages than the selection holds
    (dict(T=0, q=None), 0),
])
def test_select_pages_refuses(lib, kw, status):
    assert _call(lib.pka_select_pages, *SELECT, kw) == status


ATTN_ORDER = "q kc vc bt width qsl seq B T Hq Hkv d nb bs scale"
ATTN_TAIL = " sel K maxs out lse err stream"
ATTN = dict(q=FAKE, kc=FAKE, vc=FAKE, bt=FAKE, width=64, qsl=FAKE, seq=FAKE, B=2, T=3, Hq=8, Hkv=2, d=128, nb=100,
            bs=16, scale=0.1, sel=FAKE, K=8, maxs=1024, out=FAKE, lse=None, err=None, stream=None, k_scale=1.0,
            v_scale=1.0)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), 1), (dict(kc=None), 1), (dict(vc=None), 1), (dict(bt=None), 1), (dict(qsl=None), 1),
    (dict(seq=None), 1), (dict(sel=None), 1), (dict(out=None), 1), (dict(B=0), 1), (dict(T=-1), 1), (dict(Hq=7), 1),
    (dict(K=0), 1), (dict(maxs=0), 1), (dict(maxs=1025), 1), (dict(scale=0.0), 1), (dict(scale=-1.0), 1),
    (dict(scale=NAN), 1), (dict(q=P(0x10008)), 1), (dict(kc=P(0x10008)), 1), (dict(out=P(0x10008)), 1),
    (dict(lse=ODD), 1), (dict(sel=ODD), 1), (dict(err=ODD), 1),
    (dict(d=96), 2), (dict(Hq=34), 2), (dict(bs=24), 2), (dict(bs=4, maxs=256), 2), (dict(bs=256), 2),
    (dict(nb=1 << 31), 2), (dict(nb=1 << 27), 2), (dict(T=0, q=None), 0),
])
def test_sparse_attn_refuses(lib, kw, status):
    assert _call(lib.pka_sparse_attn_forward, ATTN_ORDER + ATTN_TAIL, ATTN, kw) == status
    assert _call(lib.pka_sparse_attn_forward_fp8, ATTN_ORDER + " k_scale v_scale" + ATTN_TAIL, ATTN, kw) == status


def test_calls_with_tensors_refuse_what_they_cannot_read(lib):
    # (RuntimeError where there is no device at all)
    t = torch.zeros(4, 2, 16, 128, dtype=torch.bfloat16)
    with pytest.raises((ValueError, RuntimeError)):
        pka.pka_page_bounds(t, t, t, t)
    with pytest.raises((TypeError, RuntimeError)):
        pka.pka_page_bounds(None, 3, "bounds", [])
    with pytest.raises(TypeError):
        pka._calls().page_bounds(t, t)


BIG = (1 << 31) - 1


def test_indexes_of_a_request_stay_in_32_bits(lib):
    # sums such as max_seq_len + block_size, and the last tile's key indexes, would pass them
    for kw in (dict(maxs=BIG, width=BIG, bs=1 << 20), dict(maxs=BIG, width=1, bs=BIG), dict(K=(1 << 30) + 1),
               dict(maxs=(1 << 30) + 1, width=65, bs=1 << 24)):
        assert _call(lib.pka_select_pages, *SELECT, kw) == 2
    for kw in (dict(maxs=BIG, width=BIG), dict(maxs=(1 << 30) + 1, width=1 << 30), dict(K=(1 << 30) + 1)):
        assert _call(lib.pka_sparse_attn_forward, ATTN_ORDER + ATTN_TAIL, ATTN, kw) == 2
        assert _call(lib.pka_sparse_attn_forward_fp8, ATTN_ORDER + " k_scale v_scale" + ATTN_TAIL, ATTN, kw) == 2
    assert _call(lib.pka_page_bounds, *BOUNDS, dict(bs=(1 << 20) + 1)) == 2
    # within the limits: one page longer than the request, no tokens
    assert _call(lib.pka_select_pages, *SELECT, dict(maxs=5, width=1, bs=BIG, T=0)) == 0


@pytest.mark.parametrize("kw,status", [(dict(d=64), 2), (dict(k_scale=0.0), 1), (dict(v_scale=NAN), 1)])
def test_sparse_attn_fp8_refuses(lib, kw, status):
    assert _call(lib.pka_sparse_attn_forward_fp8, ATTN_ORDER + " k_scale v_scale" + ATTN_TAIL, ATTN, kw) == status


# ---- the definitions


def test_unit_exponent_is_the_least():
    for a in (1e-30, 2.0 ** -53, 0.3, 1.0, 127.0, 127.5, 128.0, 3.0e38):
        e = ref.unit_exponent(a)
        assert a <= 127 * 2.0 ** e and (e == -60 or a > 127 * 2.0 ** (e - 1))
    assert ref.unit_exponent(0.0) == -60 and ref.unit_exponent(127.0) == 0 and ref.unit_exponent(127.5) == 1


def test_bounds_enclose_and_scores_are_upper_bounds():
    rng = np.random.default_rng(5)
    for _ in range(20):
        keys = rng.standard_normal((16, 64)) * rng.lognormal(0, 1, 64)
        lo, hi, unit = ref.page_bounds(keys)
        assert (lo * unit <= keys).all() and (keys <= hi * unit).all() and abs(lo).max() <= 127 and abs(hi).max() <= 127
        c, u = ref.query_codes(rng.standard_normal(64))
        bound = np.maximum(c * lo, c * hi).sum() * unit * u
        assert bound >= (keys @ (c * u)).max() * (1 - 1e-12)


def test_rope_definition_is_a_rotation_and_keeps_the_rest():
    rng = np.random.default_rng(6)
    x = rng.standard_normal((5, 2, 32))
    angle = rng.uniform(0, 6, (40, 8))
    table = np.concatenate([np.cos(angle), np.sin(angle)], 1)
    pos = np.array([0, 3, 39, 7, 7])
    for inter in (False, True):
        y, _ = ref.rope(x, None, 0.0, table, pos, inter)
        ia, ib = (slice(0, 16, 2), slice(1, 16, 2)) if inter else (slice(0, 8), slice(8, 16))
        z = (x[..., ia] + 1j * x[..., ib]) * np.exp(1j * angle[pos])[:, None]
        assert np.allclose(y[..., ia], z.real) and np.allclose(y[..., ib], z.imag)
        assert np.array_equal(y[..., 16:], x[..., 16:])


def test_sparse_attention_with_all_pages_is_dense():
    rng = np.random.default_rng(7)
    q, k, v = rng.standard_normal((1, 2, 8)), rng.standard_normal((3, 1, 4, 8)), rng.standard_normal((3, 1, 4, 8))
    out, lse, _ = ref.sparse_attn(q, k, v, np.array([[2, 0, 1]]), [0, 1], [10], np.array([[[0, 1, 2, -1]]]), 0.5)
    keys = np.concatenate([k[2, 0], k[0, 0], k[1, 0]])[:10]
    vals = np.concatenate([v[2, 0], v[0, 0], v[1, 0]])[:10]
    w = np.exp(0.5 * q[0] @ keys.T)
    assert np.allclose(out[0], w @ vals / w.sum(-1, keepdims=True)) and np.allclose(lse[0], np.log(w.sum(-1)))


def test_step_tables_definition():
    table = np.full((2, 3), 9)
    got = ref.step_tables([4, 0], [1, 3], table, 4, [5, 6, 7], 1, 5)
    assert got[0].tolist() == [[9, 6, 9], [7, 9, 9]] and got[1:4] == (3, [0, 1, 4], [5, 3])
    assert got[4] == [4, 0, 1, 2, -1] and got[5] == [24, 28, 29, 30, -1]
