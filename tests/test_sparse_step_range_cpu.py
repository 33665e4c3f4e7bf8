"""Sizes of the block-sparse step that the host refuses before any launch, and what the check of long page lists tells
apart."""
import numpy as np
import pytest

from paged_kv_attention_07_gb300 import build as B
from paged_kv_attention_07_gb300 import pka
from tests.test_gpu_sparse_step_range import SCALE, attn_of_list, each_page_case, each_page_near
from tests.test_sparse_step_cpu import ROPE, ROPE_ORDER, _call


@pytest.fixture(scope="module")
def lib():
    B.build()
    return pka.load()


# No tokens: nothing is launched where the sizes are taken.
@pytest.mark.parametrize("heads,d,status", [(1 << 23, 128, 0), ((1 << 23) + 1, 128, 2), ((1 << 31) - 1, 8, 2),
                                            (1 << 22, 256, 0), (1 << 24, 128, 2), ((1 << 22) + 1, 256, 2)])
@pytest.mark.parametrize("name", ["Hq", "Hkv"])
def test_rope_indexes_of_a_row_stay_in_32_bits(lib, name, heads, d, status):
    kw = {name: heads, "d": d, "T": 0, "rot": 0}
    assert _call(lib.pka_qk_rope_cache_write, ROPE_ORDER + " err stream", ROPE, kw) == status
    assert _call(lib.pka_qk_rope_cache_write_fp8, ROPE_ORDER + " k_scale v_scale err stream", ROPE, kw) == status


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("bs", [8, 64])
def test_a_wrong_page_of_a_long_list_is_seen(bs, fp8):
    """The lists that an error at the turn of a warp's 32 pages would leave, in float64."""
    b, caches, q, pages, look = each_page_case(bs, fp8)
    want = attn_of_list(b, q, caches, pages, SCALE)
    assert each_page_near(want[0], want[1], want, fp8).all()
    n = len(pages)
    at = [int(x) for x in look.flatten()[:60:15] if 32 <= x < n - 33]
    for j in at:
        here = look == j
        swapped, again, early, late = (pages.copy() for _ in range(4))
        swapped[j] = j - 32       # the row of the last turn
        again[j + 1] = j          # a page twice, its neighbour not at all
        early[j:-1] = pages[j + 1:]  # off by one from there on
        late[j] = j + 32
        for other in (np.delete(pages, j), swapped, again, early, late):
            o, l = attn_of_list(b, q, caches, other, SCALE)[:2]
            assert not each_page_near(o, l, want, fp8)[here].any()
