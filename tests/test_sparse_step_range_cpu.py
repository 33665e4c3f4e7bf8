"""Sizes of the block-sparse step that the host refuses before any launch."""
import pytest

from paged_kv_attention_07_gb300 import build as B
from paged_kv_attention_07_gb300 import pka
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
