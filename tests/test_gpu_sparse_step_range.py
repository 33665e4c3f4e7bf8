"""The block-sparse step at the far ends of the ranges its header names, against float64."""
import numpy as np
import pytest
import torch

from paged_kv_attention_07_gb300 import pka
from tests.test_gpu_sparse_step import BF16, I64, bounds_check, dev, word

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
