"""The calls over shared pages at the borders of what they promise: bad page ids wherever they are passed on."""
import numpy as np
import pytest

from tests.test_gpu_shared_pages import E, fork_case

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
