"""GPU tests of the shared-prefix attention where a plan over the whole cache would have more than 128 splits: one query of
129 to 148 tiles of 128 keys, with and without a prefix, bf16 and FP8 windows."""
import pytest
import torch

from tests.cmp_utils import f64
from tests.test_gpu_shared_attn import W, Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n_p,own", [(16384, 8), (300, 16200), (0, 16500), (0, 18800)])
def test_one_query_of_many_tiles(cuda_lib, n_p, own, fp8):
    c = Case(cuda_lib, 1, 1, 16, n_p, own, fp8=fp8, seed=n_p + own)
    c.check(*c.run(cuda_lib))


def test_long_cache_without_a_prefix_keeps_a_nan(cuda_lib):
    """The queries that see an entry that is not finite are NaN on this plan too, infinities of either sign included."""
    csa = cuda_lib
    c = Case(csa, 1, 1, 16, 0, 16500, n_c=[16490], seed=4)
    out, lse = c.run(csa)
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    c.cache.rope[0, 16490] = float("nan")                   # behind the last visible entry
    o2, l2 = c.run(csa)
    assert torch.equal(o2, out) and torch.equal(l2, lse)
    c.cache.rope[0, 777, 3] = float("-inf")
    o2, l2 = c.run(csa)
    assert torch.isnan(o2).all() and torch.isnan(l2).all()


def test_agrees_with_the_unshared_attention(cuda_lib):
    """bf16 windows, where hca_attn serves the length too (by another kernel)."""
    csa = cuda_lib
    c = Case(csa, 1, 1, 16, 0, 16500, seed=5)
    out, lse = c.run(csa)
    ro, rl = csa.hca_attn(*c.args[:4], *c.args[5:], ratio=c.r, window=W)
    c.check(out, lse)
    c.check(ro, rl)
    assert abs(f64(lse) - f64(rl)).max() < 2e-3             # (each within LSE_ATOL of the oracle)
