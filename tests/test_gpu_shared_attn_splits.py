"""GPU tests of the shared-prefix attention where a plan over the whole cache would have more than 128 splits: one query of
129 to 148 tiles of 128 keys, bf16 and FP8 windows."""
import pytest

from tests.test_gpu_shared_attn import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n_p,own", [(16384, 8), (300, 16200)])
def test_one_query_of_many_tiles(cuda_lib, n_p, own, fp8):
    c = Case(cuda_lib, 1, 1, 16, n_p, own, fp8=fp8, seed=n_p + own)
    c.check(*c.run(cuda_lib))
