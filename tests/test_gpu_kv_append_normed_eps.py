"""The norms of the cache append with an eps near the largest fp32 value: mean square and eps fit, their sum does not."""
import numpy as np
import pytest

from test_gpu_kv_append import slots_of
from test_gpu_kv_append_normed import NormRun

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("eps", [1e38, 3e38, float(np.finfo(np.float32).max)])
@pytest.mark.parametrize("D", [64, 128])
def test_sums_that_leave_fp32(eps, D):
    r = NormRun(8, 1, D, 16)
    size = np.exp2(np.arange(40, 128, 2.0))
    x = r.rng.uniform(0.5, 1, (len(size), 1, D)) * r.rng.choice([-1, 1], (len(size), 1, D)) * size[:, None, None]
    r.append(*slots_of(np.arange(8), 0, len(size), 16), q=x, k=x[::-1], Hq=1, eps=eps)
