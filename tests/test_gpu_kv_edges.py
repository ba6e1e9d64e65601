"""4-bit paged key/value cache on the GPU: contents and batches at the edge of
what the calls allow, against the 64-bit oracle."""
import numpy as np
import pytest

from kv_helpers import Case
from test_gpu_kv import TYPES, attend, ids

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("new", [2, 100])
@pytest.mark.parametrize("which", ["all", "some"])
def test_negative_scales(dtype, new, which):
    # a grid word is the bits of a scale, of either sign
    c = Case([(200, new), (150, new)], heads=2, share=2, dim=64, dtype=dtype, seed=new)
    rng = np.random.default_rng(new)
    for nm in "kv":
        w = c.cache[nm + "_grid"]
        w[rng.random(w.shape) < (1.0 if which == "all" else 0.5)] |= np.uint32(1 << 31)
    attend(c)
