"""Products of codes without a plan: a shared expert on block-fp8 rows, one dense product per rank. Tolerances are those
of the product's own tests (test_gpu_product.py)."""
import pytest

import combine_ep_plan_amd as ep
from gpu_util import note
from layer_ref import Dense
from test_gpu_product import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,rows,k,m,act", [(1, 1, 256, 384, ep.EP_ACT_SWIGLU), (1, 33, 128, 640, ep.EP_ACT_GELU),
                                            (3, 70, 256, 128, ep.EP_ACT_SILU), (2, 300, 128, 256, ep.EP_ACT_NONE),
                                            (1, 130, 256, 6400, ep.EP_ACT_NONE), (1, 300, 384, 3840, ep.EP_ACT_SILU),
                                            (1, 4113, 128, 2048, ep.EP_ACT_NONE)])
def test_dense_product_of_codes(n, rows, k, m, act):
    """In tiles of 32 x 64 (four sizes), 32 x 128, 128 x 128 and 256 x 256."""
    note(f"dense codes {n} {rows} {k} {m} {act}")
    Case(Dense(n, rows), n, k, m, act, fp8=True, bias=True, residual=True).check(pre=True)
