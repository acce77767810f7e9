"""Every form of the 4-bit products at its remainders: which form a shape gets is
checked against the planner, without a GPU, in test_fp4_plan.py."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from test_fp4_plan import FORMS, GROUPED_FORMS  # noqa: E402
from test_gpu_ops import Guarded, random_fp4  # noqa: E402
from test_gpu_ops import test_experts_products as experts_product  # noqa: E402
from test_gpu_ops import test_product as product  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def c3():
    from concurrent_communication_overlap_gb300 import c3 as mod
    return mod


@pytest.mark.parametrize("out", [0, 1])
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("M,N,K,budget,form", FORMS)
def test_product_in_every_form(c3, M, N, K, budget, form, fmt, out):
    product(c3, M, N, K, budget, fmt, out)


@pytest.mark.parametrize("out", [0, 1])
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("E,N,K,counts,budget,form", GROUPED_FORMS)
def test_experts_products_in_every_form(c3, E, N, K, counts, budget, form, fmt, out):
    experts_product(c3, E, N, K, counts, budget, fmt, out)


@pytest.mark.parametrize("M,budget", [(256, 0), (2048, 2)])
def test_experts_that_overlap_touch_nothing_else(c3, M, budget):
    """An error of the caller's, but one that the device finds: every count claims all rows.  What is written
    lies in C, and every row has one of the products."""
    rng = np.random.default_rng(M)
    E, N, K = 40, 200, 96
    x, _ = random_fp4(c3, rng, M, K, 0)
    w, _ = random_fp4(c3, rng, N, K, 0, count=E)
    C = Guarded((M, N), torch.float32, float("nan"))
    counts = torch.full((E,), M, dtype=torch.int32, device="cuda")
    c3.c3_fp4_gemm_experts(x, w, torch.zeros(E + 1, dtype=torch.int32, device="cuda"), counts, C.t, 0, sm_budget=budget)
    c3.c3_status_check()
    assert C.intact()
    assert bool(torch.isfinite(C.t).all())
