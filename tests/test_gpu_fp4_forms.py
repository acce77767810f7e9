"""Every form of the 4-bit products at its remainders: which form a shape gets is
checked against the planner, without a GPU, in test_fp4_plan.py."""
import pytest

pytest.importorskip("torch")

from test_fp4_plan import FORMS, GROUPED_FORMS  # noqa: E402
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
