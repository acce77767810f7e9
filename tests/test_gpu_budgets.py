"""What a budget of SMs leaves to others: a product on the other SMs runs as fast beside a chain of budgeted calls as it
does alone, up to what they share of power and of L2."""
import time

import pytest

torch = pytest.importorskip("torch")

from test_gpu_ops import c3  # noqa: F401

pytestmark = pytest.mark.gpu


def matrix(c3, n):  # noqa: F811
    new = lambda size: torch.zeros(size, dtype=torch.uint8, device="cuda")  # noqa: E731
    return c3.Fp4(n, n, c3.C3_FP4_MX, new(c3.c3_fp4_code_bytes(n, n)), new(c3.c3_fp4_scale_bytes(n, n, c3.C3_FP4_MX)))


@pytest.mark.parametrize("n,calls", [(8192, 16), (4096, 60)])
def test_4_bit_products_under_a_budget(c3, n, calls):  # noqa: F811
    """Calls on 20 SMs, one after the other.  (Where the later ones stood on other SMs already, waiting, the product on 132
    took 18 times its time alone.)"""
    a, b = matrix(c3, n), matrix(c3, n)
    out = torch.empty(n, n, dtype=torch.bfloat16, device="cuda")
    m = 4096
    x, y = torch.ones(m, m, dtype=torch.bfloat16, device="cuda"), torch.empty(m, m, device="cuda")
    one, two = torch.cuda.Stream(), torch.cuda.Stream()

    def timed():
        begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        begin.record(two)
        c3.c3_gemm(x, x, y, m, m, m, sm_budget=132, stream=two)
        end.record(two)
        return begin, end

    alone, beside = [], []
    for _ in range(6):
        torch.cuda.synchronize()
        begin, end = timed()
        torch.cuda.synchronize()
        alone.append(begin.elapsed_time(end))
        for _ in range(calls):
            c3.c3_fp4_gemm(a, b, out, c3.C3_BF16, sm_budget=20, stream=one)
        time.sleep(0.001)
        begin, end = timed()
        torch.cuda.synchronize()
        beside.append(begin.elapsed_time(end))
    c3.c3_status_check()
    print(alone, beside)
    assert min(beside) < 6 * min(alone), (alone, beside)
