"""The orthogonalisation on the GPU, against the same recurrence in 64 bits.

Tolerances (h = 2^-8 and f = 2^-11, half a step of bf16 and fp16 relative to the value).  One step, entry by entry:
A = X X^T is off by f |A| and, summed in fp32 over K, by K 2^-23 |X| |X|^T at most; P by |b| dA + |c| (dA |A| + |A| dA)
and f |P| and its own sums' m 2^-23 |c| |A| |A|; the result by dP |X| + |P| dX and K 2^-23 |P| |X|, where dX is f |X|
for fp32 inputs and 0 for bf16, and by h of itself.  Several steps, in the 2-norm: three roundings a step of f at most
each, independent of one another, each carried on by a factor of at most 3.4445, the quintic's steepest slope on the
singular values that it leaves: 3.4445 f sqrt(3 steps), and h for the output."""
import time

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from test_gpu_ops import Guarded, c3, f64  # noqa: F401

pytestmark = pytest.mark.gpu

H, F, U = 2.0 ** -8, 2.0 ** -11, 2.0 ** -24
TD = {0: torch.float32, 1: torch.bfloat16}
QUINTIC = (3.4445, -4.7750, 2.0315)


def oracle(u, coeffs, eps=1e-7):
    """The recurrence on one matrix (float64 tensor), with the coefficients as fp32 holds them."""
    x = u.T if u.shape[0] > u.shape[1] else u
    x = x / (torch.linalg.vector_norm(x) + float(np.float32(eps)))
    for a, b, c in np.asarray(coeffs, np.float32).astype(np.float64):
        g = x @ x.T
        x = a * x + (b * g + c * (g @ g)) @ x
    return x.T if u.shape[0] > u.shape[1] else x


def one_step_bound(u, coeffs, exact_input):
    """Bound of the error of one step, entry by entry, before the output's own rounding."""
    x = u.T if u.shape[0] > u.shape[1] else u
    x = (x / torch.linalg.vector_norm(x)).abs()
    a, b, c = map(abs, coeffs)
    m, n = x.shape
    dx = x * (0 if exact_input else F) + 2.0 ** -38  # (and what fp16's smallest steps leave, times 2^-13)
    g = x @ x.T
    dg = F * g + n * 2 * U * g + dx @ x.T + x @ dx.T + 2.0 ** -37
    p = a * torch.eye(m, dtype=x.dtype, device=x.device) + b * g + c * (g @ g)
    dp = b * dg + c * (dg @ g + g @ dg) + F * p + m * 2 * U * c * (g @ g) + 2.0 ** -34
    d = dp @ x + p @ dx + m * 2 * U * (p @ x)
    return d.T if u.shape[0] > u.shape[1] else d


def momentum(rng, count, m, n, rank=3, strong=3.0):
    x = rng.standard_normal((count, m, n))
    r = min(rank, m, n)
    return x + strong * rng.standard_normal((count, m, r)) @ rng.standard_normal((count, r, n))


def run(c3, x, ty, count, rows, cols, coeffs, ld=None, out_ld=None, out=None, work=None, **kw):  # noqa: F811
    out_ld = cols if out_ld is None else out_ld
    if out is None:
        out = torch.full((count, rows, out_ld), 7.0, dtype=torch.bfloat16, device="cuda")
    if work is None:
        work = torch.full((c3.c3_orthogonalize_bytes(rows, cols, count),), 0xC3, dtype=torch.uint8, device="cuda")
    c3.c3_orthogonalize(x, ty, rows, cols, out, work, coeffs, count=count, ld=ld, out_ld=out_ld, **kw)
    return out


SHAPES = [(1, 1), (1, 9), (9, 1), (2, 2), (8, 8), (7, 100), (100, 7), (64, 64), (127, 129), (128, 256), (129, 127),
          (255, 300), (256, 256), (300, 255), (257, 1000), (520, 257), (600, 640), (1000, 1000)]


@pytest.mark.parametrize("ty", [0, 1])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_one_step(c3, ty, rows, cols):  # noqa: F811
    rng = np.random.default_rng(rows * 3 + cols)
    x = torch.from_numpy(momentum(rng, 1, rows, cols)).cuda().to(TD[ty])
    scale = float(np.float32(1.3))
    for coeffs in (QUINTIC, (1.5, -0.5, 0.0), (0.0, 2.0, 0.0), (0.0, 0.0, -3.0), (1.0, 0.0, 0.0)):
        out = run(c3, x, ty, 1, rows, cols, [coeffs], scale=scale)
        u = x[0].double()
        ref = scale * oracle(u, [coeffs])
        tol = scale * one_step_bound(u, coeffs, ty == 1) + H * ref.abs() + 1e-30
        assert ((out[0].double() - ref).abs() <= tol * (1 + 1e-6)).all(), coeffs
    c3.c3_status_check()


def relative(out, ref):
    return float(torch.linalg.vector_norm(out.double() - ref) / torch.linalg.vector_norm(ref))


@pytest.mark.parametrize("ty,count,rows,cols,pad,out_pad,steps", [
    (1, 1, 64, 64, 0, 0, 5), (0, 1, 200, 300, 0, 0, 5), (1, 3, 300, 200, 0, 0, 5), (0, 2, 129, 515, 3, 5, 5),
    (1, 2, 515, 129, 8, 8, 6), (1, 5, 96, 1000, 4, 2, 3), (0, 1, 1000, 1000, 0, 0, 2), (1, 1, 1531, 700, 1, 1, 5),
    (0, 7, 40, 33, 0, 7, 5), (1, 1, 2304, 2200, 0, 0, 4), (1, 40, 256, 264, 0, 0, 5), (0, 1, 700, 5001, 0, 0, 5),
    (1, 1, 5000, 520, 0, 0, 5)])
def test_several_steps(c3, ty, count, rows, cols, pad, out_pad, steps):  # noqa: F811
    rng = np.random.default_rng(rows + cols)
    ld, out_ld = cols + pad, cols + out_pad
    g = Guarded((count, rows, ld), TD[ty])
    g.t.copy_(torch.from_numpy(momentum(rng, count, rows, ld)))
    keep = g.t.clone()
    out = Guarded((count, rows, out_ld), torch.bfloat16, 7.0)
    work = Guarded((c3.c3_orthogonalize_bytes(rows, cols, count),), torch.uint8, 0xC3)
    run(c3, g.t, ty, count, rows, cols, [QUINTIC] * steps, ld=ld, out_ld=out_ld, out=out.t, work=work.t)
    c3.c3_status_check()
    for i in range(count):
        ref = oracle(g.t[i, :, :cols].double(), [QUINTIC] * steps)
        assert relative(out.t[i, :, :cols], ref) <= 3.4445 * F * (3 * steps) ** 0.5 + H
    assert (out.t[:, :, cols:] == 7).all() and torch.equal(g.t, keep)
    assert out.intact() and work.intact() and g.intact()
    again = run(c3, g.t, ty, count, rows, cols, [QUINTIC] * steps, ld=ld, out_ld=out_ld)
    assert torch.equal(again[:, :, :cols], out.t[:, :, :cols])


def test_error_before_the_output_is_rounded(c3):  # noqa: F811
    """Roundings spread evenly over their steps are off by f / sqrt(3) in the square mean, so what they add up to is
    below 3.4445 f sqrt(3 steps / 3), 3.8e-3 for five steps.  Independent errors add up in squares, so the
    output's own rounding, found on the oracle, is taken off that way."""
    rng = np.random.default_rng(0)
    for rows, cols in ((1024, 1024), (512, 2048), (3000, 700)):
        x = torch.from_numpy(momentum(rng, 1, rows, cols, rank=8, strong=1.0)).cuda().to(torch.bfloat16)
        out = run(c3, x, 1, 1, rows, cols, [QUINTIC] * 5)[0].double()
        ref = oracle(x[0].double(), [QUINTIC] * 5)
        own, both = relative(ref.to(torch.bfloat16).double(), ref), relative(out, ref)
        print(rows, cols, own, both)
        assert both ** 2 - own ** 2 <= (3.4445 * F) ** 2 * 5, (rows, cols, own, both)


@pytest.mark.parametrize("ty,count,rows,cols,budget", [
    (1, 1, 200, 9000, 0), (1, 1, 9000, 200, 0), (0, 1, 1500, 2100, 0), (1, 1, 2100, 1500, 0), (1, 2, 300, 4000, 0),
    (1, 3, 1100, 1090, 0), (0, 1, 64, 20011, 0), (1, 1, 700, 3000, 20), (1, 1, 3000, 700, 34), (1, 1, 2600, 2700, 0)])
def test_products_that_are_cut_along_k(c3, ty, count, rows, cols, budget):  # noqa: F811
    """Long sums and few tiles: parts of a tile from several pairs, put together by the last; the same bits every time."""
    rng = np.random.default_rng(rows * 5 + cols)
    x = torch.from_numpy(momentum(rng, count, rows, cols)).cuda().to(TD[ty])
    out = run(c3, x, ty, count, rows, cols, [QUINTIC] * 3, sm_budget=budget)
    c3.c3_status_check()
    for i in range(count):
        assert relative(out[i], oracle(x[i].double(), [QUINTIC] * 3)) <= 3.4445 * F * 3 + H
    for _ in range(5):
        assert torch.equal(run(c3, x, ty, count, rows, cols, [QUINTIC] * 3, sm_budget=budget), out)


def test_singular_values_near_one(c3):  # noqa: F811
    rng = np.random.default_rng(4)
    q, _ = np.linalg.qr(rng.standard_normal((300, 200)))
    x = torch.from_numpy(q).cuda().float().unsqueeze(0) * 17
    out = run(c3, x, 0, 1, 300, 200, [(1.5, -0.5, 0.0)] * 12 )
    # all singular values alike, 1 / sqrt(200) after the norm: the cubic takes them to 1 within twelve steps
    assert relative(out[0], torch.from_numpy(q).cuda()) <= 3.4445 * F * 6 + H


def test_magnitudes(c3):  # noqa: F811
    """The norm takes any magnitude out, as far as eps lets it."""
    rng = np.random.default_rng(8)
    x = momentum(rng, 1, 70, 90)
    ref = None
    for power in (0, 60, -60, 115, -120):
        u = torch.from_numpy(x * 2.0 ** power).cuda().float()
        out = run(c3, u, 0, 1, 70, 90, [QUINTIC] * 5, eps=0.0)
        ref = out if ref is None else ref
        assert torch.equal(out, ref), power  # powers of two: the same bits
    # eps of the norm's size halves what the first step starts from
    u = torch.from_numpy(x).cuda().float()
    norm = float(torch.linalg.vector_norm(u.double()))
    out = run(c3, u, 0, 1, 70, 90, [QUINTIC] * 2, eps=norm)
    assert relative(out[0], oracle(u[0].double(), [QUINTIC] * 2, eps=norm)) <= 3.4445 * F * 6 ** 0.5 + H
    # values whose squares fp32 cannot hold, beside ordinary ones
    u[0, 0, 0] = 3e38
    out = run(c3, u, 0, 1, 70, 90, [QUINTIC] * 5)
    ref = oracle(u[0].double(), [QUINTIC] * 5)
    assert relative(out[0], ref) <= 3.4445 * F * 15 ** 0.5 + H
    # subnormal numbers
    u = torch.full((1, 3, 5), 1e-42, device="cuda")
    out = run(c3, u, 0, 1, 3, 5, [QUINTIC] * 5, eps=0.0)
    assert relative(out[0], oracle(u[0].double(), [QUINTIC] * 5, eps=0.0)) <= 3.4445 * F * 15 ** 0.5 + H


def test_zeros_and_what_is_not_finite(c3):  # noqa: F811
    rng = np.random.default_rng(6)
    for rows, cols in ((40, 70), (270, 140)):
        x = torch.from_numpy(momentum(rng, 6, rows, cols)).cuda().to(torch.bfloat16)
        clean = run(c3, x, 1, 6, rows, cols, [QUINTIC] * 5)
        x[1], x[2, rows - 1, cols - 1], x[4, 0, 3] = 0, float("nan"), -float("inf")
        out = run(c3, x, 1, 6, rows, cols, [QUINTIC] * 5)
        assert (out[1] == 0).all() and out[2].isnan().all() and out[4].isnan().all()
        for i in (0, 3, 5):
            assert torch.equal(out[i], clean[i])
        out = run(c3, x[1:2], 1, 1, rows, cols, [QUINTIC] * 5, eps=0.0)
        assert (out == 0).all()
        x[3, 5:] = 0  # of low rank, rows of zeros
        out = run(c3, x, 1, 6, rows, cols, [QUINTIC] * 5)
        assert (out[3, 5:] == 0).all()
        assert relative(out[3], oracle(x[3].double(), [QUINTIC] * 5)) <= 3.4445 * F * 15 ** 0.5 + H


def test_in_place_on_a_stream_and_in_a_graph(c3):  # noqa: F811
    rng = np.random.default_rng(2)
    rows, cols = 390, 520
    xs = [torch.from_numpy(momentum(rng, 2, rows, cols)).cuda().to(torch.bfloat16) for _ in range(3)]
    want = [run(c3, x, 1, 2, rows, cols, [QUINTIC] * 5) for x in xs]
    size = c3.c3_orthogonalize_bytes(rows, cols, 2)
    work, other = (torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(2))
    x, side, graph = xs[0].clone(), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        c3.c3_orthogonalize(x, 1, rows, cols, x, work, [QUINTIC] * 5, count=2, stream=torch.cuda.current_stream())
    for k in (1, 2, 0):
        x.copy_(xs[k])
        y = xs[(k + 1) % 3].clone()
        torch.cuda.synchronize()
        graph.replay()
        c3.c3_orthogonalize(y, 1, rows, cols, y, other, [QUINTIC] * 5, count=2, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(x, want[k]) and torch.equal(y, want[(k + 1) % 3])
    c3.c3_status_check()


@pytest.mark.parametrize("budget", [2, 3, 16, 150, 1000])
def test_budgets_change_nothing(c3, budget):  # noqa: F811
    rng = np.random.default_rng(11)
    x = torch.from_numpy(momentum(rng, 2, 700, 900)).cuda().to(torch.bfloat16)
    u = x.double()
    out = run(c3, x, 1, 2, 700, 900, [QUINTIC] * 5, sm_budget=budget)
    for i in range(2):
        assert relative(out[i], oracle(u[i], [QUINTIC] * 5)) <= 3.4445 * F * 15 ** 0.5 + H
    c3.c3_status_check()


@pytest.mark.parametrize("ty", [0, 1])
@pytest.mark.parametrize("cols", [1, 7, 8, 9, 15, 16, 17, 31, 33, 255, 257, 520, 777])
def test_rows_that_begin_anywhere(c3, ty, cols):  # noqa: F811
    """The one step X <- 1 X, where every value is the division by the norm alone: f for the conversion of fp32 (bf16 is
    exact), h for the output and 2^-20 for the norm, value by value.  What lies around the rows is NaN."""
    rng = np.random.default_rng(cols)
    rows = 5
    for off in range(9):
        for pad in (0, 1, 6, 8):
            g = Guarded((2 * rows * (cols + pad) + off,), TD[ty], float("nan"))
            x = g.t[off:].view(2, rows, cols + pad)[:, :, :cols]
            x.copy_(torch.from_numpy(rng.uniform(1, 2, (2, rows, cols)) * rng.choice([-1, 1], (2, rows, cols))))
            out = run(c3, g.t[off:], ty, 2, rows, cols, [(1, 0, 0)], ld=cols + pad)
            ref = x.double() / (torch.linalg.vector_norm(x.double(), dim=(1, 2), keepdim=True) + 1e-7)
            assert ((out.double() - ref).abs() <= (H + 2.0 ** -20 + (0 if ty else F)) * ref.abs()).all(), (off, pad)
    c3.c3_status_check()


def test_distance_that_nothing_is_read_at(c3):  # noqa: F811
    """A single row's distance to a next one may be any, also one that a tensor map cannot hold."""
    rng = np.random.default_rng(2)
    x = torch.from_numpy(momentum(rng, 1, 1, 264)).cuda().to(torch.bfloat16)
    for ld in (264, 1 << 38, 1 << 39, 1 << 42):
        out = torch.full((264,), 7.0, dtype=torch.bfloat16, device="cuda")
        c3.c3_orthogonalize(x, 1, 1, 264, out, torch.empty(c3.c3_orthogonalize_bytes(1, 264), dtype=torch.uint8, device="cuda"),
                            [QUINTIC], ld=ld, out_ld=ld)
        assert relative(out.view(1, 264), oracle(x[0].double(), [QUINTIC])) <= 3.4445 * F * 3 ** 0.5 + H
    c3.c3_status_check()


def test_past_32_bits(c3):  # noqa: F811
    """A stack of matrices whose elements pass 2^31, one step each."""
    count, rows, cols = 17, 8192, 16384  # 2.28 G elements
    x = torch.zeros(count, rows, cols, dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(1)
    for i in (0, 15, 16):
        x[i, :300, -200:] = torch.randn(300, 200, generator=gen, device="cuda").to(torch.bfloat16)
        x[i, -100:, :50] = torch.randn(100, 50, generator=gen, device="cuda").to(torch.bfloat16)
    out = run(c3, x, 1, count, rows, cols, [QUINTIC])
    c3.c3_status_check()
    for i in (0, 15, 16):
        # two blocks that share no rows or columns: each is a product of its own, with the whole matrix's norm
        norm = torch.linalg.vector_norm(x[i].double()) + 1e-7
        for r, c in ((slice(0, 300), slice(cols - 200, cols)), (slice(rows - 100, rows), slice(0, 50))):
            u = x[i, r, c].double() / norm
            a, b, q = np.asarray(QUINTIC, np.float32).astype(np.float64)
            ref = a * u + b * (u @ (u.T @ u)) + q * (u @ (u.T @ u) @ (u.T @ u))
            assert relative(out[i, r, c], ref) <= 3.4445 * F * 3 ** 0.5 + H
        assert (out[i, 300:-100] == 0).all() and (out[i, :300, :-200] == 0).all() and (out[i, -100:, 50:] == 0).all()
    for i in range(1, 15):
        assert not out[i].any()


def test_an_injected_launch_failure_is_reported(c3):  # noqa: F811
    x = torch.ones(1, 8, 8, dtype=torch.bfloat16, device="cuda")
    c3.c3_inject_fault(c3.C3_FAULT_GEMM_LAUNCH)
    with pytest.raises(c3.C3Error) as e:
        run(c3, x, 1, 1, 8, 8, [QUINTIC])
    assert e.value.status == c3.C3_ECUDA and "injected" in str(e.value)
    run(c3, x, 1, 1, 8, 8, [QUINTIC])
    c3.c3_status_check()


def blocks_of(count, rows, cols, seed):
    """A matrix of zeros but for two blocks that share no rows or columns, and where they are."""
    x = torch.zeros(count, rows, cols, dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(seed)
    at = [(slice(0, 300), slice(cols - 200, cols)), (slice(rows - 100, rows), slice(0, 50))]
    for r, c in at:
        x[:, r, c] = torch.randn(count, r.stop - r.start, c.stop - c.start, generator=gen, device="cuda").to(torch.bfloat16)
    return x, at


def test_a_chain_longer_than_a_waits_limit(c3):  # noqa: F811
    """Products on one pair of SMs that take several seconds together: the limit of a wait in a later product does not run
    while the earlier ones do."""
    rows, cols, steps = 16384, 20480, 6  # 1.25e14 operations at some 2.5e13 a second and pair
    x, at = blocks_of(1, rows, cols, 3)
    out = run(c3, x, 1, 1, rows, cols, [QUINTIC] * steps, sm_budget=2)
    c3.c3_status_check()
    norm = torch.linalg.vector_norm(x[0].double()) + float(np.float32(1e-7))
    for r, c in at:  # each block is a product of its own, with the whole matrix's norm
        u = x[0, r, c].double() / norm
        for a, b, q in np.asarray([QUINTIC] * steps, np.float32).astype(np.float64):
            g = u @ u.T
            u = a * u + (b * g + q * (g @ g)) @ u
        assert relative(out[0, r, c], u) <= 3.4445 * F * (3 * steps) ** 0.5 + H
        out[0, r, c] = 0
    assert not out.any()


def test_a_budget_leaves_the_other_sms_free(c3):  # noqa: F811
    """A product on 132 SMs beside an orthogonalisation on 20: it waits for none of the 15 products there, which take 37 ms.
    (Where the later of them stood on other SMs already, waiting, it took 30 times its time alone.)"""
    n, m = 8192, 4096
    x = torch.ones(n, n, dtype=torch.bfloat16, device="cuda")
    out, work = torch.empty_like(x), torch.empty(c3.c3_orthogonalize_bytes(n, n), dtype=torch.uint8, device="cuda")
    a, product = torch.ones(m, m, dtype=torch.bfloat16, device="cuda"), torch.empty(m, m, device="cuda")
    one, two = torch.cuda.Stream(), torch.cuda.Stream()

    def timed():
        begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        begin.record(two)
        c3.c3_gemm(a, a, product, m, m, m, sm_budget=132, stream=two)
        end.record(two)
        return begin, end

    alone, beside = [], []
    for _ in range(6):
        torch.cuda.synchronize()
        begin, end = timed()
        torch.cuda.synchronize()
        alone.append(begin.elapsed_time(end))
        c3.c3_orthogonalize(x, 1, n, n, out, work, [QUINTIC] * 5, sm_budget=20, stream=one)
        time.sleep(0.003)
        begin, end = timed()
        torch.cuda.synchronize()
        beside.append(begin.elapsed_time(end))
    c3.c3_status_check()
    assert min(beside) < 6 * min(alone), (alone, beside)


@pytest.mark.parametrize("ty", [0, 1])
@pytest.mark.parametrize("rows,cols,value", [(1024, 4096, 3e38), (4096, 1000, -2.5e38), (300, 70, 3e38), (512, 1031, 2.0 ** 127),
                                             (64, 64, 2.0 ** -133), (1024, 2048, 2.0 ** -126), (30, 20, 2.0 ** -60)])
def test_many_values_at_the_ends_of_the_range(c3, ty, rows, cols, value):  # noqa: F811
    """Finite matrices whose squares' sums neither fp32 nor one of its halves' ranges holds.  eps = 0."""
    rng = np.random.default_rng(rows)
    sign = torch.from_numpy(rng.choice([-1.0, 1.0], (1, rows, 1)) * rng.choice([-1.0, 1.0], (1, 1, cols))).cuda()
    x = (sign * value).float().to(TD[ty])
    out = run(c3, x, ty, 1, rows, cols, [QUINTIC] * 3, eps=0.0)
    c3.c3_status_check()
    # one singular value, 1 after the norm: three steps of the polynomial on it, and the vectors' product
    assert relative(out[0], oracle(x[0].double(), [QUINTIC] * 3, eps=0.0)) <= 3.4445 * F * 3 + H


def test_subnormal_numbers_of_every_size(c3):  # noqa: F811
    """fp32's smallest numbers, exact in fp64 (the sum of squares below is 2^-298 times a whole number)."""
    rng = np.random.default_rng(1)
    for power in (-149, -148, -145, -140):
        x = torch.from_numpy(rng.integers(-3, 4, (1, 90, 130)) * 2.0 ** power).cuda().float()
        assert x.double().abs().max() == 3 * 2.0 ** power
        out = run(c3, x, 0, 1, 90, 130, [QUINTIC] * 5, eps=0.0)
        assert relative(out[0], oracle(x[0].double(), [QUINTIC] * 5, eps=0.0)) <= 3.4445 * F * 15 ** 0.5 + H
    c3.c3_status_check()


@pytest.mark.parametrize("ty,count,rows,cols", [(1, 700, 20, 33), (0, 513, 65, 17), (1, 300, 130, 258)])
def test_stacks_of_many_small_matrices(c3, ty, count, rows, cols):  # noqa: F811
    test_several_steps(c3, ty, count, rows, cols, 0, 0, 4)


def test_output_scales_near_the_ends_of_the_range(c3):  # noqa: F811
    """Powers of two on top of a scale change no digit of what stays a normal bf16 number."""
    rng = np.random.default_rng(12)
    for rows, cols, steps in ((8, 8, 1), (8, 12, 5), (300, 5, 2)):
        x = torch.from_numpy(momentum(rng, 1, rows, cols)).cuda().to(torch.bfloat16)
        one = run(c3, x, 1, 1, rows, cols, [QUINTIC] * steps, scale=1.37).double()
        for power in (-60, -100, -108, -114, -120, 100, 120):
            out = run(c3, x, 1, 1, rows, cols, [QUINTIC] * steps, scale=1.37 * 2.0 ** power).double()
            normal = one.abs() * 2.0 ** power >= 2.0 ** -126
            assert normal.any() and torch.equal(out[normal], one[normal] * 2.0 ** power), (rows, cols, power)
            assert ((out - one * 2.0 ** power).abs()[~normal] <= 2.0 ** -133).all()
    c3.c3_status_check()


@pytest.mark.parametrize("ty,count,rows,cols", [(0, 1, 1024, 1024), (0, 1, 5003, 1347), (0, 1, 256, 640), (0, 2, 700, 3000),
                                                (1, 4, 512, 1024), (1, 1, 256, 640), (1, 1, 2100, 1500)])
def test_error_before_the_output_is_rounded_of_both_types(c3, ty, count, rows, cols):  # noqa: F811
    """As above, over types, stacks, odd sizes and sums that are cut: fp32 inputs have one rounding more, 3 * 5 + 1 of them, each
    f / sqrt(3) in the square mean and carried on by at most 3.4445.  Matrices between in bf16 would be off eight times as far."""
    rng = np.random.default_rng(rows)
    x = torch.from_numpy(momentum(rng, count, rows, cols, rank=8, strong=1.0)).cuda().to(TD[ty])
    out = run(c3, x, ty, count, rows, cols, [QUINTIC] * 5)
    for i in range(count):
        ref = oracle(x[i].double(), [QUINTIC] * 5)
        own, both = relative(ref.to(torch.bfloat16).double(), ref), relative(out[i], ref)
        print(ty, rows, cols, own, both, max(0.0, both ** 2 - own ** 2) ** 0.5)
        assert both ** 2 - own ** 2 <= (3.4445 * F) ** 2 * 16 / 3
    c3.c3_status_check()


@pytest.mark.parametrize("ty", [0, 1])
@pytest.mark.parametrize("rows,cols,rank", [(256, 640, 1), (640, 256, 3), (1024, 1024, 30)])
def test_matrices_of_low_rank(c3, ty, rows, cols, rank):  # noqa: F811
    """Directions that a matrix does not have: the roundings' noise there grows like the smallest singular values do, by the
    first coefficient a step.  In the Frobenius norm, of f |X| at most each and independent of one another: one of the
    conversion (none for bf16), three a step, each carried on by a for each step that is left."""
    rng = np.random.default_rng(rank)
    x = rng.standard_normal((1, rows, rank)) @ rng.standard_normal((1, rank, cols))
    x = torch.from_numpy(x).cuda().to(TD[ty])
    out = run(c3, x, ty, 1, rows, cols, [QUINTIC] * 5)
    noise = 0.0 if ty else 1.0  # in units of f^2
    for k in range(1, 6):
        norm = float(torch.linalg.vector_norm(oracle(x[0].double(), [QUINTIC] * k)))
        noise = noise * 3.4445 ** 2 + 3 * norm ** 2
    ref = oracle(x[0].double(), [QUINTIC] * 5)
    off = float(torch.linalg.vector_norm(out[0].double() - ref))
    print(ty, rows, cols, rank, off, F * noise ** 0.5, off / norm)
    assert off <= F * noise ** 0.5 + H * norm
    c3.c3_status_check()
