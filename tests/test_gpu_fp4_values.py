"""4-bit matrices of zeros under any fp32 scale, and products whose sums are long and of one sign."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from test_gpu_ops import TD, cuda, f64, new_fp4, quantise_oracle, random_fp4, read_tiles  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def c3():
    from concurrent_communication_overlap_gb300 import c3 as mod
    return mod


@pytest.mark.parametrize("ty", [0, 1])
@pytest.mark.parametrize("way", ["rows", "odd rows", "transposed", "gathered"])
@pytest.mark.parametrize("g", [0.0, 2.0 ** -140, float("inf"), 0.25])
def test_blocks_of_zeros_have_scale_zero(c3, g, way, ty):
    """Whatever tensor_scale is: that of a matrix of zeros, max|x| / 2688, is 0 and 1 / 0 infinite.  A block with
    anything else in it then holds infinities (1 / g infinite) or zeros (g infinite)."""
    R, C = 40, 200
    rng = np.random.default_rng(0)
    x = np.zeros((R, C), np.float32)
    x[3, 20] = 1.5
    x[4, 48:64] = rng.standard_normal(16)
    x[7] = -0.0
    x[39, 199] = -2.0
    src = cuda(x).to(TD[ty])
    x = src.float().cpu().numpy()
    row_of = None
    rows, cols, ld = R, C, C
    if way == "transposed":
        src, rows, cols, ld = src.t().contiguous(), C, R, R
    elif way == "odd rows":
        wide = torch.zeros(R, C + 3, dtype=TD[ty], device="cuda")
        wide[:, :C] = src
        src, ld = wide, C + 3
    elif way == "gathered":
        row_of = torch.arange(R, dtype=torch.int32, device="cuda")
    q, codes, scales = new_fp4(c3, R, C, 1, g)
    c3.c3_fp4_quantize(src, ty, rows, cols, q, ld=ld, transpose=way == "transposed", row_of=row_of)
    back = torch.empty(R, C, device="cuda")
    c3.c3_fp4_dequantize(q, back, 0, C)
    torch.cuda.synchronize()
    assert codes.intact() and scales.intact()
    bytes_, past = read_tiles(scales.t[0].cpu().numpy(), R, 13)
    empty = (np.concatenate([x, np.zeros((R, 8), np.float32)], 1).reshape(R, 13, 16) == 0).all(-1)
    assert (bytes_[empty] == 0).all() and (past == 0).all()
    code = codes.t[0].cpu().numpy()
    code = np.stack([code & 15, code >> 4], -1).reshape(R, -1)
    blank = np.concatenate([np.repeat(empty, 16, 1), np.ones((R, 16), bool)], 1)
    assert (code[blank] == 0).all()
    back = f64(back)
    blank = blank[:, :C]
    if g == 0.25:
        ref = quantise_oracle(x, 1, g)[2]
        assert np.array_equal(back, ref)
    elif g == float("inf"):
        assert np.isnan(back).all()     # 0 * inf
    else:
        assert (back[blank] == 0).all()
        assert (bytes_[~empty] == 0x7F).all() and np.isnan(back[~blank]).all()


@pytest.mark.parametrize("M,N", [(7, 50), (300, 200)])
def test_a_matrix_of_zeros_with_its_own_scale(c3, M, N):
    """The gradient of an expert that no token chose: its product is 0, and not NaN."""
    K = 96
    d = torch.zeros(M, K, device="cuda")
    w = torch.randn(N, K, device="cuda", generator=torch.Generator(device="cuda").manual_seed(0))
    a, _, _ = new_fp4(c3, M, K, 1, float(d.abs().max() / 2688))
    b, _, _ = new_fp4(c3, N, K, 1, float(w.abs().max() / 2688))
    c3.c3_fp4_quantize(d, 0, M, K, a)
    c3.c3_fp4_quantize(w, 0, N, K, b)
    C = torch.full((M, N), 7.0, device="cuda")
    c3.c3_fp4_gemm(a, b, C, 0)
    c3.c3_status_check()
    assert bool((C == 0).all())


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("M,N,K", [(20, 130, 20000), (300, 200, 20000), (64, 128, 65536)])
def test_long_sums_of_one_sign(c3, M, N, K, fmt):
    """fp32 outputs where every addition can lose something on the same side: the header's bound, (K / 64 + 64) 2^-23 of
    sum |a b|, and one rounding of the output's own."""
    rng = np.random.default_rng(K + M)
    a, va = random_fp4(c3, rng, M, K, fmt)
    b, vb = random_fp4(c3, rng, N, K, fmt)
    for q in (a, b):
        q._keep[0].bitwise_and_(0x77)   # no signs
    va, vb = np.abs(va[0]), np.abs(vb[0])
    C = torch.empty(M, N, device="cuda")
    c3.c3_fp4_gemm(a, b, C, 0)
    c3.c3_status_check()
    ref = va @ vb.T
    assert (np.abs(f64(C) - ref) <= ((K / 64 + 64) * 2.0 ** -23 + 2.0 ** -24) * ref).all()
