"""The sparse layer of examples/ on the GPU: forward and gradients against the
formula in 64 bits on the quantised operands (quantisation passes gradients
straight through), small enough to be written out.

Tolerance: bf16 roundings of the experts' rows and of the result, 2^-8 each of the
sums of magnitudes, and as much for the quantised gradient rows, whose bf16 inputs
already are roundings: 4 * 2^-8 of sum |.| in all; products add far less."""
import importlib.util
import os

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from test_gpu_ops import quantise_oracle

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def load_example():
    spec = importlib.util.spec_from_file_location("sparse_layer", os.path.join(ROOT, "examples", "sparse_layer.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def values(c3, q, count):
    """The values of a 4-bit operand, [count][rows][cols]."""
    out = torch.empty(count, q.rows, q.cols, device="cuda")
    c3.c3_fp4_dequantize(q, out, c3.C3_F32, q.cols)
    torch.cuda.synchronize()
    return f64(out)


@pytest.mark.parametrize("tokens,experts,topk,n,k", [(1, 8, 2, 64, 96), (37, 16, 3, 136, 200), (300, 8, 1, 256, 128)])
def test_forward_and_gradients(tokens, experts, topk, n, k):
    ex = load_example()
    c3 = ex.c3
    gen = torch.Generator(device="cuda").manual_seed(tokens)
    w = (torch.randn(experts, n, k, generator=gen, device="cuda") * 0.1).to(torch.bfloat16)
    layer = ex.SparseLayer(w, topk, tokens, c3.Router(experts, topk, score=c3.C3_SCORE_SIGMOID, scale=1.5))
    x = torch.randn(tokens, k, generator=gen, device="cuda").to(torch.bfloat16)
    logits = torch.randn(tokens, experts, generator=gen, device="cuda")
    dout = torch.randn(tokens, n, generator=gen, device="cuda").to(torch.bfloat16)
    out = layer.forward(x, logits).clone()
    dx, dlogits = layer.backward(logits, dout)
    c3.c3_status_check()
    again = layer.forward(x, logits)
    torch.cuda.synchronize()
    assert torch.equal(out, again)

    idx = layer.idx.cpu().numpy()
    lg = f64(logits)
    assert np.array_equal(idx, np.argsort(-lg, axis=1, kind="stable")[:, :topk])
    s = 1 / (1 + np.exp(-np.take_along_axis(lg, idx, 1)))
    W, WT = values(c3, layer.forward_weights.matrix, experts), values(c3, layer.backward_weights.matrix, experts)
    slot = layer.slot.cpu().numpy()
    xq = values(c3, layer.x_rows, 1)[0][slot]                       # [tokens][topk][k]
    y = np.einsum("tjk,tjnk->tjn", xq, W[idx])
    ymag = np.einsum("tjk,tjnk->tjn", np.abs(xq), np.abs(W)[idx])
    h = 2.0 ** -8
    ref, mag = (1.5 * s[..., None] * y).sum(1), (1.5 * s[..., None] * np.abs(y)).sum(1)
    assert (np.abs(f64(out) - ref) <= 4 * h * mag + 1e-5 * ymag.sum(1)).all()

    d = f64(dout)
    g = (d[:, None] * y).sum(-1)
    gmag = (np.abs(d)[:, None] * np.abs(y)).sum(-1)
    ref_dl, tol = np.zeros_like(lg), np.zeros_like(lg)
    np.put_along_axis(ref_dl, idx, 1.5 * g * s * (1 - s), 1)
    np.put_along_axis(tol, idx, 1.5 * 4 * h * gmag * s * (1 - s) + 1e-6, 1)
    assert (np.abs(f64(dlogits) - ref_dl) <= tol).all()
    # the rows' gradient as it was quantised, through the transposed matrices
    dyq = values(c3, layer.dy_rows, 1)[0][slot]
    ref_dx = np.einsum("tjn,tjkn->tk", dyq, WT[idx])
    parts = np.einsum("tjn,tjkn->tjk", dyq, WT[idx])
    tol = 4 * h * np.abs(parts).sum(1) + 1e-5 * np.einsum("tjn,tjkn->tk", np.abs(dyq), np.abs(WT)[idx])
    assert (np.abs(f64(dx) - ref_dx) <= tol).all()
    # those rows are w dout, rounded to bf16, and then to 4 bits exactly as defined
    want = 1.5 * s[..., None] * d[:, None]
    assert (np.abs(f64(layer.dy)[slot] - want) <= h * np.abs(want) + 1e-9).all()
    assert np.array_equal(dyq, quantise_oracle(layer.dy.float().cpu().numpy(), 0)[2][slot])


def test_experts_that_do_not_divide_by_the_ranks():
    ex = load_example()
    with pytest.raises(ValueError):
        ex.SparseLayer(torch.zeros(12, 32, 32, dtype=torch.bfloat16, device="cuda"), 2, 4)
