"""Routing where the values are hard.  Tolerances (u = 2^-24, h = 2^-8: unit
roundoffs of fp32 and bf16): weights 128 u as in test_gpu_ops.py, others as derived
beside their tests."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from test_gpu_ops import f64, run_route  # noqa: E402

pytestmark = pytest.mark.gpu
U, H = 2.0 ** -24, 2.0 ** -8
TINY = 2.0 ** -126  # below it numbers have fewer bits


@pytest.fixture(scope="module")
def c3():
    from concurrent_communication_overlap_gb300 import c3 as mod
    return mod


def name(r):
    return "_".join(f"{k}{v}" for k, v in r.items())


# ----------------------------------------------------------------------------- sigmoids that round alike

ORDER = [
    dict(E=64, k=8), dict(E=60, k=6), dict(E=2, k=1), dict(E=371, k=8), dict(E=512, k=10), dict(E=1000, k=16),
    dict(E=256, k=8, G=8, keep=4), dict(E=160, k=6, G=8, keep=3), dict(E=100, k=4, G=25, keep=5),
    dict(E=256, k=8, G=8, keep=4, best=2), dict(E=488, k=4, G=4, keep=2, best=2), dict(E=24, k=3, G=8, keep=2, best=2),
    dict(E=100, k=4, G=25, keep=5, best=2),
]


# (no sums of two saturated scores: they are equal in fp32, and so are the groups then)
BASES = [(r, b) for r in ORDER for b in (2.0, 9.0, 20.0, -9.0, -95.0) if b == 2.0 or "best" not in r]


@pytest.mark.parametrize("T", [3, 4100])
@pytest.mark.parametrize("r,base", BASES, ids=[f"{name(r)}_{b:g}" for r, b in BASES])
def test_sigmoid_orders_as_its_logits(c3, r, T, base):
    """Neighbouring fp32 logits, whose sigmoids are equal in fp32 or nearly: the larger logit is the better expert."""
    r = dict(r, score="sigmoid")
    E, k, G, keep, best = r["E"], r["k"], r.get("G", 1), r.get("keep", 1), r.get("best", 1)
    rng = np.random.default_rng(E + T)
    step = float(np.spacing(np.float32(abs(base))))
    x = base + rng.permuted(np.tile(np.arange(E), (T, 1)), axis=1) * step
    if G > 1:   # groups 1/4 apart, so that their scores do not tie
        level = rng.permuted(np.tile(np.arange(G), (T, 1)), axis=1) / (4.0 if best == 2 else 2.0 ** 20)
        x = (x.reshape(T, G, -1) + level[:, :, None]).reshape(T, E).astype(np.float32).astype(np.float64)
    idx, w, _, _ = run_route(c3, r, x, 0)
    key = x
    if G > 1:
        top = np.sort(x.reshape(T, G, -1), -1)[:, :, ::-1][:, :, :best]
        score = top[:, :, 0] if best == 1 else (1 / (1 + np.exp(-top))).sum(-1)
        kept = np.argsort(-score, axis=1, kind="stable")[:, :keep]
        stay = np.zeros((T, G), bool)
        np.put_along_axis(stay, kept, True, 1)
        key = np.where(np.repeat(stay, E // G, 1), x, -np.inf)
    want = np.argsort(-key, axis=1, kind="stable")[:, :k]
    assert np.array_equal(idx.cpu().numpy(), want)
    ref = 1 / (1 + np.exp(-np.take_along_axis(x, want, 1)))
    assert (np.abs(f64(w) - ref) <= 128 * U * ref + TINY).all()
