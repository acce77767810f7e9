"""Routing where the values are hard.  Tolerances (u = 2^-24, h = 2^-8: unit
roundoffs of fp32 and bf16): weights 128 u as in test_gpu_ops.py, others as derived
beside their tests."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from test_gpu_ops import (RAGGED_GROUPS, ROUTERS, TD, TWELVE, Guarded, cuda, f64, grid_logits,  # noqa: E402
                          route_grad_oracle, route_oracle, run_route)

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


# ----------------------------------------------------------------------------- gradients far from 0

@pytest.mark.parametrize("ty", [0, 1])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("T", [24, 4200])
@pytest.mark.parametrize("lo,hi", [(8, 20), (-20, -8), (-88.6, -85), (-88.6, 30), (30, 80)])
def test_sigmoid_gradient_keeps_its_digits(c3, lo, hi, T, renorm, ty):
    """c g s (1 - s), and with renorm c q (g - sum q g) (1 - s) with q = s / S: scores and complements near 0 have their
    digits too.  s and 1 - s are each three operations and an exponential (2 ulp): 8 u; S sums 8 terms: 16 u; so a term is
    within 64 u of itself, the terms being |g| and, with renorm, |g| + sum q |g|.  Below 2^-126 numbers are 2^-149 apart
    (bf16 2^-133): a factor that small is off by half that, 2^-150 / 3e-39 = 4 u of itself at -88.6, and so may a result
    be (three times that, for the factors it came from)."""
    E, k, scale = 40, 8, 2.5
    rng = np.random.default_rng(T)
    x = f64(cuda(rng.uniform(lo, hi, (T, E)).astype(np.float32)).to(TD[ty]))
    r = dict(E=E, k=k, score="sigmoid", renorm=renorm, scale=scale)
    idx, _, router, wide = run_route(c3, r, x, ty)
    dw = rng.standard_normal((T, k)).astype(np.float32) * 3
    dx = Guarded((T, E), TD[ty], 5.0)
    c3.c3_route_backward(router, wide, E, T, idx, cuda(dw), dx.t, E)
    torch.cuda.synchronize()
    assert dx.intact()
    idx = idx.cpu().numpy()
    z = np.take_along_axis(x, idx, 1)
    s, c, g = 1 / (1 + np.exp(-z)), 1 / (1 + np.exp(z)), scale * dw.astype(np.float64)
    if renorm:
        q = s / s.sum(1, keepdims=True)
        d, mag = q * (g - (q * g).sum(1, keepdims=True)) * c, q * (np.abs(g) + (q * np.abs(g)).sum(1, keepdims=True)) * c
    else:
        d = mag = g * s * c
    ref, tol = np.zeros((T, E)), np.zeros((T, E))
    np.put_along_axis(ref, idx, d, 1)
    np.put_along_axis(tol, idx, 64 * U * np.abs(mag) + 3 * (2.0 ** -133 if ty else 2.0 ** -149), 1)
    if ty:
        tol = tol + H * np.abs(ref)
    assert (np.abs(f64(dx.t) - ref) <= tol).all()


# ----------------------------------------------------------------------------- infinities

@pytest.mark.parametrize("T", [6, 4101])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("r", [dict(E=16, k=4), dict(E=16, k=4, bias=True), dict(E=16, k=4, G=4, keep=2, best=2),
                               dict(E=24, k=5, G=4, keep=2, bias=True), dict(E=100, k=3, G=25, keep=4, best=2),
                               dict(E=100, k=3, G=25, keep=4, best=2, bias=True), dict(E=400, k=9, bias=True)], ids=name)
def test_softmax_of_plus_infinity(c3, r, renorm, T):
    """A choice as by the logits (plus the bias), weights of NaN: the token is neither dropped nor quietly given weights."""
    r = dict(r, score="softmax", renorm=renorm)
    E, k, G, keep, best = r["E"], r["k"], r.get("G", 1), r.get("keep", 1), r.get("best", 1)
    rng = np.random.default_rng(E)
    x = grid_logits(rng, T, E)
    x[0, E // 2] = np.inf
    x[1, 1] = x[1, E - 2] = np.inf
    x[2, 0] = np.inf
    x[2, 3:9] = -np.inf
    x[T - 1] = np.inf
    bias = rng.integers(-8, 9, E) / 16.0 if r.get("bias") else np.zeros(E)
    if r.get("bias"):
        bias[2] = -np.inf
    idx, w, router, wide = run_route(c3, r, x, 0, bias if r.get("bias") else None)
    idx, w = idx.cpu().numpy(), f64(w)
    for t in (0, 1, 2, T - 1):
        with np.errstate(invalid="ignore"):
            key = x[t] + bias
        key = np.where(np.isnan(key), -np.inf, key)     # +inf under a bias of -inf: not eligible
        if G > 1:
            per = np.sort(key.reshape(G, -1), 1)[:, ::-1][:, :best]
            score = np.where(per[:, 0] > -np.inf, np.where(per > -np.inf, per, 0).sum(1), -np.inf)
            kept = np.argsort(-score, kind="stable")[:keep]
            key = np.where(np.isin(np.arange(E) // (E // G), kept), key, -np.inf)
        want = np.argsort(-key, kind="stable")[:k]
        want = np.where(key[want] > -np.inf, want, -1)
        assert np.array_equal(idx[t], want), t
        assert np.isnan(w[t][want >= 0]).all() and (w[t][want < 0] == 0).all()
    assert np.isfinite(w[3:T - 1]).all()
    dx = torch.empty(T, E, device="cuda")
    c3.c3_route_backward(router, wide, E, T, cuda(idx), cuda(rng.standard_normal((T, k)).astype(np.float32)), dx, E)
    torch.cuda.synchronize()
    dx = f64(dx)
    assert np.isfinite(dx[3:T - 1]).all()
    for t in (0, 1, 2, T - 1):
        chosen = idx[t][idx[t] >= 0]
        if renorm and not np.isinf(x[t, chosen]).any():
            continue    # the infinity was masked by its bias: the chosen logits are finite
        assert np.isnan(dx[t, chosen]).all(), t


@pytest.mark.parametrize("T", [6, 4101])
def test_sigmoid_of_infinities(c3, T):
    """1 and 0 like any other score: +inf is the best expert, -inf none."""
    E, k = 16, 4
    x = grid_logits(np.random.default_rng(1), T, E)
    x[0, 5] = x[0, 9] = np.inf
    x[1, 2:] = -np.inf
    x[2] = np.inf
    r = dict(E=E, k=k, score="sigmoid")
    idx, w, router, wide = run_route(c3, r, x, 0)
    ref_idx, ref_w = route_oracle(x[:6], E, k, "sigmoid")
    assert np.array_equal(idx.cpu().numpy()[:6], ref_idx)
    assert (np.abs(f64(w)[:6] - ref_w) <= 128 * U * ref_w).all()
    dx = torch.empty(T, E, device="cuda")
    c3.c3_route_backward(router, wide, E, T, idx, torch.ones(T, k, device="cuda"), dx, E)
    torch.cuda.synchronize()
    assert bool((dx[2] == 0).all()) and bool((dx[0, [5, 9]] == 0).all()) and bool(torch.isfinite(dx).all())


# ----------------------------------------------------------------------------- NaN rows

@pytest.mark.parametrize("T", [3, 4101])
@pytest.mark.parametrize("score,renorm", [("softmax", False), ("softmax", True), ("sigmoid", False), ("sigmoid", True)])
def test_gradient_of_a_nan_row(c3, score, renorm, T):
    """Softmax without renorm: NaN for the whole row, which every logit enters.  Else the gradient is that of the chosen
    logits (the NaN is not one of them), and NaN where dweights is."""
    E, k = 24, 4
    rng = np.random.default_rng(2)
    x = grid_logits(rng, T, E)
    x[1, 7] = np.nan
    x[2, 7] = np.nan
    r = dict(E=E, k=k, score=score, renorm=renorm)
    idx, w, router, wide = run_route(c3, r, x, 0)
    assert bool(torch.isnan(w[1:3]).all()) and bool(torch.isfinite(w[0]).all())
    dw = rng.standard_normal((T, k)).astype(np.float32)
    dw[2] = np.nan
    dx = torch.empty(T, E, device="cuda")
    c3.c3_route_backward(router, wide, E, T, idx, cuda(dw), dx, E)
    torch.cuda.synchronize()
    idx, dx = idx.cpu().numpy(), f64(dx)
    assert np.isfinite(dx[0]).all()
    assert np.isnan(dx[2, idx[2]]).all()
    if score == "softmax" and not renorm:
        assert np.isnan(dx[1:3]).all()
        return
    ref = route_grad_oracle(x[1:2], idx[1:2], dw[1:2].astype(np.float64), r)[0]
    assert (np.abs(dx[1] - ref) <= 256 * U * 4).all()
    rest = np.setdiff1d(np.arange(E), idx[2])
    assert (dx[2, rest] == 0).all()


# ----------------------------------------------------------------------------- every choice by itself

@pytest.mark.parametrize("ty", [0, 1])
@pytest.mark.parametrize("T", [77, 4101])
@pytest.mark.parametrize("r", ROUTERS + TWELVE + RAGGED_GROUPS, ids=name)
def test_every_choice_is_one_of_the_best(c3, r, T, ty):
    """Different experts, of groups that may stay, in descending order, none better left out, equal ones by number; and
    the weights of exactly these.  Keys and group scores are fp32 sums of at most two scores and a bias: a softmax score
    is 128 u off itself at most, a sigmoid less, a sum adds a u of a number of at most 4: 256 u in all."""
    E, k, G, keep, best = r["E"], r["k"], r.get("G", 1), r.get("keep", 1), r.get("best", 1)
    rng = np.random.default_rng(T * 100 + E)
    x = grid_logits(rng, T, E)
    x[rng.random((T, E)) < 0.03] = -np.inf
    bias = rng.integers(-8, 9, E) / 16.0 if r.get("bias") else None
    idx, w, _, _ = run_route(c3, r, x, ty, bias, extra=T % 3)
    idx, w = idx.cpu().numpy(), f64(w)
    some = np.arange(T) if T < 100 else rng.choice(T, 150, replace=False)
    room = 256 * U
    for t in some:
        ok = x[t] > -np.inf
        if not ok.any():
            assert (idx[t] == -1).all() and (w[t] == 0).all()
            continue
        if r["score"] == "softmax":
            s = np.exp(np.where(ok, x[t], -np.inf) - x[t][ok].max())
            s = s / s.sum()
        else:
            s = np.where(ok, 1 / (1 + np.exp(-x[t])), 0)
        key = np.where(ok, s + (0 if bias is None else bias), -np.inf)
        low = 0 if bias is None and best == 1 else room    # logits themselves: no rounding
        group = np.arange(E) // (E // G)
        top = np.sort(key.reshape(G, -1), 1)[:, ::-1][:, :best]
        score = np.where(top[:, 0] > -np.inf, np.where(top > -np.inf, top, 0).sum(1), -np.inf)
        cut = np.sort(score)[::-1][keep - 1]
        may = (score >= cut - low) & (score > -np.inf)
        if not low:
            may &= np.isin(np.arange(G), np.argsort(-score, kind="stable")[:keep])
        must = may if may.sum() <= keep else may & (score > cut + low)
        n = (idx[t] >= 0).sum()
        mine = idx[t][:n]
        assert (idx[t][n:] == -1).all() and (w[t][n:] == 0).all()
        assert len(set(mine)) == n and ok[mine].all() and may[group[mine]].all(), t
        assert len(set(group[mine])) <= keep
        if n < k:   # fewer than k only where the groups that stay have no more
            assert n >= (ok & must[group]).sum(), t
        if n:
            assert (np.diff(key[mine]) <= low).all(), t
            left = np.setdiff1d(np.nonzero(ok & must[group])[0], mine)
            if n == k and len(left):
                assert key[left].max() <= key[mine].min() + low, t
            # equal logits and biases have equal keys, whatever the rounding: the lower number goes first
            same = (x[t][mine][:, None] == x[t][left][None])
            if bias is not None:
                same &= bias[mine][:, None] == bias[left][None]
            assert not (same & (mine[:, None] > left[None]) & (group[mine][:, None] == group[left][None])).any(), t
            chosen = s[mine]
            if r.get("renorm"):
                chosen = chosen / chosen.sum()
            ref = r.get("scale", 1.0) * chosen
            assert (np.abs(w[t][:n] - ref) <= 128 * U * ref).all(), t
