"""Routing, 4-bit matrices and products, experts' products and their
combination on the GPU, against plain implementations in 64 bits written here
from the formulas.

Tolerances (u = 2^-24 and h = 2^-8, the unit roundoffs 2^-p of the 24-bit and 8-bit
significands of fp32 and bf16):
  routing weights  a softmax of logits within 20 of each other: x - max rounds
                   by 20 u, exp by 4 u, a sum of at most 1024 positive terms
                   (32 a lane, then 5 across lanes) by 37 u, the quotient and
                   the factors by 3 u; numerator and denominator both: 128 u;
  products         K products summed in fp32, each addition possibly cut off
                   instead of rounded (2 u): (K / 64 + 64) 2 u times sum |a b|,
                   one addition per 64-column instruction and at most 64 within;
  combination      topk roundings of u each on sum |w y|; inner products of
                   cols terms: cols u on sum |d y|;
  bf16 outputs     h of the value on top.
What is whole or exact (choices on a grid of logits, orders, codes, scales,
decoded values) is compared for equality."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

U, H = 2.0 ** -24, 2.0 ** -8
GRID = np.array([0, .5, 1, 1.5, 2, 3, 4, 6])
TD = {0: torch.float32, 1: torch.bfloat16}


@pytest.fixture(scope="module")
def c3():
    from concurrent_communication_overlap_gb300 import c3 as mod
    return mod


def cuda(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


class Guarded:
    """A tensor inside a larger one whose surroundings must not change."""

    def __init__(self, shape, dtype, fill=None, pad=4096):
        n = int(np.prod(shape))
        size = torch.empty(0, dtype=dtype).element_size()
        self.raw = torch.full((2 * pad + n * size,), 0xA7, dtype=torch.uint8, device="cuda")
        self.lo, self.hi = pad, pad + n * size
        self.t = self.raw[self.lo:self.hi].view(dtype).view(shape)
        if fill is not None:
            self.t.fill_(fill)

    def intact(self):
        return bool((self.raw[:self.lo] == 0xA7).all() and (self.raw[self.hi:] == 0xA7).all())


# ----------------------------------------------------------------------------- routing

def route_oracle(x, E, k, score, bias=None, G=1, keep=1, best=1, renorm=False, scale=1.0):
    """idx, weights and the scores, in 64 bits; x float64 [T, E]."""
    T = x.shape[0]
    idx = np.full((T, k), -1)
    w = np.zeros((T, k))
    for t in range(T):
        row = x[t]
        ok = ~np.isnan(row) & (row > -np.inf)
        s = np.zeros(E)
        if score == "softmax":
            if ok.any():
                with np.errstate(invalid="ignore"):
                    p = np.where(ok, np.exp(row - row[ok].max()), 0)
                s = p / p.sum()
            key = row if bias is None and best == 1 else s + (0 if bias is None else bias)
        else:
            s[ok] = 1 / (1 + np.exp(-row[ok]))
            key = s + (0 if bias is None else bias)
        key = np.where(ok, key, -np.inf)
        key = np.where(np.isnan(key), -np.inf, key)
        if G > 1:
            per = key.reshape(G, -1)
            score_g = np.full(G, -np.inf)
            for g in range(G):
                top = np.sort(per[g][per[g] > -np.inf])[::-1][:best]
                if len(top):
                    score_g[g] = top.sum()
            stay = np.argsort(-score_g, kind="stable")[:keep]
            mask = np.full(G, False)
            mask[stay] = True
            key = np.where(np.repeat(mask, E // G), key, -np.inf)
        order = np.argsort(-key, kind="stable")[:k]
        order = order[key[order] > -np.inf]
        idx[t, :len(order)] = order
        chosen = s[order]
        if renorm and len(order):
            if score == "softmax":
                e = np.exp(row[order] - row[order].max())
                chosen = e / e.sum()
            else:
                chosen = chosen / chosen.sum() if chosen.sum() > 0 else chosen * 0
        w[t, :len(order)] = scale * chosen
        if np.isnan(row).any():
            w[t, :len(order)] = np.nan
    return idx, w


def grid_logits(rng, T, E):
    """Logits on a grid of 1/8: exact in bf16, with many ties."""
    return rng.integers(-32, 33, (T, E)) / 8.0


ROUTERS = [
    dict(E=1, k=1, score="softmax"),
    dict(E=2, k=2, score="softmax", renorm=True),
    dict(E=8, k=2, score="softmax", renorm=True, scale=2.5),
    dict(E=60, k=6, score="softmax"),
    dict(E=64, k=8, score="sigmoid", renorm=True),
    dict(E=33, k=32, score="sigmoid", scale=0.5),
    dict(E=160, k=6, score="softmax", G=8, keep=3),
    dict(E=256, k=8, score="sigmoid", G=8, keep=4, best=2, renorm=True, scale=2.5, bias=True),
    dict(E=256, k=8, score="sigmoid", G=8, keep=8, best=1, bias=True),
    dict(E=96, k=5, score="sigmoid", G=32, keep=7, best=2, bias=True),
    dict(E=100, k=3, score="softmax", G=50, keep=4, best=2),
    dict(E=257, k=4, score="softmax", bias=True, renorm=True),
    dict(E=512, k=10, score="sigmoid", bias=True),
    dict(E=1000, k=32, score="softmax"),
    dict(E=1024, k=8, score="sigmoid", G=2, keep=1, best=2, renorm=True),
    dict(E=1000, k=6, score="sigmoid", G=50, keep=7, best=2, bias=True),
    dict(E=402, k=5, score="softmax", G=201, keep=100),
]


def router_of(c3, r, ty, bias):
    return c3.Router(r["E"], r["k"], score=c3.C3_SCORE_SIGMOID if r["score"] == "sigmoid" else c3.C3_SCORE_SOFTMAX,
                     groups=r.get("G", 1), topk_groups=r.get("keep", 1), group_best=r.get("best", 1),
                     renorm=r.get("renorm", False), scale=r.get("scale", 1.0), bias=bias, logits_type=ty)


def oracle_args(r):
    return {n: r[n] for n in ("G", "keep", "best", "renorm", "scale") if n in r}


def run_route(c3, r, x, ty, bias=None, extra=0, stream=None):
    T, E, k = x.shape[0], r["E"], r["k"]
    wide = torch.full((T, E + extra), 99.0, dtype=TD[ty], device="cuda")
    wide[:, :E] = cuda(x).to(TD[ty])
    idx = Guarded((T, k), torch.int32, -7)
    w = Guarded((T, k), torch.float32, -7)
    b = None if bias is None else cuda(bias.astype(np.float32))
    router = router_of(c3, r, ty, b)
    c3.c3_route(router, wide, E + extra, T, idx.t, w.t, stream=stream)
    torch.cuda.synchronize()
    assert idx.intact() and w.intact()
    return idx.t, w.t, router, wide


@pytest.mark.parametrize("ty", [0, 1])
@pytest.mark.parametrize("T,extra", [(1, 0), (77, 5)])
@pytest.mark.parametrize("r", ROUTERS, ids=lambda r: "_".join(f"{k}{v}" for k, v in r.items()))
def test_route(c3, r, T, extra, ty):
    rng = np.random.default_rng(T * 1000 + r["E"])
    x = grid_logits(rng, T, r["E"])
    bias = rng.integers(-8, 9, r["E"]) / 16.0 if r.get("bias") else None
    idx, w, _, _ = run_route(c3, r, x, ty, bias, extra)
    ref_idx, ref_w = route_oracle(x, r["E"], r["k"], r["score"], bias, **oracle_args(r))
    idx, w = idx.cpu().numpy(), f64(w)
    by_logit = r["score"] == "softmax" and bias is None and r.get("best", 1) == 1
    if by_logit:
        assert np.array_equal(idx, ref_idx)
    else:
        # keys are rounded to fp32: another choice is right where the keys differ by a rounding
        same = (idx == ref_idx).all(1)
        for t in np.nonzero(~same)[0]:
            keys = np.exp(x[t]) / np.exp(x[t]).sum() if r["score"] == "softmax" else 1 / (1 + np.exp(-x[t]))
            keys = keys + (0 if bias is None else bias)
            assert np.abs(np.sort(keys[idx[t]])[::-1] - np.sort(keys[ref_idx[t]])[::-1]).max() <= 128 * U, t
        assert same.mean() > 0.9
        ref_w = np.where(same[:, None], ref_w, w)
    assert (np.abs(w - ref_w) <= 128 * U * np.abs(ref_w)).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("G", [1, 4])
def test_route_masks_and_special_values(c3, score, G):
    E, k = 16, 4
    r = dict(E=E, k=k, score=score, G=G, keep=max(1, G // 2), renorm=True)
    rng = np.random.default_rng(3)
    x = grid_logits(rng, 9, E)
    x[0] = -np.inf                                   # nothing is left
    x[1, :] = -np.inf
    x[1, 5] = 1.0                                    # one is left
    x[2, :] = np.finfo(np.float32).min               # a mask of the lowest value: still eligible, all tied
    x[3, ::2] = -np.inf
    x[4, 3] = np.nan
    x[5, :] = 0.0
    x[5, 7] = -0.0                                   # ties with +0: the lowest number wins
    x[6, 2:] = -np.inf
    x[7, :] = -200.0 if score == "sigmoid" else 3.0  # every sigmoid is 0 in fp32
    idx, w, _, _ = run_route(c3, r, x, 0)
    ref_idx, ref_w = route_oracle(x, E, k, score, **oracle_args(r))
    if score == "sigmoid":
        # 1 / (1 + exp(200)) is not zero in 64 bits: the definition's zero sum is meant in fp32
        ref_idx[7], ref_w[7] = ref_idx[5], 0.0
        ref_idx[2], ref_w[2] = ref_idx[5], 0.0
    assert np.array_equal(idx.cpu().numpy(), ref_idx)
    w = f64(w)
    assert np.array_equal(np.isnan(w), np.isnan(ref_w))
    fine = ~np.isnan(ref_w)
    assert (np.abs(w - ref_w)[fine] <= 128 * U * np.abs(ref_w)[fine]).all()


def test_route_bias_can_mask(c3):
    E, k = 12, 3
    x = grid_logits(np.random.default_rng(0), 5, E)
    bias = np.zeros(E)
    bias[::2] = -np.inf
    bias[1] = np.nan
    for score in ("softmax", "sigmoid"):
        r = dict(E=E, k=k, score=score)
        idx, w, _, _ = run_route(c3, r, x, 0, bias)
        idx = idx.cpu().numpy()
        assert (idx % 2 == 1).all() and (idx != 1).all()
        assert np.isfinite(f64(w)).all()


def route_grad_oracle(x, idx, dw, r):
    """d sum(w dw) / dx by the formulas, 64 bits."""
    T, E = x.shape
    dx = np.zeros((T, E))
    c = r.get("scale", 1.0)
    for t in range(T):
        sel = idx[t][idx[t] >= 0]
        g = c * dw[t][idx[t] >= 0]
        if not len(sel):
            continue
        if r["score"] == "softmax":
            pool = sel if r.get("renorm") else np.nonzero(x[t] > -np.inf)[0]
            p = np.zeros(E)
            e = np.exp(x[t, pool] - x[t, pool].max())
            p[pool] = e / e.sum()
            full = np.zeros(E)
            full[sel] = g
            dx[t] = p * (full - (p * full).sum())
        else:
            s = 1 / (1 + np.exp(-x[t, sel]))
            d = g
            if r.get("renorm"):
                d = (g - (g * s).sum() / s.sum()) / s.sum()
            dx[t, sel] = d * s * (1 - s)
    return dx


@pytest.mark.parametrize("ty", [0, 1])
@pytest.mark.parametrize("r", ROUTERS, ids=lambda r: "_".join(f"{k}{v}" for k, v in r.items()))
def test_route_backward(c3, r, ty):
    rng = np.random.default_rng(r["E"])
    T, E, k = 19, r["E"], r["k"]
    x = grid_logits(rng, T, E)
    if E > 8:
        x[3, : E - k - 1] = -np.inf
        x[4] = -np.inf
    bias = rng.integers(-8, 9, E) / 16.0 if r.get("bias") else None
    idx, w, router, wide = run_route(c3, r, x, ty, bias, extra=3)
    dw = rng.standard_normal((T, k)).astype(np.float32)
    dx = Guarded((T, E + 2), TD[ty], 5.0)
    c3.c3_route_backward(router, wide, E + 3, T, idx, cuda(dw), dx.t, E + 2)
    torch.cuda.synchronize()
    assert dx.intact()
    got = f64(dx.t)
    assert (got[:, E:] == 5.0).all()
    got = got[:, :E]
    ref = route_grad_oracle(x, idx.cpu().numpy(), dw.astype(np.float64), r)
    # s (1 - s) and the differences lose up to a few u of the largest term |c dw| <= 4 c
    tol = 256 * U * 4 * r.get("scale", 1.0)
    if r["score"] == "sigmoid" and r.get("renorm"):
        s = np.where(idx.cpu().numpy() >= 0, 1 / (1 + np.exp(-np.take_along_axis(x, np.maximum(idx.cpu().numpy(), 0), 1))), 0)
        tol = tol / np.maximum(s.sum(1, keepdims=True), 1e-3)
    if ty:
        tol = tol + H * np.abs(ref)  # the output's own rounding
    assert (np.abs(got - ref) <= tol).all()
    # and against differences of the weights themselves, along a direction
    v = rng.standard_normal((T, E))
    step = 1e-5
    sel = idx.cpu().numpy()

    def weights(z):
        out = np.zeros((T, k))
        for t in range(T):
            on = sel[t] >= 0
            if not on.any():
                continue
            if r["score"] == "softmax":
                pool = sel[t][on] if r.get("renorm") else np.arange(E)
                e = np.exp(z[t] - z[t, pool].max())
                out[t, on] = e[sel[t][on]] / e[pool].sum()
            else:
                s = 1 / (1 + np.exp(-z[t, sel[t][on]]))
                out[t, on] = s / s.sum() if r.get("renorm") else s
        return out * r.get("scale", 1.0)

    live = np.where(x > -np.inf, v, 0.0)
    with np.errstate(invalid="ignore"):
        slope = ((weights(x + step * live) - weights(x - step * live)) * dw).sum(1) / (2 * step)
    along = (got * live).sum(1)
    room = (np.abs(live) * (tol + np.zeros_like(got))).sum(1) + 1e-7 * np.abs(dw).sum(1) * 16
    assert (np.abs(slope - along) <= room).all()


SMALL = [
    dict(E=1, k=1, score="softmax"),
    dict(E=5, k=2, score="sigmoid", renorm=True, bias=True),
    dict(E=8, k=8, score="softmax", renorm=True, scale=2.5),
    dict(E=60, k=6, score="softmax"),
    dict(E=64, k=8, score="sigmoid"),
    dict(E=33, k=3, score="softmax", bias=True),
    dict(E=128, k=16, score="softmax", renorm=True),
    dict(E=64, k=6, score="sigmoid", G=4, keep=2, best=2, renorm=True, bias=True),
    dict(E=256, k=8, score="sigmoid", G=8, keep=4, best=2, bias=True, scale=2.5),
    dict(E=250, k=12, score="softmax", G=2, keep=1),
    dict(E=100, k=4, score="sigmoid", G=25, keep=3),
]


@pytest.mark.parametrize("ty", [0, 1])
@pytest.mark.parametrize("T", [8192, 8237])
@pytest.mark.parametrize("r", SMALL, ids=lambda r: "_".join(f"{k}{v}" for k, v in r.items()))
def test_route_many_tokens(c3, r, T, ty):
    """Many tokens share a warp where few do not (below 4096): the same results, and the definition's."""
    rng = np.random.default_rng(T + r["E"])
    E, k = r["E"], r["k"]
    x = grid_logits(rng, T, E)
    x[5] = -np.inf
    x[6, : E // 2] = -np.inf
    x[7, E - 1] = np.nan
    x[8] = 0.0
    x[T - 1, 0] = -0.0
    bias = rng.integers(-8, 9, E) / 16.0 if r.get("bias") else None
    idx, w, router, wide = run_route(c3, r, x, ty, bias, extra=3)
    few_idx, few_w = torch.empty_like(idx), torch.empty_like(w)
    for at in range(0, T, 4095):
        n = min(4095, T - at)
        c3.c3_route(router, wide[at:], E + 3, n, few_idx[at:], few_w[at:])
    dw = cuda(rng.standard_normal((T, k)).astype(np.float32))
    dx, few_dx = Guarded((T, E + 1), TD[ty], 5.0), torch.full((T, E + 1), 5.0, dtype=TD[ty], device="cuda")
    c3.c3_route_backward(router, wide, E + 3, T, idx, dw, dx.t, E + 1)
    for at in range(0, T, 4095):
        n = min(4095, T - at)
        c3.c3_route_backward(router, wide[at:], E + 3, n, idx[at:], dw[at:], few_dx[at:], E + 1)
    torch.cuda.synchronize()
    assert dx.intact() and bool((dx.t[:, E:] == 5.0).all())
    by_logit = r["score"] == "softmax" and bias is None and r.get("best", 1) == 1
    if by_logit or r["score"] == "sigmoid":   # keys that no sum over the row enters
        assert torch.equal(idx, few_idx)
    same = (idx == few_idx).all(1)
    assert bool(same.float().mean() > 0.99)
    # both forms are 128 u off the definition at most (weights), 256 u of the largest term (gradients)
    fine = same & ~torch.isnan(few_w).any(1)
    assert torch.equal(torch.isnan(w[same]), torch.isnan(few_w[same]))
    assert bool(((w - few_w)[fine].abs() <= 256 * U * few_w[fine].abs()).all())
    some = np.r_[0:40, T - 40:T]
    ref_idx, ref_w = route_oracle(x[some], E, k, r["score"], bias, **oracle_args(r))
    got_idx, got_w = idx.cpu().numpy()[some], f64(w)[some]
    if by_logit:
        assert np.array_equal(got_idx, ref_idx)
    rows = (got_idx == ref_idx).all(1)
    assert rows.mean() > 0.9
    assert np.array_equal(np.isnan(got_w[rows]), np.isnan(ref_w[rows]))
    err = np.abs(got_w - ref_w)[rows]
    assert (err[~np.isnan(err)] <= (128 * U * np.abs(ref_w)[rows])[~np.isnan(err)]).all()
    some = some[(some != 7)]
    ref = route_grad_oracle(x[some], idx.cpu().numpy()[some], dw.cpu().numpy().astype(np.float64)[some], r)
    tol = 256 * U * 4 * r.get("scale", 1.0)
    if r["score"] == "sigmoid" and r.get("renorm"):
        sel = idx.cpu().numpy()[some]
        s = np.where(sel >= 0, 1 / (1 + np.exp(-np.take_along_axis(x[some], np.maximum(sel, 0), 1))), 0)
        tol = tol / np.maximum(s.sum(1, keepdims=True), 1e-3)
    if ty:
        tol = tol + H * np.abs(ref)
    assert (np.abs(f64(dx.t)[some, :E] - ref) <= tol).all()
    other = torch.ones(T, dtype=torch.bool, device="cuda")
    other[7] = False
    a, b = dx.t.float()[other], few_dx.float()[other]
    assert bool(((a - b).abs() <= 2 * 256 * U * 4 * r.get("scale", 1.0) * (20 if r.get("renorm") else 1) + 2 * H * b.abs()).all())


# Twelve experts a lane of 32, 16 and 8 lanes (the last two with many tokens), whole and
# ragged, rows of whole vectors and not.
TWELVE = [
    dict(E=384, k=8, score="sigmoid", G=8, keep=4, best=2, renorm=True, bias=True),
    dict(E=384, k=8, score="softmax", G=6, keep=2),
    dict(E=371, k=8, score="sigmoid", renorm=True, bias=True),
    dict(E=372, k=9, score="softmax"),
    dict(E=360, k=4, score="softmax", renorm=True),
    dict(E=192, k=8, score="sigmoid", G=4, keep=2, best=2, bias=True),
    dict(E=189, k=12, score="softmax"),
    dict(E=180, k=16, score="sigmoid", renorm=True),
    dict(E=96, k=8, score="sigmoid", G=4, keep=2, best=2, bias=True),
    dict(E=95, k=3, score="softmax"),
    dict(E=88, k=8, score="sigmoid", renorm=True, bias=True),
]


@pytest.mark.parametrize("ty", [0, 1])
@pytest.mark.parametrize("T,extra", [(1, 0), (77, 5), (33, 8)])
@pytest.mark.parametrize("r", TWELVE, ids=lambda r: "_".join(f"{k}{v}" for k, v in r.items()))
def test_route_twelve_a_lane(c3, r, T, extra, ty):
    test_route(c3, r, T, extra, ty)


@pytest.mark.parametrize("ty", [0, 1])
@pytest.mark.parametrize("extra", [0, 3, 8])
@pytest.mark.parametrize("r", TWELVE, ids=lambda r: "_".join(f"{k}{v}" for k, v in r.items()))
def test_route_twelve_many_tokens(c3, r, extra, ty):
    T, E, k = 4101, r["E"], r["k"]
    rng = np.random.default_rng(E + extra)
    x = grid_logits(rng, T, E)
    x[rng.random((T, E)) < 0.05] = -np.inf
    bias = rng.integers(-8, 9, E) / 16.0 if r.get("bias") else None
    idx, w, router, wide = run_route(c3, r, x, ty, bias, extra)
    some = rng.choice(T, 200, replace=False)
    few_idx, few_w, _, _ = run_route(c3, r, x[some], ty, bias, extra)  # a whole warp a token
    same = (idx[some] == few_idx).all(1)
    if r["score"] == "sigmoid" or bias is None:  # the keys do not depend on the number of lanes
        assert same.all()
    a, b = f64(w)[some], f64(few_w)
    assert (np.abs(a - b)[same.cpu().numpy()] <= 128 * U * np.abs(b)[same.cpu().numpy()]).all()
    ref_idx, ref_w = route_oracle(x[some], E, k, r["score"], bias, **oracle_args(r))
    hit = (few_idx.cpu().numpy() == ref_idx).all(1)
    assert hit.mean() > 0.9
    assert (np.abs(a - ref_w) <= 128 * U * np.abs(ref_w))[hit].all()


# Groups that are a power of two in number and no power of two in size: a run of lanes each, the last not full.
RAGGED_GROUPS = [
    dict(E=160, k=6, score="sigmoid", G=8, keep=3, best=2, renorm=True, bias=True),
    dict(E=488, k=4, score="sigmoid", G=4, keep=1, best=2, bias=True),
    dict(E=200, k=8, score="softmax", G=4, keep=2),
    dict(E=24, k=3, score="sigmoid", G=8, keep=2, best=2, bias=True),
    dict(E=34, k=6, score="softmax", G=2, keep=1),
    dict(E=96, k=5, score="sigmoid", G=32, keep=7, best=2, bias=True),
    dict(E=1000, k=8, score="sigmoid", G=8, keep=3, best=2, renorm=True, bias=True),
    dict(E=104, k=8, score="softmax", G=8, keep=3, renorm=True),
]


@pytest.mark.parametrize("ty", [0, 1])
@pytest.mark.parametrize("T,extra", [(1, 0), (77, 5), (33, 8)])
@pytest.mark.parametrize("r", RAGGED_GROUPS, ids=lambda r: "_".join(f"{k}{v}" for k, v in r.items()))
def test_route_ragged_groups(c3, r, T, extra, ty):
    test_route(c3, r, T, extra, ty)


@pytest.mark.parametrize("ty", [0, 1])
@pytest.mark.parametrize("extra", [0, 3, 8])
@pytest.mark.parametrize("r", RAGGED_GROUPS, ids=lambda r: "_".join(f"{k}{v}" for k, v in r.items()))
def test_route_ragged_groups_many_tokens(c3, r, extra, ty):
    test_route_twelve_many_tokens(c3, r, extra, ty)


# ----------------------------------------------------------------------------- order

def order_oracle(idx, E, rows):
    T, k = idx.shape
    flat = idx.reshape(-1)
    counts = np.array([(flat == e).sum() for e in range(E)])
    offsets = np.concatenate([[0], np.cumsum((counts + 127) // 128 * 128)])
    slot = np.full(T * k, -1)
    row_of = np.full(rows, -1)
    seen = np.zeros(E, int)
    for i, e in enumerate(flat):
        if 0 <= e < E:
            slot[i] = offsets[e] + seen[e]
            row_of[slot[i]] = i // k
            seen[e] += 1
    return slot.reshape(T, k), row_of, offsets, counts


@pytest.mark.parametrize("T,k,E", [(0, 2, 4), (1, 1, 1), (3, 2, 5), (100, 4, 7), (513, 8, 256), (4096, 1, 3),
                                   (2000, 3, 1024), (5000, 6, 60), (20011, 2, 33),
                                   (8192, 8, 16), (8193, 8, 16), (70001, 1, 1000), (40000, 3, 7)])
def test_order(c3, T, k, E):
    rng = np.random.default_rng(T + E)
    idx = rng.integers(-1, E, (T, k))
    if T > 50:
        idx[7, 0] = E       # outside: takes no row
        idx[8, 0] = -5
        idx[10:40] = 0      # a run of one expert
    rows = c3.c3_moe_rows(T, k, E) + 37
    slot, row_of = Guarded((T, k), torch.int32, -9), Guarded((rows,), torch.int32, -9)
    offsets, counts = Guarded((E + 1,), torch.int32, -9), Guarded((E,), torch.int32, -9)
    work = torch.empty(max(4, c3.c3_moe_order_bytes(T, k, E)), dtype=torch.uint8, device="cuda")
    c3.c3_moe_order(cuda(idx.astype(np.int32)), T, k, E, slot.t, row_of.t, rows, offsets.t, counts.t, work)
    torch.cuda.synchronize()
    for got, want in zip((slot, row_of, offsets, counts), order_oracle(idx, E, rows)):
        assert got.intact()
        assert np.array_equal(got.t.cpu().numpy(), want)


# ----------------------------------------------------------------------------- 4-bit matrices

def e4m3(v):
    """fp32 values >= 0 to e4m3, nearest even, at most 448 (and the byte)."""
    v = np.minimum(v.astype(np.float64), 448.0)
    with np.errstate(divide="ignore"):
        e = np.clip(np.floor(np.log2(np.maximum(v, 1e-300))), -6, 8)
    u = 2.0 ** (e - 3)
    n = np.round(v / u)                     # numpy rounds halves to even
    carry = n == 16
    e, n = np.where(carry, e + 1, e), np.where(carry, 8, n)
    byte = np.where(n >= 8, (e + 7) * 8 + n - 8, n)
    return n * 2.0 ** (e - 3), byte.astype(np.uint8)


def quantise_oracle(x, fmt, g=None):
    """x float32 [R, C] -> (codes [R, pitch], scale bytes [R, nb], values float64 [R, C])."""
    B = 16 if fmt else 32
    R, C = x.shape
    nb = -(-C // B)
    y = np.zeros((R, nb * B), np.float32)
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        y[:, :C] = x if g is None else x * (np.float32(1) / np.float32(g))
        y = y.reshape(R, nb, B)
        amax = np.abs(y).max(-1)
        bad = ~np.isfinite(y).all(-1)
        amax = np.where(bad, 1, amax).astype(np.float32)
        if fmt == 0:
            m, e = np.frexp(amax.astype(np.float64))
            e = np.where(amax == 0, -127, np.maximum(np.where(m <= 0.75, e - 3, e - 2), -127))
            scale, byte = 2.0 ** e, (e + 127).astype(np.uint8)
            q = y.astype(np.float64) / scale[..., None]
        else:
            scale, byte = e4m3(amax / np.float32(6))
            q = np.where(scale[..., None] > 0, y / np.where(scale > 0, scale, 1).astype(np.float32)[..., None], 0)
            q = q.astype(np.float64)
    byte = np.where(bad, 0x7F if fmt else 0xFF, byte).astype(np.uint8)
    mid = (GRID[1:] + GRID[:-1]) / 2
    a = np.abs(np.nan_to_num(q, nan=0.0, posinf=1e9, neginf=-1e9))
    code = np.searchsorted(mid, a, side="left")
    tie = (code < 7) & (a == mid[np.minimum(code, 6)]) & (code % 2 == 1)
    code = code + tie
    neg = np.signbit(q)
    value = GRID[code] * np.where(neg, -1, 1) * np.where(bad, np.nan, scale)[..., None]
    value = value.reshape(R, -1)[:, :C]
    if g is not None:
        value = value * np.float64(np.float32(g))
    code = (code + 8 * neg).reshape(R, -1)
    code = np.concatenate([code, np.zeros((R, -code.shape[1] % 32), code.dtype)], 1)
    return (code[:, 0::2] + 16 * code[:, 1::2]).astype(np.uint8), byte, value, np.repeat(bad, B, 1)


def read_tiles(scales, R, nb):
    """Scale bytes [R, nb] out of tiles [row tiles, k tiles, 512], and what lies past nb."""
    r = np.arange(R)[:, None]
    b = np.arange(scales.shape[1] * 4)
    all_b = scales[r // 128, b // 4, r % 32 * 16 + r % 128 // 32 * 4 + b % 4]
    return all_b[:, :nb], all_b[:, nb:]


def new_fp4(c3, R, C, fmt, g=None, count=1):
    kt = -(-C // (64 if fmt else 128))
    codes = Guarded((count, R, -(-C // 32) * 16), torch.uint8, 0xEE)
    scales = Guarded((count, -(-R // 128), kt, 512), torch.uint8, 0xEE)
    assert codes.t[0].numel() == c3.c3_fp4_code_bytes(R, C)
    assert scales.t[0].numel() == c3.c3_fp4_scale_bytes(R, C, fmt)
    tg = None if g is None else cuda(np.asarray(g, np.float32).reshape(-1))
    q = c3.Fp4(R, C, fmt, codes.t, scales.t, tg, count=count)
    return q, codes, scales


def values(rng, R, C, ty):
    x = rng.standard_normal((R, C)) * np.exp2(rng.integers(-6, 7, (R, 1)))
    x[:, ::7] *= 20
    x[R // 2] = 0
    if C > 40:
        x[0, :40] = np.repeat([6, 5, 2.5, 0.25, 0.75, 1.25, 3.5, -5], 5)   # every tie
    t = cuda(x.astype(np.float32)).to(TD[ty])
    return t, t.float().cpu().numpy()


SIZES = [(1, 1), (1, 32), (3, 17), (5, 33), (33, 130), (130, 64), (257, 1000), (64, 129), (128, 4096)]


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("ty", [0, 1])
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("R,C", SIZES)
def test_quantise(c3, R, C, fmt, ty, transpose):
    rng = np.random.default_rng(R * 7 + C)
    t, x = values(rng, R, C, ty)
    for extra, shift, g in ((0, 0, None), (3, 1, 0.37 if fmt else None), (8, 0, 1e-3 if fmt else None)):
        src = t.t().contiguous() if transpose else t
        rows, cols = src.shape
        buf = torch.full((rows * (cols + extra) + shift,), 1e30, dtype=TD[ty], device="cuda")
        view = buf[shift:].view(rows, cols + extra)
        view[:, :cols] = src
        q, codes, scales = new_fp4(c3, R, C, fmt, g)
        c3.c3_fp4_quantize(view, ty, rows, cols, q, ld=cols + extra, transpose=transpose)
        torch.cuda.synchronize()
        assert codes.intact() and scales.intact()
        ref_codes, ref_bytes, ref_v, _ = quantise_oracle(x, fmt, g)
        assert np.array_equal(codes.t[0].cpu().numpy(), ref_codes)
        got, past = read_tiles(scales.t[0].cpu().numpy(), R, ref_bytes.shape[1])
        assert np.array_equal(got, ref_bytes)
        assert (past == 0).all()
        for out in (0, 1):
            o = Guarded((R, C + 5), TD[out], 3.0)
            c3.c3_fp4_dequantize(q, o.t, out, C + 5)
            torch.cuda.synchronize()
            assert o.intact() and bool((o.t[:, C:] == 3.0).all())
            want = torch.from_numpy(ref_v.astype(np.float32)).to(TD[out]).float().numpy()
            assert np.array_equal(o.t[:, :C].float().cpu().numpy(), want)


@pytest.mark.parametrize("ty", [0, 1])
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("R,C", [(1, 5), (1, 16), (2, 47), (33, 128), (70, 333), (300, 1040)])
def test_quantise_rows_of_any_alignment(c3, R, C, gather, fmt, ty):
    """Rows that start anywhere, NaNs around them: the codes and scales of the same rows aligned."""
    rng = np.random.default_rng(R * 3 + C)
    g = 0.125 if fmt else None
    x = values(rng, R, C, ty)[0]
    wide = torch.full((R, C + 8 + -C % 8), float("nan"), dtype=TD[ty], device="cuda")
    wide[:, :C] = x
    row_of = torch.randint(-1, R, (R,), dtype=torch.int32, device="cuda") if gather else None
    for shift in range(8):
        for ld in range(C, C + 5):
            results = []
            flat = torch.full((shift + R * ld,), float("nan"), dtype=TD[ty], device="cuda")
            odd = flat[shift:].view(R, ld)
            odd[:, :C] = x
            for src, pitch in ((wide, wide.shape[1]), (odd, ld)):
                q, codes, scales = new_fp4(c3, R, C, fmt, g)
                c3.c3_fp4_quantize(src, ty, R, C, q, ld=pitch, row_of=row_of)
                torch.cuda.synchronize()
                results.append((codes.t.clone(), scales.t.clone()))
            assert torch.equal(results[0][0], results[1][0]) and torch.equal(results[0][1], results[1][1]), (shift, ld)


@pytest.mark.parametrize("ty", [0, 1])
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("R", [1, 2, 63, 65, 130, 257])
@pytest.mark.parametrize("C", [5, 128, 300])
def test_quantise_transposed_is_the_transpose_quantised(c3, R, C, fmt, ty):
    """Rows in pairs and singly, an odd last one, NaNs beside the columns."""
    rng = np.random.default_rng(R + 1000 * C)
    g = 0.3 if fmt else None
    x = values(rng, R, C, ty)[0]
    for count in (1, 2):
        want, codes, scales = new_fp4(c3, R, C, fmt, [g] * count if fmt else None, count=count)
        c3.c3_fp4_quantize(torch.stack([x] * count), ty, R, C, want)
        for ld, shift in ((R, 0), (R + 1, 0), (R + 2, 1), (R + 3, 2)):
            flat = torch.full((shift + count * C * ld,), float("nan"), dtype=TD[ty], device="cuda")
            view = flat[shift:].view(count, C, ld)
            view[:, :, :R] = x.t()
            q, c2, s2 = new_fp4(c3, R, C, fmt, [g] * count if fmt else None, count=count)
            c3.c3_fp4_quantize(view, ty, C, R, q, ld=ld, transpose=True)
            torch.cuda.synchronize()
            assert c2.intact() and s2.intact()
            assert torch.equal(c2.t, codes.t) and torch.equal(s2.t, scales.t), (ld, shift, count)


def test_quantise_every_nv_scale(c3):
    """Each e4m3 scale with each tie between codes and its neighbours in fp32; and maxima around the scales' own ties."""
    bits = np.arange(1, 127)
    s = np.where(bits < 8, bits * 2.0 ** -9, (8 + bits % 8) * 2.0 ** (bits // 8 - 10)).astype(np.float32)
    ties = np.float32([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 6])
    x = []
    for way in (0, -np.inf, np.inf):
        t = s[:, None] * ties[None]
        x.append(t if way == 0 else np.nextafter(t, np.float32(way)))
        x[-1][:, -1] = 6 * s
    # 16 columns: eight ties and their negatives, without the maximum's
    blocks = np.concatenate([np.concatenate([b, -b], 1) for b in x])
    mid = np.float32(6) * (s[1:] + s[:-1]) / 2
    peaks = np.concatenate([mid, np.nextafter(mid, np.float32(np.inf)), np.nextafter(mid, np.float32(0)),
                            np.float32([1e-45, 1e-38, 6 * 2.0 ** -11, 6 * 2.0 ** -10, 5.9 * 2.0 ** -10, 3e38, 2688, 2800])])
    more = np.zeros((len(peaks), 16), np.float32)
    more[:, 3] = peaks
    more[:, 5] = -peaks / 2
    x = np.concatenate([blocks, more]).astype(np.float32)
    R, C = x.shape
    for transpose in (False, True):
        q, codes, scales = new_fp4(c3, R, C, 1)
        src = cuda(np.ascontiguousarray(x.T) if transpose else x)
        c3.c3_fp4_quantize(src, 0, src.shape[0], src.shape[1], q, transpose=transpose)
        torch.cuda.synchronize()
        ref_codes, ref_bytes, _, _ = quantise_oracle(x, 1)
        assert np.array_equal(read_tiles(scales.t[0].cpu().numpy(), R, 1)[0], ref_bytes)
        assert np.array_equal(codes.t[0].cpu().numpy(), ref_codes)


@pytest.mark.parametrize("ty", [0, 1])
@pytest.mark.parametrize("fmt", [0, 1])
def test_quantise_special_values(c3, fmt, ty):
    x = np.ones((6, 64), np.float32)
    x[0, 3] = np.nan
    x[1, 40] = np.inf
    x[2, 33] = -np.inf
    x[3] = 1e-44                       # subnormal
    x[4] = np.finfo(np.float32).max
    x[5, :32] = 0
    x[5, 5] = -0.0
    x[5, 32:] = np.repeat([6, 5, 2.5, 0.25, 0.75, 1.25, 3.5, -5], 4)
    q, codes, scales = new_fp4(c3, 6, 64, fmt)
    if ty:
        x[4] = 3.3e38
    t = cuda(x).to(TD[ty])
    x = t.float().cpu().numpy()
    c3.c3_fp4_quantize(t, ty, 6, 64, q)
    o = torch.empty(6, 64, device="cuda")
    c3.c3_fp4_dequantize(q, o, 0, 64)
    torch.cuda.synchronize()
    ref_codes, ref_bytes, ref_v, bad = quantise_oracle(x, fmt)
    got, _ = read_tiles(scales.t[0].cpu().numpy(), 6, ref_bytes.shape[1])
    assert np.array_equal(got, ref_bytes)
    o = o.cpu().numpy()
    assert np.array_equal(np.isnan(o), bad[:, :64])
    assert np.array_equal(o[~np.isnan(o)], ref_v.astype(np.float32)[~np.isnan(o)])


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("transpose", [False, True])
def test_quantise_several_matrices(c3, fmt, transpose):
    rng = np.random.default_rng(5)
    R, C, n = 70, 200, 3
    x = rng.standard_normal((n, R, C)).astype(np.float32)
    g = [0.5, 0.1, 2.0] if fmt else None
    q, codes, scales = new_fp4(c3, R, C, fmt, g, count=n)
    src = cuda(x.transpose(0, 2, 1) if transpose else x)
    c3.c3_fp4_quantize(src, 0, C if transpose else R, R if transpose else C, q, transpose=transpose)
    back = torch.empty(n, R, C, device="cuda")
    c3.c3_fp4_dequantize(q, back, 0, C)
    torch.cuda.synchronize()
    assert codes.intact() and scales.intact()
    for i in range(n):
        ref_codes, ref_bytes, ref_v, _ = quantise_oracle(x[i], fmt, g[i] if g else None)
        assert np.array_equal(codes.t[i].cpu().numpy(), ref_codes)
        assert np.array_equal(read_tiles(scales.t[i].cpu().numpy(), R, ref_bytes.shape[1])[0], ref_bytes)
        assert np.array_equal(back[i].cpu().numpy(), ref_v.astype(np.float32))


@pytest.mark.parametrize("ty", [0, 1])
def test_quantise_gathers_rows(c3, ty):
    rng = np.random.default_rng(9)
    T, C, R = 50, 97, 300
    t, x = values(rng, T, C, ty)
    row_of = rng.integers(0, T, R)
    row_of[::5] = -1
    row_of[3], row_of[4] = T, 1 << 30   # outside
    q, codes, scales = new_fp4(c3, R, C, 0)
    c3.c3_fp4_quantize(t, ty, T, C, q, row_of=cuda(row_of.astype(np.int32)))
    torch.cuda.synchronize()
    assert codes.intact() and scales.intact()
    have = (row_of >= 0) & (row_of < T)
    ref_codes, ref_bytes, _, _ = quantise_oracle(x[np.where(have, row_of, 0)], 0)
    got = codes.t[0].cpu().numpy()
    assert np.array_equal(got[have], ref_codes[have])
    assert (got[~have] == 0xEE).all()
    assert np.array_equal(read_tiles(scales.t[0].cpu().numpy(), R, ref_bytes.shape[1])[0][have], ref_bytes[have])


# ----------------------------------------------------------------------------- products

def random_fp4(c3, rng, R, C, fmt, g=None, count=1, spread=3):
    """A matrix of random codes and scales, and its values (float64)."""
    q, codes, scales = new_fp4(c3, R, C, fmt, g, count)
    B = 16 if fmt else 32
    code = rng.integers(0, 16, (count, R, -(-C // 32) * 32))
    code[:, :, C:] = 0
    codes.t.copy_(cuda((code[..., 0::2] + 16 * code[..., 1::2]).astype(np.uint8)))
    # padding rows of a tile hold NaN scales: they must not matter
    s = np.full(tuple(scales.t.shape), 0x7F if fmt else 0xFF, np.uint8)
    kb = s.shape[2] * 4
    nb = -(-C // B)
    byte = (rng.integers(127 - spread, 128 + spread, (count, R, kb)) if fmt == 0
            else rng.integers(40, 72, (count, R, kb))).astype(np.uint8)
    byte[:, :, nb:] = 0
    r, b = np.arange(R)[:, None], np.arange(kb)
    for i in range(count):
        s[i][r // 128, b // 4, r % 32 * 16 + r % 128 // 32 * 4 + b % 4] = byte[i]
    scales.t.copy_(cuda(s))
    v = np.concatenate([GRID, -GRID])[code[:, :, :C]]
    sv = 2.0 ** (byte.astype(np.float64) - 127) if fmt == 0 else np.where(
        byte >= 8, (8 + byte % 8) * 2.0 ** (byte // 8 - 10.0), byte % 8 * 2.0 ** -9)
    v = v * np.repeat(sv, B, 2)[:, :, :C]
    if g is not None:
        v = v * np.asarray(g, np.float32).astype(np.float64).reshape(-1, 1, 1)
    return q, v


def close(got, a, b, out, K):
    ref, mag = a @ b.T, np.abs(a) @ np.abs(b).T
    tol = (K / 64 + 64) * 2 * U * mag + (H * np.abs(ref) if out else 2 * U * np.abs(ref))
    return bool((np.abs(got - ref) <= tol).all())


@pytest.mark.parametrize("out", [0, 1])
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("M,N,K,budget", [
    (1, 1, 1, 0), (1, 128, 64, 0), (7, 5, 33, 0), (128, 128, 256, 0), (129, 127, 257, 0), (16, 1000, 520, 0),
    (300, 200, 1000, 0), (512, 640, 768, 3), (255, 513, 96, 1), (200, 264, 4104, 0), (64, 4096, 2048, 0),
    (1000, 1032, 130, 0), (13, 384, 8072, 0), (2100, 520, 320, 0), (500, 1600, 2000, 0),
    # few rows, long K, more tiles than would be split: every ring goes round several times
    (128, 20000, 2304, 0), (64, 20000, 2304, 0), (20, 20000, 2304, 0), (100, 300, 9000, 2), (50, 300, 9000, 1),
    (1100, 400, 9000, 4)])
def test_product(c3, M, N, K, budget, fmt, out):
    rng = np.random.default_rng(M + N + K)
    a, va = random_fp4(c3, rng, M, K, fmt, 0.75 if fmt else None)
    b, vb = random_fp4(c3, rng, N, K, fmt, 0.3 if fmt else None)
    C = Guarded((M, N), TD[out], float("nan"))
    c3.c3_fp4_gemm(a, b, C.t, out, sm_budget=budget)
    c3.c3_status_check()
    assert C.intact()
    assert close(f64(C.t), va[0], vb[0], out, K)


def test_product_is_exact_where_fp32_is(c3):
    """Unit scales: every partial sum is a multiple of 1/4 below 2^22, so any order gives the same."""
    rng = np.random.default_rng(1)
    M, N, K = 200, 328, 1000
    a, va = random_fp4(c3, rng, M, K, 0, spread=0)
    b, vb = random_fp4(c3, rng, N, K, 0, spread=0)
    C = torch.empty(M, N, device="cuda")
    c3.c3_fp4_gemm(a, b, C, 0)
    c3.c3_status_check()
    assert np.array_equal(f64(C), va[0] @ vb[0].T)


@pytest.mark.parametrize("fmt", [0, 1])
def test_product_carries_nan_blocks(c3, fmt):
    M, N, K = 140, 130, 300
    x = np.ones((M, K), np.float32)
    x[3, 7] = np.nan
    x[139, 299] = np.inf
    w = np.ones((N, K), np.float32)
    w[128, 0] = -np.inf
    a, _, _ = new_fp4(c3, M, K, fmt)
    b, _, _ = new_fp4(c3, N, K, fmt)
    c3.c3_fp4_quantize(cuda(x), 0, M, K, a)
    c3.c3_fp4_quantize(cuda(w), 0, N, K, b)
    C = torch.empty(M, N, device="cuda")
    c3.c3_fp4_gemm(a, b, C, 0)
    c3.c3_status_check()
    nan = np.zeros((M, N), bool)
    nan[3], nan[139], nan[:, 128] = True, True, True
    C = C.cpu().numpy()
    assert np.array_equal(np.isnan(C), nan)
    assert np.allclose(C[~nan], K, rtol=0.1)   # ones become 6/6, 4 * .25 or the like


def test_an_injected_launch_failure_is_reported_once(c3):
    rng = np.random.default_rng(3)
    for M in (16, 300):   # both forms of the product
        a, va = random_fp4(c3, rng, M, 128, 0)
        b, vb = random_fp4(c3, rng, 200, 128, 0)
        C = torch.full((M, 200), 7.0, device="cuda")
        c3.c3_inject_fault(c3.C3_FAULT_GEMM_LAUNCH)
        assert c3.c3_fp4_gemm(a, b, C, 0, check=False) == c3.C3_ECUDA
        assert "injected" in c3.c3_last_error()
        torch.cuda.synchronize()
        assert bool((C == 7.0).all())
        c3.c3_fp4_gemm(a, b, C, 0)
        c3.c3_status_check()
        assert close(f64(C), va[0], vb[0], 0, 128)


def test_product_gradients_are_products(c3):
    """dA = dC B and dB = dC^T A through transposed operands, against the formula on the quantised values."""
    rng = np.random.default_rng(2)
    M, N, K = 96, 80, 160
    A, B, D = (rng.standard_normal(s).astype(np.float32) for s in ((M, K), (N, K), (M, N)))

    def quantised(x, transpose):
        R, C = x.shape[::-1] if transpose else x.shape
        q, _, _ = new_fp4(c3, R, C, 1, 0.01)
        c3.c3_fp4_quantize(cuda(x), 0, x.shape[0], x.shape[1], q, transpose=transpose)
        return q, quantise_oracle(x.T.copy() if transpose else x, 1, 0.01)[2]
    for (l, lt), (r, rt), K_ in (((D, False), (B, True), N), ((D, True), (A, True), M)):
        ql, vl = quantised(l, lt)
        qr, vr = quantised(r, rt)
        C = torch.empty(ql.rows, qr.rows, device="cuda")
        c3.c3_fp4_gemm(ql, qr, C, 0)
        c3.c3_status_check()
        assert close(f64(C), vl, vr, 0, K_)


@pytest.mark.parametrize("out", [0, 1])
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("E,N,K,counts,budget", [
    (1, 128, 256, [5], 0), (4, 130, 200, [0, 3, 0, 129], 0), (7, 256, 520, [1, 128, 127, 0, 300, 2, 0], 0),
    (3, 1000, 64, [64, 64, 64], 5), (5, 72, 1030, [0, 0, 0, 0, 1], 0), (2, 512, 300, [0, 0], 0),
    (64, 384, 128, [i % 5 for i in range(64)], 0), (3, 640, 2048, [700, 1, 513], 0),
    (40, 1024, 2304, [1 + i % 70 for i in range(40)], 0), (6, 260, 5000, [3, 0, 130, 65, 1, 2], 2),
    (3, 500, 5000, [400, 300, 513], 6)])
def test_experts_products(c3, E, N, K, counts, budget, fmt, out):
    rng = np.random.default_rng(E + N + K)
    offsets = np.concatenate([[0], np.cumsum([(c + 127) // 128 * 128 for c in counts])]).astype(np.int32)
    R = int(offsets[-1]) + 128
    x, vx = random_fp4(c3, rng, R, K, fmt, 0.5 if fmt else None)
    w, vw = random_fp4(c3, rng, N, K, fmt, rng.uniform(0.1, 2, E) if fmt else None, count=E)
    C = Guarded((R, N), TD[out], 77.0)
    c3.c3_fp4_gemm_experts(x, w, cuda(offsets), cuda(np.array(counts, np.int32)), C.t, out, sm_budget=budget)
    c3.c3_status_check()
    assert C.intact()
    got = f64(C.t)
    mine = np.zeros(R, bool)
    for e, c in enumerate(counts):
        rows = slice(offsets[e], offsets[e] + c)
        mine[rows] = True
        assert close(got[rows], vx[0][rows], vw[e], out, K), e
    assert (got[~mine] == 77.0).all()


@pytest.mark.parametrize("out", [0, 1])
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("E,N,K,counts,budget", [
    (64, 100, 2048, [1] * 20 + [5100] + [2] * 43, 0), (40, 250, 1100, [4900] + [0, 1, 64] * 13, 0),
    (6, 1440, 2690, [26] * 6, 0)])
def test_experts_products_more_tiles_than_clusters(c3, E, N, K, counts, budget, fmt, out):
    """K split over clusters that each do several tiles: an expert has far more rows than the rest."""
    test_experts_products(c3, E, N, K, counts, budget, fmt, out)


def test_experts_products_skip_bad_ranges(c3):
    rng = np.random.default_rng(4)
    E, N, K, R = 5, 128, 128, 512
    x, vx = random_fp4(c3, rng, R, K, 0)
    w, vw = random_fp4(c3, rng, N, K, 0, count=E)
    offsets = np.array([-128, 64, 128, 512, 384, 0], np.int32)
    counts = np.array([10, 10, 20, 1, 129, 0][:E], np.int32)
    C = Guarded((R, N), torch.float32, 77.0)
    c3.c3_fp4_gemm_experts(x, w, cuda(offsets), cuda(counts), C.t, 0)
    c3.c3_status_check()
    assert C.intact()
    got = f64(C.t)
    assert close(got[128:148], vx[0][128:148], vw[2], 0, K)
    got[128:148] = 77.0
    assert (got == 77.0).all()


# ----------------------------------------------------------------------------- combine

@pytest.mark.parametrize("yt,ot", [(0, 0), (0, 1), (1, 0), (1, 1)])
@pytest.mark.parametrize("T,k,cols,shift", [(1, 1, 1, 0), (5, 3, 7, 0), (17, 8, 64, 0), (9, 32, 2056, 0), (40, 2, 4096, 0),
                                            (6, 6, 1000, 1), (300, 4, 136, 0)])
def test_combine(c3, T, k, cols, shift, yt, ot):
    rng = np.random.default_rng(T + cols)
    rows = T * k + 20
    y = rng.standard_normal((rows, cols)).astype(np.float32)
    buf = torch.empty(rows * cols + shift, dtype=TD[yt], device="cuda")
    ty = buf[shift:].view(rows, cols)
    ty.copy_(cuda(y))
    vy = f64(ty)
    slot = rng.permutation(rows)[:T * k].reshape(T, k).astype(np.int32)
    slot[0, 0] = -1
    if T > 4:
        slot[2] = -1                # a token without experts
        slot[3, 0] = rows           # outside
    w = rng.standard_normal((T, k)).astype(np.float32)
    have = (slot >= 0) & (slot < rows)
    sel = np.where(have, slot, 0)
    dslot, dw_ = cuda(slot), cuda(w)
    for weights in (w, None):
        eff = np.where(have, 1.0 if weights is None else weights.astype(np.float64), 0)
        out = Guarded((T, cols), TD[ot], float("nan"))
        c3.c3_moe_combine(ty, yt, rows, cols, dslot, None if weights is None else dw_, T, k, out.t, ot)
        torch.cuda.synchronize()
        assert out.intact()
        ref = (eff[..., None] * vy[sel]).sum(1)
        mag = (np.abs(eff)[..., None] * np.abs(vy[sel])).sum(1)
        assert (np.abs(f64(out.t) - ref) <= k * 2 * U * mag + (H * np.abs(ref) if ot else 0)).all()
        # backward: dout in `ot`, dy in `yt`
        d = cuda(rng.standard_normal((T, cols)).astype(np.float32)).to(TD[ot])
        vd = f64(d)
        dy = Guarded((rows, cols), TD[yt], 9.0)
        dwt = Guarded((T, k), torch.float32, float("nan"))
        c3.c3_moe_combine_backward(d, ot, ty, yt, rows, cols, dslot, None if weights is None else dw_, T, k, dy.t, dwt.t)
        torch.cuda.synchronize()
        assert dy.intact() and dwt.intact()
        ref_dw = np.where(have, (vd[:, None] * vy[sel]).sum(-1), 0)
        mag = np.where(have, (np.abs(vd)[:, None] * np.abs(vy[sel])).sum(-1), 0)
        assert (np.abs(f64(dwt.t) - ref_dw) <= (cols + 1) * U * mag).all()
        ref_dy = np.full((rows, cols), 9.0)
        for t, j in zip(*np.nonzero(have)):
            ref_dy[slot[t, j]] = eff[t, j] * vd[t]
        assert (np.abs(f64(dy.t) - ref_dy) <= (H if yt else 2 * U) * np.abs(ref_dy)).all()
        # the same dy without dweights
        again = Guarded((rows, cols), TD[yt], 9.0)
        c3.c3_moe_combine_backward(d, ot, None, yt, rows, cols, dslot, None if weights is None else dw_, T, k, again.t, None)
        torch.cuda.synchronize()
        assert again.intact() and torch.equal(again.t, dy.t)


def test_combine_gradient_against_differences(c3):
    rng = np.random.default_rng(8)
    T, k, cols, rows = 12, 4, 40, 64
    y, v = rng.standard_normal((2, rows, cols)).astype(np.float32)
    w, u = rng.standard_normal((2, T, k)).astype(np.float32)
    d = rng.standard_normal((T, cols)).astype(np.float32)
    slot = cuda(rng.permutation(rows)[:T * k].reshape(T, k).astype(np.int32))
    dy, dw = torch.zeros(rows, cols, device="cuda"), torch.empty(T, k, device="cuda")
    c3.c3_moe_combine_backward(cuda(d), 0, cuda(y), 0, rows, cols, slot, cuda(w), T, k, dy, dw)

    def loss(s):
        out = torch.empty(T, cols, device="cuda")
        c3.c3_moe_combine(cuda(y + np.float32(s) * v), 0, rows, cols, slot, cuda(w + np.float32(s) * u), T, k, out, 0)
        return (f64(out) * d).sum()
    # the loss is quadratic along the direction: central differences have no error but rounding,
    # k + 2 roundings of u on terms that sum to `mag`, over the step
    step = 0.25
    mag = (np.abs(d)[:, None] * (np.abs(w) + np.abs(u))[..., None] * (np.abs(y) + np.abs(v))[slot.cpu().numpy()]).sum()
    slope = (loss(step) - loss(-step)) / (2 * step)
    along = (f64(dy) * v).sum() + (f64(dw) * u).sum()
    assert abs(slope - along) <= (k + 4) * U * mag / step + cols * U * mag


# ----------------------------------------------------------------------------- together

def test_other_streams_and_repeatability(c3):
    """Every operator on a stream of its own, twice: the same bits."""
    rng = np.random.default_rng(6)
    T, E, k, Kd, N = 333, 24, 3, 264, 200
    x = cuda(rng.standard_normal((T, Kd)).astype(np.float32))
    logits = cuda(rng.standard_normal((T, E)).astype(np.float32))
    w, vw = random_fp4(c3, rng, N, Kd, 0, count=E)
    st = torch.cuda.Stream()
    rows = c3.c3_moe_rows(T, k, E)
    torch.cuda.synchronize()
    seen = []
    for _ in range(2):
        idx = torch.empty(T, k, dtype=torch.int32, device="cuda")
        wt = torch.empty(T, k, device="cuda")
        slot, row_of = torch.empty_like(idx), torch.empty(rows, dtype=torch.int32, device="cuda")
        offsets, counts = torch.empty(E + 1, dtype=torch.int32, device="cuda"), torch.empty(E, dtype=torch.int32, device="cuda")
        work = torch.empty(c3.c3_moe_order_bytes(T, k, E), dtype=torch.uint8, device="cuda")
        q, _, _ = new_fp4(c3, rows, Kd, 0)
        y, out = torch.empty(rows, N, device="cuda"), torch.empty(T, N, device="cuda")
        torch.cuda.synchronize()
        c3.c3_route(c3.Router(E, k, renorm=True), logits, E, T, idx, wt, stream=st)
        c3.c3_moe_order(idx, T, k, E, slot, row_of, rows, offsets, counts, work, stream=st)
        c3.c3_fp4_quantize(x, 0, T, Kd, q, row_of=row_of, stream=st)
        c3.c3_fp4_gemm_experts(q, w, offsets, counts, y, 0, stream=st)
        c3.c3_moe_combine(y, 0, rows, N, slot, wt, T, k, out, 0, stream=st)
        c3.c3_status_check(st)
        seen.append((idx.clone(), out.clone()))
    assert torch.equal(seen[0][0], seen[1][0]) and torch.equal(seen[0][1], seen[1][1])
    xq = quantise_oracle(x.cpu().numpy(), 0)[2]
    idx, wt = seen[0][0].cpu().numpy(), f64(wt)
    ref = np.einsum("tk,tkn->tn", wt, np.einsum("tc,tknc->tkn", xq, vw[idx]))
    mag = np.einsum("tk,tkn->tn", wt, np.einsum("tc,tknc->tkn", np.abs(xq), np.abs(vw)[idx]))
    assert (np.abs(f64(seen[0][1]) - ref) <= ((Kd / 64 + 64) * 2 + k * 2) * U * mag).all()


def test_offsets_past_32_bits(c3):
    """Rows whose elements lie past 2^31: quantised, multiplied and combined like the first ones."""
    rows, cols = 70016, 32768          # 2.29e9 elements
    few = cuda(np.random.default_rng(0).standard_normal((128, cols)).astype(np.float32)).to(torch.bfloat16)
    big = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    big[-128:] = few
    q, codes, scales = new_fp4(c3, rows, cols, 0)
    c3.c3_fp4_quantize(big, 1, rows, cols, q)
    p, pc, ps = new_fp4(c3, 128, cols, 0)
    c3.c3_fp4_quantize(few, 1, 128, cols, p)
    torch.cuda.synchronize()
    assert torch.equal(codes.t[0, -128:], pc.t[0]) and torch.equal(scales.t[0, -1], ps.t[0, 0])
    c3.c3_fp4_dequantize(q, big, 1, cols)
    back = torch.empty(128, cols, dtype=torch.bfloat16, device="cuda")
    c3.c3_fp4_dequantize(p, back, 1, cols)
    torch.cuda.synchronize()
    assert torch.equal(big[-128:], back)
    # combine: the last rows of y
    slot = torch.arange(rows - 128, rows, dtype=torch.int32, device="cuda").view(128, 1)
    out = torch.empty(128, cols, dtype=torch.bfloat16, device="cuda")
    c3.c3_moe_combine(big, 1, rows, cols, slot, None, 128, 1, out, 1)
    torch.cuda.synchronize()
    assert torch.equal(out, back)
    del codes, scales
    # a product whose output has its last rows past 2^31 elements
    small, vs = random_fp4(c3, np.random.default_rng(1), rows, 64, 0)
    wide, vw = random_fp4(c3, np.random.default_rng(2), cols, 64, 0)
    c3.c3_fp4_gemm(small, wide, big, 1)
    c3.c3_status_check()
    assert close(f64(big[-128:]), vs[0][-128:], vw[0], 1, 64)
