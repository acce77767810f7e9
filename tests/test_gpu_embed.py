"""The lookup of embeddings and its gradient on the GPU, against plain implementations in 64 bits.

Tolerances (u = 2^-24 and h = 2^-8, half a step of fp32 and bf16 relative to the value): a lookup is one product,
u of it, and h where the output is bf16.  A row of the gradient is a sum of k terms, k u of the sum of their
magnitudes in any order, a product, and an addition where it accumulates: (k + 2) u of scale * sum |d| + |old|, and
h of the value where the table is bf16."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from test_gpu_ops import Guarded, c3, f64  # noqa: F401

pytestmark = pytest.mark.gpu

U, H = 2.0 ** -24, 2.0 ** -8
TD = {0: torch.float32, 1: torch.bfloat16}


def rows_in(shape, ld, dtype, off=0, fill=None):
    """A guarded [rows][ld] tensor whose rows begin `off` elements in, and the view of its columns."""
    rows, cols = shape
    g = Guarded((rows * ld + off,), dtype)
    if fill is not None:
        g.t.copy_(fill)
    return g, g.t[off:].view(rows, ld)[:, :cols]


def some_ids(rng, tokens, rows, first, kind):
    if kind == "hot":      # a few rows hold nearly everything
        ids = np.where(rng.random(tokens) < 0.9, rng.integers(0, min(3, rows), tokens), rng.integers(0, rows, tokens))
    elif kind == "one":
        ids = np.full(tokens, rows - 1)
    elif kind == "none":
        ids = np.full(tokens, rows)
    else:
        ids = rng.integers(0, rows, tokens)
    ids = ids + first
    if kind == "padded":   # ids of other shards, and padding
        ids = np.where(rng.random(tokens) < 0.4, rng.choice([-1, -2 ** 31, first - 1, first + rows, 2 ** 31 - 1], tokens), ids)
    return ids.astype(np.int64).astype(np.int32)


def vector(rng, n, dtype):
    return torch.from_numpy(rng.standard_normal(n).astype(np.float32)).cuda().to(dtype)


# ----------------------------------------------------------------------------- lookup

@pytest.mark.parametrize("tt", [0, 1])
@pytest.mark.parametrize("ot", [0, 1])
@pytest.mark.parametrize("tokens,rows,cols,pad,off,first", [
    (1, 1, 1, 0, 0, 0), (1, 7, 8, 0, 0, 0), (3, 5, 255, 0, 0, 2), (17, 100, 256, 0, 0, 1000), (33, 9, 257, 3, 1, 5),
    (64, 50, 1030, 0, 0, 0), (64, 50, 1026, 2, 2, 7), (129, 300, 2048, 8, 8, 12), (40, 30, 520, 0, 4, 0),
    (2000, 1111, 8, 0, 0, 3)])
def test_lookup(c3, tt, ot, tokens, rows, cols, pad, off, first):  # noqa: F811
    rng = np.random.default_rng(tokens * 7 + cols)
    ld = cols + pad
    ids = some_ids(rng, tokens, rows, first, "padded")
    gt, table = rows_in((rows, cols), ld, TD[tt], off, vector(rng, rows * ld + off, TD[tt]))
    go, out = rows_in((tokens, cols), ld, TD[ot], off, torch.full((tokens * ld + off,), 7.0, device="cuda"))
    scale = float(np.float32(1.7))
    c3.c3_embed(table, tt, rows, cols, torch.from_numpy(ids).cuda(), tokens, out, ot, scale=scale, first=first, ld=ld, out_ld=ld)
    torch.cuda.synchronize()
    at = ids.astype(np.int64) - first
    have = (at >= 0) & (at < rows)
    ref = np.where(have[:, None], f64(table)[np.clip(at, 0, rows - 1)] * scale, 0)
    assert (np.abs(f64(out) - ref) <= (U + (H if ot else 0)) * np.abs(ref)).all()
    assert go.intact() and gt.intact()
    rest = go.t[off:].view(tokens, ld)[:, cols:]
    assert (rest == 7).all() and (go.t[:off] == 7).all()


def test_lookup_of_special_values(c3):  # noqa: F811
    table = torch.tensor([[float("inf"), float("nan"), -0.0, 1e-40, -float("inf"), 3e38, 0.0, 1.0]] * 2, device="cuda")
    ids = torch.tensor([1, 5, 0], dtype=torch.int32, device="cuda")
    out = torch.full((3, 8), 9.0, device="cuda")
    c3.c3_embed(table, 0, 2, 8, ids, 3, out, 0, scale=2.0)
    o = out.cpu().numpy()
    assert (o[1] == 0).all()  # no row: zeros, whatever the table holds
    with np.errstate(over="ignore"):
        want = table[0].cpu().numpy() * np.float32(2)
    assert np.array_equal(o[0], want, equal_nan=True) and np.array_equal(o[2], want, equal_nan=True)


def test_lookup_past_32_bits(c3):  # noqa: F811
    rows, cols = 140000, 20008  # 2.8 G elements
    table = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    table[rows - 1] = 3.0
    table[107400] = 2.0  # its end passes 2^31 elements
    ids = torch.tensor([rows - 1, 0, 107400, rows], dtype=torch.int32, device="cuda")
    out = torch.empty(4, cols, device="cuda")
    c3.c3_embed(table, 1, rows, cols, ids, 4, out, 0)
    assert (out.amin(1).tolist(), out.amax(1).tolist()) == ([3.0, 0.0, 2.0, 0.0],) * 2
    # the gradient of such a table, into those rows
    work = torch.empty(c3.c3_embed_backward_bytes(4, rows, cols), dtype=torch.uint8, device="cuda")
    dout = torch.ones(4, cols, device="cuda")
    c3.c3_embed_backward(dout, 0, ids, 4, table, 1, rows, cols, work, scale=5.0, accumulate=True)
    torch.cuda.synchronize()
    assert (table[rows - 1] == 8).all() and (table[107400] == 7).all() and (table[0] == 5).all() and (table[1] == 0).all()
    assert (table[rows - 2] == 0).all()


# ----------------------------------------------------------------------------- gradient

def gradient_oracle(ids, dout, rows, first, scale, old):
    at = ids.astype(np.int64) - first
    mine = np.nonzero((at >= 0) & (at < rows))[0]
    total, mag = np.zeros((rows, dout.shape[1])), np.zeros((rows, dout.shape[1]))
    np.add.at(total, at[mine], dout[mine])
    np.add.at(mag, at[mine], np.abs(dout[mine]))
    count = np.bincount(at[mine], minlength=rows)[:, None]
    return scale * total + old, (count + 2) * U * (scale * mag + np.abs(old)), count[:, 0]


def check_gradient(c3, dt, tt, tokens, rows, cols, pad, off, first, kind, accumulate, seed=0):  # noqa: F811
    rng = np.random.default_rng(seed + tokens * 13 + cols)
    ld = cols + pad
    ids = some_ids(rng, tokens, rows, first, kind)
    gd, dout = rows_in((max(tokens, 1), cols), ld, TD[dt], off, vector(rng, max(tokens, 1) * ld + off, TD[dt]))
    before = vector(rng, rows * ld + off, TD[tt])
    gt, table = rows_in((rows, cols), ld, TD[tt], off, before)
    old = f64(table)
    dids = torch.from_numpy(ids).cuda()
    work = Guarded((c3.c3_embed_backward_bytes(tokens, rows, cols),), torch.uint8)
    scale = float(np.float32(0.3))

    def call():
        c3.c3_embed_backward(dout, dt, dids, tokens, table, tt, rows, cols, work.t, scale=scale, first=first,
                             accumulate=accumulate, dout_ld=ld, ld=ld)
        torch.cuda.synchronize()
    call()
    got = table.clone()
    ref, tol, count = gradient_oracle(ids, f64(dout)[:tokens], rows, first, scale, old if accumulate else 0 * old)
    g = f64(got)
    assert (np.abs(g - ref) <= tol + (H * np.abs(ref) if tt else 0)).all()
    if accumulate:  # rows that no token names are left as they were
        assert np.array_equal(g[count == 0], old[count == 0])
    else:
        assert (g[count == 0] == 0).all()
    assert gd.intact() and gt.intact() and work.intact()
    whole = gt.t[off:].view(rows, ld)
    assert torch.equal(whole[:, cols:], before[off:].view(rows, ld)[:, cols:]) and torch.equal(gt.t[:off], before[:off])
    # again, over a workspace full of something else: the same bits
    gt.t.copy_(before)
    work.t.fill_(0xC3)
    call()
    assert torch.equal(got, table)


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("dt,tt", [(0, 0), (1, 1), (1, 0), (0, 1)])
@pytest.mark.parametrize("tokens,rows,cols,pad,off,first,kind", [
    (1, 1, 1, 0, 0, 0, "any"), (1, 1000, 8, 0, 0, 3, "any"), (2, 1, 8, 0, 0, 0, "one"), (7, 33, 255, 0, 0, 2, "padded"),
    (8, 3, 256, 0, 0, 0, "any"), (9, 40, 257, 3, 1, 5, "padded"), (31, 1025, 520, 0, 4, 0, "any"),
    (33, 1024, 40, 2, 2, 9, "hot"), (64, 64, 1030, 0, 0, 0, "one"), (100, 500, 2048, 8, 8, 100, "padded"),
    (257, 5000, 2, 0, 0, 0, "hot"), (300, 7, 513, 0, 0, 0, "none"), (0, 9, 12, 1, 0, 0, "any"),
    (1024, 700, 257, 0, 0, 4, "hot"), (1023, 5, 48, 0, 0, 0, "one"), (1025, 100, 56, 0, 0, 0, "hot"),
    (600, 33, 2050, 0, 0, 0, "padded"), (1000, 20, 8, 0, 0, 0, "any")])
def test_gradient(c3, dt, tt, tokens, rows, cols, pad, off, first, kind, accumulate):  # noqa: F811
    check_gradient(c3, dt, tt, tokens, rows, cols, pad, off, first, kind, accumulate)


@pytest.mark.parametrize("tokens,rows,cols,kind", [
    (2000, 70000, 520, "padded"), (3000, 2500000, 2, "hot"), (4096, 5000, 300, "hot"), (4097, 5000, 300, "hot"),
    (4000, 1, 16, "one"), (3001, 77, 16, "none"), (1100, 33, 2304, "any"), (4095, 1000, 24, "any"), (4096, 1023, 8, "hot"), (4097, 1024, 8, "padded"), (5000, 1025, 40, "one"),
    (8191, 70001, 16, "any"), (20011, 50021, 24, "hot"), (70001, 131072, 8, "padded"), (66000, 40, 264, "any"),
    (65536, 3, 1040, "hot"), (33000, 1100000, 8, "any"), (300007, 600, 8, "hot"), (12345, 2000, 1347, "padded")])
@pytest.mark.parametrize("accumulate", [False, True])
def test_gradient_of_many_tokens(c3, tokens, rows, cols, kind, accumulate):  # noqa: F811
    check_gradient(c3, 1, 0, tokens, rows, cols, 0, 0, 11, kind, accumulate)


@pytest.mark.parametrize("tokens", [513, 520, 768, 769, 1025, 8439, 8448, 8449, 8456, 38912, 38913])
@pytest.mark.parametrize("kind,cols", [("one", 8), ("hot", 8), ("one", 2500)])
def test_gradient_of_rows_cut_into_many_parts(c3, tokens, kind, cols):  # noqa: F811
    """Around the numbers of parts at which their count takes another turn: 1 + 32, 1 + 32 + 32, 1 + 32 + 1024 of 8 tokens."""
    check_gradient(c3, 0, 0, tokens, 90, cols, 0, 0, 3, kind, True)


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("tokens,rows,cols,kind", [(1, 3, 1050001, "any"), (40, 2, 1048600, "one"), (5, 600, 700001, "padded")])
def test_gradient_of_long_rows(c3, tokens, rows, cols, kind, accumulate):  # noqa: F811
    """Few tokens of so many columns that they are put in order first."""
    check_gradient(c3, 1, 1, tokens, rows, cols, 0, 0, 11, kind, accumulate)


def test_gradient_of_infinities(c3):  # noqa: F811
    """An infinity or a NaN stays in its row and column."""
    dout = torch.zeros(40, 16, device="cuda")
    dout[3, 5], dout[4, 6], dout[5, 7], dout[6, 7] = float("inf"), float("nan"), float("inf"), -float("inf")
    ids = torch.arange(40, dtype=torch.int32, device="cuda") % 8
    ids[5] = ids[6] = 2
    table = torch.empty(8, 16, device="cuda")
    work = torch.empty(c3.c3_embed_backward_bytes(40, 8, 16), dtype=torch.uint8, device="cuda")
    c3.c3_embed_backward(dout, 0, ids, 40, table, 0, 8, 16, work)
    ref = torch.zeros(8, 16, dtype=torch.float64)
    for t in range(40):
        ref[int(ids[t])] += dout[t].cpu().double()
    assert np.array_equal(f64(table), ref.numpy(), equal_nan=True)


def test_gradient_is_the_lookups(c3):  # noqa: F811
    """<dout, lookup(table + e) - lookup(table)> against <gradient, e>: the lookup is linear, so differences are exact
    up to roundings (values on a grid make them exact)."""
    rng = np.random.default_rng(5)
    tokens, rows, cols = 500, 64, 48
    ids = torch.from_numpy(some_ids(rng, tokens, rows, 10, "padded")).cuda()
    grid = lambda *s: torch.from_numpy(rng.integers(-8, 9, s).astype(np.float32)).cuda()  # noqa: E731
    table, e, dout = grid(rows, cols), grid(rows, cols), grid(tokens, cols)
    a, b = (torch.empty(tokens, cols, device="cuda") for _ in range(2))
    c3.c3_embed(table, 0, rows, cols, ids, tokens, a, 0, scale=0.5, first=10)
    c3.c3_embed(table + e, 0, rows, cols, ids, tokens, b, 0, scale=0.5, first=10)
    grad = torch.empty(rows, cols, device="cuda")
    work = torch.empty(c3.c3_embed_backward_bytes(tokens, rows, cols), dtype=torch.uint8, device="cuda")
    c3.c3_embed_backward(dout, 0, ids, tokens, grad, 0, rows, cols, work, scale=0.5, first=10)
    assert (dout.double() * (b - a).double()).sum().item() == (grad.double() * e.double()).sum().item()


def test_calls_in_a_graph_and_on_streams(c3):  # noqa: F811
    """Two micro-batches captured together, replayed on other inputs, beside eager calls on a second stream."""
    rng = np.random.default_rng(9)
    tokens, rows, cols = 6000, 5000, 136
    size = c3.c3_embed_backward_bytes(tokens, rows, cols)
    ids = [torch.from_numpy(some_ids(rng, tokens, rows, 0, "hot")).cuda() for _ in range(4)]
    douts = [vector(rng, tokens * cols, torch.bfloat16).view(tokens, cols) for _ in range(4)]

    def both(i, d, table, work, s):
        for k in range(2):
            c3.c3_embed_backward(d[k], 1, i[k], tokens, table, 0, rows, cols, work, accumulate=k > 0, stream=s)

    want = []
    for k in (0, 2):
        table, work = torch.empty(rows, cols, device="cuda"), torch.empty(size, dtype=torch.uint8, device="cuda")
        both(ids[k:k + 2], douts[k:k + 2], table, work, torch.cuda.current_stream())
        torch.cuda.synchronize()
        want.append(table)
    gi, gd = [t.clone() for t in ids[:2]], [t.clone() for t in douts[:2]]
    table, work = torch.empty(rows, cols, device="cuda"), torch.empty(size, dtype=torch.uint8, device="cuda")
    other, other_work = torch.empty_like(table), torch.empty_like(work)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both(gi, gd, table, work, torch.cuda.current_stream())
    torch.cuda.synchronize()
    for k in (0, 2, 0):
        for j in range(2):
            gi[j].copy_(ids[k + j])
            gd[j].copy_(douts[k + j])
        torch.cuda.synchronize()
        graph.replay()
        both(ids[2 - k:4 - k], douts[2 - k:4 - k], other, other_work, side)
        torch.cuda.synchronize()
        assert torch.equal(table, want[k // 2]) and torch.equal(other, want[1 - k // 2])


def test_lookup_of_shards_is_the_whole_lookup(c3):  # noqa: F811
    """Eight shards' lookups, put together by the library's all-reduce: one of them has each row."""
    rng = np.random.default_rng(3)
    per, cols, tokens = 125, 64, 333
    table = vector(rng, 8 * per * cols, torch.bfloat16).view(8 * per, cols)
    ids = torch.from_numpy(some_ids(rng, tokens, 8 * per, 0, "padded")).cuda()
    count = -(-tokens * cols // 32) * 32
    parts = [torch.zeros(count, device="cuda") for _ in range(8)]
    for r in range(8):
        c3.c3_embed(table[r * per:(r + 1) * per], 1, per, cols, ids, tokens, parts[r], 0, scale=3.0, first=r * per)
    out = torch.empty(8, count, device="cuda")
    c3.c3_allreduce(parts, out, count, 8)
    whole = torch.empty(tokens, cols, device="cuda")
    c3.c3_embed(table, 1, 8 * per, cols, ids, tokens, whole, 0, scale=3.0)
    torch.cuda.synchronize()
    for r in range(8):
        assert torch.equal(out[r, :tokens * cols].view(tokens, cols), whole)
