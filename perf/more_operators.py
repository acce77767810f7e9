"""Measured cases of a training step's two ends: the lookup of embeddings with its gradient by sorted tokens, and
the orthogonalisation of an update by Newton-Schulz products.

`run` computes an operator in plain torch operations, or, with `own` set, through the library's binding.
"""
import math

import numpy as np
import torch

own = False

F32, BF16 = 0, 1
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
CODES = {"f32": F32, "bf16": BF16}
SIZE = {"f32": 4, "bf16": 2}
# the quintic that the Muon optimiser iterates
QUINTIC = (3.4445, -4.7750, 2.0315)
STEPS = 5
EPS = 1e-7


# ----------------------------------------------------------------------------- cases

def listed():
    look = dict(op="lookup", vocab=131072, first=0, rows=131072, table="bf16", out="bf16", padded=False)
    grad = dict(op="gradient", vocab=131072, first=0, rows=131072, dout="bf16", table="bf16", batches=1, padded=False)
    orth = dict(op="orthogonalise", count=1, type="bf16")
    return [
        # one serving step: eight sequences, one token each; latency is all that counts
        dict(look, name="lookup decode", tokens=8, cols=8192),
        # a long prefill batch against a whole table
        dict(look, name="lookup prefill", tokens=65536, cols=8192),
        # one of eight shards of a vocabulary, fp32 master table, odd rows, a padded batch: what the ranks all-reduce
        dict(look, name="lookup shard", tokens=10007, cols=2051, first=3 * 16384, rows=16384, table="f32", padded=True),
        # a small fine-tuning step on one shard; latency counts
        dict(grad, name="gradient small", tokens=96, cols=1024, vocab=32768, first=4096, rows=4096, dout="f32", table="f32"),
        # a training step's gradient of a whole table in the working type, frequent tokens thousands of times
        dict(grad, name="gradient step", tokens=16384, cols=8192),
        # two micro-batches, the second added to the first's fp32 gradient, on one of eight shards
        dict(grad, name="gradient accumulated", tokens=32768, cols=4096, first=16384, rows=16384, table="f32", batches=2),
        # odd sizes and padding throughout, fp32
        dict(grad, name="gradient ragged", tokens=40009, cols=1347, vocab=50021, rows=50021, dout="f32", table="f32",
             padded=True),
        # the smallest matrices of a model: an adapter or a projection of few heads
        dict(orth, name="orthogonalise small", rows=256, cols=640),
        # experts' matrices, one stack
        dict(orth, name="orthogonalise experts", rows=1024, cols=2048, count=16),
        # a tall matrix of odd sizes, the momentum in fp32
        dict(orth, name="orthogonalise tall", rows=5003, cols=1347, type="f32"),
        # a square projection
        dict(orth, name="orthogonalise square", rows=4096, cols=4096),
        # the feed-forward weight of this library's workloads
        dict(orth, name="orthogonalise feed-forward", rows=8192, cols=28672),
    ]


def _size(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["lookup", "gradient", "gradient", "orthogonalise", "orthogonalise"])
    kind = lambda: rng.choice(["f32", "bf16"])  # noqa: E731
    if op == "orthogonalise":
        rows, cols = _size(rng, 64, 8192), _size(rng, 64, 16384)
        count = _size(rng, 1, 32) if rng.random() < 0.4 else 1
        while count > 1 and count * rows * cols > 1 << 26:
            count //= 2
        return dict(op=op, rows=rows, cols=cols, count=count, type=kind())
    vocab, cols = _size(rng, 1000, 131072), _size(rng, 64, 8192)
    shards = rng.choice([1, 1, 2, 4, 8])
    rows = -(-vocab // shards)
    first = rng.randrange(shards) * rows
    rows = min(rows, vocab - first)
    tokens = _size(rng, 1, 65536)
    case = dict(op=op, vocab=vocab, first=first, rows=rows, tokens=tokens, cols=cols, padded=rng.random() < 0.3)
    if op == "lookup":
        return dict(case, table=kind(), out=kind())
    return dict(case, dout=kind(), table=kind(), batches=rng.choice([1, 1, 2]))


# ----------------------------------------------------------------------------- inputs

def _rng(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _shares(vocab):
    """How often each rank of a vocabulary comes up: a power law, as tokens have it."""
    p = 1.0 / (np.arange(vocab) + 2.7)
    return p / p.sum()


def _spread(vocab):
    """A step that takes ranks to ids one to one, so that every shard has frequent tokens."""
    step = 7919
    while math.gcd(step, vocab) > 1:
        step += 2
    return step


def _ids(c, gen):
    """int32 token ids; padding is -1."""
    cdf = torch.from_numpy(np.cumsum(_shares(c["vocab"]))).cuda()
    u = torch.rand(c["tokens"], generator=gen, device="cuda", dtype=torch.float64)
    rank = torch.searchsorted(cdf, u).clamp_max(c["vocab"] - 1)
    ids = rank * _spread(c["vocab"]) % c["vocab"]
    if c["padded"]:
        ids = torch.where(torch.rand(c["tokens"], generator=gen, device="cuda") < 0.1, -1, ids)
    return ids.to(torch.int32)


def _normal(shape, gen, scale, dtype):
    return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype)


def prepare(case, seed):
    gen = _rng(seed)
    c = case
    new = lambda shape, kind: torch.zeros(shape, dtype=TYPES[kind], device="cuda")  # noqa: E731
    if c["op"] == "lookup":
        return dict(case=c, ids=_ids(c, gen), table=_normal((c["rows"], c["cols"]), gen, 0.02, TYPES[c["table"]]),
                    scale=math.sqrt(c["cols"]), out=new((c["tokens"], c["cols"]), c["out"]))
    if c["op"] == "gradient":
        batches = [(_ids(c, gen), _normal((c["tokens"], c["cols"]), gen, 1e-3, TYPES[c["dout"]]))
                   for _ in range(c["batches"])]
        return dict(case=c, batches=batches, scale=math.sqrt(c["cols"]),
                    dtable=new((c["rows"], c["cols"]), c["table"]))
    # a momentum: a few strong directions over noise, as gradients of weights have them
    m, n, k = c["rows"], c["cols"], c["count"]
    r = min(8, m, n)
    x = torch.randn((k, m, n), generator=gen, device="cuda")
    strong = torch.linspace(1.0, 0.1, r, device="cuda")
    left = torch.randn((k, m, r), generator=gen, device="cuda") * strong
    x += torch.matmul(left, torch.randn((k, r, n), generator=gen, device="cuda"))
    x *= 1e-3
    return dict(case=c, x=x.to(TYPES[c["type"]]), scale=math.sqrt(max(1.0, m / n)), out=new((k, m, n), "bf16"))


# ----------------------------------------------------------------------------- plain forms

def _place(ids, c):
    """Rows of the shard, and which tokens have one."""
    at = ids.long() - c["first"]
    have = (at >= 0) & (at < c["rows"])
    return at, have


def _plain(s):
    c = s["case"]
    if c["op"] == "lookup":
        at, have = _place(s["ids"], c)
        rows = s["table"][at.clamp(0, c["rows"] - 1)].float() * s["scale"]
        return torch.where(have.unsqueeze(1), rows, 0.0).to(TYPES[c["out"]])
    if c["op"] == "gradient":
        total = torch.zeros(c["rows"] + 1, c["cols"], device="cuda")
        # tokens of other shards add to a row of their own, which is cut off
        for i, (ids, dout) in enumerate(s["batches"]):
            at, have = _place(ids, c)
            total.index_add_(0, torch.where(have, at, c["rows"]), dout.float() * s["scale"])
            if i + 1 < len(s["batches"]):  # what the table holds between two micro-batches is of its type
                total = total.to(TYPES[c["table"]]).float()
        return total[:-1].to(TYPES[c["table"]])
    a, b, q = QUINTIC
    x = s["x"].float()
    tall = c["rows"] > c["cols"]
    x = x.transpose(-1, -2) if tall else x
    x = x / (x.square().sum((-1, -2), keepdim=True).sqrt() + EPS)
    for _ in range(STEPS):
        g = torch.matmul(x, x.transpose(-1, -2))
        x = a * x + torch.matmul(b * g + q * torch.matmul(g, g), x)
    x = x.transpose(-1, -2) if tall else x
    return (x * s["scale"]).to(torch.bfloat16)


# ----------------------------------------------------------------------------- the library's calls

def _own(s):
    from concurrent_communication_overlap_gb300 import c3
    c = s["case"]
    if c["op"] == "lookup":
        c3.c3_embed(s["table"], CODES[c["table"]], c["rows"], c["cols"], s["ids"], c["tokens"], s["out"], CODES[c["out"]],
                    scale=s["scale"], first=c["first"])
        return s["out"]
    if "work" not in s:  # the workspace is the program's own
        size = (c3.c3_embed_backward_bytes(c["tokens"], c["rows"], c["cols"]) if c["op"] == "gradient"
                else c3.c3_orthogonalize_bytes(c["rows"], c["cols"], c["count"]))
        s["work"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    if c["op"] == "gradient":
        for i, (ids, dout) in enumerate(s["batches"]):
            c3.c3_embed_backward(dout, CODES[c["dout"]], ids, c["tokens"], s["dtable"], CODES[c["table"]], c["rows"],
                                 c["cols"], s["work"], scale=s["scale"], first=c["first"], accumulate=i > 0)
        return s["dtable"]
    c3.c3_orthogonalize(s["x"], CODES[c["type"]], c["rows"], c["cols"], s["out"], s["work"], [QUINTIC] * STEPS,
                        scale=s["scale"], eps=EPS, count=c["count"])
    return s["out"]


def run(state):
    return _own(state) if own else _plain(state)


# ----------------------------------------------------------------------------- what a pass cannot do without

def _distinct(c):
    """Rows of the shard that a batch names, on average; and its tokens with a row."""
    n = c["tokens"] * (0.9 if c["padded"] else 1.0)
    p = _shares(c["vocab"])
    ids = np.arange(c["vocab"]) * _spread(c["vocab"]) % c["vocab"]
    p = p[(ids >= c["first"]) & (ids < c["first"] + c["rows"])]
    return float(-np.expm1(n * np.log1p(-p)).sum()), float(n * p.sum())


def work(case):
    c = case
    if c["op"] == "lookup":
        rows, tokens = _distinct(c)
        return {"bytes": rows * c["cols"] * SIZE[c["table"]] + c["tokens"] * (c["cols"] * SIZE[c["out"]] + 4),
                "flops": tokens * c["cols"]}
    if c["op"] == "gradient":
        rows, tokens = _distinct(c)
        b = c["rows"] * c["cols"] * SIZE[c["table"]]                       # every row is written once
        b += c["batches"] * (tokens * c["cols"] * SIZE[c["dout"]] + 4 * c["tokens"])
        b += (c["batches"] - 1) * 2 * rows * c["cols"] * SIZE[c["table"]]  # rows that are added to
        return {"bytes": b, "flops": c["batches"] * tokens * c["cols"]}
    m, n = min(c["rows"], c["cols"]), max(c["rows"], c["cols"])
    # the two symmetric products need one half each
    return {"bytes": c["count"] * m * n * (SIZE[c["type"]] + 2),
            "flops": c["count"] * STEPS * (m * m * n + m * m * m + 2 * m * m * n)}


# ----------------------------------------------------------------------------- the definitions, in 64 bits

def exact(case, seed):
    c = case
    if c["op"] == "orthogonalise":
        m, n = min(c["rows"], c["cols"]), max(c["rows"], c["cols"])
        if c["count"] * STEPS * 6.0 * m * m * n > 8e12:
            return None  # too long in 64 bits
        s = prepare(c, seed)
        a, b, q = QUINTIC
        out = torch.empty(s["out"].shape, dtype=torch.float64, device="cuda")
        for i in range(c["count"]):
            x = s["x"][i].double()
            x /= torch.linalg.vector_norm(x) + EPS
            for _ in range(STEPS):  # the polynomial inside out, without a product of the square matrices
                if c["rows"] <= c["cols"]:
                    g = x @ x.T
                    x = a * x + g @ (b * x + q * (g @ x))
                else:
                    g = x.T @ x
                    x = a * x + (b * x + q * (x @ g)) @ g
            out[i] = s["scale"] * x
        return out
    s = prepare(c, seed)
    if c["op"] == "lookup":
        out = torch.zeros(c["tokens"], c["cols"], dtype=torch.float64, device="cuda")
        mine = ((s["ids"] >= c["first"]) & (s["ids"] < c["first"] + c["rows"])).nonzero()[:, 0]
        out[mine] = s["table"][s["ids"][mine].long() - c["first"]].double() * s["scale"]
        return out
    total = torch.zeros(c["rows"], c["cols"], dtype=torch.float64, device="cuda")
    for ids, dout in s["batches"]:
        mine = ((ids >= c["first"]) & (ids < c["first"] + c["rows"])).nonzero()[:, 0]
        # sorted by row, then the rows of each by differences of running sums, a slice of columns at a time
        row, order = torch.sort(ids[mine].long() - c["first"], stable=True)
        last = torch.ones_like(row, dtype=torch.bool)
        last[:-1] = row[1:] != row[:-1]
        end = last.nonzero()[:, 0]
        for j in range(0, c["cols"], 512):
            run_sum = torch.cumsum(dout[mine[order], j:j + 512].double(), 0)[end]
            run_sum[1:] -= run_sum[:-1].clone()
            total[row[end], j:j + 512] += s["scale"] * run_sum
    return total
