"""Measured cases of the routing and 4-bit operators: routing to experts, microscaled 4-bit quantisation and
products, the experts' products and the combination of their outputs.

`run` computes an operator in plain torch operations, or, with `own` set, through the library's binding.
"""
import math

import torch

own = False

TILE = 128  # rows of a scale tile; an expert's rows start at a multiple of it
MX, NV = 0, 1
BLOCK = {MX: 32, NV: 16}
F32, BF16 = 0, 1
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
CODES = {"f32": F32, "bf16": BF16}


# ----------------------------------------------------------------------------- cases

def listed():
    route = dict(op="route", score="sigmoid", bias=True, groups=8, keep=4, best=2, renorm=True, scale=2.5,
                 masked=False, train=False)
    return [
        # the router of one serving step: eight sequences, one token each; latency is all that counts
        dict(route, name="route decode", tokens=8, experts=256, topk=8, type="bf16"),
        # the router over a long prefill batch, grouped experts, fp32 scores
        dict(route, name="route prefill", tokens=65536, experts=256, topk=8, type="f32"),
        # a training step's router with a softmax, some experts masked off, forward and backward
        dict(op="route", name="route train", tokens=32768, experts=60, topk=6, type="bf16", score="softmax",
             bias=False, groups=1, keep=1, best=1, renorm=False, scale=1.0, masked=True, train=True),
        # a square weight to 4 bits and back, as a training step with 4-bit forward numerics does it
        dict(op="quantise", name="quantise weight", rows=8192, cols=8192, type="bf16", format="mx", transpose=False),
        # a gradient laid out along its rows for the weight's product: transposed, two-level scales, odd sizes
        dict(op="quantise", name="quantise gradient", rows=2050, cols=4100, type="f32", format="nv", transpose=True),
        # a dense layer of a serving step: few tokens against a whole weight, odd sizes
        dict(op="product", name="product decode", m=13, n=8200, k=8072, format="nv", out="bf16"),
        # the memory-bound product of this library's workloads
        dict(op="product", name="product batch", m=256, n=28672, k=8192, format="mx", out="bf16"),
        # the feed-forward product of this library's workloads
        dict(op="product", name="product feed-forward", m=8192, n=28672, k=8192, format="mx", out="bf16"),
        # experts of a serving step: most experts get a handful of tokens, the weights' bytes count
        dict(op="experts", name="experts decode", tokens=32, experts=64, topk=6, n=2048, k=4096, format="mx"),
        # experts of a prefill batch, uneven loads
        dict(op="experts", name="experts prefill", tokens=8192, experts=32, topk=4, n=4096, k=4096, format="nv"),
        # the experts' outputs of one serving step put together
        dict(op="combine", name="combine decode", tokens=32, topk=6, experts=64, cols=4096, type="bf16", train=False),
        # the same in training, forward and backward
        dict(op="combine", name="combine train", tokens=8192, topk=8, experts=64, cols=4096, type="bf16", train=True),
    ]


def _size(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    n = min(hi, max(lo, n))
    return n - 1 if n == 3072 else n


def draw(rng):
    op = rng.choice(["route", "route", "quantise", "product", "product", "experts", "combine"])
    if op == "route":
        sigmoid = rng.random() < 0.5
        experts = _size(rng, 8, 512)
        groups = rng.choice([1, 2, 4, 8]) if rng.random() < 0.5 else 1
        if groups > 1:
            experts = max(2, experts // groups) * groups
        keep = rng.randint(1, groups)
        topk = rng.randint(1, min(12, experts // groups * keep))
        train = rng.random() < 0.4
        return dict(op="route", tokens=_size(rng, 1, 32768 if train else 65536 * 256 // max(256, experts)),
                    experts=experts, topk=topk, type=rng.choice(["f32", "bf16"]),
                    score="sigmoid" if sigmoid else "softmax", bias=sigmoid and rng.random() < 0.7, groups=groups,
                    keep=keep, best=2 if sigmoid and groups > 1 and rng.random() < 0.5 else 1,
                    renorm=topk > 1 and rng.random() < 0.5, scale=rng.choice([1.0, 2.5]), masked=rng.random() < 0.3, train=train)
    if op == "quantise":
        rows, cols = _size(rng, 1, 16384), _size(rng, 16, 16384)
        while rows * cols > 8192 * 8192:
            rows, cols = max(1, rows // 2), max(16, cols // 2)
        return dict(op="quantise", rows=rows, cols=cols, type=rng.choice(["f32", "bf16"]),
                    format=rng.choice(["mx", "nv"]), transpose=rng.random() < 0.4)
    if op == "product":
        m, n, k = _size(rng, 1, 8192), _size(rng, 128, 28672), _size(rng, 128, 8192)
        fmt = rng.choice(["mx", "nv"])
        # 32-bit outputs go with short sums: a router's scores, a low-rank update
        return dict(op="product", m=m, n=n, k=k, format=fmt,
                    out="f32" if fmt == "mx" and k <= 1024 else "bf16")
    if op == "experts":
        experts = _size(rng, 2, 64)
        return dict(op="experts", tokens=_size(rng, 1, 8192), experts=experts, topk=rng.randint(1, min(6, experts)),
                    n=_size(rng, 256, 4096), k=_size(rng, 256, 4096), format=rng.choice(["mx", "nv"]))
    return dict(op="combine", tokens=_size(rng, 1, 8192), topk=rng.randint(1, 8), experts=_size(rng, 8, 64),
                cols=_size(rng, 64, 4096), type=rng.choice(["f32", "bf16"]), train=rng.random() < 0.5)


# ----------------------------------------------------------------------------- 4-bit matrices in torch

def _e2m1(a):
    """Nearest of 0 .5 1 1.5 2 3 4 6 to a >= 0, ties to the even code."""
    q = torch.where(a < 2, torch.round(a * 2) / 2, torch.where(a < 4, torch.round(a), torch.round(a / 2) * 2))
    return torch.clamp(q, max=6.0)


def _blocks(x, fmt):
    b = BLOCK[fmt]
    pad = -x.shape[-1] % b
    if pad:
        x = torch.nn.functional.pad(x, (0, pad))
    return x.reshape(*x.shape[:-1], -1, b)


def _power(e):
    """2^e as fp32 for whole e (int32) from -127 on."""
    return torch.where(e > -127, (e + 127) << 23, 1 << 22).to(torch.int32).view(torch.float32)


def _quantise(x, fmt, g=None):
    """x (fp32) as [..., blocks, block] signed 4-bit values, the scales' values and the scales' bytes."""
    y = _blocks(x if g is None else x * (1.0 / g), fmt)
    amax = y.abs().amax(-1)
    if fmt == MX:
        m, e = torch.frexp(amax)  # amax = m 2^e, m in [.5, 1)
        e = torch.where(m <= 0.75, e - 3, e - 2)
        e = torch.where(amax == 0, -127, torch.clamp(e, -127, 126)).to(torch.int32)
        # powers of two put together from their exponents: exact
        scale = _power(e)
        q = y * ((127 - e) << 23).view(torch.float32).unsqueeze(-1)
        byte = (e + 127).to(torch.uint8)
    else:
        s8 = torch.clamp(amax / 6, max=448.0).to(torch.float8_e4m3fn)
        scale = s8.float()
        q = torch.where(scale.unsqueeze(-1) > 0, y / scale.unsqueeze(-1), 0.0)
        byte = s8.view(torch.uint8)
    return torch.copysign(_e2m1(q.abs()), q), scale, byte


def _pack(q):
    """Signed 4-bit values [..., blocks, block] as bytes, the even column in the low half, rows of 16-byte units."""
    q = q.reshape(*q.shape[:-2], -1)
    pad = -q.shape[-1] % 32
    if pad:
        q = torch.nn.functional.pad(q, (0, pad))
    a = q.abs()
    code = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code = code + 8 * torch.signbit(q).to(torch.uint8)
    return (code[..., 0::2] + 16 * code[..., 1::2]).contiguous()


def _tile(byte):
    """Scale bytes [..., rows, blocks] in tiles of 128 rows x 4 blocks: byte (r % 32) * 16 + (r / 32) * 4 + block."""
    rows, nb = byte.shape[-2:]
    byte = torch.nn.functional.pad(byte, (0, -nb % 4, 0, -rows % TILE))
    lead = byte.shape[:-2]
    t = byte.reshape(*lead, byte.shape[-2] // TILE, 4, 32, byte.shape[-1] // 4, 4)
    n = len(lead)
    return t.permute(*range(n), n, n + 3, n + 2, n + 1, n + 4).contiguous()


def _untile(t, rows, nb):
    """The scale bytes [..., rows, blocks] of tiled ones."""
    lead = t.shape[:-5]
    n = len(lead)
    b = t.permute(*range(n), n, n + 3, n + 2, n + 1, n + 4)
    return b.reshape(*lead, b.shape[n] * TILE, -1)[..., :rows, :nb]


_VALUES = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]


def _decode(codes, scales, g, rows, cols, fmt):
    """The fp32 values of a packed matrix."""
    table = torch.tensor(_VALUES, device=codes.device)
    v = torch.stack((table[(codes & 15).long()], table[(codes >> 4).long()]), -1).flatten(-2)
    nb = -(-cols // BLOCK[fmt])
    byte = _untile(scales, rows, nb)
    s = _power(byte.to(torch.int32) - 127) if fmt == MX else byte.contiguous().view(torch.float8_e4m3fn).float()
    v = v[..., :nb * BLOCK[fmt]].reshape(*v.shape[:-1], nb, BLOCK[fmt]) * s.unsqueeze(-1)
    v = v.flatten(-2)[..., :cols]
    return v if g is None else v * g


def _values(gen, shape, std=1.0):
    """Normal values with a few large channels, as activations and weights have them."""
    x = torch.randn(shape, generator=gen, device="cuda") * std
    x[..., ::97] *= 8
    return x


def _packed(gen, rows, cols, fmt, std, count=None):
    """A quantised matrix in hand: codes, tiled scales, the matrix's fp32 scale (two-level format only)."""
    lead = () if count is None else (count,)
    codes, scales = [], []
    g = None
    if fmt == NV:
        g = torch.full(lead or (1,), std * 40.0 / (6 * 448), device="cuda")
    for i in range(count or 1):
        q, _, byte = _quantise(_values(gen, (rows, cols), std), fmt, None if g is None else g[i])
        codes.append(_pack(q))
        scales.append(_tile(byte))
    if count is None:
        return codes[0], scales[0], g
    return torch.stack(codes), torch.stack(scales), g


# ----------------------------------------------------------------------------- inputs

def _fmt(c):
    return MX if c["format"] == "mx" else NV


def _cap(tokens, topk, experts):
    n = tokens * topk
    return (n + (TILE - 1) * min(experts, n)) // TILE * TILE


def _chosen(gen, tokens, topk, experts):
    """topk different experts a token, some experts far more often than others."""
    lean = torch.randn(experts, generator=gen, device="cuda") * 0.7
    r = torch.rand(tokens, experts, generator=gen, device="cuda").clamp_min(1e-9)
    gumbel = lean - torch.log(-torch.log(r))
    return torch.argsort(gumbel, dim=1, descending=True)[:, :topk].to(torch.int32).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case=case)
    op = case["op"]
    if op == "route":
        T, E = case["tokens"], case["experts"]
        x = torch.randn(T, E, generator=gen, device="cuda") * 1.5 + torch.randn(E, generator=gen, device="cuda") * 0.5
        if case["masked"]:
            x[:, torch.rand(E, generator=gen, device="cuda") < 0.1] = -math.inf
            if T > 1:
                x[T // 2] = -math.inf  # a padding token
        s["logits"] = x.to(TYPES[case["type"]])
        s["bias"] = torch.randn(E, generator=gen, device="cuda") * 0.05 if case["bias"] else None
        s["idx"] = torch.empty(T, case["topk"], dtype=torch.int32, device="cuda")
        s["weights"] = torch.empty(T, case["topk"], device="cuda")
        if case["train"]:
            s["dweights"] = torch.randn(T, case["topk"], generator=gen, device="cuda")
            s["dlogits"] = torch.empty_like(s["logits"])
    elif op == "quantise":
        fmt, rows, cols = _fmt(case), case["rows"], case["cols"]
        s["x"] = _values(gen, (rows, cols), 0.02).to(TYPES[case["type"]])
        s["g"] = torch.full((1,), 0.02 * 40.0 / (6 * 448), device="cuda") if fmt == NV else None
        if case["transpose"]:
            rows, cols = cols, rows
        nb = -(-cols // BLOCK[fmt])
        s["codes"] = torch.empty(rows, -(-cols // 32) * 16, dtype=torch.uint8, device="cuda")
        s["scales"] = torch.empty(-(-rows // TILE), -(-nb // 4), 32, 4, 4, dtype=torch.uint8, device="cuda")
        s["values"] = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    elif op == "product":
        fmt, m, n, k = _fmt(case), case["m"], case["n"], case["k"]
        s["a"] = _packed(gen, m, k, fmt, 1.0)
        s["b"] = _packed(gen, n, k, fmt, 0.02)
        s["c"] = torch.empty(m, n, dtype=TYPES[case["out"]], device="cuda")
    elif op == "experts":
        T, E, topk, n, k, fmt = (case["tokens"], case["experts"], case["topk"], case["n"], case["k"], _fmt(case))
        s["x"] = _values(gen, (T, k)).to(torch.bfloat16)
        s["idx"] = _chosen(gen, T, topk, E)
        s["w"] = _packed(gen, n, k, fmt, 0.02, E)
        s["g"] = torch.full((1,), 40.0 / (6 * 448), device="cuda") if fmt == NV else None
        cap = _cap(T, topk, E)
        nb = -(-k // BLOCK[fmt])
        # the most tokens of one expert: the plain form's padded batch
        s["most"] = int(torch.bincount(s["idx"].flatten().long(), minlength=E).max())
        s["slot"] = torch.empty(T, topk, dtype=torch.int32, device="cuda")
        s["row_of"] = torch.empty(cap, dtype=torch.int32, device="cuda")
        s["offsets"] = torch.empty(E + 1, dtype=torch.int32, device="cuda")
        s["counts"] = torch.empty(E, dtype=torch.int32, device="cuda")
        s["codes"] = torch.zeros(cap, -(-k // 32) * 16, dtype=torch.uint8, device="cuda")
        s["scales"] = torch.zeros(cap // TILE, -(-nb // 4), 32, 4, 4, dtype=torch.uint8, device="cuda")
        s["y"] = torch.zeros(cap, n, dtype=torch.bfloat16, device="cuda")
    else:
        T, E, topk, cols = case["tokens"], case["experts"], case["topk"], case["cols"]
        dt = TYPES[case["type"]]
        rows = _cap(T, topk, E)
        s["y"] = torch.randn(rows, cols, generator=gen, device="cuda").to(dt)
        # any different rows will do as slots; a few choices are dropped
        slot = torch.randperm(rows, generator=gen, device="cuda")[:T * topk].reshape(T, topk).to(torch.int32)
        drop = torch.rand(T, topk, generator=gen, device="cuda") < 0.02
        s["slot"] = torch.where(drop, -1, slot)
        s["weights"] = torch.softmax(torch.randn(T, topk, generator=gen, device="cuda"), -1)
        s["out"] = torch.empty(T, cols, dtype=dt, device="cuda")
        if case["train"]:
            s["dout"] = torch.randn(T, cols, generator=gen, device="cuda").to(dt)
            s["dy"] = torch.zeros_like(s["y"])  # rows that no slot names stay zero
            s["dweights"] = torch.empty(T, topk, device="cuda")
    return s


# ----------------------------------------------------------------------------- the plain forms

def _route_plain(s):
    c = s["case"]
    x = s["logits"].float()
    T, E, k, G = c["tokens"], c["experts"], c["topk"], c["groups"]
    low = -math.inf
    ok = x > low
    if c["score"] == "softmax":
        top = x.amax(-1, keepdim=True)
        e = torch.where(ok, torch.exp(x - top), 0.0)
        total = e.sum(-1, keepdim=True)
        score = torch.where(total > 0, e / total, 0.0)
        key = x  # orders as the scores do
    else:
        score = torch.where(ok, 1.0 / (1.0 + torch.exp(-x)), 0.0)
        key = score if s["bias"] is None else score + s["bias"]
    key = torch.where(ok, key, low)
    if G > 1:
        per = key.view(T, G, E // G)
        best = torch.sort(per, dim=-1, descending=True)[0][..., :c["best"]]
        some = best[..., 0] > low
        group = torch.where(some, torch.where(best > low, best, 0.0).sum(-1), low)
        kept = torch.sort(group, dim=-1, descending=True, stable=True)[1][:, :c["keep"]]
        stay = torch.zeros(T, G, dtype=torch.bool, device=x.device).scatter(1, kept, True)
        key = torch.where(stay.unsqueeze(-1), per, low).view(T, E)
    val, idx = torch.sort(key, dim=-1, descending=True, stable=True)
    val, idx = val[:, :k], idx[:, :k]
    have = val > low
    w = torch.where(have, score.gather(1, idx), 0.0)
    S = w.sum(-1, keepdim=True)
    if c["renorm"]:
        if c["score"] == "softmax":
            xs = torch.where(have, x.gather(1, idx), low)
            xs = torch.exp(xs - torch.where(have[:, :1], xs.amax(-1, keepdim=True), 0.0))
            share = torch.where(have, xs / xs.sum(-1, keepdim=True), 0.0)
        else:
            share = torch.where(S > 0, w / S, 0.0)
    else:
        share = w
    out = dict(idx=torch.where(have, idx, -1).to(torch.int32), weights=share * c["scale"])
    if c["train"]:
        g = torch.where(have, s["dweights"] * c["scale"], 0.0)
        if c["score"] == "softmax" and not c["renorm"]:
            full = torch.zeros_like(x).scatter(1, idx, g)
            dx = score * (full - (share * g).sum(-1, keepdim=True))
        else:
            if c["score"] == "softmax":
                d = share * (g - (share * g).sum(-1, keepdim=True))
            elif c["renorm"]:
                d = torch.where(S > 0, (g - (share * g).sum(-1, keepdim=True)) / S, 0.0) * w * (1 - w)
            else:
                d = g * w * (1 - w)
            dx = torch.zeros_like(x).scatter(1, idx, d)
        out["dlogits"] = dx.to(s["logits"].dtype)
    return out


def _order_plain(idx, E, cap):
    """Slots of the choices, sorted by expert and then by choice, each expert at a multiple of 128 rows."""
    T, k = idx.shape
    flat = idx.flatten().long()
    order = torch.argsort(flat, stable=True)
    counts = torch.zeros(E, dtype=torch.long, device=idx.device).scatter_add(0, flat, torch.ones_like(flat))
    ends = torch.cumsum((counts + TILE - 1) // TILE * TILE, 0)
    offsets = torch.nn.functional.pad(ends, (1, 0))
    first = torch.cumsum(counts, 0) - counts
    sorted_e = flat[order]
    row = offsets[sorted_e] + torch.arange(T * k, device=idx.device) - first[sorted_e]
    slot = torch.zeros_like(flat).scatter(0, order, row)
    row_of = torch.full((cap,), -1, dtype=torch.long, device=idx.device).scatter(0, row, order // k)
    return slot.view(T, k), row_of, offsets, counts


def _experts_plain(s):
    c, fmt = s["case"], _fmt(s["case"])
    E, n, k = c["experts"], c["n"], c["k"]
    cap = s["y"].shape[0]
    slot, row_of, offsets, counts = _order_plain(s["idx"], E, cap)
    x = torch.where((row_of >= 0).unsqueeze(1), s["x"].float()[row_of.clamp_min(0)], 0.0)
    q, scale, _ = _quantise(x, fmt, s["g"])
    x = (q * scale.unsqueeze(-1)).flatten(-2)[:, :k]
    x = x if s["g"] is None else x * s["g"]
    codes, scales, g = s["w"]
    w = _decode(codes, scales, None if g is None else g.view(E, 1, 1), n, k, fmt)
    place = torch.arange(s["most"], device=x.device)
    rows = (offsets[:-1].unsqueeze(1) + place).clamp_max(cap - 1)
    y = torch.bmm(x[rows], w.transpose(1, 2))
    mine = (place < counts.unsqueeze(1)).view(-1)
    # places past an expert's count go to a row of their own, which is cut off
    rows = torch.where(mine, rows.view(-1), cap)
    out = torch.zeros(cap + 1, n, device=x.device).index_copy(0, rows, y.view(-1, n))
    return dict(slot=slot.to(torch.int32), counts=counts.to(torch.int32), y=out[:cap].to(torch.bfloat16))


def _combine_plain(s):
    c = s["case"]
    have = (s["slot"] >= 0).unsqueeze(-1)
    at = s["slot"].clamp_min(0).long()
    rows = torch.where(have, s["y"].float()[at], 0.0)
    w = s["weights"].unsqueeze(-1)
    out = dict(out=(rows * w).sum(1).to(s["y"].dtype))
    if c["train"]:
        d = s["dout"].float().unsqueeze(1)
        out["dweights"] = (rows * d).sum(-1)
        n, cols = s["y"].shape
        flat = torch.where(have, at.unsqueeze(-1), n).view(-1)
        out["dy"] = torch.zeros(n + 1, cols, device=w.device).index_copy(0, flat, (w * d).reshape(-1, cols))[:n].to(s["y"].dtype)
    return out


def _plain(s):
    c = s["case"]
    if c["op"] == "route":
        return _route_plain(s)
    if c["op"] == "quantise":
        x = s["x"].float()
        x = x.t() if c["transpose"] else x
        q, scale, _ = _quantise(x, _fmt(c), s["g"])
        v = (q * scale.unsqueeze(-1)).flatten(-2)[:, :x.shape[1]]
        return (v if s["g"] is None else v * s["g"]).to(torch.bfloat16)
    if c["op"] == "product":
        a = _decode(*s["a"], c["m"], c["k"], _fmt(c))
        b = _decode(*s["b"], c["n"], c["k"], _fmt(c))
        return torch.matmul(a, b.t()).to(s["c"].dtype)
    return _experts_plain(s) if c["op"] == "experts" else _combine_plain(s)


# ----------------------------------------------------------------------------- the library's calls

def _records(s, c3):
    """The descriptions of the router and of the 4-bit matrices, and the workspace: what a program keeps."""
    c, op = s["case"], s["case"]["op"]
    if op == "route":
        return c3.Router(c["experts"], c["topk"], score=c3.C3_SCORE_SIGMOID if c["score"] == "sigmoid" else c3.C3_SCORE_SOFTMAX,
                         groups=c["groups"], topk_groups=c["keep"], group_best=c["best"], renorm=c["renorm"],
                         scale=c["scale"], bias=s["bias"], logits_type=CODES[c["type"]])
    fmt = _fmt(c)
    if op == "quantise":
        return c3.Fp4(s["values"].shape[0], s["values"].shape[1], fmt, s["codes"], s["scales"], s["g"])
    if op == "product":
        return tuple(c3.Fp4(r, c["k"], fmt, *q) for r, q in ((c["m"], s["a"]), (c["n"], s["b"])))
    x = c3.Fp4(s["y"].shape[0], c["k"], fmt, s["codes"], s["scales"], s["g"])
    w = c3.Fp4(c["n"], c["k"], fmt, *s["w"], count=c["experts"])
    size = c3.c3_moe_order_bytes(c["tokens"], c["topk"], c["experts"])
    return x, w, torch.empty(size, dtype=torch.uint8, device="cuda")


def _own(s):
    from concurrent_communication_overlap_gb300 import c3
    c, op = s["case"], s["case"]["op"]
    if op == "combine":
        T, topk, cols, ty = c["tokens"], c["topk"], c["cols"], CODES[c["type"]]
        rows = s["y"].shape[0]
        c3.c3_moe_combine(s["y"], ty, rows, cols, s["slot"], s["weights"], T, topk, s["out"], ty)
        if not c["train"]:
            return dict(out=s["out"])
        c3.c3_moe_combine_backward(s["dout"], ty, s["y"], ty, rows, cols, s["slot"], s["weights"], T, topk, s["dy"], s["dweights"])
        return dict(out=s["out"], dweights=s["dweights"], dy=s["dy"])
    if "records" not in s:
        s["records"] = _records(s, c3)
    r = s["records"]
    if op == "route":
        T, E = c["tokens"], c["experts"]
        c3.c3_route(r, s["logits"], E, T, s["idx"], s["weights"])
        if not c["train"]:
            return dict(idx=s["idx"], weights=s["weights"])
        c3.c3_route_backward(r, s["logits"], E, T, s["idx"], s["dweights"], s["dlogits"], E)
        return dict(idx=s["idx"], weights=s["weights"], dlogits=s["dlogits"])
    if op == "quantise":
        c3.c3_fp4_quantize(s["x"], CODES[c["type"]], c["rows"], c["cols"], r, transpose=c["transpose"])
        c3.c3_fp4_dequantize(r, s["values"], BF16, r.cols)
        return s["values"]
    if op == "product":
        c3.c3_fp4_gemm(r[0], r[1], s["c"], CODES[c["out"]])
        return s["c"]
    x, w, work = r
    c3.c3_moe_order(s["idx"], c["tokens"], c["topk"], c["experts"], s["slot"], s["row_of"], s["row_of"].numel(),
                    s["offsets"], s["counts"], work)
    c3.c3_fp4_quantize(s["x"], BF16, c["tokens"], c["k"], x, row_of=s["row_of"])
    c3.c3_fp4_gemm_experts(x, w, s["offsets"], s["counts"], s["y"], BF16)
    return dict(slot=s["slot"], counts=s["counts"], y=s["y"])


def run(state):
    return _own(state) if own else _plain(state)


# ----------------------------------------------------------------------------- what a pass cannot do without

def _fp4_bytes(rows, cols, fmt):
    return rows * cols * (0.5 + 1.0 / BLOCK[fmt])


def work(case):
    op = case["op"]
    size = {"f32": 4, "bf16": 2}
    if op == "route":
        T, E, k, sz = case["tokens"], case["experts"], case["topk"], size[case["type"]]
        b = T * E * sz + 8 * T * k
        if case["train"]:
            b += 2 * T * E * sz + 8 * T * k
        return {"bytes": b, "flops": 10 * T * E}
    if op == "quantise":
        n = case["rows"] * case["cols"]
        return {"bytes": n * (size[case["type"]] + 2) + 2 * _fp4_bytes(case["rows"], case["cols"], _fmt(case)), "flops": 4 * n}
    if op == "product":
        m, n, k, fmt = case["m"], case["n"], case["k"], _fmt(case)
        return {"bytes": _fp4_bytes(m + n, k, fmt) + m * n * size[case["out"]], "flops": 2 * m * n * k}
    if op == "experts":
        T, E, topk, n, k, fmt = (case["tokens"], case["experts"], case["topk"], case["n"], case["k"], _fmt(case))
        rows = T * topk
        busy = min(E, rows)  # the experts that any token can have chosen
        return {"bytes": 2 * T * k + 4 * rows + 2 * _fp4_bytes(rows, k, fmt) + busy * _fp4_bytes(n, k, fmt) + 2 * rows * n + 4 * rows,
                "flops": 2 * rows * n * k}
    T, topk, cols, sz = case["tokens"], case["topk"], case["cols"], size[case["type"]]
    b = T * topk * cols * sz + T * cols * sz + 8 * T * topk
    if case["train"]:
        b += 2 * T * topk * cols * sz + T * cols * sz + 12 * T * topk
    return {"bytes": b, "flops": (6 if case["train"] else 2) * T * topk * cols}


# ----------------------------------------------------------------------------- the definitions, in 64 bits

def _exact_power(e):
    """2^e in 64 bits for whole e, without a rounding."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_fp4(x, fmt, g):
    """The quantised values of x (64 bits) by the formats' definitions."""
    grid = torch.tensor(_VALUES[:8], dtype=torch.float64, device=x.device)
    b = BLOCK[fmt]
    rows, cols = x.shape
    full = torch.zeros(rows, -(-cols // b) * b, dtype=torch.float64, device=x.device)
    full[:, :cols] = x if g is None else x / g.double()
    y = full.view(rows, -1, b)
    amax = y.abs().max(-1, keepdim=True)[0]
    if fmt == MX:
        s = _exact_power(torch.ceil(torch.log2(amax.clamp_min(1e-30) / 6)).clamp(-127, 127))
        s = torch.where(s * 6 < amax, s * 2, torch.where((s * 3 >= amax) & (s > 2.0 ** -127), s / 2, s))
    else:
        t = (amax / 6).clamp(max=448)
        u = _exact_power(torch.floor(torch.log2(t.clamp_min(2.0 ** -6))) - 3)  # the spacing of e4m3 at t
        s = torch.round(t / u) * u
    r = torch.where(s > 0, y / torch.where(s > 0, s, 1.0), 0.0)
    mid = (grid[1:] + grid[:-1]) / 2
    a = r.abs()
    up = torch.bucketize(a, mid, right=False)  # the codes whose lower midpoint lies below a
    tie = up < 7
    tie &= a == mid[up.clamp_max(6)]
    code = torch.where(tie & (up % 2 == 1), up + 1, up)
    v = grid[code] * torch.sign(r) * s
    v = v.view(rows, -1)[:, :cols]
    return v if g is None else v * g.double()


def _exact_values(q, rows, cols, fmt):
    """The values (64 bits) of one packed matrix, read off byte by byte."""
    codes, scales, g = q
    grid = torch.tensor(_VALUES, dtype=torch.float64, device=codes.device)
    col = torch.arange(cols, device=codes.device)
    nib = codes[:, col // 2] >> (4 * (col % 2)).to(torch.uint8) & 15
    row = torch.arange(rows, device=codes.device).unsqueeze(1)
    blk = torch.arange(-(-cols // BLOCK[fmt]), device=codes.device)
    byte = scales[row // TILE, blk // 4, row % 32, row % TILE // 32, blk % 4].double()
    if fmt == MX:
        s = _exact_power(byte - 127)
    else:
        e, m = torch.floor(byte / 8), byte % 8
        s = torch.where(e > 0, (8 + m) * _exact_power(e - 10), m * 2.0 ** -9)
    v = grid[nib.long()] * s.repeat_interleave(BLOCK[fmt], 1)[:, :cols]
    return v if g is None else v * g.double()


def _exact_route(s):
    c = s["case"]
    x = s["logits"].double()
    T, E = x.shape
    ok = ~torch.isneginf(x)
    if c["score"] == "softmax":
        p = torch.nan_to_num(torch.softmax(x, -1), nan=0.0)
        rank = x.clone()
    else:
        p = torch.sigmoid(x)
        rank = p if s["bias"] is None else p + s["bias"].double()
    rank = rank.masked_fill(~ok, -math.inf)
    if c["groups"] > 1:
        per = rank.reshape(T, c["groups"], -1)
        best = per.topk(c["best"], -1)[0]
        total = best.masked_fill(torch.isneginf(best), 0).sum(-1).masked_fill(torch.isneginf(best[..., 0]), -math.inf)
        keep = torch.zeros_like(total, dtype=torch.bool)
        keep.scatter_(1, total.argsort(dim=-1, descending=True, stable=True)[:, :c["keep"]], True)
        rank = per.masked_fill(~keep.unsqueeze(-1), -math.inf).reshape(T, E)
    idx = rank.argsort(dim=-1, descending=True, stable=True)[:, :c["topk"]]
    have = ~torch.isneginf(rank.gather(1, idx))
    taken = torch.zeros(T, E, dtype=torch.bool, device=x.device).scatter(1, idx, have)

    def weights(logits):
        z = torch.softmax(logits, -1) if c["score"] == "softmax" else torch.sigmoid(logits)
        z = z.gather(1, idx) * have
        if c["renorm"]:
            z = z / z.sum(-1, keepdim=True)
        return z * c["scale"]

    out = dict(idx=None)
    if c["train"]:
        dead = ~have.any(-1)
        safe = x.masked_fill(dead.unsqueeze(1), 0.0).requires_grad_(True)
        with torch.enable_grad():
            w = weights(safe)
            w = torch.where(have, w, torch.zeros_like(w))
            (w * s["dweights"].double()).sum().backward()
        dx = safe.grad.masked_fill(dead.unsqueeze(1) | ~ok, 0.0)
        out["dlogits"] = dx if not c["renorm"] and c["score"] == "softmax" else dx * taken
        out["weights"] = w.detach()
    else:
        out["weights"] = torch.where(have, weights(x), torch.zeros((), dtype=torch.float64, device=x.device))
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        return _exact_route(s)
    if op == "quantise":
        x = s["x"].double()
        return _exact_fp4(x.t().contiguous() if case["transpose"] else x, _fmt(case), s["g"])
    if op == "product":
        if 2.0 * case["m"] * case["n"] * case["k"] > 1.2e12:
            return None  # too long in 64 bits
        return _exact_values(s["a"], case["m"], case["k"], _fmt(case)) @ _exact_values(s["b"], case["n"], case["k"], _fmt(case)).t()
    if op == "experts":
        if 2.0 * case["tokens"] * case["topk"] * case["n"] * case["k"] > 1.2e12:
            return None
        fmt, E = _fmt(case), case["experts"]
        x = _exact_fp4(s["x"].double(), fmt, s["g"])
        y = torch.zeros(s["y"].shape, dtype=torch.float64, device="cuda")
        codes, scales, g = s["w"]
        at = 0
        for e in range(E):
            token = (s["idx"] == e).nonzero()[:, 0]
            w = _exact_values((codes[e], scales[e], None if g is None else g[e]), case["n"], case["k"], fmt)
            y[at:at + len(token)] = x[token] @ w.t()
            at += -(-len(token) // TILE) * TILE
        return dict(slot=None, counts=None, y=y)
    slot, w = s["slot"].long(), s["weights"].double()
    y = s["y"].double()
    total = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    dw, dy = torch.zeros_like(w), torch.zeros_like(y)
    d = s["dout"].double() if case["train"] else None
    for j in range(case["topk"]):
        at = (slot[:, j] >= 0).nonzero()[:, 0]
        rows = slot[at, j]
        total[at] += w[at, j].unsqueeze(1) * y[rows]
        if case["train"]:
            dw[at, j] = (d[at] * y[rows]).sum(1)
            dy[rows] = w[at, j].unsqueeze(1) * d[at]
    return dict(out=total, dweights=dw, dy=dy) if case["train"] else dict(out=total)
