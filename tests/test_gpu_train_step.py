"""The two ends of a data-parallel training step on eight virtual ranks, as a program would run them, against the same
in 64 bits: each rank looks the tokens up in its shard of the vocabulary and the all-reduce adds the shards'
rows up; the gradient of the rows goes back into each rank's shard over two micro-batches; shards of a momentum are
gathered on a second stream and orthogonalised.  Eagerly, and captured into a graph with other inputs at replay.

Tolerances (u = 2^-24, h = 2^-8, f = 2^-11): lookups are one product each and the all-reduce adds zeros: u.  A row of
the gradient is a sum of k terms over both micro-batches, (k + 4) u of scale * sum |d|.  The update: three roundings a
step of f, each carried on by a slope of at most 3.4445, and h for the output, in the 2-norm."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from test_gpu_ops import c3, f64  # noqa: F401

pytestmark = pytest.mark.gpu

U, H, F = 2.0 ** -24, 2.0 ** -8, 2.0 ** -11
RANKS = 8
QUINTIC = (3.4445, -4.7750, 2.0315)


class Step:
    def __init__(self, c3, per, cols, tokens, wrows, wcols):  # noqa: F811
        self.c3, self.per, self.cols, self.tokens, self.wrows, self.wcols = c3, per, cols, tokens, wrows, wcols
        new = lambda *s, dtype=torch.float32: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
        self.count = -(-tokens * cols // (4 * RANKS)) * 4 * RANKS
        self.tables = [new(per, cols, dtype=torch.bfloat16) for _ in range(RANKS)]
        self.ids = [new(tokens, dtype=torch.int32) for _ in range(2)]
        self.douts = [new(tokens, cols, dtype=torch.bfloat16) for _ in range(2)]
        self.parts = [new(self.count) for _ in range(RANKS)]
        self.rows = new(RANKS, self.count)
        self.grads = [new(per, cols) for _ in range(RANKS)]
        self.shards = [new(wrows // RANKS * wcols, dtype=torch.bfloat16) for _ in range(RANKS)]
        self.momentum, self.update = (new(wrows, wcols, dtype=torch.bfloat16) for _ in range(2))
        # a workspace for each of the calls that may run side by side
        self.work = torch.empty(c3.c3_embed_backward_bytes(tokens, per, cols), dtype=torch.uint8, device="cuda")
        self.owork = torch.empty(c3.c3_orthogonalize_bytes(wrows, wcols), dtype=torch.uint8, device="cuda")
        self.side = torch.cuda.Stream()

    def fill(self, rng):
        vocab = RANKS * self.per
        for t in self.tables + self.douts + self.shards:
            t.copy_(torch.from_numpy(rng.standard_normal(tuple(t.shape)).astype(np.float32)))
        for t in self.ids:
            ids = np.where(rng.random(self.tokens) < 0.5, rng.integers(0, 5, self.tokens) * 13 % vocab, rng.integers(-9, vocab, self.tokens))
            t.copy_(torch.from_numpy(ids.astype(np.int32)))

    def run(self):
        c3, here = self.c3, torch.cuda.current_stream()  # noqa: F811
        self.side.wait_stream(here)
        c3.c3_allgather(self.shards, self.momentum, self.shards[0].numel() * 2, RANKS, stream=self.side)
        c3.c3_orthogonalize(self.momentum, c3.C3_BF16, self.wrows, self.wcols, self.update, self.owork, [QUINTIC] * 5, scale=0.2,
                            stream=self.side)
        for r in range(RANKS):
            c3.c3_embed(self.tables[r], c3.C3_BF16, self.per, self.cols, self.ids[0], self.tokens, self.parts[r], c3.C3_F32, scale=4.0,
                        first=r * self.per, stream=here)
        c3.c3_allreduce(self.parts, self.rows, self.count, RANKS, stream=here)
        for r in range(RANKS):
            for k in range(2):
                c3.c3_embed_backward(self.douts[k], c3.C3_BF16, self.ids[k], self.tokens, self.grads[r], c3.C3_F32, self.per, self.cols,
                                     self.work, scale=4.0, first=r * self.per, accumulate=k > 0, stream=here)
        here.wait_stream(self.side)

    def check(self):
        table = np.concatenate([f64(t) for t in self.tables])
        ids = [t.cpu().numpy().astype(np.int64) for t in self.ids]
        have = ids[0] >= 0
        ref = np.where(have[:, None], table[np.clip(ids[0], 0, None)] * 4.0, 0)
        for r in (0, RANKS - 1):
            got = f64(self.rows[r, :self.tokens * self.cols]).reshape(self.tokens, self.cols)
            assert (np.abs(got - ref) <= U * np.abs(ref)).all()
        total, mag, many = (np.zeros_like(table) for _ in range(3))
        for i, d in zip(ids, self.douts):
            mine = np.nonzero(i >= 0)[0]
            np.add.at(total, i[mine], 4.0 * f64(d)[mine])
            np.add.at(mag, i[mine], 4.0 * np.abs(f64(d)[mine]))
            np.add.at(many, i[mine], 1.0)
        got = np.concatenate([f64(t) for t in self.grads])
        assert (np.abs(got - total) <= (many + 4) * U * mag).all()
        x = torch.cat([s.view(-1, self.wcols) for s in self.shards]).double()
        assert torch.equal(self.momentum.double(), x)
        x = x / (torch.linalg.vector_norm(x) + 1e-7)
        a, b, c = np.asarray(QUINTIC, np.float32).astype(np.float64)
        for _ in range(5):
            g = x.T @ x if self.wrows > self.wcols else x @ x.T
            x = a * x + (x @ (b * g + c * (g @ g)) if self.wrows > self.wcols else (b * g + c * (g @ g)) @ x)
        off = torch.linalg.vector_norm(self.update.double() - 0.2 * x) / torch.linalg.vector_norm(0.2 * x)
        assert off <= 3.4445 * F * 15 ** 0.5 + H
        self.c3.c3_status_check()


@pytest.mark.parametrize("per,cols,tokens,wrows,wcols", [(50, 40, 100, 64, 96), (333, 129, 1000, 520, 264), (1000, 256, 5000, 256, 1200)])
def test_eager_and_captured(c3, per, cols, tokens, wrows, wcols):  # noqa: F811
    rng = np.random.default_rng(per)
    step = Step(c3, per, cols, tokens, wrows, wcols)
    step.fill(rng)
    step.run()
    torch.cuda.synchronize()
    step.check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.run()
    for _ in range(2):
        step.fill(rng)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        step.check()
