"""A sparse layer on the library's operators, forward and backward.

    out[t] = sum_j w[t, j] * W[e(t, j)] x[t]

The router chooses `topk` of `experts` matrices for each token.  The matrices are
stored over 8 virtual ranks, in 4 bits: a rank's shard is its experts' codes and
scales.  Before they are used, c3_allgather puts the shards together on a second
stream, while the first stream routes the tokens, sorts them by expert and
quantises their rows: the gather moves 4.25 bits a weight where bf16 would move 16.

  forward   c3_route, c3_moe_order, c3_fp4_quantize (rows gathered by expert),
            c3_fp4_gemm_experts, c3_moe_combine
  backward  c3_moe_combine_backward, c3_fp4_quantize, c3_fp4_gemm_experts with the
            transposed matrices, c3_moe_combine (weights of one) for the tokens'
            gradient, c3_route_backward for the logits'

Quantisation passes gradients straight through.  `python examples/sparse_layer.py`
times a step and compares the bytes the gather moves.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from concurrent_communication_overlap_gb300 import c3  # noqa: E402

RANKS = 8


class ShardedWeights:
    """One 4-bit operand of all experts: shards over the ranks, and the gathered copy."""

    def __init__(self, weights, transpose):
        experts, n, k = weights.shape
        rows, cols = (k, n) if transpose else (n, k)
        self.rows, self.cols, self.experts = rows, cols, experts
        per = experts // RANKS
        code, scale = c3.c3_fp4_code_bytes(rows, cols), c3.c3_fp4_scale_bytes(rows, cols, c3.C3_FP4_MX)
        self.shards = []
        for r in range(RANKS):
            codes = torch.empty(per * code, dtype=torch.uint8, device="cuda")
            scales = torch.zeros(per * scale, dtype=torch.uint8, device="cuda")
            q = c3.Fp4(rows, cols, c3.C3_FP4_MX, codes, scales, count=per)
            c3.c3_fp4_quantize(weights[r * per:(r + 1) * per], c3.C3_BF16, n, k, q, transpose=transpose)
            self.shards.append((codes, scales))
        self.codes = torch.empty(experts * code, dtype=torch.uint8, device="cuda")
        self.scales = torch.empty(experts * scale, dtype=torch.uint8, device="cuda")
        self.matrix = c3.Fp4(rows, cols, c3.C3_FP4_MX, self.codes, self.scales, count=experts)

    def gather(self, stream):
        for i, out in enumerate((self.codes, self.scales)):
            parts = [s[i] for s in self.shards]
            c3.c3_allgather(parts, out, parts[0].numel(), RANKS, stream=stream)


class SparseLayer:
    """weights: bf16 [experts][n][k], experts a multiple of 8; tokens: how many a step takes."""

    def __init__(self, weights, topk, tokens, router=None):
        self.experts, self.n, self.k = weights.shape
        if self.experts % RANKS:
            raise ValueError("experts must be a multiple of 8")
        self.topk, self.tokens = topk, tokens
        self.forward_weights = ShardedWeights(weights, transpose=False)
        self.backward_weights = ShardedWeights(weights, transpose=True)
        self.router = router or c3.Router(self.experts, topk, renorm=True)
        self.rows = c3.c3_moe_rows(tokens, topk, self.experts)
        new = lambda shape, dtype: torch.empty(shape, dtype=dtype, device="cuda")  # noqa: E731
        self.idx, self.weights = new((tokens, topk), torch.int32), new((tokens, topk), torch.float32)
        self.slot, self.row_of = new((tokens, topk), torch.int32), new(self.rows, torch.int32)
        self.offsets, self.counts = new(self.experts + 1, torch.int32), new(self.experts, torch.int32)
        self.work = new(max(16, c3.c3_moe_order_bytes(tokens, topk, self.experts)), torch.uint8)
        self.x_rows, self.dy_rows = self._operand(self.k), self._operand(self.n)
        self.y, self.dy = (torch.zeros(self.rows, self.n, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.dx_rows = torch.zeros(self.rows, self.k, dtype=torch.bfloat16, device="cuda")
        self.out, self.dx = new((tokens, self.n), torch.bfloat16), new((tokens, self.k), torch.bfloat16)
        self.dweights, self.dlogits = new((tokens, topk), torch.float32), new((tokens, self.experts), torch.float32)
        self.side = torch.cuda.Stream()

    def _operand(self, cols):
        codes = torch.zeros(c3.c3_fp4_code_bytes(self.rows, cols), dtype=torch.uint8, device="cuda")
        scales = torch.zeros(c3.c3_fp4_scale_bytes(self.rows, cols, c3.C3_FP4_MX), dtype=torch.uint8, device="cuda")
        return c3.Fp4(self.rows, cols, c3.C3_FP4_MX, codes, scales)

    def _gather_beside(self, weights, work):
        """Gather on the second stream while `work` runs on the current one; both are done afterwards."""
        here = torch.cuda.current_stream()
        self.side.wait_stream(here)
        weights.gather(self.side)
        work(here)
        here.wait_stream(self.side)
        return here

    def forward(self, x, logits):
        """x bf16 [tokens][k], logits fp32 [tokens][experts] -> out bf16 [tokens][n]."""
        T, E = self.tokens, self.experts

        def rows(s):
            c3.c3_route(self.router, logits, E, T, self.idx, self.weights, stream=s)
            c3.c3_moe_order(self.idx, T, self.topk, E, self.slot, self.row_of, self.rows, self.offsets, self.counts,
                            self.work, stream=s)
            c3.c3_fp4_quantize(x, c3.C3_BF16, T, self.k, self.x_rows, row_of=self.row_of, stream=s)

        s = self._gather_beside(self.forward_weights, rows)
        c3.c3_fp4_gemm_experts(self.x_rows, self.forward_weights.matrix, self.offsets, self.counts, self.y, c3.C3_BF16,
                               stream=s)
        c3.c3_moe_combine(self.y, c3.C3_BF16, self.rows, self.n, self.slot, self.weights, T, self.topk, self.out,
                          c3.C3_BF16, stream=s)
        return self.out

    def backward(self, logits, dout):
        """The gradients with respect to x (bf16) and to the logits (fp32) of the last forward pass."""
        T, E = self.tokens, self.experts

        def rows(s):
            c3.c3_moe_combine_backward(dout, c3.C3_BF16, self.y, c3.C3_BF16, self.rows, self.n, self.slot,
                                       self.weights, T, self.topk, self.dy, self.dweights, stream=s)
            c3.c3_route_backward(self.router, logits, E, T, self.idx, self.dweights, self.dlogits, E, stream=s)
            c3.c3_fp4_quantize(self.dy, c3.C3_BF16, self.rows, self.n, self.dy_rows, stream=s)

        s = self._gather_beside(self.backward_weights, rows)
        c3.c3_fp4_gemm_experts(self.dy_rows, self.backward_weights.matrix, self.offsets, self.counts, self.dx_rows,
                               c3.C3_BF16, stream=s)
        c3.c3_moe_combine(self.dx_rows, c3.C3_BF16, self.rows, self.k, self.slot, None, T, self.topk, self.dx,
                          c3.C3_BF16, stream=s)
        return self.dx, self.dlogits


def main():
    experts, n, k, topk, tokens = 32, 4096, 4096, 4, 8192
    gen = torch.Generator(device="cuda").manual_seed(0)
    w = (torch.randn(experts, n, k, generator=gen, device="cuda") * 0.02).to(torch.bfloat16)
    layer = SparseLayer(w, topk, tokens)
    x = torch.randn(tokens, k, generator=gen, device="cuda").to(torch.bfloat16)
    logits = torch.randn(tokens, experts, generator=gen, device="cuda")
    dout = torch.randn(tokens, n, generator=gen, device="cuda").to(torch.bfloat16)
    begin, middle, end = (torch.cuda.Event(enable_timing=True) for _ in range(3))
    for _ in range(5):
        begin.record()
        layer.forward(x, logits)
        middle.record()
        layer.backward(logits, dout)
        end.record()
    torch.cuda.synchronize()
    c3.c3_status_check()
    bits = 8 * (layer.forward_weights.codes.numel() + layer.forward_weights.scales.numel()) / w.numel()
    print(f"{tokens} tokens, {topk} of {experts} experts {n} x {k}: forward {begin.elapsed_time(middle) * 1e3:.0f} us, "
          f"backward {middle.elapsed_time(end) * 1e3:.0f} us; a gathered weight takes {bits:.2f} bits")


if __name__ == "__main__":
    main()
