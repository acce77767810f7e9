"""Host side of the routing and 4-bit operators: sizes, and the refusals that
come back before any CUDA call (safe without a GPU)."""
import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 0x10000  # an aligned address that is never touched


@pytest.fixture(scope="module")
def c3():
    from concurrent_communication_overlap_gb300 import build
    build.build()
    from concurrent_communication_overlap_gb300 import c3 as mod
    return mod


def test_record_layouts_match_the_header(c3, tmp_path):
    probe = tmp_path / "probe.c"
    probe.write_text(r'''
#include <stdio.h>
#include <stddef.h>
#include "c3_api.h"
#define F(T, f) printf(#T "." #f " %zu\n", offsetof(T, f))
int main(void) {
  printf("c3_router %zu\nc3_fp4 %zu\n", sizeof(c3_router), sizeof(c3_fp4));
  F(c3_router, bias); F(c3_router, experts); F(c3_router, topk); F(c3_router, groups); F(c3_router, topk_groups);
  F(c3_router, group_best); F(c3_router, score); F(c3_router, renorm); F(c3_router, logits_type); F(c3_router, scale);
  F(c3_fp4, codes); F(c3_fp4, scales); F(c3_fp4, tensor_scale); F(c3_fp4, rows); F(c3_fp4, cols); F(c3_fp4, count);
  F(c3_fp4, format);
  return 0;
}
''')
    exe = tmp_path / "probe"
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), str(probe), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout
    cls = {"c3_router": c3.C3Router, "c3_fp4": c3.C3Fp4}
    for line in out.splitlines():
        key, val = line.rsplit(" ", 1)
        if "." in key:
            rec, field = key.split(".")
            assert getattr(cls[rec], field).offset == int(val), key
        else:
            assert ctypes.sizeof(cls[key]) == int(val), key


def test_sizes(c3):
    assert c3.c3_fp4_code_bytes(3, 1) == 3 * 16
    assert c3.c3_fp4_code_bytes(3, 33) == 3 * 32
    assert c3.c3_fp4_code_bytes(0, 33) == 0
    assert c3.c3_fp4_scale_bytes(1, 1, c3.C3_FP4_MX) == 512
    assert c3.c3_fp4_scale_bytes(129, 129, c3.C3_FP4_MX) == 4 * 512
    assert c3.c3_fp4_scale_bytes(129, 129, c3.C3_FP4_NV) == 6 * 512
    assert c3.c3_fp4_scale_bytes(1, 0, c3.C3_FP4_NV) == 0
    assert c3.c3_fp4_scale_bytes(1, 1, 2) == 0
    # the most rows a choice can need: every expert that can be chosen may waste up to 127
    assert c3.c3_moe_rows(0, 4, 8) == 0
    assert c3.c3_moe_rows(1, 1, 8) == 128
    assert c3.c3_moe_rows(1, 4, 8) == 4 * 128
    assert c3.c3_moe_rows(128, 1, 1) == 128
    for tokens, topk, experts in ((5, 3, 4), (100, 2, 7), (129, 1, 2), (1000, 8, 64)):
        n = tokens * topk
        busy = min(experts, n)
        worst = (busy - 1) * 128 + -(-(n - busy + 1) // 128) * 128  # all but one expert get one choice
        assert worst <= c3.c3_moe_rows(tokens, topk, experts) < worst + 128 * busy
    with pytest.raises(c3.C3Error):
        c3.c3_moe_rows(1 << 31, 1, 8)
    with pytest.raises(c3.C3Error):
        c3.c3_moe_rows(4, 33, 64)
    assert c3.c3_moe_order_bytes(4, 33, 64) == 0
    assert c3.c3_moe_order_bytes(4, 2, 64) > 0


@pytest.mark.parametrize("kw", [
    dict(experts=0), dict(experts=1025), dict(topk=0), dict(topk=33, experts=64), dict(topk=9), dict(groups=3),
    dict(groups=0), dict(groups=2, topk_groups=3), dict(groups=2, topk_groups=0), dict(groups=4, topk_groups=1, topk=3),
    dict(group_best=3), dict(group_best=0), dict(groups=8, group_best=2, topk=1), dict(score=2), dict(logits_type=2),
    dict(scale=float("inf")), dict(scale=float("nan"))])
def test_router_records_that_are_refused(c3, kw):
    base = dict(experts=8, topk=2)
    base.update(kw)
    r = c3.Router(**base)
    assert c3.c3_route(r, P, 1 << 12, 4, P, P, check=False) == c3.C3_EINVAL
    assert c3.c3_route_backward(r, P, 1 << 12, 4, P, P, P, 1 << 12, check=False) == c3.C3_EINVAL
    assert c3.c3_last_error()


def test_route_refusals(c3):
    r = c3.Router(8, 2)
    h = c3.Router(8, 2, logits_type=c3.C3_BF16)
    assert c3.c3_route(r, P, 8, 0, None, None, check=False) == c3.C3_OK
    assert c3.c3_route(r, P, 7, 4, P, P, check=False) == c3.C3_EINVAL
    assert c3.c3_route(r, P, 8, -1, P, P, check=False) == c3.C3_EINVAL
    assert c3.c3_route(r, P, 8, 1 << 30, P, P, check=False) == c3.C3_EUNSUP
    assert c3.c3_route(r, None, 8, 4, P, P, check=False) == c3.C3_EINVAL
    assert c3.c3_route(r, P, 8, 4, None, P, check=False) == c3.C3_EINVAL
    assert c3.c3_route(r, P, 8, 4, P, None, check=False) == c3.C3_EINVAL
    assert c3.c3_route(r, P + 2, 8, 4, P, P, check=False) == c3.C3_EALIGN
    assert c3.c3_route(h, P + 1, 8, 4, P, P, check=False) == c3.C3_EALIGN
    assert c3.c3_route(r, P, 8, 4, P + 2, P, check=False) == c3.C3_EALIGN
    assert c3.c3_route(c3.Router(8, 2, bias=P + 2), P, 8, 4, P, P, check=False) == c3.C3_EALIGN
    assert c3.lib().c3_route(None, P, 8, 4, P, P, None) == c3.C3_EINVAL
    assert c3.c3_route_backward(r, P, 8, 4, P, P, P, 7, check=False) == c3.C3_EINVAL
    assert c3.c3_route_backward(r, P, 8, 4, P, P, None, 8, check=False) == c3.C3_EINVAL
    assert c3.c3_route_backward(r, P, 8, 4, P, None, P, 8, check=False) == c3.C3_EINVAL
    assert c3.c3_route_backward(r, P, 8, 4, P, P, P + 2, 8, check=False) == c3.C3_EALIGN
    assert c3.c3_route_backward(r, P, 8, 0, None, None, None, 8, check=False) == c3.C3_OK


def test_order_refusals(c3):
    def order(idx=P, tokens=4, topk=2, experts=8, slot=P, row_of=P, rows=4096, offsets=P, counts=P, work=P, nbytes=1 << 20):
        return c3.c3_moe_order(idx, tokens, topk, experts, slot, row_of, rows, offsets, counts, work, nbytes, check=False)
    assert order(tokens=-1) == c3.C3_EINVAL
    assert order(topk=0) == c3.C3_EINVAL
    assert order(experts=0) == c3.C3_EINVAL
    assert order(experts=1025) == c3.C3_EINVAL
    assert order(rows=c3.c3_moe_rows(4, 2, 8) - 1) == c3.C3_EINVAL
    assert order(rows=1 << 31) == c3.C3_EINVAL
    assert order(nbytes=c3.c3_moe_order_bytes(4, 2, 8) - 1) == c3.C3_EINVAL
    for name in ("idx", "slot", "row_of", "offsets", "counts", "work"):
        assert order(**{name: None}) == c3.C3_EINVAL, name
        assert order(**{name: P + 2}) == c3.C3_EALIGN, name


def test_fp4_refusals(c3):
    def m(rows=4, cols=64, fmt=0, codes=P, scales=P, g=None, count=1):
        return c3.Fp4(rows, cols, fmt, codes, scales, g, count)
    bad = [(m(rows=-1), c3.C3_EINVAL), (m(cols=0), c3.C3_EINVAL), (m(count=0), c3.C3_EINVAL), (m(fmt=2), c3.C3_EINVAL),
           (m(codes=None), c3.C3_EINVAL), (m(scales=None), c3.C3_EINVAL), (m(codes=P + 8), c3.C3_EALIGN),
           (m(scales=P + 8), c3.C3_EALIGN), (m(g=P), c3.C3_EINVAL), (m(fmt=1, g=P + 2), c3.C3_EALIGN),
           (m(rows=1 << 30, count=4), c3.C3_EUNSUP)]
    for q, want in bad:
        assert c3.c3_fp4_quantize(P, 0, q.rows, max(q.cols, 0), q, check=False) == want
        assert c3.c3_fp4_dequantize(q, P, 0, 1 << 12, check=False) == want
        assert c3.c3_fp4_gemm(q, m(), P, 0, check=False) == want
        assert c3.c3_fp4_gemm(m(), q, P, 0, check=False) == want
        assert c3.c3_fp4_gemm_experts(q, m(), P, P, P, 0, check=False) == want
    q = m()
    for kw, want in ((dict(x=None), -1), (dict(x=P + 2), -2), (dict(x_type=2), -1), (dict(x_rows=5), -1),
                     (dict(x_cols=63), -1), (dict(ld=63), -1), (dict(transpose=True), -1), (dict(transpose=2), -1),
                     (dict(row_of=P, x_cols=60), -1), (dict(row_of=P + 2), -2), (dict(x_rows=-4), -1)):
        a = dict(x=P, x_type=0, x_rows=4, x_cols=64, ld=None, transpose=False, row_of=None)
        a.update(kw)
        assert c3.c3_fp4_quantize(a["x"], a["x_type"], a["x_rows"], a["x_cols"], q, ld=a["ld"],
                                  transpose=a["transpose"], row_of=a["row_of"], check=False) == want, kw
    assert c3.c3_fp4_quantize(P, 0, 64, 4, q, transpose=True, row_of=P, check=False) == c3.C3_EINVAL
    assert c3.c3_fp4_quantize(P, 0, 4, 64, m(count=2), row_of=P, check=False) == c3.C3_EINVAL
    assert c3.c3_fp4_quantize(P, 0, 0, 64, m(rows=0), check=False) == c3.C3_OK
    assert c3.c3_fp4_dequantize(q, P, 2, 64, check=False) == c3.C3_EINVAL
    assert c3.c3_fp4_dequantize(q, P, 0, 63, check=False) == c3.C3_EINVAL
    assert c3.c3_fp4_dequantize(q, None, 0, 64, check=False) == c3.C3_EINVAL
    assert c3.c3_fp4_dequantize(q, P + 2, 0, 64, check=False) == c3.C3_EALIGN
    assert c3.c3_fp4_dequantize(m(rows=0), None, 0, 64, check=False) == c3.C3_OK


def test_product_refusals(c3):
    def m(rows=4, cols=64, fmt=0, count=1):
        return c3.Fp4(rows, cols, fmt, P, P, None, count)
    assert c3.c3_fp4_gemm(m(), m(cols=96), P, 0, check=False) == c3.C3_EINVAL
    assert c3.c3_fp4_gemm(m(), m(fmt=1), P, 0, check=False) == c3.C3_EINVAL
    assert c3.c3_fp4_gemm(m(), m(count=2), P, 0, check=False) == c3.C3_EINVAL
    assert c3.c3_fp4_gemm(m(count=2), m(), P, 0, check=False) == c3.C3_EINVAL
    assert c3.c3_fp4_gemm(m(), m(), P, 2, check=False) == c3.C3_EINVAL
    assert c3.c3_fp4_gemm(m(), m(), P, 0, sm_budget=-1, check=False) == c3.C3_EINVAL
    assert c3.c3_fp4_gemm(m(), m(), None, 0, check=False) == c3.C3_EINVAL
    assert c3.c3_fp4_gemm(m(), m(), P + 4, 0, check=False) == c3.C3_EALIGN
    assert c3.c3_fp4_gemm(m(rows=0), m(), None, 0, check=False) == c3.C3_OK
    assert c3.lib().c3_fp4_gemm(None, m().ref, P, 0, 0, None) == c3.C3_EINVAL
    assert c3.c3_fp4_gemm_experts(m(), m(count=4), None, P, P, 0, check=False) == c3.C3_EINVAL
    assert c3.c3_fp4_gemm_experts(m(), m(count=4), P, None, P, 0, check=False) == c3.C3_EINVAL
    assert c3.c3_fp4_gemm_experts(m(), m(count=4), P + 2, P, P, 0, check=False) == c3.C3_EALIGN
    assert c3.c3_fp4_gemm_experts(m(), m(count=1025), P, P, P, 0, check=False) == c3.C3_EINVAL
    assert c3.c3_fp4_gemm_experts(m(count=2), m(), P, P, P, 0, check=False) == c3.C3_EINVAL
    assert c3.c3_fp4_gemm_experts(m(rows=0), m(count=4), P, P, None, 0, check=False) == c3.C3_OK


def test_combine_refusals(c3):
    def fwd(y=P, yt=0, rows=8, cols=4, slot=P, w=P, tokens=2, topk=2, out=P, ot=0):
        return c3.c3_moe_combine(y, yt, rows, cols, slot, w, tokens, topk, out, ot, check=False)

    def bwd(d=P, dt=0, y=P, yt=0, rows=8, cols=4, slot=P, w=P, tokens=2, topk=2, dy=P, dw=P):
        return c3.c3_moe_combine_backward(d, dt, y, yt, rows, cols, slot, w, tokens, topk, dy, dw, check=False)
    for f in (fwd, bwd):
        assert f(yt=2) == c3.C3_EINVAL
        assert f(rows=-1) == c3.C3_EINVAL
        assert f(cols=-1) == c3.C3_EINVAL
        assert f(tokens=-1) == c3.C3_EINVAL
        assert f(topk=33) == c3.C3_EINVAL
        assert f(rows=1 << 31) == c3.C3_EUNSUP
        assert f(slot=None) == c3.C3_EINVAL
        assert f(slot=P + 2) == c3.C3_EALIGN
        assert f(w=P + 2) == c3.C3_EALIGN
        assert f(y=None) == c3.C3_EINVAL
        assert f(y=P + 2) == c3.C3_EALIGN
        assert f(tokens=0) == c3.C3_OK
    assert fwd(out=None) == c3.C3_EINVAL
    assert fwd(ot=3) == c3.C3_EINVAL
    assert fwd(cols=0) == c3.C3_OK
    assert bwd(d=None) == c3.C3_EINVAL
    assert bwd(dy=None) == c3.C3_EINVAL
    assert bwd(dt=3) == c3.C3_EINVAL
    assert bwd(dw=P + 2) == c3.C3_EALIGN
