"""Host side of the orthogonalisation: sizes, the refusals that come back before any CUDA call, and the powers of
two that its fp16 matrices are held in (ortho_plan.h)."""
import math
import os
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "concurrent_communication_overlap_gb300", "csrc")
P = 0x10000  # an aligned address that is never touched
QUINTIC = (3.4445, -4.7750, 2.0315)


@pytest.fixture(scope="module")
def c3():
    from concurrent_communication_overlap_gb300 import build
    build.build()
    from concurrent_communication_overlap_gb300 import c3 as mod
    return mod


def test_workspace_sizes(c3):
    size = c3.c3_orthogonalize_bytes
    assert size(-1, 8) == size(8, -1) == size(8, 8, -1) == size(1 << 25, 8) == size(8, 1 << 25) == size(8, 8, 65536) == 0
    # two fp16 copies of x and two square matrices on the shorter side, rows of whole 32 bytes
    for m, n, k in ((1, 1, 1), (5, 9, 3), (300, 77, 2), (1024, 1000, 7), (4096, 4096, 1)):
        s = min(m, n)
        need = k * (2 * m * -(-n // 16) * 32 + 2 * s * -(-s // 16) * 32)
        parts = 160 * 256 * 256 * 4 if max(m, n) > 448 else 0  # fp32 sums of parts of products
        assert need + parts <= size(m, n, k) <= need + parts + k * 512 * 8 + 4 * k + 80 * 64 + 2048, (m, n, k)


def test_refusals(c3):
    def f(x=P, type=0, rows=8, cols=4, out=P, work=P, coeffs=[QUINTIC] * 5, nbytes=1 << 24, **kw):  # noqa: B006
        return c3.c3_orthogonalize(x, type, rows, cols, out, work, coeffs, work_bytes=nbytes, check=False, **kw)
    need = c3.c3_orthogonalize_bytes(8, 4)
    inf, nan = float("inf"), float("nan")
    for kw in (dict(type=2), dict(rows=-1), dict(cols=-1), dict(count=-1), dict(ld=3), dict(out_ld=3), dict(coeffs=[]),
               dict(coeffs=None), dict(coeffs=[QUINTIC] * 33), dict(coeffs=[(nan, 0, 0)]), dict(coeffs=[(1, 0, inf)]),
               dict(coeffs=[(100, 0, 0)] * 8), dict(eps=-1e-9), dict(eps=nan), dict(eps=inf), dict(scale=nan), dict(x=None),
               dict(out=None), dict(work=None), dict(nbytes=need - 1), dict(sm_budget=-1), dict(sm_budget=1)):
        assert f(**kw) == c3.C3_EINVAL, kw
        assert c3.c3_last_error()
    for kw in (dict(rows=1 << 25), dict(cols=1 << 25, ld=1 << 25, out_ld=1 << 25), dict(count=65536)):
        assert f(**kw) == c3.C3_EUNSUP, kw
    # sizes whose workspace would pass 64 bits, and the first above the limit
    for m, n, k in ((1 << 24, 1 << 24, 65535), (1 << 24, 1 << 24, 1), (1 << 20, 1 << 20, 2), (1 << 16, (1 << 24) - 1, 2)):
        assert f(rows=m, cols=n, count=k, nbytes=2 ** 64 - 1) == c3.C3_EUNSUP, (m, n, k)
        assert c3.c3_orthogonalize_bytes(m, n, k) == 0
    assert c3.c3_orthogonalize_bytes(1 << 20, 1 << 20) > 1 << 43
    for kw in (dict(x=P + 2), dict(x=P + 1, type=1), dict(out=P + 1), dict(work=P + 16)):
        assert f(**kw) == c3.C3_EALIGN, kw
    for kw in (dict(rows=0), dict(cols=0), dict(count=0)):
        assert f(x=None, out=None, work=None, **kw) == c3.C3_OK, kw


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    at = tmp_path_factory.mktemp("plan")
    src = at / "plan.cpp"
    src.write_text(r'''
#include <cstdio>
#include <cstdlib>
#include "ortho_plan.h"
int main(int n, char** v) {
  if (v[1][0] == 't') {
    const c3::OrthoTiles t{atoi(v[2]), atoi(v[3]), atoi(v[4])};
    printf("%lld", (long long)t.total());
    for (int i = 0; i <= t.rows; ++i) printf(" %lld", (long long)t.before(i));
    return 0;
  }
  if (v[1][0] == 's') {
    const c3::OrthoPlan p = c3::ortho_plan(atoll(v[2]), atoll(v[3]), atoi(v[4]) != 0, atoi(v[5]), atoi(v[6]), atoi(v[7]));
    const c3::OrthoSplit& s = p.cut;
    printf("%d %lld %d %d\n", p.nt, (long long)p.total, s.split, s.runs);
    if (s.runs) {
      for (int r = 0; r <= s.runs; ++r) printf("%lld ", (long long)s.begin(r));
      printf("\n");
      for (long long u = 0; u < (long long)s.split * s.num_kb; ++u) printf("%d ", s.run_of((unsigned)u));
    }
    return 0;
  }
  float c[c3::kOrthoSteps][3];
  const int steps = (n - 1) / 3;
  for (int i = 0; i < 3 * steps; ++i) c[i / 3][i % 3] = (float)atof(v[1 + i]);
  c3::OrthoStep s[c3::kOrthoSteps];
  if (!c3::ortho_steps(c, steps, s)) { printf("no\n"); return 0; }
  for (int i = 0; i < steps; ++i) printf("%d %d %d %d\n", s[i].x, s[i].g, s[i].p, s[i].next);
}
''')
    exe = at / "plan"
    subprocess.run(["g++", "-std=c++17", "-I", CSRC, str(src), "-o", str(exe)], check=True)

    def run(*args):
        return subprocess.run([str(exe), *map(str, args)], capture_output=True, text=True, check=True).stdout
    return run


@pytest.mark.parametrize("coeffs", [
    [QUINTIC] * 6, [(1.5, -0.5, 0)] * 9, [(1, 0, 0)], [(-2, 0.5, -0.1)] * 3, [(0, 0, 0)] * 2, [(2, -1.5, 0.5)] * 4,
    [(8.28721, -23.5959, 17.3004), (4.1071, -2.9479, 0.5448), (3.9487, -2.9089, 0.5518), (2.3037, -1.6904, 0.4189)],
    [(0, 0, 1)] * 2, [(0, -3, 0), (5, 1, 1)]])
def test_powers_keep_every_matrix_within_fp16(plan, coeffs):
    """Singular values from 0 to 1, followed through the steps: entries are at most them, and what is stored stays
    8 times below fp16's largest.  Where the bound is not tiny it lies above 2^8, so that entries down to 2^-22 of the
    largest keep 11 bits (the planner's bound grows by 0.2% a step and by the polynomial's steepness there)."""
    lines = plan(*[v for c in coeffs for v in c]).split("\n")
    s = np.linspace(0, 1, 200001)
    for (a, b, c), line in zip(coeffs, lines):
        x, g, p, nxt = map(int, line.split())
        poly = np.abs(a + b * s ** 2 + c * s ** 4)
        t = s * poly
        for power, top in ((x, s.max()), (g, (s * s).max()), (p, poly.max()), (nxt, t.max())):
            assert top * 2.0 ** power <= 2.0 ** 13 * 1.0001
            assert top < 1e-5 or top * 2.0 ** power >= 2.0 ** 8
        s = t


def test_coefficients_that_run_away(plan):
    assert plan(*[100, 0, 0] * 8).strip() == "no"
    assert plan(*[3e38, 0, 0]).strip() == "no"
    assert plan(*[100, 0, 0] * 3).strip() != "no"


@pytest.mark.parametrize("n,width", [(1, 256), (256, 256), (257, 256), (1000, 128), (1024, 128), (5000, 256), (300, 128)])
def test_tiles_cover_the_upper_triangle_once(plan, n, width):
    rows, cols, skip = math.ceil(n / 256), math.ceil(n / width), 256 // width
    out = list(map(int, plan("t", rows, cols, skip).split()))
    total, before = out[0], out[1:]
    seen = set()
    for t in range(total):
        i = max(k for k in range(rows) if before[k] <= t)
        seen.add((i, t - before[i] + skip * i))
    want = {(i, j) for i in range(rows) for j in range(cols) if (j + 1) * width > i * 256}
    assert seen == want and total == len(want)


# M, N, symmetric, K blocks, matrices, pairs and what the plan is to be: tiles' width, whether some are cut
PLANS = [
    (1347, 1347, 1, 79, 1, 76, 128, True), (5003, 1347, 0, 22, 1, 76, 256, False), (200, 200, 1, 141, 1, 76, 128, True),
    (4096, 4096, 1, 64, 1, 76, 256, False), (4096, 4096, 0, 64, 1, 76, 256, True), (1024, 1024, 1, 32, 16, 76, 256, True),
    (256, 640, 0, 4, 1, 76, 128, False), (256, 256, 1, 10, 1, 76, 128, False), (8192, 28672, 0, 128, 1, 76, 256, True),
    (1024, 1024, 1, 16, 1, 76, 128, False), (3000, 700, 0, 11, 1, 17, 256, False), (700, 700, 1, 47, 1, 17, 128, False),
    (700, 700, 1, 79, 1, 76, 128, True), (300, 5000, 0, 500, 3, 1, 256, False), (2600, 2700, 0, 41, 1, 76, 256, True),
    (1, 1, 1, 3, 1, 76, 128, False)]


@pytest.mark.parametrize("M,N,sym,num_kb,count,pairs,nt,cut", PLANS)
def test_a_products_tiles_are_dealt_out_once(plan, M, N, sym, num_kb, count, pairs, nt, cut):
    """Every K block of every tile that is left over goes to one pair, no run is longer than a tile, and the runs that
    a block's tile is put together from are those that have a part of it."""
    out = plan("s", M, N, sym, num_kb, count, pairs).split("\n")
    got_nt, total, split, runs = map(int, out[0].split())
    rows, cols = -(-M // 256), -(-N // got_nt)
    assert total == count * (sum(cols - 256 // got_nt * i for i in range(rows)) if sym else rows * cols)
    assert (got_nt, runs > 0) == (nt, cut)
    assert split == 0 or (split == total % pairs and split < runs <= min(pairs, 80) and num_kb >= 8)
    if not split:
        return
    begin = list(map(int, out[1].split()))
    assert begin[0] == 0 and begin[-1] == split * num_kb and len(begin) == runs + 1
    assert all(3 <= b - a <= num_kb for a, b in zip(begin, begin[1:]))
    owner = list(map(int, out[2].split()))
    assert owner == [max(q for q in range(runs) if begin[q] <= u) for u in range(split * num_kb)]


@pytest.mark.parametrize("coeffs", [
    [(3, -3, c), (1.5, -0.5, 0)] for c in (1e-16, -1e-16, 1e-12, 1e-7, -1e-7, 1e-30, 1e-38)] + [
    [(1e-30, -3, 1e-16), (5, 1, 1)], [(3, -3e-16, -3), (1, 0, 0)], [(2, 0, -1), (1, 0, 0)], [(-3, 3, -1e-16), (1, 0, 0)]])
def test_powers_where_a_coefficient_is_tiny_beside_the_others(plan, coeffs):
    """The polynomial's turning points, of which an equation's textbook roots lose one there."""
    test_powers_keep_every_matrix_within_fp16(plan, coeffs)


@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (8, 8, 65535), (5, 9, 3), (300, 77, 511), (300, 77, 512), (300, 77, 513), (449, 3, 1),
                                   (2, 448, 40000), (4096, 4096, 1)])
def test_workspace_is_what_the_header_says(c3, m, n, k):
    s, up = min(m, n), lambda v: -(-v // 16) * 16
    need = 4 * k * (m * up(n) + s * up(s)) + (160 * 256 * 256 * 4 if max(m, n) > 448 else 0)
    # sums: 8 bytes each, at most 512 and one more a matrix; 4 bytes a matrix, 5120 of counts, eight parts' roundings to 256
    assert need <= c3.c3_orthogonalize_bytes(m, n, k) <= need + 12 * k + 4096 + 5120 + 8 * 256
    assert c3.c3_orthogonalize_bytes(m, n, 0) < need + (8 << 10)
