"""Which form a 4-bit product takes, by the planner alone (no GPU): test_gpu_fp4_forms.py
runs the shapes listed here, and a retuned planner must not take a form out of its reach."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "concurrent_communication_overlap_gb300", "csrc")
SMS = 152

# M, N, K, sm_budget and the form: rows x columns of a tile.  Last tiles of a few rows, of most of
# them and of whole ones; columns that end in the first and in the second accumulator; K that ends
# within each of a stage's four steps; more tiles than pairs of SMs, and fewer.
FORMS = [
    (4000, 190, 4090, 2, (512, 192)), (1025, 190, 9100, 6, (512, 192)), (1536, 383, 6001, 4, (512, 192)),
    (2048, 1001, 4033, 6, (512, 192)), (2600, 577, 8100, 6, (512, 192)),
    (250, 3800, 4090, 2, (256, 384)), (256, 1151, 4160, 2, (256, 384)), (129, 1919, 8200, 2, (256, 384)),
    (250, 1153, 6017, 4, (256, 384)), (256, 768, 6090, 2, (256, 384)),
    (512, 640, 768, 3, (256, 192)), (385, 193, 520, 2, (256, 192)), (1100, 400, 9000, 4, (256, 192)),
    (200, 264, 4104, 0, (256, 192)),
    (128, 300, 9000, 2, (128, 128)), (100, 130, 2100, 0, (128, 128)), (129, 127, 600, 1, (128, 128)),
    (64, 300, 9000, 1, (64, 128)), (33, 260, 2049, 0, (64, 128)), (32, 260, 2049, 0, (32, 128)), (1, 1, 1, 0, (32, 128)),
]
# experts, N, K, their counts (in a buffer of the rows they take and 128 more), sm_budget and the form
GROUPED_FORMS = [
    (2, 3800, 4090, [250, 255], 2, (256, 384)), (2, 3801, 4100, [900, 700], 2, (256, 384)),
    (4, 1100, 6150, [0, 300, 511, 1025], 2, (256, 384)), (3, 1150, 6001, [513, 256, 700], 4, (256, 384)),
    (3, 640, 2048, [700, 1, 513], 0, (256, 192)), (2, 385, 700, [250, 255], 2, (256, 192)),
    (6, 260, 5000, [3, 0, 130, 65, 1, 2], 2, (64, 128)), (6, 260, 5000, [3, 0, 130, 65, 1, 2], 0, (64, 128)),
]


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    at = tmp_path_factory.mktemp("plan")
    src = at / "plan.cpp"
    src.write_text(r'''
#include <cstdio>
#include <cstdlib>
#include "fp4_plan.h"
int main(int, char** v) {
  const c3::Fp4Plan p = c3::fp4_plan(atoll(v[1]), atoll(v[2]), atoll(v[3]), atoi(v[4]), atoi(v[5]) != 0, atoi(v[6]), atoi(v[7]));
  printf("%d %d %d %d\n", p.rows, p.cols, p.split, p.ctas);
}
''')
    exe = at / "plan"
    subprocess.run(["g++", "-std=c++17", "-I", CSRC, str(src), "-o", str(exe)], check=True)

    def run(M, N, K, experts=1, grouped=False, cap=SMS):
        args = [M, N, K, experts, int(grouped), cap or SMS, SMS]
        return tuple(int(x) for x in subprocess.run([str(exe), *map(str, args)], check=True, capture_output=True, text=True).stdout.split())
    return run


def check(rows, cols, split, ctas, cap):
    two_sms = rows >= 256
    limit = cap if 0 < cap < SMS else SMS if two_sms else 2 * SMS    # few rows: two CTAs an SM of the whole machine
    assert 1 <= ctas <= limit
    assert split in ((1,) if two_sms else (1, 2, 4, 8)) and split * 4 <= max(rows, 4)
    assert ctas % (2 if two_sms else split) == 0


@pytest.mark.parametrize("M,N,K,budget,form", FORMS)
def test_form_of_a_product(plan, M, N, K, budget, form):
    rows, cols, split, ctas = plan(M, N, K, cap=budget)
    assert (rows, cols) == form
    check(rows, cols, split, ctas, budget)


def buffer_rows(counts):
    return sum((c + 127) // 128 * 128 for c in counts) + 128


@pytest.mark.parametrize("E,N,K,counts,budget,form", GROUPED_FORMS)
def test_form_of_the_experts_products(plan, E, N, K, counts, budget, form):
    rows, cols, split, ctas = plan(buffer_rows(counts), N, K, E, True, budget)
    assert (rows, cols) == form
    check(rows, cols, split, ctas, budget)


def test_every_form_is_listed():
    assert {f[-1] for f in FORMS} == {(512, 192), (256, 384), (256, 192), (128, 128), (64, 128), (32, 128)}
    assert {f[-1] for f in GROUPED_FORMS} == {(256, 384), (256, 192), (64, 128)}


def test_forms_of_the_measured_products(plan):
    assert plan(8192, 28672, 8192)[:2] == (512, 192)
    assert plan(256, 28672, 8192)[:2] == (256, 192)
    assert plan(4096, 7680, 8192)[:2] == (256, 192)
    assert plan(13, 8200, 8072)[:3] == (32, 128, 4)
    assert plan(8192 * 4 + 127 * 32, 4096, 4096, 32, True)[:2] == (256, 384)
    assert plan(192 + 127 * 64, 2048, 4096, 64, True)[:2] == (64, 128)


def test_overlapping_experts_stay_in_32_bits(tmp_path):
    """Counts that claim the whole matrix for each of 1024 experts: the running sum of row tiles, as the kernels form it,
    times the column tiles would pass 2^31 (1024 x 31250 x 224); held at the limit it is monotone and in range."""
    src = tmp_path / "tiles.cpp"
    src.write_text(r'''
#include <cstdio>
#include "fp4_plan.h"
int main() {
  const long long M = 2000000, rows = 64, experts = 1024, num_n = 224, num_m = (M + rows - 1) / rows;
  const long long limit = num_m + experts;
  int run = 0, prefix[1025] = {0};
  for (int e0 = 0; e0 < experts; e0 += 32) {
    int incl = 0;
    for (int l = 0; l < 32; ++l) {
      incl += (int)num_m;
      prefix[e0 + l + 1] = c3::tiles_up_to(run, incl, limit);
    }
    run = c3::tiles_up_to(run, incl, limit);
  }
  for (int e = 0; e < experts; ++e)
    if (prefix[e + 1] < prefix[e] || prefix[e + 1] > limit) return 1;
  if (prefix[1] != num_m || prefix[experts] != limit) return 2;
  return (long long)prefix[experts] * num_n > 0x7fffffffLL ? 3 : 0;
}
''')
    exe = tmp_path / "tiles"
    subprocess.run(["g++", "-std=c++17", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)]).returncode == 0
