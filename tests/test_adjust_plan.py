"""How the logit rules' kernels are cut (csrc/adjust_plan.h), compiled for the host and computed for sizes over
the whole range: a plan exists, fits a block's shared memory, covers the row, and was estimated to
take some time. Around the size where the table of touched tokens, the stages and the biases fill a block's
shared memory the last block that fits still counts as one that runs.
"""
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "chunked_kl_loss_gb300", "csrc")
SMS = 152
SMEM = 226 << 10     # of a block
COUNTS, SEEN, GRAD = 0, 1, 2

PROGRAM = r"""
#include <cinttypes>
#include <cstdio>
#include "adjust_plan.h"
using namespace fckl;
int main() {
  int ve, kind, staged, sms, V, L, B, streams;
  int64_t N;
  while (scanf("%d %d %d %d %" SCNd64 " %d %d %d %d", &ve, &kind, &staged, &sms, &N, &V, &L, &B, &streams) == 9) {
    AdjustPlan p;
#define CASE(VE, KIND, STAGED) \
  if (ve == VE && kind == KIND && staged == STAGED) p = adjust_plan<VE, KIND, STAGED>(sms, N, V, L, B, streams != 0);
#define STAGED_CASES(VE) CASE(VE, ADJUST_COUNTS, true) CASE(VE, ADJUST_SEEN, true) CASE(VE, ADJUST_GRAD, true)
#define OTHER_CASES(VE) CASE(VE, ADJUST_COUNTS, false) CASE(VE, ADJUST_GRAD, false)
    STAGED_CASES(4) STAGED_CASES(8) OTHER_CASES(1) OTHER_CASES(4) OTHER_CASES(8)
    printf("%zu %d %d %d %d %d %d %.17g\n", p.smem, p.threads, p.segs, p.seg_vecs, p.stages, p.slots_log2, p.resident, p.us);
  }
}
"""


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    """A function from cases (ve, kind, staged, N, V, L, B, streams) to their plans."""
    where = tmp_path_factory.mktemp("plan")
    src, exe = where / "plan.cpp", where / "plan"
    src.write_text(PROGRAM)
    cxx = os.environ.get("CXX") or shutil.which("g++") or "c++"
    done = subprocess.run([cxx, "-std=c++17", "-O1", "-I", CSRC, str(src), "-o", str(exe)], capture_output=True, text=True)
    assert done.returncode == 0, done.stderr

    def run(cases):
        lines = "".join(f"{ve} {kind} {staged} {SMS} {N} {V} {L} {B} {streams}\n" for ve, kind, staged, N, V, L, B, streams in cases)
        done = subprocess.run([str(exe)], input=lines, capture_output=True, text=True)
        rows = [line.split() for line in done.stdout.splitlines()]
        assert done.returncode == 0 and len(rows) == len(cases), (done.returncode, cases[min(len(rows), len(cases) - 1)])
        names = ("smem", "threads", "segs", "seg_vecs", "stages", "slots_log2", "resident", "us")
        return [dict(zip(names, [*map(int, row[:-1]), float(row[-1])])) for row in rows]

    return run


def check(case, p):
    ve, kind, staged, N, V, L, B, streams = case
    assert p["threads"] in ((128, 512) if staged else (512,)), (case, p)
    assert 0 < p["smem"] <= SMEM and p["resident"] >= 1, (case, p)
    assert p["segs"] >= 1 and p["segs"] * p["seg_vecs"] * ve >= V + ve - 1, (case, p)
    assert p["stages"] in ((2, 3) if staged else (0,)), (case, p)
    assert p["slots_log2"] < 0 or 3 << p["slots_log2"] >= 4 * (L + B), (case, p)
    assert 2.5 <= p["us"] < 1e12, (case, p)  # at least one wave's gathering


# what fills a block's shared memory beside the largest table: a set of bits (V / 8) and 12 bytes a bias
NEAR_THE_LIMIT = [(201088, 8192, 100), (201088, 6100, 100), (201088, 12100, 100), (201500, 9000, 100), (182000, 8000, 300),
                  (210000, 8192, 0), (210000, 8000, 0), (112000, 8000, 1024), (128256, 8000, 860)]


@pytest.mark.parametrize("V,L,B", NEAR_THE_LIMIT)
def test_near_the_limit_of_shared_memory(plans, V, L, B):
    cases = [(ve, COUNTS, 1, N, V, L, B, streams) for ve in (4, 8) for N in (1, 2, 16, 256, 4096) for streams in (0, 1)]
    for case, p in zip(cases, plans(cases)):
        check(case, p)
        if case[3] <= 16:  # few rows are cut so that more SMs than rows take part
            assert p["segs"] > 1, (case, p)
    # the choice goes on as beside the limit: as many segments, give or take one step, as with fewer biases
    near, beside = plans([(8, COUNTS, 1, 16, V, L, B, 1), (8, COUNTS, 1, 16, V, L, B // 2, 1)])
    assert 0.7 <= near["segs"] / beside["segs"] <= 1.4, (near, beside)


def test_every_number_of_biases_and_ids_across_the_limit(plans):
    cases = [(8, COUNTS, 1, 4, 201088, 8000, B, 1) for B in range(0, 1025)]
    cases += [(ve, COUNTS, 1, 4, V, 8000, B, 1) for ve in (4, 8) for V in range(100000, 263000, 500) for B in (0, 1024)]
    for case, p in zip(cases, plans(cases)):
        check(case, p)


def test_sizes_over_the_whole_range(plans):
    rng = random.Random(5)

    def log(lo, hi):
        return int(lo * (hi / lo) ** rng.random())

    cases = []
    for _ in range(20000):
        staged = rng.random() < 0.6
        ve = rng.choice((4, 8) if staged else (1, 4, 8))
        kind = rng.choice((COUNTS, SEEN, GRAD) if staged else (COUNTS, GRAD))
        V = rng.choice((log(1, 300000), log(1, 1 << 30), rng.randint(100000, 262144)))
        L = rng.choice((0, log(1, 1048576), rng.randint(5900, 12500)))
        B = rng.choice((0, log(1, 1025), 1024)) if kind == COUNTS else 0
        cases.append((ve, kind, int(staged), log(1, 100000), V, L, B, rng.randint(0, 1)))
    for case, p in zip(cases, plans(cases)):
        check(case, p)
