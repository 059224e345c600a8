// How the work of the logit rules' kernels (adjust.cuh) is cut: threads, segments, stages and shared memory.
// Plain C++ without CUDA, so that the choice can be computed for any size without a device.
#pragma once

#include <algorithm>
#include <cstddef>
#include <cstdint>

#include "sizes.h"

namespace fckl {

constexpr int ADJUST_THREADS = 512;
constexpr int ADJUST_STAGED_THREADS = 512;  // of a block, or for short segments
constexpr int ADJUST_STAGED_FEW = 128;
constexpr int ADJUST_STAGES = 3;       // of each warp's ring in the staged kernel at most
constexpr int ADJUST_STAGE_VECS = 96;  // vectors of a stage (1.5 KB)
constexpr int ADJUST_STAGE_BYTES = ADJUST_STAGE_VECS * 16;

// What a row's rules have to know of its history.
enum AdjustKind {
  ADJUST_COUNTS,  // counts and biases too
  ADJUST_SEEN,    // which tokens stand in it: the repetition penalty alone
  ADJUST_GRAD     // the same, and the signs of their logits
};

constexpr int ADJUST_SEG_WORDS = 16384;   // tokens of a segment at most where each has a word (64 KB)
constexpr int ADJUST_SEG_BITS = 1 << 18;  // and where each has a bit (32 KB)
constexpr int ADJUST_TABLE_LOG2 = 14;     // slots of the table of touched tokens at most (128 KB)
constexpr size_t ADJUST_SMEM = 226 << 10;
// Segments up to which blocks of 128 threads are considered: more rows are then under way on an SM. 4096
// rows with 1000 history entries, with 512 / 128 threads: V = 8000 bf16 115 / 70 us, 30000 191 / 160,
// 128256 376 / 481; 2000 rows of 4000 41 / 18.
constexpr int ADJUST_FEW_VECS = 4096;

// Shared memory of a block: its warps' rings (staged kernel), sets of bits, the table's or the tokens' words
// and the biases.
inline size_t adjust_smem(int64_t tokens, int rings, int sets, bool words, int slots_log2, int B) {
  size_t n = size_t(rings) * ADJUST_STAGE_BYTES + sets * size_t(rup(tokens, 128)) / 8 + size_t(B) * 12;
  if (words) n += slots_log2 >= 0 ? size_t(8) << slots_log2 : size_t(tokens) * 4;
  return n;
}

struct AdjustPlan {
  size_t smem = 0;
  int threads = 0;             // 0: no plan
  int segs = 0, seg_vecs = 0;  // segments of a row, vectors of a segment
  int stages = 0;              // of a warp's ring in the staged kernel
  int slots_log2 = 0;          // of the table of touched tokens; < 0: one word for every token of the segment
  int resident = 0;            // blocks that run on an SM at once
  double us = 0;               // estimated time
};

// How the work is cut: into how many segments a row, with the table of touched tokens or a word for each,
// and in the staged kernel with how many threads and stages. Taken is the least estimated time, in us, of
// waves of blocks that each gather first (2.5 us, 1 us for every 8 history entries a thread reads, 0.6 us
// for each that it puts into the table or 0.3 into words, 1 us for every 64 KB of shared memory cleared)
// and then stream at their share of an SM's 44 GB/s, 10% slower with two stages than with three (4096 x 128256:
// 15%). The estimates are mostly 10 to 40% below what is
// measured, alike for the choices of one shape: 64 x 50001 fp32 with 16384 history entries in 4 segments and
// 2 stages 14 us, in 8 segments 24, with 3 stages 23; 16 x 128256 with 4000 in 1, 4 and 16 segments 29, 12
// and 7.6.
template <int VE, AdjustKind KIND, bool STAGED>
AdjustPlan adjust_plan(int sms, int64_t N, int V, int L, int B, bool streams) {
  constexpr bool WORDS = !STAGED || KIND == ADJUST_COUNTS;
  const int64_t nvec = cdiv(int64_t(V) + VE - 1, VE);
  // The table is at most three quarters full.
  int log2 = 8;
  while ((int64_t(3) << log2) < 4 * (int64_t(L) + B)) ++log2;
  double best = 1e30;
  AdjustPlan plan;
  for (int way = 0; way < 2; ++way) {
    const bool table = way == 0;
    if (table ? log2 > ADJUST_TABLE_LOG2 : !WORDS && plan.smem) continue;
    const int64_t most = WORDS && !table ? ADJUST_SEG_WORDS : STAGED ? ADJUST_SEG_BITS : int64_t(1) << 31;
    const int64_t least = cdiv(nvec * VE, most);
    // from the fewest segments on, in finer steps first, until they are short or the GPU is full many times
    for (int64_t segs = least; segs == least || (segs < least + 64 && nvec * VE / segs >= 2048 &&
                                                 N * segs <= 12 * int64_t(sms)); segs += std::max<int64_t>(1, segs / 8)) {
      const int64_t vecs = rup(cdiv(nvec, segs), 4);
      for (int choice = 0; choice < (STAGED ? 4 : 1); ++choice) {
        if ((choice & 2) && vecs > ADJUST_FEW_VECS) continue;
        const int threads = !STAGED ? ADJUST_THREADS : choice & 2 ? ADJUST_STAGED_FEW : ADJUST_STAGED_THREADS;
        const int stages = !STAGED ? 0 : choice & 1 ? 2 : ADJUST_STAGES;
        const int rings = threads / 32 * stages;
        const int sets = STAGED && KIND == ADJUST_GRAD ? 2 : STAGED || !table ? 1 : 0;  // of bits
        const size_t smem = adjust_smem(vecs * VE, rings, sets, WORDS, table ? log2 : -1, B);
        if (smem > ADJUST_SMEM) continue;
        // blocks of an SM: by shared memory, and 64 registers a thread. 1.5 KB a block is more than it takes
        // beside its dynamic part (1 KB and the barriers), so the last blocks that fit would count as none.
        const int64_t by_smem = std::max<int64_t>(1, (227 << 10) / int64_t(smem + 1536));
        const int64_t resident = std::min<int64_t>(1024 / threads, by_smem);
        const int64_t blocks = N * segs, on_sm = std::min(resident, cdiv(blocks, sms));
        const double gather = 2.5 + double(cdiv(L, threads * 8)) +
                              (WORDS && table ? 0.6 : 0.3) * double(L) / double(threads * segs) +
                              double(smem - size_t(rings) * ADJUST_STAGE_BYTES) / 65536;
        // a small block's few copies under way do not draw an SM's whole share
        const double share = STAGED ? std::min(44e3 / double(on_sm), 44e3 * rings / 32.0) : 44e3 / double(on_sm);
        const double stream = streams ? double(vecs) * 32.0 / share * (stages == 2 ? 1.1 : 1.0) : 0.0;
        const double us = double(cdiv(blocks, resident * sms)) * (gather + stream);
        if (us < 0.98 * best) {
          best = us;
          plan = {smem, threads, static_cast<int>(segs), static_cast<int>(vecs), stages, table ? log2 : -1,
                  static_cast<int>(resident), us};
        }
      }
    }
  }
  return plan;
}

}  // namespace fckl
