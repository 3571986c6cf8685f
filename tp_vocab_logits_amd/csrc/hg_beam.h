// Internal declarations of the beam search operators (hg_beam.hip). The C ABI
// is in include/hg.h; argument checks and workspace layout in hg_beam_api.cpp.
#pragma once

#include "hg_internal.h"

namespace hg {

// What one workgroup leaves of its part of a row: the largest logit, and the
// sum of exp(scale * (z - top)).
struct BeamStat {
  double sum;
  float top;
  int unused;
};

struct BeamPlan {
  int requests, beams, keep;
  int tp, shard, vocab;  // the blocks that hold a part of the vocabulary, and their rows' stride
  int dtype, pad;
  float scale;
  int vecs;              // 16-byte vectors per thread of the scan: 1, 2 or 4
  int per_block, parts;  // parts (workgroups) per block of a row, and per row
  BeamStat *stat;              // [rows][parts]
  unsigned long long *keys;    // [rows][parts][keep], descending, 0: none
};

constexpr int kScanThreads = 256;

// Elements of a 16-byte vector.
inline int beam_lane_elements(int dtype) { return dtype == HG_FP32 ? 4 : 8; }

hipError_t launch_beam_scan(const BeamPlan &p, const ShardTable &logits, const float *scores,
                            const unsigned char *finished, hipStream_t s);
hipError_t launch_beam_join(const BeamPlan &p, const float *scores, const unsigned char *finished,
                            float *out, long long *parents, long long *tokens, hipStream_t s);

// States of one geometry, moved by one launch (up to kStates of them).
constexpr int kStates = 64;
constexpr int kFewStates = 8;
template <int N>
struct StateTable {
  unsigned char *p[N];
};
struct ReorderPlan {
  int requests, beams, count;
  long long row_stride, outer_stride;
  unsigned long long step_bytes;
  int outer, steps;
  const void *parents, *lengths;
  int parent_bytes, length_bytes;
};
hipError_t launch_beam_reorder(const ReorderPlan &p, unsigned char *const *states, hipStream_t s);
// Workgroups' worth of work of such a launch; one of 2^31 or more is refused.
long long beam_reorder_items(const ReorderPlan &p);

}  // namespace hg
