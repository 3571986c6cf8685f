// Workgroups of the zero fill that runs beside the embedding gradient's sort
// (hg_embed.hip). Plain C++: the host chooses the grid with it.
#pragma once

namespace hg {

constexpr int kFillVecs = 1024;           // 16-byte vectors, one per thread of a workgroup
constexpr long long kFillMost = 1 << 18;  // workgroups: a launch stays far below 2^32 lanes

// One store per thread up to kFillMost workgroups (4.3 GB); with more to fill the
// workgroups go through it in strides of all of them.
inline int fill_groups(long long vecs) {
  const long long want = vecs > 0 ? (vecs + kFillVecs - 1) / kFillVecs : 0;
  return static_cast<int>(want < kFillMost ? want : kFillMost);
}

}  // namespace hg
