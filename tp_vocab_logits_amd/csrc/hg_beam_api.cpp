// Host side of the beam search operators: argument checks, workspace layout and
// launch order of hg_beam_select and hg_beam_reorder. The C ABI is declared in
// include/hg.h.

#include <math.h>
#include <string.h>

#include "hg_beam.h"
#include "hg_ranges.h"

#define HG_API extern "C" __attribute__((visibility("default")))

namespace {

using hg::aligned;
using hg::BeamPlan;

#define HIP_TRY(expr)                                            \
  do {                                                           \
    hipError_t e_ = (expr);                                      \
    if (e_ != hipSuccess) return hg::record_hip_error(e_, #expr); \
  } while (0)

constexpr long long kMaxGroups = 1 << 23;  // of 256 lanes: a launch has fewer than 2^32 lanes

bool shape_ok(const hg_beam_shape *s) {
  if (!s || s->requests < 0 || s->beams < 1 || s->beams > HG_MAX_BEAMS || s->keep < 1 ||
      s->keep > HG_MAX_KEEP || s->tp < 1 || s->tp > HG_MAX_TP || s->shard < 1)
    return false;
  if (s->vocab < 1 || s->vocab > (1 << 20) || s->vocab > static_cast<long long>(s->tp) * s->shard)
    return false;
  if (s->dtype != HG_BF16 && s->dtype != HG_FP16 && s->dtype != HG_FP32) return false;
  return s->pad >= 0 && s->pad < s->vocab && s->scale > 0.f && s->scale < INFINITY;
}

// Lays the workspace out from `ws`; 0 bytes if a launch cannot cover the shape.
size_t plan(const hg_beam_shape &s, char *ws, BeamPlan *p) {
  memset(p, 0, sizeof *p);
  p->requests = s.requests;
  p->beams = s.beams;
  p->keep = s.keep;
  p->shard = s.shard;
  p->vocab = s.vocab;
  p->dtype = s.dtype;
  p->pad = s.pad;
  p->scale = s.scale;
  p->tp = (s.vocab + static_cast<long long>(s.shard) - 1) / s.shard;  // blocks that hold a real entry
  // A row's part per workgroup: as small as keeps the launch at 2048 workgroups
  // (a few rows are a matter of latency) and a row at 64 parts, one per lane of
  // the join.
  const long long rows = static_cast<long long>(s.requests) * s.beams;
  const int lanes = hg::beam_lane_elements(s.dtype);
  const long long width = s.shard < s.vocab ? s.shard : s.vocab;
  for (p->vecs = 1;; p->vecs *= 2) {
    const long long part = static_cast<long long>(p->vecs) * hg::kScanThreads * lanes;
    p->per_block = static_cast<int>((width + part - 1) / part);
    p->parts = p->per_block * p->tp;
    if (p->vecs == 4 || (rows * p->parts <= 2048 && p->parts <= 64)) break;
  }
  if (rows * p->parts > kMaxGroups || s.requests > kMaxGroups) return 0;
  const size_t n = static_cast<size_t>(rows) * p->parts;
  p->stat = reinterpret_cast<hg::BeamStat *>(ws);
  p->keys = reinterpret_cast<unsigned long long *>(ws + n * sizeof(hg::BeamStat));
  return n * (sizeof(hg::BeamStat) + 8 * static_cast<size_t>(s.keep));
}

}  // namespace

HG_API int hg_beam_workspace(const hg_beam_shape *s, size_t *bytes) {
  if (!bytes || !shape_ok(s)) return HG_EINVAL;
  *bytes = 0;
  if (s->requests == 0) return HG_OK;
  BeamPlan p;
  *bytes = plan(*s, nullptr, &p);
  return *bytes ? HG_OK : HG_EINVAL;
}

HG_API int hg_beam_select(const hg_beam_shape *s, const void *const *logits, const float *scores,
                          const void *finished, float *out, long long *parents, long long *tokens,
                          void *ws, size_t ws_bytes, void *stream) {
  if (!shape_ok(s)) return HG_EINVAL;
  if (s->requests == 0) return HG_OK;
  BeamPlan p;
  const size_t need = plan(*s, static_cast<char *>(ws), &p);
  if (!need || !logits || !scores || !aligned(scores, 4) || !out || !aligned(out, 4) || !parents ||
      !aligned(parents, 8) || !tokens || !aligned(tokens, 8) || !ws || !aligned(ws, 256))
    return HG_EINVAL;
  const size_t esize = s->dtype == HG_FP32 ? 4 : 2;
  const size_t rows = static_cast<size_t>(s->requests) * s->beams;
  const size_t places = static_cast<size_t>(s->requests) * s->keep;
  hg::ShardTable t;
  memset(&t, 0, sizeof t);
  hg::Ranges r;
  for (int k = 0; k < p.tp; ++k) {
    if (!logits[k] || !aligned(logits[k], esize)) return HG_EINVAL;
    t.p[k] = static_cast<const hg::u32x4 *>(logits[k]);
    r.add(logits[k], rows * s->shard * esize, false);
  }
  r.add(scores, rows * 4, false);
  if (finished) r.add(finished, rows, false);
  r.add(out, places * 4, true);
  r.add(parents, places * 8, true);
  r.add(tokens, places * 8, true);
  r.add(ws, ws_bytes, true);
  if (r.clash()) return HG_EINVAL;
  if (need > ws_bytes) {
    hg::record_error("the workspace is smaller than hg_beam_workspace asks");
    return HG_ESIZE;
  }
  hipStream_t st = static_cast<hipStream_t>(stream);
  const unsigned char *const done = static_cast<const unsigned char *>(finished);
  HIP_TRY(hg::launch_beam_scan(p, t, scores, done, st));
  HIP_TRY(hg::launch_beam_join(p, scores, done, out, parents, tokens, st));
  return HG_OK;
}

namespace {

// The bytes of a state: `rows` x `outer` runs of `run` bytes.
struct Extent {
  uintptr_t at;
  long long rows, outer, row_stride, outer_stride, run;
  size_t span() const { return (rows - 1) * row_stride + (outer - 1) * outer_stride + run; }
};

// Runs of one state apart from each other: the smaller stride takes a run, the
// larger one all of the smaller's.
bool apart(const Extent &e) {
  const bool rows_inside = e.row_stride <= e.outer_stride;
  const long long small = rows_inside ? e.row_stride : e.outer_stride;
  const long long large = rows_inside ? e.outer_stride : e.row_stride;
  const long long many = rows_inside ? e.rows : e.outer, times = rows_inside ? e.outer : e.rows;
  if (many > 1 && small < e.run) return false;
  return times == 1 || large >= (many - 1) * small + e.run;
}

// Whether two states share a byte. States of one geometry may lie between each
// other's runs (views of one cache); others have to lie apart as a whole.
bool meet(const Extent &a, const Extent &b) {
  const Extent &x = a.at <= b.at ? a : b, &y = a.at <= b.at ? b : a;
  if (y.at - x.at >= x.span()) return false;
  if (a.rows != b.rows || a.outer != b.outer || a.row_stride != b.row_stride ||
      a.outer_stride != b.outer_stride || a.run != b.run)
    return true;
  // d + i*row_stride + j*outer_stride within a run of 0, |i| < rows, |j| < outer
  const long long d = static_cast<long long>(y.at - x.at);
  for (long long j = -(a.outer - 1); j < a.outer; ++j) {
    const long long left = d + j * a.outer_stride;
    const long long near = a.rows > 1 ? -left / a.row_stride : 0;
    for (long long i = near - 1; i <= near + 1; ++i) {
      const long long gap = left + i * a.row_stride;
      if (i > -a.rows && i < a.rows && gap < a.run && gap > -a.run) return true;
    }
  }
  return false;
}

}  // namespace

HG_API int hg_beam_reorder(int requests, int beams, int count, const hg_beam_state *states,
                           const void *parents, int parent_bytes, const void *lengths,
                           int length_bytes, void *stream) {
  if (requests < 0 || beams < 1 || beams > HG_MAX_BEAMS || count < 0 || count > (1 << 16) ||
      (parent_bytes != 4 && parent_bytes != 8) || (lengths && length_bytes != 4 && length_bytes != 8))
    return HG_EINVAL;
  if (requests == 0 || count == 0) return HG_OK;
  if (!states || !parents || !aligned(parents, parent_bytes) ||
      (lengths && !aligned(lengths, length_bytes)))
    return HG_EINVAL;
  const long long rows = static_cast<long long>(requests) * beams;
  constexpr long long kMost = 1ll << 46;  // bytes of a state: strides and offsets stay far from 2^63
  auto extent = [&](const hg_beam_state &t) {
    return Extent{reinterpret_cast<uintptr_t>(t.ptr), rows, t.outer, t.row_stride, t.outer_stride,
                  t.steps * t.step_bytes};
  };
  auto empty = [](const hg_beam_state &t) { return t.outer == 0 || t.steps == 0 || t.step_bytes == 0; };
  for (int i = 0; i < count; ++i) {
    const hg_beam_state &t = states[i];
    if (t.outer < 0 || t.outer > (1 << 20) || t.steps < 0 || t.step_bytes < 0 || t.step_bytes > kMost)
      return HG_EINVAL;
    if (empty(t)) continue;
    if (!t.ptr || t.step_bytes > kMost / t.steps || t.row_stride < 0 || t.outer_stride < 0 ||
        t.row_stride > kMost / rows || t.outer_stride > kMost / t.outer)
      return HG_EINVAL;
    const Extent e = extent(t);
    if (!apart(e)) return HG_EINVAL;
    const uintptr_t end = e.at + e.span();
    auto touches = [&](const void *p, size_t bytes) {
      const uintptr_t at = reinterpret_cast<uintptr_t>(p);
      return p && at < end && e.at < at + bytes;
    };
    if (touches(parents, rows * parent_bytes) ||
        touches(lengths, static_cast<size_t>(requests) * length_bytes))
      return HG_EINVAL;
    for (int k = 0; k < i; ++k)
      if (!empty(states[k]) && meet(e, extent(states[k]))) return HG_EINVAL;
  }
  hipStream_t st = static_cast<hipStream_t>(stream);
  // States of one geometry that follow one another share a launch. The sizes of
  // all launches are checked before the first.
  for (const bool run : {false, true}) {
    for (int i = 0; i < count;) {
      const hg_beam_state &t = states[i];
      unsigned char *table[hg::kStates];
      hg::ReorderPlan p{requests, beams, 0, t.row_stride, t.outer_stride,
                        static_cast<unsigned long long>(t.step_bytes), t.outer, t.steps,
                        parents, lengths, parent_bytes, length_bytes};
      for (; i < count && p.count < hg::kStates; ++i) {
        const hg_beam_state &o = states[i];
        if (o.row_stride != t.row_stride || o.outer_stride != t.outer_stride ||
            o.step_bytes != t.step_bytes || o.outer != t.outer || o.steps != t.steps)
          break;
        table[p.count++] = static_cast<unsigned char *>(o.ptr);
      }
      if (empty(t)) continue;
      if (!run && hg::beam_reorder_items(p) >= (1ll << 31)) return HG_EINVAL;
      if (run) HIP_TRY(hg::launch_beam_reorder(p, table, st));
    }
  }
  return HG_OK;
}
