// Host side of the beam search operators: argument checks, workspace layout and
// launch order of hg_beam_select and hg_beam_reorder. The C ABI is declared in
// include/hg.h.

#include <math.h>
#include <string.h>

#include <algorithm>
#include <memory>
#include <new>

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

// The bytes of a state: runs of `run` bytes, `many` of them `small` apart, and that
// (`block` bytes from end to end) `times` over, `large` apart. A stride that nothing
// takes is 0.
struct Extent {
  uintptr_t at;
  size_t run, small, large, block, span;
  size_t many, times;
};

// False if runs of the state lie in each other.
bool extent(const hg_beam_state &t, size_t rows, Extent *e) {
  size_t n[2] = {rows, static_cast<size_t>(t.outer)};
  size_t step[2] = {static_cast<size_t>(t.row_stride), static_cast<size_t>(t.outer_stride)};
  for (int k = 0; k < 2; ++k)
    if (n[k] == 1) step[k] = 0;
  const int s = step[0] <= step[1] ? 0 : 1;
  e->at = reinterpret_cast<uintptr_t>(t.ptr);
  e->run = static_cast<size_t>(t.steps) * t.step_bytes;
  e->many = n[s];
  e->small = step[s];
  e->times = n[1 - s];
  e->large = step[1 - s];
  e->block = (e->many - 1) * e->small + e->run;
  e->span = (e->times - 1) * e->large + e->block;
  return (e->many == 1 || e->small >= e->run) && (e->times == 1 || e->large >= e->block);
}

// The stride that two counts share (0: neither has one); false if they differ.
bool shared(size_t a, size_t b, size_t *step) {
  *step = a ? a : b;
  return !a || !b || a == b;
}

// Whether two states, a first, share a byte; true as well if their strides differ where
// it depends on them.
bool meet(const Extent &a, const Extent &b) {
  typedef long long wide;
  const size_t apart = b.at - a.at;
  if (apart >= a.span) return false;
  size_t large, small;
  if (!shared(a.large, b.large, &large)) return true;
  // Blocks meet where b's is moved by `large` to within a block of a's: two or three
  // places at most. The same of their runs.
  if (large && (a.block > large || b.block > large)) return true;
  const wide d = static_cast<wide>(apart), step = static_cast<wide>(large ? large : 1);
  const wide near = large ? -(d / step) : 0;
  for (wide j = near - 1; j <= near + 1; ++j) {
    if (j <= -static_cast<wide>(a.times) || j >= static_cast<wide>(b.times)) continue;
    const wide e = d + (large ? j * step : 0);
    if (e >= static_cast<wide>(a.block) || e <= -static_cast<wide>(b.block)) continue;
    if (!shared(a.small, b.small, &small)) return true;
    if (small && (a.run > small || b.run > small)) return true;
    const wide inner = static_cast<wide>(small ? small : 1), close = small ? -(e / inner) : 0;
    for (wide i = close - 1; i <= close + 1; ++i) {
      if (i <= -static_cast<wide>(a.many) || i >= static_cast<wide>(b.many)) continue;
      const wide gap = e + (small ? i * inner : 0);
      if (gap < static_cast<wide>(a.run) && gap > -static_cast<wide>(b.run)) return true;
    }
  }
  return false;
}

// Whether no two of the states' runs (blocks) of `bytes` meet at any multiple of `step`
// from where they are: then nor do they where they are. `order`: room for n places.
bool apart_around(const Extent *e, size_t n, size_t step, size_t Extent::*bytes, uint32_t *order) {
  for (size_t k = 0; k < n; ++k) {
    if (e[k].*bytes > step) return false;
    order[k] = static_cast<uint32_t>(k);
  }
  std::sort(order, order + n, [&](uint32_t a, uint32_t b) { return e[a].at % step < e[b].at % step; });
  for (size_t k = 0; k < n; ++k) {
    const Extent &a = e[order[k]], &b = e[order[k + 1 < n ? k + 1 : 0]];
    if (a.at % step + a.*bytes > b.at % step + (k + 1 < n ? 0 : step)) return false;
  }
  return true;
}

// The same of all their bytes: of n states, sorted by address, those whose spans are
// linked. Views of one cache lie apart by their places between two rows, or between two
// runs, which takes a sort; other ones go by pairs.
bool all_apart(const Extent *e, size_t n, uint32_t *order) {
  size_t large = 0, small = 0;
  bool one = true, same = true;
  for (size_t k = 0; k < n && one; ++k) one = shared(large, e[k].large, &large);
  for (size_t k = 0; k < n && same; ++k) same = shared(small, e[k].small, &small);
  if (one && large && apart_around(e, n, large, &Extent::block, order)) return true;
  if (one && large && same && small && large % small == 0 && apart_around(e, n, small, &Extent::run, order)) return true;
  for (size_t k = 1; k < n; ++k)
    for (size_t i = 0; i < k; ++i)
      if (meet(e[i], e[k])) return false;
  return true;
}

// Whether the states lie apart: a sort by address, then all_apart where spans are linked
// (64 separate caches, the most of a launch, with the call's other checks: 3 us; 64 views
// of one cache, 32 heads: 10 us, 4096 views 0.5 ms).
bool disjoint(Extent *e, size_t n, uint32_t *order) {
  std::sort(e, e + n, [](const Extent &a, const Extent &b) { return a.at < b.at; });
  for (size_t k = 0; k < n;) {
    uintptr_t end = e[k].at + e[k].span;
    size_t first = k++;
    for (; k < n && e[k].at < end; ++k) end = std::max<uintptr_t>(end, e[k].at + e[k].span);
    if (k - first > 1 && !all_apart(e + first, k - first, order)) return false;
  }
  return true;
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
  auto empty = [](const hg_beam_state &t) { return t.outer == 0 || t.steps == 0 || t.step_bytes == 0; };
  constexpr int kFew = 64;  // (a few states need no memory of the host)
  Extent few[kFew];
  uint32_t few_order[kFew];
  std::unique_ptr<Extent[]> more(count > kFew ? new (std::nothrow) Extent[count] : nullptr);
  std::unique_ptr<uint32_t[]> more_order(count > kFew ? new (std::nothrow) uint32_t[count] : nullptr);
  if (count > kFew && (!more || !more_order)) return HG_ENOMEM;
  Extent *const e = count > kFew ? more.get() : few;
  size_t n = 0;
  for (int i = 0; i < count; ++i) {
    const hg_beam_state &t = states[i];
    if (t.outer < 0 || t.outer > (1 << 20) || t.steps < 0 || t.step_bytes < 0 || t.step_bytes > kMost)
      return HG_EINVAL;
    if (empty(t)) continue;
    if (!t.ptr || t.step_bytes > kMost / t.steps || t.row_stride < 0 || t.outer_stride < 0 ||
        t.row_stride > kMost / rows || t.outer_stride > kMost / t.outer)
      return HG_EINVAL;
    if (!extent(t, rows, e + n)) {
      hg::record_error("a state's rows overlap each other");
      return HG_EINVAL;
    }
    const uintptr_t begin = e[n].at, end = begin + e[n].span;
    auto touches = [&](const void *p, size_t bytes) {
      const uintptr_t at = reinterpret_cast<uintptr_t>(p);
      return p && at < end && begin < at + bytes;
    };
    if (touches(parents, rows * parent_bytes) ||
        touches(lengths, static_cast<size_t>(requests) * length_bytes)) {
      hg::record_error("a state overlaps the parents or the lengths");
      return HG_EINVAL;
    }
    ++n;
  }
  if (!disjoint(e, n, count > kFew ? more_order.get() : few_order)) {
    hg::record_error("states overlap each other, or lie between each other's rows with other strides");
    return HG_EINVAL;
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
      if (!run && hg::beam_reorder_items(p) >= (1ll << 31)) {
        hg::record_error("more runs of rows than a launch covers");
        return HG_EINVAL;
      }
      if (run) HIP_TRY(hg::launch_beam_reorder(p, table, st));
    }
  }
  return HG_OK;
}
