// Host side of the low-rank adapters: argument checks, workspace layout and
// launch order of hg_adapt and hg_adapt_grad. The C ABI is declared in
// include/hg.h.

#include <string.h>

#include "hg_adapt.h"
#include "hg_ranges.h"

#define HG_API extern "C" __attribute__((visibility("default")))

namespace {

using hg::AdaptPlan;
using hg::AdaptRows;
using hg::aligned;
using hg::Blocked;

#define HIP_TRY(expr)                                            \
  do {                                                           \
    hipError_t e_ = (expr);                                      \
    if (e_ != hipSuccess) return hg::record_hip_error(e_, #expr); \
  } while (0)

constexpr long long kMaxGroups = 1 << 23;  // of 256 lanes: a launch has fewer than 2^32 lanes

long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }

bool shape_ok(const hg_adapt_shape *s, int kind) {
  if (!s || s->tp < 1 || s->tp > HG_MAX_TP || s->shard < 8 || s->shard % 8 != 0 || s->hidden < 8 ||
      s->hidden % 8 != 0 || s->hidden > (1 << 20) || s->m < 0 || s->m > (1 << 24))
    return false;
  const long long columns = static_cast<long long>(s->tp) * s->shard;
  if (columns >= (1ll << 29) || s->m * columns > (1ll << 40)) return false;
  if (s->adapters < 1 || s->adapters > (1 << 15) || s->rank < 8 || s->rank > HG_MAX_RANK || s->rank % 8 != 0)
    return false;
  if (s->dtype != HG_BF16 && s->dtype != HG_FP16) return false;
  if (s->index_bytes != 4 && s->index_bytes != 8) return false;
  // the largest launch: adapters x 64 columns x rank chunks
  const long long strips = s->tp * ceil_div(s->shard, 64), other = ceil_div(s->hidden, 64);
  const long long wide = strips > other ? strips : other;
  return kind == HG_ADAPT_ADD || s->adapters * wide * ceil_div(s->rank, hg::kRankChunk) < kMaxGroups;
}

// Lays the workspace out from `ws`; returns its size.
size_t lay_out(const hg_adapt_shape &s, int kind, char *ws, AdaptPlan *p) {
  memset(p, 0, sizeof *p);
  p->m = s.m;
  p->adapters = s.adapters;
  p->rank = s.rank;
  p->hidden = s.hidden;
  p->tp = s.tp;
  p->shard = s.shard;
  p->half = s.dtype == HG_FP16;
  p->few = kind == HG_ADAPT_ADD && s.m <= hg::kFewRows;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    char *q = ws + at;
    at += (bytes + 255) & ~static_cast<size_t>(255);
    return q;
  };
  auto floats = [&](size_t n) { return reinterpret_cast<float *>(take(4 * n)); };
  const size_t low = static_cast<size_t>(s.m) * s.rank;
  if (p->few) {
    p->few_keys = reinterpret_cast<int *>(take(8 * hg::kFewRows));
  } else {
    p->sort = hg::sort_plan(s.adapters, s.m);
    p->sort_ws = take(p->sort.bytes);
  }
  p->split_u = hg::adapt_splits(s.m, 1, s.hidden, s.rank, p->few);
  p->pu = floats(low * p->split_u);
  if (hg::adapt_streams(s.m, s.adapters, s.rank)) {
    p->low = reinterpret_cast<unsigned short *>(take(static_cast<size_t>(s.m) * (s.rank <= 16 ? 96 : 384)));
    p->back = floats(s.m);
  } else if (kind == HG_ADAPT_ADD && !p->few) {
    p->u = floats(low);
  }
  if (kind == HG_ADAPT_ADD) return at;
  p->split_g = hg::adapt_splits(s.m, s.tp, s.shard, s.rank, false);
  p->pg = floats(low * p->split_g);
  p->u = floats(low);
  p->g = floats(low);
  if (p->half) p->head = reinterpret_cast<int *>(take(8 * static_cast<size_t>(s.adapters)));
  p->seg = reinterpret_cast<int *>(take(4 * (static_cast<size_t>(s.adapters) + 1)));
  p->padded = static_cast<int>(ceil_div(s.m + 8, 32) * 32);  // (eight are read at once from any row on)
  p->ut = reinterpret_cast<unsigned short *>(take(6 * static_cast<size_t>(s.rank) * p->padded));
  p->gt = reinterpret_cast<unsigned short *>(take(6 * static_cast<size_t>(s.rank) * p->padded));
  p->at = reinterpret_cast<unsigned short *>(take(2 * static_cast<size_t>(s.adapters) * s.rank * s.hidden));
  p->parts_a = hg::adapt_parts(s.m, s.adapters, 1, s.hidden, s.rank);
  p->parts_b = hg::adapt_parts(s.m, s.adapters, s.tp, s.shard, s.rank);
  const size_t pairs = static_cast<size_t>(s.adapters) * s.rank;
  if (p->parts_a > 1) p->pa = floats(pairs * s.hidden * p->parts_a);
  if (p->parts_b > 1) p->pb = floats(pairs * s.tp * s.shard * p->parts_b);
  return at;
}

// Bytes of the arguments.
struct Sizes {
  size_t y, x, a, b, scale, index;
};
Sizes sizes(const hg_adapt_shape &s) {
  const size_t m = s.m, columns = static_cast<size_t>(s.tp) * s.shard, n = s.adapters;
  return {2 * m * columns, 2 * m * s.hidden, 2 * n * s.rank * s.hidden, 2 * n * columns * s.rank, 4 * n,
          m * s.index_bytes};
}

bool inputs_ok(const hg_adapt_shape &s, const void *y, const void *x, const void *a, const void *b,
               const float *scale, const void *index, const void *ws) {
  return y && aligned(y, 16) && x && aligned(x, 16) && a && aligned(a, 16) && b && aligned(b, 16) &&
         aligned(scale, 4) && index && aligned(index, s.index_bytes) && ws && aligned(ws, 256);
}

int too_small() {
  hg::record_error("the workspace is smaller than hg_adapt_workspace asks");
  return HG_ESIZE;
}

AdaptRows rows_of(const hg_adapt_shape &s, const void *index) {
  return AdaptRows{nullptr, nullptr, index, s.index_bytes};
}

int sort_rows(const AdaptPlan &p, AdaptRows *r, hipStream_t st) {
  hg::Sorted sorted;
  HIP_TRY(hg::launch_sort(p.sort, p.sort_ws, p.adapters, r->index, r->index_bytes, p.m, p.seg, &sorted, st));
  r->keys = sorted.keys;
  r->pos = sorted.pos;
  return HG_OK;
}

}  // namespace

HG_API int hg_adapt_workspace(const hg_adapt_shape *s, int kind, size_t *bytes) {
  if (!bytes || (kind != HG_ADAPT_ADD && kind != HG_ADAPT_GRAD) || !shape_ok(s, kind)) return HG_EINVAL;
  *bytes = 0;
  if (s->m == 0) return HG_OK;
  AdaptPlan p;
  *bytes = lay_out(*s, kind, nullptr, &p);
  return HG_OK;
}

HG_API int hg_adapt(const hg_adapt_shape *s, const void *y, const void *x, const void *a, const void *b,
                    const float *scale, const void *index, void *out, void *ws, size_t ws_bytes,
                    void *stream) {
  if (!shape_ok(s, HG_ADAPT_ADD)) return HG_EINVAL;
  if (s->m == 0) return HG_OK;
  if (!inputs_ok(*s, y, x, a, b, scale, index, ws) || !out || !aligned(out, 16)) return HG_EINVAL;
  const Sizes n = sizes(*s);
  hg::Ranges r;
  if (out != y) r.add(y, n.y, false);
  r.add(x, n.x, false);
  r.add(a, n.a, false);
  r.add(b, n.b, false);
  if (scale) r.add(scale, n.scale, false);
  r.add(index, n.index, false);
  r.add(out, n.y, true);
  r.add(ws, ws_bytes, true);
  if (r.clash()) return HG_EINVAL;
  AdaptPlan p;
  if (lay_out(*s, HG_ADAPT_ADD, static_cast<char *>(ws), &p) > ws_bytes) return too_small();
  hipStream_t st = static_cast<hipStream_t>(stream);
  AdaptRows rows = rows_of(*s, index);
  if (p.few) {
    rows.keys = p.few_keys;
    rows.pos = p.few_keys + hg::kFewRows;
  } else {
    const int rc = sort_rows(p, &rows, st);
    if (rc != HG_OK) return rc;
  }
  HIP_TRY(hg::launch_adapt_low(p, rows, Blocked{x, 1, s->hidden}, a, Blocked{nullptr, 1, 8}, nullptr, st));
  // The second product's workgroups each read all of their rows' parts: of many
  // rows they are added up first (2047 rows, 28 parts: 578 us against 365).
  const Blocked wide_y{y, s->tp, s->shard};
  if (p.u) {
    HIP_TRY(hg::launch_adapt_join(p, rows, scale, st));
    HIP_TRY(hg::launch_adapt_up(p, rows, p.u, 1, nullptr, b, wide_y, out, st));
  } else {
    HIP_TRY(hg::launch_adapt_up(p, rows, p.pu, p.split_u, scale, b, wide_y, out, st));
  }
  return HG_OK;
}

HG_API int hg_adapt_grad(const hg_adapt_shape *s, const void *dy, const void *x, const void *a,
                         const void *b, const float *scale, const void *index, void *dx, void *da,
                         void *db, int wide, void *ws, size_t ws_bytes, void *stream) {
  if (!shape_ok(s, HG_ADAPT_GRAD) || (wide != 0 && wide != 1)) return HG_EINVAL;
  if ((!dx && !da && !db) || !aligned(dx, 16) || !aligned(da, 16) || !aligned(db, 16)) return HG_EINVAL;
  const Sizes n = sizes(*s);
  const size_t times = wide ? 2 : 1;
  hg::Ranges r;
  if (s->m) {
    if (!inputs_ok(*s, dy, x, a, b, scale, index, ws)) return HG_EINVAL;
    r.add(dy, n.y, false);
    r.add(x, n.x, false);
    r.add(a, n.a, false);
    r.add(b, n.b, false);
    if (scale) r.add(scale, n.scale, false);
    r.add(index, n.index, false);
    r.add(ws, ws_bytes, true);
  }
  if (dx) r.add(dx, n.x, true);
  if (da) r.add(da, n.a * times, true);
  if (db) r.add(db, n.b * times, true);
  if (r.clash()) return HG_EINVAL;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (s->m == 0) {
    if (da) HIP_TRY(hg::launch_zero(da, n.a * times, st));
    if (db) HIP_TRY(hg::launch_zero(db, n.b * times, st));
    return HG_OK;
  }
  AdaptPlan p;
  if (lay_out(*s, HG_ADAPT_GRAD, static_cast<char *>(ws), &p) > ws_bytes) return too_small();
  AdaptRows rows = rows_of(*s, index);
  const int rc = sort_rows(p, &rows, st);
  if (rc != HG_OK) return rc;
  const Blocked none{nullptr, 1, 8}, wide_x{x, 1, s->hidden}, wide_y{dy, s->tp, s->shard};
  if (!db) p.u = nullptr, p.ut = nullptr;
  if (!dx && !da) p.g = nullptr;
  if (!da) p.gt = nullptr;
  if (!dx) p.at = nullptr;
  HIP_TRY(hg::launch_adapt_low(p, rows, p.u ? wide_x : none, a, p.g ? wide_y : none, b, st));
  HIP_TRY(hg::launch_adapt_prepare(p, rows, scale, a, st));
  if (da || db) HIP_TRY(hg::launch_adapt_outer(p, rows, wide_x, da, wide_y, db, wide != 0, st));
  if (dx) {
    const float *const g = hg::adapt_prepares_rows(p) ? nullptr : p.g;
    HIP_TRY(hg::launch_adapt_up(p, rows, g, 1, nullptr, p.at, Blocked{nullptr, 1, s->hidden}, dx, st));
  }
  return HG_OK;
}
