// Host side of the vocabulary matrix's training operators: argument checks,
// workspace layout and launch order of the cross entropy (hg_xent*) and the
// embedding (hg_embed*). The C ABI is declared in include/hg.h.

#include <stdint.h>
#include <string.h>

#include "hg_ranges.h"
#include "hg_vocab.h"

#define HG_API extern "C" __attribute__((visibility("default")))

namespace {

using hg::aligned;
using hg::Ranges;
using hg::VocabMatrix;
using hg::XentPlan;

#define HIP_TRY(expr)                                            \
  do {                                                           \
    hipError_t e_ = (expr);                                      \
    if (e_ != hipSuccess) return hg::record_hip_error(e_, #expr); \
  } while (0)

constexpr int kCus = 256;  // compute units of the one device these kernels are built for
constexpr int kTile = 256, kStep = 64;
constexpr long long kMaxTiles = 1 << 22;  // of 512 lanes: a launch has fewer than 2^32 lanes

int ceil_div(long long a, long long b) { return static_cast<int>((a + b - 1) / b); }
size_t up256(size_t b) { return (b + 255) & ~static_cast<size_t>(255); }

bool shape_ok(const hg_xent_shape *s) {
  if (!s || s->tp < 1 || s->tp > HG_MAX_TP || s->shard < 32 || s->shard % 32 != 0 ||
      s->hidden < 8 || s->hidden % 8 != 0 || s->hidden > (1 << 20) || s->m < 0 ||
      s->m > (1 << 24))
    return false;
  const long long rows = static_cast<long long>(s->tp) * s->shard;
  if (rows >= (1ll << 30) || s->vocab < 1 || s->vocab > rows) return false;
  const long long tm = ceil_div(s->m, kTile), tv = ceil_div(rows, kTile),
                  th = ceil_div(s->hidden, kTile);
  if (tm * tv > kMaxTiles || tm * th > kMaxTiles / 4 || tv * th > kMaxTiles / 4) return false;
  if (s->dtype != HG_BF16 && s->dtype != HG_FP16) return false;
  return s->label_bytes == 4 || s->label_bytes == 8;
}

// Splits of a product of `tiles` tiles and `steps` steps of k whose partial
// sums take `bytes` per split: the split that ends first, counting rounds of
// one tile per CU, 6 steps of pipeline fill and epilogue per tile, a step of
// about 1 us, and the partial sums written and read at 5 TB/s. One split that
// needs no partial sums (`direct`) pays no traffic.
int pick_split(long long tiles, int steps, double bytes, bool direct) {
  int best = 1;
  double least = 0;
  long long most = kMaxTiles / 2 / tiles;
  if (most > steps / 8) most = steps / 8;
  if (most > 64) most = 64;
  if (most < 1) most = 1;
  for (int s = 1; s <= most; ++s) {
    const double rounds = static_cast<double>((tiles * s + kCus - 1) / kCus);
    const double cost = rounds * (ceil_div(steps, s) + 6) +
                        (s == 1 && direct ? 0.0 : 2.0 * s * bytes / 5e6);
    if (s == 1 || cost < least) {
      best = s;
      least = cost;
    }
  }
  return best;
}

// Lays the workspace out from `ws` for one kind of call and a piece of the
// vocabulary, with the products split or not; returns its size. kind: HG_XENT_*,
// with the flags of what is not wanted.
size_t lay_out(const hg_xent_shape &s, int kind, int piece, bool splits, char *ws, XentPlan *p) {
  const bool want_dx = !(kind & HG_XENT_NO_DX), want_dw = !(kind & HG_XENT_NO_DW);
  kind &= ~(HG_XENT_NO_DX | HG_XENT_NO_DW);
  memset(p, 0, sizeof *p);
  p->m = s.m;
  p->hidden = s.hidden;
  p->vocab = s.vocab;
  p->rows = s.tp * s.shard;
  p->half = s.dtype == HG_FP16;
  p->scale = s.scale;
  p->z_weight = s.z_weight;
  p->ignore = s.ignore;
  p->label_bytes = s.label_bytes;
  p->piece = piece;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    char *q = ws + at;
    at += up256(bytes);
    return q;
  };
  const size_t m = static_cast<size_t>(s.m), h = static_cast<size_t>(s.hidden);
  p->r.head = reinterpret_cast<int *>(take(256));
  p->r.idx = reinterpret_cast<int *>(take(4 * m));
  p->r.inv = reinterpret_cast<int *>(take(4 * m));
  p->r.lab = reinterpret_cast<int *>(take(4 * m));
  p->r.zt = reinterpret_cast<float *>(take(4 * m));
  p->r.lse2 = reinterpret_cast<float *>(take(4 * m));
  p->r.ca = reinterpret_cast<float *>(take(4 * m));
  p->r.cb = reinterpret_cast<float *>(take(4 * m));
  p->r.res = reinterpret_cast<float *>(take(4 * m));
  // The small tile while the big one would give work to half of the CUs at
  // most. It takes about 1.5 times as long per product (2047 rows at V = 32000,
  // H = 2048: logits 255 us against 165, gradient products 505 us against 310),
  // so beyond that the big one's single round is the shorter. Up to 128 rows the
  // logits' big tile would be half empty, and few rows show a single loss's last
  // digits, which the small tile keeps: a step at V = 163840, H = 7168 takes 1636 us
  // with one row and 1988 with 128, with the big tile 1680 and 2004.
  const long long tm = ceil_div(s.m, kTile), tn = ceil_div(s.hidden, kTile);
  p->small_logits = s.m <= kTile / 2 ||
                    tm * ceil_div(kind == HG_XENT_GRAD ? piece : s.vocab, kTile) <= kCus / 2;
  p->small_grads = ceil_div(piece, kTile) * tn <= kCus / 2;
  p->ref = p->small_logits ? kTile / 2 : kTile;
  const size_t tiles = static_cast<size_t>(ceil_div(s.vocab, p->ref));
  if (kind == HG_XENT_SCORE && s.m <= hg::kScoreRows) {
    p->part = reinterpret_cast<float *>(take(8 * m * hg::kScoreGroups));
    return at;
  }
  p->xc = take(2 * m * hg::kPanel * ceil_div(s.hidden, hg::kPanel));
  if (kind != HG_XENT_GRAD) p->part = reinterpret_cast<float *>(take(8 * tiles * m));
  if (kind != HG_XENT_SCORE) {
    const int edge = p->small_grads ? kTile / 2 : kTile;
    const long long hn = ceil_div(s.hidden, edge);
    p->split_dx = p->split_dw = 1;
    if (splits) {
      p->split_dx = pick_split(ceil_div(s.m, edge) * hn, ceil_div(piece, kStep), 4.0 * m * h, false);
      p->split_dw = pick_split(piece / edge * hn, ceil_div(s.m, kStep), 4.0 * piece * h, true);
    }
    p->d = take(2 * m * piece);
    if (want_dx) p->dxp = reinterpret_cast<float *>(take(4 * m * h * p->split_dx));
    if (want_dw && p->split_dw > 1)
      p->dwp = reinterpret_cast<float *>(take(4 * static_cast<size_t>(piece) * h * p->split_dw));
  }
  return at;
}

// The plan for a workspace of `limit` bytes (0: any size), and its bytes: the
// fewest pieces of the vocabulary that fit, all about equally wide; if none do,
// the fewest that fit with no product split; if none do, the narrowest of those,
// which no plan takes less than. Every width is tried, widest first, so the plan
// for the bytes of a plan is that plan: what did not fit the limit does not fit
// them either.
size_t plan(const hg_xent_shape &s, int kind, size_t limit, char *ws, XentPlan *p) {
  for (const bool splits : {true, false}) {
    for (int pieces = 1;;) {
      const int piece = ceil_div(ceil_div(s.vocab, pieces), kTile) * kTile;
      const size_t bytes = lay_out(s, kind, piece, splits, ws, p);
      if (kind == HG_XENT_SCORE || limit == 0 || bytes <= limit) return bytes;
      if (piece == kTile) {
        if (!splits) return bytes;
        break;
      }
      pieces = ceil_div(s.vocab, piece - kTile);  // the fewest that are narrower
    }
  }
  return 0;
}

int matrix(int tp, int shard, int hidden, const void *const *w, size_t row_bytes, VocabMatrix *v) {
  if (!w) return HG_EINVAL;
  memset(v, 0, sizeof *v);
  bool joined = true;
  for (int r = 0; r < tp; ++r) {
    if (!w[r] || !aligned(w[r], 16)) return HG_EINVAL;
    v->t.p[r] = static_cast<const hg::u32x4 *>(w[r]);
    if (r && static_cast<const char *>(w[r]) !=
                 static_cast<const char *>(w[r - 1]) + static_cast<size_t>(shard) * row_bytes)
      joined = false;
  }
  v->tp = joined ? 1 : tp;
  v->shard = joined ? tp * shard : shard;
  v->hidden = hidden;
  return HG_OK;
}

// Checks shared by the three calls; fills the plan and the matrix.
int begin(const hg_xent_shape *s, int kind, const void *x, const void *const *w,
          const void *labels, const float *lse_in, const float *grad, float *loss, float *lse,
          void *dx, void *dw, int wide, int accumulate, void *ws, size_t ws_bytes, VocabMatrix *v,
          XentPlan *p) {
  if (!shape_ok(s)) return HG_EINVAL;
  if ((wide != 0 && wide != 1) || (accumulate != 0 && accumulate != 1)) return HG_EINVAL;
  const size_t m = static_cast<size_t>(s->m), h = static_cast<size_t>(s->hidden);
  const size_t rows = static_cast<size_t>(s->tp) * s->shard;
  const bool grads = kind != HG_XENT_SCORE;
  if (grads && !dw && (kind != HG_XENT_GRAD || (m && !dx))) return HG_EINVAL;
  if (!aligned(dw, 16)) return HG_EINVAL;
  Ranges r;
  if (m) {
    const int rc = matrix(s->tp, s->shard, s->hidden, w, 2 * h, v);
    if (rc != HG_OK) return rc;
    if (!x || !aligned(x, 16) || !labels || !aligned(labels, s->label_bytes)) return HG_EINVAL;
    if (kind != HG_XENT_GRAD && (!loss || !lse || !aligned(loss, 4) || !aligned(lse, 4)))
      return HG_EINVAL;
    if (grads && (!grad || !aligned(grad, 4) || (!dx && kind != HG_XENT_GRAD) || !aligned(dx, 16)))
      return HG_EINVAL;
    if (kind == HG_XENT_GRAD && (!lse_in || !aligned(lse_in, 4))) return HG_EINVAL;
    if (!ws || !aligned(ws, 256)) return HG_EINVAL;
    for (int k = 0; k < v->tp; ++k)
      r.add(v->t.p[k], 2 * h * v->shard, false);
    r.add(x, 2 * m * h, false);
    r.add(labels, m * s->label_bytes, false);
    if (kind == HG_XENT_GRAD) r.add(lse_in, 4 * m, false);
    if (grads) r.add(grad, 4 * m, false);
    if (kind != HG_XENT_GRAD) {
      r.add(loss, 4 * m, true);
      r.add(lse, 4 * m, true);
    }
    if (dx) r.add(dx, 2 * m * h, true);
    r.add(ws, ws_bytes, true);
  }
  if (dw) r.add(dw, rows * h * (wide ? 4 : 2), true);
  if (r.clash()) return HG_EINVAL;
  if (kind == HG_XENT_GRAD) kind |= (dx ? 0 : HG_XENT_NO_DX) | (dw ? 0 : HG_XENT_NO_DW);
  if (m && plan(*s, kind, ws_bytes, static_cast<char *>(ws), p) > ws_bytes) {
    hg::record_error("the workspace is smaller than hg_xent_workspace asks");
    return HG_ESIZE;
  }
  return HG_OK;
}

// dX and dW from d, piece by piece. `ready`: d of the whole vocabulary is
// there; otherwise each piece's is computed first.
int products(const XentPlan &p, const VocabMatrix &v, bool ready, void *dx, void *dw, int wide,
             int accumulate, hipStream_t s) {
  for (int v0 = 0; v0 < p.vocab; v0 += p.piece) {
    const int cols = p.vocab - v0 < p.piece ? p.vocab - v0 : p.piece;
    if (!ready) HIP_TRY(hg::launch_xent_logits(p, v, 2, v0, cols, s));
    HIP_TRY(hg::launch_xent_grads(p, v, v0, cols, v0 == 0, dw, wide != 0, accumulate != 0, s));
  }
  if (dx) HIP_TRY(hg::launch_xent_dx_join(p, v, dx, s));
  return HG_OK;
}

int no_rows(const hg_xent_shape *s, void *dw, int wide, int accumulate, hipStream_t st) {
  if (accumulate || !dw) return HG_OK;
  const size_t n = static_cast<size_t>(s->tp) * s->shard * s->hidden * (wide ? 4 : 2);
  HIP_TRY(hg::launch_zero(dw, n, st));
  return HG_OK;
}

}  // namespace

HG_API int hg_xent_workspace(const hg_xent_shape *s, int kind, size_t limit, size_t *bytes) {
  const bool one_of_two = kind == (HG_XENT_GRAD | HG_XENT_NO_DX) || kind == (HG_XENT_GRAD | HG_XENT_NO_DW);
  if (!bytes || !shape_ok(s) || ((kind < HG_XENT_SCORE || kind > HG_XENT_STEP) && !one_of_two))
    return HG_EINVAL;
  *bytes = 0;
  if (s->m == 0) return HG_OK;
  XentPlan p;
  *bytes = plan(*s, kind, limit, nullptr, &p);
  return HG_OK;
}

HG_API int hg_xent(const hg_xent_shape *s, const void *x, const void *const *w, const void *labels,
                   float *loss, float *lse, void *ws, size_t ws_bytes, void *stream) {
  VocabMatrix v;
  XentPlan p;
  const int rc = begin(s, HG_XENT_SCORE, x, w, labels, nullptr, nullptr, loss, lse, nullptr,
                       nullptr, 0, 0, ws, ws_bytes, &v, &p);
  if (rc != HG_OK || s->m == 0) return rc;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (s->m <= hg::kScoreRows) {
    HIP_TRY(hg::launch_xent_score(p, v, x, labels, loss, lse, st));
    return HG_OK;
  }
  HIP_TRY(hg::launch_xent_pack(p, x, labels, loss, lse, st));
  HIP_TRY(hg::launch_xent_logits(p, v, 0, 0, p.vocab, st));
  HIP_TRY(hg::launch_xent_join(p, nullptr, loss, lse, st));
  return HG_OK;
}

HG_API int hg_xent_grad(const hg_xent_shape *s, const void *x, const void *const *w,
                        const void *labels, const float *lse, const float *grad, void *dx,
                        void *dw, int dw_wide, int accumulate, void *ws, size_t ws_bytes,
                        void *stream) {
  VocabMatrix v;
  XentPlan p;
  const int rc = begin(s, HG_XENT_GRAD, x, w, labels, lse, grad, nullptr, nullptr, dx, dw, dw_wide,
                       accumulate, ws, ws_bytes, &v, &p);
  if (rc != HG_OK) return rc;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (s->m == 0) return no_rows(s, dw, dw_wide, accumulate, st);
  HIP_TRY(hg::launch_xent_pack(p, x, labels, nullptr, nullptr, st));
  HIP_TRY(hg::launch_xent_factors(p, lse, grad, st));
  return products(p, v, false, dx, dw, dw_wide, accumulate, st);
}

HG_API int hg_xent_step(const hg_xent_shape *s, const void *x, const void *const *w,
                        const void *labels, const float *grad, float *loss, float *lse, void *dx,
                        void *dw, int dw_wide, int accumulate, void *ws, size_t ws_bytes,
                        void *stream) {
  VocabMatrix v;
  XentPlan p;
  const int rc = begin(s, HG_XENT_STEP, x, w, labels, nullptr, grad, loss, lse, dx, dw, dw_wide,
                       accumulate, ws, ws_bytes, &v, &p);
  if (rc != HG_OK) return rc;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (s->m == 0) return no_rows(s, dw, dw_wide, accumulate, st);
  const bool whole = p.piece >= p.vocab;
  HIP_TRY(hg::launch_xent_pack(p, x, labels, loss, lse, st));
  HIP_TRY(hg::launch_xent_logits(p, v, whole ? 1 : 0, 0, p.vocab, st));
  if (whole && hg::xent_joins_in_place(p)) {
    HIP_TRY(hg::launch_xent_join_normalise(p, grad, loss, lse, st));
  } else {
    HIP_TRY(hg::launch_xent_join(p, grad, loss, lse, st));
    if (whole) HIP_TRY(hg::launch_xent_normalise(p, st));
  }
  return products(p, v, whole, dx, dw, dw_wide, accumulate, st);
}

namespace {

bool embed_shape_ok(int tp, int shard, int hidden, int n) {
  return tp >= 1 && tp <= HG_MAX_TP && shard >= 1 && hidden >= 8 && hidden % 8 == 0 &&
         hidden <= (1 << 20) && n >= 0 && static_cast<long long>(tp) * shard < (1ll << 29);
}
bool embed_type_ok(int dtype) { return dtype == HG_BF16 || dtype == HG_FP16 || dtype == HG_FP32; }

}  // namespace

HG_API int hg_embed(int tp, int shard, int hidden, int dtype, const void *const *w,
                    const void *tokens, int token_bytes, int n, float scale, void *out,
                    void *stream) {
  if (!embed_shape_ok(tp, shard, hidden, n) || !embed_type_ok(dtype) ||
      (token_bytes != 4 && token_bytes != 8))
    return HG_EINVAL;
  if (n == 0) return HG_OK;
  const size_t row = static_cast<size_t>(hidden) * (dtype == HG_FP32 ? 4 : 2);
  VocabMatrix v;
  const int rc = matrix(tp, shard, hidden, w, row, &v);
  if (rc != HG_OK) return rc;
  if (!tokens || !aligned(tokens, token_bytes) || !out || !aligned(out, 16)) return HG_EINVAL;
  Ranges r;
  for (int k = 0; k < v.tp; ++k) r.add(v.t.p[k], row * v.shard, false);
  r.add(tokens, static_cast<size_t>(n) * token_bytes, false);
  r.add(out, row * n, true);
  if (r.clash()) return HG_EINVAL;
  HIP_TRY(hg::launch_embed(v, tp * shard, dtype, tokens, token_bytes, n, scale, out,
                           static_cast<hipStream_t>(stream)));
  return HG_OK;
}

HG_API int hg_embed_workspace(int tp, int shard, int hidden, int n, size_t *bytes) {
  if (!bytes || !embed_shape_ok(tp, shard, hidden, n)) return HG_EINVAL;
  *bytes = n ? hg::embed_plan(tp * shard, hidden, n).bytes : 0;
  return HG_OK;
}

HG_API int hg_embed_grad(int tp, int shard, int hidden, int dtype, const void *tokens,
                         int token_bytes, int n, const void *dy, float scale, void *dw,
                         int dw_wide, int accumulate, void *ws, size_t ws_bytes, void *stream) {
  if (!embed_shape_ok(tp, shard, hidden, n) || !embed_type_ok(dtype) ||
      (token_bytes != 4 && token_bytes != 8) || (dw_wide != 0 && dw_wide != 1) ||
      (accumulate != 0 && accumulate != 1))
    return HG_EINVAL;
  if (!dw || !aligned(dw, 16)) return HG_EINVAL;
  const size_t esize = dtype == HG_FP32 ? 4 : 2;
  const size_t rows = static_cast<size_t>(tp) * shard;
  const hg::EmbedPlan p = hg::embed_plan(static_cast<int>(rows), hidden, n);
  Ranges r;
  r.add(dw, rows * hidden * (dw_wide ? 4 : esize), true);
  if (n) {
    if (!tokens || !aligned(tokens, token_bytes) || !dy || !aligned(dy, 16) ||
        (p.bytes && (!ws || !aligned(ws, 256))))
      return HG_EINVAL;
    r.add(tokens, static_cast<size_t>(n) * token_bytes, false);
    r.add(dy, static_cast<size_t>(n) * hidden * esize, false);
    if (p.bytes) r.add(ws, ws_bytes, true);
  }
  if (r.clash()) return HG_EINVAL;
  if (p.bytes > ws_bytes) {
    hg::record_error("the workspace is smaller than hg_embed_workspace asks");
    return HG_ESIZE;
  }
  if (n == 0 && accumulate) return HG_OK;
  HIP_TRY(hg::launch_embed_grad(p, ws, static_cast<int>(rows), hidden, dtype, tokens, token_bytes, n,
                                dy, scale, dw, dw_wide != 0, accumulate != 0,
                                static_cast<hipStream_t>(stream)));
  return HG_OK;
}
