// Internal declarations of the low-rank adapters (hg_adapt.hip). The C ABI is in
// include/hg.h; argument checks and workspace layout in hg_adapt_api.cpp.
#pragma once

#include "hg_vocab.h"

namespace hg {

// Up to this many rows hg_adapt takes a workgroup (or several) for each row's u, and
// sorts the rows beside them.
constexpr int kFewRows = 64;
constexpr int kRankChunk = 64;  // ranks that a workgroup holds at once

// A matrix of 16-bit elements in blocks: column c of row j is at
// ((c / shard) * m + j) * shard + c % shard. One block is a plain matrix.
struct Blocked {
  const void *p;
  int blocks, shard;
};

// The rows' adapters, sorted (keys ascending, rows without one last, as the key
// `adapters`), and as the caller gave them.
struct AdaptRows {
  const int *keys, *pos;
  const void *index;
  int index_bytes;
};

struct AdaptPlan {
  int m, adapters, rank, hidden, tp, shard;
  bool half;
  int few;               // not above kFewRows, and no gradients
  int *few_keys;         // [2][kFewRows] then: keys and places
  SortPlan sort;
  int split_u, split_g;  // parts of the sums over hidden and over the vocabulary
  int padded;            // rows, up to a multiple of 32
  void *sort_ws;
  float *pu, *pg;        // [split][m][rank] partial sums of u and g
  float *u, *g;          // [m][rank] scaled sums, by sorted position
  unsigned short *low;   // [m][3][16 or 64] their pieces, where the second product streams
  float *back;           // [m] and fp16's factors
  int *head;             // [2][adapters]: bits of the largest |u| and |g| (fp16)
  int *seg;              // [adapters + 1] sorted positions where they begin
  unsigned short *ut, *gt;  // [3][ranks][padded] pieces of u and g
  unsigned short *at;    // [adapters][hidden][rank]: A turned
  int parts_a, parts_b;  // of the rows in the sums of dA and dB
  float *pa, *pb;        // [parts][adapters][..], where there are several
};

// Whether the second product goes through many rows with W's fragments kept
// (k_adapt_stream): sorted rows, 64 or more for each adapter of the bank, ranks that fit.
// (How many of the adapters the rows use is on the device alone; see APART in
// hg_adapt.hip for what it costs where they are few.)
inline bool adapt_streams(int m, int adapters, int rank) {
  return m > kFewRows && m / 64 >= adapters && rank <= kRankChunk;
}

// Whether launch_adapt_prepare leaves g's pieces in `low` for it (dx of bf16: fp16's need
// a row's largest): a launch less, gradients of 2047 rows of 32000 columns 77
// us instead of 80 (with two pieces).
inline bool adapt_prepares_rows(const AdaptPlan &p) {
  return p.at && !p.half && adapt_streams(p.m, p.adapters, p.rank);
}

// pu and pg: u's parts from x and A, g's from y and B ([adapters][rank][columns] and
// [adapters][columns][rank]); a side without p is left out.
hipError_t launch_adapt_low(const AdaptPlan &p, const AdaptRows &r, const Blocked &x, const void *a,
                            const Blocked &y, const void *b, hipStream_t s);
// out = y + (sum of the parts) W^T per row; y NULL: zeros; part NULL: their pieces are
// in `low` (k_adapt_stream's sizes).
hipError_t launch_adapt_up(const AdaptPlan &p, const AdaptRows &r, const float *part, int splits,
                           const float *scale, const void *w, const Blocked &y, void *out,
                           hipStream_t s);
// u and g from their parts, scaled; each adapter's largest.
hipError_t launch_adapt_join(const AdaptPlan &p, const AdaptRows &r, const float *scale, hipStream_t s);
// The same and their pieces by rank (ut, gt), and A turned (at), those that are there.
hipError_t launch_adapt_prepare(const AdaptPlan &p, const AdaptRows &r, const float *scale, const void *a,
                                hipStream_t s);
// da and db, those that are there: the sums over an adapter's rows, in parts of the
// rows that are added up if there are several.
hipError_t launch_adapt_outer(const AdaptPlan &p, const AdaptRows &r, const Blocked &x, void *da, const Blocked &y,
                              void *db, bool wide, hipStream_t s);

// Parts that a sum over `columns` columns of `m` rows is cut into.
int adapt_splits(int m, int blocks, int shard, int rank, bool few);
// Parts of the rows in the sums over an adapter's rows, if they are spread over the bank.
int adapt_parts(int m, int adapters, int blocks, int shard, int rank);

}  // namespace hg
