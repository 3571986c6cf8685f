// Internal declarations of the vocabulary matrix's training operators: the
// softmax cross entropy of the lm_head product (hg_xent.hip) and the
// embedding lookup with its gradient (hg_embed.hip). The C ABI is in
// include/hg.h; argument checks and workspace layout in hg_vocab_api.cpp.
#pragma once

#include "hg_internal.h"

namespace hg {

// Rank blocks of the vocabulary matrix. Blocks that follow one another in
// memory are one block of tp*shard rows (NT = 1); others keep the table.
struct VocabMatrix {
  ShardTable t;
  int tp;       // table entries in use: 1 when the blocks are contiguous
  int shard;    // rows per entry
  int hidden;
};

// Per-row work arrays of the cross entropy, in the caller's workspace. Rows
// that count are packed: packed row p is row idx[p] of the call.
struct XentRows {
  int *head;      // [0] packed rows, [1] bits of the largest gradient factor (fp32)
  int *idx;       // [m] packed -> row
  int *inv;       // [m] row -> packed, or -1
  int *lab;       // [m] packed labels
  float *zt;      // [m] packed: the label's logit (base 2), relative to its tile's largest;
                  // few rows: by row, the label's product
  float *lse2;    // [m] packed: log-sum-exp in base 2
  float *ca;      // [m] packed: factor of the probability in d
  float *cb;      // [m] packed: factor of the label's one in d
  float *res;     // [m] packed: what the rounding of the label's d left out
};

// The 16-bit work arrays (packed x, d) lie in panels of 256 columns: element
// (row, col) at ((col / 256) * m + row) * 256 + col % 256. The products read
// such an array along its rows and along its columns; in panels both runs stay
// in a few adjacent pages. Row-major, a column tile's rows of d are 328 KB
// apart (V = 163840), each in a page of its own: at 4096 rows and H = 7168
// dW = d^T X took 9.05 ms (matrix cores 49 % busy) instead of 7.56, dX = d W
// 7.45 instead of 7.36.
constexpr int kPanel = 256;

struct XentPlan {
  int m, hidden, vocab, rows;  // rows = tp*shard
  bool half;                   // fp16 inputs (bf16 otherwise)
  float scale, z_weight;
  long long ignore;
  int label_bytes;
  int piece;       // vocabulary columns per piece, a multiple of 256
  bool small_logits, small_grads;  // products on 128 x 128 tiles (256 x 256 otherwise)
  int ref;         // columns that share a probability reference: the logits' tile edge
  int split_dx;    // splits of the vocabulary in dX = d W
  int split_dw;    // splits of the rows in dW = d^T X
  XentRows r;
  void *xc;        // packed rows of X, [hidden / 256 up][m][256]
  void *d;         // d (or unnormalised probabilities) of one piece, [piece / 256][m][256]
  float *part;     // [2][tiles][m] per tile of `ref` columns: maximum (base 2), sum; few rows:
                   // [m][kScoreGroups][2]
  float *dxp;      // [split_dx][m][hidden]
  float *dwp;      // [split_dw][piece][hidden] when split_dw > 1
};

hipError_t launch_xent_pack(const XentPlan &p, const void *x, const void *labels, float *loss,
                            float *lse, hipStream_t s);
// Logits of columns v0 .. v0+cols-1: mode 0 keeps the row statistics alone, 1
// also the unnormalised probabilities, 2 writes d (the row factors are known).
hipError_t launch_xent_logits(const XentPlan &p, const VocabMatrix &w, int mode, int v0, int cols,
                              hipStream_t s);
// Few rows (m <= kScoreRows): loss and lse straight from x, with no packing.
constexpr int kScoreRows = 128;
constexpr int kScoreGroups = 512;  // workgroups at most, each with a run of the vocabulary
hipError_t launch_xent_score(const XentPlan &p, const VocabMatrix &w, const void *x,
                             const void *labels, float *loss, float *lse, hipStream_t s);
// Row statistics -> loss, lse and the rows' factors (grad null: none).
hipError_t launch_xent_join(const XentPlan &p, const float *grad, float *loss, float *lse,
                            hipStream_t s);
// The rows' factors for a known lse.
hipError_t launch_xent_factors(const XentPlan &p, const float *lse, const float *grad,
                               hipStream_t s);
// Unnormalised probabilities -> d, in place.
hipError_t launch_xent_normalise(const XentPlan &p, hipStream_t s);
// Both of the above in one launch, every workgroup merging its rows' tiles by
// itself: while a row's tiles fit two per lane of its 32 lanes and the rows'
// largest factor, which fp16's d needs, can be found on the way (m labels per
// workgroup; it must not depend on lse).
inline bool xent_joins_in_place(const XentPlan &p) {
  return (p.vocab + p.ref - 1) / p.ref <= 64 && p.m <= 1024 && (!p.half || p.z_weight == 0.f);
}
hipError_t launch_xent_join_normalise(const XentPlan &p, const float *grad, float *loss, float *lse,
                                      hipStream_t s);
// dX's partial sums and dW's rows of the piece, in one launch (without the one
// whose output is not there: p.dxp or dw null).
hipError_t launch_xent_grads(const XentPlan &p, const VocabMatrix &w, int v0, int cols, bool first,
                             void *dw, bool wide, bool accumulate, hipStream_t s);
hipError_t launch_xent_dx_join(const XentPlan &p, const VocabMatrix &w, void *dx, hipStream_t s);

// `bytes` zero bytes at a 16-byte aligned address (bytes a multiple of 16).
hipError_t launch_zero(void *p, size_t bytes, hipStream_t s);

// out[j] = scale * W[tokens[j]], zero for tokens outside 0 .. rows-1.
hipError_t launch_embed(const VocabMatrix &w, int rows, int dtype, const void *tokens,
                        int token_bytes, int n, float scale, void *out, hipStream_t s);

// A stable sort of n keys index[j] (int32 or int64) in 0 .. rows-1, those outside
// last, as the key `rows`: the sorted keys and the places that they came from, both
// in the workspace; in seg[rows + 1], if given, where each key's run begins.
struct SortPlan {
  int passes, tiles;
  size_t off[5], bytes;
};
struct Sorted {
  const int *keys, *pos;
};
SortPlan sort_plan(int rows, long long n);
hipError_t launch_sort(const SortPlan &p, void *ws, int rows, const void *index, int index_bytes,
                       long long n, int *seg, Sorted *sorted, hipStream_t s);

// Workspace of an embedding gradient over n tokens: the sort's, then partial rows.
struct EmbedPlan {
  int per, blocks;  // sorted positions per block of the sums
  size_t part, bytes;
};
EmbedPlan embed_plan(int rows, int hidden, long long n);
hipError_t launch_embed_grad(const EmbedPlan &p, void *ws, int rows, int hidden, int dtype,
                             const void *tokens, int token_bytes, long long n, const void *dy,
                             float scale, void *dw, bool wide, bool accumulate, hipStream_t s);

}  // namespace hg
