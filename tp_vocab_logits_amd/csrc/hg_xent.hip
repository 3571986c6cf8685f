// Softmax cross entropy of the lm_head product, on gfx950 matrix cores,
// without keeping the logits.
//
// For the rows i that count (label t_i, not the ignored value), logits over
// the real vocabulary v < vocab of the rank blocks W_r (rank r at r*shard):
//   z_iv = scale * x_i . W_v
//   lse_i = log sum_v exp z_iv
//   loss_i = lse_i - z_it + z_weight * lse_i^2
//   d_iv = scale * g_i * ((1 + 2 z_weight lse_i) exp(z_iv - lse_i) - [v = t_i])
//   dx_i = sum_v d_iv W_v,   dW_v = sum_i d_iv x_i
//
// The rows that count are packed first (k_pack, k_pack_rows): rows left out
// cost nothing in the products, and what their x holds (NaN, infinities) is
// never multiplied. All products then run over the packed rows, whose number
// stays on the device.
//
// Logits: 256 x 256 tiles (hg_tile.h). The epilogue reduces each row of its
// tile to a maximum and a sum of exponentials (one pass, in base 2, fp32);
// k_join merges a row's tiles. For the gradient either
//  - the epilogue also stores the unnormalised probabilities exp(z - tile
//    maximum), and k_normalise turns them into d once lse is known: the logits
//    are computed once (hg_xent_step), or
//  - lse is known, and the epilogue writes d itself (hg_xent_grad, and steps
//    whose workspace holds fewer columns than the vocabulary).
// d is 16 bits wide, as the matrix cores take it: one rounding to the type on
// each term of sums over many. A label's d is no term among many: it is the
// largest of its row by far, and often the one large term of its row of dW, and
// its rounding would show in the results as one more rounding of their own. What
// it leaves out (XentRows::res) joins both products in fp32, as a multiple of
// the label's row of W and of x. fp16 has 5 exponent bits: there d is scaled by a
// power of two that brings its largest row factor to 2^13..2^14, so that terms
// down to about 2^-27 of the largest keep all their bits; the scale is exact
// and is taken back in fp32.
// The unnormalised probabilities, all in 0..1, wait in 16 bits without a sign
// (see Prob): 10 bits of mantissa for bf16 and 11 for fp16, so that this first
// rounding is off by at most an eighth (fp16: a half) of what d's own is.

#include <type_traits>

#include "hg_tile.h"
#include "hg_vocab.h"

namespace hg {

namespace {

constexpr int kCus = 256;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// An unnormalised probability p in 0..1 in 16 bits: the top of its fp32 bits,
// exponents 2^-(2^E - 1) .. 2^0 with M mantissa bits, E + M = 16, rounded to
// nearest; what is smaller (2^-63 for bf16, 2^-31 for fp16) becomes 0.
template <class T>
struct Prob {
  static constexpr int M = T::kHalf ? 11 : 10, E = 16 - M, S = 23 - M;
  static constexpr int kLow = (127 - ((1 << E) - 1)) << M;
  static __device__ __forceinline__ uint32_t put(float p) {
    const uint32_t b = (__builtin_bit_cast(uint32_t, p) + (1u << (S - 1))) >> S;
    return __builtin_elementwise_sub_sat(b, static_cast<uint32_t>(kLow));
  }
  static __device__ __forceinline__ float get(uint32_t c) {
    return c ? __builtin_bit_cast(float, static_cast<int>(c + kLow) << S) : 0.f;
  }
};

__device__ __forceinline__ float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }

// The power of two by which d is scaled (and its inverse) for the bits of the
// largest row factor: 1 for bf16.
template <class T>
__device__ __forceinline__ float d_scale_of(int largest, bool inverse) {
  if constexpr (!T::kHalf) return 1.f;
  // 2^(13 - exponent of the largest factor): products end in 2^13..2^14
  const int e = static_cast<int>((static_cast<unsigned>(largest) >> 23) & 255u);
  int up = e == 0 ? 0 : 13 - (e - 127);
  up = up > 126 ? 126 : up < -126 ? -126 : up;
  return __builtin_bit_cast(float, static_cast<unsigned>(127 + (inverse ? -up : up)) << 23);
}

// A row's results from its largest logit (base 2), the sum of exponentials
// relative to it, and how far its label's logit lies below it. For a confident
// row that gap and the sum's logarithm are small, while lse and the logit are
// large and nearly equal: they never meet in a difference. The sum holds the
// largest logit's 1, so the logarithm is that of 1 + (sum - 1).
struct RowLoss {
  float lse2, lse, loss;
};
__device__ __forceinline__ RowLoss row_loss(float top, float sum, float gap, float z_weight) {
  const float log_sum = log1pf(sum - 1.f);
  RowLoss o;
  o.lse2 = top + log_sum * kLog2e;
  o.lse = top * kLn2 + log_sum;
  o.loss = gap * kLn2 + log_sum + z_weight * o.lse * o.lse;
  return o;
}

__device__ __forceinline__ long long label_at(const void *labels, int bytes, int i) {
  return bytes == 8 ? static_cast<const long long *>(labels)[i]
                    : static_cast<const int *>(labels)[i];
}

// What the rounding of a label's d leaves out; nothing where d is not finite.
template <class T>
__device__ __forceinline__ float residue(float d) {
  const float r = d - from16<T>(bits16<T>(d));
  return fabsf(r) < __builtin_inff() ? r : 0.f;
}

// What a row left out gets: loss = lse = 0, or NaN in both for a label outside
// the vocabulary.
__device__ __forceinline__ void leave_out(long long t, long long ignore, int i, float *loss,
                                          float *lse) {
  if (!loss) return;
  const float v = t == ignore ? 0.f : __builtin_nanf("");
  loss[i] = v;
  lse[i] = v;
}

template <class T>
__device__ __forceinline__ float d_scale(const XentRows &r, bool inverse) {
  return d_scale_of<T>(T::kHalf ? r.head[1] : 0, inverse);
}

// The packed rows' x, 16 bytes per lane.
__device__ __forceinline__ void pack_row(const u32x4 *x, u32x4 *xc, int i, int p, int m, int hv) {
  const u32x4 *src = x + static_cast<long long>(i) * hv;
  u32x4 *dst = xc + static_cast<long long>(p) * 32;
  for (int k = static_cast<int>(threadIdx.x); k < hv; k += 256)
    dst[static_cast<long long>(k >> 5) * m * 32 + (k & 31)] = src[k];
}

// Packs the rows that count, in order, in one launch: a workgroup per row
// counts the rows before it that count. Up to kPackRows rows, where the labels
// (32 KB) stay in the caches; one launch less than the two below.
constexpr int kPackRows = 4096;
__global__ __launch_bounds__(256) void k_pack_few(XentRows r, const void *labels, int label_bytes,
                                                  int m, int vocab, long long ignore,
                                                  const u32x4 *x, u32x4 *xc, int hv, float *loss,
                                                  float *lse) {
  __shared__ int wave_sum[4];
  const int tid = static_cast<int>(threadIdx.x), i = static_cast<int>(blockIdx.x);
  const long long t = label_at(labels, label_bytes, i);
  const bool kept = t != ignore && t >= 0 && t < vocab;
  int before = 0;
  for (int k = tid; k < i; k += 256) {
    const long long o = label_at(labels, label_bytes, k);
    before += o != ignore && o >= 0 && o < vocab;
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) before += __shfl_xor(before, d);
  if ((tid & 63) == 0) wave_sum[tid >> 6] = before;
  __syncthreads();
  const int p = wave_sum[0] + wave_sum[1] + wave_sum[2] + wave_sum[3];
  if (tid == 0) {
    if (kept) {
      r.idx[p] = i;
      r.lab[p] = static_cast<int>(t);
    } else {
      leave_out(t, ignore, i, loss, lse);
    }
    r.inv[i] = kept ? p : -1;
    if (i == m - 1) {
      r.head[0] = p + kept;
      r.head[1] = 0;
    }
  }
  if (kept) pack_row(x, xc, i, p, m, hv);
}

// The same for more rows: one workgroup walks the labels 1024 at a time (a
// running total in LDS), a second launch copies.
__global__ __launch_bounds__(1024) void k_pack(XentRows r, const void *labels, int label_bytes,
                                               int m, int vocab, long long ignore, float *loss,
                                               float *lse) {
  __shared__ int wave_sum[16];
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 63, wave = tid >> 6;
  int base = 0;
  for (int i0 = 0; i0 < m; i0 += 1024) {
    const int i = i0 + tid;
    const long long t = i < m ? label_at(labels, label_bytes, i) : ignore;
    const bool kept = i < m && t != ignore && t >= 0 && t < vocab;
    const unsigned long long votes = __ballot(kept);
    if (lane == 0) wave_sum[wave] = __popcll(votes);
    __syncthreads();
    int before = base, total = 0;
    for (int k = 0; k < 16; ++k) {
      if (k < wave) before += wave_sum[k];
      total += wave_sum[k];
    }
    const int p = before + __popcll(votes & ((1ull << lane) - 1));
    if (kept) {
      r.idx[p] = i;
      r.lab[p] = static_cast<int>(t);
    }
    if (i < m) {
      r.inv[i] = kept ? p : -1;
      if (!kept) leave_out(t, ignore, i, loss, lse);
    }
    base += total;
    __syncthreads();
  }
  if (tid == 0) {
    r.head[0] = base;
    r.head[1] = 0;
  }
}

__global__ __launch_bounds__(256) void k_pack_rows(XentRows r, const u32x4 *x, u32x4 *xc, int m,
                                                   int hv) {
  const int kept = r.head[0];
  for (int p = static_cast<int>(blockIdx.x); p < kept; p += static_cast<int>(gridDim.x))
    pack_row(x, xc, r.idx[p], p, m, hv);
}

enum LogitsMode { kStats = 0, kProb = 1, kGrad = 2 };

template <class T, class Tile, int NT, int MODE>
__global__ __launch_bounds__(512, 2) void k_logits(XentPlan pl, const u32x4 *xc, ShardTableN<NT> w,
                                                   int shard, int v0, int vend, int tn) {
  __shared__ __attribute__((aligned(1024))) unsigned char lds[kTileLds];
  constexpr int kEdge = Tile::kEdge, MI = Tile::MI, NJ = Tile::NJ;
  const int kept = pl.r.head[0];
  int z, mt, nt;
  if (!tile_at(static_cast<int>(blockIdx.x), static_cast<int>(gridDim.x),
               (kept + kEdge - 1) / kEdge, tn, 1, &z, &mt, &nt))
    return;
  const int m0 = mt * kEdge, n0 = v0 + nt * kEdge;
  const int lane = static_cast<int>(threadIdx.x) & 63;
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
  const int wr = wave >> 2, wc = wave & 3, l16 = lane & 15, g = lane >> 4;

  PanelRowSource a;
  const int rows = kept - m0 < kEdge ? kept - m0 : kEdge;
  a.init(xc + static_cast<long long>(m0) * 32, rows, pl.m * 512ll, 0, pl.hidden, lane);
  RankRowSource<NT, Tile::kBLoads> b;
  b.init(w, shard, vend, pl.hidden, n0, Tile::b_sub(wave), Tile::b_first(wave), lane);
  f32x4 acc[MI][NJ];
  Tile::template product<T>(a, b, (pl.hidden + kStep - 1) / kStep, lds, acc);

  const float s2 = pl.scale * kLog2e;
  const int nl = n0 + Tile::kCols * wc + 4 * g;  // the lane's column of block 0
  // d's panel of this tile, from the wave's columns on
  unsigned short *dout = static_cast<unsigned short *>(pl.d) +
                         static_cast<long long>((n0 - v0) / kPanel) * pl.m * kPanel +
                         (n0 - v0) % kPanel + (nl - n0);
  if constexpr (MODE == kGrad) {
    const float up = d_scale<T>(pl.r, false);
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const int row = m0 + Tile::kRows * wr + 16 * i + l16;
      if (row >= kept) continue;
      const float lse2 = pl.r.lse2[row], ca = pl.r.ca[row] * up, cb = pl.r.cb[row] * up;
      const int lab = pl.r.lab[row];
      unsigned short *o = dout + static_cast<long long>(row) * kPanel;
      // few of a tile's rows have their label in it, and few tiles columns past
      // the vocabulary
      auto emit = [&](auto special) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          uint32_t q[4];
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            float v = exp2_(fmaf(acc[i][j][t], s2, -lse2)) * ca;
            if constexpr (decltype(special)::value) {
              const int n = nl + 16 * j + t;
              if (n == lab) {
                v -= cb;
                pl.r.res[row] = residue<T>(v);
              }
              v = n < vend ? v : 0.f;
            }
            q[t] = bits16<T>(v);
          }
          *reinterpret_cast<uint2 *>(o + 16 * j) = uint2{q[0] | q[1] << 16, q[2] | q[3] << 16};
        }
      };
      if (n0 + kEdge > vend || __any(lab >= nl && lab < nl + 16 * NJ))
        emit(std::integral_constant<bool, true>{});
      else
        emit(std::integral_constant<bool, false>{});
    }
    return;
  } else {
    // A row's columns of the tile lie in 4 waves x 4 lane groups x 4*NJ registers: the
    // maximum, then the sum of exponentials, each reduced in registers, over
    // the lane groups, and over the waves through LDS.
    float *red = reinterpret_cast<float *>(lds);  // [4][kEdge] maxima, then [4][kEdge] sums
    float top[MI];
    // Columns past the vocabulary, in its last tile alone, become -inf logits.
    const float masked = s2 < 0.f ? __builtin_inff() : -__builtin_inff();
    const bool last = n0 + kEdge > vend;
    if (last) {
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
          for (int t = 0; t < 4; ++t)
            if (nl + 16 * j + t >= vend) acc[i][j][t] = masked;
    }
    // The largest logit is the largest product, or the smallest if the scale
    // is negative.
    auto row_top = [&](auto pick) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        float mx = acc[i][0][0];
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
          for (int t = 0; t < 4; ++t) mx = pick(mx, acc[i][j][t]);
        mx = pick(mx, __shfl_xor(mx, 16));
        mx = pick(mx, __shfl_xor(mx, 32));
        if (g == 0) red[wc * kEdge + Tile::kRows * wr + 16 * i + l16] = mx * s2;
      }
    };
    if (s2 < 0.f)
      row_top([](float a, float b) __attribute__((always_inline)) { return fminf(a, b); });
    else
      row_top([](float a, float b) __attribute__((always_inline)) { return fmaxf(a, b); });
    __syncthreads();
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const int at = Tile::kRows * wr + 16 * i + l16;
      const float mx = fmaxf(fmaxf(red[at], red[kEdge + at]),
                             fmaxf(red[2 * kEdge + at], red[3 * kEdge + at]));
      top[i] = mx == -__builtin_inff() ? 0.f : mx;  // a row of -inf: every exponential is 0
    }
    float *sums = red + 4 * kEdge;
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const int row = m0 + Tile::kRows * wr + 16 * i + l16;
      const int lab = row < kept ? pl.r.lab[row] - nl : -1;
      // few of a tile's rows have their label in it
      if (__any(lab >= 0 && lab < 16 * NJ)) {
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
          for (int t = 0; t < 4; ++t)
            if (lab == 16 * j + t) pl.r.zt[row] = fmaf(acc[i][j][t], s2, -top[i]);
      }
      float sum = 0.f;
      unsigned short *o = dout + static_cast<long long>(row) * kPanel;
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        uint32_t q[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          float e = exp2_(fmaf(acc[i][j][t], s2, -top[i]));
          if (last && nl + 16 * j + t >= vend) e = 0.f;  // (at scale 0 too)
          sum += e;
          if (MODE == kProb) q[t] = Prob<T>::put(e);
        }
        if (MODE == kProb && row < kept)
          *reinterpret_cast<uint2 *>(o + 16 * j) = uint2{q[0] | q[1] << 16, q[2] | q[3] << 16};
      }
      sum += __shfl_xor(sum, 16);
      sum += __shfl_xor(sum, 32);
      if (g == 0) sums[wc * kEdge + Tile::kRows * wr + 16 * i + l16] = sum;
    }
    __syncthreads();
    const int at = static_cast<int>(threadIdx.x);
    if (at < kEdge && m0 + at < kept) {
      const float mx = fmaxf(fmaxf(red[at], red[kEdge + at]),
                             fmaxf(red[2 * kEdge + at], red[3 * kEdge + at]));
      const float sum = (sums[at] + sums[kEdge + at]) + (sums[2 * kEdge + at] + sums[3 * kEdge + at]);
      const int tiles = (pl.vocab + kEdge - 1) / kEdge;
      float *part = pl.part + static_cast<long long>(n0 / kEdge) * pl.m + m0 + at;
      part[0] = mx;
      part[static_cast<long long>(tiles) * pl.m] = sum;
    }
  }
}

// ---------------------------------------------------------------------------
// Few rows (decode, speculative tokens): the matrix is read once and bounds the
// call, so every CU streams its own run of the vocabulary, without a break from
// its first row to its last: workgroup b takes the 16-row units b*units/G ..,
// in tiles of 256 rows x 64 k, the loads running on across tile ends.
//
// A stage is 256 rows of W (32 KB) and 16*MB rows of x, read back from L2 by
// every workgroup (rows from m on lie beyond the resource and cost nothing).
// Wave v loads and multiplies rows 32v .. 32v+31 of the tile, so a barrier per
// step is needed for x alone. v_mfma_f32_16x16x32 with W as its rows: a lane
// holds, of one row of x, 8 columns per tile, and keeps a running maximum and
// sum over all of its columns; lanes, waves and workgroups are joined at the
// end. As many stages as LDS holds, up to four: 64 KB or more in flight per CU.
// HBM-bound: one row at V = 163840, H = 7168 takes 343 us, 6.85 TB/s of weights
// (64 rows: 370 us; on 256 x 256 tiles, 2.5 rounds of the CUs, 445 and 460).
//
// KC: a run of at most 128 or 64 rows leaves sub-tiles of the 256 empty, and
// with them bytes in flight. Its stage holds KC = 2 or 4 times as much k instead:
// sub-tile s is the rows 64*(s % RB) of chunk s / RB of the step's 64*KC k, and
// the waves of the chunks add up their parts of the one tile at the end. (One
// row at V = 20480, H = 7168, a rank's share at TP = 8: 64 us with KC = 1, 49
// with KC = 2.)
//
// A logit is summed in chains of kChain steps, each added to a total of its own:
// every addition to a sum rounds at the sum's size, and a label's logit is a sum
// of terms of one sign, which has its full size for much of a chain of 7168
// products. (Losses of rows whose labels' logits are about 12, V = 163840: off by
// 1.0 * 2^-24 of the logit, rms, instead of 6; the same time.)
template <class T, int NT, int MB, int KC>
__global__ __launch_bounds__(512, 2) void k_score(XentPlan pl, const u32x4 *x, const void *labels,
                                                  ShardTableN<NT> w, int shard) {
  constexpr int RB = 4 / KC;                                 // 64-row blocks of a tile
  constexpr int XR = 16 * MB > 64 / KC ? 16 * MB : 64 / KC;  // rows of x in a chunk's stage
  constexpr int XI = KC * XR / 64;                           // x loads per wave and step
  constexpr int kStageB = 4 * kSubBytes + KC * XR * 128;
  constexpr int ST = 4 * kStageB <= 160 * 1024 ? 4 : 3 * kStageB <= 160 * 1024 ? 3 : 2;
  constexpr int kLoads = 4 + XI;
  __shared__ __attribute__((aligned(1024))) unsigned char lds[ST * kStageB];
  const int lane = static_cast<int>(threadIdx.x) & 63;
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  const long long units = (pl.vocab + 15) >> 4;
  const int r0 = static_cast<int>(units * blockIdx.x / gridDim.x) * 16;
  int r1 = static_cast<int>(units * (blockIdx.x + 1) / gridDim.x) * 16;
  if (r1 > pl.vocab) r1 = pl.vocab;
  const int ks = (pl.hidden + kStep * KC - 1) / (kStep * KC);
  const int steps = r1 > r0 ? (r1 - r0 + 64 * RB - 1) / (64 * RB) * ks : 0;

  const LoadLane ll = load_lane<false>(lane);
  const rsrc_t xr = resource(x, static_cast<long long>(pl.m) * pl.hidden * 2);
  const int k8 = pl.hidden >> 3;
  const int sub = wave >> 1, q0 = 4 * (wave & 1);
  const int block = sub % RB, chunk = sub / RB;  // of the wave's sub-tile
  RankRowSource<NT, 4, true> b;
  int lt = 0, lk = 0;  // tile and step of k of the next loads
  b.init(w, shard, r1, pl.hidden, r0, block, q0, lane);
  auto load = [&](int s) __attribute__((always_inline)) {
    unsigned char *st = lds + (s % ST) * kStageB;
    // steps past the last one load nothing and keep the counts
    const int kk = s < steps ? lk : ks;
#pragma unroll
    for (int i = 0; i < XI; ++i) {
      const int all = 8 * i + wave, q = all % (XR / 8), o = q & 1;
      const int k64 = kk * KC + all / (XR / 8);
      const unsigned v = static_cast<unsigned>((8 * q + ll.row) * pl.hidden * 2 + k64 * 128 +
                                               ll.chunk[o] * 16);
      load_lds(xr, st + 4 * kSubBytes + all * 1024, k64 * 8 + ll.chunk[o] < k8 ? v : kBeyond);
    }
#pragma unroll
    for (int t = 0; t < 4; ++t) b.load(st + sub * kSubBytes, block, q0 + t, kk * KC + chunk);
    if (++lk == ks && s + 1 < steps) {
      lk = 0;
      ++lt;
      b.init(w, shard, r1, pl.hidden, r0 + lt * 64 * RB, block, q0, lane);
    }
  };

  FragLane<false> f;
  f.init(lane);
  f32x4 acc[2][MB], total[2][MB];
  float top[MB], sum[MB];
  int lab[MB];
#pragma unroll
  for (int j = 0; j < MB; ++j) {
    acc[0][j] = acc[1][j] = total[0][j] = total[1][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    top[j] = -__builtin_inff();
    sum[j] = 0.f;
    const int row = 16 * j + l16;
    const long long t = row < pl.m ? label_at(labels, pl.label_bytes, row) : -1;
    lab[j] = t >= 0 && t < pl.vocab ? static_cast<int>(t) : -1;
  }
  const float s2 = pl.scale * kLog2e;
  __asm__ __volatile__("s_waitcnt vmcnt(0)" ::: "memory");  // the labels: only the loads below count

  int n0 = r0 + 64 * block + 32 * (wave & 1) + 4 * g;
  // A chain ends: into the totals.
  auto chain_done = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < MB; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        total[h][j] += acc[h][j];
        acc[h][j] = f32x4{0.f, 0.f, 0.f, 0.f};
      }
  };
  // The tile's columns are done: into the running statistics. An exponential is
  // of a logit less a reference, rounded once; the reference may be any number
  // near the largest logit, so its own rounding takes nothing from it.
  auto tile_done = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < MB; ++j) {
      float mx = top[j];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const int n = n0 + 16 * h + t;
          if (n == lab[j] && n < r1) pl.r.zt[16 * j + l16] = total[h][j][t];  // past r1: another's
          mx = fmaxf(mx, n < r1 ? total[h][j][t] * s2 : -__builtin_inff());
        }
      const float ref = mx == -__builtin_inff() ? 0.f : mx;
      float e = sum[j] * exp2_(top[j] - ref);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int t = 0; t < 4; ++t)
          e += n0 + 16 * h + t < r1 ? exp2_(fmaf(total[h][j][t], s2, -ref)) : 0.f;
      sum[j] = e;
      top[j] = mx;
      total[0][j] = total[1][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
  };

#pragma unroll
  for (int s = 0; s < ST - 1; ++s) load(s);
  int ck = 0;
  for (int s = 0; s < steps; ++s) {
    wait_vm_lds<kLoads * (ST - 2)>();
    tile_barrier();
    load(s + ST - 1);
    const unsigned char *st = lds + (s % ST) * kStageB;
    const unsigned char *sw = st + sub * kSubBytes + (wave & 1) * 32 * 128;
    const unsigned char *sx = st + 4 * kSubBytes + chunk * XR * 128;
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      const s16x8 w0 = f.read(sw, 0, kk), w1 = f.read(sw, 1, kk);
#pragma unroll
      for (int j = 0; j < MB; ++j) {
        const s16x8 xv = f.read(sx, j, kk);
        acc[0][j] = T::mma(w0, xv, acc[0][j]);
        acc[1][j] = T::mma(w1, xv, acc[1][j]);
      }
    }
    ++ck;
    const bool last = ck == ks;
    if (ck % kChain == 0 || last) chain_done();
    if (KC == 1 && last) {
      ck = 0;
      tile_done();
      n0 += 64 * RB;
    }
  }
  wait_vm_lds<0>();
  tile_barrier();
  if constexpr (KC > 1) {
    f32x4 *part = reinterpret_cast<f32x4 *>(lds);  // [8][2 * MB][64]
#pragma unroll
    for (int j = 0; j < MB; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h) part[((wave * MB + j) * 2 + h) * 64 + lane] = total[h][j];
    wait_lds();
    tile_barrier();
    if (chunk == 0) {
#pragma unroll
      for (int j = 0; j < MB; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int c = 1; c < KC; ++c)
            total[h][j] += part[(((wave + 2 * RB * c) * MB + j) * 2 + h) * 64 + lane];
      tile_done();
    }
    wait_lds();
    tile_barrier();
  }
  float *red = reinterpret_cast<float *>(lds);  // [8][16*MB][2]
#pragma unroll
  for (int j = 0; j < MB; ++j) {
    float mx = top[j];
    mx = fmaxf(mx, __shfl_xor(mx, 16));
    mx = fmaxf(mx, __shfl_xor(mx, 32));
    float e = sum[j] * exp2_(top[j] - (mx == -__builtin_inff() ? 0.f : mx));
    e += __shfl_xor(e, 16);
    e += __shfl_xor(e, 32);
    if (g == 0) {
      red[(wave * 16 * MB + 16 * j + l16) * 2] = mx;
      red[(wave * 16 * MB + 16 * j + l16) * 2 + 1] = e;
    }
  }
  __syncthreads();
  const int row = static_cast<int>(threadIdx.x);
  if (row < 16 * MB && row < pl.m) {
    float mx = -__builtin_inff(), e = 0.f;
#pragma unroll
    for (int v = 0; v < 8; ++v) mx = fmaxf(mx, red[(v * 16 * MB + row) * 2]);
    const float ref = mx == -__builtin_inff() ? 0.f : mx;
#pragma unroll
    for (int v = 0; v < 8; ++v)
      e += red[(v * 16 * MB + row) * 2 + 1] * exp2_(red[(v * 16 * MB + row) * 2] - ref);
    float2 *part = reinterpret_cast<float2 *>(pl.part);
    part[static_cast<long long>(row) * kScoreGroups + blockIdx.x] = float2{mx, e};
  }
}

// One wave per row joins the workgroups' statistics.
__global__ __launch_bounds__(64) void k_score_join(XentPlan pl, const void *labels, int groups,
                                                   float *loss, float *lse) {
  const int row = static_cast<int>(blockIdx.x), lane = static_cast<int>(threadIdx.x);
  const float2 *part = reinterpret_cast<const float2 *>(pl.part) +
                       static_cast<long long>(row) * kScoreGroups;
  const long long t = label_at(labels, pl.label_bytes, row);
  const float zt = pl.r.zt[row];
  float2 p[kScoreGroups / 64];
  float mx = -__builtin_inff(), sum = 0.f;
#pragma unroll
  for (int k = 0; k < kScoreGroups / 64; ++k) {
    p[k] = lane + 64 * k < groups ? part[lane + 64 * k] : float2{-__builtin_inff(), 0.f};
    mx = fmaxf(mx, p[k].x);
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) mx = fmaxf(mx, __shfl_xor(mx, d));
  const float ref = mx == -__builtin_inff() ? 0.f : mx;
#pragma unroll
  for (int k = 0; k < kScoreGroups / 64; ++k) sum += p[k].y * exp2_(p[k].x - ref);
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d);
  if (lane != 0) return;
  float a = 0.f, b = 0.f;
  if (t != pl.ignore) {
    const RowLoss o = row_loss(ref, sum, -fmaf(zt, pl.scale * kLog2e, -ref), pl.z_weight);
    const bool real = t >= 0 && t < pl.vocab;
    b = real ? o.lse : __builtin_nanf("");
    a = real ? o.loss : b;
  }
  loss[row] = a;
  lse[row] = b;
}

// Merges a row's tiles: 16 rows per workgroup, 16 threads a row, eight tiles in
// flight each (4096 rows of 640 tiles: 13 us; one at a time 26).
__global__ __launch_bounds__(256) void k_join(XentPlan pl, const float *grad, float *loss,
                                              float *lse) {
  __shared__ float smax[16][17], ssum[16][17];
  const int kept = pl.r.head[0];
  const int tiles = (pl.vocab + pl.ref - 1) / pl.ref;
  const int c = static_cast<int>(threadIdx.x) & 15, k = static_cast<int>(threadIdx.x) >> 4;
  const int row = static_cast<int>(blockIdx.x) * 16 + c;
  float mx = -__builtin_inff(), sum = 0.f;
  if (row < kept) {
    const float *pm = pl.part + row;
    const float *ps = pm + static_cast<long long>(tiles) * pl.m;
    for (int t0 = k; t0 < tiles; t0 += 16 * 8) {  // eight tiles in flight
      float a[8], b[8], hi = mx;
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int t = t0 + 16 * u;
        a[u] = t < tiles ? pm[static_cast<long long>(t) * pl.m] : -__builtin_inff();
        b[u] = t < tiles ? ps[static_cast<long long>(t) * pl.m] : 0.f;
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) hi = fmaxf(hi, a[u]);
      const float ref = hi == -__builtin_inff() ? 0.f : hi;
      sum *= exp2_(mx - ref);
#pragma unroll
      for (int u = 0; u < 8; ++u) sum += b[u] * exp2_(a[u] - ref);
      mx = hi;
    }
  }
  smax[k][c] = mx;
  ssum[k][c] = sum;
  __syncthreads();
  if (k != 0 || row >= kept) return;
  for (int t = 1; t < 16; ++t) mx = fmaxf(mx, smax[t][c]);
  const float ref = mx == -__builtin_inff() ? 0.f : mx;
  sum = 0.f;
  for (int t = 0; t < 16; ++t) sum += ssum[t][c] * exp2_(smax[t][c] - ref);
  const float own = pl.part[static_cast<long long>(pl.r.lab[row] / pl.ref) * pl.m + row];
  const RowLoss o = row_loss(ref, sum, (ref - own) - pl.r.zt[row], pl.z_weight);
  const float l2 = o.lse2, l = o.lse;
  const int i = pl.r.idx[row];
  loss[i] = o.loss;
  lse[i] = l;
  if (!grad) return;
  const float u = pl.scale * grad[i];
  const float ca = u * (1.f + 2.f * pl.z_weight * l);
  pl.r.lse2[row] = l2;
  pl.r.ca[row] = ca;
  pl.r.cb[row] = u;
  const float f = fmaxf(fabsf(u), fabsf(ca));
  if (f < __builtin_inff()) atomicMax(pl.r.head + 1, __builtin_bit_cast(int, f));
}

__global__ __launch_bounds__(256) void k_factors(XentPlan pl, const float *lse, const float *grad) {
  const int row = static_cast<int>(blockIdx.x) * 256 + static_cast<int>(threadIdx.x);
  if (row >= pl.r.head[0]) return;
  const int i = pl.r.idx[row];
  const float l = lse[i], u = pl.scale * grad[i];
  const float ca = u * (1.f + 2.f * pl.z_weight * l);
  pl.r.lse2[row] = l * kLog2e;
  pl.r.ca[row] = ca;
  pl.r.cb[row] = u;
  const float f = fmaxf(fabsf(u), fabsf(ca));
  if (f < __builtin_inff()) atomicMax(pl.r.head + 1, __builtin_bit_cast(int, f));
}

// 16 bytes (8 columns) of a row's unnormalised probabilities -> d: times c, less
// cb at column `at` of them. The label's probability comes from its logit, not
// from the 16 bits that waited.
template <class T>
__device__ __forceinline__ u32x4 normalised(const XentRows &r, int row, u32x4 v, float c, float cb,
                                            int at) {
  float label = 0.f;
  if (at >= 0 && at < 8) {
    label = exp2_(r.zt[row]) * c - cb;
    r.res[row] = residue<T>(label);
  }
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    float lo = Prob<T>::get(v[t] & 0xFFFFu) * c, hi = Prob<T>::get(v[t] >> 16) * c;
    if (at == 2 * t) lo = label;
    if (at == 2 * t + 1) hi = label;
    v[t] = bits16<T>(lo) | bits16<T>(hi) << 16;
  }
  return v;
}

// Unnormalised probabilities -> d in place: 16 bytes per lane and step, 8 rows
// of a panel per workgroup and step. HBM-bound: reads and writes d once (4096
// rows, V = 163840: 0.51 ms, 5.3 TB/s).
template <class T>
__global__ __launch_bounds__(256) void k_normalise(XentPlan pl) {
  const int kept = pl.r.head[0];
  const int panel = static_cast<int>(blockIdx.x);
  const float up = d_scale<T>(pl.r, false);
  const int k = static_cast<int>(threadIdx.x) & 31;
  const int tile = (panel * kPanel + 8 * k) / pl.ref;
  if (tile >= (pl.vocab + pl.ref - 1) / pl.ref) return;  // columns no tile wrote or reads
  const float *part = pl.part + static_cast<long long>(tile) * pl.m;
  u32x4 *d = static_cast<u32x4 *>(pl.d) + static_cast<long long>(panel) * pl.m * 32;
  for (int row = static_cast<int>(blockIdx.y * 8 + threadIdx.x / 32); row < kept;
       row += static_cast<int>(gridDim.y) * 8) {
    const float mx = part[row];
    const float ref = mx == -__builtin_inff() ? 0.f : mx;
    const float c = exp2_(ref - pl.r.lse2[row]) * (pl.r.ca[row] * up), cb = pl.r.cb[row] * up;
    u32x4 *o = d + static_cast<long long>(row) * 32 + k;
    *o = normalised<T>(pl.r, row, *o, c, cb, pl.r.lab[row] - panel * kPanel - 8 * k);
  }
}

// k_join and k_normalise in one (see xent_joins_in_place): the 32 lanes of a
// row merge its tiles, two at most each. One launch less where launches are
// what a call takes: 33 rows at V = 4096, H = 264 take 31.7 us a step instead of
// 36.2.
template <class T>
__global__ __launch_bounds__(256) void k_join_normalise(XentPlan pl, const float *grad, float *loss,
                                                        float *lse) {
  __shared__ int wave_top[4];
  const int kept = pl.r.head[0];
  const int panel = static_cast<int>(blockIdx.x), tid = static_cast<int>(threadIdx.x);
  const int tiles = (pl.vocab + pl.ref - 1) / pl.ref;
  int largest = 0;
  if constexpr (T::kHalf) {
    for (int row = tid; row < kept; row += 256) {
      const float f = fabsf(pl.scale * grad[pl.r.idx[row]]);
      const int bits = f < __builtin_inff() ? __builtin_bit_cast(int, f) : 0;
      largest = largest > bits ? largest : bits;
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_xor(largest, d);
      largest = largest > o ? largest : o;
    }
    if ((tid & 63) == 0) wave_top[tid >> 6] = largest;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 4; ++k) largest = largest > wave_top[k] ? largest : wave_top[k];
    if (panel == 0 && blockIdx.y == 0 && tid == 0) pl.r.head[1] = largest;
  }
  const float up = d_scale_of<T>(largest, false);
  const int k = tid & 31, mine = (panel * kPanel + 8 * k) / pl.ref;
  u32x4 *d = static_cast<u32x4 *>(pl.d) + static_cast<long long>(panel) * pl.m * 32;
  for (int row = static_cast<int>(blockIdx.y * 8 + tid / 32); row < kept;
       row += static_cast<int>(gridDim.y) * 8) {
    const float *pm = pl.part + row;
    const float *ps = pm + static_cast<long long>(tiles) * pl.m;
    const float a0 = k < tiles ? pm[static_cast<long long>(k) * pl.m] : -__builtin_inff();
    const float b0 = k < tiles ? ps[static_cast<long long>(k) * pl.m] : 0.f;
    const bool two = k + 32 < tiles;
    const float a1 = two ? pm[static_cast<long long>(k + 32) * pl.m] : -__builtin_inff();
    const float b1 = two ? ps[static_cast<long long>(k + 32) * pl.m] : 0.f;
    float mx = fmaxf(a0, a1);
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) mx = fmaxf(mx, __shfl_xor(mx, s));
    const float all = mx == -__builtin_inff() ? 0.f : mx;
    float sum = b0 * exp2_(a0 - all) + b1 * exp2_(a1 - all);
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) sum += __shfl_xor(sum, s);
    const float own = pm[static_cast<long long>(pl.r.lab[row] / pl.ref) * pl.m];
    const RowLoss r = row_loss(all, sum, (all - own) - pl.r.zt[row], pl.z_weight);
    const float l2 = r.lse2, l = r.lse;
    const int i = pl.r.idx[row];
    const float u = pl.scale * grad[i];
    if (panel == 0 && k == 0) {
      loss[i] = r.loss;
      lse[i] = l;
    }
    if (mine >= tiles) continue;
    const float top = pm[static_cast<long long>(mine) * pl.m];
    const float ref = top == -__builtin_inff() ? 0.f : top;
    const float c = exp2_(ref - l2) * (u * (1.f + 2.f * pl.z_weight * l) * up);
    u32x4 *o = d + static_cast<long long>(row) * 32 + k;
    *o = normalised<T>(pl.r, row, *o, c, u * up, pl.r.lab[row] - panel * kPanel - 8 * k);
  }
}

// Four consecutive columns of dW, in fp32 or 16 bits.
template <class T>
__device__ __forceinline__ void dw_store(void *dw, long long at, f32x4 v, int wide,
                                         int accumulate) {
  if (wide) {
    f32x4 *o = reinterpret_cast<f32x4 *>(static_cast<float *>(dw) + at);
    *o = accumulate ? *o + v : v;
  } else {
    uint2 *o = reinterpret_cast<uint2 *>(static_cast<unsigned short *>(dw) + at);
    if (accumulate) {
      const uint2 old = *o;
      v += f32x4{from16<T>(old.x & 0xFFFFu), from16<T>(old.x >> 16), from16<T>(old.y & 0xFFFFu),
                 from16<T>(old.y >> 16)};
    }
    *o = uint2{bits16<T>(v[0]) | bits16<T>(v[1]) << 16, bits16<T>(v[2]) | bits16<T>(v[3]) << 16};
  }
}

// The two products of the gradient, in one launch: the first workgroups take
// dX's tiles (few and long, so they start first), the others dW's, which fill
// the CUs that dX leaves over.
struct GradArgs {
  int v0, vend;       // the piece's columns
  int xgroups, per, first;  // dX: workgroups, steps per split, whether sums start at 0
  int wm, tn;         // dW: tile rows; both: tile columns
  void *dw;
  int wide, accumulate;
};

// The residues of the labels' d in a dW tile of vocabulary rows v0 .. and columns
// n0 .., over the packed rows k0 .. k1-1. The rows with a label in the tile are
// listed, each wave's in a part of the list of its own, and 64 of them at a time
// are the k of one more step of the product: their x is gathered into LDS as a
// column operand, beside an operand of zeros with one residue for each k. The first
// labels are loaded before the product, which covers their latency.
// (Both products of the gradient of 4096 rows at V = 163840, H = 7168 take 14.86 ms
// with the residues and 14.68 without, of 8192 rows at V = 32768, H = 1024 779 us and
// 759, of 777 rows at V = 32768, H = 4096 406 and 386. One row at a time, from
// registers, 225 us more at 8192 rows, 780 of which share a label; the residues'
// operand compared together in registers 8 us more there; gathered behind the
// product's first loads, the same.)
typedef int i32x8 __attribute__((ext_vector_type(8)));
template <class T, class Tile>
struct Residues {
  static constexpr int kTurn = 8 * 512;                    // labels listed at a time
  static constexpr int kSubs = Tile::kEdge / 64;           // sub-tiles of an operand
  static constexpr int kX = 0, kA = kSubs * kSubBytes, kList = 2 * kA, kCounts = kList + 4 * kTurn;
  static_assert(kCounts + 32 <= kTileLds);

  // The thread's labels of the turn from `base` on.
  static __device__ __forceinline__ i32x8 load(const XentPlan &pl, int base, int k1) {
    i32x8 at;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int p = base + 512 * u + static_cast<int>(threadIdx.x);
      at[u] = p < k1 ? pl.r.lab[p] : -1;
    }
    return at;
  }
  // After the product, when LDS is free; `at`: the first turn's labels.
  static __device__ __forceinline__ void add(const XentPlan &pl, i32x8 at, int v0, int n0, int k0,
                                             int k1, unsigned char *lds,
                                             f32x4 (&acc)[Tile::MI][Tile::NJ]) {
    const int tid = static_cast<int>(threadIdx.x), lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wr = wave >> 2, wc = wave & 3;
    unsigned *list = reinterpret_cast<unsigned *>(lds + kList);  // tile row << 24 | packed row
    int *count = reinterpret_cast<int *>(lds + kCounts);
    const unsigned char *x = static_cast<const unsigned char *>(pl.xc) +
                             static_cast<long long>(n0 / kPanel) * pl.m * (2 * kPanel) +
                             n0 % kPanel * 2;
    auto clear = [&]() __attribute__((always_inline)) {
#pragma unroll
      for (int u = 0; u < kSubs; ++u)
        *reinterpret_cast<u32x4 *>(lds + kA + (u * 512 + tid) * 16) = u32x4{0u, 0u, 0u, 0u};
    };
    FragLane<true> f;
    f.init(lane);
    for (int base = k0; base < k1; base += kTurn) {
      if (base > k0) {
        at = load(pl, base, k1);
        __syncthreads();
      }
      int run = 0;
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int row = at[u] - v0;  // (no label: -1, below every tile)
        const bool in = at[u] >= v0 && row < Tile::kEdge;
        const unsigned long long lanes = __ballot(in);
        if (in)
          list[wave * 512 + run + __popcll(lanes & ((1ull << lane) - 1))] =
              static_cast<unsigned>(row) << 24 | static_cast<unsigned>(base + 512 * u + tid);
        run += __popcll(lanes);
      }
      if (lane == 0) count[wave] = run;
      clear();
      __syncthreads();
      int first[9];  // of each wave's rows among all
      first[0] = 0;
#pragma unroll
      for (int w = 0; w < 8; ++w)
        first[w + 1] = first[w] + __builtin_amdgcn_readfirstlane(count[w]);
      const int all = first[8];
      auto listed = [&](int q) __attribute__((always_inline)) {
        int at_q = q;
#pragma unroll
        for (int w = 1; w < 8; ++w) at_q = q >= first[w] ? q - first[w] + 512 * w : at_q;
        return list[at_q];
      };
      for (int q0 = 0; q0 < all; q0 += 64) {
        if (q0) {
          __syncthreads();
          clear();
          __syncthreads();
        }
        const int here = all - q0 < 64 ? all - q0 : 64, steps = here > 32 ? 2 : 1;
        if (tid < here) {
          const unsigned e = listed(q0 + tid), row = e >> 24;
          const int fk = ((tid >> 1) & 1) | ((tid >> 3) & 1) << 1;
          *reinterpret_cast<unsigned short *>(lds + kA + (row >> 6) * kSubBytes + tid * 128 +
                                              ((((row >> 3) & 7) ^ (2 * fk)) << 4) + (row & 7) * 2) =
              static_cast<unsigned short>(bits16<T>(pl.r.res[e & 0xFFFFFFu]));
        }
        constexpr int kChunks = Tile::kEdge / 8;  // of 16 bytes in a row of x
#pragma unroll
        for (int u = 0; u < kSubs; ++u) {
          const int q = (u * 512 + tid) / kChunks, c = tid % kChunks;
          if (u >= kSubs / 2 && steps == 1) break;
          u32x4 v = {0u, 0u, 0u, 0u};
          if (q < here)
            v = *reinterpret_cast<const u32x4 *>(
                x + static_cast<long long>(listed(q0 + q) & 0xFFFFFFu) * (2 * kPanel) + 16 * c);
          const int fk = ((q >> 1) & 1) | ((q >> 3) & 1) << 1;
          *reinterpret_cast<u32x4 *>(lds + kX + (c >> 3) * kSubBytes + q * 128 +
                                     (((c & 7) ^ (2 * fk)) << 4)) = v;
        }
        __syncthreads();
#pragma unroll 1
        for (int ks = 0; ks < steps; ++ks) {
          s16x8 ra[Tile::MI], rb[Tile::NJ];
#pragma unroll
          for (int j = 0; j < Tile::NJ; ++j) {
            if constexpr (Tile::NJ == 4)
              rb[j] = f.read(lds + kX + wc * kSubBytes, j, ks);
            else
              rb[j] = (wc & 1) ? f.read(lds + kX + (wc >> 1) * kSubBytes, 2 + j, ks)
                               : f.read(lds + kX + (wc >> 1) * kSubBytes, j, ks);
          }
#pragma unroll
          for (int i = 0; i < Tile::MI; ++i)
            ra[i] = f.read(lds + kA + (wr * (Tile::MI / 4) + i / 4) * kSubBytes, i % 4, ks);
#pragma unroll
          for (int i = 0; i < Tile::MI; ++i)
#pragma unroll
            for (int j = 0; j < Tile::NJ; ++j) acc[i][j] = T::mma(rb[j], ra[i], acc[i][j]);
        }
      }
    }
  }
};

template <class T, class Tile, int NT>
__global__ __launch_bounds__(512, 2) void k_grads(XentPlan pl, ShardTableN<NT> w, int shard,
                                                  GradArgs ga) {
  __shared__ __attribute__((aligned(1024))) unsigned char lds[kTileLds];
  constexpr int kEdge = Tile::kEdge, MI = Tile::MI, NJ = Tile::NJ;
  const int lane = static_cast<int>(threadIdx.x) & 63;
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
  const int wr = wave >> 2, wc = wave & 3, l16 = lane & 15, g = lane >> 4;
  const int kept = pl.r.head[0];
  const int v0 = ga.v0, vend = ga.vend;
  int z, mt, nt;
  f32x4 acc[MI][NJ];
  if (static_cast<int>(blockIdx.x) < ga.xgroups) {
    // dX = d W over a run of the piece's columns; fp32 partial sums, joined in a
    // fixed order by k_dx_join
    if (!tile_at(static_cast<int>(blockIdx.x), ga.xgroups, (kept + kEdge - 1) / kEdge, ga.tn,
                 pl.split_dx, &z, &mt, &nt))
      return;
    const int m0 = mt * kEdge, n0 = nt * kEdge;
    const int k0 = z * ga.per * kStep;
    int k1 = k0 + ga.per * kStep;
    if (k1 > vend - v0) k1 = vend - v0;
    const int steps = k1 > k0 ? (k1 - k0 + kStep - 1) / kStep : 0;
    PanelRowSource a;
    const int rows = kept - m0 < kEdge ? kept - m0 : kEdge;
    // d's columns past the vocabulary are zero up to a whole tile
    a.init(static_cast<const unsigned char *>(pl.d) + m0 * 512ll, rows, pl.m * 512ll, k0,
           steps * kStep, lane);
    RankColumnSource<NT> b;
    b.init(w, shard, v0 + (k1 > k0 ? k1 : k0), v0 + k0, n0, pl.hidden, lane);
    Tile::template product<T>(a, b, steps, lds, acc);
    float *out = pl.dxp + static_cast<long long>(z) * pl.m * pl.hidden;
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const int row = m0 + Tile::kRows * wr + 16 * i + l16;
      if (row >= kept) continue;
      float *o = out + static_cast<long long>(row) * pl.hidden;
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const int n = n0 + Tile::kCols * wc + 16 * j + 4 * g;
        if (n >= pl.hidden) continue;
        f32x4 *at = reinterpret_cast<f32x4 *>(o + n);
        *at = ga.first ? acc[i][j] : *at + acc[i][j];
      }
    }
    return;
  }
  // dW rows of the piece = d^T X over the packed rows, or over a run of them
  // (fp32 partial sums, joined by k_dw_join)
  if (!tile_at(static_cast<int>(blockIdx.x) - ga.xgroups,
               static_cast<int>(gridDim.x) - ga.xgroups, ga.wm, ga.tn, pl.split_dw, &z, &mt, &nt))
    return;
  const int c0 = mt * kEdge, n0 = nt * kEdge;  // column of the piece
  int k0 = 0, k1 = kept;
  const bool split = pl.split_dw > 1;
  if (split) {
    const int per = ((kept + kStep - 1) / kStep + pl.split_dw - 1) / pl.split_dw * kStep;
    k0 = z * per < kept ? z * per : kept;
    k1 = k0 + per < kept ? k0 + per : kept;
  }
  const int kdim = k1 - k0;
  PanelColumnSource a, b;
  a.init(static_cast<const unsigned char *>(pl.d) +
             (static_cast<long long>(c0 / kPanel) * pl.m + k0) * 512,
         c0 % kPanel, kdim, lane);
  b.init(static_cast<const unsigned char *>(pl.xc) +
             (static_cast<long long>(n0 / kPanel) * pl.m + k0) * 512,
         n0 % kPanel, kdim, lane);
  using Res = Residues<T, Tile>;
  const i32x8 labels = Res::load(pl, k0, k1);
  Tile::template product<T>(a, b, (kdim + kStep - 1) / kStep, lds, acc);
  Res::add(pl, labels, v0 + c0, n0, k0, k1, lds, acc);
  const float down = split ? 1.f : d_scale<T>(pl.r, true);
  void *out = split ? static_cast<void *>(pl.dwp +
                                          static_cast<long long>(z) * pl.piece * pl.hidden)
                    : ga.dw;
  const int wide = split ? 1 : ga.wide, accumulate = split ? 0 : ga.accumulate;
  // rows past the vocabulary get no gradient, whatever x holds: zeros as far as
  // the tile goes, or nothing
  const int wend = split || ga.accumulate ? vend : pl.rows;
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    const int row = v0 + c0 + Tile::kRows * wr + 16 * i + l16;
    if (row >= wend) continue;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int n = n0 + Tile::kCols * wc + 16 * j + 4 * g;
      if (n >= pl.hidden) continue;
      const f32x4 v = row < vend ? acc[i][j] * down : f32x4{0.f, 0.f, 0.f, 0.f};
      dw_store<T>(out, static_cast<long long>(split ? row - v0 : row) * pl.hidden + n, v, wide,
                  accumulate);
    }
  }
}

// The sum of n partial sums, in order, eight loads in flight.
__device__ __forceinline__ f32x4 add_planes(const f32x4 *src, long long plane, int n) {
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
  for (int z0 = 0; z0 < n; z0 += 8) {
    f32x4 p[8];
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (z0 + u < n) p[u] = src[(z0 + u) * plane];
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (z0 + u < n) v += p[u];
  }
  return v;
}

// Partial sums and the label's residue -> dx rows (zero where the row is left
// out): four columns per lane.
template <class T, int NT>
__global__ __launch_bounds__(256) void k_dx_join(XentPlan pl, ShardTableN<NT> w, int shard,
                                                 uint2 *dx) {
  const float down = d_scale<T>(pl.r, true);
  const int hq = pl.hidden >> 2;
  const long long plane = static_cast<long long>(pl.m) * hq;
  for (int row = static_cast<int>(blockIdx.y); row < pl.m; row += static_cast<int>(gridDim.y)) {
    const int p = pl.r.inv[row];
    const float res = p >= 0 ? pl.r.res[p] : 0.f;
    const int lab = p >= 0 ? pl.r.lab[p] : 0, rank = NT == 1 ? 0 : lab / shard;
    const uint2 *wl = reinterpret_cast<const uint2 *>(w.p[rank]) +
                      static_cast<long long>(lab - rank * shard) * hq;
    for (int k = static_cast<int>(blockIdx.x * 256 + threadIdx.x); k < hq;
         k += static_cast<int>(gridDim.x) * 256) {
      uint2 o = {0u, 0u};
      if (p >= 0) {
        const f32x4 *src = reinterpret_cast<const f32x4 *>(pl.dxp) + static_cast<long long>(p) * hq + k;
        const uint2 wv = wl[k];
        f32x4 v = add_planes(src, plane, pl.split_dx);
        if (res != 0.f)
          v += f32x4{from16<T>(wv.x & 0xFFFFu), from16<T>(wv.x >> 16), from16<T>(wv.y & 0xFFFFu),
                     from16<T>(wv.y >> 16)} * res;
        v *= down;
        o = uint2{bits16<T>(v[0]) | bits16<T>(v[1]) << 16, bits16<T>(v[2]) | bits16<T>(v[3]) << 16};
      }
      dx[static_cast<long long>(row) * hq + k] = o;
    }
  }
}

// Partial sums -> the piece's `cols` rows of dw; zeros from there to `rows`.
template <class T>
__global__ __launch_bounds__(256) void k_dw_join(XentPlan pl, int v0, int cols, int rows, void *dw,
                                                 int wide, int accumulate) {
  const float down = d_scale<T>(pl.r, true);
  const int hq = pl.hidden >> 2;
  const long long sums = static_cast<long long>(cols) * hq, n = static_cast<long long>(rows) * hq;
  const long long plane = static_cast<long long>(pl.piece) * hq;
  for (long long k = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x; k < n;
       k += static_cast<long long>(gridDim.x) * 256) {
    const f32x4 *src = reinterpret_cast<const f32x4 *>(pl.dwp) + k;
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
    if (k < sums) v = add_planes(src, plane, pl.split_dw);
    dw_store<T>(dw, static_cast<long long>(v0) * pl.hidden + 4 * k, v * down, wide, accumulate);
  }
}

template <int NT>
ShardTableN<NT> small_table(const ShardTable &t) {
  ShardTableN<NT> o;
  for (int r = 0; r < NT; ++r) o.p[r] = t.p[r];
  return o;
}

int ceil_div(int a, int b) { return (a + b - 1) / b; }

template <class F>
void by_type(bool half, F f) {
  if (half) f(TypeF16{});
  else f(TypeBf16{});
}
template <class F>
void by_tile(bool small, F f) {
  if (small) f(SmallTile{});
  else f(BigTile{});
}
template <class F>
void by_table(int tp, F f) {
  if (tp == 1) f(std::integral_constant<int, 1>{});
  else f(std::integral_constant<int, HG_MAX_TP>{});
}

}  // namespace

hipError_t launch_xent_pack(const XentPlan &p, const void *x, const void *labels, float *loss,
                            float *lse, hipStream_t s) {
  if (p.m <= kPackRows) {
    hipLaunchKernelGGL(k_pack_few, dim3(p.m), dim3(256), 0, s, p.r, labels, p.label_bytes, p.m,
                       p.vocab, p.ignore, static_cast<const u32x4 *>(x),
                       static_cast<u32x4 *>(p.xc), p.hidden >> 3, loss, lse);
    return hipGetLastError();
  }
  hipLaunchKernelGGL(k_pack, dim3(1), dim3(1024), 0, s, p.r, labels, p.label_bytes, p.m, p.vocab,
                     p.ignore, loss, lse);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_pack_rows, dim3(p.m < 2048 ? p.m : 2048), dim3(256), 0, s, p.r,
                     static_cast<const u32x4 *>(x), static_cast<u32x4 *>(p.xc), p.m, p.hidden >> 3);
  return hipGetLastError();
}

hipError_t launch_xent_logits(const XentPlan &p, const VocabMatrix &w, int mode, int v0, int cols,
                              hipStream_t s) {
  const int edge = p.small_logits ? SmallTile::kEdge : BigTile::kEdge;
  const int tm = ceil_div(p.m, edge), tn = ceil_div(cols, edge);
  const int vend = v0 + cols;
  by_type(p.half, [&](auto type) {
    by_table(w.tp, [&](auto nt) {
      by_tile(p.small_logits, [&](auto tile) {
        using T = decltype(type);
        using Tile = decltype(tile);
        constexpr int NT = decltype(nt)::value;
        auto go = [&](auto kernel) {
          hipLaunchKernelGGL(kernel, dim3(tm * tn), dim3(512), 0, s, p,
                             static_cast<const u32x4 *>(p.xc), small_table<NT>(w.t), w.shard, v0,
                             vend, tn);
        };
        if (mode == kStats) go(k_logits<T, Tile, NT, kStats>);
        else if (mode == kProb) go(k_logits<T, Tile, NT, kProb>);
        else go(k_logits<T, Tile, NT, kGrad>);
      });
    });
  });
  return hipGetLastError();
}

hipError_t launch_xent_score(const XentPlan &p, const VocabMatrix &w, const void *x,
                             const void *labels, float *loss, float *lse, hipStream_t s) {
  // One run per CU; runs of 129 to 256 rows become two of up to 128, which fill
  // their stages (13 rows at V = 44480, H = 3528: 74 us instead of 80).
  const int units = ceil_div(p.vocab, 16);
  int groups = units < kCus ? units : kCus;
  if (units > 8 * kCus && units <= 16 * kCus) groups = kScoreGroups;
  by_type(p.half, [&](auto type) {
    by_table(w.tp, [&](auto nt) {
      using T = decltype(type);
      constexpr int NT = decltype(nt)::value;
      auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3(groups), dim3(512), 0, s, p, static_cast<const u32x4 *>(x),
                           labels, small_table<NT>(w.t), w.shard);
      };
      auto by_rows = [&](auto chunks) {
        constexpr int KC = decltype(chunks)::value;
        if (p.m <= 16) go(k_score<T, NT, 1, KC>);
        else if (p.m <= 32) go(k_score<T, NT, 2, KC>);
        else if (p.m <= 64) go(k_score<T, NT, 4, KC>);
        else go(k_score<T, NT, 8, KC < 2 ? 1 : 2>);  // x of 128 rows and 256 k fills the LDS
      };
      const int run = ceil_div(units, groups) * 16;  // rows of a workgroup
      if (run > 128) by_rows(std::integral_constant<int, 1>{});
      else if (run > 64) by_rows(std::integral_constant<int, 2>{});
      else by_rows(std::integral_constant<int, 4>{});
    });
  });
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_score_join, dim3(p.m), dim3(64), 0, s, p, labels, groups, loss, lse);
  return hipGetLastError();
}

hipError_t launch_xent_join(const XentPlan &p, const float *grad, float *loss, float *lse,
                            hipStream_t s) {
  hipLaunchKernelGGL(k_join, dim3(ceil_div(p.m, 16)), dim3(256), 0, s, p, grad, loss, lse);
  return hipGetLastError();
}

hipError_t launch_xent_factors(const XentPlan &p, const float *lse, const float *grad,
                               hipStream_t s) {
  hipLaunchKernelGGL(k_factors, dim3(ceil_div(p.m, 256)), dim3(256), 0, s, p, lse, grad);
  return hipGetLastError();
}

hipError_t launch_xent_normalise(const XentPlan &p, hipStream_t s) {
  const int per = ceil_div(p.m, 8 * 16);  // 16 steps of 8 rows per workgroup
  const dim3 grid(p.piece / kPanel, per < 65535 ? per : 65535);
  by_type(p.half, [&](auto type) {
    hipLaunchKernelGGL(k_normalise<decltype(type)>, grid, dim3(256), 0, s, p);
  });
  return hipGetLastError();
}

hipError_t launch_xent_dx_join(const XentPlan &p, const VocabMatrix &w, void *dx, hipStream_t s) {
  const dim3 grid(ceil_div(p.hidden >> 2, 1024), p.m < 16384 ? p.m : 16384);
  by_type(p.half, [&](auto type) {
    by_table(w.tp, [&](auto nt) {
      constexpr int NT = decltype(nt)::value;
      hipLaunchKernelGGL((k_dx_join<decltype(type), NT>), grid, dim3(256), 0, s, p,
                         small_table<NT>(w.t), w.shard, static_cast<uint2 *>(dx));
    });
  });
  return hipGetLastError();
}

hipError_t launch_xent_join_normalise(const XentPlan &p, const float *grad, float *loss, float *lse,
                                      hipStream_t s) {
  const dim3 grid(p.piece / kPanel, ceil_div(p.m, 8));
  by_type(p.half, [&](auto type) {
    hipLaunchKernelGGL(k_join_normalise<decltype(type)>, grid, dim3(256), 0, s, p, grad, loss, lse);
  });
  return hipGetLastError();
}

hipError_t launch_xent_grads(const XentPlan &p, const VocabMatrix &w, int v0, int cols, bool first,
                             void *dw, bool wide, bool accumulate, hipStream_t s) {
  const int vend = v0 + cols;
  const int edge = p.small_grads ? SmallTile::kEdge : BigTile::kEdge;
  GradArgs a;
  a.v0 = v0;
  a.vend = vend;
  a.tn = ceil_div(p.hidden, edge);
  a.xgroups = p.dxp ? ceil_div(p.m, edge) * a.tn * p.split_dx : 0;
  a.per = ceil_div(ceil_div(cols, kStep), p.split_dx);
  a.first = first ? 1 : 0;
  a.wm = dw ? ceil_div(cols, edge) : 0;
  a.dw = dw;
  a.wide = wide ? 1 : 0;
  a.accumulate = accumulate ? 1 : 0;
  const dim3 grid(a.xgroups + a.wm * a.tn * p.split_dw);
  by_type(p.half, [&](auto type) {
    using T = decltype(type);
    by_table(w.tp, [&](auto nt) {
      constexpr int NT = decltype(nt)::value;
      by_tile(p.small_grads, [&](auto tile) {
        hipLaunchKernelGGL((k_grads<T, decltype(tile), NT>), grid, dim3(512), 0, s, p,
                           small_table<NT>(w.t), w.shard, a);
      });
    });
    if (dw && p.split_dw > 1) {
      const int rows = vend < p.vocab || accumulate ? cols : p.rows - v0;
      const long long quads = static_cast<long long>(rows) * (p.hidden >> 2);
      const long long want = (quads + 255) / 256;
      const dim3 g2(static_cast<unsigned>(want < 4096 ? want : 4096));
      hipLaunchKernelGGL((k_dw_join<T>), g2, dim3(256), 0, s, p, v0, cols, rows, dw, a.wide,
                         a.accumulate);
    }
  });
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !dw || p.split_dw > 1 || vend < p.vocab || accumulate) return e;
  // the matrix's rows past the tiles that the vocabulary ends in
  const int from = v0 + a.wm * edge;
  if (from >= p.rows) return hipSuccess;
  const size_t row_bytes = static_cast<size_t>(p.hidden) * (wide ? 4 : 2);
  return launch_zero(static_cast<char *>(dw) + from * row_bytes, (p.rows - from) * row_bytes, s);
}

}  // namespace hg
