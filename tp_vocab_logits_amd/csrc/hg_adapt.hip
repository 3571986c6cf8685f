// Low-rank adapters of many requests beside the shared head, and their gradients.
//
//   u_j = A_i x_j,  out_j = y_j + s_i B_i u_j            i = index[j]
//   g_j = s_i B_i^T dy_j,  dx_j = A_i^T g_j,  dA_i = sum_j g_j x_j^T,
//   dB_i = sum_j s_i dy_j u_j^T
//
// Everything with a side of the vocabulary's length is bound by HBM: y read and
// written, dy, B, dB. The products run on the matrix cores all the same
// (v_mfma_f32_16x16x32, tiles of 16 rows), so that nothing else comes near.
//
// Rows. A tile is 16 rows next to each other, sorted by adapter. A tile with rows of
// several adapters runs through each of them and every row takes its own one's
// result: no tile lists, y passes once whatever the mixture, and no value of one
// adapter (an infinity in its B) reaches the rows of another.
//
// Precision. u and g are fp32 sums that enter a second product of 16-bit operands.
// They enter as the sum of three 16-bit numbers, which hold all of fp32's 24 bits
// (bf16: 8 each, over the same exponents). For fp16 they are first scaled by a power
// of two that brings the largest of the row (out, dx) or of the adapter's rows (dA,
// dB) to 2^13 .. 2^14; what lies 2^-38 below it is lost. (Comparisons below of forms
// that were not kept were measured with two pieces, 2 to 4 % faster.)
#include <type_traits>

#include "hg_adapt.h"
#include "hg_tile.h"

namespace hg {

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ s16x8 load8(const unsigned short *p) {
  return *reinterpret_cast<const s16x8 *>(p);
}
__device__ __forceinline__ s16x8 stream8(const unsigned short *p) {  // read once
  return __builtin_nontemporal_load(reinterpret_cast<const s16x8 *>(p));
}
__device__ __forceinline__ s16x8 zero8() { return s16x8{0, 0, 0, 0, 0, 0, 0, 0}; }

// A power of two that brings `largest` to 2^13 .. 2^14 (1 for bf16, whose exponent
// needs none), and its inverse. (Both are normal for every exponent from 14 to 254;
// an infinity goes by the largest of them.)
__device__ __forceinline__ uint32_t exponent(float largest) {
  const uint32_t e = __builtin_bit_cast(uint32_t, largest) >> 23 & 255;
  return e < 14 ? 14 : e > 254 ? 254 : e;
}
template <class T>
__device__ __forceinline__ float to_range(float largest) {
  return T::kHalf ? __builtin_bit_cast(float, (267 - exponent(largest)) << 23) : 1.f;
}
template <class T>
__device__ __forceinline__ float from_range(float largest) {
  return T::kHalf ? __builtin_bit_cast(float, (exponent(largest) - 13) << 23) : 1.f;
}

// f as the sum of three, descending. Each takes what the ones before leave, which fp32
// holds exactly; an infinity or a NaN leaves nothing.
constexpr int kPieces = 3;
template <class T>
__device__ __forceinline__ void pieces(float f, uint32_t (&h)[kPieces]) {
  h[0] = bits16<T>(f);
  // (bf16: between its largest value and fp32's, a finite value rounds to infinity)
  if (!T::kHalf && (h[0] & 0x7FFF) == 0x7F80 && fabsf(f) < __builtin_inff()) --h[0];
#pragma unroll
  for (int k = 1; k < kPieces; ++k) {
    f -= from16<T>(h[k - 1]);
    h[k] = f == f ? bits16<T>(f) : 0u;
  }
}

// ---------------------------------------------------------------------------
// Few rows: u of one row, or a part of it, per workgroup. A lane holds 8 elements
// of x and meets them with those of each rank's row of A. The last workgroup sorts
// the rows by adapter meanwhile (up to 64: a lane each). Latency: 3.8 us for one row,
// 5.1 for 64 (hidden 7168, rank 16, 32 adapters).

struct RowArgs {
  const void *index;
  int index_bytes;
  const unsigned short *x, *a;
  int m, adapters, rank, hidden, splits;
  float *part;
  int *keys, *pos;
};

__device__ __forceinline__ int key_of_row(const RowArgs &r, int j) {
  const long long i = r.index_bytes == 8 ? static_cast<const long long *>(r.index)[j]
                                         : static_cast<const int *>(r.index)[j];
  return i >= 0 && i < r.adapters ? static_cast<int>(i) : r.adapters;
}

template <class T>
__global__ __launch_bounds__(kThreads) void k_adapt_row(RowArgs a) {
  const int lane = static_cast<int>(threadIdx.x) & 63;
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
  const int j = static_cast<int>(blockIdx.x) / a.splits, split = static_cast<int>(blockIdx.x) - j * a.splits;
  if (j == a.m) {
    if (wave > 0) return;
    const int key = lane < a.m ? key_of_row(a, lane) : 0x7FFFFFFF;
    int rank = 0;
#pragma unroll
    for (int o = 0; o < kFewRows; ++o) {
      const int other = __builtin_amdgcn_readlane(key, o);
      rank += other < key || (other == key && o < lane);
    }
    if (lane < a.m) {
      a.keys[rank] = key;
      a.pos[rank] = lane;
    }
    return;
  }
  const int i = key_of_row(a, j);
  if (i >= a.adapters) return;
  const unsigned short *const xr = a.x + static_cast<size_t>(j) * a.hidden;
  const unsigned short *const ai = a.a + static_cast<size_t>(i) * a.rank * a.hidden;
  float *const out = a.part + (static_cast<size_t>(split) * a.m + j) * a.rank;
  const int steps = (a.hidden + 511) / 512, from = steps * split / a.splits, to = steps * (split + 1) / a.splits;
  constexpr int kRows = 4;  // ranks at once per wave
  for (int r0 = wave * kRows; r0 < a.rank; r0 += 4 * kRows) {  // (rank is a multiple of 8)
    float sum[kRows] = {0.f, 0.f, 0.f, 0.f};
    for (int step = from; step < to; ++step) {
      const int k = step * 512 + lane * 8;
      if (k >= a.hidden) continue;
      const s16x8 xv = load8(xr + k);
      s16x8 av[kRows];
#pragma unroll
      for (int t = 0; t < kRows; ++t) av[t] = load8(ai + static_cast<size_t>(r0 + t) * a.hidden + k);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float f = from16<T>(static_cast<unsigned short>(xv[e]));
#pragma unroll
        for (int t = 0; t < kRows; ++t)
          sum[t] = __builtin_fmaf(f, from16<T>(static_cast<unsigned short>(av[t][e])), sum[t]);
      }
    }
#pragma unroll
    for (int t = 0; t < kRows; ++t) {
#pragma unroll
      for (int d = 32; d; d >>= 1) sum[t] += __shfl_xor(sum[t], d);
      if (lane == t) out[r0 + t] = sum[t];
    }
  }
}

// ---------------------------------------------------------------------------
// Loads straight into LDS (16 bytes per lane, at lds + 16 * lane), three stages deep,
// for the two kernels that stream the wide matrices. Written as an instruction
// because the compiler, which knows that the builtin form writes LDS, waits for
// every load in flight before it reads LDS; there is no output register, and the
// order against LDS reads is kept by the waits and barriers below. Each lane has
// an address of its own (rows are gathered); what lies outside is read from kZeros,
// so that every wave's count of loads is the same in every step.

__device__ __align__(16) unsigned char kZeros[16];

// PAST: past the caches, for a matrix that they cannot hold until it is read again
// (dy of 1.3 GB: 33 us of 657; dy of 131 MB: 6 of 87 more).
template <bool PAST = false>
__device__ __forceinline__ void async16(const void *src, unsigned char *lds) {
  const uint32_t at = static_cast<uint32_t>(
      reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) unsigned char *)lds));
  if constexpr (PAST)
    __asm__ __volatile__("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off nt"
                         :
                         : "s"(at), "v"(src)
                         : "memory");
  else
    __asm__ __volatile__("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
                         :
                         : "s"(at), "v"(src)
                         : "memory");
}
// The same for 4 bytes per lane.
__device__ __forceinline__ void async4(const void *src, unsigned char *lds) {
  const uint32_t at = static_cast<uint32_t>(
      reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) unsigned char *)lds));
  __asm__ __volatile__("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off"
                       :
                       : "s"(at), "v"(src)
                       : "memory");
}

constexpr int kStages = 3;
constexpr int kWaveBytes = 32 * 128;                   // 32 rows x 64 columns, or the like
constexpr int kStageAll = 4 * kWaveBytes + kSubBytes;  // four waves' and 8 KB that they share (or 2 KB each)

// The kernels of the second products hold low-rank values as well, 32 rows' a step
// in three pieces: 12 KB that the waves share, or 3 KB each up to 16 ranks. These
// come from the L2 and are loaded one step ahead only, the rows two steps: 72 KB and the
// rows' places leave two workgroups per CU, a third stage would leave one.
constexpr int kRowStage = 4 * kWaveBytes;
constexpr int kLowWave = 3 * 1024, kLowStage = 4 * kLowWave;
constexpr int kSecondLds = kStages * kRowStage + 2 * kLowStage;

// ---------------------------------------------------------------------------
// Low-rank products of many rows: part[split][p][rank] = sum over the split's
// columns of of[p][c] w_i[rank][c]. A workgroup has 128 rows (two tiles per wave), a
// part of the columns and up to 64 ranks (RB blocks of 16). Its waves share w's
// 64 columns of a step, so that w comes through the L2 once per 128 rows, half of
// what the rows themselves take; up to 16 ranks (2 KB) every wave loads its own
// and none waits for another. w's columns are next to each other in memory (A), or,
// if TURNED, its ranks are (B): those are turned while they are read from LDS.
//
// The workgroups of a split follow one another on one XCD, whose L2 then has w's
// part for all of them, and each begins at a place of its own in the split's columns:
// rows are a power of two times a small number apart, and at one column they would
// all be on a few of the memory's channels. 4096 rows of 163840 columns, rank 64, two
// adapters, gradients: 630 us with neither, 642 with the first alone, 627 with the
// second alone (a step apart), 606 with both. This kernel's part of it is 257 to 304
// us, 4.4 to 5.2 TB/s of dy: HBM bounds it; x, A and B come on top (a tenth: 1.48 GB in
// all are read past the L2).

struct LowSide {
  const unsigned short *of, *w;
  int blocks, shard, per_block, chunks;  // chunks of 64 columns per block, in all
  int splits;                            // 0: not wanted
  float *part;
};
struct LowArgs {
  const int *keys, *pos;
  int m, adapters, rank;
  int *head;     // [2][adapters], cleared for the join, or NULL
  LowSide x, y;  // u = A x, g = B^T dy
};

constexpr int kLowRows = 128;

template <class T, bool TURNED, int RB, bool PAST>
__device__ __forceinline__ void low_products(const LowArgs &a, const LowSide &s, int id, unsigned char *lds) {
  static_assert(RB == 1 || RB == 4);
  constexpr int TT = 2;
  const int lane = static_cast<int>(threadIdx.x) & 63;
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
  const int ml = lane & 15, g = lane >> 4;
  const int groups = (a.m + kLowRows - 1) / kLowRows;
  const int split = id / groups, group = id - split * groups;
  const int rc = static_cast<int>(blockIdx.y) * kRankChunk;
  const int ranks = a.rank - rc < RB * 16 ? a.rank - rc : RB * 16;  // a multiple of 8
  const int from = static_cast<int>(static_cast<long long>(s.chunks) * split / s.splits);
  const int to = static_cast<int>(static_cast<long long>(s.chunks) * (split + 1) / s.splits);
  const int p0 = group * kLowRows;
  // the rows that go through an adapter together: a wave's where none waits for another
  const int begin = RB == 1 ? p0 + wave * 32 : p0, most = begin + (RB == 1 ? 32 : kLowRows);
  const int pend = a.m < most ? a.m : most;
  if (begin >= a.m) return;
  const size_t columns = static_cast<size_t>(s.blocks) * s.shard;
  const LoadLane lr = load_lane<false>(lane), lc = load_lane<true>(lane);
  FragLane<false> fr;
  FragLane<true> fc;
  fr.init(lane);
  fc.init(lane);

  int key[TT];  // of the rows whose results this lane holds
#pragma unroll
  for (int t = 0; t < TT; ++t) {
    const int p = p0 + (wave * TT + t) * 16 + ml;
    key[t] = p < a.m ? a.keys[p] : a.adapters;
  }
  int lkey[4];  // of the rows that it loads
  const unsigned short *src[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int p = p0 + wave * 32 + 8 * q + lr.row;
    lkey[q] = p < a.m ? a.keys[p] : a.adapters;
    src[q] = s.of + static_cast<size_t>(p < a.m ? a.pos[p] : 0) * s.shard + lr.chunk[q & 1] * 8;
  }
  int at = begin;  // the first position of the adapter in turn
  int cur = __builtin_amdgcn_readfirstlane(a.keys[at]);
  while (cur < a.adapters) {
    bool active[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) active[t] = __ballot(key[t] == cur) != 0;
    f32x4 acc[TT][RB];
#pragma unroll
    for (int t = 0; t < TT; ++t)
#pragma unroll
      for (int b = 0; b < RB; ++b) acc[t][b] = f32x4{0.f, 0.f, 0.f, 0.f};
    const unsigned short *const wi = s.w + static_cast<size_t>(cur) * a.rank * columns;

    // six loads per wave and step
    auto issue = [&](int chunk, int stage) __attribute__((always_inline)) {
      const int block = chunk / s.per_block, c0 = (chunk - block * s.per_block) * 64;
      const int left = s.shard - c0;  // columns of the block from here on
      const size_t off = static_cast<size_t>(block) * a.m * s.shard + c0;
      const size_t col = static_cast<size_t>(block) * s.shard + c0;
      unsigned char *const st = lds + stage * kStageAll + wave * kWaveBytes;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const bool real = lkey[q] == cur && lr.chunk[q & 1] * 8 < left;
        async16<PAST>(real ? static_cast<const void *>(src[q] + off) : kZeros, st + q * 1024);
      }
      unsigned char *const sw = lds + stage * kStageAll + 4 * kWaveBytes + wave * 2048;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int q = RB == 1 ? t : 2 * wave + t;
        bool real;
        const unsigned short *p;
        if constexpr (!TURNED) {
          const int r = 8 * q + lr.row, c = lr.chunk[t] * 8;
          real = r < ranks && c < left;
          p = wi + static_cast<size_t>(rc + r) * columns + col + c;
        } else if constexpr (RB == 1) {  // lines of 16 ranks
          const int v = 32 * q + (lane >> 1), e = (lane & 1) * 8;
          real = v < left && e < ranks;
          p = wi + (col + v) * a.rank + e;
        } else {
          const int v = 8 * q + lc.row, e = lc.chunk[t] * 8;
          real = v < left && e < ranks;
          p = wi + (col + v) * a.rank + rc + e;
        }
        async16(real ? static_cast<const void *>(p) : kZeros, sw + t * 1024);
      }
    };
    auto multiply = [&](int stage) __attribute__((always_inline)) {
      const unsigned char *const st = lds + stage * kStageAll + wave * kWaveBytes;
      unsigned char *const sw = lds + stage * kStageAll + 4 * kWaveBytes + (RB == 1 ? wave * 2048 : 0);
      s16x8 xf[TT][2];
#pragma unroll
      for (int t = 0; t < TT; ++t)
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) xf[t][ks] = fr.read(st, t, ks);
#pragma unroll
      for (int ks = 0; ks < 2; ++ks)
#pragma unroll
        for (int b = 0; b < RB; ++b) {
          s16x8 wf;
          if constexpr (!TURNED) {
            wf = fr.read(sw, b, ks);
          } else if constexpr (RB == 1) {
            typedef __attribute__((address_space(3))) s16x4 *lds4;
            unsigned char *const q = sw + (ks * 32 + g * 8 + (ml >> 2)) * 32 + (ml & 3) * 8;
            const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(q));
            const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(q + 4 * 32));
            wf = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
          } else {
            wf = fc.read(sw, b, ks);
          }
#pragma unroll
          for (int t = 0; t < TT; ++t)
            if (active[t]) acc[t][b] = T::mma(wf, xf[t][ks], acc[t][b]);
        }
    };
    const int n = to - from;
    const int turn = static_cast<int>(static_cast<long long>(n) * group / groups);
    auto chunk_of = [&](int k) __attribute__((always_inline)) {
      k += turn;
      return from + (k < n ? k : k - n);
    };
    if (n > 0) issue(chunk_of(0), 0);
    if (n > 1) issue(chunk_of(1), 1);
    int stage = 0;
    for (int k = 0; k < n; ++k) {
      // this step has landed, and the last one's reads are done, here and (RB > 1) in
      // every wave
      if (k + 1 < n)
        wait_vm_lds<6>();
      else
        wait_vm_lds<0>();
      if constexpr (RB > 1)
        tile_barrier();
      else
        __asm__ __volatile__("" ::: "memory");
      if (k + 2 < n) issue(chunk_of(k + 2), stage >= 1 ? stage - 1 : kStages - 1);
      multiply(stage);
      stage = stage + 1 < kStages ? stage + 1 : 0;
    }
    wait_vm_lds<0>();
    if constexpr (RB > 1) tile_barrier();
#pragma unroll
    for (int t = 0; t < TT; ++t)
#pragma unroll
      for (int b = 0; b < RB; ++b) {
        const int r = b * 16 + 4 * g;
        if (key[t] == cur && r < ranks)
          *reinterpret_cast<f32x4 *>(
              s.part + (static_cast<size_t>(split) * a.m + p0 + (wave * TT + t) * 16 + ml) * a.rank + rc + r) =
              acc[t][b];
      }
    // the next adapter among the workgroup's rows (they are sorted)
    for (int same = 64; same == 64 && at < pend;) {
      const int p = at + lane;
      same = __popcll(__ballot(p < pend && a.keys[p < pend ? p : at] == cur));
      at += same;
    }
    cur = at < pend ? __builtin_amdgcn_readfirstlane(a.keys[at]) : a.adapters;
  }
}

// u's workgroups first (there are fewer), then g's.
template <class T, int RB, bool PAST>
__global__ __launch_bounds__(kThreads) void k_adapt_low(LowArgs a) {
  __shared__ __align__(1024) unsigned char lds[kStages * kStageAll];
  const int id = static_cast<int>(blockIdx.x);
  const int first = (a.m + kLowRows - 1) / kLowRows * a.x.splits;
  if (a.head && blockIdx.y == 0)
    for (int k = id * kThreads + static_cast<int>(threadIdx.x); k < 2 * a.adapters;
         k += static_cast<int>(gridDim.x) * kThreads)
      a.head[k] = 0;
  // consecutive workgroups go to the eight XCDs in turn: each XCD's are a run
  auto in_runs = [](int k, int all) __attribute__((always_inline)) {
    const int each = all / 8;
    return k < each * 8 ? k % 8 * each + k / 8 : k;
  };
  if (id < first)
    low_products<T, false, RB, false>(a, a.x, in_runs(id, first), lds);
  else
    low_products<T, true, RB, PAST>(a, a.y, in_runs(id - first, static_cast<int>(gridDim.x) - first), lds);
}

// ---------------------------------------------------------------------------
// A row's low-rank values: the parts' sum, scaled, as three 16-bit numbers each (fp16:
// brought to its range). PER threads next to each other share a row, each has TIMES
// times eight ranks.

template <class T, int PER, int TIMES>
__device__ __forceinline__ void low_values(const float *part, const float *scale, int key, int p, int sub,
                                           int m, int adapters, int rank, int splits,
                                           u32x4 (&low)[kPieces][TIMES], float &back) {
  float v[TIMES][8];
  float largest = 0.f;
  const float s = key < adapters && scale ? scale[key] : 1.f;
#pragma unroll
  for (int q = 0; q < TIMES; ++q) {
    const int e = (q * PER + sub) * 8;
#pragma unroll
    for (int t = 0; t < 8; ++t) v[q][t] = 0.f;
    if (key < adapters && e < rank) {
      for (int k0 = 0; k0 < splits; k0 += 4) {  // (eight loads in flight)
        f32x4 w[4][2];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (k0 + k < splits) {
            const f32x4 *const from =
                reinterpret_cast<const f32x4 *>(part + (static_cast<size_t>(k0 + k) * m + p) * rank + e);
            w[k][0] = from[0];
            w[k][1] = from[1];
          }
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (k0 + k < splits)
#pragma unroll
            for (int t = 0; t < 8; ++t) v[q][t] += w[k][t >> 2][t & 3];
      }
    }
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      v[q][t] *= s;
      largest = fmaxf(largest, fabsf(v[q][t]));
    }
  }
  if constexpr (T::kHalf) {
#pragma unroll
    for (int d = 1; d < PER; d <<= 1) largest = fmaxf(largest, __shfl_xor(largest, d));
  }
  const float factor = to_range<T>(largest);
  back = from_range<T>(largest);
#pragma unroll
  for (int q = 0; q < TIMES; ++q)
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      uint32_t a[kPieces], b[kPieces];
      pieces<T>(v[q][2 * t] * factor, a);
      pieces<T>(v[q][2 * t + 1] * factor, b);
#pragma unroll
      for (int h = 0; h < kPieces; ++h) low[h][q][t] = a[h] | b[h] << 16;
    }
}

// All rows' values by sorted position: [m][3][RANKS] (16 or 64 ranks, zeros past
// `rank`), and fp16's factors back. (2047 rows of 64 ranks in 28 parts: 7 us.)
template <class T, int RANKS>
__global__ __launch_bounds__(kThreads) void k_adapt_values(const float *part, const float *scale, const int *keys,
                                                           int m, int adapters, int rank, int splits,
                                                           unsigned short *low, float *back) {
  constexpr int kPer = RANKS / 8;
  const int tid = static_cast<int>(threadIdx.x);
  const int p = static_cast<int>(blockIdx.x) * (kThreads / kPer) + tid / kPer, sub = tid % kPer;
  if (p >= m) return;
  u32x4 v[kPieces][1];
  float inv;
  low_values<T, kPer, 1>(part, scale, keys[p], p, sub, m, adapters, rank, splits, v, inv);
  unsigned short *const row = low + static_cast<size_t>(p) * (kPieces * RANKS) + sub * 8;
#pragma unroll
  for (int h = 0; h < kPieces; ++h) *reinterpret_cast<u32x4 *>(row + h * RANKS) = v[h][0];
  if (T::kHalf && sub == 0) back[p] = inv;
}

// ---------------------------------------------------------------------------
// out = y + low W^T: W is [adapters][columns][rank]. A workgroup has a tile of 16
// rows and 64 columns for each of its four waves. A lane of a tile holds one row's
// 8 + 8 columns: the rows of W are dealt to the matrix cores' rows so that these are
// next to each other (stores of 64 bytes per row). For few rows, and for rows of
// many adapters. 64 rows of 32 adapters (V = 163840, rank 16): 36 to 38 us for 190 MB,
// 5.0 TB/s where a copy reaches 4.8, most of it W read once.

// acc += W's fragments x a row's values, given by read(piece, ks); BOTH: two pieces of
// up to 16 ranks are one fragment, the third one and zeros another.
template <class T, bool BOTH, int KF, class F>
__device__ __forceinline__ void add_low(f32x4 (&acc)[4], const s16x8 (&wf)[4][KF], F read) {
#pragma unroll
  for (int ks = 0; ks < KF; ++ks)
#pragma unroll
    for (int h = 0; h < (BOTH ? 2 : kPieces); ++h) {
      const s16x8 f = read(h, ks);
#pragma unroll
      for (int v = 0; v < 4; ++v) acc[v] = T::mma(wf[v][ks], f, acc[v]);
    }
}

// y + inv * res, eight of a row, rounded once.
template <class T>
__device__ __forceinline__ u32x4 sum8(s16x8 y, const f32x4 *res, float inv) {
  u32x4 o;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float f0 = __builtin_fmaf(res[e >> 1][(2 * e) & 3], inv, from16<T>(static_cast<unsigned short>(y[2 * e])));
    const float f1 =
        __builtin_fmaf(res[e >> 1][(2 * e + 1) & 3], inv, from16<T>(static_cast<unsigned short>(y[2 * e + 1])));
    o[e] = bits16<T>(f0) | bits16<T>(f1) << 16;
  }
  return o;
}

struct UpArgs {
  const int *keys, *pos;
  int by_row;  // the parts are in the caller's order of rows, not in the sorted one
  const float *part;
  const float *scale;
  const unsigned short *w, *y;
  unsigned short *out;
  int m, adapters, rank, splits;
  int blocks, shard, per_block, chunks;  // chunks of 64 columns per block, in all
  int first, groups, strips;             // groups of 16 rows of this launch, from `first` on
};

// RANKS: 16 (two pieces share one fragment), 64, or 256: in turns of 64.
// APART: as many adapters as tiles, or more, so that each tile is taken to have its own.
// (Which ones the rows use is on the device alone: rows of few adapters of a large bank
// pay for it. 2047 rows of 4 adapters, rank 64, V = 163840: 693 us in a bank of 32, where
// the tiles share, 880 of 256, apart; 335 of 4 in the form below. 64 rows of one adapter,
// rank 16: 23 us in a bank of 1, 25 of 256.)
template <class T, int RANKS, bool APART>
__global__ __launch_bounds__(kThreads) void k_adapt_up(UpArgs a) {
  constexpr bool kBoth = RANKS == 16;
  constexpr int kRow = kPieces * RANKS + 8;  // 16-bit elements of an LDS row, piece by piece
  constexpr int kTimes = RANKS == 256 ? 2 : 1;
  constexpr int KF = kBoth ? 1 : 2;
  constexpr int kBatch = kBoth ? 2 : 1;  // adapters whose fragments are loaded together
  __shared__ __align__(16) unsigned short low[16 * kRow];
  __shared__ float back[16];
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int ml = lane & 15, g = lane >> 4;
  // Tiles that share adapters: one strip's go to one XCD (workgroups are dealt to the
  // eight in turn) and find W's strip in its L2. Otherwise a tile's strips follow one
  // another, so that W is read in longer runs, and past the caches (64 rows of 32
  // adapters, V = 163840, rank 16: 43.5 us; through the caches 47.7, the other way 51).
  const int id = static_cast<int>(blockIdx.x);
  int strip, group;
  if constexpr (APART) {
    group = id / a.strips;
    strip = id - group * a.strips;
  } else {
    const int eight = id / (8 * a.groups), in = id - eight * 8 * a.groups;
    strip = eight * 8 + in % 8;
    group = in / 8;
  }
  if (strip >= a.strips) return;
  const int p0 = (a.first + group) * 16;
  const int p = p0 + ml;
  const int key = p < a.m ? a.keys[p] : -1;  // -1: no row
  const size_t row = static_cast<size_t>(p < a.m ? a.pos[p] : 0) * a.shard;
  const int chunk = strip * 4 + wave;
  const bool there = chunk < a.chunks;
  const int block = there ? chunk / a.per_block : 0, c0 = there ? (chunk - block * a.per_block) * 64 : 0;
  const int left = there ? a.shard - c0 : 0;
  const size_t at = static_cast<size_t>(block) * a.m * a.shard + c0;
  const unsigned short *const wcol = a.w + (static_cast<size_t>(block) * a.shard + c0) * a.rank;
  const size_t each = static_cast<size_t>(a.blocks) * a.shard * a.rank;

  // y and the first adapter's fragments are on their way before the low-rank values
  s16x8 yv[2];
#pragma unroll
  for (int h = 0; h < 2; ++h)
    yv[h] = a.y && key >= 0 && h * 32 + 8 * g < left ? load8(a.y + at + row + h * 32 + 8 * g) : zero8();
  s16x8 wf[kBatch][4][KF];
  int cur[kBatch];
  auto fragments = [&](int i, int rc, s16x8 (&w)[4][KF]) __attribute__((always_inline)) {
    const unsigned short *const wi = wcol + static_cast<size_t>(i) * each;
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int col = 32 * (v >> 1) + 8 * (ml >> 2) + 4 * (v & 1) + (ml & 3);
#pragma unroll
      for (int ks = 0; ks < KF; ++ks) {
        const int r = kBoth ? 8 * (g & 1) : rc + ks * 32 + 8 * g;
        const unsigned short *const from = wi + static_cast<size_t>(col) * a.rank + r;
        w[v][ks] = zero8();
        if (col < left && r < a.rank) w[v][ks] = APART ? stream8(from) : load8(from);
      }
    }
  };
  unsigned todo = static_cast<unsigned>(__ballot(key >= 0 && key < a.adapters)) & 0xFFFF;
  auto begin = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int n = 0; n < kBatch; ++n) {
      cur[n] = -1;
      if (todo) {
        cur[n] = __builtin_amdgcn_readlane(key, __builtin_ctz(todo));
        todo &= ~static_cast<unsigned>(__ballot(key == cur[n]));
        fragments(cur[n], 0, wf[n]);
      }
    }
  };
  begin();

  {
    const int r = tid / 16, sub = tid % 16, q0 = p0 + r;
    const int other = q0 < a.m ? a.keys[q0] : a.adapters;
    u32x4 v[kPieces][kTimes];
    float inv;
    low_values<T, 16, kTimes>(a.part, a.scale, other, a.by_row && q0 < a.m ? a.pos[q0] : q0, sub, a.m, a.adapters,
                              a.rank, a.splits, v, inv);
    if (sub == 0) back[r] = inv;
#pragma unroll
    for (int q = 0; q < kTimes; ++q) {
      const int e = (q * 16 + sub) * 8;
      if (e < RANKS) {
#pragma unroll
        for (int h = 0; h < kPieces; ++h) *reinterpret_cast<u32x4 *>(low + r * kRow + h * RANKS + e) = v[h][q];
      }
    }
  }
  __syncthreads();

  f32x4 res[4];
#pragma unroll
  for (int v = 0; v < 4; ++v) res[v] = f32x4{0.f, 0.f, 0.f, 0.f};
  const unsigned short *const mine = low + ml * kRow;
  while (cur[0] >= 0) {
#pragma unroll
    for (int n = 0; n < kBatch; ++n) {
      if (cur[n] < 0) break;
      f32x4 acc[4];
#pragma unroll
      for (int v = 0; v < 4; ++v) acc[v] = f32x4{0.f, 0.f, 0.f, 0.f};
      for (int rc = 0;;) {
        add_low<T, kBoth>(acc, wf[n], [&](int h, int ks) __attribute__((always_inline)) {
          if (kBoth && h == 1) return g < 2 ? load8(mine + 2 * RANKS + 8 * g) : zero8();
          return load8(mine + (kBoth ? 8 * g : h * RANKS + rc + ks * 32 + 8 * g));
        });
        rc += kRankChunk;
        if (RANKS <= kRankChunk || rc >= a.rank) break;
        fragments(cur[n], rc, wf[n]);
      }
      const bool take = key == cur[n];
#pragma unroll
      for (int v = 0; v < 4; ++v)
#pragma unroll
        for (int e = 0; e < 4; ++e) res[v][e] = take ? acc[v][e] : res[v][e];
    }
    begin();
  }
  const bool has = key < a.adapters;
  if (key < 0 || (a.y == a.out && !has)) return;
  const float inv = back[ml];
#pragma unroll
  for (int h = 0; h < 2; ++h)
    if (h * 32 + 8 * g < left)
      *reinterpret_cast<u32x4 *>(a.out + at + row + h * 32 + 8 * g) =
          has ? sum8<T>(yv[h], &res[2 * h], inv) : __builtin_bit_cast(u32x4, yv[h]);
}

// The same for many rows of few adapters: a workgroup keeps its 256 columns (64 per
// wave), and with them W's fragments, and goes through the rows, or a part of them,
// 32 at a time, y and the low-rank values loaded straight into LDS as above. The
// first form reads W's 8 KB for every 16 rows of 64 columns (2 KB); with 64 rows it
// still took 365 us; this one takes 312 to 340, 4.0 to 4.3 TB/s of y read and written,
// where a copy reaches 4.8 (2047 rows, V = 163840, rank 64). The form above has any rank:
// at 72, 2047 rows of 4 adapters take 964 us, at 64 in this form 335.

struct StreamArgs {
  const int *keys, *pos;
  const unsigned short *low, *w, *y;
  const float *back;
  unsigned short *out;
  int m, adapters, rank, blocks, shard, per_block, chunks;  // chunks of 64 columns
};

// RB: blocks of 16 ranks, 1 or 4.
template <class T, int RB, bool PAST>
__global__ __launch_bounds__(kThreads) void k_adapt_stream(StreamArgs a) {
  static_assert(RB == 1 || RB == 4);
  constexpr int KF = RB == 1 ? 1 : 2;
  constexpr int kPlaces = 4, kPlace = 512;          // per wave and step: places, keys, factors
  constexpr int kRowLoads = T::kHalf ? 6 : 5;       // per wave and step, places and factors among them
  __shared__ __align__(1024) unsigned char lds[kSecondLds + 4 * kPlaces * kPlace];
  unsigned char *const low_lds = lds + kStages * kRowStage;
  const int lane = static_cast<int>(threadIdx.x) & 63;
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
  const int ml = lane & 15, g = lane >> 4;
  const int chunk = static_cast<int>(blockIdx.x) * 4 + wave;
  const bool has = chunk < a.chunks;
  const int block = has ? chunk / a.per_block : 0, c0 = has ? (chunk - block * a.per_block) * 64 : 0;
  const int left = has ? a.shard - c0 : 0;
  const int steps = (a.m + 31) / 32;
  const int s0 = static_cast<int>(static_cast<long long>(steps) * blockIdx.y / gridDim.y);
  const int n = static_cast<int>(static_cast<long long>(steps) * (blockIdx.y + 1) / gridDim.y) - s0;
  const LoadLane lr = load_lane<false>(lane);
  FragLane<false> fr;
  fr.init(lane);
  const size_t at = static_cast<size_t>(block) * a.m * a.shard + c0;
  const unsigned short *const wcol = a.w + (static_cast<size_t>(block) * a.shard + c0) * a.rank;
  const size_t each = static_cast<size_t>(a.blocks) * a.shard * a.rank;
  unsigned char *const places = lds + kSecondLds + wave * kPlaces * kPlace;

  // the places and keys of step k's rows (positions past the last row: that one's)
  auto locate = [&](int k) __attribute__((always_inline)) {
    const int want = (s0 + k) * 32 + (lane & 31), p = want < a.m ? want : a.m - 1;
    unsigned char *const to = places + (k & (kPlaces - 1)) * kPlace;
    async4((lane < 32 ? a.pos : a.keys) + p, to);
    if constexpr (T::kHalf) async4(a.back + p, to + 256);
  };
  auto issue_rows = [&](int k, int stage) __attribute__((always_inline)) {
    locate(k + 2);
    const int p0 = (s0 + k) * 32;
    unsigned char *const st = lds + stage * kRowStage + wave * kWaveBytes;
    const int *const place = reinterpret_cast<const int *>(places + (k & (kPlaces - 1)) * kPlace);
    int row[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) row[q] = place[8 * q + lr.row];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int c = lr.chunk[q & 1] * 8;
      const bool real = a.y && p0 + 8 * q + lr.row < a.m && c < left;
      async16<PAST>(
          real ? static_cast<const void *>(a.y + at + static_cast<size_t>(row[q]) * a.shard + c) : kZeros,
          st + q * 1024);
    }
  };
  auto issue_low = [&](int k) __attribute__((always_inline)) {
    const int p0 = (s0 + k) * 32;
    unsigned char *const sl = low_lds + (k & 1) * kLowStage;
#pragma unroll
    for (int t = 0; t < kPieces; ++t) {
      int p, e;  // position, and 16-bit element of its values
      unsigned char *to;
      if constexpr (RB == 1) {
        to = sl + wave * kLowWave + t * 1024;
        if (t < 2) {  // 64 bytes a row, its four chunks swizzled by (row >> 2) & 3
          p = p0 + t * 16 + (lane >> 2);
          e = ((lane & 3) ^ (lane >> 4)) * 8;
        } else {  // the third piece's 32
          p = p0 + (lane >> 1);
          e = 32 + (lane & 1) * 8;
        }
      } else {  // 128 bytes of a row's piece, as an operand's row
        to = sl + t * 4096 + wave * 1024;
        p = p0 + wave * 8 + lr.row;
        e = t * kRankChunk + (wave & 1 ? lr.chunk[1] : lr.chunk[0]) * 8;
      }
      async16(p < a.m ? static_cast<const void *>(a.low + static_cast<size_t>(p) * (RB * 16 * kPieces) + e) : kZeros,
              to);
    }
  };
  if (n > 0) {
    locate(0);
    locate(1);
    wait_vm_lds<0>();
    __asm__ __volatile__("" ::: "memory");
    issue_rows(0, 0);
    issue_low(0);
  }
  if (n > 1) issue_rows(1, 1);
  int stage = 0, stored = 0;  // stores of the last step
  int have = -1;
  s16x8 wf[4][KF];
  for (int k = 0; k < n; ++k) {
    // Loads and stores share one counter and are counted off in order: the next step's
    // rows and the last step's stores may be under way.
    if (k + 1 >= n)
      wait_vm_lds<0>();
    else if (stored == 4)
      wait_vm_lds<kRowLoads + 4>();
    else
      wait_vm_lds<kRowLoads>();
    if constexpr (RB > 1)
      tile_barrier();
    else
      __asm__ __volatile__("" ::: "memory");
    // (the loads that issue_rows() starts overwrite this step's places)
    const int p0 = (s0 + k) * 32;
    int keys[2], rows[2];
    float factors[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int *const place = reinterpret_cast<const int *>(places + (k & (kPlaces - 1)) * kPlace) + t * 16 + ml;
      keys[t] = p0 + t * 16 + ml < a.m ? place[32] : -1;  // -1: no row
      rows[t] = place[0];
      factors[t] = T::kHalf ? __builtin_bit_cast(float, place[64]) : 1.f;
    }
    wait_lds();
    if (k + 1 < n) issue_low(k + 1);
    if (k + 2 < n) issue_rows(k + 2, stage >= 1 ? stage - 1 : kStages - 1);
    stored = 0;
    const unsigned char *const st = lds + stage * kRowStage + wave * kWaveBytes;
    const unsigned char *const sl = low_lds + (k & 1) * kLowStage + (RB == 1 ? wave * kLowWave : 0);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int key = keys[t];
      f32x4 res[4];
#pragma unroll
      for (int v = 0; v < 4; ++v) res[v] = f32x4{0.f, 0.f, 0.f, 0.f};
      unsigned todo = static_cast<unsigned>(__ballot(key >= 0 && key < a.adapters)) & 0xFFFF;
      while (todo) {
        const int cur = __builtin_amdgcn_readlane(key, __builtin_ctz(todo));
        todo &= ~static_cast<unsigned>(__ballot(key == cur));
        if (have != cur) {
          const unsigned short *const wi = wcol + static_cast<size_t>(cur) * each;
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            const int col = 32 * (v >> 1) + 8 * (ml >> 2) + 4 * (v & 1) + (ml & 3);
#pragma unroll
            for (int ks = 0; ks < KF; ++ks) {
              const int r = RB == 1 ? 8 * (g & 1) : ks * 32 + 8 * g;
              wf[v][ks] = col < left && r < a.rank ? load8(wi + static_cast<size_t>(col) * a.rank + r) : zero8();
            }
          }
          have = cur;
        }
        f32x4 acc[4];
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[v] = f32x4{0.f, 0.f, 0.f, 0.f};
        add_low<T, RB == 1>(acc, wf, [&](int h, int ks) __attribute__((always_inline)) {
          if constexpr (RB == 1) {
            const s16x8 f = *reinterpret_cast<const s16x8 *>(
                h == 0 ? sl + (t * 16 + ml) * 64 + ((g ^ (ml >> 2)) << 4) : sl + 2048 + (t * 16 + ml) * 32 + ((g & 1) << 4));
            return h == 0 || g < 2 ? f : zero8();
          } else {
            return fr.read(sl + h * 4096, t, ks);
          }
        });
        const bool take = key == cur;
#pragma unroll
        for (int v = 0; v < 4; ++v)
#pragma unroll
          for (int e = 0; e < 4; ++e) res[v][e] = take ? acc[v][e] : res[v][e];
      }
      const bool mine = key >= 0 && key < a.adapters;
      const bool writes = mine || (key >= 0 && a.y != a.out);
      if (__ballot(writes) == 0) continue;
      unsigned short *const to = a.out + at + static_cast<size_t>(rows[t]) * a.shard;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (h * 32 >= left) continue;
        const s16x8 yv = fr.read(st, t, h);
        const u32x4 o = mine ? sum8<T>(yv, &res[2 * h], factors[t]) : __builtin_bit_cast(u32x4, yv);
        if (writes && h * 32 + 8 * g < left) *reinterpret_cast<u32x4 *>(to + h * 32 + 8 * g) = o;
        ++stored;
      }
    }
    stage = stage + 1 < kStages ? stage + 1 : 0;
  }
}

// ---------------------------------------------------------------------------
// The gradients' small pieces.

// Four values' sums over the parts, [splits][n], at k.
__device__ __forceinline__ f32x4 sum_parts(const float *part, int splits, size_t n, size_t k) {
  f32x4 sum = {0.f, 0.f, 0.f, 0.f};
  for (int s0 = 0; s0 < splits; s0 += 8) {  // (eight loads in flight)
    f32x4 v[8];
#pragma unroll
    for (int t = 0; t < 8; ++t)
      if (s0 + t < splits) v[t] = *reinterpret_cast<const f32x4 *>(part + (s0 + t) * n + k);
#pragma unroll
    for (int t = 0; t < 8; ++t)
      if (s0 + t < splits) sum += v[t];
  }
  return sum;
}

// The parts' sums, scaled, and (fp16) the largest of each adapter's: blockIdx.y 0: u,
// 1: g. Four ranks of a row per thread.
struct JoinSide {
  const float *part;
  float *sum;
  int splits;  // 0: not wanted
};
template <class T>
__global__ __launch_bounds__(kThreads) void k_adapt_join(JoinSide u, JoinSide g, const int *keys,
                                                         const float *scale, int m, int adapters,
                                                         int rank, int *head) {
  const JoinSide side = blockIdx.y ? g : u;
  if (!side.splits) return;
  const size_t n = static_cast<size_t>(m) * rank;
  for (size_t k0 = static_cast<size_t>(blockIdx.x) * kThreads * 4; k0 < n;
       k0 += static_cast<size_t>(gridDim.x) * kThreads * 4) {
    const size_t k = k0 + threadIdx.x * 4;
    const int key = k < n ? keys[k / rank] : adapters;
    float largest = 0.f;
    f32x4 sum = {0.f, 0.f, 0.f, 0.f};
    if (key < adapters) {
      sum = sum_parts(side.part, side.splits, n, k);
      const float f = scale ? scale[key] : 1.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        sum[e] *= f;
        const float size = fabsf(sum[e]);
        if (size > largest && size < __builtin_inff()) largest = size;
      }
    }
    if (k < n) *reinterpret_cast<f32x4 *>(side.sum + k) = sum;
    if constexpr (T::kHalf) {
      // The largest of all does not depend on the order. Thousands of atomics on one
      // address took 25 us (4096 rows of 64 ranks, one adapter): a workgroup's
      // largest where it has one adapter, if it is more than what is there.
      __shared__ float tops[4];
      __shared__ int whose[4];  // adapters: none, or already done
      auto note = [&](int i, float top) __attribute__((always_inline)) {
        int *const to = head + static_cast<size_t>(blockIdx.y) * adapters + i;
        const int bits = static_cast<int>(__builtin_bit_cast(uint32_t, top));
        if (bits > __hip_atomic_load(to, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT)) atomicMax(to, bits);
      };
      const int first = __builtin_amdgcn_readfirstlane(key);  // (keys ascend, `adapters` comes last)
      const bool one = __ballot(key != first && key < adapters) == 0;
      if (one) {
#pragma unroll
        for (int d = 32; d; d >>= 1) largest = fmaxf(largest, __shfl_xor(largest, d));
      } else if (key < adapters) {
        note(key, largest);
      }
      if ((threadIdx.x & 63) == 0) {
        tops[threadIdx.x >> 6] = largest;
        whose[threadIdx.x >> 6] = one ? first : adapters;
      }
      __syncthreads();
      if (threadIdx.x < 4 && whose[threadIdx.x] < adapters) {
        const int w = static_cast<int>(threadIdx.x);
        bool last = true;
        float top = tops[w];
        for (int o = 0; o < 4; ++o)
          if (whose[o] == whose[w]) {
            top = fmaxf(top, tops[o]);
            if (o > w) last = false;
          }
        if (last) note(whose[w], top);
      }
      __syncthreads();
    }
  }
}

// low [m][rank] -> turned [3][rank][padded], piece by piece, zeros past m: 64 rows of 32
// ranks. fp16: one factor for all of an adapter's rows, by the largest of them, which the
// sums over them take back.
struct TurnSide {
  const float *part;  // JOIN: the parts, of which `splits`, and where their scaled sums
  int splits;         // go (or NULL)
  float *low;         // otherwise: those
  unsigned short *turned;  // (or NULL: the sums alone)
  unsigned short *rows;    // or NULL: the pieces by row as well, as k_adapt_values lays
  int of_row;              // them out for `of_row` ranks (JOIN, bf16)
  int *largest;            // [adapters]
};
struct TurnLds {
  float t[64][33];
  float of_row[64];
  int key[64];
};
// JOIN: the parts are added up here, a launch less than by k_adapt_join before it
// (gradients of 2047 rows of 32000 columns, 8 adapters: 80 us instead of 82; 33 rows of
// 4096: 32.6 instead of 34). fp16 knows its factors then only if the tile has all rows
// and ranks.
template <class T, bool JOIN>
__device__ __forceinline__ void turn_pieces(const TurnSide &s, const int *keys, const float *scale, int adapters, int m,
                                            int rank, int padded, int p0, int r0, TurnLds &l) {
  const int tid = static_cast<int>(threadIdx.x);
  if (tid < 64) l.key[tid] = p0 + tid < m ? keys[p0 + tid] : adapters;
  __syncthreads();
  for (int k = tid; k < 64 * 8; k += kThreads) {
    const int row = k / 8, e = k % 8 * 4, p = p0 + row, r = r0 + e, key = l.key[row];
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
    if (p < m && r < rank) {  // (four ranks are there or not)
      const size_t at = static_cast<size_t>(p) * rank + r;
      if constexpr (JOIN) {
        if (key < adapters) {
          v = sum_parts(s.part, s.splits, static_cast<size_t>(m) * rank, at);
          const float f = scale ? scale[key] : 1.f;
#pragma unroll
          for (int t = 0; t < 4; ++t) v[t] *= f;
        }
        if (s.low) *reinterpret_cast<f32x4 *>(s.low + at) = v;
      } else {
        v = *reinterpret_cast<const f32x4 *>(s.low + at);
      }
    }
#pragma unroll
    for (int t = 0; t < 4; ++t) l.t[row][e + t] = v[t];
  }
  __syncthreads();
  if constexpr (JOIN && !T::kHalf) {
    if (s.rows) {
      const int last = r0 + 32 >= rank ? s.of_row : r0 + 32, width = (last - r0) / 8;
      for (int k = tid; k < 64 * width; k += kThreads) {
        const int row = k / width, e = k % width * 8, p = p0 + row;
        if (p >= m) continue;
        u32x4 v[kPieces];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          uint32_t x[kPieces] = {}, y[kPieces] = {};
          if (e < 32) {
            pieces<T>(l.t[row][e + 2 * t], x);
            pieces<T>(l.t[row][e + 2 * t + 1], y);
          }
#pragma unroll
          for (int h = 0; h < kPieces; ++h) v[h][t] = x[h] | y[h] << 16;
        }
        unsigned short *const to = s.rows + static_cast<size_t>(p) * (kPieces * s.of_row) + r0 + e;
#pragma unroll
        for (int h = 0; h < kPieces; ++h) *reinterpret_cast<u32x4 *>(to + h * s.of_row) = v[h];
      }
    }
  }
  if (JOIN && !s.turned) return;
  if constexpr (T::kHalf) {
    if constexpr (JOIN) {
      if (tid < 64) {
        float top = 0.f;
        for (int e = 0; e < 32; ++e) {
          const float size = fabsf(l.t[tid][e]);
          if (size > top && size < __builtin_inff()) top = size;
        }
        l.of_row[tid] = top;
      }
      __syncthreads();
    }
    float top = 0.f;
    if (tid < 64) {
      const int key = l.key[tid];
      if constexpr (JOIN) {
        for (int o = 0; o < 64; ++o)
          if (l.key[o] == key) top = fmaxf(top, l.of_row[o]);
        if (key < adapters) s.largest[key] = static_cast<int>(__builtin_bit_cast(uint32_t, top));
      } else if (key < adapters) {
        top = __builtin_bit_cast(float, s.largest[key]);
      }
    }
    __syncthreads();
    if (tid < 64) l.of_row[tid] = to_range<T>(top);
    __syncthreads();
  }
  for (int k = tid; k < 64 * 32; k += kThreads) {
    const int p = p0 + k % 64, r = r0 + k / 64;
    if (p >= padded || r >= rank) continue;
    uint32_t v[kPieces];
    pieces<T>(T::kHalf ? l.t[k % 64][k / 64] * l.of_row[k % 64] : l.t[k % 64][k / 64], v);
#pragma unroll
    for (int h = 0; h < kPieces; ++h)
      s.turned[static_cast<size_t>(h * rank + r) * padded + p] = static_cast<unsigned short>(v[h]);
  }
}

// A [rank][hidden] -> [hidden][rank]: 64 x 64, 16 bytes at a time.
__device__ __forceinline__ void turn_block(const unsigned short *a, unsigned short *at, int rank, int hidden, int h0,
                                           int r0, unsigned short (&t)[64][72]) {
  for (int k = static_cast<int>(threadIdx.x); k < 64 * 8; k += kThreads) {
    const int r = r0 + k / 8, h = h0 + k % 8 * 8;
    if (r < rank && h < hidden)
      *reinterpret_cast<s16x8 *>(&t[k / 8][k % 8 * 8]) = load8(a + static_cast<size_t>(r) * hidden + h);
  }
  __syncthreads();
  for (int k = static_cast<int>(threadIdx.x); k < 64 * 8; k += kThreads) {
    const int h = h0 + k / 8, r = r0 + k % 8 * 8;
    if (r >= rank || h >= hidden) continue;
    s16x8 v;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = static_cast<short>(t[k % 8 * 8 + e][k / 8]);
    *reinterpret_cast<s16x8 *>(at + static_cast<size_t>(h) * rank + r) = v;
  }
}

// What the gradients' wide products take, in one launch: the pieces of u and g by
// rank, and A turned, for the adapters that have rows.
struct PrepareArgs {
  TurnSide u, g;
  unsigned short *at;
  const unsigned short *a;
  const int *seg, *keys;
  const float *scale;
  int m, rank, hidden, padded, adapters;
  int tiles, across, blocks;  // workgroups of one side's pieces, of which per rank chunk; of an adapter's A
  int first, second;          // workgroups before g's pieces, before A's
};
template <class T, bool JOIN>
__global__ __launch_bounds__(kThreads) void k_adapt_prepare(PrepareArgs a) {
  __shared__ union {
    TurnLds f;
    __align__(16) unsigned short h[64][72];
  } t;
  int id = static_cast<int>(blockIdx.x);
  if (id < a.second) {
    const bool g = id >= a.first;
    if (g) id -= a.first;
    turn_pieces<T, JOIN>(g ? a.g : a.u, a.keys, a.scale, a.adapters, a.m, a.rank, a.padded, id % a.across * 64,
                         id / a.across * 32, t.f);
  } else {
    id -= a.second;
    const int i = id / a.blocks, block = id - i * a.blocks, wide = (a.hidden + 63) / 64;
    if (a.seg[i] == a.seg[i + 1]) return;
    const size_t base = static_cast<size_t>(i) * a.rank * a.hidden;
    turn_block(a.a + base, a.at + base, a.rank, a.hidden, block % wide * 64, block / wide * 64, t.h);
  }
}

// ---------------------------------------------------------------------------
// Sums over an adapter's rows: out_i[rank][column] = sum_p low[p][rank] of[p][column]
// (dA, of = x), or turned, [column][rank] (dB, of = dy). A workgroup has one
// adapter, 64 columns for each of its four waves and up to 64 ranks, and goes
// through the rows, or a part of them, 32 at a time, as above: the waves share the
// rows' low-rank values (half of the bytes that their own columns take; up to 16
// ranks each loads its own), of is turned while it is read from LDS. The rows'
// places are loaded two steps before the rows. dB and dA of 4096 rows (V = 163840,
// hidden 7168, rank 64, two adapters): 305 to 330 us for 1.44 GB, 4.4 to 4.7 TB/s; 1336
// equal workgroups on 512 places are 2.6 rounds. Neighbouring columns on one XCD: 25 us
// slower. A fragment of the low-rank values, 16 lines of 64 bytes, is read in four cycles
// more than one without bank conflicts, 16.4 M cycles in all or 10 % of the LDS's time.

struct OuterSide {
  const int *largest;  // of each adapter's low-rank values (fp16)
  const unsigned short *of, *low;
  void *out;
  int blocks, shard, per_block, chunks;  // chunks of 64 columns
  int strips, parts;                     // 256 columns; parts of the rows (0: not wanted)
  int wide;                              // out is fp32, [parts][adapters]...
};
struct OuterArgs {
  const int *pos, *seg;
  int m, adapters, rank, padded;
  OuterSide y, x;  // dB, dA
};

template <class T, bool TURNED, int RB, bool PAST>
__device__ __forceinline__ void outer_products(const OuterArgs &a, const OuterSide &s, int id, unsigned char *lds) {
  static_assert(RB == 1 || RB == 4);
  constexpr int kPlaces = 4;  // steps' places at once, 256 bytes each, per wave
  const int lane = static_cast<int>(threadIdx.x) & 63;
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
  const int ml = lane & 15, g = lane >> 4;
  const int pair = id / s.strips;  // part and adapter
  const int part = pair / a.adapters, i = pair - part * a.adapters;
  const int rc = static_cast<int>(blockIdx.y) * kRankChunk;
  const int ranks = a.rank - rc < RB * 16 ? a.rank - rc : RB * 16;
  const int chunk = (id - pair * s.strips) * 4 + wave;
  const bool has = chunk < s.chunks;
  const int block = has ? chunk / s.per_block : 0, c0 = has ? (chunk - block * s.per_block) * 64 : 0;
  const int left = has ? s.shard - c0 : 0;
  const int from = a.seg[i], to = a.seg[i + 1];
  const int first = from & ~7;  // (low is read eight rows at a time)
  const int steps = (to - first + 31) / 32;
  const int s0 = static_cast<int>(static_cast<long long>(steps) * part / s.parts);
  const int n = static_cast<int>(static_cast<long long>(steps) * (part + 1) / s.parts) - s0;
  const LoadLane lc = load_lane<true>(lane);
  FragLane<true> fc;
  fc.init(lane);
  const unsigned short *const of = s.of + static_cast<size_t>(block) * a.m * s.shard + c0;
  unsigned char *const low_lds = lds + kStages * kRowStage;
  unsigned char *const places = lds + kSecondLds + wave * kPlaces * 256;
  f32x4 acc[RB][4];
#pragma unroll
  for (int b = 0; b < RB; ++b)
#pragma unroll
    for (int v = 0; v < 4; ++v) acc[b][v] = f32x4{0.f, 0.f, 0.f, 0.f};

  // the places of step k's rows (positions past the last row: that one's)
  auto locate = [&](int k) __attribute__((always_inline)) {
    const int p = first + (s0 + k) * 32 + (lane & 31);
    async4(a.pos + (p < a.m ? p : a.m - 1), places + (k & (kPlaces - 1)) * 256);
  };
  // five loads per wave and step
  auto issue_rows = [&](int k, int stage) __attribute__((always_inline)) {
    locate(k + 2);
    const int p0 = first + (s0 + k) * 32;
    unsigned char *const st = lds + stage * kRowStage + wave * kWaveBytes;
    const int *const place = reinterpret_cast<const int *>(places + (k & (kPlaces - 1)) * 256);
    int row[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) row[q] = place[8 * q + lc.row];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int p = p0 + 8 * q + lc.row, c = lc.chunk[q & 1] * 8;
      const bool real = p >= from && p < to && c < left;
      async16<PAST>(real ? static_cast<const void *>(of + static_cast<size_t>(row[q]) * s.shard + c) : kZeros,
                    st + q * 1024);
    }
  };
  // three: 16 ranks' 32 rows of each piece, a rank's four chunks swizzled by (rank >> 2) & 3
  auto issue_low = [&](int k) __attribute__((always_inline)) {
    const int p0 = first + (s0 + k) * 32;
    unsigned char *const sl = low_lds + (k & 1) * kLowStage + (RB == 1 ? wave * kLowWave : wave * 1024);
#pragma unroll
    for (int h = 0; h < kPieces; ++h) {
      const int r = (RB == 1 ? 0 : wave * 16) + (lane >> 2);
      const int p = p0 + ((lane & 3) ^ (lane >> 4)) * 8;
      const bool real = r < ranks && p < to;
      async16(real ? static_cast<const void *>(s.low + static_cast<size_t>(h * a.rank + rc + r) * a.padded + p) : kZeros,
              sl + h * (RB * 1024));
    }
  };
  auto multiply = [&](int k, int stage) __attribute__((always_inline)) {
    const int p0 = first + (s0 + k) * 32;
    const unsigned char *const st = lds + stage * kRowStage + wave * kWaveBytes;
    const unsigned char *const sl = low_lds + (k & 1) * kLowStage + (RB == 1 ? wave * kLowWave : 0);
    s16x8 lf[RB][kPieces];
#pragma unroll
    for (int b = 0; b < RB; ++b)
#pragma unroll
      for (int h = 0; h < kPieces; ++h) {
        const int line = h * (RB * 16) + b * 16 + ml;
        lf[b][h] = *reinterpret_cast<const s16x8 *>(sl + line * 64 + ((g ^ (ml >> 2)) << 4));
      }
    if (p0 < from || p0 + 32 > to) {  // rows of other adapters
      const int p = p0 + 8 * g;
#pragma unroll
      for (int b = 0; b < RB; ++b)
#pragma unroll
        for (int h = 0; h < kPieces; ++h)
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (p + e < from || p + e >= to) lf[b][h][e] = 0;
    }
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const s16x8 of8 = fc.read(st, v, 0);
#pragma unroll
      for (int b = 0; b < RB; ++b)
#pragma unroll
        for (int h = 0; h < kPieces; ++h)
          acc[b][v] = TURNED ? T::mma(lf[b][h], of8, acc[b][v]) : T::mma(of8, lf[b][h], acc[b][v]);
    }
  };
  if (n > 0) {
    locate(0);
    locate(1);
    wait_vm_lds<0>();
    __asm__ __volatile__("" ::: "memory");
    issue_rows(0, 0);
    issue_low(0);
  }
  if (n > 1) issue_rows(1, 1);
  int stage = 0;
  for (int k = 0; k < n; ++k) {
    if (k + 1 < n)  // the next step's rows may be under way
      wait_vm_lds<5>();
    else
      wait_vm_lds<0>();
    if constexpr (RB > 1)
      tile_barrier();
    else
      __asm__ __volatile__("" ::: "memory");
    if (k + 1 < n) issue_low(k + 1);
    if (k + 2 < n) issue_rows(k + 2, stage >= 1 ? stage - 1 : kStages - 1);
    multiply(k, stage);
    stage = stage + 1 < kStages ? stage + 1 : 0;
  }
  const float inv = T::kHalf ? from_range<T>(__builtin_bit_cast(float, s.largest[i])) : 1.f;
  const size_t columns = static_cast<size_t>(s.blocks) * s.shard;
  const size_t col0 = static_cast<size_t>(block) * s.shard + c0;
#pragma unroll
  for (int b = 0; b < RB; ++b)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const f32x4 sum = acc[b][v] * inv;
      size_t at;
      if constexpr (TURNED) {  // column v*16 + ml, ranks b*16 + 4g ..
        if (v * 16 + ml >= left || b * 16 + 4 * g >= ranks) continue;
        at = (static_cast<size_t>(pair) * columns + col0 + v * 16 + ml) * a.rank + rc + b * 16 + 4 * g;
      } else {  // rank b*16 + ml, columns v*16 + 4g ..
        if (b * 16 + ml >= ranks || v * 16 + 4 * g >= left) continue;
        at = (static_cast<size_t>(pair) * a.rank + rc + b * 16 + ml) * columns + col0 + v * 16 + 4 * g;
      }
      if (s.wide) {
        *reinterpret_cast<f32x4 *>(static_cast<float *>(s.out) + at) = sum;
      } else {
        typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
        *reinterpret_cast<u32x2 *>(static_cast<unsigned short *>(s.out) + at) =
            u32x2{bits16<T>(sum[0]) | bits16<T>(sum[1]) << 16, bits16<T>(sum[2]) | bits16<T>(sum[3]) << 16};
      }
    }
}

// dB's workgroups first, then dA's.
template <class T, int RB, bool PAST>
__global__ __launch_bounds__(kThreads) void k_adapt_outer(OuterArgs a) {
  __shared__ __align__(1024) unsigned char lds[kSecondLds + 4 * 4 * 256];
  const int id = static_cast<int>(blockIdx.x), first = a.y.strips * a.y.parts * a.adapters;
  if (id < first)
    outer_products<T, true, RB, PAST>(a, a.y, id, lds);
  else
    outer_products<T, false, RB, false>(a, a.x, id - first, lds);
}

// out = the sum of the parts, [n] each, n a multiple of 8.
template <class T, bool WIDE>
__global__ __launch_bounds__(kThreads) void k_adapt_parts(const float *part, int parts, size_t n, void *out) {
  for (size_t k = (static_cast<size_t>(blockIdx.x) * kThreads + threadIdx.x) * 8; k < n;
       k += static_cast<size_t>(gridDim.x) * kThreads * 8) {
    f32x4 sum[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
    for (int p0 = 0; p0 < parts; p0 += 4) {  // (eight loads in flight)
      f32x4 v[4][2];
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (p0 + t < parts) v[t][h] = *reinterpret_cast<const f32x4 *>(part + (p0 + t) * n + k + 4 * h);
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (p0 + t < parts) sum[h] += v[t][h];
    }
    if constexpr (WIDE) {
      f32x4 *const o = reinterpret_cast<f32x4 *>(static_cast<float *>(out) + k);
      o[0] = sum[0];
      o[1] = sum[1];
    } else {
      u32x4 o;
#pragma unroll
      for (int t = 0; t < 4; ++t)
        o[t] = bits16<T>(sum[t >> 1][2 * (t & 1)]) | bits16<T>(sum[t >> 1][2 * (t & 1) + 1]) << 16;
      *reinterpret_cast<u32x4 *>(static_cast<unsigned short *>(out) + k) = o;
    }
  }
}

template <int V>
using Int = std::integral_constant<int, V>;

template <class F>
void by_type(bool half, F f) {
  half ? f(TypeF16{}) : f(TypeBf16{});
}
// f(blocks of 16 ranks held at once, whether a matrix of m rows is read past the
// caches: more than the 256 MB of the memory-side one).
template <class F>
void by_size(int rank, int m, const Blocked &of, F f) {
  const bool past = of.p && 2ll * m * of.blocks * of.shard > (256ll << 20);
  if (rank <= 16)
    past ? f(Int<1>{}, Int<1>{}) : f(Int<1>{}, Int<0>{});
  else
    past ? f(Int<4>{}, Int<1>{}) : f(Int<4>{}, Int<0>{});
}

int ceil_div(long long a, long long b) { return static_cast<int>((a + b - 1) / b); }

constexpr int kMaxGroups = 1 << 23;  // workgroups of a launch

}  // namespace

int adapt_splits(int m, int blocks, int shard, int rank, bool few) {
  if (few) {  // k_adapt_row: steps of 512 columns, about 256 workgroups
    const int steps = ceil_div(shard, 512), want = 256 / m;
    return want < 1 ? 1 : want < steps ? want : steps;
  }
  // k_adapt_low: about 512 workgroups (two per CU), at least four steps each
  const long long groups = ceil_div(m, kLowRows) * static_cast<long long>(ceil_div(rank, kRankChunk));
  const int chunks = blocks * ceil_div(shard, 64);
  long long s = 512 / groups;
  if (s > chunks / 4) s = chunks / 4;
  if (s > 64) s = 64;
  return s < 1 ? 1 : static_cast<int>(s);
}

int adapt_parts(int m, int adapters, int blocks, int shard, int rank) {
  // k_adapt_outer: about 1024 workgroups, of at least eight steps of rows
  const long long have = static_cast<long long>(ceil_div(static_cast<long long>(blocks) * ceil_div(shard, 64), 4)) *
                         adapters * ceil_div(rank, kRankChunk);
  long long s = 1024 / have;
  const long long steps = m / (32ll * adapters);
  if (s > steps / 8) s = steps / 8;
  return s < 1 ? 1 : static_cast<int>(s);
}

hipError_t launch_adapt_low(const AdaptPlan &p, const AdaptRows &r, const Blocked &x, const void *a,
                            const Blocked &y, const void *b, hipStream_t s) {
  const auto *xp = static_cast<const unsigned short *>(x.p), *ap = static_cast<const unsigned short *>(a);
  if (p.few) {
    const RowArgs args{r.index, r.index_bytes, xp, ap, p.m, p.adapters, p.rank, x.shard, p.split_u, p.pu,
                       p.few_keys, p.few_keys + kFewRows};
    by_type(p.half, [&](auto type) {
      hipLaunchKernelGGL((k_adapt_row<decltype(type)>), dim3(p.m * p.split_u + 1), dim3(kThreads), 0, s, args);
    });
    return hipGetLastError();
  }
  auto side = [&](const Blocked &of, const void *w, int splits, float *part) {
    const int per = ceil_div(of.shard, 64);
    return LowSide{static_cast<const unsigned short *>(of.p), static_cast<const unsigned short *>(w), of.blocks,
                   of.shard, per, per * of.blocks, of.p ? splits : 0, part};
  };
  const LowArgs args{r.keys, r.pos, p.m, p.adapters, p.rank, p.head, side(x, a, p.split_u, p.pu), side(y, b, p.split_g, p.pg)};
  const dim3 grid(static_cast<unsigned>(ceil_div(p.m, kLowRows)) * (args.x.splits + args.y.splits),
                  ceil_div(p.rank, kRankChunk));
  by_type(p.half, [&](auto type) {
    by_size(p.rank, p.m, y, [&](auto rb, auto past) {
      hipLaunchKernelGGL((k_adapt_low<decltype(type), decltype(rb)::value, decltype(past)::value != 0>), grid,
                         dim3(kThreads), 0, s, args);
    });
  });
  return hipGetLastError();
}

hipError_t launch_adapt_up(const AdaptPlan &p, const AdaptRows &r, const float *part, int splits,
                           const float *scale, const void *w, const Blocked &y, void *out,
                           hipStream_t s) {
  const int per = ceil_div(y.shard, 64), chunks = per * y.blocks;
  const auto *wp = static_cast<const unsigned short *>(w), *yp = static_cast<const unsigned short *>(y.p);
  auto *op = static_cast<unsigned short *>(out);
  by_type(p.half, [&](auto type) {
    using T = decltype(type);
    if (adapt_streams(p.m, p.adapters, p.rank)) {
      by_size(p.rank, p.m, y, [&](auto rb, auto past) {
        constexpr int RB = decltype(rb)::value;
        if (part)
          hipLaunchKernelGGL((k_adapt_values<T, RB * 16>), dim3(ceil_div(p.m, kThreads / (RB * 2))), dim3(kThreads), 0,
                             s, part, scale, r.keys, p.m, p.adapters, p.rank, splits, p.low, p.back);
        const StreamArgs a{r.keys, r.pos, p.low, wp, yp, p.back, op, p.m, p.adapters, p.rank, y.blocks, y.shard, per,
                           chunks};
        // about 2048 workgroups, four rounds of two per CU, of two steps at least (2047 rows,
        // V = 163840: 335 us; 1024 of them 362, 5100 349; with two pieces)
        const int strips = ceil_div(chunks, 4), most = ceil_div(p.m, 64), want = ceil_div(2048, strips);
        hipLaunchKernelGGL((k_adapt_stream<T, RB, decltype(past)::value != 0>),
                           dim3(strips, want < most ? want : most), dim3(kThreads), 0, s, a);
      });
    } else {
      const int groups = ceil_div(p.m, 16), strips = ceil_div(chunks, 4);
      UpArgs a{r.keys, r.pos, p.few, part, scale, wp, yp, op, p.m, p.adapters, p.rank, splits, y.blocks,
               y.shard, per, chunks, 0, groups, strips};
      // (a launch has fewer than 2^32 lanes: 212000 rows of 163840 columns are two)
      const int most = kMaxGroups / (strips + 8);
      auto go = [&](auto ranks) {
        for (; a.first < groups; a.first += most) {
          a.groups = groups - a.first < most ? groups - a.first : most;
          if (p.adapters >= groups)
            hipLaunchKernelGGL((k_adapt_up<T, decltype(ranks)::value, true>),
                               dim3(static_cast<unsigned>(strips) * a.groups), dim3(kThreads), 0, s, a);
          else
            hipLaunchKernelGGL((k_adapt_up<T, decltype(ranks)::value, false>),
                               dim3(static_cast<unsigned>(ceil_div(strips, 8)) * 8 * a.groups), dim3(kThreads), 0, s, a);
        }
      };
      p.rank <= 16 ? go(Int<16>{}) : p.rank <= kRankChunk ? go(Int<kRankChunk>{}) : go(Int<HG_MAX_RANK>{});
    }
  });
  return hipGetLastError();
}

hipError_t launch_adapt_join(const AdaptPlan &p, const AdaptRows &r, const float *scale, hipStream_t s) {
  const int want = ceil_div(static_cast<long long>(p.m) * p.rank, 4 * kThreads);
  const dim3 grid(want < 1024 ? want : 1024, p.g ? 2 : 1);
  const JoinSide u{p.pu, p.u, p.u ? p.split_u : 0}, g{p.pg, p.g, p.g ? p.split_g : 0};
  by_type(p.half && p.head, [&](auto type) {
    hipLaunchKernelGGL((k_adapt_join<decltype(type)>), grid, dim3(kThreads), 0, s, u, g, r.keys, scale, p.m, p.adapters,
                       p.rank, p.head);
  });
  return hipGetLastError();
}

hipError_t launch_adapt_prepare(const AdaptPlan &p, const AdaptRows &r, const float *scale, const void *a,
                                hipStream_t s) {
  const bool join = !p.half || (p.padded <= 64 && p.rank <= 32);
  if (!join) {
    const hipError_t e = launch_adapt_join(p, r, scale, s);
    if (e != hipSuccess) return e;
  }
  PrepareArgs args{};
  // (u itself goes nowhere else, g to dx)
  const bool rows = adapt_prepares_rows(p);
  args.u = TurnSide{p.pu, p.split_u, join ? nullptr : p.u, p.ut, nullptr, 0, p.head};
  args.g = TurnSide{p.pg, p.split_g, join && (rows || !p.at) ? nullptr : p.g, p.gt, rows ? p.low : nullptr,
                    p.rank <= 16 ? 16 : kRankChunk, p.half ? p.head + p.adapters : nullptr};
  args.at = p.at;
  args.a = static_cast<const unsigned short *>(a);
  args.seg = p.seg;
  args.keys = r.keys;
  args.scale = scale;
  args.m = p.m;
  args.rank = p.rank;
  args.hidden = p.hidden;
  args.padded = p.padded;
  args.adapters = p.adapters;
  args.across = ceil_div(p.padded, 64);
  args.tiles = args.across * ceil_div(p.rank, 32);
  args.blocks = ceil_div(p.hidden, 64) * ceil_div(p.rank, 64);
  args.first = p.ut ? args.tiles : 0;
  args.second = args.first + (p.gt || (join && p.g) ? args.tiles : 0);
  const int all = args.second + (p.at ? args.blocks * p.adapters : 0);
  by_type(p.half, [&](auto type) {
    using T = decltype(type);
    if (join)
      hipLaunchKernelGGL((k_adapt_prepare<T, true>), dim3(all), dim3(kThreads), 0, s, args);
    else
      hipLaunchKernelGGL((k_adapt_prepare<T, false>), dim3(all), dim3(kThreads), 0, s, args);
  });
  return hipGetLastError();
}

hipError_t launch_adapt_outer(const AdaptPlan &p, const AdaptRows &r, const Blocked &x, void *da, const Blocked &y,
                              void *db, bool wide, hipStream_t s) {
  auto side = [&](const Blocked &of, const int *largest, const unsigned short *low, int parts, float *part, void *out) {
    const int per = ceil_div(of.shard, 64), chunks = per * of.blocks;
    return OuterSide{largest, static_cast<const unsigned short *>(of.p), low, parts > 1 ? part : out, of.blocks,
                     of.shard, per, chunks, ceil_div(chunks, 4), out ? parts : 0, wide || parts > 1};
  };
  const OuterArgs a{r.pos, p.seg, p.m, p.adapters, p.rank, p.padded, side(y, p.head, p.ut, p.parts_b, p.pb, db),
                    side(x, p.head + p.adapters, p.gt, p.parts_a, p.pa, da)};
  const dim3 grid(static_cast<unsigned>(a.y.strips * a.y.parts + a.x.strips * a.x.parts) * p.adapters,
                  ceil_div(p.rank, kRankChunk));
  by_type(p.half, [&](auto type) {
    using T = decltype(type);
    by_size(p.rank, p.m, y, [&](auto rb, auto past) {
      hipLaunchKernelGGL((k_adapt_outer<T, decltype(rb)::value, decltype(past)::value != 0>), grid, dim3(kThreads), 0, s,
                         a);
    });
    auto sum = [&](const Blocked &of, int parts, const float *part, void *out) {
      if (!out || parts == 1) return;
      const size_t n = static_cast<size_t>(p.adapters) * p.rank * of.blocks * of.shard;
      const int want = ceil_div(static_cast<long long>(n), 8 * kThreads);
      const dim3 sums(want < 2048 ? want : 2048);
      if (wide)
        hipLaunchKernelGGL((k_adapt_parts<T, true>), sums, dim3(kThreads), 0, s, part, parts, n, out);
      else
        hipLaunchKernelGGL((k_adapt_parts<T, false>), sums, dim3(kThreads), 0, s, part, parts, n, out);
    };
    sum(y, p.parts_b, p.pb, db);
    sum(x, p.parts_a, p.pa, da);
  });
  return hipGetLastError();
}

}  // namespace hg
