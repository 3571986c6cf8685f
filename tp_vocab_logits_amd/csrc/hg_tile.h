// The 256 x 256 matrix-product tile of the vocabulary operators, on gfx950
// matrix cores: 16-bit operands, fp32 accumulation in registers.
//
// C[m][n] = sum_k A[m][k] B[n][k] for one 256 x 256 tile. Either operand may
// lie in memory with k contiguous in a row ("row" operands: [m][k]) or with k
// as the row index ("column" operands: [k][m]); the column form is turned
// while it is read from LDS (ds_read_b64_tr_b16), so no operand is ever
// transposed in memory.
//
// LDS: two stages of 64 k; a stage is eight 64 x 64 sub-tiles of 8 KB (four
// of A, four of B), 128 bytes per LDS row (a row is an m for a row operand, a
// k for a column operand). Sub-tiles arrive by buffer loads straight into LDS,
// 1 KB (8 LDS rows) per instruction; the lanes' global addresses carry the
// swizzle of the eight 16-byte chunks of a row that keeps the fragment reads
// off one another's banks:
//   row operand:    chunk ^ ((row >> 1) & 7); a fragment read takes 16
//                   consecutive rows at one chunk
//   column operand: chunk ^ 2*f(k), f(k) = bit 1 of k | bit 3 of k << 1; a
//                   transposed read takes 8 k rows (k0..k0+3 and k0+8..k0+11)
//                   at one pair of chunks
//
// Waves: 8, as 2 (m) x 4 (n); a wave owns 128 x 64 of C as 8 x 4 blocks of
// v_mfma_f32_16x16x32. The operands are given to the MFMA in the order (B, A),
// so a lane holds four consecutive n of one m: the epilogues store 8 or 16
// bytes at a time and reduce over n mostly inside the lane.
//
// Schedule: the two waves of a SIMD (w and w + 4) alternate between reading
// fragments and multiplying. A step of 64 k has two phases per wave -- the
// upper and the lower 64 rows of A, each against the wave's 64 columns of B --
// and each phase is a memory part (fragment reads, loads of later steps into
// sub-tiles whose last reader is done) and a part of 32 MFMAs, with a barrier
// after each. Waves 4-7 run one barrier behind, so that one wave of every SIMD
// multiplies while the other one reads.
//   memory part 1 of step k reads A's upper half and B, and loads A's lower
//   half of step k+1; part 2 reads A's lower half, and loads B and A's upper
//   half of step k+2. Each ends with vmcnt(8): everything but the newest eight
//   loads of the wave has landed, which is what the next part reads.
// Measured (4096 rows, V = 163840, H = 7168): logits 6.45 to 6.8 ms, 1.41 to
// 1.49 PFLOP/s, the matrix cores busy 83 % of the cycles at 1.63 to 1.7 GHz, the
// clock that the power limit leaves; the gradient's products (a column operand on
// one or both sides, the labels' residues included) 14.7 to 15.6 ms, 1.23 to 1.31
// PFLOP/s, busy 68 % at 1.73 GHz. The memory parts bound it: five wait states more
// per load cost 3 to 5 %. Not kept, measured the same or
// slower: a third stage of B (160 KB of LDS), B's reads spread over both parts,
// the loads spread over both parts (logits 5 % slower) or all in the second (6 %
// slower) or among the MFMAs (15 % slower), X turned in memory for dW, workgroups
// that stay and load ahead of their epilogue (3 % slower here, 2 % faster at
// H = 1024), no s_setprio (logits 1 % faster, gradients 1 % slower).
// Loads past the last step, past K or past an operand's rows lie beyond their
// buffer resource, which fills LDS with zeros without touching memory: the
// counts stay the same to the end and no operand needs padding.
#pragma once

#include "hg_internal.h"

namespace hg {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));

// The two 16-bit types: their product and their rounding (to nearest even).
struct TypeBf16 {
  using elt = __bf16;
  static __device__ __forceinline__ f32x4 mma(s16x8 a, s16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  }
  static constexpr bool kHalf = false;
};
struct TypeF16 {
  using elt = _Float16;
  static __device__ __forceinline__ f32x4 mma(s16x8 a, s16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  }
  static constexpr bool kHalf = true;
};

template <class T>
__device__ __forceinline__ uint32_t bits16(float f) {
  return __builtin_bit_cast(unsigned short, static_cast<typename T::elt>(f));
}
template <class T>
__device__ __forceinline__ float from16(uint32_t b) {
  return static_cast<float>(__builtin_bit_cast(typename T::elt, static_cast<unsigned short>(b)));
}

constexpr int kTile = 256;           // C tile edge (the small tile's is half of it)
constexpr int kStep = 64;            // k per step
constexpr int kChain = 16;           // steps that are summed before they join a total
constexpr int kSubBytes = 64 * 128;  // one 64 x 64 sub-tile
constexpr int kStageBytes = 8 * kSubBytes;
constexpr int kTileLds = 2 * kStageBytes;
constexpr unsigned kBeyond = 0x80000000u;  // an offset past every buffer resource used here
constexpr int kRawWord3 = 0x00020000;      // buffer resource word 3: raw 32-bit data

typedef uint32_t rsrc_t __attribute__((ext_vector_type(4)));

// Raw buffer resource of `bytes` bytes (none if negative) at a wave-uniform base.
__device__ __forceinline__ rsrc_t resource(const void *base, long long bytes) {
  const unsigned long long p = reinterpret_cast<unsigned long long>(base);
  return rsrc_t{static_cast<uint32_t>(p), static_cast<uint32_t>(p >> 32) & 0xFFFFu,
                static_cast<uint32_t>(bytes > 0 ? bytes : 0), kRawWord3};
}

// One load of 16 bytes per lane straight into LDS, at lds + 16*lane. Written
// as an instruction because the compiler, which knows that the builtin form
// writes LDS, waits for every load in flight (vmcnt(0)) before a transposed LDS
// read: the gradient's two products of 4096 rows at V = 163840, H = 7168 take
// 14.55 ms so and 14.78 with the builtin, of 8192 rows at V = 32768, H = 1024
// 781 us and 818. The load has no output register; its order against the LDS
// reads is kept by the waits and barriers of the products and by the memory
// clobber. What the compiler does not see it does not guard: the resource must
// come from scalar instructions (a vector instruction that writes a scalar
// register needs five wait states before this reads it), which
// tests/test_vocab_asm.py checks in the compiled kernels.
// STREAM: data that is read once (non-temporal).
template <bool STREAM = false>
__device__ __forceinline__ void load_lds(rsrc_t r, unsigned char *lds, unsigned offset) {
  const uint32_t at = static_cast<uint32_t>(
      reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) unsigned char *)lds));
  if constexpr (STREAM)
    __asm__ __volatile__(
        "s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen nt lds"
        :
        : "s"(at), "v"(offset), "s"(r)
        : "memory");
  else
    __asm__ __volatile__("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                         :
                         : "s"(at), "v"(offset), "s"(r)
                         : "memory");
}

// Lane constants of the loads: LDS row l >> 3 of the instruction's eight, slot
// l & 7; the chunk that belongs there, by the parity of the instruction.
struct LoadLane {
  int row;
  int chunk[2];
};
template <bool COLUMN>
__device__ __forceinline__ LoadLane load_lane(int lane) {
  LoadLane p;
  p.row = lane >> 3;
#pragma unroll
  for (int odd = 0; odd < 2; ++odd)
    p.chunk[odd] = COLUMN ? (lane & 7) ^ ((((lane >> 4) & 1) | (odd << 1)) << 1)
                          : (lane & 7) ^ ((odd << 2) | (lane >> 4));
  return p;
}

// Operand sources. load(lds, sub, q, step): instruction q (LDS rows 8q..8q+7)
// of sub-tile `sub` at step `step`.

// Row operand in panels of 256 k: row m of the tile at base + m*512 bytes,
// the k of panel i at base + i*panel; k counts from column `k0` (a multiple of
// 64), K a multiple of 8.
struct PanelRowSource {
  static constexpr bool kColumn = false;
  const unsigned char *base;
  long long panel;
  unsigned off[2];
  int chunk[2];
  int k8, s0, bytes;
  __device__ __forceinline__ void init(const void *base_, int rows, long long panel_bytes, int k0,
                                       int k_, int lane) {
    const LoadLane p = load_lane<false>(lane);
    base = static_cast<const unsigned char *>(base_);
    panel = panel_bytes;
    bytes = rows * 512;
    s0 = k0 >> 6;
    k8 = k_ >> 3;
#pragma unroll
    for (int o = 0; o < 2; ++o) {
      chunk[o] = p.chunk[o];
      off[o] = static_cast<unsigned>(p.row * 512 + p.chunk[o] * 16);
    }
  }
  __device__ __forceinline__ void load(unsigned char *lds, int sub, int q, int step) const {
    const int o = q & 1, s = s0 + step;
    const unsigned v = off[o] + static_cast<unsigned>((64 * sub + 8 * q) * 512 + (s & 3) * 128);
    load_lds(resource(base + (s >> 2) * panel, bytes), lds + q * 1024,
             step * 8 + chunk[o] < k8 ? v : kBeyond);
  }
};

// Row operand in rank blocks (NT table entries): tile row m is matrix row
// n0 + m. Blocks are a multiple of 32 rows, so eight rows share a block. A
// wave always loads the same L instructions of the same sub-tile, so it keeps
// one resource for each.
template <int NT, int L, bool STREAM = false>
struct RankRowSource {
  static constexpr bool kColumn = false;
  rsrc_t r[L];
  unsigned off[2];
  int chunk[2];
  int k8;
  __device__ __forceinline__ void init(const ShardTableN<NT> &w, int shard, int limit, int hidden,
                                       int n0, int sub, int q0, int lane) {
    const LoadLane p = load_lane<false>(lane);
    k8 = hidden >> 3;
#pragma unroll
    for (int o = 0; o < 2; ++o) {
      chunk[o] = p.chunk[o];
      off[o] = static_cast<unsigned>(p.row * hidden * 2 + p.chunk[o] * 16);
    }
#pragma unroll
    for (int t = 0; t < L; ++t) {
      const int n = n0 + 64 * sub + 8 * (q0 + t);
      const int left = limit - n;
      const int rank = NT == 1 || left <= 0 ? 0 : n / shard;
      const int at = left <= 0 ? 0 : n - rank * shard;
      const unsigned char *base = reinterpret_cast<const unsigned char *>(w.p[rank]) +
                                  static_cast<long long>(at) * hidden * 2;
      r[t] = resource(base, left <= 0 ? 0 : (left < 8 ? left : 8) * hidden * 2);
    }
  }
  __device__ __forceinline__ void load(unsigned char *lds, int, int q, int step) const {
    const int o = q & 1;
    const unsigned v = step * 8 + chunk[o] < k8 ? off[o] + static_cast<unsigned>(step * 128)
                                                : kBeyond;
    // A step's 128 bytes of a row are a cache line only if rows are whole lines;
    // of others the next step needs the rest of the line (13 rows at V = 44480,
    // H = 3528: 71.5 us instead of 74).
    if (STREAM && (k8 & 7) == 0)
      load_lds<true>(r[q & (L - 1)], lds + q * 1024, v);
    else
      load_lds(r[q & (L - 1)], lds + q * 1024, v);
  }
};

// Column operand in one panel, from its column `col` on: k row k at base +
// k*512 bytes; K rows.
struct PanelColumnSource {
  static constexpr bool kColumn = true;
  const unsigned char *base;
  unsigned off[2];
  int rows, col;
  __device__ __forceinline__ void init(const void *base_, int col_, int rows_, int lane) {
    const LoadLane p = load_lane<true>(lane);
    base = static_cast<const unsigned char *>(base_) + 2 * col_;
    col = col_;
    rows = rows_;
#pragma unroll
    for (int o = 0; o < 2; ++o) off[o] = static_cast<unsigned>(p.row * 512 + p.chunk[o] * 16);
  }
  __device__ __forceinline__ void load(unsigned char *lds, int sub, int q, int step) const {
    // Past the last row the resource is empty, wherever it points. (Without the
    // test of that and with one minimum for the length: 14.83 ms for the gradient's
    // products of 4096 rows at V = 163840, H = 7168, with them 15.06.)
    const int left = rows - step * 64;
    const rsrc_t r = resource(base + static_cast<long long>(step) * (64 * 512),
                              (left < 64 ? left : 64) * 512 - 2 * col);
    load_lds(r, lds + q * 1024, off[q & 1] + static_cast<unsigned>(8 * q * 512 + sub * 128));
  }
};

// Column operand in rank blocks: k row k is matrix row v0 + k (v0 a multiple
// of 8); rows from `limit` on read as zero.
template <int NT>
struct RankColumnSource {
  static constexpr bool kColumn = true;
  const ShardTableN<NT> *w;
  unsigned off[2];
  int shard, limit, v0, stride, col;
  __device__ __forceinline__ void init(const ShardTableN<NT> &w_, int shard_, int limit_, int v0_,
                                       int col_, int hidden, int lane) {
    const LoadLane p = load_lane<true>(lane);
    w = &w_;
    shard = shard_;
    limit = limit_;
    v0 = v0_;
    col = col_;
    stride = hidden * 2;
#pragma unroll
    for (int o = 0; o < 2; ++o) off[o] = static_cast<unsigned>(p.row * stride + p.chunk[o] * 16);
  }
  __device__ __forceinline__ void load(unsigned char *lds, int sub, int q, int step) const {
    // The resource ends with the block's (or the limit's) last row: counted
    // from this tile's columns it is 2*col short of whole rows. Reads past a
    // row's end belong to columns that no one stores.
    const unsigned v_off = off[q & 1] + static_cast<unsigned>(sub * 128);
    if constexpr (NT == 1) {  // one block: the step's 64 rows share a resource
      const int v = v0 + step * 64, left = limit - v;
      const int n = left > 64 ? 64 * stride : left * stride - 2 * col;
      const unsigned char *base = reinterpret_cast<const unsigned char *>(w->p[0]) +
                                  static_cast<long long>(left > 0 ? v : 0) * stride + 2 * col;
      load_lds(resource(base, left > 0 ? n : 0), lds + q * 1024,
               v_off + static_cast<unsigned>(8 * q * stride));
    } else {
      const int v = v0 + step * 64 + 8 * q;
      const int left = limit - v;
      const int rank = left <= 0 ? 0 : v / shard;
      const int at = left <= 0 ? 0 : v - rank * shard;
      const int n = left <= 0 ? 0 : (left < 8 ? left : 8) * stride - 2 * col;
      const unsigned char *base = reinterpret_cast<const unsigned char *>(w->p[rank]) +
                                  static_cast<long long>(at) * stride + 2 * col;
      load_lds(resource(base, n), lds + q * 1024, v_off);
    }
  }
};

// Fragment of a 16-row block: eight consecutive k (of the step's slice ks) of
// one row per lane.
template <bool COLUMN>
struct FragLane {
  int off[COLUMN ? 4 : 2];
  __device__ __forceinline__ void init(int lane) {
    const int i = lane & 15, g = lane >> 4;
    if constexpr (COLUMN) {
      const int f = (i >> 3) | ((g & 1) << 1);
#pragma unroll
      for (int b = 0; b < 4; ++b)
        off[b] = (g * 8 + (i >> 2)) * 128 + ((b ^ f) << 5) + (i & 3) * 8;
    } else {
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) off[ks] = i * 128 + (((ks * 4 + g) ^ (i >> 1)) << 4);
    }
  }
  __device__ __forceinline__ s16x8 read(const unsigned char *sub, int block, int ks) const {
    if constexpr (COLUMN) {
      typedef __attribute__((address_space(3))) s16x4 *lds4;
      const unsigned char *p = sub + off[block] + ks * 32 * 128;
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(p));
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(p + 4 * 128));
      return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    } else {
      return *reinterpret_cast<const s16x8 *>(sub + off[ks] + block * 16 * 128);
    }
  }
};

// s_waitcnt vmcnt(N) lgkmcnt(0) (N < 64).
template <int N>
__device__ __forceinline__ void wait_vm_lds() {
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | 0x70);
}

__device__ __forceinline__ void wait_lds() { __builtin_amdgcn_s_waitcnt(0xC07F); }  // lgkmcnt(0)

__device__ __forceinline__ void tile_barrier() {
  __asm__ __volatile__("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
  __asm__ __volatile__("" ::: "memory");
}

// The two tiles. acc[i][j][t] is row kRows*(wave >> 2) + 16*i + (lane & 15) and
// column kCols*(wave & 3) + 16*j + 4*(lane >> 4) + t. On return of product()
// every load has landed and every wave is past its last LDS read.
struct BigTile {
  static constexpr int kEdge = 256, MI = 8, NJ = 4, kRows = 128, kCols = 64;
  static constexpr int kBLoads = 4;  // B's load instructions per wave and step,
  static __device__ __forceinline__ int b_sub(int wave) { return wave & 3; }  // their sub-tile
  static __device__ __forceinline__ int b_first(int wave) { return 4 * (wave >> 2); }  // and first

  template <class T, class SA, class SB>
  static __device__ __forceinline__ void product(const SA &a, const SB &b, int steps,
                                               unsigned char *lds, f32x4 (&acc)[8][4]) {
    const int lane = static_cast<int>(threadIdx.x) & 63;
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
    const int wr = wave >> 2, wc = wave & 3;
    FragLane<SA::kColumn> fa;
    FragLane<SB::kColumn> fb;
    fa.init(lane);
    fb.init(lane);

    // A: each half (64 rows) of the wave's 128 is a sub-tile, loaded by the
    // four waves that read it; B: sub-tile wc, half of it per wave.
    auto load_a = [&](int half, int step) __attribute__((always_inline)) {
      const int sub = 2 * wr + half;
      unsigned char *st = lds + (step & 1) * kStageBytes + sub * kSubBytes;
      a.load(st, sub, 2 * wc, step);
      a.load(st, sub, 2 * wc + 1, step);
    };
    auto load_b = [&](int step) __attribute__((always_inline)) {
      unsigned char *st = lds + (step & 1) * kStageBytes + (4 + wc) * kSubBytes;
#pragma unroll
      for (int t = 0; t < 4; ++t) b.load(st, wc, 4 * wr + t, step);
    };

#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    load_b(0);
    load_a(0, 0);
    load_a(1, 0);
    load_b(1);
    load_a(0, 1);
    wait_vm_lds<8>();
    tile_barrier();
    if (wr == 1) tile_barrier();

    s16x8 ra[4][2], rb[4][2];
    auto multiply = [&](int half) __attribute__((always_inline)) {
      __builtin_amdgcn_s_setprio(1);
#pragma unroll
      for (int ks = 0; ks < 2; ++ks)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            acc[4 * half + i][j] = T::mma(rb[j][ks], ra[i][ks], acc[4 * half + i][j]);
      __builtin_amdgcn_s_setprio(0);
    };
    for (int kb = 0; kb < steps; ++kb) {
      const unsigned char *st = lds + (kb & 1) * kStageBytes;
      const unsigned char *sa = st + 2 * wr * kSubBytes;
      const unsigned char *sb = st + (4 + wc) * kSubBytes;
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
#pragma unroll
        for (int j = 0; j < 4; ++j) rb[j][ks] = fb.read(sb, j, ks);
#pragma unroll
        for (int i = 0; i < 4; ++i) ra[i][ks] = fa.read(sa, i, ks);
      }
      load_a(1, kb + 1);
      wait_vm_lds<8>();
      tile_barrier();
      multiply(0);
      tile_barrier();
#pragma unroll
      for (int ks = 0; ks < 2; ++ks)
#pragma unroll
        for (int i = 0; i < 4; ++i) ra[i][ks] = fa.read(sa + kSubBytes, i, ks);
      load_b(kb + 2);
      load_a(0, kb + 2);
      wait_vm_lds<8>();
      tile_barrier();
      multiply(1);
      tile_barrier();
    }
    if (wr == 0) tile_barrier();
    wait_vm_lds<0>();
    tile_barrier();
  }
};

// 128 x 128 for problems whose 256 x 256 tiles would leave CUs idle: a quarter
// of the work per tile, a ring of four 32 KB stages loaded three steps ahead
// and one barrier per step. 33 rows over V = 4096, H = 264 take 8.7 us for their
// logits on 32 small tiles and 16 us on 16 big ones. Long sums are taken in
// chains of kChain steps, each added to a total: an addition rounds at the size
// that the sum has by then. (The big tile has no registers for a total.)
struct SmallTile {
  static constexpr int kEdge = 128, MI = 4, NJ = 2, kRows = 64, kCols = 32;
  static constexpr int kBLoads = 2;
  static __device__ __forceinline__ int b_sub(int wave) { return wave >> 2; }
  static __device__ __forceinline__ int b_first(int wave) { return 2 * (wave & 3); }

  template <class T, class SA, class SB>
  static __device__ __forceinline__ void product(const SA &a, const SB &b, int steps,
                                                 unsigned char *lds, f32x4 (&acc)[4][2]) {
    constexpr int kBytes = 4 * kSubBytes;
    const int lane = static_cast<int>(threadIdx.x) & 63;
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
    const int wr = wave >> 2, wc = wave & 3;
    FragLane<SA::kColumn> fa;
    FragLane<SB::kColumn> fb;
    fa.init(lane);
    fb.init(lane);
    auto load = [&](int step) __attribute__((always_inline)) {
      unsigned char *st = lds + (step & 3) * kBytes + wr * kSubBytes;
#pragma unroll
      for (int t = 0; t < 2; ++t) a.load(st, wr, 2 * wc + t, step);
#pragma unroll
      for (int t = 0; t < 2; ++t) b.load(st + 2 * kSubBytes, wr, 2 * wc + t, step);
    };
    f32x4 chain[4][2];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[i][j] = chain[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < 3; ++s) load(s);
    for (int s = 0; s < steps; ++s) {
      wait_vm_lds<8>();
      tile_barrier();
      load(s + 3);
      const unsigned char *sa = lds + (s & 3) * kBytes + wr * kSubBytes;
      const unsigned char *sb = lds + (s & 3) * kBytes + (2 + (wc >> 1)) * kSubBytes;
      s16x8 ra[4], rb[2];
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        // block 2*(wc & 1) + j: the selection stays in the lane offsets
#pragma unroll
        for (int j = 0; j < 2; ++j) rb[j] = (wc & 1) ? fb.read(sb, 2 + j, ks) : fb.read(sb, j, ks);
#pragma unroll
        for (int i = 0; i < 4; ++i) ra[i] = fa.read(sa, i, ks);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j) chain[i][j] = T::mma(rb[j], ra[i], chain[i][j]);
      }
      if ((s + 1) % kChain == 0 || s + 1 == steps) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            acc[i][j] += chain[i][j];
            chain[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
          }
      }
    }
    wait_vm_lds<0>();
    tile_barrier();
  }
};

// The tile of workgroup `bid` of `groups`, out of tm x tn x tz: false if there
// is none left for it. Workgroups are dealt to the 8 XCDs in turn; each XCD
// takes a contiguous run of ids, which go through groups of 8 tile rows, columns
// inside a group, rows fastest, so that the workgroups in flight on an XCD share
// operands in its L2. `tm` may be the number of tile rows that the device found
// (rows that count), with workgroups launched for more: the ones left over are
// the last of each XCD. (Cut by the launched number, 1228 of 2047 rows at
// V = 32000, H = 2048 took 212 us for their logits instead of 172.)
__device__ __forceinline__ bool tile_at(int bid, int groups, int tm, int tn, int tz, int *z,
                                        int *mt, int *nt) {
  const int plane = tm * tn, total = plane * tz;
  const int n = groups < 8 ? groups : 8;
  const int xcd = bid % n, per = total / n, more = total % n;
  if (bid / n >= per + (xcd < more ? 1 : 0)) return false;
  int id = xcd * per + (xcd < more ? xcd : more) + bid / n;
  *z = id / plane;
  id -= *z * plane;
  const int group = id / (8 * tn);
  const int first = group * 8;
  const int gm = tm - first < 8 ? tm - first : 8;
  const int in = id - group * 8 * tn;
  *mt = first + in % gm;
  *nt = in / gm;
  return true;
}

}  // namespace hg
