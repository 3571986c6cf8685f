// The embedding lookup with scaling, and its gradient by sorted tokens.
//
//   out_j = scale * W[t_j]                 (0 where t_j lies outside W)
//   dW_v  = scale * sum over j with t_j = v of dy_j
//
// Both move rows and hardly compute: HBM bounds them, latency the small ones.
//
// The gradient sorts the (token, position) pairs by token, stably, so that
// every sum runs over its positions in increasing order and repeated calls
// give the same bits. The sort is a radix sort, least significant digit first,
// of 9 bits a pass (two passes up to 2^18 entries, the smallest number that
// covers a large vocabulary): one workgroup in LDS while its 4096-key tile
// holds all tokens, one launch each for counts, offsets and scatter beyond.
// The sorted run is then cut into blocks of equally many positions, whatever
// their tokens: a frequent token's sum is spread over many workgroups. A sum
// inside one block is written at once; one that crosses a block's edge leaves
// fp32 partial rows, joined in order by a second launch. The whole gradient is
// first filled with zeros, beside the sort and in its launches; rows that get a
// sum are written twice. (65536 tokens of 2048 columns into 163840 rows: 240 us,
// 140 of them fill and sort, 80 sums, 18 joins; filled after the sort by the
// launch that sums, 350.)
// Up to 256 tokens, one launch does it all without a sort (k_sum_few).

#include <type_traits>

#include "hg_fill.h"
#include "hg_tile.h"
#include "hg_vocab.h"

namespace hg {

namespace {

struct TypeF32 {};

// 16 bytes of a row as fp32 values, and back (rounded to nearest even).
template <class T>
struct Vec {
  static constexpr int N = 8;
  static __device__ __forceinline__ void get(u32x4 v, float *f) {
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      f[2 * t] = from16<T>(v[t] & 0xFFFFu);
      f[2 * t + 1] = from16<T>(v[t] >> 16);
    }
  }
  static __device__ __forceinline__ u32x4 put(const float *f) {
    u32x4 v;
#pragma unroll
    for (int t = 0; t < 4; ++t) v[t] = bits16<T>(f[2 * t]) | bits16<T>(f[2 * t + 1]) << 16;
    return v;
  }
};
template <>
struct Vec<TypeF32> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void get(u32x4 v, float *f) {
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const uint32_t b = v[t];  // (a bit cast of a vector's element takes the first one)
      f[t] = __builtin_bit_cast(float, b);
    }
  }
  static __device__ __forceinline__ u32x4 put(const float *f) {
    u32x4 v;
#pragma unroll
    for (int t = 0; t < 4; ++t) v[t] = __builtin_bit_cast(uint32_t, f[t]);
    return v;
  }
};

__device__ __forceinline__ long long token_at(const void *tokens, int bytes, long long i) {
  return bytes == 8 ? static_cast<const long long *>(tokens)[i]
                    : static_cast<const int *>(tokens)[i];
}

// U 16-byte vectors per lane, 256 apart; a workgroup takes 256*U vectors of a
// row.
template <class T, int NT, int U>
__global__ __launch_bounds__(256) void k_embed(ShardTableN<NT> w, int shard, int rows,
                                               const void *tokens, int token_bytes, int n, int hv,
                                               float scale, u32x4 *out) {
  const int k = static_cast<int>(blockIdx.x * (256 * U) + threadIdx.x);
  for (int j = static_cast<int>(blockIdx.y); j < n; j += static_cast<int>(gridDim.y)) {
    const long long t = token_at(tokens, token_bytes, j);
    const bool real = t >= 0 && t < rows;
    const int rank = NT == 1 || !real ? 0 : static_cast<int>(t) / shard;
    const u32x4 *src = w.p[rank] + (real ? t - static_cast<long long>(rank) * shard : 0) * hv;
    u32x4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (real && k + 256 * u < hv) v[u] = src[k + 256 * u];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (k + 256 * u >= hv) break;
      if (real) {
        float f[Vec<T>::N];
        Vec<T>::get(v[u], f);
#pragma unroll
        for (int e = 0; e < Vec<T>::N; ++e) f[e] *= scale;
        v[u] = Vec<T>::put(f);
      } else {
        v[u] = u32x4{0u, 0u, 0u, 0u};
      }
      u32x4 *o = out + static_cast<long long>(j) * hv + k + 256 * u;
      if constexpr (U > 1) __builtin_nontemporal_store(v[u], o);
      else *o = v[u];
    }
  }
}

size_t up256(size_t b) { return (b + 255) & ~static_cast<size_t>(255); }

// ---------------------------------------------------------------------------
// The sort. A key is the token, or `rows` where the token lies outside.

constexpr int kSortTile = 4096;  // keys per workgroup
constexpr int kDigits = 512;
constexpr int kSortWaves = 16;

__device__ __forceinline__ int key_at(const void *tokens, int bytes, long long i, int rows) {
  const long long t = token_at(tokens, bytes, i);
  return t >= 0 && t < rows ? static_cast<int>(t) : rows;
}

// Lanes of the wave (of those in `live`) with this lane's digit.
__device__ __forceinline__ unsigned long long same_digit(int digit, unsigned long long live) {
  unsigned long long m = live;
#pragma unroll
  for (int b = 0; b < 9; ++b) {
    const unsigned long long votes = __ballot((digit >> b) & 1);
    m &= ((digit >> b) & 1) ? votes : ~votes;
  }
  return m;
}

// Exclusive scan of 8 values per thread over the 1024 threads of a workgroup.
__device__ __forceinline__ void scan8(int (&v)[8], int *wave_sum) {
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 63, wave = tid >> 6;
  int sum = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) sum += v[e];
  int up = sum;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(up, d);
    if (lane >= d) up += o;
  }
  if (lane == 63) wave_sum[wave] = up;
  __syncthreads();
  int run = up - sum;
  for (int k = 0; k < wave; ++k) run += wave_sum[k];
  __syncthreads();
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int c = v[e];
    v[e] = run;
    run += c;
  }
}

// The per-wave digit counts [kDigits][kSortWaves] of a workgroup's keys; wave
// w holds keys w*per .. of the tile, in order.
template <class K>
__device__ __forceinline__ void count_digits(int *count, int n, int per, int shift, K key) {
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 63, wave = tid >> 6;
  for (int k = tid; k < kDigits * kSortWaves; k += 1024) count[k] = 0;
  __syncthreads();
  const int end = (wave + 1) * per < n ? (wave + 1) * per : n;
  for (int k = wave * per + lane; k < end; k += 64)
    atomicAdd(&count[((key(k) >> shift) & (kDigits - 1)) * kSortWaves + wave], 1);
  __syncthreads();
}

// Each wave hands its keys, in order, the places its counters hold.
template <class K, class P>
__device__ __forceinline__ void place_keys(volatile int *place, int n, int per, int shift, K key, P put) {
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 63, wave = tid >> 6;
  const int end = (wave + 1) * per < n ? (wave + 1) * per : n;
  for (int k0 = wave * per; k0 < end; k0 += 64) {
    const int k = k0 + lane;
    const bool live = k < end;
    const int v = live ? key(k) : 0;
    const int digit = (v >> shift) & (kDigits - 1);
    const unsigned long long lanes = same_digit(digit, __ballot(live));
    const int at = live ? place[digit * kSortWaves + wave] : 0;
    const int rank = __popcll(lanes & ((1ull << lane) - 1));
    // the counter is the wave's own; its last lane of the digit moves it on
    if (live && (lanes >> lane) == 1ull) place[digit * kSortWaves + wave] = at + rank + 1;
    if (live) put(k, v, at + rank);
  }
}

// Zeros, written by the workgroups of a sort launch that the sort leaves over:
// the sort is a chain of latencies on few CUs, the fill needs HBM alone. One
// store per thread: the chip then writes one front through memory (671 MB: 110
// us; 8 stores per thread, a front per workgroup, 119, 16 stores 125).
struct Fill {
  u32x4 *p;
  long long vecs;
  int groups;
};
__device__ __forceinline__ void fill_part(const Fill &f, int k) {
  for (long long i = static_cast<long long>(k) * kFillVecs + threadIdx.x; i < f.vecs;
       i += static_cast<long long>(f.groups) * kFillVecs)
    f.p[i] = u32x4{0u, 0u, 0u, 0u};
}

// Where the sorted keys begin: seg[i] is the first place of a key of i or more, for i
// in 0 .. rows; place j writes those between its key and the one before it.
template <class K>
__device__ __forceinline__ void begin_segments(K key, int j, int n, int rows, int *seg) {
  const int before = j > 0 ? key(j - 1) : -1, here = j < n ? key(j) : rows;
  for (int i = before + 1; i <= here; ++i) seg[i] = j;
}
__global__ __launch_bounds__(256) void k_sort_segments(const int *keys, int n, int rows, int *seg) {
  const int j = static_cast<int>(blockIdx.x * 256 + threadIdx.x);
  if (j <= n) begin_segments([&](int k) { return keys[k]; }, j, n, rows, seg);
}

// All keys in one workgroup's LDS. seg may be NULL.
__global__ __launch_bounds__(1024) void k_sort_tile(const void *tokens, int token_bytes, int n,
                                                    int rows, int passes, int *keys, int *pos,
                                                    int *seg, Fill fill) {
  if (blockIdx.x > 0) {
    fill_part(fill, static_cast<int>(blockIdx.x) - 1);
    return;
  }
  __shared__ int count[kDigits * kSortWaves];
  __shared__ int sk[2][kSortTile], sp[2][kSortTile];
  __shared__ int wave_sum[16];
  const int tid = static_cast<int>(threadIdx.x);
  const int per = ((n + 1023) / 1024) * 64;
  for (int k = tid; k < n; k += 1024) {
    sk[0][k] = key_at(tokens, token_bytes, k, rows);
    sp[0][k] = k;
  }
  __syncthreads();
  for (int p = 0; p < passes; ++p) {
    const int *ik = sk[p & 1], *ip = sp[p & 1];
    int *ok = sk[(p & 1) ^ 1], *op = sp[(p & 1) ^ 1];
    auto key = [&](int k) { return ik[k]; };
    count_digits(count, n, per, 9 * p, key);
    int v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = count[8 * tid + e];
    scan8(v, wave_sum);
#pragma unroll
    for (int e = 0; e < 8; ++e) count[8 * tid + e] = v[e];
    __syncthreads();
    place_keys(count, n, per, 9 * p, key, [&](int k, int kv, int at) {
      ok[at] = kv;
      op[at] = ip[k];
    });
    __syncthreads();
  }
  for (int k = tid; k < n; k += 1024) {
    keys[k] = sk[passes & 1][k];
    pos[k] = sp[passes & 1][k];
  }
  if (seg)
    for (int k = tid; k <= n; k += 1024)
      begin_segments([&](int j) { return sk[passes & 1][j]; }, k, n, rows, seg);
}

// Counts of one pass: hist[digit][tile].
__global__ __launch_bounds__(1024) void k_sort_count(const void *tokens, int token_bytes,
                                                     const int *keys, long long n, int rows,
                                                     int shift, int *hist, int tiles, Fill fill) {
  if (static_cast<int>(blockIdx.x) >= tiles) {
    fill_part(fill, static_cast<int>(blockIdx.x) - tiles);
    return;
  }
  __shared__ int count[kDigits];
  const int tid = static_cast<int>(threadIdx.x);
  const long long base = static_cast<long long>(blockIdx.x) * kSortTile;
  if (tid < kDigits) count[tid] = 0;
  __syncthreads();
  for (int k = tid; k < kSortTile && base + k < n; k += 1024) {
    const int v = keys ? keys[base + k] : key_at(tokens, token_bytes, base + k, rows);
    atomicAdd(&count[(v >> shift) & (kDigits - 1)], 1);
  }
  __syncthreads();
  if (tid < kDigits) hist[tid * tiles + blockIdx.x] = count[tid];
}

// Exclusive scan of the counts, in place; one workgroup, 8192 at a time.
__global__ __launch_bounds__(1024) void k_sort_scan(int *hist, int n, Fill fill) {
  if (blockIdx.x > 0) {
    fill_part(fill, static_cast<int>(blockIdx.x) - 1);
    return;
  }
  __shared__ int wave_sum[16], total;
  const int tid = static_cast<int>(threadIdx.x);
  int carry = 0;
  for (int k0 = 0; k0 < n; k0 += 8192) {
    int v[8], last = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int k = k0 + 8 * tid + e;
      v[e] = k < n ? hist[k] : 0;
      last = v[e];
    }
    scan8(v, wave_sum);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int k = k0 + 8 * tid + e;
      if (k < n) hist[k] = carry + v[e];
    }
    if (tid == 1023) total = v[7] + last;
    __syncthreads();
    carry += total;
    __syncthreads();
  }
}

// Scatter of one pass.
__global__ __launch_bounds__(1024) void k_sort_place(const void *tokens, int token_bytes,
                                                     const int *keys, const int *pos, long long n,
                                                     int rows, int shift, const int *hist,
                                                     int tiles, int *okeys, int *opos, Fill fill) {
  if (static_cast<int>(blockIdx.x) >= tiles) {
    fill_part(fill, static_cast<int>(blockIdx.x) - tiles);
    return;
  }
  __shared__ int count[kDigits * kSortWaves];
  __shared__ int sk[kSortTile];
  const int tid = static_cast<int>(threadIdx.x);
  const long long base = static_cast<long long>(blockIdx.x) * kSortTile;
  const int here = n - base < kSortTile ? static_cast<int>(n - base) : kSortTile;
  for (int k = tid; k < here; k += 1024)
    sk[k] = keys ? keys[base + k] : key_at(tokens, token_bytes, base + k, rows);
  __syncthreads();
  auto key = [&](int k) { return sk[k]; };
  const int per = kSortTile / kSortWaves;
  count_digits(count, here, per, shift, key);
  if (tid < kDigits) {
    int run = hist[tid * tiles + blockIdx.x];
    for (int w = 0; w < kSortWaves; ++w) {
      const int c = count[tid * kSortWaves + w];
      count[tid * kSortWaves + w] = run;
      run += c;
    }
  }
  __syncthreads();
  place_keys(count, here, per, shift, key, [&](int k, int kv, int at) {
    okeys[at] = kv;
    opos[at] = pos ? pos[base + k] : static_cast<int>(base + k);
  });
}

// ---------------------------------------------------------------------------
// The sums.

struct SumArgs {
  const int *keys, *pos;
  const u32x4 *dy;
  void *dw;
  float *part;      // [blocks][2][hidden]
  long long n;
  int rows, hidden, per;  // per: positions per block
  int blocks, slabs;      // slabs of 256 vectors in a row
  float scale;
  int accumulate;
};

template <class T, class D>
__device__ __forceinline__ void write_row(const SumArgs &a, int v, int col, const float *sum) {
  constexpr int N = Vec<T>::N;
  float f[N];
#pragma unroll
  for (int e = 0; e < N; ++e) f[e] = sum[e] * a.scale;
  const long long at = static_cast<long long>(v) * a.hidden + col;
  if constexpr (std::is_same_v<T, D>) {
    u32x4 *o = reinterpret_cast<u32x4 *>(static_cast<char *>(a.dw) + at * (16 / N));
    if (a.accumulate) {
      float old[N];
      Vec<T>::get(*o, old);
#pragma unroll
      for (int e = 0; e < N; ++e) f[e] += old[e];
    }
    *o = Vec<T>::put(f);
  } else {  // 16-bit dy, fp32 gradient
    f32x4 *o = reinterpret_cast<f32x4 *>(static_cast<float *>(a.dw) + at);
#pragma unroll
    for (int h = 0; h < N / 4; ++h) {
      f32x4 x = {f[4 * h], f[4 * h + 1], f[4 * h + 2], f[4 * h + 3]};
      o[h] = a.accumulate ? o[h] + x : x;
    }
  }
}

// Workgroup: one block of sorted positions and 256 vectors of a row.
template <class T, class D>
__global__ __launch_bounds__(256) void k_sum(SumArgs a) {
  constexpr int N = Vec<T>::N;
  const int tid = static_cast<int>(threadIdx.x);
  const int bid = static_cast<int>(blockIdx.x);
  const int hv = a.hidden / N;
  const int blk = bid / a.slabs, k = (bid - blk * a.slabs) * 256 + tid;
  const long long j0 = static_cast<long long>(blk) * a.per;
  const int here = a.n - j0 < a.per ? static_cast<int>(a.n - j0) : a.per;
  const int *keys = a.keys + j0, *pos = a.pos + j0;
  const int before = blk > 0 ? keys[-1] : -1;
  const int after = j0 + here < a.n ? keys[here] : -2;
  const int lane = tid & 63;
  float sum[N];
#pragma unroll
  for (int e = 0; e < N; ++e) sum[e] = 0.f;
  float *part = a.part + static_cast<long long>(blk) * 2 * a.hidden + k * N;
  // Rows in flight: 16, or half as many positions per block, measured the same
  // (79 us at 65536 tokens of 2048 columns, the fill's zeros still on their way).
  constexpr int kAhead = 8;
  for (int j64 = 0; j64 < here; j64 += 64) {
    // 64 keys and positions at once, a lane each; handed out as scalars
    const int some = here - j64 < 64 ? here - j64 : 64;
    const int mykey = lane < some ? keys[j64 + lane] : a.rows;
    const int mypos = lane < some ? pos[j64 + lane] : 0;
    const int beyond = j64 + 64 < here ? keys[j64 + 64] : -2;  // the key after these
    // tokens outside sort last
    const int real = __popcll(__ballot(mykey < a.rows));
    for (int j = 0; j < real; j += kAhead) {
      u32x4 v[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int p = __builtin_amdgcn_readlane(mypos, j + u < real ? j + u : 0);
        if (j + u < real && k < hv)
          v[u] = __builtin_nontemporal_load(a.dy + static_cast<long long>(p) * hv + k);
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        if (j + u >= real) break;
        const int key = __builtin_amdgcn_readlane(mykey, j + u);
        const bool last = j64 + j + u + 1 == here;  // of the block
        const int next = last ? after
                              : j + u + 1 < 64 ? __builtin_amdgcn_readlane(mykey, j + u + 1) : beyond;
        float f[N];
        Vec<T>::get(v[u], f);
#pragma unroll
        for (int e = 0; e < N; ++e) sum[e] += f[e];
        if (key == next && !last) continue;
        // the sum of `key` ends here, or goes on in the next block
        if (k < hv) {
          if (key == before || key == next) {
            f32x4 *o = reinterpret_cast<f32x4 *>(part + (key == before ? 0 : a.hidden));
#pragma unroll
            for (int h = 0; h < N / 4; ++h)
              o[h] = f32x4{sum[4 * h], sum[4 * h + 1], sum[4 * h + 2], sum[4 * h + 3]};
          } else {
            write_row<T, D>(a, key, k * N, sum);
          }
        }
#pragma unroll
        for (int e = 0; e < N; ++e) sum[e] = 0.f;
      }
    }
  }
}

// Sums that cross block edges: the block in which such a sum begins adds the
// partial rows of the blocks it runs through, in order.
template <class T, class D>
__global__ __launch_bounds__(256) void k_sum_join(SumArgs a) {
  constexpr int N = Vec<T>::N;
  const int hv = a.hidden / N;
  const int blk = static_cast<int>(blockIdx.x) / a.slabs;
  const int k = (static_cast<int>(blockIdx.x) - blk * a.slabs) * 256 + static_cast<int>(threadIdx.x);
  const long long j1 = static_cast<long long>(blk + 1) * a.per;
  if (j1 >= a.n) return;
  const int key = a.keys[j1 - 1];
  if (key >= a.rows || a.keys[j1] != key) return;  // nothing crosses this edge
  // a sum that began before this block is joined there
  if (blk > 0 && a.keys[j1 - a.per - 1] == key) return;
  // the blocks the sum runs through: 64 of their first keys at a time
  int end = blk + 1;
  for (bool on = true; on;) {
    const int b = end + (static_cast<int>(threadIdx.x) & 63);
    const bool same = b < a.blocks && a.keys[static_cast<long long>(b) * a.per] == key;
    const int run = __ffsll(~__ballot(same)) - 1;  // -1: all 64
    end += run < 0 ? 64 : run;
    on = run < 0;
  }
  if (k >= hv) return;
  float sum[N];
  const float *p = a.part + (static_cast<long long>(blk) * 2 + 1) * a.hidden + k * N;
#pragma unroll
  for (int e = 0; e < N; ++e) sum[e] = p[e];
  p = a.part + static_cast<long long>(blk + 1) * 2 * a.hidden + k * N;
  constexpr int kAhead = 8;
  for (int b = blk + 1; b < end; b += kAhead) {
    f32x4 v[kAhead][N / 4];
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
#pragma unroll
      for (int h = 0; h < N / 4; ++h)
        v[u][h] = b + u < end ? reinterpret_cast<const f32x4 *>(p + 2ll * u * a.hidden)[h]
                              : f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (b + u < end) {
#pragma unroll
        for (int e = 0; e < N; ++e) sum[e] += v[u][e / 4][e % 4];
      }
    p += 2ll * kAhead * a.hidden;
  }
  write_row<T, D>(a, key, k * N, sum);
}

// Few tokens: everything in one launch, with no sort. The first workgroups take
// a position and 256 vectors of its row each; the one whose position is its
// token's first adds up the rows of all of them, in order. The others write
// zeros, 64 rows each, but for the rows that a token names.
constexpr int kFewTokens = 256;  // one per thread
template <class T, class D>
__global__ __launch_bounds__(256) void k_sum_few(SumArgs a, const void *tokens, int token_bytes) {
  constexpr int N = Vec<T>::N;
  const int tid = static_cast<int>(threadIdx.x), bid = static_cast<int>(blockIdx.x);
  const int n = static_cast<int>(a.n), hv = a.hidden / N;
  __shared__ unsigned long long named[4];
  const int mine = tid < n ? key_at(tokens, token_bytes, tid, a.rows) : a.rows;
  if (bid < n * a.slabs) {
    const int j = bid / a.slabs, k = (bid - j * a.slabs) * 256 + tid;
    const int key = key_at(tokens, token_bytes, j, a.rows);
    if (key >= a.rows) return;
    const unsigned long long votes = __ballot(mine == key);
    if ((tid & 63) == 0) named[tid >> 6] = votes;
    __syncthreads();
    unsigned long long m[4];
#pragma unroll
    for (int w = 0; w < 4; ++w) m[w] = named[w];
    for (int w = 0; w < (j >> 6); ++w)
      if (m[w]) return;
    if (m[j >> 6] & ((1ull << (j & 63)) - 1)) return;  // an earlier position has the token
    if (k >= hv) return;
    float sum[N];
#pragma unroll
    for (int e = 0; e < N; ++e) sum[e] = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      while (m[w]) {
        u32x4 v[8];
        int got = 0;
#pragma unroll
        for (int u = 0; u < 8; ++u)
          if (m[w]) {
            const int p = 64 * w + __ffsll(m[w]) - 1;
            m[w] &= m[w] - 1;
            v[u] = a.dy[static_cast<long long>(p) * hv + k];
            got = u + 1;
          }
#pragma unroll
        for (int u = 0; u < 8; ++u)
          if (u < got) {
            float f[N];
            Vec<T>::get(v[u], f);
#pragma unroll
            for (int e = 0; e < N; ++e) sum[e] += f[e];
          }
      }
    }
    write_row<T, D>(a, key, k * N, sum);
    return;
  }
  const int v0 = (bid - n * a.slabs) * 64;
  if (tid == 0) named[0] = 0;
  __syncthreads();
  if (mine >= v0 && mine < v0 + 64 && mine < a.rows) atomicOr(&named[0], 1ull << (mine - v0));
  __syncthreads();
  const unsigned long long skip = named[0];
  const int vecs = hv * (std::is_same_v<T, D> ? 1 : 2);
  u32x4 *dw = static_cast<u32x4 *>(a.dw) + static_cast<long long>(v0) * vecs;
  const int last = a.rows - v0 < 64 ? a.rows - v0 : 64;
  if (!skip) {  // one run of memory
    const long long all = static_cast<long long>(last) * vecs;
    for (long long k = tid; k < all; k += 256) dw[k] = u32x4{0u, 0u, 0u, 0u};
    return;
  }
  for (int r = 0; r < last; ++r) {
    if ((skip >> r) & 1) continue;
    for (int k = tid; k < vecs; k += 256)
      dw[static_cast<long long>(r) * vecs + k] = u32x4{0u, 0u, 0u, 0u};
  }
}

// One store per thread, as above (671 MB: 102 us, 6.6 TB/s).
__global__ __launch_bounds__(256) void k_zero(u32x4 *p, long long vecs) {
  for (long long k = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x; k < vecs;
       k += static_cast<long long>(gridDim.x) * 256)
    p[k] = u32x4{0u, 0u, 0u, 0u};
}

template <class F>
void by_dtype(int dtype, F f) {
  if (dtype == HG_BF16) f(TypeBf16{});
  else if (dtype == HG_FP16) f(TypeF16{});
  else f(TypeF32{});
}

}  // namespace

hipError_t launch_embed(const VocabMatrix &w, int rows, int dtype, const void *tokens,
                        int token_bytes, int n, float scale, void *out, hipStream_t s) {
  by_dtype(dtype, [&](auto type) {
    using T = decltype(type);
    const int hv = w.hidden / Vec<T>::N;
    auto go = [&](auto nt, auto vecs) {
      constexpr int NT = decltype(nt)::value, U = decltype(vecs)::value;
      const dim3 grid((hv + 256 * U - 1) / (256 * U), n < 32768 ? n : 32768);
      ShardTableN<NT> t;
      for (int r = 0; r < NT; ++r) t.p[r] = w.t.p[r];
      hipLaunchKernelGGL((k_embed<T, NT, U>), grid, dim3(256), 0, s, t, w.shard, rows, tokens,
                         token_bytes, n, hv, scale, static_cast<u32x4 *>(out));
    };
    using One = std::integral_constant<int, 1>;
    using All = std::integral_constant<int, HG_MAX_TP>;
    using Four = std::integral_constant<int, 4>;
    // Four vectors in flight per lane, and stores that pass the caches, once
    // every CU has work without them: 16383 rows of 14 KB take 57 us instead of
    // 90 with one vector per lane and plain stores. Fewer rows spread over more
    // waves (4 rows: 2.5 us).
    const bool many = static_cast<long long>(n) * hv >= (1 << 18);
    if (w.tp == 1) many ? go(One{}, Four{}) : go(One{}, One{});
    else many ? go(All{}, Four{}) : go(All{}, One{});
  });
  return hipGetLastError();
}

hipError_t launch_zero(void *p, size_t bytes, hipStream_t s) {
  const long long vecs = static_cast<long long>(bytes / 16);
  if (vecs == 0) return hipSuccess;
  const long long want = (vecs + 255) / 256;
  hipLaunchKernelGGL(k_zero, dim3(static_cast<unsigned>(want < (1 << 22) ? want : 1 << 22)),
                     dim3(256), 0, s, static_cast<u32x4 *>(p), vecs);
  return hipGetLastError();
}

SortPlan sort_plan(int rows, long long n) {
  SortPlan p = {};
  int bits = 1;
  while ((1ll << bits) <= rows) ++bits;  // the largest key is `rows`
  p.passes = (bits + 8) / 9;
  p.tiles = static_cast<int>((n + kSortTile - 1) / kSortTile);
  size_t at = 0;
  for (int k = 0; k < 4; ++k) {
    p.off[k] = at;  // keys, positions, and the other side of each pass
    at += up256(static_cast<size_t>(n) * sizeof(int));
  }
  p.off[4] = at;  // counts
  at += up256(static_cast<size_t>(p.tiles) * kDigits * sizeof(int));
  p.bytes = at;
  return p;
}

namespace {

int sort_launches(const SortPlan &p) { return p.tiles <= 1 ? 1 : 3 * p.passes; }

// fill(&groups) gives each launch its share of zeros to write beside the sort, and
// adds the workgroups that it takes.
template <class F>
Sorted launch_sort(const SortPlan &p, char *base, int rows, const void *tokens, int token_bytes,
                   long long n, int *seg, hipStream_t s, F fill) {
  int *buf[4], *hist = reinterpret_cast<int *>(base + p.off[4]);
  for (int k = 0; k < 4; ++k) buf[k] = reinterpret_cast<int *>(base + p.off[k]);
  int side = 0;
  if (p.tiles <= 1) {
    int groups = 1;
    const Fill f = fill(&groups);
    hipLaunchKernelGGL(k_sort_tile, dim3(groups), dim3(1024), 0, s, tokens, token_bytes,
                       static_cast<int>(n), rows, p.passes, buf[0], buf[1], seg, f);
  } else {
    for (int k = 0; k < p.passes; ++k) {
      const int *ik = k ? buf[2 * side] : nullptr, *ip = k ? buf[2 * side + 1] : nullptr;
      if (k) side ^= 1;
      int g1 = p.tiles, g2 = 1, g3 = p.tiles;
      const Fill f1 = fill(&g1), f2 = fill(&g2), f3 = fill(&g3);
      hipLaunchKernelGGL(k_sort_count, dim3(g1), dim3(1024), 0, s, tokens, token_bytes, ik, n, rows,
                         9 * k, hist, p.tiles, f1);
      hipLaunchKernelGGL(k_sort_scan, dim3(g2), dim3(1024), 0, s, hist, p.tiles * kDigits, f2);
      hipLaunchKernelGGL(k_sort_place, dim3(g3), dim3(1024), 0, s, tokens, token_bytes, ik, ip, n,
                         rows, 9 * k, hist, p.tiles, buf[2 * side], buf[2 * side + 1], f3);
    }
    if (seg)
      hipLaunchKernelGGL(k_sort_segments, dim3(static_cast<unsigned>(n / 256 + 1)), dim3(256), 0, s, buf[2 * side],
                         static_cast<int>(n), rows, seg);
  }
  return Sorted{buf[2 * side], buf[2 * side + 1]};
}

}  // namespace

hipError_t launch_sort(const SortPlan &p, void *ws, int rows, const void *index, int index_bytes,
                       long long n, int *seg, Sorted *sorted, hipStream_t s) {
  *sorted = launch_sort(p, static_cast<char *>(ws), rows, index, index_bytes, n, seg, s,
                        [](int *) { return Fill{nullptr, 0, 1}; });
  return hipGetLastError();
}

EmbedPlan embed_plan(int rows, int hidden, long long n) {
  EmbedPlan p = {};
  if (n <= kFewTokens) return p;  // no workspace
  // Positions per block: at least 8 (the rows in flight), and no more blocks
  // than about eight workgroups per CU need.
  long long per = n / 2048;
  p.per = static_cast<int>(per < 8 ? 8 : per > 256 ? 256 : per);
  p.blocks = static_cast<int>((n + p.per - 1) / p.per);
  p.part = sort_plan(rows, n).bytes;
  p.bytes = p.part + up256(static_cast<size_t>(p.blocks) * 2 * hidden * sizeof(float));
  return p;
}

hipError_t launch_embed_grad(const EmbedPlan &p, void *ws, int rows, int hidden, int dtype,
                             const void *tokens, int token_bytes, long long n, const void *dy,
                             float scale, void *dw, bool wide, bool accumulate, hipStream_t s) {
  const long long zeros = accumulate ? 0
                                     : static_cast<long long>(rows) * hidden *
                                           (wide || dtype == HG_FP32 ? 4 : 2) / 16;
  if (n == 0) return launch_zero(dw, static_cast<size_t>(zeros) * 16, s);
  SumArgs a = {};
  a.dy = static_cast<const u32x4 *>(dy);
  a.dw = dw;
  a.n = n;
  a.rows = rows;
  a.hidden = hidden;
  a.scale = scale;
  a.accumulate = accumulate ? 1 : 0;
  auto with_types = [&](auto go) {
    by_dtype(dtype, [&](auto type) {
      using T = decltype(type);
      a.slabs = (hidden / Vec<T>::N + 255) / 256;
      if constexpr (!std::is_same_v<T, TypeF32>) {
        if (wide) {
          go(type, TypeF32{});
          return;
        }
      }
      go(type, type);
    });
  };
  if (n <= kFewTokens) {
    // a long fill is faster as a launch of its own, with one store per thread
    const bool apart = zeros > (32 << 20) / 16;
    if (apart) {
      const hipError_t e = launch_zero(dw, static_cast<size_t>(zeros) * 16, s);
      if (e != hipSuccess) return e;
    }
    const int fills = accumulate || apart ? 0 : (rows + 63) / 64;
    with_types([&](auto t, auto d) {
      hipLaunchKernelGGL((k_sum_few<decltype(t), decltype(d)>),
                         dim3(static_cast<unsigned>(n) * a.slabs + fills), dim3(256), 0, s, a,
                         tokens, token_bytes);
    });
    return hipGetLastError();
  }
  char *base = static_cast<char *>(ws);
  const SortPlan sort = sort_plan(rows, n);
  const int launches = sort_launches(sort);
  const long long share = (zeros + launches - 1) / launches;
  int part = 0;
  // the zeros, cut into one part per launch of the sort
  const Sorted sorted = launch_sort(sort, base, rows, tokens, token_bytes, n, nullptr, s, [&](int *groups) {
    Fill f;
    const long long at = share * part++;
    f.p = static_cast<u32x4 *>(dw) + at;
    f.vecs = zeros - at < share ? zeros - at : share;
    f.groups = fill_groups(f.vecs);
    *groups += f.groups;
    return f;
  });
  a.keys = sorted.keys;
  a.pos = sorted.pos;
  a.part = reinterpret_cast<float *>(base + p.part);
  a.per = p.per;
  a.blocks = p.blocks;
  with_types([&](auto t, auto d) {
    using T = decltype(t);
    using D = decltype(d);
    hipLaunchKernelGGL((k_sum<T, D>), dim3(a.blocks * a.slabs), dim3(256), 0, s, a);
    if (a.blocks > 1)
      hipLaunchKernelGGL((k_sum_join<T, D>), dim3((a.blocks - 1) * a.slabs), dim3(256), 0, s, a);
  });
  return hipGetLastError();
}

}  // namespace hg
