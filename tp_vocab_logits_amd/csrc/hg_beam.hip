// Beam search on the logits: which continuations of a request's beams to keep,
// and the beams' states put in their order.
//
//   c_kv = score_k + scale * z_kv - log sum_v exp(scale * z_kv)
//
// Selection, two launches. The scan reads every logit once: a workgroup holds
// its part of a row in registers, finds its maximum, its sum of exponentials
// and its `keep` largest entries. The join (a workgroup per request, a wave per
// beam) merges the parts' sums and lists, and the beams' lists by c.
//
// An entry is a 64-bit key: the logit's bits in the order of its value above the
// complement of its place, so that larger keys are better entries and equal
// logits go by the lowest place. Largest entries are found by a bound from below:
// the keep-th largest of a wave's 64 lane maxima (found bit by bit, a ballot
// each). No more than the lanes at or above it hold entries of interest: those
// go to LDS, where each counts the larger ones. Where equal logits make them too
// many for LDS, the bound is found among all entries, ties included.
//
// Order over beams: the candidates of different beams are compared through their
// rows' sums, so an error of a sum shifts a whole beam. fp32's, about 1e-6 of a
// logarithm of 12, would swap two candidates in about one of a thousand requests
// (16 of them, about 0.02 apart); sums and scores are therefore in 64 bits, the
// exponentials to 6e-11, a
// polynomial of degree 7 for 2^f on [-1/2, 1/2] (interpolated at the Chebyshev
// points). The 64-bit instructions run at fp32's rate on this chip.
//
// Measured: 512 rows of 163837 bf16 entries, a tenth of them finished, keep 16: scan
// 70 to 75 us, join 13. Reading alone takes 28 of them; vector instructions, 31 an entry
// with half of them the exponentials', are issued in 88 % of the cycles and bound it. Four
// rows of 163840 are bound by latency: 5.7 and 7.3 us. With 64 to keep the lanes' maxima
// are no bound worth the name (the least of 64), most entries are of interest and a part
// falls back to the search among all: 512 rows 1.3 ms.
#include <type_traits>

#include "hg_beam.h"
#include "hg_tile.h"

namespace hg {

namespace {

typedef unsigned long long u64;

constexpr int kFound = 1024;            // entries in LDS that a workgroup ranks
constexpr uint32_t kLeast = 0x00800000u;  // order of the lowest finite fp32

struct BeamF32 {};

// 16 bytes as fp32 values, and which bits an order of theirs can differ in.
template <class T>
struct Lane {
  static constexpr int N = 8, kLow = T::kHalf ? 13 : 16;
  static constexpr uint32_t kNone = T::kHalf ? 0xFC00u : 0xFF80u;  // minus infinity
  using elt = unsigned short;
  typedef uint32_t anywhere __attribute__((ext_vector_type(4), aligned(2)));  // 16 bytes at any element
  static __device__ __forceinline__ void get(u32x4 v, float *f) {
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      f[2 * t] = from16<T>(v[t] & 0xFFFFu);
      f[2 * t + 1] = from16<T>(v[t] >> 16);
    }
  }
  // The largest value, NaN left out, of N vectors: pairs of 16-bit integers in the
  // values' order (one and a half instructions an element); positive NaN are above
  // infinity there and taken out if one shows, negative ones below it.
  template <int J>
  static __device__ __forceinline__ float largest(const u32x4 (&v)[J]) {
    typedef short pair __attribute__((ext_vector_type(2)));
    constexpr short kTop = T::kHalf ? 0x7C00 : 0x7F80;
    pair top = {-32768, -32768};
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const uint32_t w = v[j][t];
        const uint32_t sign = __builtin_bit_cast(uint32_t, __builtin_bit_cast(pair, w) >> 15);
        top = __builtin_elementwise_max(top, __builtin_bit_cast(pair, w ^ (sign & 0x7FFF7FFFu)));
      }
    short most = top[0] > top[1] ? top[0] : top[1];
    if (__ballot(most > kTop)) {
      most = -32768;
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int t = 0; t < 8; ++t) {
          const short b = static_cast<short>(v[j][t / 2] >> 16 * (t & 1));
          const short o = static_cast<short>(b ^ (b >> 15 & 0x7FFF));
          most = o > most && o <= kTop ? o : most;
        }
    }
    const float z = from16<T>(static_cast<unsigned short>(most ^ (most >> 15 & 0x7FFF)));
    return z == z ? z : -__builtin_inff();  // (negative NaN alone)
  }
};
template <>
struct Lane<BeamF32> {
  static constexpr int N = 4, kLow = 0;
  static constexpr uint32_t kNone = 0xFF800000u;
  using elt = uint32_t;
  typedef uint32_t anywhere __attribute__((ext_vector_type(4), aligned(4)));
  static __device__ __forceinline__ void get(u32x4 v, float *f) {
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const uint32_t b = v[t];
      f[t] = __builtin_bit_cast(float, b);
    }
  }
  template <int J>
  static __device__ __forceinline__ float largest(const u32x4 (&v)[J]) {
    float top = -__builtin_inff();
#pragma unroll
    for (int j = 0; j < J; ++j) {
      float f[4];
      get(v[j], f);
#pragma unroll
      for (int t = 0; t < 4; ++t) top = f[t] > top ? f[t] : top;
    }
    return top;
  }
};

// The order of a value's bits: larger values, larger orders; one zero.
__device__ __forceinline__ uint32_t order_of(float z) {
  const uint32_t b = __builtin_bit_cast(uint32_t, z + 0.0f);
  return b ^ (static_cast<uint32_t>(static_cast<int>(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t o) {
  return __builtin_bit_cast(float, o & 0x80000000u ? o ^ 0x80000000u : ~o);
}
__device__ __forceinline__ u64 key_of(float z, int place) {
  return static_cast<u64>(order_of(z)) << 32 | ~static_cast<uint32_t>(place);
}

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int d = 32; d; d >>= 1) v = fmaxf(v, __shfl_xor(v, d));
  return v;
}
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

// The n-th largest of the lanes' orders, cut to the bits from LOW on; the least
// order of a finite value if fewer than n lanes have one (0: a lane without).
template <int LOW>
__device__ __forceinline__ uint32_t nth_order(uint32_t o, int n) {
  uint32_t t = 0;
#pragma unroll
  for (int bit = 31; bit >= LOW; --bit) {
    const uint32_t trial = t | 1u << bit;
    if (__popcll(__ballot(o >= trial)) >= n) t = trial;
  }
  return t > kLeast ? t : kLeast;
}

// exp2(t) for t <= 0 (NaN and what is below -1000: as at -1000, which adds nothing
// to a sum of at least 2^-1).
__device__ __forceinline__ double exp2_of(double t) {
  constexpr double kRound = 6755399441055744.0;  // 1.5 * 2^52: its low bits are the rounded t
  t = t > -1000.0 ? t : -1000.0;
  const double k = t + kRound;
  const double f = t - (k - kRound);
  double p = 0.000015303700711365693939;
  p = __builtin_fma(p, f, 0.00015469729214118297093);
  p = __builtin_fma(p, f, 0.0013333478473685415281);
  p = __builtin_fma(p, f, 0.0096180256133180342494);
  p = __builtin_fma(p, f, 0.055504109063258666119);
  p = __builtin_fma(p, f, 0.24022651213498092661);
  p = __builtin_fma(p, f, 0.69314718055683241353);
  p = __builtin_fma(p, f, 0.99999999995956175074);
  return __builtin_ldexp(p, static_cast<int>(static_cast<uint32_t>(__builtin_bit_cast(u64, k))));
}

struct ScanArgs {
  int shard, vocab, keep, per_block, parts;
  double rate;  // scale * log2(e)
  const float *scores;
  const unsigned char *finished;
  BeamStat *stat;
  u64 *keys;
};

__device__ __forceinline__ bool is_live(float score) {
  return score > -__builtin_inff() && score < __builtin_inff();
}

template <class T, int J, int NT>
__global__ __launch_bounds__(kScanThreads) void k_beam_scan(ShardTableN<NT> logits, ScanArgs a) {
  using L = Lane<T>;
  constexpr float kNoneF = -__builtin_inff();
  constexpr int kMine = J * L::N;  // entries of a lane
  __shared__ u64 found[kFound];
  __shared__ u32x4 held[kScanThreads * J];
  __shared__ double sums[4];
  __shared__ float tops[4];
  __shared__ uint32_t bounds[4];
  __shared__ int count;

  const int tid = static_cast<int>(threadIdx.x);
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int row = static_cast<int>(blockIdx.x) / a.parts;
  const int part = static_cast<int>(blockIdx.x) - row * a.parts;
  const int rank = NT == 1 ? 0 : part / a.per_block;
  const int piece = part - rank * a.per_block;
  const int first = rank * a.shard;  // the block's first place in the vocabulary
  const int width = a.vocab - first < a.shard ? a.vocab - first : a.shard;
  BeamStat *const stat = a.stat + blockIdx.x;
  u64 *const out = a.keys + static_cast<size_t>(blockIdx.x) * a.keep;

  // Rows may start anywhere: vectors are counted from the row's first element, so
  // that equal rows are summed in the same order and their candidates tie. (The
  // last one may not be whole and is read element by element.)
  const typename L::elt *const base =
      reinterpret_cast<const typename L::elt *>(logits.p[rank]) + static_cast<size_t>(row) * a.shard;
  const int at0 = (piece * (J * kScanThreads) + tid) * L::N;
  // A beam that is not there, or finished: the join asks for nothing, and nothing is
  // read of it. (Asking while the logits are on their way saves nothing: 5.7 us of four
  // rows of 163840 both ways.)
  if (!is_live(a.scores[row]) || (a.finished && a.finished[row])) return;
  u32x4 v[J];
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int at = at0 + j * (kScanThreads * L::N);
    if (at + L::N <= width) {
      v[j] = __builtin_nontemporal_load(reinterpret_cast<const typename L::anywhere *>(base + at));
    } else {
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        if constexpr (L::N == 4) {
          v[j][t] = at + t < width ? base[at + t] : L::kNone;
        } else {
          const int e = at + 2 * t;
          const uint32_t lo = e < width ? base[e] : L::kNone;
          const uint32_t hi = e + 1 < width ? base[e + 1] : L::kNone;
          v[j][t] = lo | hi << 16;
        }
      }
    }
  }
  if (tid == 0) count = 0;

  const float top = L::largest(v);
  const float wtop = wave_max(top);
  const uint32_t bound = nth_order<L::kLow>(top > kNoneF ? order_of(top) : 0u, a.keep);

  double sum = 0.0;
  if (wtop == __builtin_inff()) {  // these alone have a share
    float n = 0.f;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      float f[L::N];
      L::get(v[j], f);
#pragma unroll
      for (int e = 0; e < L::N; ++e) n += f[e] == wtop ? 1.f : 0.f;
    }
    sum = n;
  } else if (wtop > kNoneF) {
    const double from = -static_cast<double>(wtop) * a.rate;
    double s[2] = {0.0, 0.0};
#pragma unroll
    for (int j = 0; j < J; ++j) {
      float f[L::N];
      L::get(v[j], f);
#pragma unroll
      for (int e = 0; e < L::N; ++e)
        s[e & 1] += exp2_of(__builtin_fma(static_cast<double>(f[e]), a.rate, from));
    }
    sum = s[0] + s[1];
  }
  sum = wave_sum(sum);
  if ((tid & 63) == 0) {
    sums[wave] = sum;
    tops[wave] = wtop;
    bounds[wave] = bound;
  }
  __syncthreads();

  // any wave's bound is one of the workgroup's
  uint32_t best = bounds[0];
#pragma unroll
  for (int w = 1; w < 4; ++w) best = bounds[w] > best ? bounds[w] : best;
  float least = value_of(best);
  auto each = [&](auto &&use) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < J; ++j) {
      float f[L::N];
      L::get(v[j], f);
      const int place = first + at0 + j * (kScanThreads * L::N);
#pragma unroll
      for (int e = 0; e < L::N; ++e) use(f[e], place + e);
    }
  };
  // Which of the lane's entries are of interest: a bit each, without a branch; the few
  // that are, are looked up again in LDS.
  static_assert(kMine <= 32);
  uint32_t bits = 0;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    float f[L::N];
    L::get(v[j], f);
#pragma unroll
    for (int e = 0; e < L::N; ++e) bits = bits + bits + (f[e] >= least ? 1u : 0u);
  }
  if (bits) {
#pragma unroll
    for (int j = 0; j < J; ++j) held[j * kScanThreads + tid] = v[j];
    do {
      const int k = 31 - __builtin_clz(bits);  // the last entry is bit 0
      bits &= ~(1u << k);
      const int i = kMine - 1 - k, j = i / L::N, e = i % L::N;
      const u32x4 *const from = held + j * kScanThreads + tid;
      float z;
      if constexpr (L::N == 4)
        z = reinterpret_cast<const float *>(from)[e];
      else
        z = from16<T>(reinterpret_cast<const unsigned short *>(from)[e]);
      const int n = atomicAdd(&count, 1);
      if (n < kFound) found[n] = key_of(z, first + at0 + j * (kScanThreads * L::N) + e);
    } while (bits);
  }
  if (tid == 0) {
    float t = tops[0];
    for (int w = 1; w < 4; ++w) t = fmaxf(t, tops[w]);
    double s = 0.0;
    for (int w = 0; w < 4; ++w)
      if (tops[w] == t)
        s += sums[w];
      else if (t < __builtin_inff() && tops[w] > kNoneF)
        s += sums[w] * exp2_of((static_cast<double>(tops[w]) - static_cast<double>(t)) * a.rate);
    *stat = BeamStat{s, t, 0};
  }
  __syncthreads();
  int n = count;
  if (n > kFound) {  // many equal ones: the keep-th largest key of all, bit by bit
    u64 bar = 0;
    for (int bit = 63; bit >= 0; --bit) {
      const u64 trial = bar | 1ull << bit;
      int mine = 0;
      each([&](float z, int place) __attribute__((always_inline)) {
        mine += z >= least && key_of(z, place) >= trial;
      });
      __syncthreads();
      if (tid == 0) count = 0;
      __syncthreads();
      if (mine) atomicAdd(&count, mine);
      __syncthreads();
      if (count >= a.keep) bar = trial;
    }
    __syncthreads();
    if (tid == 0) count = 0;
    __syncthreads();
    each([&](float z, int place) __attribute__((always_inline)) {
      if (z >= least && key_of(z, place) >= bar) found[atomicAdd(&count, 1)] = key_of(z, place);
    });
    __syncthreads();
    n = count;
  }
  // an entry's place: how many are larger, counted by four threads
  for (int i = tid >> 2; i < n; i += kScanThreads / 4) {
    const u64 key = found[i];
    int larger = 0;
    for (int k0 = tid & 3; k0 < n; k0 += 16) {
#pragma unroll
      for (int t = 0; t < 4; ++t) larger += k0 + 4 * t < n && found[k0 + 4 * t] > key;
    }
    larger += __shfl_xor(larger, 1);
    larger += __shfl_xor(larger, 2);
    if ((tid & 3) == 0 && larger < a.keep) out[larger] = key;
  }
  for (int i = n + tid; i < a.keep; i += kScanThreads) out[i] = 0;
}

struct JoinArgs {
  int beams, keep, parts, vocab, pad, room;
  double scale, rate;
  const float *scores;
  const unsigned char *finished;
  const BeamStat *stat;
  const u64 *keys;
  float *out;
  long long *parents, *tokens;
};

// LDS of the join: scores [beams][keep], tokens [beams][keep], entries per beam
// [64], per wave a counter and `room` entries.
struct JoinLds {
  int score, token, filled, counter, found, bytes;
};
__host__ __device__ inline JoinLds join_lds(int beams, int keep, int waves, int room) {
  JoinLds l;
  l.score = 0;
  l.found = l.score + beams * keep * 8;
  l.token = l.found + waves * room * 8;
  l.filled = l.token + beams * keep * 4;
  l.counter = l.filled + 64 * 4;
  l.bytes = l.counter + waves * 4;
  return l;
}

__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "workgroup");
  __builtin_amdgcn_wave_barrier();
}

// Beam k of the request: its best entries' scores and tokens, and how many.
__device__ __forceinline__ int join_row(const JoinArgs &a, int row, int lane, double *score, int *token,
                                        u64 *found, int *counter) {
  const float s = a.scores[row];
  if (!is_live(s)) return 0;
  if (a.finished && a.finished[row]) {
    if (lane == 0) {
      score[0] = s;
      token[0] = a.pad;
    }
    return 1;
  }
  const BeamStat *const stat = a.stat + static_cast<size_t>(row) * a.parts;
  const u64 *const keys = a.keys + static_cast<size_t>(row) * a.parts * a.keep;
  // The entries, eight of a lane in registers (all there are, mostly): with the
  // parts' sums, they are one round trip.
  const int all = a.parts * a.keep;
  u64 mine[8];
  auto load8 = [&](int i0, u64 (&k)[8]) __attribute__((always_inline)) {
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      const int i = i0 + t * 64 + lane;
      k[t] = i < all ? keys[i] : 0;
    }
  };
  load8(0, mine);
  auto each = [&](auto &&use) __attribute__((always_inline)) {
#pragma unroll
    for (int t = 0; t < 8; ++t) use(mine[t]);
    for (int i0 = 512; i0 < all; i0 += 512) {
      u64 k[8];
      load8(i0, k);
#pragma unroll
      for (int t = 0; t < 8; ++t) use(k[t]);
    }
  };
  // the row's largest and its sum
  BeamStat one = lane < a.parts ? stat[lane] : BeamStat{0.0, -__builtin_inff(), 0};
  float top = one.top;
  for (int p = lane + 64; p < a.parts; p += 64) top = fmaxf(top, stat[p].top);
  top = wave_max(top);
  if (top == -__builtin_inff()) return 0;
  const bool boundless = top == __builtin_inff();
  double sum = 0.0;
  for (int p = lane;;) {
    if (one.top == top)
      sum += one.sum;
    else if (!boundless && one.top > -__builtin_inff())
      sum += one.sum * exp2_of((static_cast<double>(one.top) - static_cast<double>(top)) * a.rate);
    if ((p += 64) >= a.parts) break;
    one = stat[p];
  }
  sum = wave_sum(sum);
  const double lse = boundless ? log(sum) : a.scale * static_cast<double>(top) + log(sum);

  // Entries at or above the keep-th of the lanes' best logits: at most keep lanes
  // have any that are above it, about twice keep entries in all for logits in no
  // order.
  u64 head = 0;
  each([&](u64 k) __attribute__((always_inline)) { head = k > head ? k : head; });
  u64 bar = static_cast<u64>(nth_order<0>(static_cast<uint32_t>(head >> 32), a.keep)) << 32;
  auto collect = [&]() __attribute__((always_inline)) {
    wave_fence();
    if (lane == 0) *counter = 0;
    wave_fence();
    each([&](u64 k) __attribute__((always_inline)) {
      if (k >= bar) {
        const int at = atomicAdd(counter, 1);
        if (at < a.room) found[at] = k;
      }
    });
    wave_fence();
    return *reinterpret_cast<volatile int *>(counter);
  };
  auto total = [](int c) __attribute__((always_inline)) {
#pragma unroll
    for (int d = 32; d; d >>= 1) c += __shfl_xor(c, d);
    return c;
  };
  int n = collect();
  if (n > a.room) {  // lanes that hold most of the best, or equal logits: the keep-th itself
    bar = 0;
    for (int bit = 63; bit >= 0; --bit) {
      const u64 trial = bar | 1ull << bit;
      int c = 0;
      each([&](u64 k) __attribute__((always_inline)) { c += k >= trial; });
      if (total(c) >= a.keep) bar = trial;
    }
    if (bar == 0) bar = 1;
    n = collect();
  }
  int filled = 0;
  for (int i = lane; i < n; i += 64) {
    const u64 key = found[i];
    int larger = 0;
    for (int k = 0; k < n; ++k) larger += found[k] > key;
    const float z = value_of(static_cast<uint32_t>(key >> 32));
    if (larger < a.keep && (!boundless || z == top)) {
      // (the first of a row of infinities have its share)
      score[larger] = boundless ? s - lse : s + (a.scale * static_cast<double>(z) - lse);
      token[larger] = static_cast<int>(~static_cast<uint32_t>(key));
      ++filled;
    }
  }
  return total(filled);
}

__global__ __launch_bounds__(1024) void k_beam_join(JoinArgs a) {
  extern __shared__ __align__(16) unsigned char lds[];
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), waves = static_cast<int>(blockDim.x) >> 6;
  const JoinLds l = join_lds(a.beams, a.keep, waves, a.room);
  double *const score = reinterpret_cast<double *>(lds + l.score);
  int *const token = reinterpret_cast<int *>(lds + l.token);
  int *const filled = reinterpret_cast<int *>(lds + l.filled);
  const int q = static_cast<int>(blockIdx.x);
  for (int k = wave; k < a.beams; k += waves) {
    const int n = join_row(a, q * a.beams + k, lane, score + k * a.keep, token + k * a.keep,
                           reinterpret_cast<u64 *>(lds + l.found) + wave * a.room,
                           reinterpret_cast<int *>(lds + l.counter) + wave);
    if (lane == 0) filled[k] = n;
    wave_fence();
  }
  __syncthreads();
  // An entry's rank over the beams: every beam's list descends, so the entries of
  // another one that come first are found by bisection.
  float *const out = a.out + static_cast<size_t>(q) * a.keep;
  long long *const parents = a.parents + static_cast<size_t>(q) * a.keep;
  long long *const tokens = a.tokens + static_cast<size_t>(q) * a.keep;
  for (int id = tid; id < a.beams * a.keep; id += static_cast<int>(blockDim.x)) {
    const int k = id / a.keep, i = id - k * a.keep;
    if (i >= filled[k]) continue;
    const double c = score[id];
    int rank = i;
    for (int o = 0; o < a.beams && rank < a.keep; ++o) {
      if (o == k) continue;
      const double *const list = score + o * a.keep;
      int lo = 0, hi = filled[o];
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        const bool first = o < k ? list[mid] >= c : list[mid] > c;
        if (first)
          lo = mid + 1;
        else
          hi = mid;
      }
      rank += lo;
    }
    if (rank < a.keep) {
      out[rank] = static_cast<float>(c);
      parents[rank] = k;
      tokens[rank] = token[id];
    }
  }
  int total = 0;
  for (int k = 0; k < a.beams && total < a.keep; ++k) total += filled[k];
  for (int i = total + tid; i < a.keep; i += static_cast<int>(blockDim.x)) {
    out[i] = -__builtin_inff();
    parents[i] = -1;
    tokens[i] = -1;
  }
}

template <class T, int J, int NT>
void scan(const BeamPlan &p, const ShardTable &logits, const ScanArgs &a, hipStream_t s) {
  ShardTableN<NT> t;
  for (int r = 0; r < NT; ++r) t.p[r] = logits.p[r];
  hipLaunchKernelGGL((k_beam_scan<T, J, NT>), dim3(p.requests * p.beams * p.parts), dim3(kScanThreads), 0,
                     s, t, a);
}
template <class T, int J>
void scan(const BeamPlan &p, const ShardTable &logits, const ScanArgs &a, hipStream_t s) {
  if (p.tp == 1)
    scan<T, J, 1>(p, logits, a, s);
  else if (p.tp <= kSmallTable)
    scan<T, J, kSmallTable>(p, logits, a, s);
  else
    scan<T, J, HG_MAX_TP>(p, logits, a, s);
}
template <class T>
void scan(const BeamPlan &p, const ShardTable &logits, const ScanArgs &a, hipStream_t s) {
  switch (p.vecs) {
    case 1: return scan<T, 1>(p, logits, a, s);
    case 2: return scan<T, 2>(p, logits, a, s);
    default: return scan<T, 4>(p, logits, a, s);
  }
}

constexpr double kLog2E = 1.4426950408889634074;

}  // namespace

hipError_t launch_beam_scan(const BeamPlan &p, const ShardTable &logits, const float *scores,
                            const unsigned char *finished, hipStream_t s) {
  const ScanArgs a{p.shard, p.vocab, p.keep, p.per_block, p.parts, p.scale * kLog2E,
                   scores, finished, p.stat, p.keys};
  if (p.dtype == HG_FP32)
    scan<BeamF32>(p, logits, a, s);
  else if (p.dtype == HG_FP16)
    scan<TypeF16>(p, logits, a, s);
  else
    scan<TypeBf16>(p, logits, a, s);
  return hipGetLastError();
}

hipError_t launch_beam_join(const BeamPlan &p, const float *scores, const unsigned char *finished,
                            float *out, long long *parents, long long *tokens, hipStream_t s) {
  // A wave per beam, up to 16, each with room for the most entries that are ranked as
  // they are (128; more than keep in any case).
  constexpr int room = 128;
  int waves = p.beams < 16 ? p.beams : 16;
  if (join_lds(p.beams, p.keep, waves, room).bytes > 65536) waves = 8;
  const JoinArgs a{p.beams, p.keep, p.parts, p.vocab, p.pad, room, p.scale, p.scale * kLog2E,
                   scores, finished, p.stat, p.keys, out, parents, tokens};
  hipLaunchKernelGGL(k_beam_join, dim3(p.requests), dim3(64 * waves),
                     join_lds(p.beams, p.keep, waves, room).bytes, s, a);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Reordering in place. A thread owns one column (16 bytes, or 4 where there are
// many beams) of all of a request's rows: it reads what every changed row
// becomes, then writes. No other thread touches the column, so nothing is read
// after it was overwritten. Bytes bound it: changed rows are written once, rows
// that several take are read again from the caches (1.8 GB in 347 to 356 us, 5.1 TB/s;
// a copy reaches 4.8).

namespace {

constexpr int kMoveThreads = 256;

struct MoveArgs {
  int requests, beams, outer, chunks, steps;
  unsigned items;
  long long row_stride, outer_stride;
  u64 step_bytes;
  const void *parents, *lengths;
  int parent_bytes, length_bytes;
};

__device__ __forceinline__ long long int_at(const void *p, int bytes, size_t i) {
  return bytes == 8 ? static_cast<const long long *>(p)[i] : static_cast<const int *>(p)[i];
}

template <int W, bool ALIGNED>
struct Column;
template <>
struct Column<16, true> {
  typedef u32x4 type;
};
template <>
struct Column<16, false> {
  typedef uint32_t type __attribute__((ext_vector_type(4), aligned(1)));
};
template <>
struct Column<4, true> {
  typedef uint32_t type;
};
template <>
struct Column<4, false> {
  typedef uint32_t type __attribute__((aligned(1)));
};

// KM: beams at most; W: bytes of a column. A thread has one column: with four of them,
// states of 2.1 GB took 385 us instead of 353, 165 rows of 28 KB 21 instead of 11.
template <int KM, int W, bool ALIGNED, int NT>
__global__ __launch_bounds__(kMoveThreads) void k_beam_move(StateTable<NT> states, MoveArgs a) {
  typedef typename Column<W, ALIGNED>::type memory;
  __shared__ int from[KM];
  const int tid = static_cast<int>(threadIdx.x);
  for (unsigned item = blockIdx.x; item < a.items; item += gridDim.x) {
    unsigned rest = item / a.chunks;
    const unsigned chunk = item - rest * a.chunks;
    const unsigned o = rest % a.outer;
    rest /= a.outer;
    const unsigned q = rest % a.requests, st = rest / a.requests;
    long long len = a.steps;
    if (a.lengths) {
      const long long l = int_at(a.lengths, a.length_bytes, q);
      len = l < 0 ? 0 : l < len ? l : len;
    }
    const u64 run = static_cast<u64>(len) * a.step_bytes;
    const u64 at0 = static_cast<u64>(chunk) * (kMoveThreads * W);
    if (at0 >= run) continue;
    __syncthreads();  // (the last item's reads are done)
    bool moves = false;
    if (tid < KM) {
      int p = -1;
      if (tid < a.beams) {
        const long long want = int_at(a.parents, a.parent_bytes, static_cast<size_t>(q) * a.beams + tid);
        if (want >= 0 && want < a.beams && want != tid) p = static_cast<int>(want);
      }
      from[tid] = p;
      moves = p >= 0;
    }
    if (!__syncthreads_or(moves)) continue;
    unsigned char *const base = states.p[st] + static_cast<long long>(q) * a.beams * a.row_stride +
                                static_cast<long long>(o) * a.outer_stride;
    const u64 at = at0 + static_cast<u64>(tid) * W;
    if (at + W <= run) {
      memory v[KM];
#pragma unroll
      for (int k = 0; k < KM; ++k) {
        const int p = __builtin_amdgcn_readfirstlane(from[k]);
        if (p >= 0) v[k] = *reinterpret_cast<const memory *>(base + p * a.row_stride + at);
      }
#pragma unroll
      for (int k = 0; k < KM; ++k)
        if (__builtin_amdgcn_readfirstlane(from[k]) >= 0)
          *reinterpret_cast<memory *>(base + k * a.row_stride + at) = v[k];
    } else {
      for (u64 b = at; b < run; ++b) {  // the run's last bytes
        unsigned char v[KM];
#pragma unroll
        for (int k = 0; k < KM; ++k)
          if (from[k] >= 0) v[k] = base[from[k] * a.row_stride + b];
#pragma unroll
        for (int k = 0; k < KM; ++k)
          if (from[k] >= 0) base[k * a.row_stride + b] = v[k];
      }
    }
  }
}

struct MoveShape {
  int width, chunks;
  long long items;
};
MoveShape move_shape(const ReorderPlan &p) {
  MoveShape m;
  m.width = p.beams <= 16 ? 16 : 4;
  const u64 run = static_cast<u64>(p.steps) * p.step_bytes;
  const long long runs = static_cast<long long>(p.requests) * p.outer * p.count;
  const u64 bytes = static_cast<u64>(kMoveThreads) * m.width;
  const u64 chunks = (run + bytes - 1) / bytes;
  m.chunks = chunks < (1u << 30) ? static_cast<int>(chunks) : 1 << 30;
  m.items = runs * m.chunks;
  return m;
}

template <int KM, int W, bool ALIGNED, int NT>
void move(const MoveArgs &a, unsigned char *const *states, int count, hipStream_t s) {
  StateTable<NT> t;
  for (int i = 0; i < NT; ++i) t.p[i] = states[i < count ? i : 0];
  const unsigned grid = a.items < (1u << 22) ? a.items : 1u << 22;
  hipLaunchKernelGGL((k_beam_move<KM, W, ALIGNED, NT>), dim3(grid), dim3(kMoveThreads), 0, s, t, a);
}
template <int KM, int W, bool ALIGNED>
void move(const MoveArgs &a, unsigned char *const *states, int count, hipStream_t s) {
  if (count <= kFewStates)
    move<KM, W, ALIGNED, kFewStates>(a, states, count, s);
  else
    move<KM, W, ALIGNED, kStates>(a, states, count, s);
}
template <int KM, int W>
void move(const MoveArgs &a, bool aligned, unsigned char *const *states, int count, hipStream_t s) {
  if (aligned)
    move<KM, W, true>(a, states, count, s);
  else
    move<KM, W, false>(a, states, count, s);
}

}  // namespace

long long beam_reorder_items(const ReorderPlan &p) { return move_shape(p).items; }

hipError_t launch_beam_reorder(const ReorderPlan &p, unsigned char *const *states, hipStream_t s) {
  const MoveShape m = move_shape(p);
  if (m.items == 0) return hipSuccess;
  const MoveArgs a{p.requests, p.beams, p.outer, m.chunks, p.steps, static_cast<unsigned>(m.items),
                   p.row_stride, p.outer_stride, p.step_bytes, p.parents, p.lengths, p.parent_bytes,
                   p.length_bytes};
  uintptr_t bits = static_cast<uintptr_t>(p.row_stride) | static_cast<uintptr_t>(p.outer_stride);
  for (int i = 0; i < p.count; ++i) bits |= reinterpret_cast<uintptr_t>(states[i]);
  const bool aligned = (bits & (m.width - 1)) == 0;
  if (p.beams <= 4)
    move<4, 16>(a, aligned, states, p.count, s);
  else if (p.beams <= 8)
    move<8, 16>(a, aligned, states, p.count, s);
  else if (p.beams <= 16)
    move<16, 16>(a, aligned, states, p.count, s);
  else
    move<64, 4>(a, aligned, states, p.count, s);
  return hipGetLastError();
}

}  // namespace hg
