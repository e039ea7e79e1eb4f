// The next token from a row of logits (uw_sample): temperature, top-k, top-p,
// min-p and the draw from a given uniform number.
//
// A row is read from memory once, by a cluster of CTAs (a run of the row each);
// the later passes find it in L2, where the rows in work (one CTA per SM) fit.
// The ids kept by top-k and top-p are a prefix of the falling order, so nothing
// sorts the row.  A histogram over the distance from the maximum bounds where
// the prefix ends: for top-k the bin in which the count crosses, for top-p the
// few bins in which the weight can cross, since a bin's weights are alike.
// Then
//   - where all logits down to there are few (top_k up to about a thousand, a
//     nucleus of a peaked row), they are gathered and ordered, and one CTA
//     finishes the row from that list;
//   - else one pass sums the exact weight above the open bins and lists the
//     logits in them; those are cut into key ranges until few are left, and the
//     order of the few gives the threshold: a logit, and how many of its ties
//     stay (the lowest ids).  The kept weight of each warp's stretch of the row
//     says where the choice lies, and that stretch is searched.
//
// Weights are whole multiples of 2^-40 of the largest one, summed in 64 bits:
// no order of additions and no launch shape changes a result, and every CTA of
// a cluster takes the same decisions from the same merged numbers.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>
#include <type_traits>

#include "gemm_sm100.cuh"
#include "handle.h"
#include "pdl.cuh"
#include "serving.h"

namespace uw {
namespace {

using namespace sm100;
typedef unsigned long long u64;

constexpr int kMaxVocab = 1 << 18;
constexpr int kThreads = 1024;
constexpr int kWarpsPer = kThreads / 32;
constexpr int kPer = 4;               // bins per thread in the scan over them
constexpr int kBins = kPer * kThreads;
constexpr int kFine = kThreads;       // bins of a cut into key ranges: count and three pieces of the weight
constexpr int kCap = kThreads;        // logits that are ordered exactly: one per thread, at most
constexpr int kFew = 256;             // logits down to which a cut is narrowed
constexpr int kFixBits = 40;          // 2^18 weights of at most 2^40 fit in 64 bits
constexpr int kPiece = 14;            // a weight in three pieces of 14 bits, whose 2^18 sums fit in 32
constexpr int kMaxListed = 38;        // keys per thread of the logits that may end a prefix
constexpr int kMaxCluster = 8;
constexpr float kSpan = 28.f;         // weights of e^-28 and less are 0 in 40 bits
constexpr float kPerUnit = (kBins - 1) / kSpan;
constexpr uint32_t kAll = 0xFFFFFFFFu;
constexpr float kMagic = 24576.f;     // 1.5 * 2^14: one unit is 2^-9

struct SampleParams {
  uw_sample_args a;
  int32_t run;     // elements of a row per CTA
  int32_t listed;  // keys per thread that have room
  int32_t ordered; // rows that take long come first
};

struct Shared {
  uint2 table[512];        // of the weights
  uint32_t count[4 * kFine];   // kBins, or the cut's
  u64 list[kCap];          // this CTA's gathered entries
  u64 order[kCap];         // entries in order
  u64 post[2][4];          // numbers published to the cluster, two rounds
  u64 scratch[4 * kWarpsPer];
  float bound[2 * kWarpsPer];
  u64 found[4];
  uint32_t ends[4];
  uint32_t n_list;
};

// With room for `listed` keys per thread, and the `v` that a step may write behind them.
constexpr size_t shared_bytes(int listed, int v) {
  return (sizeof(Shared) + 15) / 16 * 16 + sizeof(float) * kThreads * (listed + v);
}
constexpr size_t kSharedBytes = shared_bytes(0, 0);
static_assert(shared_bytes(kMaxListed, 8) <= 227 * 1024, "shared memory");

__device__ __forceinline__ uint32_t peer(const void* p, uint32_t rank) { return mapa_shared(smem_u32(p), rank); }

__device__ __forceinline__ u64 ld_peer_u64(const void* p, uint32_t rank) {
  u64 v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(peer(p, rank)) : "memory");
  return v;
}

__device__ __forceinline__ uint32_t ld_peer_u32(const void* p, uint32_t rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(peer(p, rank)) : "memory");
  return v;
}

__device__ __forceinline__ uint4 ld_peer_u32x4(const void* p, uint32_t rank) {
  uint4 v;
  asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(peer(p, rank)) : "memory");
  return v;
}

// Unsigned keys in the order of the floats.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t u = __float_as_uint(x);
  return u ^ ((u >> 31) ? kAll : 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : kAll));
}

// The least key above lo that fits, where all from some key on do; hi if none
// below it does.  A warp halves the range five times per step.
template <typename F>
__device__ __forceinline__ uint32_t least_key(uint32_t lo, uint32_t hi, F fits) {
  const int lane = threadIdx.x & 31;
  while (hi - lo > 1) {
    const uint32_t step = (hi - lo + 31) / 32, at = lo + (lane + 1) * step;
    const bool past = at >= hi, fit = fits(at);  // (both: a branch would cost more)
    const uint32_t f = __ffs(__ballot_sync(kAll, past | fit)) - 1;  // (the last lane's is past the end)
    hi = min(hi, lo + (f + 1) * step);
    lo += f * step;
  }
  return hi;
}

// One row's weights: w(x) = 2^40 e^((x - max) / t), to 2^-29.8 of itself (2^-31.7 in the mean of squares: a table
// entry and a correction, each rounded to a unit of a number of 31 bits), the bits below one dropped.
// y = (max - x) log2(e) / t = i / 512 + g with g small, and the weight is a table
// entry times the Taylor polynomial of 2^-g (the table-driven scheme of Tang,
// 1989), whose correction is added to the entry as a whole number.  log2(e) / t is
// carried in two floats, hi + lo, and max (hi + lo) as a multiple of 2^-9 and a
// rest: then one multiply-add rounds x hi to i, and a second gives what that
// left, x hi being exact inside both.  That holds while |x hi| stays below 2^12;
// where the maximum's does not, x is taken less the maximum, a difference that is
// exact for all that have a weight (they lie within a hundredth of it).
// About 20 instructions, six of them for the integer unit, which bounds the
// passes over a row (with differences in two floats 256 rows without a cut took
// 104 us, so 59; FP64 arithmetic takes eight times the first).
// Temperatures far from one are brought near it, and the logits by the same power
// of two, inside the multiply-adds (where the temperature is tiny only if that
// keeps the maximum finite: else all differences are far above it).
struct Weights {
  float max, scale;            // the largest logit; of all logits, a power of two
  float top, per_bin;          // max * scale; bins per unit of x * scale
  float hi, lo;                // log2(e) / t, t scaled
  float origin;                // 0, or `top`
  float whole, rest;           // of (top - origin) (hi + lo) - 9
  float near;                  // x above which a weight may exceed 32 bits
  float floor;                 // x * scale - origin below which weights are taken as 0
  const uint2* table;          // [512] 2^31 2^(-i / 512), whole (less kWhole's bits) and as a float

  static constexpr float kWhole = 12582912.f;  // 1.5 * 2^23: |2^31 c| < 2^22
  static constexpr uint32_t kWholeBits = 0x4B400000u;

  __device__ __forceinline__ void set(float peak, float t) {
    constexpr float kLog2e = (float)1.4426950408889634074, kLog2eLow = (float)(1.4426950408889634074 - (double)kLog2e);
    max = peak;
    scale = t > 1e20f ? 0x1p-100f : (t < 1e-20f && fabsf(max) < 1e6f ? 0x1p100f : 1.f);
    t *= scale;
    top = max * scale;
    hi = fminf(kLog2e / t, 1e30f);  // (finite: the maximum's distance is 0)
    lo = hi < 1e30f && hi > 1e-30f ? (fmaf(-hi, t, kLog2e) + kLog2eLow) / t : 0.f;  // from hi's remainder
    per_bin = hi * (kPerUnit / kLog2e);
    origin = fabsf(top) * hi < 4000.f ? 0.f : top;
    const float over = top - origin, units = fmaf(over, hi, kMagic) - kMagic;
    rest = fmaf(over, lo, fmaf(over, hi, -units));
    whole = units - 9.f;
    near = __fdiv_rd(__fadd_rd(over - 9.01f / hi, origin), scale);
    lower(40.5f);
  }
  // Take weights of 2^-octaves and less as 0.
  __device__ __forceinline__ void lower(float octaves) { floor = fmaxf(top - origin - octaves / hi, -FLT_MAX); }
  __device__ __forceinline__ bool weighs(float x) const { return fmaf(x, scale, -origin) >= floor; }
  // Whether one of x may have a weight near the maximum's, of more than 32 bits.
  template <int V>
  __device__ __forceinline__ bool is_near(const float (&x)[V]) const {
    float most = x[0];
#pragma unroll
    for (int j = 1; j < V; ++j) most = fmaxf(most, x[j]);
    return most > near;
  }
  // The weight as m 2^-n, the bits below one to be dropped, in two steps; *at holds
  // n (its nine are in `whole`) from bit 9 on.  (No branch: a lane with nothing to
  // weigh would not spare the others' work.  NaN and infinite x are not above
  // `floor`.)
  __device__ __forceinline__ uint32_t parts(float x, uint32_t* at) const {
    x = fmaf(x, scale, -origin);
    const float t = fmaf(x, -hi, whole + kMagic);
    const float g = fmaf(x, -hi, whole - (t - kMagic)) + fmaf(x, -lo, rest);
    constexpr float kA = -0.69314718055994531f, kB = 0.24022650695910071f, kC = -0.055504108664821580f;  // of 2^-g
    const float c = g * fmaf(g, fmaf(g, kC, kB), kA);
    *at = __float_as_uint(t);
    const uint2 entry = table[*at & 511];
    const uint32_t m = entry.x + __float_as_uint(fmaf(__uint_as_float(entry.y), c, kWhole));
    return x >= floor ? m : 0u;
  }
  // of any x
  static __device__ __forceinline__ u64 wide(uint32_t m, uint32_t at) {
    return ((u64)m << 9) >> ((at + 9 * 512) >> 9 & 63);
  }
  // of an x that is not near: n is 0 to 31
  static __device__ __forceinline__ uint32_t small(uint32_t m, uint32_t at) { return __funnelshift_r(m, 0u, at >> 9); }
  __device__ __forceinline__ u64 operator()(float x) const {
    uint32_t at;
    const uint32_t m = parts(x, &at);
    return wide(m, at);
  }
  // Distance from the maximum in bins; NaN for NaN.
  __device__ __forceinline__ float place(float x) const { return fmaf(x, -scale, top) * per_bin; }
  // The least finite x, as it compares, whose place is `lim` or less; above the
  // maximum if there is none.  (place does not fall as x falls: each of its steps
  // is monotone.)
  __device__ __forceinline__ float lowest(float lim) const {
    if (lim == INFINITY) return -FLT_MAX;
    const auto fits = [&](uint32_t k) { return place(of_key(k)) <= lim; };
    uint32_t lo = key_of(-FLT_MAX) - 1, hi = key_of(max) + 1;
    // nearer, where that holds: about where place is lim
    const float at = (top - lim / per_bin) / scale, off = fabsf(max) * 4e-7f;
    const uint32_t a = key_of(at - off), b = key_of(at + off);
    if (a > lo && a < hi && !fits(a)) lo = a;
    if (b > lo && b < hi && fits(b)) hi = b;
    return of_key(least_key(lo, hi, fits));
  }
  // Histogram bin of x: it does not fall as x falls (each step is monotone).
  __device__ __forceinline__ uint32_t bin(float x) const {
    return __float_as_uint(fminf(place(x), (float)(kBins - 1)) + 8388608.f) & (kBins - 1);
  }
  // The largest place() of bins up to b (its rounding to even takes b + 1/2 down
  // where b is even).
  static __device__ __forceinline__ float limit(int b) {
    if (b < 0) return -1.f;
    if (b >= kBins - 1) return INFINITY;
    return b % 2 ? __uint_as_float(__float_as_uint((float)b + 0.5f) - 1) : (float)b + 0.5f;
  }
};
static_assert((kBins & (kBins - 1)) == 0 && kBins <= 4096, "bin() keeps the low bits");

__device__ __forceinline__ u64 min_u64(u64 a, u64 b) { return a < b ? a : b; }
__device__ __forceinline__ u64 max_u64(u64 a, u64 b) { return a > b ? a : b; }

// Inclusive running sums over the lanes of a warp.
__device__ __forceinline__ uint32_t scan_warp(uint32_t v) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t x = __shfl_up_sync(kAll, v, d);
    if ((threadIdx.x & 31) >= d) v += x;
  }
  return v;
}

// Sum over a warp, in pieces whose sums fit in 32 bits (three reductions; ten
// shuffles took three times as long).
__device__ __forceinline__ u64 sum_warp(u64 v) {
  const uint32_t a = (uint32_t)v & 0x3FFFFFFu, b = (uint32_t)(v >> 26) & 0x3FFFFFFu, c = (uint32_t)(v >> 52);
  return __reduce_add_sync(kAll, a) + ((u64)__reduce_add_sync(kAll, b) << 26) + ((u64)__reduce_add_sync(kAll, c) << 52);
}

// sum += v, as a product, which does not burden the integer unit; `one` is 1 (and
// known to be only when the kernel runs).
__device__ __forceinline__ void add_wide(u64* sum, uint32_t v, uint32_t one) {
  asm("mad.wide.u32 %0, %1, %2, %0;" : "+l"(*sum) : "r"(v), "r"(one));
}

// One cluster's view of a row; T: float, or uint16_t for BF16.
template <typename T>
struct Row {
  static constexpr int V = 16 / sizeof(T);  // elements per load
  Shared& s;
  const T* base;   // 16-byte aligned, at or before this CTA's run
  int skip, n;     // the run: elements skip .. skip + n - 1 from base
  int id0;         // id of the element at base
  int rank, ranks;
  int round;       // of the exchange
  bool infinite;   // the largest logit is +infinity: 0 then, and all others nothing
  Weights w;

  __device__ __forceinline__ int warp() const { return threadIdx.x >> 5; }
  __device__ __forceinline__ int lane() const { return threadIdx.x & 31; }
  // A warp's elements are one stretch, a lane's V neighbours of each step:
  // ids rise with warp, step, lane and place.
  __device__ __forceinline__ int stretch() const { return (skip + n + kThreads * V - 1) / (kThreads * V) * (32 * V); }

  // NaN counts as -infinity, as does what lies outside the run; there is one
  // zero.  (Passes that only compare take the values as they are.)
  static __device__ __forceinline__ float clean(float x) {
    x = x + 0.f;
    return x == x ? x : -INFINITY;
  }
  __device__ __forceinline__ uint4 fetch(int e) const {  // V elements from e on
    if (e >= skip && e + V <= skip + n) return __ldg(reinterpret_cast<const uint4*>(base + e));
    uint32_t r[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (V == 4) {
        r[j] = 0xFF800000u;
        if (e + j >= skip && e + j < skip + n) r[j] = __ldg(reinterpret_cast<const uint32_t*>(base) + e + j);
      } else {
        uint32_t h[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int i = e + 2 * j + k;
          h[k] = 0xFF80u;
          if (i >= skip && i < skip + n) h[k] = __ldg(reinterpret_cast<const uint16_t*>(base) + i);
        }
        r[j] = h[0] | h[1] << 16;
      }
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
  }
  __device__ __forceinline__ void split(const uint4& v, float (&x)[V]) const {
    const uint32_t r[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (V == 4) {
        x[j] = __uint_as_float(r[j]);
      } else {
        x[2 * j] = __uint_as_float(r[j] << 16);
        x[2 * j + 1] = __uint_as_float(r[j] & 0xFFFF0000u);
      }
    }
    if (infinite)
#pragma unroll
      for (int j = 0; j < V; ++j) x[j] = x[j] == INFINITY ? 0.f : -INFINITY;
  }

  __device__ __forceinline__ float one(int e) const {  // element e of the run
    float x;
    if constexpr (V == 4) x = __ldg(reinterpret_cast<const float*>(base) + e);
    else x = __uint_as_float((uint32_t)__ldg(reinterpret_cast<const uint16_t*>(base) + e) << 16);
    return infinite ? (x == INFINITY ? 0.f : -INFINITY) : x;
  }

  // f(values, first element) for each step of this lane, in id order; all lanes
  // of a warp take the same steps.  kAhead steps are loaded at a time; kEarly: while
  // those before them are worked on (else all warps wait for memory together, and
  // then work together; where the work is short it is the other way round).
  template <int kAhead = 4, bool kEarly = false, typename F>
  __device__ __forceinline__ void steps(F f) const {
    constexpr int kStep = 32 * V;
    const int end = min((warp() + 1) * stretch(), skip + n);
    const auto load = [&](int at, uint4 (&v)[kAhead]) {  // at: the warp's first element
      const int e = at + lane() * V;
      if (at >= skip && at + kAhead * kStep <= end) {
#pragma unroll
        for (int j = 0; j < kAhead; ++j) v[j] = __ldg(reinterpret_cast<const uint4*>(base + e + j * kStep));
      } else {
#pragma unroll
        for (int j = 0; j < kAhead; ++j) v[j] = at + j * kStep < end ? fetch(e + j * kStep) : make_uint4(0, 0, 0, 0);
      }
    };
    int at = warp() * stretch();
    uint4 v[kAhead], next[kAhead];
    if (kEarly) load(at, next);
    for (; at < end; at += kAhead * kStep) {
      if (kEarly) {
#pragma unroll
        for (int j = 0; j < kAhead; ++j) v[j] = next[j];
        load(at + kAhead * kStep, next);
      } else {
        load(at, v);
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        if (at + j * kStep >= end) break;
        float x[V];
        split(v[j], x);
        f(x, at + lane() * V + j * kStep);
      }
    }
  }
  template <typename F>
  __device__ __forceinline__ void each_raw(F f) const {
    steps([&](const float (&x)[V], int e) {
#pragma unroll
      for (int j = 0; j < V; ++j) f(x[j], e + j);
    });
  }

  __device__ __forceinline__ void sync_cluster() const {
    if (ranks > 1) cluster_sync();
  }

  // Lane r gets the number that CTA r has at `p`, lanes past the cluster `none`.
  // (Shared memory of other CTAs is slow to read, about 20 bytes a clock: each
  // warp asks each CTA once.)
  __device__ __forceinline__ u64 of_ranks(const u64* p, u64 none) const {
    return lane() < ranks ? ld_peer_u64(p, lane()) : none;
  }

  // The largest of one number per thread of the cluster.
  __device__ u64 largest(u64 v) {
#pragma unroll
    for (int d = 16; d; d >>= 1) v = max_u64(v, __shfl_xor_sync(kAll, v, d));
    __syncthreads();
    if (lane() == 0) s.scratch[warp()] = v;
    __syncthreads();
    v = s.scratch[lane()];
#pragma unroll
    for (int d = 16; d; d >>= 1) v = max_u64(v, __shfl_xor_sync(kAll, v, d));
    if (ranks == 1) return v;
    u64* post = s.post[round++ & 1];
    if (threadIdx.x == 0) *post = v;
    cluster_sync();
    v = of_ranks(post, 0);
#pragma unroll
    for (int d = kMaxCluster / 2; d; d >>= 1) v = max_u64(v, __shfl_xor_sync(kAll, v, d));
    return __shfl_sync(kAll, v, 0);
  }

  // Sums of N numbers per thread over the cluster.
  template <int N>
  __device__ void sums(u64 (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = sum_warp(v[i]);
    __syncthreads();
    if (lane() == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) s.scratch[i * kWarpsPer + warp()] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = sum_warp(s.scratch[i * kWarpsPer + lane()]);
    if (ranks == 1) return;
    u64* post = s.post[round++ & 1];
    if (threadIdx.x == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) post[i] = v[i];
    cluster_sync();
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = sum_warp(of_ranks(post + i, 0));
  }

  // Inclusive running sums over the block's threads; *total gets the last.
  __device__ u64 scan(u64 v, u64* total) {
    u64 in = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const u64 x = __shfl_up_sync(kAll, in, d);
      if (lane() >= d) in += x;
    }
    __syncthreads();
    if (lane() == 31) s.scratch[warp()] = in;
    __syncthreads();
    const u64 t = s.scratch[lane()];
    *total = sum_warp(t);
    return in + sum_warp(lane() < warp() ? t : 0);
  }
  __device__ uint32_t scan(uint32_t v, uint32_t* total) {
    uint32_t* room = reinterpret_cast<uint32_t*>(s.scratch);
    const uint32_t in = scan_warp(v);
    __syncthreads();
    if (lane() == 31) room[warp()] = in;
    __syncthreads();
    const uint32_t t = room[lane()];
    *total = __reduce_add_sync(kAll, t);
    return in + __reduce_add_sync(kAll, lane() < warp() ? t : 0);
  }
  // The sum before this thread's (never by a subtraction: of a small sum before
  // large ones it would leave the large ones' rounding).
  __device__ float before_float(float v, float* total, float* room) {
    float in = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const float x = __shfl_up_sync(kAll, in, d);
      if (lane() >= d) in += x;
    }
    __syncthreads();
    if (lane() == 31) room[warp()] = in;
    __syncthreads();
    float t = room[lane()];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const float x = __shfl_up_sync(kAll, t, d);
      if (lane() >= d) t += x;
    }
    *total = __shfl_sync(kAll, t, 31);
    const float before = __shfl_sync(kAll, t, warp() ? warp() - 1 : 0);
    const float left = __shfl_up_sync(kAll, in, 1);
    return (lane() ? left : 0.f) + (warp() ? before : 0.f);
  }

  __device__ void clear_bins() {
    __syncthreads();
    reinterpret_cast<uint4*>(s.count)[threadIdx.x] = make_uint4(0, 0, 0, 0);
    __syncthreads();
  }

  // Sum the first `words` of every CTA's s.count: each CTA sums a slice of them in
  // place, and merged() finds it there.  (All of them read by every CTA would be
  // four times as much with eight CTAs; with two it is as much, and two read all.)
  __device__ void merge(int words) {
    __syncthreads();
    if (ranks == 1) return;
    cluster_sync();
    if (ranks == 2) return;
    const int slice = words / ranks;
    for (int i = threadIdx.x; i < slice; i += kThreads) {
      uint32_t* at = s.count + rank * slice + i;
      uint32_t v[kMaxCluster], sum = 0;
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) v[r] = r < ranks ? ld_peer_u32(at, r) : 0;
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) sum += v[r];
      *at = sum;
    }
    cluster_sync();
  }
  __device__ __forceinline__ uint32_t merged(int words, int i) const {
    if (ranks <= 2) return s.count[i] + (ranks == 2 ? ld_peer_u32(s.count + i, rank ^ 1) : 0);
    return ld_peer_u32(s.count + i, i / (words / ranks));
  }

  // Bins of all finite logits, merged: this thread's counts.  (The bins are clear.)
  __device__ uint4 histogram() {
    each_raw([&](float x, int) {
      const uint32_t b = w.bin(x);
      if (x > -INFINITY) atomicAdd(&s.count[b], 1u);
    });
    merge(kBins);
    const uint32_t* mine = s.count + kPer * threadIdx.x;
    if (ranks > 2) return ld_peer_u32x4(mine, threadIdx.x / (kThreads / ranks));
    uint4 c = *reinterpret_cast<const uint4*>(mine);
    if (ranks == 2) {
      const uint4 other = ld_peer_u32x4(mine, rank ^ 1);
      c = make_uint4(c.x + other.x, c.y + other.y, c.z + other.z, c.w + other.w);
    }
    return c;
  }

  // Put the entries that visit(push) pushes in the CTAs into one list, in every
  // CTA of the cluster (or the first only), the largest first, with n_extra more
  // that are alike.  Returns how many there are; they are known to be kCap at
  // most.
  template <typename F>
  __device__ int gather(F visit, bool first_only, u64 extra, uint32_t n_extra) {
    __syncthreads();
    if (threadIdx.x == 0) s.n_list = 0;
    __syncthreads();
    visit([&](u64 entry) {
      const uint32_t at = atomicAdd(&s.n_list, 1u);
      if (at < kCap) s.list[at] = entry;
    });
    __syncthreads();
    sync_cluster();
    int total = 0;
    if (!first_only || rank == 0) {
      // the lists end to end, in rank order: thread i takes entry i
      const int theirs = lane() < ranks ? (int)ld_peer_u32(&s.n_list, lane()) : 0;
      int from = 0, at = 0;
      for (int r = 0; r < ranks; ++r) {
        if ((int)threadIdx.x >= total) from = r, at = threadIdx.x - total;
        total += __shfl_sync(kAll, theirs, r);
      }
      const int listed = min(total, kCap), i = threadIdx.x;
      if (i < listed) s.order[i] = ranks == 1 ? s.list[at] : ld_peer_u64(&s.list[at], from);
      total = min(listed + (int)n_extra, kCap);
      if (i >= listed && i < total) s.order[i] = extra;
      __syncthreads();
      sort(total, true);
    }
    return total;
  }

  // Order s.order[0 .. total), total <= kCap.  Each warp orders 32 entries in a
  // bitonic network; then runs are merged in pairs, an entry's place in the other
  // run found by bisection.  (One network over all entries took 12 kclk for 400 of
  // them, 7 so.)
  __device__ void sort(int total, bool falling) {
    const int i = threadIdx.x;
    u64 v = i < total ? (falling ? s.order[i] : ~s.order[i]) : 0;  // (no entry is 0 here)
    if (warp() * 32 < total) {
#pragma unroll
      for (int k = 2; k <= 32; k <<= 1)
#pragma unroll
        for (int j = k >> 1; j; j >>= 1) {
          const u64 other = __shfl_xor_sync(kAll, v, j);
          v = ((i & k) == 0 || k == 32) == ((i & j) == 0) ? max_u64(v, other) : min_u64(v, other);
        }
    }
    int size = 32;
    for (; size < total; size *= 2) {}
    for (int length = 32; length < size; length *= 2) {
      __syncthreads();
      if (i < size) s.order[i] = v;
      __syncthreads();
      int place = 0;
      if (i < size) {
        const u64* run = s.order + ((i & -length) ^ length);
        const bool second = i & length;  // (equal entries of the first run go first)
        const auto before = [&](u64 other) { return second ? other >= v : other > v; };
        int at = 0;  // entries of the other run that go before v
        for (int d = length / 2; d; d /= 2) at += before(run[at + d - 1]) ? d : 0;
        at += before(run[at]);
        place = (i & -(2 * length)) + (i & (length - 1)) + at;
      }
      __syncthreads();
      if (i < size) s.order[place] = v;
      __syncthreads();
      if (i < size) v = s.order[i];
    }
    __syncthreads();
    if (i < total) s.order[i] = falling ? v : ~v;
    __syncthreads();
  }

  // Logits of which `inside` have a key in lo .. hi, with before_c logits and
  // before_m weight above.
  struct Cut {
    u64 before_c, before_m, inside;
    uint32_t lo, hi;
    __device__ __forceinline__ bool in(uint32_t k) const { return k >= lo && k <= hi; }
    __device__ __forceinline__ int shift() const {  // of kFine bins of keys, the first at hi
      const int width = 32 - __clz(hi - lo);
      return width > 10 ? width - 10 : 0;
    }
  };
  __device__ __forceinline__ void add_fine(const Cut& cut, uint32_t k, uint32_t times, bool by_mass) {
    const uint32_t b = (cut.hi - k) >> cut.shift();
    atomicAdd(&s.count[b], times);
    if (!by_mass) return;
    const u64 v = w(of_key(k));
#pragma unroll
    for (int j = 0; j < 3; ++j) {
      const uint32_t d = (uint32_t)(v >> (j * kPiece)) & ((1u << kPiece) - 1);
      if (d) atomicAdd(&s.count[(j + 1) * kFine + b], d * times);
    }
  }
  // From the fine bins of `cut`, filled by every CTA: the one in which the
  // running count, or weight, reaches target.
  __device__ void narrow_to_bin(bool by_mass, u64 target, Cut* cut) {
    const int words = by_mass ? 4 * kFine : kFine;
    merge(words);
    const u64 c = merged(words, threadIdx.x);
    u64 m = 0;
    if (by_mass)
#pragma unroll
      for (int j = 1; j < 4; ++j) m += (u64)merged(words, j * kFine + threadIdx.x) << ((j - 1) * kPiece);
    // (there is such a bin; were there none, every CTA had to agree on one)
    if (threadIdx.x == 0) {
      s.found[0] = 0;
      s.found[1] = cut->before_c;
      s.found[2] = cut->before_m;
      s.found[3] = 0;
    }
    u64 total;
    const u64 ci = scan(c, &total) + cut->before_c;
    const u64 mi = by_mass ? scan(m, &total) + cut->before_m : 0;
    const u64 now = by_mass ? mi : ci, was = by_mass ? mi - m : ci - c;
    if (was < target && (now >= target || threadIdx.x == kFine - 1)) {
      s.found[0] = threadIdx.x;
      s.found[1] = ci - c;
      s.found[2] = mi - m;
      s.found[3] = c;
    }
    __syncthreads();
    const int shift = cut->shift();
    const uint32_t b = (uint32_t)s.found[0], top = cut->hi, low = cut->lo;
    cut->before_c = s.found[1];
    cut->before_m = s.found[2];
    cut->inside = s.found[3];
    cut->hi = top - (b << shift);
    const u64 depth = ((u64)(b + 1) << shift) - 1;
    cut->lo = top - low > depth ? (uint32_t)(top - depth) : low;
    __syncthreads();
    sync_cluster();  // (the bins are cleared only after every CTA has read them)
  }
  // Narrow the cut down to kFew logits, or to a single key.  visit(f) calls f
  // with the key of every logit that takes part; `extra` more have key `top`.
  // `target` counts logits, or (by_mass) weight, of the whole falling order.
  template <typename F>
  __device__ void narrow(F visit, bool by_mass, u64 target, uint32_t top, uint32_t extra, Cut* cut) {
    // (a cut takes ten bits off the keys that are left: four at most)
    for (int round = 0; round < 4 && cut->inside > kFew && cut->hi != cut->lo; ++round) {
      clear_bins();
      visit([&](uint32_t k) {
        if (cut->in(k)) add_fine(*cut, k, 1, by_mass);
      });
      if (extra && cut->in(top) && rank == 0 && threadIdx.x == 0) add_fine(*cut, top, extra, by_mass);
      narrow_to_bin(by_mass, target, cut);
    }
  }
  // Keys that hold all logits of bins b0 .. b1 (the borders lie a hundredth of a
  // bin, a ten-thousandth and two keys further out than the arithmetic needs).
  __device__ __forceinline__ void keys_of_bins(uint32_t b0, uint32_t b1, Cut* cut) const {
    const uint32_t top = key_of(w.max), bottom = key_of(-FLT_MAX);
    const float high = (w.top - ((float)b0 - 0.51f) / w.per_bin * 0.9999f) / w.scale;
    const float low = (w.top - ((float)b1 + 0.51f) / w.per_bin * 1.0001f) / w.scale;
    cut->hi = b0 == 0 || !(high < w.max && high > -FLT_MAX) ? top : min(key_of(high) + 2, top);
    cut->lo = b1 == kBins - 1 || !(low > -FLT_MAX) ? bottom : max(key_of(low) - 2, bottom);
  }

  // The place in s.order[0 .. n) at which the running weight, `before` above
  // it, reaches target (it does).
  __device__ int crossing(int n, u64 before, u64 target) {
    const u64 v = (int)threadIdx.x < n ? w(of_key((uint32_t)(s.order[threadIdx.x] >> 32))) : 0;
    u64 total;
    if (threadIdx.x == 0) s.found[0] = n > 0 ? n - 1 : 0;
    const u64 upto = scan(v, &total) + before;
    if (upto - v < target && upto >= target) s.found[0] = threadIdx.x;
    __syncthreads();
    const int j = (int)s.found[0];
    __syncthreads();
    return j;
  }

  // The threshold at place j of the n entries of s.order: its key, how many of
  // its ties (all of them are in the list) lie at or before j, and whether none
  // lies behind.
  __device__ void threshold_at(int n, int j, uint32_t* key, uint32_t* ties, bool* whole) {
    const uint32_t k = n > 0 ? (uint32_t)(s.order[j] >> 32) : 0;
    const int above = __syncthreads_count((int)threadIdx.x < j && (uint32_t)(s.order[threadIdx.x] >> 32) > k);
    *key = k;
    *ties = (uint32_t)(j + 1 - above);
    *whole = j + 1 >= n || (uint32_t)(s.order[j + 1] >> 32) != k;
  }
};

// floor(f total) of a float 0 <= f < 1, exactly: f is a whole number of 24 bits
// times a power of two.
__device__ __forceinline__ u64 floor_share(float f, u64 total, bool* exact) {
  const uint32_t u = __float_as_uint(f), e = u >> 23;
  const u64 m = e ? (u & 0x7FFFFFu) | 0x800000u : u;
  const uint32_t s = 150 - (e ? e : 1);  // f = m 2^-s, s >= 24
  const u64 lo = total * m, hi = __umul64hi(total, m);
  const u64 out = s < 64 ? hi << (64 - s) | lo >> s : (s < 128 ? hi >> (s - 64) : 0);
  *exact = s < 64 ? (lo << (64 - s)) == 0 : (lo | (s == 64 ? 0 : hi << (128 - min(s, 128u)))) == 0 && s < 128;
  return out;
}
// The least weight that is `share` of total, and no less than one unit.
__device__ __forceinline__ u64 share_of(float share, u64 total) {
  bool exact;
  const u64 f = floor_share(share, total, &exact);
  return max_u64(f + !exact, 1);
}

// The row that this CTA takes where the rows are more than the SMs: of each 1024
// in turn, those that take long first (a batch of 256 rows of 100 003, every kind
// in it, took 110 us in the order in which they lie, 78 so; finding the row
// takes 1 of those).  Such a row takes 73 us with top-p alone, 37 to 45 with a top-k of
// hundreds, 30 with any other cut or none, 11 without a draw.
__device__ int64_t heavy_first(const uw_sample_args& a, Shared& s, int64_t r) {
  const int64_t first = r / kThreads * kThreads, mine = first + threadIdx.x;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int weight = -1;
  if (mine < a.n_rows) {
    const float t = a.temperature_dev ? a.temperature_dev[mine] : 1.f, share = a.top_p_dev ? a.top_p_dev[mine] : 1.f;
    const int k = a.top_k_dev ? a.top_k_dev[mine] : 0;
    const bool cut_k = k > 0 && k < a.vocab;
    weight = !(t > 0.f) ? 0 : (cut_k ? (k > kFew ? 2 : 1) : (share < 1.f ? 3 : 1));
  }
  int at = (int)(r - first), kind = 3;  // the at-th of the kind
  for (; kind > 0; --kind) {
    const int n = __syncthreads_count(weight == kind);
    if (at < n) break;
    at -= n;
  }
  const uint32_t votes = __ballot_sync(kAll, weight == kind);
  if (lane == 0) s.count[warp] = __popc(votes);
  __syncthreads();
  const int before = __reduce_add_sync(kAll, lane < warp ? s.count[lane] : 0) + __popc(votes & ((1u << lane) - 1));
  if (weight == kind && before == at) s.ends[0] = threadIdx.x;
  __syncthreads();
  return first + s.ends[0];
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 1) sample_kernel(const __grid_constant__ SampleParams p) {
  extern __shared__ __align__(16) unsigned char raw[];
  Shared& s = *reinterpret_cast<Shared*>(raw);
  const uw_sample_args& a = p.a;
  const int ranks = (int)(gridDim.x / a.n_rows), rank = blockIdx.x % ranks;
  const int start = min(rank * p.run, a.vocab);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float* listed = reinterpret_cast<float*>(raw + kSharedBytes) + threadIdx.x;  // [p.listed + V][kThreads]
  if (threadIdx.x < 512) {
    const double e = exp2((double)threadIdx.x * (-1.0 / 512.0)) * 2147483648.0;
    s.table[threadIdx.x] = make_uint2((uint32_t)__double2uint_rn(e) - Weights::kWholeBits, __float_as_uint((float)e));
  }
  pdl_wait();
  pdl_release();
  int64_t r = blockIdx.x / ranks;
  if (p.ordered) r = heavy_first(a, s, r);
  const float t = a.temperature_dev ? a.temperature_dev[r] : 1.f;
  const int k = a.top_k_dev ? a.top_k_dev[r] : 0;
  const float share = a.top_p_dev ? a.top_p_dev[r] : 1.f, min_p = a.min_p_dev ? a.min_p_dev[r] : 0.f;
  float u = a.u_dev[r];
  const T* src = static_cast<const T*>(a.logits_dev) + r * a.row_stride + start;
  const int skip = (int)((reinterpret_cast<uintptr_t>(src) & 15) / sizeof(T));
  Row<T> row{s, src - skip, skip, min(p.run, a.vocab - start), start - skip, rank, ranks, 0, false, {}};
  constexpr int V = Row<T>::V;

  row.clear_bins();  // (for the histogram)
  // the largest logit (a NaN loses against every other)
  float best = -INFINITY;
  row.steps([&](const float (&x)[V], int) {
#pragma unroll
    for (int j = 0; j < V; ++j) best = fmaxf(best, x[j]);
  });
  const uint32_t best_key = __reduce_max_sync(kAll, key_of(best + 0.f));
  float peak = of_key((uint32_t)row.largest(best_key));
  const auto choose = [&](int64_t id, float prob) {
    a.ids_dev[r] = id;
    if (a.prob_dev) a.prob_dev[r] = prob;
  };
  if (peak == -INFINITY || !(t > 0.f)) {
    if (peak == -INFINITY) {
      if (rank == 0 && threadIdx.x == 0) choose(-1, 0.f);
    } else {  // its lowest id, in a warp that has it
      u64 id = 0;
      if (of_key(best_key) == peak)
        row.each_raw([&](float x, int e) { id = x == peak ? max_u64(id, (uint32_t)~(row.id0 + e)) : id; });
      id = row.largest(id);
      if (rank == 0 && threadIdx.x == 0) choose((int64_t)(uint32_t)~(uint32_t)id, 1.f);
    }
    row.sync_cluster();
    return;
  }
  if (peak == INFINITY) {
    row.infinite = true;
    peak = 0.f;
  }
  row.w.set(peak, t);
  row.w.table = s.table;

  const u64 least = min_p > 0.f ? (u64)ceil(fmin((double)min_p, 1.0) * (double)(u64(1) << kFixBits)) : 0;
  u = u > 0.f ? fminf(u, 0.99999994f) : 0.f;
  bool cut_k = k > 0 && k < a.vocab;
  const bool cut_p = share < 1.f;
  const float part = fmaxf(share, 0.f);

  const auto across = [&](u64 mine, u64* total) {  // sums before this warp, over the cluster's warps
    __syncthreads();
    if (lane == 0) s.scratch[warp] = mine;
    __syncthreads();
    u64 v = s.scratch[lane], before = sum_warp(lane < warp ? v : 0);
    v = sum_warp(v);
    if (ranks > 1) {
      u64* post = s.post[row.round++ & 1];
      if (threadIdx.x == 0) *post = v;
      cluster_sync();
      v = row.of_ranks(post, 0);
      before += sum_warp(lane < rank ? v : 0);
      v = sum_warp(v);
    }
    *total = v;
    return before;
  };
  uint32_t key = 0, ties = 0;  // keys above `key` stay, and the first `ties` equal to it
  bool all_ties = false;       // which are known to be all of them
  u64 sum = 0;           // of this thread's kept weights, and whether that is done
  bool summed = false;
  u64 tie_from = 0;      // ties before this warp's stretch
  // (exact sums for top-p count every weight; without it those under min_p, by
  // a margin far above the rounding of y, need no more than a comparison)
  if (!cut_p && min_p > 0.f)
    row.w.lower(fminf(40.5f, 0.01f - __log2f(fminf(min_p, 1.f))));
  // the weights of all logits, this thread's
  const uint32_t one = blockDim.y;  // 1
  const auto weigh_all_of = [&]() {
    u64 all = 0;
    row.template steps<2, true>([&](const float (&x)[V], int) {
      uint32_t m[V], at[V];
#pragma unroll
      for (int j = 0; j < V; ++j) m[j] = row.w.parts(x[j], &at[j]);
      if (__any_sync(kAll, row.w.is_near(x))) {
#pragma unroll
        for (int j = 0; j < V; ++j) all += Weights::wide(m[j], at[j]);
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j) add_wide(&all, Weights::small(m[j], at[j]), one);
      }
    });
    return all;
  };
  if (cut_k || cut_p) {
    const uint4 bins = row.histogram();
    const uint32_t counts[kPer] = {bins.x, bins.y, bins.z, bins.w};
    uint32_t logits;
    const uint32_t mine = bins.x + bins.y + bins.z + bins.w, from0 = row.scan(mine, &logits) - mine;
    cut_k = cut_k && (uint32_t)k < logits;
    if (threadIdx.x == 0) {
      s.ends[0] = kBins - 1;
      s.ends[1] = 0;
      s.ends[2] = 0;
      s.ends[3] = kBins - 1;
      s.found[3] = 0;
    }
    __syncthreads();
    // bin of the k-th logit, and the count before it
    if (cut_k) {
      uint32_t at = from0;
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        if (at < (uint32_t)k && at + counts[j] >= (uint32_t)k) {
          s.ends[0] = threadIdx.x * kPer + j;
          s.ends[1] = at;
          s.found[3] = counts[j];
        }
        at += counts[j];
      }
    }
    __syncthreads();
    const uint32_t bin_k = s.ends[0], before_k = s.ends[1];
    const u64 inside_k = s.found[3];
    uint32_t b0 = 0, b1 = bin_k;  // bins in which the prefix may end
    u64 down_to = logits;         // logits in bins up to b1, and above b0
    u64 above_b0 = 0;
    if (cut_p && !(cut_k && before_k + inside_k <= kCap)) {
      // Bounds of the running weight from the counts: the weights of bin b lie
      // between those of its two borders (a hundredth of a bin allows for the
      // rounding of bin(), a ten-thousandth for these sums).
      float low[kPer], high[kPer], lows = 0.f, highs = 0.f;
      const float step = __expf(-1.f / kPerUnit), wide = __expf(1.02f / kPerUnit);
      float border = __expf(-((float)(threadIdx.x * kPer) + 0.51f) / kPerUnit);  // the lower one's weight
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const uint32_t b = threadIdx.x * kPer + j;
        u64 m = counts[j];
        if (cut_k) m = b < bin_k ? m : (b == bin_k ? (u64)k - before_k : 0);
        low[j] = b == kBins - 1 ? 0.f : (float)m * border;
        high[j] = b == 0 ? (float)m : (float)m * (border * wide);
        border *= step;
        lows += low[j];
        highs += high[j];
      }
      float low_all, high_all;
      float l = row.before_float(lows, &low_all, s.bound);
      float h = row.before_float(highs, &high_all, s.bound + kWarpsPer);
      const float from = part * low_all * 0.9999f, to = part * high_all * 1.0001f;
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        // (the sums' rounding only widens what is taken: the smallest and the
        // largest bin stand)
        if ((h + high[j]) * 1.0001f >= from) atomicMin(&s.ends[3], threadIdx.x * kPer + j);
        if (l * 0.9999f <= to && counts[j]) atomicMax(&s.ends[2], threadIdx.x * kPer + j);
        l += low[j];
        h += high[j];
      }
      __syncthreads();
      b0 = min(s.ends[3], bin_k);
      b1 = min(s.ends[2], bin_k);
      b0 = min(b0, b1);
      uint32_t at = from0;
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const uint32_t b = threadIdx.x * kPer + j;
        if (b == b0) s.found[1] = at;
        at += counts[j];
        if (b == b1) s.found[2] = at;
      }
      __syncthreads();
      above_b0 = s.found[1];
      down_to = s.found[2];
    }
    row.sync_cluster();  // (every CTA has read the merged bins)

    // With top-k the list reaches to its end, for top-p's total; else to b1.
    const uint32_t deep = cut_k ? bin_k : b1;
    const u64 n_deep = cut_k ? before_k + inside_k : down_to;
    if (n_deep <= kCap) {
      u64 total = 0;
      if (cut_p && !cut_k) {
        u64 one[1] = {weigh_all_of()};
        row.sums(one);
        total = one[0];
      }
      const float from = row.w.lowest(Weights::limit((int)deep));
      const int n = row.gather(
          [&](auto push) {
            row.steps([&](const float (&x)[V], int e) {
              bool any = false;
#pragma unroll
              for (int j = 0; j < V; ++j) any |= x[j] >= from;
              if (any)
#pragma unroll
                for (int j = 0; j < V; ++j)
                  if (x[j] >= from)
                    push((u64)key_of(Row<T>::clean(x[j])) << 32 | (uint32_t)~(row.id0 + e + j));
            });
          },
          true, 0, 0);
      if (rank == 0) {
        // entry i of the falling order (equal logits by rising id)
        const int i = threadIdx.x;
        const u64 entry = i < n ? s.order[i] : 0;
        const u64 v = i < (cut_k ? min(n, k) : n) ? row.w(of_key((uint32_t)(entry >> 32))) : 0;
        u64 all;
        const u64 sums = row.scan(v, &all);
        bool stay = v > 0 && v >= least;
        if (cut_p) stay = stay && sums - v < share_of(part, cut_k ? all : total);
        __syncthreads();
        // The kept ones are the first of the order (weights fall with it but for
        // their last bits, which do not reopen it); now by rising id.
        const int kept = __syncthreads_count(stay);
        stay = i < kept;
        s.order[i] = stay ? (u64)(uint32_t)~(uint32_t)entry << 32 | (uint32_t)i : ~u64(0);
        s.list[i] = v;
        __syncthreads();
        row.sort(kept, false);
        const u64 mine = i < kept ? s.order[i] : 0;
        const u64 weight = i < kept ? s.list[(uint32_t)mine] : 0;
        u64 kept_all;
        const u64 to = row.scan(weight, &kept_all);
        bool exact;
        const u64 target = floor_share(u, kept_all, &exact);
        if (to - weight <= target && target < to)
          choose((int64_t)(mine >> 32), (float)((double)weight / (double)kept_all));
      }
      row.sync_cluster();
      return;
    }

    // The open bins hold every logit that may be the end of a prefix.  One pass
    // sums the weights above them and copies the keys inside to shared memory, a
    // list per thread (a list per warp, its places found by votes: 86 kclk for this
    // pass over a flat row of 100 000 in place of 77); all that follows goes by the
    // lists.  Where they do not hold them, it goes over the row again.
    const uint32_t first = cut_p ? b0 : bin_k, last = cut_k ? bin_k : b1;
    const float from_up = row.w.lowest(Weights::limit((int)first - 1)), from_in = row.w.lowest(Weights::limit((int)last));
    const bool weigh_all = cut_p && !cut_k;
    u64 every = 0, above = 0;
    int filled = 0;
    bool over = false;
    row.template steps<2, true>([&](const float (&x)[V], int) {
      bool up[V], any = weigh_all;
#pragma unroll
      for (int j = 0; j < V; ++j) any |= up[j] = x[j] >= from_up;
      if (__any_sync(kAll, any)) {
        uint32_t m[V], at[V];
#pragma unroll
        for (int j = 0; j < V; ++j) m[j] = row.w.parts(x[j], &at[j]);
        if (__any_sync(kAll, row.w.is_near(x))) {
#pragma unroll
          for (int j = 0; j < V; ++j) {
            const u64 v = Weights::wide(m[j], at[j]);
            every += v;
            if (up[j]) above += v;
          }
        } else {
#pragma unroll
          for (int j = 0; j < V; ++j) {
            const uint32_t v = Weights::small(m[j], at[j]);
            add_wide(&every, v, one);
            if (up[j]) add_wide(&above, v, one);
          }
        }
        if (least)
#pragma unroll
          for (int j = 0; j < V; ++j) {
            const u64 v = Weights::wide(m[j], at[j]);
            sum += up[j] && v >= least ? v : 0;
          }
      }
      // (a store for each, of which those inside stay: no branches)
      over |= filled > p.listed;
      filled = min(filled, p.listed);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        listed[filled * kThreads] = x[j];
        filled += x[j] >= from_in && !up[j];
      }
    });
    over |= filled > p.listed;
    filled = min(filled, p.listed);
    if (!least) sum = above;
    u64 sums[3] = {over, above, every};
    row.sums(sums);
    const bool fits = sums[0] == 0;
    // f(key) for the logits of the open bins
    const auto visit = [&](auto f) {
      if (fits) {
        for (int i = 0; i < filled; ++i) f(key_of(listed[i * kThreads] + 0.f));
      } else {
        row.each_raw([&](float raw, int) {
          if (raw >= from_in && !(raw >= from_up)) f(key_of(Row<T>::clean(raw)));
        });
      }
    };
    if (cut_k) {
      typename Row<T>::Cut cut = {before_k, 0, inside_k};
      row.keys_of_bins(bin_k, bin_k, &cut);
      const auto visit_k = [&](auto f) {
        visit([&](uint32_t q) {
          if (cut.in(q) && row.w.bin(of_key(q)) == bin_k) f(q);
        });
      };
      row.narrow(visit_k, false, (u64)k, 0, 0, &cut);
      if (cut.inside > kFew) {
        key = cut.hi;
        ties = (uint32_t)((u64)k - cut.before_c);
      } else {
        const int n = row.gather([&](auto push) { visit_k([&](uint32_t q) { push((u64)q << 32); }); }, false, 0, 0);
        row.threshold_at(n, (int)((u64)k - cut.before_c) - 1, &key, &ties, &all_ties);
        row.sync_cluster();
      }
    }
    if (cut_p) {
      const uint32_t top = key, top_ties = ties;
      const auto visit_p = [&](auto f) {
        visit([&](uint32_t q) {
          if (q > top) f(q);
        });
      };
      // (without top-k all of the weight is known, and how many take part)
      u64 part_sums[2] = {down_to - above_b0, sums[2]};
      if (cut_k) {
        part_sums[0] = part_sums[1] = 0;
        visit_p([&](uint32_t q) {
          ++part_sums[0];
          part_sums[1] += row.w(of_key(q));
        });
        row.sums(part_sums);
      }
      typename Row<T>::Cut cut = {above_b0, sums[1], part_sums[0] + top_ties};
      row.keys_of_bins(first, last, &cut);
      const u64 total = weigh_all ? part_sums[1] : cut.before_m + part_sums[1] + top_ties * row.w(of_key(top));
      const u64 target = share_of(part, total);
      row.narrow(visit_p, true, target, top, top_ties, &cut);
      if (cut.inside > kFew) {
        key = cut.hi;
        const u64 one = row.w(of_key(key));
        ties = (uint32_t)((target - cut.before_m + one - 1) / one);
        all_ties = false;
      } else {
        const int n = row.gather(
            [&](auto push) {
              visit_p([&](uint32_t q) {
                if (cut.in(q)) push((u64)q << 32);
              });
            },
            false, (u64)top << 32, cut.in(top) ? top_ties : 0);
        bool whole = false;
        row.threshold_at(n, row.crossing(n, cut.before_m, target), &key, &ties, &whole);
        // (top-k's own threshold: whether all of its ties stay was settled there)
        all_ties = whole && (key != top || all_ties);
        row.sync_cluster();
      }
    }
    if (fits) {
      // the kept weights of each warp, from its list
      uint32_t tied_here = 0;
      visit([&](uint32_t q) {
        tied_here += q == key;
        const u64 v = q > key ? row.w(of_key(q)) : 0;
        sum += v >= least ? v : 0;
      });
      tied_here = __reduce_add_sync(kAll, tied_here);
      u64 keep = tied_here;
      if (!all_ties) {
        u64 total;
        tie_from = across(tied_here, &total);
        keep = tie_from >= ties ? 0 : min_u64(ties - tie_from, tied_here);
      }
      const u64 one = row.w(of_key(key));
      if (lane == 0 && one >= least) sum += keep * one;
      summed = true;
    } else {
      sum = 0;
    }
  }

  // Ties that stay are the lowest ids: where not all do, count those before
  // each warp's stretch.
  const float edge = ties ? of_key(key) : -INFINITY;  // (comparisons of floats: NaN fails them, zeros are equal)
  if (!ties) all_ties = true;
  if (!all_ties && !summed) {
    uint32_t mine = 0;
    row.each_raw([&](float x, int) { mine += x == edge; });
    mine = __reduce_add_sync(kAll, mine);
    u64 total;
    tie_from = across(mine, &total);
    all_ties = total <= ties;
  }
  // The kept weights, summed per warp.  Where few logits are kept, a step of
  // 32 x V neighbours is weighed only if it holds one of them.
  const bool some_ties = ties != 0 && all_ties, sparse = ties != 0 || least != 0;
  u64 tied = tie_from;
  if (!summed && !sparse) {
    sum = weigh_all_of();
  } else if (!summed) row.template steps<2>([&](const float (&x)[V], int) {
    bool stay[V], any = false;
#pragma unroll
    for (int j = 0; j < V; ++j) stay[j] = x[j] > edge || (some_ties && x[j] == edge);
    if (!all_ties) {
      uint32_t mine = 0;
#pragma unroll
      for (int j = 0; j < V; ++j) mine += x[j] == edge;
      if (__any_sync(kAll, mine != 0)) {
        const uint32_t upto = scan_warp(mine);
        u64 at = tied + upto - mine;  // this lane's first tie, among the row's
        tied += __shfl_sync(kAll, upto, 31);
#pragma unroll
        for (int j = 0; j < V; ++j)
          if (x[j] == edge) stay[j] = at++ < ties;
      }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      stay[j] = stay[j] && row.w.weighs(x[j]);
      any |= stay[j];
    }
    if (!__any_sync(kAll, any)) return;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const u64 v = row.w(x[j]);
      sum += stay[j] && v >= least ? v : 0;
    }
  });
  sum = sum_warp(sum);
  if (threadIdx.x == 0) s.ends[0] = kAll;
  u64 total;
  const u64 from = across(sum, &total);
  bool exact;
  const u64 target = floor_share(u, total, &exact);  // the choice's running sum exceeds this
  if (from <= target && target < from + sum && lane == 0) {
    s.ends[0] = warp;
    s.found[0] = from;
    s.found[1] = tie_from;
  }
  __syncthreads();
  // The warp whose stretch holds the choice: all threads of its CTA go through
  // that stretch again, a few neighbours each.
  const uint32_t owner = s.ends[0];
  if (owner != kAll) {
    const u64 before = s.found[0], ties_before = s.found[1];
    const int e0 = max((int)owner * row.stretch(), row.skip), e1 = min(((int)owner + 1) * row.stretch(), row.skip + row.n);
    const int each = (e1 - e0 + kThreads - 1) / kThreads;
    const int i0 = e0 + threadIdx.x * each, i1 = min(i0 + each, e1);
    u64 tie = 0;
    if (!all_ties) {
      uint32_t mine = 0, unused;
      for (int i = i0; i < i1; ++i) mine += row.one(i) == edge;
      tie = ties_before + row.scan(mine, &unused) - mine;
    }
    const u64 first_tie = tie;
    const auto weight = [&](int i) -> u64 {
      const float x = row.one(i);
      const bool stay = x > edge || (some_ties && x == edge) || (!all_ties && x == edge && tie++ < ties);
      const u64 v = stay ? row.w(x) : 0;
      return v >= least ? v : 0;
    };
    u64 mine = 0, unused;
    for (int i = i0; i < i1; ++i) mine += weight(i);
    const u64 upto = before + row.scan(mine, &unused);
    if (upto - mine <= target && target < upto) {
      u64 run = upto - mine;
      tie = first_tie;
      for (int i = i0; i < i1; ++i) {
        const u64 v = weight(i);
        run += v;
        if (run > target) {
          choose(row.id0 + i, (float)((double)v / (double)total));
          break;
        }
      }
    }
  }
  row.sync_cluster();
}

// CTAs per row: as many as give each SM one CTA, while each has work for its
// threads.
int cluster_for(const uw_sample_args& a, int sms) {
  int c = 1;
  while (c < kMaxCluster && a.n_rows * c * 2 <= sms && a.vocab / c >= 8 * kThreads) c *= 2;
  return c;
}

template <typename T>
cudaError_t launch_sample(const uw_sample_args& a, int sms, cudaStream_t s) {
  const int c = cluster_for(a, sms);
  SampleParams p;
  p.a = a;
  p.run = (a.vocab + c - 1) / c;
  p.ordered = a.n_rows > sms;
  // Room for a third of the logits, as long as that is there.  (No more than
  // that: what is left of the SM's memory is the cache that holds loads in flight.
  // 256 rows of 100 003 without a draw took 29 us with 38, 24 with this.)
  p.listed = std::min(kMaxListed, std::max(16, p.run / (3 * kThreads)));
  const size_t smem = shared_bytes(p.listed, Row<T>::V);
  // The limit belongs to the kernel and the device, not to this call: it is always set to the most that
  // any call needs, so that no other thread's call lowers it between here and the launch.
  const cudaError_t e = cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)shared_bytes(kMaxListed, Row<T>::V));
  if (e != cudaSuccess) return e;
  return launch_pdl_cluster(sample_kernel<T>, dim3((unsigned)(a.n_rows * c)), c, dim3(kThreads), smem, s, p);
}

}  // namespace
}  // namespace uw

using namespace uw;

extern "C" uw_status uw_sample(const uw_sample_args* a, void* stream) {
  if (!a) return UW_ERR_ARG;
  if (a->vocab < 1 || a->vocab > kMaxVocab || a->n_rows < 0 || a->n_rows > (int64_t(1) << 27)) return UW_ERR_SHAPE;
  if (a->n_rows == 0) return UW_OK;
  if (!a->logits_dev || !a->u_dev || !a->ids_dev) return UW_ERR_ARG;
  if (a->row_stride < 0 || (a->n_rows > 1 && a->row_stride < a->vocab)) return UW_ERR_ARG;
  if (!aligned(a->logits_dev, a->logits_bf16 ? 2 : 4) || !aligned(a->u_dev, 4) || !aligned(a->ids_dev, 8) ||
      !aligned(a->temperature_dev, 4) || !aligned(a->top_k_dev, 4) || !aligned(a->top_p_dev, 4) ||
      !aligned(a->min_p_dev, 4) || !aligned(a->prob_dev, 4))
    return UW_ERR_ARG;
  int dev = 0;
  const uw_status st = device_of(a->logits_dev, &dev);
  if (st != UW_OK) return st;
  DeviceGuard g(dev);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int sms = sm_count_of(dev);
  return map_launch(a->logits_bf16 ? launch_sample<uint16_t>(*a, sms, s) : launch_sample<float>(*a, sms, s));
}
