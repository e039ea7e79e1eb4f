// Attention of new tokens over the paged cache (uw_paged_attention), for any
// mix of single tokens and prompt chunks, in one kernel and a small second one.
//
//   * Work is (request, key/value head, group of new tokens) units, each a run
//     of 128-position key/value tiles.  Lengths are only known on the device:
//     every CTA sums the units' tiles over all requests and takes an equal,
//     contiguous share of the flattened tile list (one CTA per SM), so a single
//     long request spreads over the GPU and a ragged batch stays balanced.  A
//     unit that CTAs share leaves (maximum, sum, output) partials in the
//     workspace; the second kernel joins them in order.
//   * A tile is 128 rows of (token, query head of the group) against 128
//     positions: S = Q K^T and O += P V on the tensor cores (tcgen05, both
//     accumulators in TMEM; P replaces S there as BF16 and is the A operand of
//     the second product).  V is used as it lies in the cache: an MN-major B
//     operand.
//   * Two streams keep the tensor cores and the exponentials busy at the same
//     time: units of more than 128 rows run two row tiles against each K/V tile;
//     smaller ones (single tokens) run their one row tile against alternating
//     K/V tiles with an accumulator each, and join the two at the end.
//   * K and V pages come by TMA, one box per page and 64 values, into a ring
//     that is ordered as the products use it, so the loads run ahead across
//     units.  Only pages with a visible position are read; V rows beyond the
//     visible ones are zeroed in shared memory (what lies there is unknown).
//   * Warps: 0-3 and 4-7 softmax of stream 0 and 1 (a thread per row), 8 loads Q and K,
//     11 loads V, 9 issues the products, 10 walks the CTA's share and hands out units.
//   * Every wait is bounded; on expiry the kernel raises UW_FLAG_TIMEOUT, waits
//     for its copies and products in flight (once all warps have stopped: one that
//     was through before the expiry has left some too), frees TMEM and returns.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdlib>

#include "attention_sm100.cuh"
#include "handle.h"
#include "pdl.cuh"
#include "serving.h"
#include "tma_map.h"

namespace uw {
namespace {

using namespace sm100;

constexpr int kAttnMaxRequests = 8192;
constexpr int kMaxCtas = 160;
constexpr int kRows = 128;                // rows of a stream's tile = TMEM lanes
constexpr int kKeys = 128;                // positions per K/V tile
constexpr int kThreads = 12 * 32;
constexpr int kRegsSoftmax = 224, kRegsOther = 56;  // 256 * 224 + 128 * 56 = 384 * 168, the launch's registers
constexpr int kLoadWarp = 8, kMmaWarp = 9, kWalkWarp = 10, kLoadVWarp = 11;
constexpr int kDescs = 4;                 // units handed out ahead
constexpr int kSmemLimit = 232448;
constexpr float kLazy = 8.f;              // the kept maximum may lag the true one by 2^8

// The first page of the workspace: one record per CTA for the second kernel.
struct JoinRecord {
  int32_t pieces;   // CTAs that hold a part of the unit this CTA began (0: none to join)
  int32_t tok, n_tok, kv_head;
  int32_t pad[4];
};
constexpr size_t kJoinBytes = kMaxCtas * sizeof(JoinRecord);

struct Unit {
  int32_t request, kv_head;
  int32_t tok, n_tok;    // rows of q: first, and how many
  int32_t pos;           // position of the first
  int32_t two;           // more than one row tile
  int32_t lo, hi;        // positions that some row sees
  int32_t tile, n_tiles; // this CTA's share of the unit's tiles
  int32_t slot;          // -1: all of it; else the partial's slot (0: from before, 1: begun here)
  int32_t stop;          // no further units
};

struct AttnParams {
  CUtensorMap q, q_one, k, v;  // q_one: boxes of one token
  uw_paged_attention_args a;
  int32_t group, per_tile;  // query heads per key/value head; tokens per row tile
  int32_t page_shift;
  float scale_log2;         // |scale| * log2(e)
  int32_t turn;             // scale <= 0: scores are taken as (x & s_and) ^ s_xor
  uint32_t s_and, s_xor;
  int32_t withhold;         // failure-detection tests: the second row tile's last signal stays away
  uint64_t wait_ns;
};

template <int D>
struct Layout {
  static constexpr int kTile = kKeys * D * 2;             // one K or V tile, one Q tile
  static constexpr int kStats = 2048, kAside = kStats + 1024;  // statistics; they, descriptors and barriers
  static constexpr int kRing = (kSmemLimit - 2 * kTile - kAside) / kTile > 12 ? 12 : (kSmemLimit - 2 * kTile - kAside) / kTile;
  static constexpr int oRing = 2 * kTile;
  static constexpr int oStats = oRing + kRing * kTile;    // float2 [2][128]
  static constexpr int oDesc = oStats + kStats;             // Unit [kDescs]
  static constexpr int oBar = oDesc + kDescs * 64;
  static constexpr int bFull = 0, bEmpty = kRing, bScore = 2 * kRing, bWeight = bScore + 2, bOut = bWeight + 2,
                       bQ = bOut + 2, bQEmpty = bQ + 2, bStats = bQEmpty + 2, bDone = bStats + 1, bDescFull = bDone + 1,
                       bDescEmpty = bDescFull + kDescs, bDrain = bDescEmpty + kDescs, kBars = bDrain + 1;
  static constexpr int oMisc = oBar + kBars * 8;          // TMEM base, abort flag
  static constexpr int kBytes = oMisc + 64;
  static_assert(kBytes <= kSmemLimit, "shared memory");
  static_assert(sizeof(Unit) <= 64, "descriptor");
};
constexpr uint32_t kColScore = 0, kColOut = 256;          // TMEM columns: S0 S1 O0 O1

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two FP32 operations per instruction.
__device__ __forceinline__ float2 fma2(float2 x, float2 y, float2 z) {
  float2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<uint64_t&>(r))
      : "l"(reinterpret_cast<uint64_t&>(x)), "l"(reinterpret_cast<uint64_t&>(y)), "l"(reinterpret_cast<uint64_t&>(z)));
  return r;
}
__device__ __forceinline__ float2 add2(float2 x, float2 y) {
  float2 r;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t&>(r))
      : "l"(reinterpret_cast<uint64_t&>(x)), "l"(reinterpret_cast<uint64_t&>(y)));
  return r;
}

// The weights 2^(x c - mc) of a row's 128 scores: BF16 into TMEM, their FP32 sum
// returned.  They are the product's operand, whose type V's is; that rounding, at
// most 2^-8 of each, is the only one beside FP32's.  It takes the root mean square
// error of a BF16 output from 0.0017 of its size, its own rounding, to 0.0020 to
// 0.0023.  Weights in two parts would be exact to 2^-16, for twice the product.
__device__ __forceinline__ float exponentials(const uint32_t (&x)[kKeys], float c, float mc, uint32_t to) {
  const float2 c2 = make_float2(c, c), mc2 = make_float2(-mc, -mc);
  float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
  for (int i = 0; i < kKeys / 32; ++i) {
    uint32_t w[16];
#pragma unroll
    for (int q = 0; q < 16; ++q) {
      const float2 y = fma2(make_float2(__uint_as_float(x[i * 32 + 2 * q]), __uint_as_float(x[i * 32 + 2 * q + 1])), c2, mc2);
      const float2 e = make_float2(ex2(y.x), ex2(y.y));
      sum[q & 1] = add2(sum[q & 1], e);
      w[q] = bf16_pair(e.x, e.y);
    }
    tmem_st16(to + i * 16, w);
  }
  const float2 both = add2(sum[0], sum[1]);
  return both.x + both.y;
}

// Softmax of a tile whose live rows are at most 16 (single tokens): one warp,
// four threads per row with 32 scores each, so that the exponentials take a
// quarter of the time that a thread per row needs.  Each thread serves rows t / 4
// and t / 4 + 8 of the tile (t: thread of the warp).
struct FewRows {
  float m[2], l[2];  // the rows' maxima, and this thread's part of their sums

  template <int D>
  __device__ __forceinline__ void tile(uint32_t score, uint32_t out, bool first, bool eight, float c, const int (&from)[2],
                                       const int (&to)[2], bool edge, bool turn, uint32_t s_and, uint32_t s_xor) {
    const int col = 2 * (threadIdx.x & 3);
    uint32_t x[64];
    tmem_ld_16x256b_x8(score, x);
    tmem_ld_16x256b_x8(score + 64, x + 32);
    tmem_ld_wait();
    if (turn) {
#pragma unroll
      for (int i = 0; i < 64; ++i) x[i] = (x[i] & s_and) ^ s_xor;
    }
    uint32_t w[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) w[i] = 0;
    float f[2] = {1.f, 1.f};
    bool lag = false;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      if (r == 1 && eight) break;  // (eight rows at most)
      if (edge) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
#pragma unroll
          for (int q = 0; q < 2; ++q)
            if (8 * i + col + q < from[r] || 8 * i + col + q >= to[r]) x[4 * i + 2 * r + q] = 0xFF800000u;
      }
      float top = m[r];
#pragma unroll
      for (int i = 0; i < 16; ++i)
        top = fmaxf(top, fmaxf(__uint_as_float(x[4 * i + 2 * r]), __uint_as_float(x[4 * i + 2 * r + 1])));
      top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
      if (first) {
        m[r] = top;
      } else if (top > m[r] && !((top - m[r]) * c <= kLazy)) {
        f[r] = ex2((m[r] - top) * c);
        m[r] = top;
        l[r] *= f[r];
        lag = true;
      }
      const float mc = m[r] == -INFINITY ? 0.f : m[r] * c;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float e0 = ex2(fmaf(__uint_as_float(x[4 * i + 2 * r]), c, -mc));
        const float e1 = ex2(fmaf(__uint_as_float(x[4 * i + 2 * r + 1]), c, -mc));
        l[r] += e0 + e1;
        w[2 * i + r] = bf16_pair(e0, e1);
      }
    }
    tmem_st_16x128b_x16(score, w);
    if (__any_sync(0xFFFFFFFFu, lag)) {
#pragma unroll 1
      for (int k = 0; k < D; k += 64) {
        uint32_t o[32];
        tmem_ld_16x256b_x8(out + k, o);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f[i / 2 % 2]);
        tmem_st_16x256b_x8(out + k, o);
      }
    }
    tmem_st_wait();
  }
};

// All warps are through their work: `abort` keeps its value from here on.  (A barrier of its own, since the
// warps come to it from different places.)
__device__ __forceinline__ void work_ends() {
  __syncwarp();
  asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory");
}

// log sum of exponentials, from base-two maximum and sum.
__device__ __forceinline__ float lse_of(float m, float l) {
  return l > 0.f ? (m + log2f(l)) * 0.69314718055994531f : (l == 0.f ? -INFINITY : l);
}

// What a request asks for, cut to what the arrays hold.
struct Request {
  int32_t row, n, kv;  // first row of q, rows, stored positions
};

__device__ __forceinline__ Request request_of(const AttnParams& p, int b, bool* bad) {
  const int64_t rows = p.a.n_rows, from = __ldg(p.a.cu_q_dev + b), to = __ldg(p.a.cu_q_dev + b + 1);
  if (from < 0 || to < from || to > rows) *bad = true;
  const int64_t c0 = min(max(from, (int64_t)0), rows), c1 = min(max(to, c0), rows);
  const int64_t most = min((int64_t)p.a.table_width << p.page_shift, (int64_t)INT32_MAX - 2 * kKeys);
  const int64_t kv = __ldg(p.a.kv_len_dev + b);
  if (c1 > c0 && (kv < 0 || kv > most)) *bad = true;
  Request r;
  r.row = (int32_t)c0;
  r.n = (int32_t)(c1 - c0);
  r.kv = (int32_t)min(max(kv, (int64_t)0), most);
  return r;
}

// What a unit costs beside its tiles (loads of Q, first scores, epilogue), in
// tiles of one row tile.  A mixed batch of short and long requests took 80 us
// with 0, 70 with 2 and 4; a chunk of a long prompt 874 with 2, 899 with 4.
constexpr int kUnitCost = 2;

// The unit of the request's tokens [first, first + 2 * per_tile): its visible
// positions and tiles.
struct Span {
  int32_t n_tok, pos, lo, hi, tile, n_tiles, two;
  // weight of a tile in the shares: two row tiles take twice the products
  __device__ __forceinline__ int64_t cost() const { return kUnitCost + ((int64_t)max(n_tiles, 1) << two); }
};

__device__ __forceinline__ Span span_of(const AttnParams& p, const Request& r, int first) {
  Span s;
  s.n_tok = min(2 * p.per_tile, r.n - first);
  s.two = s.n_tok > p.per_tile;
  s.pos = r.kv - r.n + first;
  s.hi = max(0, s.pos + s.n_tok);
  s.lo = p.a.window > 0 ? max(0, s.pos - p.a.window + 1) : 0;
  s.tile = s.lo / kKeys;
  s.n_tiles = s.hi > s.lo ? (s.hi + kKeys - 1) / kKeys - s.tile : 0;
  return s;
}

__device__ __forceinline__ int64_t request_cost(const AttnParams& p, const Request& r) {
  int64_t c = 0;
  for (int t = 0; t < r.n; t += 2 * p.per_tile) c += span_of(p, r, t).cost();
  return c;
}

// Ranks of ring buffers: where tile j's K and V lie in the order of use, over a
// piece of n tiles (K0 V0 K1 V1 .. with two row tiles; K0 K1 V0 K2 V1 .. else).
__device__ __forceinline__ int ring_k(int j, int two) { return two ? 2 * j : (j == 0 ? 0 : 2 * j - 1); }
__device__ __forceinline__ int ring_v(int j, int n, int two) { return two ? 2 * j + 1 : min(2 * j + 2, 2 * n - 1); }

template <int D>
__global__ void __launch_bounds__(kThreads, 1) paged_attention_kernel(const __grid_constant__ AttnParams p) {
  using L = Layout<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t s0 = smem_u32(smem);
  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + L::oMisc);
  volatile int* abort = reinterpret_cast<volatile int*>(misc + 1);
  float2* stats = reinterpret_cast<float2*>(smem + L::oStats);
  volatile Unit* descs = reinterpret_cast<volatile Unit*>(smem + L::oDesc);
  const auto bar = [&](int i) { return s0 + L::oBar + 8 * i; };
  const uw_paged_attention_args& a = p.a;

  if (warp == kMmaWarp) {
    tmem_alloc(s0 + L::oMisc, 512);
    tmem_relinquish();
  }
  if (tid == 0) {
    for (int i = 0; i < L::kRing; ++i) {
      mbar_init(bar(L::bFull + i), 1);
      mbar_init(bar(L::bEmpty + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(L::bScore + i), 1);
      mbar_init(bar(L::bWeight + i), 4);
      mbar_init(bar(L::bOut + i), 1);
      mbar_init(bar(L::bQ + i), 1);
      mbar_init(bar(L::bQEmpty + i), 1);
    }
    mbar_init(bar(L::bStats), 8);
    mbar_init(bar(L::bDone), 8);
    for (int i = 0; i < kDescs; ++i) {
      mbar_init(bar(L::bDescFull + i), 1);
      mbar_init(bar(L::bDescEmpty + i), 11);
    }
    mbar_init(bar(L::bDrain), 1);
    fence_mbar_init();
    misc[1] = 0;
    prefetch_tensormap(&p.q);
    prefetch_tensormap(&p.k);
    prefetch_tensormap(&p.v);
  }
  for (int i = tid; i < 2 * L::kTile / 16; i += kThreads)
    reinterpret_cast<uint4*>(smem)[i] = make_uint4(0, 0, 0, 0);  // both Q buffers
  pdl_wait();
  pdl_release();

  // The total work, and the request in which this CTA's share begins: each
  // thread sums a run of consecutive requests (the scratch lies in the ring).
  int64_t* sums = reinterpret_cast<int64_t*>(smem + L::oRing);
  const int per = (a.n_requests + kThreads - 1) / kThreads;
  bool pairs = false;  // some unit has two row tiles
  {
    int64_t mine = 0;
    bool bad = false;
    for (int b = tid * per; b < min((tid + 1) * per, a.n_requests); ++b) {
      const Request r = request_of(p, b, &bad);
      mine += request_cost(p, r);
      pairs |= r.n > p.per_tile;
    }
    if (bad && a.flags_dev && blockIdx.x == 0) atomicOr(a.flags_dev, (uint32_t)UW_FLAG_BAD_INPUT);
    int64_t in = mine * a.cache.n_kv_heads;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t x = __shfl_up_sync(0xFFFFFFFFu, in, d);
      if (lane >= d) in += x;
    }
    sums[tid] = in;
  }
  tc_fence_before();
  pairs = __syncthreads_or(pairs);
  tc_fence_after();
  const uint32_t tmem = misc[0];
  int64_t total = 0;
  for (int w = 0; w < kThreads / 32; ++w) total += sums[w * 32 + 31];

  // Shares of a tile at least, so that a unit's pieces lie in successive CTAs.
  const int cta = blockIdx.x, G = (int)min((int64_t)gridDim.x, max(pairs ? total >> 1 : total, (int64_t)1));
  const int64_t share0 = cta < G ? total * cta / G : total, share1 = cta < G ? total * (cta + 1) / G : total;
  float* part = reinterpret_cast<float*>(static_cast<uint8_t*>(a.ws_dev) + kJoinBytes);
  constexpr int64_t kPart = 2 * kRows * (D + 2);  // floats of a partial
  int64_t start_sum = 0;
  int start_b = 0;
  if (warp == kWalkWarp) {
    // the thread whose run of requests holds share0: the warp by its sum, then
    // the thread in it
    int64_t upto = lane < kThreads / 32 ? sums[lane * 32 + 31] : 0;
#pragma unroll
    for (int d = 1; d < 16; d <<= 1) {
      const int64_t x = __shfl_up_sync(0xFFFFFFFFu, upto, d);
      if (lane >= d) upto += x;
    }
    const int w = __ffs(__ballot_sync(0xFFFFFFFFu, lane < kThreads / 32 && share0 < upto)) - 1;
    start_b = a.n_requests;
    if (w >= 0) {
      start_sum = w > 0 ? __shfl_sync(0xFFFFFFFFu, upto, w - 1) : 0;
      const int64_t in = sums[w * 32 + lane];
      const int t = __ffs(__ballot_sync(0xFFFFFFFFu, share0 < start_sum + in)) - 1;
      start_sum += t > 0 ? __shfl_sync(0xFFFFFFFFu, in, t - 1) : 0;
      start_b = min((w * 32 + t) * per, a.n_requests);
    }
  }
  fence_proxy_async_smem();  // (the scratch becomes ring buffers)
  __syncthreads();

  const auto fail = [&]() {
    if (!*abort) {
      *abort = 1;
      if (a.flags_dev) atomicOr(a.flags_dev, (uint32_t)UW_FLAG_TIMEOUT);
    }
  };
  const auto wait = [&](int i, uint32_t parity) {
    if (mbar_wait_bounded(bar(i), parity, abort, p.wait_ns)) return true;
    fail();
    return false;
  };
  // Read unit n's descriptor once it is there; false: aborted.  (Each warp frees the descriptor itself.)
  const auto take = [&](uint32_t n, Unit* u) {
    const int i = n % kDescs;
    if (!wait(L::bDescFull + i, (n / kDescs) & 1)) return false;
    const volatile Unit& d = descs[i];
    u->request = d.request;
    u->kv_head = d.kv_head;
    u->tok = d.tok;
    u->n_tok = d.n_tok;
    u->pos = d.pos;
    u->two = d.two;
    u->lo = d.lo;
    u->hi = d.hi;
    u->tile = d.tile;
    u->n_tiles = d.n_tiles;
    u->slot = d.slot;
    u->stop = d.stop;
    return true;
  };

  if (warp >= kLoadWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
    if (warp == kWalkWarp) {
      if (lane == 0) {
        uint32_t n = 0;
        const auto hand = [&](const Unit& u) {
          const int i = n % kDescs;
          if (!wait(L::bDescEmpty + i, ((n / kDescs) & 1) ^ 1)) return false;
          volatile Unit& d = descs[i];
          d.request = u.request;
          d.kv_head = u.kv_head;
          d.tok = u.tok;
          d.n_tok = u.n_tok;
          d.pos = u.pos;
          d.two = u.two;
          d.lo = u.lo;
          d.hi = u.hi;
          d.tile = u.tile;
          d.n_tiles = u.n_tiles;
          d.slot = u.slot;
          d.stop = u.stop;
          mbar_arrive(bar(L::bDescFull + i));
          ++n;
          return true;
        };
        JoinRecord rec = {};
        int64_t at = start_sum;  // weight before the unit under consideration
        bool ok = true, bad = false;
        for (int b = start_b; b < a.n_requests && at < share1 && ok; ++b) {
          const Request r = request_of(p, b, &bad);
          if (r.n == 0) continue;
          const int64_t per_head = request_cost(p, r);
          if (at + per_head * a.cache.n_kv_heads <= share0) {
            at += per_head * a.cache.n_kv_heads;
            continue;
          }
          for (int h = 0; h < a.cache.n_kv_heads && at < share1 && ok; ++h) {
            if (at + per_head <= share0) {
              at += per_head;
              continue;
            }
            for (int t = 0; t < r.n && at < share1 && ok; t += 2 * p.per_tile) {
              const Span s = span_of(p, r, t);
              const int64_t cost = s.cost(), end = at + cost;
              if (end <= share0) {
                at = end;
                continue;
              }
              // the tiles whose weight begins inside the share
              const int64_t unit = int64_t(1) << s.two;
              const int n_all = max(1, s.n_tiles);
              const int64_t from = at + kUnitCost;
              const int t0 = (int)((max(share0 - from, (int64_t)0) + unit - 1) >> s.two);
              const int t1 = (int)min((int64_t)n_all, (max(share1 - from, (int64_t)0) + unit - 1) >> s.two);
              if (t0 < min(t1, n_all)) {
                Unit u;
                u.request = b;
                u.kv_head = h;
                u.tok = r.row + t;
                u.n_tok = s.n_tok;
                u.pos = s.pos;
                u.two = s.two;
                u.lo = s.lo;
                u.hi = s.hi;
                u.tile = s.tile + t0;
                u.n_tiles = s.n_tiles ? t1 - t0 : 0;
                u.slot = t1 - t0 == n_all ? -1 : (t0 == 0 ? 1 : 0);
                u.stop = 0;
                if (u.slot == 1) {
                  // weight x is in the share of CTA ((x + 1) G - 1) / total
                  const int64_t x = from + ((int64_t)(n_all - 1) << s.two);
                  rec.pieces = (int32_t)(((x + 1) * G - 1) / total) - cta + 1;
                  rec.tok = u.tok;
                  rec.n_tok = u.n_tok;
                  rec.kv_head = h;
                }
                ok = hand(u);
              }
              at = end;
            }
          }
        }
        if (ok) {
          Unit u = {};
          u.stop = 1;
          hand(u);
        }
        reinterpret_cast<JoinRecord*>(a.ws_dev)[cta] = rec;
      }
      work_ends();
    } else if (warp == kLoadWarp || warp == kLoadVWarp) {
      // One warp loads Q and K, the other V.  A lane per box of the tile: its
      // page's id is fetched a tile ahead, and each lane issues its own copies,
      // which a warp does one lane after the other (with 16-slot pages one thread
      // that walked all boxes took 815 us for a ragged decoding batch of 2.1 GB, one
      // warp 462, two 337).
      const bool is_v = warp == kLoadVWarp;
      const CUtensorMap* map = is_v ? &p.v : &p.k;
      const int page_rows = min(kKeys, 1 << p.page_shift), boxes = kKeys / page_rows;
      uint32_t n = 0, rank = 0, pieces = 0;  // rank: ring buffers used before this unit
      uint32_t q_used[2] = {0, 0}, last = 0;
      bool ok = true, bad = false;
      Unit u;
      while (ok) {
        ok = __all_sync(0xFFFFFFFFu, take(n, &u));
        if (!ok) break;
        if (lane == 0) mbar_arrive(bar(L::bDescEmpty + n % kDescs));
        ++n;
        if (u.stop) break;
        if (u.n_tiles == 0) continue;
        // Q: the rows of (token, head) as they lie, one box per row tile and 64
        // values; units of one row tile take the two buffers in turn.  A single
        // token comes alone, and the tile's other rows stay as they are: zero in a
        // batch of single tokens, else what the buffer's last longer unit left.
        // With zeros the products are as long, but take less power, which bounds the
        // clock of a long decoding run (seconds of the ragged batch: 367 us a call
        // with the neighbouring tokens' rows in the tile, 357 so).
        for (int t = 0; t <= u.two && ok && !is_v; ++t) {
          const int buf = u.two ? t : (int)(pieces & 1);
          ok = __all_sync(0xFFFFFFFFu, wait(L::bQEmpty + buf, (q_used[buf] & 1) ^ 1));
          if (!ok) break;
          if (lane == 0) {
            const bool one = u.n_tok == 1;
            mbar_expect_tx(bar(L::bQ + buf), (uint32_t)(p.group * (one ? 1 : p.per_tile)) * D * 2);
#pragma unroll
            for (int c = 0; c < D / 64; ++c)
              tma_load_3d(s0 + buf * L::kTile + c * kRows * 128, one ? &p.q_one : &p.q, bar(L::bQ + buf), c * 64,
                          u.kv_head * p.group, u.tok + t * p.per_tile);
          }
          __syncwarp();
          ++q_used[buf];
        }
        if (!ok) break;
        ++pieces;
        const int32_t* table = a.table_dev + (int64_t)u.request * a.table_stride;
        // page of this lane's box of tile j; -1: nothing of it is visible
        const auto page_of = [&](int j) {
          const int at = (u.tile + j) * kKeys + lane * page_rows;
          if (lane >= boxes || j >= u.n_tiles || at >= u.hi || at + page_rows <= u.lo) return -1;
          const int32_t page = __ldg(table + (at >> p.page_shift));
          if (page >= 0 && page < a.cache.n_pages) return page;
          bad = true;
          return -1;
        };
        int page = page_of(0);
        for (int j = 0; j < u.n_tiles; ++j) {
          const int next = page_of(j + 1);
          const uint32_t at = rank + (is_v ? ring_v(j, u.n_tiles, u.two) : ring_k(j, u.two));
          const int buf = at % L::kRing;
          ok = __all_sync(0xFFFFFFFFu, wait(L::bEmpty + buf, ((at / L::kRing) & 1) ^ 1));
          if (!ok) break;
          last = at + 1;
          const uint32_t full = bar(L::bFull + buf);
          const uint32_t some = __ballot_sync(0xFFFFFFFFu, page >= 0);
          if (lane == 0) mbar_expect_tx(full, (uint32_t)__popc(some) * page_rows * D * 2);
          __syncwarp();
          if (page >= 0) {
            const int slot = ((u.tile + j) * kKeys + lane * page_rows) & ((1 << p.page_shift) - 1);
            const uint32_t dst = s0 + L::oRing + buf * L::kTile + lane * page_rows * 128;
#pragma unroll
            for (int c = 0; c < D / 64; ++c)
              tma_load_4d(dst + c * kKeys * 128, map, full, c * 64, slot, u.kv_head, page);
          }
          page = next;
        }
        rank += 2 * u.n_tiles;
      }
      if (bad && a.flags_dev) atomicOr(a.flags_dev, (uint32_t)UW_FLAG_BAD_INPUT);
      work_ends();
      if (*abort && lane == 0) {  // leave no copy in flight
        // (a buffer's phase that this warp did not fill is over or never began;
        // the wait for it is bounded like every other)
        volatile int none = 0;
        for (uint32_t q = last > L::kRing ? last - L::kRing : 0; q < last; ++q)
          mbar_wait_bounded(bar(L::bFull + q % L::kRing), (q / L::kRing) & 1, &none, p.wait_ns);
        for (int t = 0; t < 2; ++t)
          if (q_used[t]) mbar_wait_bounded(bar(L::bQ + t), (q_used[t] - 1) & 1, &none, p.wait_ns);
      }
      __syncwarp();
    } else {
      // The products.  The warp stays together and elects a lane per
      // instruction: descriptors are then in uniform registers, and an issue
      // takes 41 clocks, of the 64 that a 128 x 128 x 16 product runs (one lane
      // in a branch of its own took 69).
      const auto wait_all = [&](int i, uint32_t parity) { return (bool)__all_sync(0xFFFFFFFFu, wait(i, parity)); };
      const auto uniform = [](int x) { return __shfl_sync(0xFFFFFFFFu, x, 0); };
      constexpr uint32_t kIdScore = idesc_bf16(kRows, kKeys), kIdOut = idesc_bf16_b_mn(kRows, D);
      const uint32_t acc = uniform(tmem);
      uint32_t n = 0, pieces = 0, head = 0, phase = 0;  // head, phase: of the ring
      uint32_t weights[2] = {0, 0};  // weight tiles taken per stream
      uint32_t q_used[2] = {0, 0};
      bool ok = true;
      while (ok) {
        ok = wait_all(L::bDescFull + n % kDescs, (n / kDescs) & 1);
        if (!ok) break;
        const int two = uniform(descs[n % kDescs].two), n_tiles = uniform(descs[n % kDescs].n_tiles);
        const bool stop = uniform(descs[n % kDescs].stop);
        if (lane == 0) mbar_arrive(bar(L::bDescEmpty + n % kDescs));
        __syncwarp();
        ++n;
        if (stop) break;
        if (n_tiles == 0) continue;
        const int q0 = two ? 0 : (int)(pieces & 1), q1 = two ? 1 : q0;  // Q buffer of each stream
        // The next buffer of the ring, loaded (the order of use is the ring's).
        int taken = 0;
        const auto next = [&]() {
          ok = ok && wait_all(L::bFull + head, phase);
          taken = head;
          if (++head == L::kRing) {
            head = 0;
            phase ^= 1;
          }
          return s0 + L::oRing + (uint32_t)taken * L::kTile;
        };
        const auto score = [&](int s, int j, uint32_t k, bool last_use) {
          const uint64_t kb = smem_desc_sw128(k), qb = smem_desc_sw128(s0 + (s ? q1 : q0) * L::kTile);
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            const uint32_t off = ((c / 4) * (kKeys * 128) + (c % 4) * 32) >> 4;
            mma_bf16_elect(acc + kColScore + s * kKeys, qb + off, kb + off, kIdScore, c > 0);
          }
          if (last_use) mma_commit_elect(bar(L::bEmpty) + (k - s0 - L::oRing) / L::kTile * 8);
          if (j == n_tiles - 1) mma_commit_elect(bar(L::bQEmpty + (s ? q1 : q0)));
          mma_commit_elect(bar(L::bScore + s));
        };
        const auto output = [&](int s, uint32_t v, bool first, bool last_use) {
          const uint64_t vb = smem_desc_sw128_mn(v, kKeys * 128);
#pragma unroll
          for (int c = 0; c < kKeys / 16; ++c)
            mma_bf16_tmem_a_elect(acc + kColOut + s * D, acc + kColScore + s * kKeys + c * 8, vb + c * (2048 >> 4), kIdOut,
                                  !first || c > 0);
          if (last_use) mma_commit_elect(bar(L::bEmpty) + (v - s0 - L::oRing) / L::kTile * 8);
        };
        for (int t = q0; t <= q1 && ok; ++t) ok = wait_all(L::bQ + t, q_used[t]++ & 1);
        // scores run one tile of each stream ahead of the outputs
        const int steps = two ? 2 * n_tiles : n_tiles;  // (tile, stream) pairs
        uint32_t k = 0, v = 0;
        for (int i = 0; i < min(2, steps) && ok; ++i) {
          if (i == 0 || !two) k = next();
          tc_fence_after();
          if (ok) score(i, two ? 0 : i, k, !two || i == 1);
        }
        // the accumulators are free once the last unit's outputs have been read
        if (ok) ok = wait_all(L::bDone, (pieces & 1) ^ 1);
        for (int i = 0; i < steps && ok; ++i) {
          const int s = i & 1;
          // (what the products read is awaited before what the softmax makes:
          // it is there already, but for the first tiles)
          if (s == 0 || !two) {
            v = next();
            if (i + 2 < steps) k = next();
          }
          ok = ok && wait_all(L::bWeight + s, weights[s] & 1);
          if (!ok) break;
          ++weights[s];
          tc_fence_after();
          output(s, v, i < 2, !two || s == 1);
          if (i + 2 >= steps) {
            if (!(p.withhold && two && s == 1)) mma_commit_elect(bar(L::bOut + s));
          } else score(s, two ? (i + 2) >> 1 : i + 2, k, !two || s == 1);
        }
        ++pieces;
      }
      work_ends();
      if (*abort) {  // leave no product in flight
        volatile int none = 0;
        mma_commit_elect(bar(L::bDrain));
        mbar_wait_bounded(bar(L::bDrain), 0, &none, p.wait_ns);
      }
      __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    // softmax of stream s: thread = row of its tile
    const int s = warp >> 2, row = tid & 127;
    const uint32_t lanes = tmem + ((uint32_t)(warp & 3) * 32 << 16);
    const float c = p.scale_log2;
    uint32_t n = 0, rank = 0, pieces = 0, scores = 0, joins = 0, outs1 = 0;
    // (one decision per warp: its lanes stay together)
    const auto wait_all = [&](int i, uint32_t parity) { return (bool)__all_sync(0xFFFFFFFFu, wait(i, parity)); };
    while (wait_all(L::bDescFull + n % kDescs, (n / kDescs) & 1)) {
      // What the tiles need is held in registers, the rest is read again after
      // them (the row's scores take most of a thread's registers).
      const volatile Unit& u = descs[n % kDescs];
      if (u.stop) break;
      const int two = u.two, n_tiles = u.n_tiles, lo = u.lo, hi = u.hi, tile0 = u.tile * kKeys;
      // this thread's row of q: in its stream's tile with two row tiles, else
      // in the one tile of both streams
      const int tok = (two ? s * p.per_tile : 0) + row / p.group;
      const bool live = row < p.per_tile * p.group && tok < u.n_tok;
      const bool warp_live = __any_sync(0xFFFFFFFFu, live);
      const int pos = u.pos + tok;
      // tiles that every row of the unit sees whole need no mask
      const int whole_to = u.pos + 1, whole_from = a.window > 0 ? u.pos + u.n_tok - a.window : 0;

      float m = -INFINITY, l = 0.f;  // of the raw scores; of the weights
      // 0: a thread per row; else at most 8 rows (1) or 16 (2), four threads each
      const int rows = u.n_tok * p.group, few = two || rows > 16 ? 0 : (rows > 8 ? 2 : 1);
      FewRows q16 = {{-INFINITY, -INFINITY}, {0.f, 0.f}};
      bool ok = true;
      for (int j = two ? 0 : s; j < n_tiles; j += two ? 1 : 2) {
        const int first = tile0 + j * kKeys;
        ok = wait_all(L::bScore + s, scores & 1);
        ++scores;
        if (!ok) break;
        tc_fence_after();
        const bool edge = first < whole_from || first + kKeys > whole_to;
        if (few != 0 && warp_live) {
          int from[2], to[2];
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const int at = whole_to - 1 + (lane / 4 + 8 * r) / p.group - first;  // (whole_to - 1: the first row's position)
            from[r] = a.window > 0 ? at - a.window + 1 : -first;
            to[r] = at + 1;
          }
          q16.template tile<D>(lanes + kColScore + s * kKeys, lanes + kColOut + s * D, j < 2, few == 1, c, from, to, edge,
                               p.turn, p.s_and, p.s_xor);
        } else if (warp_live) {
          const uint32_t score = lanes + kColScore + s * kKeys;
          uint32_t x[kKeys];
#pragma unroll
          for (int i = 0; i < kKeys / 32; ++i) tmem_ld32(score + i * 32, x + i * 32);
          tmem_ld_wait();
          if (p.turn) {
#pragma unroll
            for (int i = 0; i < kKeys; ++i) x[i] = (x[i] & p.s_and) ^ p.s_xor;
          }
          if (edge) {
            const int from = a.window > 0 ? pos - a.window + 1 - first : -first, to = pos + 1 - first;
#pragma unroll
            for (int i = 0; i < kKeys; ++i)
              if (i < from || i >= to) x[i] = 0xFF800000u;
          }
          // (four chains: one alone would take as long as the exponentials)
          float tops[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) tops[i] = fmaxf(__uint_as_float(x[i]), __uint_as_float(x[i + 4]));
#pragma unroll
          for (int i = 8; i < kKeys; i += 8)
#pragma unroll
            for (int q = 0; q < 4; ++q)
              tops[q] = fmaxf(tops[q], fmaxf(__uint_as_float(x[i + q]), __uint_as_float(x[i + 4 + q])));
          const float top = fmaxf(m, fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3])));
          // Keep the old maximum while it lags by less than 2^8: the weights
          // stay below 2^8, and sum and output keep their scale.
          const bool lag = top > m && !((top - m) * c <= kLazy);
          if (j < 2 - two) {  // the stream's first tile
            m = top;
          } else if (__any_sync(0xFFFFFFFFu, lag)) {
            const float f = lag ? ex2((m - top) * c) : 1.f;
            if (lag) m = top;
            l *= f;
#pragma unroll 1
            for (int i = 0; i < D; i += 16) {
              uint32_t o[16];
              tmem_ld16(lanes + kColOut + s * D + i, o);
              tmem_ld_wait();
#pragma unroll
              for (int q = 0; q < 16; ++q) o[q] = __float_as_uint(__uint_as_float(o[q]) * f);
              tmem_st16(lanes + kColOut + s * D + i, o);
            }
            tmem_st_wait();
          }
          const float mc = m == -INFINITY ? 0.f : m * c;
          l += exponentials(x, c, mc, score);
          tmem_st_wait();
        }
        // V rows that no row of the unit sees hold anything: make them zero
        if ((first < lo || first + kKeys > hi) && (!two || s == 0)) {
          const uint32_t at = rank + ring_v(j, n_tiles, two);
          ok = wait_all(L::bFull + at % L::kRing, (at / L::kRing) & 1);
          if (!ok) break;
          if (first + row < lo || first + row >= hi) {
            uint8_t* v = smem + L::oRing + (at % L::kRing) * L::kTile + row * 128;
#pragma unroll
            for (int i = 0; i < D / 8; ++i)
              *reinterpret_cast<uint4*>(v + (i / 8) * (kKeys * 128) + (i & 7) * 16) = make_uint4(0, 0, 0, 0);
            fence_proxy_async_smem();
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(L::bWeight + s));
      }
      if (!ok) break;
      rank += 2 * n_tiles;

      // Join the two streams of a single row tile: each writes half of the
      // values.  (The statistics may be replaced once both have read the last
      // unit's.)
      const bool both = !two && n_tiles > 1;  // two accumulators of the same rows
      float f0 = 1.f, f1 = 0.f;               // factors of the accumulators
      if (n_tiles > 0) {
        if (!two) {
          if (pieces > 0) ok = wait_all(L::bDone, (pieces - 1) & 1);
          if (!ok) break;
          if (few == 0) {
            stats[s * kRows + row] = make_float2(m, l);
          } else if (warp_live) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              float sum = q16.l[r];
              sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
              sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 2);
              if (lane % 4 == 0) stats[s * kRows + lane / 4 + 8 * r] = make_float2(q16.m[r], sum);
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(L::bStats));
        }
        if (!two || s == 0) ok = wait_all(L::bOut, pieces & 1);
        if (ok && (both || (two && s == 1))) ok = wait_all(L::bOut + 1, outs1 & 1);
        if (two || both) ++outs1;
        if (ok && !two) ok = wait_all(L::bStats, joins++ & 1);
        if (!ok) break;
        ++pieces;
        tc_fence_after();
        if (!two) {
          const float2 x = stats[row], y = stats[kRows + row];
          m = fmaxf(x.x, y.x);
          const float mc = m == -INFINITY ? 0.f : m * c;
          f0 = ex2(fmaf(x.x, c, -mc));
          f1 = ex2(fmaf(y.x, c, -mc));
          l = x.y * f0 + (both ? y.y * f1 : 0.f);
        }
      }
      const int slot = u.slot, head = u.kv_head * p.group + row % p.group;
      const int64_t q_row = (int64_t)u.tok + tok;
      // (a row that sees nothing gives zeros, whatever the accumulators hold)
      const bool none = l == 0.f;
      const float inv = slot >= 0 ? 1.f : (l > 0.f ? 1.f / l : 0.f);
      const int64_t piece = (int64_t)(2 * cta + slot) * kPart;
      const int in_part = (two ? s * kRows : 0) + row;
      if (warp_live) {
        const int col1 = two ? D : (s + 1) * (D / 2);
#pragma unroll 1
        for (int col = two ? 0 : s * (D / 2); col < col1; col += 32) {
          uint32_t x[32];
          if (n_tiles > 0) {
            tmem_ld32(lanes + kColOut + (two ? s * D : 0) + col, x);
            tmem_ld_wait();
          }
#pragma unroll
          for (int i = 0; i < 32; ++i) x[i] = none ? 0u : __float_as_uint(__uint_as_float(x[i]) * f0);
          if (both) {
            uint32_t y[32];
            tmem_ld32(lanes + kColOut + D + col, y);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i)
              x[i] = none ? 0u : __float_as_uint(fmaf(__uint_as_float(y[i]), f1, __uint_as_float(x[i])));
          }
          const auto val = [&](int i) { return __uint_as_float(x[i]) * inv; };
          if (!live) continue;
          if (slot >= 0 || a.out_f32) {
            float* o = slot >= 0 ? part + piece + (int64_t)in_part * D
                                 : static_cast<float*>(a.out_dev) + q_row * a.out_stride + (int64_t)head * D;
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              *reinterpret_cast<float4*>(o + col + i) = make_float4(val(i), val(i + 1), val(i + 2), val(i + 3));
          } else {
            uint16_t* o = static_cast<uint16_t*>(a.out_dev) + q_row * a.out_stride + (int64_t)head * D;
#pragma unroll
            for (int i = 0; i < 32; i += 8)
              *reinterpret_cast<uint4*>(o + col + i) =
                  make_uint4(bf16_pair(val(i), val(i + 1)), bf16_pair(val(i + 2), val(i + 3)),
                             bf16_pair(val(i + 4), val(i + 5)), bf16_pair(val(i + 6), val(i + 7)));
          }
        }
        if (live && (two || s == 0)) {
          if (slot >= 0)
            reinterpret_cast<float2*>(part + piece + 2 * kRows * D)[in_part] = make_float2(m * c, l);
          else if (a.lse_dev)
            a.lse_dev[q_row * a.n_heads + head] = lse_of(m * c, l);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (n_tiles > 0) mbar_arrive(bar(L::bDone));
        mbar_arrive(bar(L::bDescEmpty + n % kDescs));
      }
      ++n;
    }
    work_ends();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Join the partials of the units that CTAs shared, a row's pieces in order.
// Latency is its time: with 32 warps for the up to 256 rows of a unit a mixed batch
// took 72 us in all, with 128 62.  A warp takes a row; where the pieces are many
// and the rows few, the warps of a CTA share a row's pieces (one token over 4096
// positions took 16.6 us in all with a warp per row, 14.1 so).
constexpr int kJoinWarps = 8, kJoinSplit = 16;

template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(const __grid_constant__ AttnParams p) {
  constexpr int64_t kPart = 2 * kRows * (D + 2);
  constexpr int E = D / 32;
  __shared__ float shared_o[kJoinWarps][D], shared_l[kJoinWarps];
  const uw_paged_attention_args& a = p.a;
  pdl_wait();
  pdl_release();
  const int cta = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const JoinRecord r = reinterpret_cast<const JoinRecord*>(a.ws_dev)[cta];
  if (r.pieces <= 0) return;
  const float* part = reinterpret_cast<const float*>(static_cast<const uint8_t*>(a.ws_dev) + kJoinBytes);
  const int rows = r.n_tok * p.group, tile = p.per_tile * p.group;
  const bool many = r.pieces > 4 && rows <= 2 * kJoinSplit;
  const int q0 = many ? warp : 0, step = many ? kJoinWarps : 1;
  const float inv_group = 1.f / (float)p.group;
  const float* begun = part + (int64_t)(2 * cta + 1) * kPart;  // piece 0; piece q is slot 0 of CTA cta + q
  const auto piece = [&](int q) { return q == 0 ? begun : begun + (int64_t)(2 * q - 1) * kPart; };
  for (int i = many ? blockIdx.y : blockIdx.y * kJoinWarps + warp; i < rows; i += many ? kJoinSplit : kJoinWarps * kJoinSplit) {
    const int tok = (int)(((float)i + 0.5f) * inv_group), g = i - tok * p.group;  // (exact: i < 256)
    const int at = i < tile ? i : kRows + i - tile;                              // row of the partial
    float m = -INFINITY;
    if (r.pieces <= 4) {
      for (int q = 0; q < r.pieces; ++q) m = fmaxf(m, reinterpret_cast<const float2*>(piece(q) + 2 * kRows * D)[at].x);
    } else {
      for (int q = lane; q < r.pieces; q += 32) m = fmaxf(m, reinterpret_cast<const float2*>(piece(q) + 2 * kRows * D)[at].x);
      for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
    }
    const float top = m == -INFINITY ? 0.f : m;
    float l = 0.f, o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.f;
#pragma unroll 4
    for (int q = q0; q < r.pieces; q += step) {
      const float* x = piece(q);
      const float2 ml = reinterpret_cast<const float2*>(x + 2 * kRows * D)[at];
      const float f = ex2(ml.x - top);
      l = fmaf(ml.y, f, l);
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        const float2 v = reinterpret_cast<const float2*>(x + at * D + e * 32)[lane];
        o[e] = fmaf(v.x, f, o[e]);
        o[e + 1] = fmaf(v.y, f, o[e + 1]);
      }
    }
    if (many) {
      __syncthreads();  // (the row before has been read)
#pragma unroll
      for (int e = 0; e < E; ++e) shared_o[warp][e * 32 + lane] = o[e];
      if (lane == 0) shared_l[warp] = l;
      __syncthreads();
      if (warp != 0) continue;
      for (int w = 1; w < kJoinWarps; ++w) {
        l += shared_l[w];
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] += shared_o[w][e * 32 + lane];
      }
    }
    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
    const int64_t row = r.tok + tok;
    const int head = r.kv_head * p.group + g;
    const int64_t to = row * a.out_stride + (int64_t)head * D + lane * 2;  // a lane's pairs lie 64 values apart
#pragma unroll
    for (int e = 0; e < E; e += 2) {
      if (a.out_f32) {
        *reinterpret_cast<float2*>(static_cast<float*>(a.out_dev) + to + e * 32) = make_float2(o[e] * inv, o[e + 1] * inv);
      } else {
        *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out_dev) + to + e * 32) = bf16_pair(o[e] * inv, o[e + 1] * inv);
      }
    }
    if (a.lse_dev && lane == 0)
      a.lse_dev[row * a.n_heads + head] = lse_of(m, l);
  }
}

// [page, head, slot, value] of the cache; a box is 64 values of a page's slots
// (128 at most) of one head, stored as rows of 128 swizzled bytes.  L2 fetches
// what a head's row has in one place: 256 bytes for the 128 of a 64-value head
// would bring the neighbouring head's too (decoding over 0.96 GB of those took
// 233 us so, 167 with 128).
bool make_map(CUtensorMap* m, const uint16_t* base, const uw_paged_cache& c) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[4] = {(cuuint64_t)c.head_dim, (cuuint64_t)c.page_size, (cuuint64_t)c.n_kv_heads, (cuuint64_t)c.n_pages};
  const cuuint64_t strides[3] = {(cuuint64_t)c.slot_stride * 2, (cuuint64_t)c.head_stride * 2, (cuuint64_t)c.page_stride * 2};
  const cuuint32_t box[4] = {64, (cuuint32_t)std::min(c.page_size, kKeys), 1, 1};
  const cuuint32_t one[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<uint16_t*>(base), dims, strides, box, one,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            c.head_dim == 64 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// [row, head, value] of q; a box is 64 values of the heads of one key/value head
// over some tokens.
bool make_q_map(CUtensorMap* m, const uw_paged_attention_args& a, int group, int tokens) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const uint64_t width = (uint64_t)a.n_heads * a.cache.head_dim;
  const cuuint64_t dims[3] = {(cuuint64_t)a.cache.head_dim, (cuuint64_t)a.n_heads, (cuuint64_t)a.n_rows};
  const cuuint64_t strides[2] = {(cuuint64_t)a.cache.head_dim * 2, std::max((uint64_t)a.q_stride, width) * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)group, (cuuint32_t)tokens};
  const cuuint32_t one[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t*>(a.q_dev), dims, strides, box, one,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

size_t workspace_bytes(int head_dim) {
  return kJoinBytes + (size_t)kMaxCtas * 2 * (2 * kRows) * (head_dim + 2) * 4;
}

template <int D>
cudaError_t launch_attention(const AttnParams& p, int sms, cudaStream_t s) {
  using L = Layout<D>;
  cudaError_t e = cudaFuncSetAttribute(paged_attention_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kBytes);
  if (e != cudaSuccess) return e;
  const int grid = std::min(sms, kMaxCtas);
  e = launch_pdl(paged_attention_kernel<D>, dim3(grid), dim3(kThreads), L::kBytes, s, p);
  if (e != cudaSuccess) return e;
  return launch_pdl(join_kernel<D>, dim3(grid, kJoinSplit), dim3(kJoinWarps * 32), 0, s, p);
}

}  // namespace
}  // namespace uw

using namespace uw;

extern "C" {

uw_status uw_paged_attention_workspace_bytes(int32_t n_heads, int32_t n_kv_heads, int32_t head_dim,
                                             size_t* bytes) {
  if (!bytes) return UW_ERR_ARG;
  if (n_heads < 1 || n_kv_heads < 1 || n_heads % n_kv_heads) return UW_ERR_SHAPE;
  if ((head_dim != 64 && head_dim != 128) || n_heads / n_kv_heads > kRows) return UW_ERR_UNSUPPORTED;
  *bytes = workspace_bytes(head_dim);
  return UW_OK;
}

uw_status uw_paged_attention(const uw_paged_attention_args* a, void* stream) {
  if (!a) return UW_ERR_ARG;
  if (a->n_rows < 0 || a->n_rows > (int64_t(1) << 30) || a->n_requests < 0 ||
      a->n_requests > kAttnMaxRequests || a->table_width < 0 || a->window < 0 || a->n_heads < 1)
    return UW_ERR_SHAPE;
  uw_status st = check_cache(a->cache);
  if (st != UW_OK) return st;
  size_t need = 0;
  st = uw_paged_attention_workspace_bytes(a->n_heads, a->cache.n_kv_heads, a->cache.head_dim, &need);
  if (st != UW_OK) return st;
  if (!std::isfinite(a->scale)) return UW_ERR_ARG;
  // a window that no stored position lies outside of is none; behind this check
  // the kernel's position arithmetic stays in 32 bits
  const bool windowed = a->window > 0 && (int64_t)a->window < (int64_t)a->table_width * a->cache.page_size;
  if (windowed && a->window >= 1 << 30) return UW_ERR_UNSUPPORTED;
  if (a->n_rows == 0 || a->n_requests == 0) return UW_OK;
  if (!a->q_dev || !a->out_dev || !a->cu_q_dev || !a->kv_len_dev ||
      (a->table_width > 0 && (!a->table_dev || a->table_stride < a->table_width)))
    return UW_ERR_ARG;
  if (!aligned(a->q_dev, 16) || !aligned(a->out_dev, 16) || !aligned(a->cu_q_dev, 4) ||
      !aligned(a->kv_len_dev, 4) || !aligned(a->table_dev, 4) || !aligned(a->lse_dev, 4) ||
      !aligned(a->flags_dev, 4))
    return UW_ERR_ARG;
  const int64_t width = (int64_t)a->n_heads * a->cache.head_dim;
  if (a->q_stride % 8 || a->out_stride % 8 || a->q_stride < 0 || a->out_stride < 0 ||
      (a->n_rows > 1 && (a->q_stride < width || a->out_stride < width)))
    return UW_ERR_ARG;
  if (!a->ws_dev || !aligned(a->ws_dev, 256)) return UW_ERR_ARG;
  if (a->ws_bytes < need) return UW_ERR_WORKSPACE;
  int dev = 0;
  st = device_of(a->q_dev, &dev);
  if (st != UW_OK) return st;
  DeviceGuard g(dev);
  AttnParams p;
  p.a = *a;
  p.group = a->n_heads / a->cache.n_kv_heads;
  p.per_tile = kRows / p.group;
  p.page_shift = 0;
  while ((1 << p.page_shift) < a->cache.page_size) ++p.page_shift;
  // s = scale q . k with the scale's size in the exponent's factor; a negative
  // one turns the scores' signs, zero makes them zero
  p.scale_log2 = std::fabs(a->scale) * 1.4426950408889634f;
  p.turn = !(a->scale > 0.f);
  p.s_and = p.scale_log2 == 0.f ? 0 : 0xFFFFFFFFu;
  p.s_xor = a->scale < 0.f && p.s_and ? 0x80000000u : 0;
  if (!p.s_and) {
    p.turn = 1;
    p.scale_log2 = 1.f;
  }
  if (!windowed) p.a.window = 0;
  p.wait_ns = wait_limit_ns();
  // Failure-detection tests (the GEMM's switch, read once per process): units of two row tiles never signal
  // the second one's outputs, so that waits run out; single tokens go on as ever.
  static const int withhold = std::getenv("UW_TEST_WITHHOLD_HANDOFF") ? 1 : 0;
  p.withhold = withhold;
  if (!make_q_map(&p.q, *a, p.group, p.per_tile) || !make_q_map(&p.q_one, *a, p.group, 1) ||
      !make_map(&p.k, a->cache.k_dev, a->cache) ||
      !make_map(&p.v, a->cache.v_dev, a->cache))
    return UW_ERR_UNSUPPORTED;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int sms = sm_count_of(dev);
  return map_launch(a->cache.head_dim == 64 ? launch_attention<64>(p, sms, s) : launch_attention<128>(p, sms, s));
}

}  // extern "C"
