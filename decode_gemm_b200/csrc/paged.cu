// The paged key/value cache around the attention: block tables and slot maps
// from the requests' lengths (uw_paged_plan), and the norms and the rotation of
// queries and keys in the pass that writes the cache (uw_qk_norm_rope).
#include <cuda_runtime.h>

#include <algorithm>
#include <mutex>

#include "gemm_sm100.cuh"
#include "handle.h"
#include "pdl.cuh"
#include "serving.h"

namespace uw {

int sm_count_of(int dev) {
  static std::mutex mu;
  static int known[64] = {0};
  if (dev < 0 || dev >= 64) return 148;
  std::lock_guard<std::mutex> lock(mu);
  if (!known[dev]) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = 148;
    known[dev] = n;
  }
  return known[dev];
}

uw_status check_cache(const uw_paged_cache& c) {
  if (!c.k_dev || !c.v_dev || !aligned(c.k_dev, 16) || !aligned(c.v_dev, 16)) return UW_ERR_ARG;
  if (c.n_pages < 1 || c.n_pages > INT32_MAX || c.n_kv_heads < 1 || c.head_dim < 1) return UW_ERR_SHAPE;
  if (c.page_size < 8 || c.page_size > 1024 || (c.page_size & (c.page_size - 1))) return UW_ERR_UNSUPPORTED;
  const int64_t top = int64_t(1) << 39;
  int64_t st[3] = {c.page_stride, c.slot_stride, c.head_stride};
  int64_t n[3] = {c.n_pages, c.page_size, c.n_kv_heads};
  for (int64_t s : st)
    if (s <= 0 || s % 8 || s >= top) return UW_ERR_ARG;
  // no overlap: with the axes by rising stride, each steps over all that lies
  // inside it (an axis of one entry is never stepped along)
  for (int i = 0; i < 2; ++i)
    for (int j = i + 1; j < 3; ++j)
      if (st[j] < st[i]) {
        std::swap(st[i], st[j]);
        std::swap(n[i], n[j]);
      }
  int64_t extent = c.head_dim;
  for (int i = 0; i < 3; ++i) {
    if (n[i] > 1 && st[i] < extent) return UW_ERR_ARG;
    extent += st[i] * (n[i] - 1);
    if (extent > (int64_t(1) << 46)) return UW_ERR_SHAPE;
  }
  return UW_OK;
}

namespace {

using namespace sm100;

// ---------------------------------------------------------------- the plan ----
//
// A few integers per request and per row: latency is all of its time.  One
// launch: a cluster of CTAs, each of which scans all requests for itself (the
// scan's inputs are a few KB in L2) and then writes its share of the rows and
// of the new pages' table entries, each found by bisection in the scan.  The
// cluster's barrier separates everyone's reads from the first write, so lengths
// and list head may be updated in place.

constexpr int kPlanThreads = 512;
constexpr int kPlanMaxRequests = 8192;
constexpr size_t plan_shared_bytes(int requests) { return ((size_t)4 * requests + 2) * 4; }

struct PlanParams {
  uw_paged_plan_args a;
  int shift;  // log2(page_size)
};

__device__ __forceinline__ int64_t pages_of(int64_t tokens, int shift) {
  return (tokens + (int64_t(1) << shift) - 1) >> shift;
}

// Largest b in [0, n) with first[b] <= x (first[0] = 0 <= x, first rising).
__device__ __forceinline__ int bisect(const int32_t* first, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kPlanThreads) paged_plan_kernel(const __grid_constant__ PlanParams p) {
  const uw_paged_plan_args& a = p.a;
  extern __shared__ int32_t sh[];
  const int n = a.n_requests, t = threadIdx.x, lane = t & 31, warp = t >> 5;
  int32_t* s_cu = sh;               // [n + 1] first row
  int32_t* s_first = s_cu + n + 1;  // [n + 1] first taken entry, among this call's
  int32_t* s_ctx = s_first + n + 1; // [n] stored tokens; -1: refused
  int32_t* s_at = s_ctx + n;        // [n] first position (what a refused request's rows still get)
  __shared__ int64_t s_rows[kPlanThreads / 32], s_need[kPlanThreads / 32];
  __shared__ int32_t s_taken;
  pdl_wait();
  pdl_release();
  const int32_t head0 = a.head_in_dev ? *a.head_in_dev : 0;
  const int32_t head = head0 < 0 ? 0 : (head0 > a.n_free ? a.n_free : head0);
  bool bad = head != head0;
  const int64_t avail = a.n_free - head;
  const int64_t most = min((int64_t)a.table_width << p.shift, (int64_t)INT32_MAX);
  // each thread scans a run of consecutive requests
  const int per = (n + kPlanThreads - 1) / kPlanThreads;
  const int b0 = min(t * per, n), b1 = min(b0 + per, n);
  int64_t rows = 0, need = 0;
  for (int b = b0; b < b1; ++b) {
    const int64_t ctx = a.ctx_len_dev[b], fresh = a.new_len_dev[b];
    rows += fresh > 0 ? fresh : 0;
    if (ctx >= 0 && fresh >= 0 && ctx + fresh <= most)
      need += pages_of(ctx + fresh, p.shift) - pages_of(ctx, p.shift);
  }
  int64_t rows_in = rows, need_in = need;  // inclusive scans over the block
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t r = __shfl_up_sync(0xFFFFFFFFu, rows_in, d), q = __shfl_up_sync(0xFFFFFFFFu, need_in, d);
    if (lane >= d) {
      rows_in += r;
      need_in += q;
    }
  }
  if (lane == 31) {
    s_rows[warp] = rows_in;
    s_need[warp] = need_in;
  }
  if (t == 0) s_taken = 0;
  __syncthreads();
  for (int w = 0; w < warp; ++w) {
    rows_in += s_rows[w];
    need_in += s_need[w];
  }
  int64_t row = rows_in - rows, first = need_in - need;
  int32_t taken = 0;
  for (int b = b0; b < b1; ++b) {
    const int64_t ctx = a.ctx_len_dev[b], len = a.new_len_dev[b], fresh = len > 0 ? len : 0;
    const bool sound = ctx >= 0 && len >= 0 && ctx + fresh <= most;
    const int64_t want = sound ? pages_of(ctx + fresh, p.shift) - pages_of(ctx, p.shift) : 0;
    const bool fits = row + fresh <= a.n_rows || fresh == 0;
    const bool granted = sound && fits && (want == 0 || first + want <= avail);
    s_cu[b] = (int32_t)min(row, a.n_rows);
    s_first[b] = (int32_t)min(first, avail);
    s_ctx[b] = granted ? (int32_t)ctx : -1;
    s_at[b] = (int32_t)(sound ? ctx : 0);
    if (granted && want > 0) taken = (int32_t)(first + want);
    bad |= !granted;
    row += fresh;
    // a request whose rows do not fit takes no pages, but none behind it has rows either
    first += want;
  }
  if (b1 == n && b0 < b1) {
    s_cu[n] = (int32_t)min(row, a.n_rows);
    s_first[n] = (int32_t)min(first, avail);
  }
  if (n == 0 && t == 0) s_cu[0] = s_first[0] = 0;
  if (taken) atomicMax(&s_taken, taken);
  if (bad && a.flags_dev && blockIdx.x == 0) atomicOr(a.flags_dev, (uint32_t)UW_FLAG_BAD_INPUT);
  __syncthreads();
  // every CTA has read the lengths and the list's head: now they may change
  if (gridDim.x > 1) cluster_sync();

  const int64_t me = (int64_t)blockIdx.x * kPlanThreads + t, all = (int64_t)gridDim.x * kPlanThreads;
  const int32_t got = s_taken;
  if (me == 0) {
    *a.head_out_dev = head + got;
    a.cu_q_dev[n] = s_cu[n];
  }
  for (int64_t b = me; b < n; b += all) {
    const int32_t ctx = s_ctx[b];
    a.cu_q_dev[b] = s_cu[b];
    // (a granted request's rows all fit, so its cu_q difference is its new length)
    a.kv_len_dev[b] = ctx < 0 ? 0 : ctx + (s_cu[b + 1] - s_cu[b]);
  }
  for (int64_t j = me; j < got; j += all) {
    const int b = bisect(s_first, n, (int)j);
    if (s_ctx[b] < 0) continue;
    const int64_t col = pages_of(s_ctx[b], p.shift) + (j - s_first[b]);
    a.table_dev[b * a.table_stride + col] = a.free_pages_dev[head + j];
  }
  const int32_t live = s_cu[n];
  // a few rows at a time, so that their page ids are fetched together
  constexpr int kAhead = 4;
  for (int64_t r0 = me; r0 < a.n_rows; r0 += kAhead * all) {
    int32_t pos[kAhead], page[kAhead];
    bool wanted[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int64_t r = r0 + j * all;
      pos[j] = page[j] = 0;
      wanted[j] = false;
      if (r < live) {
        const int b = bisect(s_cu, n, (int)r);
        const int32_t ctx = s_ctx[b];
        pos[j] = s_at[b] + ((int32_t)r - s_cu[b]);
        if (ctx >= 0) {
          const int64_t col = pos[j] >> p.shift, held = pages_of(ctx, p.shift);
          wanted[j] = true;
          page[j] = col < held ? a.table_dev[b * a.table_stride + col]
                               : a.free_pages_dev[head + s_first[b] + (int32_t)(col - held)];
        }
      }
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int64_t r = r0 + j * all;
      if (r >= a.n_rows) break;
      if (wanted[j] && page[j] < 0 && a.flags_dev) atomicOr(a.flags_dev, (uint32_t)UW_FLAG_BAD_INPUT);
      a.positions_dev[r] = pos[j];
      a.slots_dev[r] = wanted[j] && page[j] >= 0
                           ? ((int64_t)page[j] << p.shift) + (pos[j] & ((1 << p.shift) - 1))
                           : -1;
    }
  }
}

// ---------------------------------------------- norms, rotation, cache update --
//
// Every value is read once and written once; at a few instructions per value
// that stays bound by memory.  A warp takes one row, or a share of a row's
// heads where the rows are too few to fill the GPU.  LANES lanes hold a head,
// each four of its pairs (eight values, two 8-byte loads), and the warp steps
// over its heads: so a pair lies in one lane, the lane keeps the same pairs of
// every head, and their turns, multiplied with the norm's weights, stay in
// registers.  8192 rows of 32 + 2 x 8 heads of 128: 40 us, 5.0 TB/s (the
// first form, with partners in other lanes and 94 registers, 66 us).

constexpr int kRopeWarps = 4;
constexpr int kRopeMaxPairs = 128;  // rot_dim / 2

struct RopeParams {
  uw_qk_norm_rope_args a;
  int32_t share;      // warps per row
  int32_t n_q, n_k;   // head groups (32 / LANES heads) of q, and of k or v
  int32_t page_shift;
};

__device__ __forceinline__ float low_of(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high_of(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// A lane's eight values of a head as four pairs (first[i], second[i]).
struct Eight {
  uint2 x, y;  // as they lie at the lane's two places
};
template <bool INTERLEAVED>
__device__ __forceinline__ void pairs_of(const Eight& v, float (&first)[4], float (&second)[4]) {
  if constexpr (INTERLEAVED) {
    const uint32_t w[4] = {v.x.x, v.x.y, v.y.x, v.y.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) first[i] = low_of(w[i]), second[i] = high_of(w[i]);
  } else {
    first[0] = low_of(v.x.x), first[1] = high_of(v.x.x), first[2] = low_of(v.x.y), first[3] = high_of(v.x.y);
    second[0] = low_of(v.y.x), second[1] = high_of(v.y.x), second[2] = low_of(v.y.y), second[3] = high_of(v.y.y);
  }
}
template <bool INTERLEAVED>
__device__ __forceinline__ Eight eight_of(const float (&first)[4], const float (&second)[4]) {
  if constexpr (INTERLEAVED)
    return {make_uint2(bf16_pair(first[0], second[0]), bf16_pair(first[1], second[1])),
            make_uint2(bf16_pair(first[2], second[2]), bf16_pair(first[3], second[3]))};
  else
    return {make_uint2(bf16_pair(first[0], first[1]), bf16_pair(first[2], first[3])),
            make_uint2(bf16_pair(second[0], second[1]), bf16_pair(second[2], second[3]))};
}

template <int LANES, bool INTERLEAVED>
__global__ void __launch_bounds__(kRopeWarps * 32, 8) qk_norm_rope_kernel(const __grid_constant__ RopeParams p) {
  const uw_qk_norm_rope_args& a = p.a;
  __shared__ float2 s_turn[kRopeWarps][kRopeMaxPairs];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t unit = (int64_t)blockIdx.x * kRopeWarps + warp;
  const int64_t row = unit / p.share;
  const int part = (int)(unit - row * p.share);
  pdl_wait();
  pdl_release();
  if (row >= a.n_rows) return;
  constexpr int kPer = 32 / LANES;              // heads per step
  const int dim = a.cache.head_dim, half = a.rot_dim >> 1;
  const int e = lane % LANES, sub = lane / LANES;
  const bool on = e * 8 < dim;                  // (dim / 8 need not be a power of two)
  const bool turned = e * 8 < a.rot_dim;
  // the lane's two places in a head: the halves of its pairs, or eight values
  // in a row (neighbouring pairs, and what is not turned)
  const int at0 = INTERLEAVED || !turned ? e * 8 : e * 4;
  const int at1 = INTERLEAVED || !turned ? e * 8 + 4 : half + e * 4;
  const int64_t slot = a.slots_dev[row];
  const int64_t page = slot >> p.page_shift;
  const bool stored = slot >= 0 && page < a.cache.n_pages;
  if (!stored && slot != -1 && lane == 0 && part == 0 && a.flags_dev)
    atomicOr(a.flags_dev, (uint32_t)UW_FLAG_BAD_INPUT);
  // the row's angles: position times frequency in 64 bits, brought to one turn
  // there, so that far positions keep the precision of near ones
  const double pos = (double)a.positions_dev[row];
  for (int i = lane; i < half; i += 32) {
    const double turns = pos * (double)a.inv_freq_dev[i] * 0.15915494309189533577;  // 1 / (2 pi)
    float2 cs;
    sincospif((float)((turns - rint(turns)) * 2.0), &cs.y, &cs.x);
    s_turn[warp][i] = cs;
  }
  __syncwarp();

  const float inv_dim = 1.f / (float)dim;
  constexpr int kAhead = 4;  // steps whose loads are in flight together
  // heads [h0, h1) of `src`, turned, to `dst`; both point at the lane's first head
  const auto run = [&](const uint16_t* src, uint16_t* dst, int64_t dst_stride, const uint16_t* weight, int heads,
                       int s0, int s1) {
    // (f, g) -> (f A - g B, g C + f D)
    float A[4], B[4], C[4], D[4];
    {
      float w0[4] = {1.f, 1.f, 1.f, 1.f}, w1[4] = {1.f, 1.f, 1.f, 1.f};
      if (on && weight) {
        const Eight w = {*reinterpret_cast<const uint2*>(weight + at0), *reinterpret_cast<const uint2*>(weight + at1)};
        pairs_of<INTERLEAVED>(w, w0, w1);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 cs = turned ? s_turn[warp][e * 4 + i] : make_float2(1.f, 0.f);
        A[i] = w0[i] * cs.x;
        B[i] = w1[i] * cs.y;
        C[i] = w1[i] * cs.x;
        D[i] = w0[i] * cs.y;
      }
    }
    for (int st = s0; st < s1; st += kAhead) {
      Eight raw[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int h = (st + j) * kPer + sub;
        raw[j] = {make_uint2(0, 0), make_uint2(0, 0)};
        if (st + j < s1 && on && h < heads) {
          raw[j].x = *reinterpret_cast<const uint2*>(src + (int64_t)h * dim + at0);
          raw[j].y = *reinterpret_cast<const uint2*>(src + (int64_t)h * dim + at1);
        }
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        if (st + j >= s1) break;  // (the same in the whole warp)
        float f[4], g[4], y[4], z[4];
        pairs_of<INTERLEAVED>(raw[j], f, g);
        float r = 1.f;
        if (weight) {
          float ss = 0.f;
#pragma unroll
          for (int i = 0; i < 4; ++i) ss = fmaf(f[i], f[i], fmaf(g[i], g[i], ss));
#pragma unroll
          for (int d = LANES / 2; d; d >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, d);
          r = rsqrtf(fmaf(ss, inv_dim, a.eps));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          y[i] = r * (turned ? fmaf(f[i], A[i], -(g[i] * B[i])) : f[i] * A[i]);
          z[i] = r * (turned ? fmaf(g[i], C[i], f[i] * D[i]) : g[i] * C[i]);
        }
        const int h = (st + j) * kPer + sub;
        if (on && h < heads) {
          const Eight o = eight_of<INTERLEAVED>(y, z);
          *reinterpret_cast<uint2*>(dst + h * dst_stride + at0) = o.x;
          *reinterpret_cast<uint2*>(dst + h * dst_stride + at1) = o.y;
        }
      }
    }
  };
  // this warp's share of the row's steps, over q, k and v
  const int steps = p.n_q + 2 * p.n_k, per_part = (steps + p.share - 1) / p.share;
  const int st0 = part * per_part, st1 = min(st0 + per_part, steps);
  if (st0 < p.n_q)
    run(a.q_dev + row * a.q_stride, a.q_out_dev + row * a.q_out_stride, dim, a.q_weight_dev, a.n_heads, st0,
        min(st1, p.n_q));
  if (!stored) return;
  const int64_t at = page * a.cache.page_stride + (slot & ((1 << p.page_shift) - 1)) * a.cache.slot_stride;
  if (st0 < p.n_q + p.n_k && st1 > p.n_q)
    run(a.k_dev + row * a.k_stride, a.cache.k_dev + at, a.cache.head_stride, a.k_weight_dev, a.cache.n_kv_heads,
        max(st0 - p.n_q, 0), min(st1 - p.n_q, p.n_k));
  const uint16_t* v = a.v_dev + row * a.v_stride;
  for (int st = max(st0 - p.n_q - p.n_k, 0); st < st1 - p.n_q - p.n_k; st += kAhead) {
    uint4 raw[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int h = (st + j) * kPer + sub;
      if (st + j < st1 - p.n_q - p.n_k && on && h < a.cache.n_kv_heads)
        raw[j] = *reinterpret_cast<const uint4*>(v + (int64_t)h * dim + e * 8);
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int h = (st + j) * kPer + sub;
      if (st + j < st1 - p.n_q - p.n_k && on && h < a.cache.n_kv_heads)
        *reinterpret_cast<uint4*>(a.cache.v_dev + at + h * a.cache.head_stride + e * 8) = raw[j];
    }
  }
}

template <bool INTERLEAVED>
cudaError_t launch_rope(const RopeParams& p, int lanes, dim3 grid, cudaStream_t s) {
  const dim3 block(kRopeWarps * 32);
  switch (lanes) {
    case 2: return launch_pdl(qk_norm_rope_kernel<2, INTERLEAVED>, grid, block, 0, s, p);
    case 4: return launch_pdl(qk_norm_rope_kernel<4, INTERLEAVED>, grid, block, 0, s, p);
    case 8: return launch_pdl(qk_norm_rope_kernel<8, INTERLEAVED>, grid, block, 0, s, p);
    case 16: return launch_pdl(qk_norm_rope_kernel<16, INTERLEAVED>, grid, block, 0, s, p);
    default: return launch_pdl(qk_norm_rope_kernel<32, INTERLEAVED>, grid, block, 0, s, p);
  }
}

int log2_of(int x) {
  int s = 0;
  while ((1 << s) < x) ++s;
  return s;
}

}  // namespace
}  // namespace uw

using namespace uw;

extern "C" {

uw_status uw_paged_plan(const uw_paged_plan_args* a, void* stream) {
  if (!a) return UW_ERR_ARG;
  if (a->n_requests < 0 || a->n_requests > kPlanMaxRequests || a->n_rows < 0 ||
      a->n_rows > (int64_t(1) << 30) || a->n_free < 0 || a->table_width < 0)
    return UW_ERR_SHAPE;
  if (a->page_size < 1 || a->page_size > 1024 || (a->page_size & (a->page_size - 1)))
    return UW_ERR_UNSUPPORTED;
  if (!a->cu_q_dev || !a->head_out_dev) return UW_ERR_ARG;
  if (a->n_requests > 0) {
    if (!a->ctx_len_dev || !a->new_len_dev || !a->kv_len_dev) return UW_ERR_ARG;
    if (a->table_width > 0 && (!a->table_dev || a->table_stride < a->table_width)) return UW_ERR_ARG;
  }
  if (a->n_free > 0 && !a->free_pages_dev) return UW_ERR_ARG;
  if (a->n_rows > 0 && (!a->positions_dev || !a->slots_dev)) return UW_ERR_ARG;
  for (const void* q : {(const void*)a->ctx_len_dev, (const void*)a->new_len_dev,
                        (const void*)a->free_pages_dev, (const void*)a->head_in_dev,
                        (const void*)a->head_out_dev, (const void*)a->table_dev,
                        (const void*)a->cu_q_dev, (const void*)a->kv_len_dev,
                        (const void*)a->positions_dev, (const void*)a->flags_dev})
    if (!aligned(q, 4)) return UW_ERR_ARG;
  if (!aligned(a->slots_dev, 8)) return UW_ERR_ARG;
  int dev = 0;
  const uw_status st = device_of(a->cu_q_dev, &dev);
  if (st != UW_OK) return st;
  DeviceGuard g(dev);
  PlanParams p;
  p.a = *a;
  p.shift = log2_of(a->page_size);
  // one CTA while a few rows per thread are all there is (no barrier between
  // CTAs then), else the eight of the largest portable cluster
  const int cluster = a->n_rows <= 4 * kPlanThreads && a->n_requests <= 4 * kPlanThreads ? 1 : 8;
  const size_t smem = plan_shared_bytes(a->n_requests);
  // (The limit is the kernel's, not this call's: set to the most that any call needs, so that no other
  // thread's call lowers it before the launch.  Without it 48 KB are the limit of this and of the kernel's
  // own arrays together; half of that leaves them room.)
  if (smem > 24 * 1024 &&
      cudaFuncSetAttribute(paged_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           (int)plan_shared_bytes(kPlanMaxRequests)) != cudaSuccess)
    return map_launch(cudaGetLastError());
  return map_launch(launch_pdl_cluster(paged_plan_kernel, dim3(cluster), cluster, dim3(kPlanThreads), smem,
                                       static_cast<cudaStream_t>(stream), p));
}

uw_status uw_qk_norm_rope(const uw_qk_norm_rope_args* a, void* stream) {
  if (!a) return UW_ERR_ARG;
  if (a->n_rows < 0 || a->n_rows > (int64_t(1) << 30) || a->n_heads < 1 || a->n_heads > 65536) return UW_ERR_SHAPE;
  const uw_status cs = check_cache(a->cache);
  if (cs != UW_OK) return cs;
  const int dim = a->cache.head_dim;
  if (dim % 16 || dim < 16 || dim > 256) return UW_ERR_UNSUPPORTED;
  if (a->rot_dim < 0 || a->rot_dim > dim || a->rot_dim % 16) return UW_ERR_UNSUPPORTED;
  if (!(a->eps >= 0.f)) return UW_ERR_ARG;
  if (a->n_rows == 0) return UW_OK;
  if (!a->q_dev || !a->k_dev || !a->v_dev || !a->q_out_dev || !a->positions_dev || !a->slots_dev ||
      (a->rot_dim > 0 && !a->inv_freq_dev))
    return UW_ERR_ARG;
  for (const void* q : {(const void*)a->q_dev, (const void*)a->k_dev, (const void*)a->v_dev,
                        (const void*)a->q_out_dev, (const void*)a->q_weight_dev, (const void*)a->k_weight_dev})
    if (!aligned(q, 16)) return UW_ERR_ARG;
  if (!aligned(a->positions_dev, 4) || !aligned(a->inv_freq_dev, 4) || !aligned(a->flags_dev, 4) ||
      !aligned(a->slots_dev, 8))
    return UW_ERR_ARG;
  const int64_t qw = (int64_t)a->n_heads * dim, kw = (int64_t)a->cache.n_kv_heads * dim;
  const int64_t st4[4] = {a->q_stride, a->k_stride, a->v_stride, a->q_out_stride};
  const int64_t w4[4] = {qw, kw, kw, qw};
  for (int i = 0; i < 4; ++i)
    if (st4[i] % 8 || st4[i] < 0 || (a->n_rows > 1 && st4[i] < w4[i])) return UW_ERR_ARG;
  if (a->q_out_dev == a->q_dev && a->q_out_stride != a->q_stride) return UW_ERR_ARG;
  int dev = 0;
  const uw_status st = device_of(a->q_dev, &dev);
  if (st != UW_OK) return st;
  DeviceGuard g(dev);
  RopeParams p;
  p.a = *a;
  int lanes = 2;
  while (lanes * 8 < dim) lanes *= 2;
  const int per = 32 / lanes;
  p.n_q = (a->n_heads + per - 1) / per;
  p.n_k = (a->cache.n_kv_heads + per - 1) / per;
  p.page_shift = log2_of(a->cache.page_size);
  // a warp per row once that gives every SM 16 warps, else the row's head
  // groups over as many warps as reach that
  const int64_t want = (int64_t)sm_count_of(dev) * 16;
  p.share = (int)std::max<int64_t>(1, std::min<int64_t>(p.n_q + 2 * p.n_k, want / a->n_rows));
  const int64_t units = a->n_rows * p.share;
  const int64_t grid = (units + kRopeWarps - 1) / kRopeWarps;
  if (grid > INT32_MAX) return UW_ERR_SHAPE;
  const dim3 blocks((unsigned)grid);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return map_launch(a->interleaved ? launch_rope<true>(p, lanes, blocks, s) : launch_rope<false>(p, lanes, blocks, s));
}

}  // extern "C"
