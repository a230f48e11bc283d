// gla_cache.cuh -- the paged 8-bit rollout cache of the softmax anchor layers:
// the plan (block tables and slot maps from sequence lengths) and the store
// (e4m3 codes with one power-of-two scale for each page and key/value head).
//
// Cache layout: k, v codes [pages, Hkv, P, d] (one page of one head is P * d
// contiguous bytes), scales fp32 [pages, Hkv].  block_table[r][j] is the page
// that holds tokens j P .. j P + P - 1 of sequence r.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "sm100_ptx.cuh"

namespace gla {

constexpr int kCacheMaxSeqs = 8192;   // sequences of one call (their prefix sums sit in shared
                                      // memory)

__host__ __device__ __forceinline__ int64_t ceil_div64(int64_t a, int64_t b) {
  return (a + b - 1) / b;
}

// First index of `a[0 .. n]` (ascending, a[0] = 0) whose successor exceeds x:
// the owner of item x of a prefix sum.  0 <= x < a[n].
template <typename T>
__device__ __forceinline__ int prefix_owner(const T* a, int n, T x) {
  int lo = 0, hi = n;  // a[lo] <= x < a[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a[mid] <= x)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// Exclusive prefix sums over the threads of a block (whole warps, at most
// 1024 threads); `total` is the sum over all of them.  `scratch`: 33 values.
// Ends with every thread past its reads of `scratch`.
template <typename T>
__device__ __forceinline__ T block_exclusive_scan(T v, T* scratch, T& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  T x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) scratch[warp] = x;
  __syncthreads();
  if (warp == 0) {
    T w = lane < warps ? scratch[lane] : T(0);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const T y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    scratch[lane] = w;
  }
  __syncthreads();
  const T base = warp > 0 ? scratch[warp - 1] : T(0);
  total = scratch[warps - 1];
  __syncthreads();
  return base + x - v;
}

// ------------------------------------------------------------------- plan

struct PlanParams {
  const int *lens, *held, *new_lens, *free_count;
  int *free_pages, *table, *lens_out, *held_out, *free_count_out, *cu, *slots, *status;
  int R, max_pages, pages, P, tokens, F, W, n_sink;
};

constexpr int kPlanThreads = 1024;

// The pages of one sequence in this step.
struct PlanSeq {
  int64_t L, n;        // cached tokens, new tokens (0 for a finished sequence)
  int64_t np_old, np_new;
  int64_t held_out;
  int64_t sink_back;   // finished: pages 0 .. sink_back - 1 go back too
  int64_t back_lo, back_hi;
  bool done;
  __device__ int64_t back() const { return sink_back + back_hi - back_lo; }
};

__device__ __forceinline__ PlanSeq plan_seq(const PlanParams& p, int r) {
  PlanSeq s;
  s.L = p.lens[r] > 0 ? p.lens[r] : 0;
  const int64_t nl = p.new_lens[r];
  const int64_t held = p.held[r] > 0 ? p.held[r] : 0;
  s.done = nl < 0;
  s.n = s.done ? 0 : nl;
  const int64_t sp = ceil_div64(p.n_sink, p.P);
  s.np_old = ceil_div64(s.L, p.P);
  s.np_new = s.done ? s.np_old : ceil_div64(s.L + s.n, p.P);
  int64_t low = 0;
  if (p.W > 0) {
    const int64_t w_lo = (s.L / p.F - p.W + 1) * p.F;
    low = w_lo > 0 ? w_lo / p.P : 0;
  }
  const int64_t upto = s.done ? s.np_old : (held > low ? held : low);
  s.held_out = s.done ? 0 : upto;
  s.back_lo = held > sp ? held : sp;
  s.back_hi = upto > s.back_lo ? upto : s.back_lo;
  s.sink_back = s.done ? (s.np_old < sp ? s.np_old : sp) : 0;
  return s;
}

__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

// One thread-block cluster does a whole step in one launch.  Every CTA sums
// new tokens, new pages and returned pages over all sequences for itself (a
// few KB from L2; cheaper than a second launch), pushes its share of the
// returned pages, and after the cluster barrier, which also orders those
// pushes and everybody's reads of the lengths before any write over them (the
// outputs may be the inputs), takes its share of the slots.  The new page of
// rank i in (sequence, page) order is entry free + returned - 1 - i of the
// stack, so no thread depends on another one's pop.
// Bound by latency: measured at 256 sequences and 256 tokens 1 CTA, at 2048
// sequences and half a million tokens 8 CTAs.
__global__ void __launch_bounds__(kPlanThreads, 1) gla_cache_plan_kernel(const PlanParams p) {
  extern __shared__ int plan_smem[];
  __shared__ long long scratch[33];
  int* s_cu = plan_smem;              // [R + 1] new tokens
  int* s_need = s_cu + p.R + 1;       // [R + 1] new pages
  int* s_back = s_need + p.R + 1;     // [R + 1] returned pages
  int* s_len = s_back + p.R + 1;      // [R] cached tokens
  const int tid = threadIdx.x;
  const int ctas = gridDim.x, cta = blockIdx.x;

  // sums over this thread's sequences, then over the block
  const int per = (p.R + kPlanThreads - 1) / kPlanThreads;
  const int r0 = min(p.R, tid * per), r1 = min(p.R, r0 + per);
  long long tok = 0, need = 0, back = 0;
  int wide = 0;
  for (int r = r0; r < r1; ++r) {
    const PlanSeq s = plan_seq(p, r);
    tok += s.n;
    need += s.np_new - s.np_old;
    back += s.back();
    wide |= s.np_new > p.max_pages;
  }
  const int too_wide = __syncthreads_or(wide);
  long long tok_all, need_all, back_all;
  tok = block_exclusive_scan<long long>(tok, scratch, tok_all);
  need = block_exclusive_scan<long long>(need, scratch, need_all);
  back = block_exclusive_scan<long long>(back, scratch, back_all);
  const long long free0 = *p.free_count;
  int status = 0;
  if (free0 + back_all < need_all) status |= 1;
  if (tok_all > p.tokens) status |= 2;
  if (too_wide) status |= 4;
  if (free0 < 0 || free0 + back_all > p.pages) status |= 8;
  if (status == 0) {
    for (int r = r0; r < r1; ++r) {
      const PlanSeq s = plan_seq(p, r);
      s_cu[r] = static_cast<int>(tok);
      s_need[r] = static_cast<int>(need);
      s_back[r] = static_cast<int>(back);
      s_len[r] = static_cast<int>(s.L);
      tok += s.n;
      need += s.np_new - s.np_old;
      back += s.back();
    }
    if (tid == 0) {
      s_cu[p.R] = static_cast<int>(tok_all);
      s_need[p.R] = static_cast<int>(need_all);
      s_back[p.R] = static_cast<int>(back_all);
    }
    __syncthreads();
    for (long long i = cta * kPlanThreads + tid; i < back_all; i += ctas * kPlanThreads) {
      const int r = prefix_owner<int>(s_back, p.R, static_cast<int>(i));
      const PlanSeq s = plan_seq(p, r);
      const int64_t k = i - s_back[r];
      const int64_t j = k < s.sink_back ? k : s.back_lo + (k - s.sink_back);
      p.free_pages[free0 + i] = p.table[static_cast<int64_t>(r) * p.max_pages + j];
    }
  }
  // the per-sequence outputs of this CTA's share, computed before the barrier
  // (the inputs may be overwritten after it)
  constexpr int kKeep = kCacheMaxSeqs / kPlanThreads;
  int keep_len[kKeep], keep_held[kKeep];
  if (cta == 0) {
#pragma unroll
    for (int k = 0; k < kKeep; ++k) {
      const int r = tid + k * kPlanThreads;
      if (r < p.R) {
        const PlanSeq s = plan_seq(p, r);
        keep_len[k] = status ? p.lens[r] : (s.done ? 0 : static_cast<int>(s.L + s.n));
        keep_held[k] = status ? p.held[r] : static_cast<int>(s.held_out);
      }
    }
  }
  cluster_sync_all();
  if (cta == 0) {
#pragma unroll
    for (int k = 0; k < kKeep; ++k) {
      const int r = tid + k * kPlanThreads;
      if (r < p.R) {
        p.lens_out[r] = keep_len[k];
        p.held_out[r] = keep_held[k];
      }
    }
    for (int r = tid; r <= p.R; r += kPlanThreads) p.cu[r] = status ? 0 : s_cu[r];
    if (tid == 0) {
      *p.free_count_out = static_cast<int>(status ? free0 : free0 + back_all - need_all);
      *p.status = status;
    }
  }
  // slots, four neighbouring tokens a thread: one search, then a walk
  const long long top = free0 + back_all - 1;
  const int quads = (p.tokens + 3) >> 2;
  const bool vec = (reinterpret_cast<uintptr_t>(p.slots) & 15) == 0;
  for (int qd = cta * kPlanThreads + tid; qd < quads; qd += ctas * kPlanThreads) {
    int out[4] = {-1, -1, -1, -1};
    const int i0 = qd * 4;
    if (status == 0 && i0 < tok_all) {
      int r = prefix_owner<int>(s_cu, p.R, i0);
      int64_t have = ceil_div64(s_len[r], p.P);
      int page = -1;
      int64_t page_j = -1;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = i0 + e;
        if (i >= tok_all) break;
        while (i >= s_cu[r + 1]) {
          ++r;
          have = ceil_div64(s_len[r], p.P);
          page_j = -1;
        }
        const int64_t pos = static_cast<int64_t>(s_len[r]) + (i - s_cu[r]);
        const int64_t j = pos / p.P;
        if (j != page_j) {
          page_j = j;
          int* entry = p.table + static_cast<int64_t>(r) * p.max_pages + j;
          if (j < have) {
            page = *entry;
          } else {
            page = p.free_pages[top - (s_need[r] + (j - have))];
            if (pos % p.P == 0) *entry = page;
          }
        }
        out[e] = page * p.P + static_cast<int>(pos % p.P);
      }
    }
    if (vec && i0 + 3 < p.tokens) {
      *reinterpret_cast<int4*>(p.slots + i0) = make_int4(out[0], out[1], out[2], out[3]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (i0 + e < p.tokens) p.slots[i0 + e] = out[e];
    }
  }
}

// ------------------------------------------------------------------ store

struct StoreParams {
  const __nv_bfloat16 *k, *v;
  const int *lens, *cu, *slots;
  uint8_t *k8, *v8;
  float *ks, *vs;
  int* nonfinite;
  int R, tokens, H, pages;
};

constexpr int kStoreThreads = 128;
constexpr int kScaleMinExp = -60, kScaleMaxExp = 60;

// Exponent e of the smallest power of two with a <= 448 * 2^e, for |a| given
// as finite bf16 bits (448 = 1.75 * 2^8 is the largest e4m3 value), held in
// the range of the scales; 0 takes the smallest.
__device__ __forceinline__ int scale_exponent(uint32_t a) {
  const int e = static_cast<int>(a >> 7) - 127 - 8 + ((a & 127u) > 96u ? 1 : 0);
  return e < kScaleMinExp ? kScaleMinExp : (e > kScaleMaxExp ? kScaleMaxExp : e);
}

__device__ __forceinline__ float exp2_int(int e) {  // 2^e, -126 <= e <= 127
  return __int_as_float((e + 127) << 23);
}

// Two fp32 -> two e4m3 codes (round to nearest even, saturating), `lo` in the
// low byte.
__device__ __forceinline__ uint32_t pack_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Two e4m3 codes (low byte first) -> two fp16, exactly.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t w) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(w)));
  return r;
}

// One work item = the new tokens that one sequence adds to one page, for one
// head and one of K and V: at most P rows of d values, read once into
// registers (the maximum needs all of them before the first code), coded and
// written once.  Items are dealt out with the heads fastest, so that CTAs of
// neighbouring items read whole token rows together.  128 threads keep P d / 8
// / 128 16-byte loads each in flight and many CTAs share an SM.
// Bound by HBM: 2 bytes in and 1 byte out for each value.
template <int D, int P>
__global__ void __launch_bounds__(kStoreThreads) gla_cache_store_kernel(const StoreParams p) {
  constexpr int kRowChunks = D / 8;  // 16-byte chunks of a token row
  constexpr int kRowsPerPass = kStoreThreads / kRowChunks;
  constexpr int kPasses = P > kRowsPerPass ? P / kRowsPerPass : 1;
  extern __shared__ int s_items[];  // [R + 1] prefix sums of the pages each sequence writes
  __shared__ long long scratch[33];
  __shared__ uint32_t s_max[2][kStoreThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int col = tid % kRowChunks, row0 = tid / kRowChunks;

  auto seq = [&](int r, int& c0, int& n, int& old) {
    c0 = min(max(p.cu[r], 0), p.tokens);
    n = max(min(p.cu[r + 1], p.tokens) - c0, 0);
    old = max(p.lens[r] - n, 0);
  };
  {
    const int per = (p.R + kStoreThreads - 1) / kStoreThreads;
    const int r0 = min(p.R, tid * per), r1 = min(p.R, r0 + per);
    long long sum = 0, all;
    for (int r = r0; r < r1; ++r) {
      int c0, n, old;
      seq(r, c0, n, old);
      sum += n > 0 ? (static_cast<int64_t>(old) + n + P - 1) / P - old / P : 0;
    }
    sum = block_exclusive_scan<long long>(sum, scratch, all);
    for (int r = r0; r < r1; ++r) {
      int c0, n, old;
      seq(r, c0, n, old);
      s_items[r] = static_cast<int>(sum);
      sum += n > 0 ? (static_cast<int64_t>(old) + n + P - 1) / P - old / P : 0;
    }
    if (tid == 0) s_items[p.R] = static_cast<int>(all);
    __syncthreads();
  }
  const int64_t items = static_cast<int64_t>(s_items[p.R]) * p.H * 2;
  int bad = 0;
  int flip = 0;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x, flip ^= 1) {
    const int64_t run = it / (2 * p.H);
    const int rest = static_cast<int>(it - run * (2 * p.H));
    const bool is_v = rest >= p.H;
    const int h = is_v ? rest - p.H : rest;
    const int r = prefix_owner<int>(s_items, p.R, static_cast<int>(run));
    int c0, n, old;
    seq(r, c0, n, old);
    const int j = old / P + static_cast<int>(run - s_items[r]);  // page of the sequence
    const int64_t p0 = max(static_cast<int64_t>(j) * P, static_cast<int64_t>(old));
    const int t0 = c0 + static_cast<int>(p0 - old);
    const int slot = p.slots[t0];
    const int page = slot >= 0 ? slot / P : p.pages;
    const int at = slot >= 0 ? slot % P : 0;
    int m = static_cast<int>(min(static_cast<int64_t>(j + 1) * P, static_cast<int64_t>(old) + n) - p0);
    m = page < p.pages ? min(m, P - at) : 0;  // a slot outside the cache: nothing to write

    const __nv_bfloat16* src =
        (is_v ? p.v : p.k) + (static_cast<int64_t>(t0) * p.H + h) * D + col * 8;
    uint4 x[kPasses];
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const int row = row0 + i * kRowsPerPass;
      x[i] = make_uint4(0, 0, 0, 0);
      if (row < m)
        x[i] = __ldcs(reinterpret_cast<const uint4*>(src + static_cast<int64_t>(row) * p.H * D));
    }
    // largest finite magnitude (packed 16-bit maxima of the bf16 bits); NaN
    // becomes 0, infinities stay for the saturating conversion
    uint32_t mx = 0;
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      uint32_t* w = reinterpret_cast<uint32_t*>(&x[i]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t a = w[e] & 0x7FFF7FFFu;
        const uint32_t odd = __vcmpgeu2(a, 0x7F807F80u);  // 0xFFFF where not finite
        if (odd) {
          bad += __popc(odd) >> 4;
          w[e] &= ~__vcmpgtu2(a, 0x7F807F80u);
        }
        mx = __vmaxu2(mx, a & ~odd);
      }
    }
    mx = max(mx & 0xFFFFu, mx >> 16);
    mx = __reduce_max_sync(0xffffffffu, mx);
    if (lane == 0) s_max[flip][warp] = mx;
    __syncthreads();  // the other half of s_max is free again after this barrier
    mx = max(max(s_max[flip][0], s_max[flip][1]), max(s_max[flip][2], s_max[flip][3]));
    if (m <= 0) continue;  // uniform over the block
    const int64_t blk = static_cast<int64_t>(page) * p.H + h;
    float* scale_p = (is_v ? p.vs : p.ks) + blk;
    uint8_t* dst = (is_v ? p.v8 : p.k8) + blk * (P * D);
    float scale = exp2_int(scale_exponent(mx));
    float was = 0.f;
    if (at > 0) {
      was = *scale_p;
      scale = fmaxf(scale, was);
    }
    const float inv = 1.0f / scale;  // exact: a power of two unless `was` is not one
    const bool exact = (__float_as_uint(scale) & 0x7FFFFFu) == 0;
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const int row = row0 + i * kRowsPerPass;
      const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
      uint32_t c[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float lo = bf16lo_to_f32(w[e]), hi = bf16hi_to_f32(w[e]);
        c[e] = exact ? pack_e4m3x2(lo * inv, hi * inv) : pack_e4m3x2(lo / scale, hi / scale);
      }
      if (row < m)
        *reinterpret_cast<uint2*>(dst + (at + row) * D + col * 8) =
            make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
    }
    if (at > 0 && scale != was) {  // the page's scale grew: its earlier tokens are coded again
      const float ratio = was / scale;
      for (int i = tid; i < at * (D / 4); i += kStoreThreads) {
        uint32_t* w = reinterpret_cast<uint32_t*>(dst) + i;
        const uint32_t q = *w;
        const uint32_t f0 = e4m3x2_to_f16x2(q & 0xFFFFu), f1 = e4m3x2_to_f16x2(q >> 16);
        const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&f0));
        const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&f1));
        *w = pack_e4m3x2(a.x * ratio, a.y * ratio) | (pack_e4m3x2(b.x * ratio, b.y * ratio) << 16);
      }
    }
    // every thread has read the old scale before one replaces it
    if (at > 0) __syncthreads();
    if (tid == 0) *scale_p = scale;
  }
  if (p.nonfinite != nullptr) {
    bad = __reduce_add_sync(0xffffffffu, bad);
    if (lane == 0 && bad) atomicAdd(p.nonfinite, bad);
  }
}

}  // namespace gla
