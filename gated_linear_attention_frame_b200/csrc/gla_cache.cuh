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
// 1024 threads) of N values at once; `total` are the sums over all of them.
// `scratch`: 33 N values.  Ends with every thread past its reads of `scratch`.
template <int N, typename T>
__device__ __forceinline__ void block_exclusive_scan_n(T (&v)[N], T (*scratch)[33], T (&total)[N]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  T x[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    x[i] = v[i];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const T y = __shfl_up_sync(0xffffffffu, x[i], o);
      if (lane >= o) x[i] += y;
    }
    if (lane == 31) scratch[i][warp] = x[i];
  }
  __syncthreads();
  if (warp < N) {
    T w = lane < warps ? scratch[warp][lane] : T(0);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const T y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    scratch[warp][lane] = w;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    v[i] = (warp > 0 ? scratch[i][warp - 1] : T(0)) + x[i] - v[i];
    total[i] = scratch[i][warps - 1];
  }
  __syncthreads();
}

template <typename T>
__device__ __forceinline__ T block_exclusive_scan(T v, T* scratch, T& total) {
  T x[1] = {v}, all[1];
  block_exclusive_scan_n<1, T>(x, reinterpret_cast<T(*)[33]>(scratch), all);
  total = all[0];
  return x[0];
}

// ------------------------------------------------------------------- plan

struct PlanParams {
  const int *lens, *held, *new_lens, *free_count;
  int *free_pages, *table, *lens_out, *held_out, *free_count_out, *cu, *slots, *status;
  int R, max_pages, pages, p_shift, tokens, F, W, n_sink;  // P = 1 << p_shift
};

constexpr int kPlanThreads = 1024;

// The pages of one sequence in this step.
struct PlanSeq {
  int L, n;             // cached tokens, new tokens (0 for a finished sequence)
  int np_old;           // pages held before and after the step, but for the window
  int64_t np_new;
  int held_out;
  int sink_back;        // finished: pages 0 .. sink_back - 1 go back too
  int back_lo, back_hi;
  bool done;
  __device__ int64_t back() const { return static_cast<int64_t>(sink_back) + back_hi - back_lo; }
};

__device__ __forceinline__ int pages_of(int64_t tokens, int p_shift) {
  return static_cast<int>((tokens + (1 << p_shift) - 1) >> p_shift);
}

__device__ __forceinline__ PlanSeq plan_seq(const PlanParams& p, int r) {
  PlanSeq s;
  s.L = max(p.lens[r], 0);
  const int nl = p.new_lens[r];
  const int held = max(p.held[r], 0);
  s.done = nl < 0;
  s.n = s.done ? 0 : nl;
  const int sp = pages_of(p.n_sink, p.p_shift);
  s.np_old = pages_of(s.L, p.p_shift);
  s.np_new = s.done ? s.np_old
                    : (static_cast<int64_t>(s.L) + s.n + (1 << p.p_shift) - 1) >> p.p_shift;
  int low = 0;
  if (p.W > 0) {
    const int64_t w_lo = (static_cast<int64_t>(s.L / p.F) - p.W + 1) * p.F;
    low = w_lo > 0 ? static_cast<int>(w_lo >> p.p_shift) : 0;
  }
  const int upto = s.done ? s.np_old : max(held, low);
  s.held_out = s.done ? 0 : upto;
  s.back_lo = max(held, sp);
  s.back_hi = max(upto, s.back_lo);
  s.sink_back = s.done ? min(s.np_old, sp) : 0;
  return s;
}

// Slots of four neighbouring tokens 4 q .. 4 q + 3 (one search, then a walk along
// the sequences), and the table entries of the pages that begin there.  cu and
// need: prefix sums of the new tokens and new pages; len(r): tokens of sequence
// r before the step; top: stack entry of the first new page.
template <typename Len>
__device__ __forceinline__ void plan_slots(const PlanParams& p, int q, int tokens, const int* cu,
                                           const int* need, int top, Len len) {
  int out[4] = {-1, -1, -1, -1};
  const int i0 = q * 4;
  if (i0 < tokens) {
    int r = prefix_owner<int>(cu, p.R, i0);
    int L = len(r);
    int page = -1, page_j = -1;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = i0 + e;
      if (i >= tokens) break;
      while (i >= cu[r + 1]) {
        L = len(++r);
        page_j = -1;
      }
      const int pos = L + (i - cu[r]);
      const int j = pos >> p.p_shift, at = pos & ((1 << p.p_shift) - 1);
      if (j != page_j) {
        page_j = j;
        const int have = pages_of(L, p.p_shift);
        int* entry = p.table + static_cast<int64_t>(r) * p.max_pages + j;
        if (j < have) {
          page = *entry;
        } else {
          page = p.free_pages[top - (need[r] + (j - have))];
          if (at == 0) *entry = page;
        }
      }
      out[e] = (page << p.p_shift) + at;
    }
  }
  if (i0 + 3 < p.tokens && (reinterpret_cast<uintptr_t>(p.slots) & 15) == 0) {
    *reinterpret_cast<int4*>(p.slots + i0) = make_int4(out[0], out[1], out[2], out[3]);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (i0 + e < p.tokens) p.slots[i0 + e] = out[e];
  }
}

// One CTA: sums new tokens, new pages and returned pages over the sequences,
// pushes the returned pages and writes the lengths.  The outputs may be the
// inputs: everything is read before the barrier that the writes follow.  The new
// page of rank i in (sequence, page) order is entry free + returned - 1 - i of
// the stack, so no thread depends on another one's pop.  kSlots: the slots too
// (few tokens: one launch); otherwise gla_cache_slots_kernel takes them.
// Bound by latency: a handful of dependent trips to L2 (256 sequences: 8 us cold).
template <bool kSlots>
__global__ void __launch_bounds__(kPlanThreads, 1) gla_cache_plan_kernel(const PlanParams p) {
  extern __shared__ int plan_smem[];
  __shared__ long long scratch[3][33];
  int* s_cu = plan_smem;              // [R + 1] new tokens
  int* s_need = s_cu + p.R + 1;       // [R + 1] new pages
  int* s_back = s_need + p.R + 1;     // [R + 1] returned pages
  int* s_len = s_back + p.R + 1;      // [R] cached tokens
  const int tid = threadIdx.x;

  // sums over this thread's sequences, then over the block
  const int per = (p.R + kPlanThreads - 1) / kPlanThreads;
  const int r0 = min(p.R, tid * per), r1 = min(p.R, r0 + per);
  const long long free0 = *p.free_count;
  long long sum[3] = {0, 0, 0}, all[3];  // new tokens, new pages, returned pages
  int wide = 0;
  for (int r = r0; r < r1; ++r) {
    const PlanSeq s = plan_seq(p, r);
    sum[0] += s.n;
    sum[1] += s.np_new - s.np_old;
    sum[2] += s.back();
    wide |= s.np_new > p.max_pages;
  }
  const int too_wide = __syncthreads_or(wide);
  block_exclusive_scan_n<3, long long>(sum, scratch, all);
  int status = 0;
  if (free0 + all[2] < all[1]) status |= 1;
  if (all[0] > p.tokens) status |= 2;
  if (too_wide) status |= 4;
  if (free0 < 0 || free0 + all[2] > p.pages) status |= 8;
  // what the sequences become: kept in registers over the barrier below
  constexpr int kKeep = kCacheMaxSeqs / kPlanThreads;
  int keep_len[kKeep], keep_held[kKeep];
#pragma unroll
  for (int k = 0; k < kKeep; ++k) {
    const int r = r0 + k;
    if (r < r1) {
      const PlanSeq s = plan_seq(p, r);
      keep_len[k] = status ? p.lens[r] : (s.done ? 0 : s.L + s.n);
      keep_held[k] = status ? p.held[r] : s.held_out;
      if (status == 0) {
        s_cu[r] = static_cast<int>(sum[0]);
        s_need[r] = static_cast<int>(sum[1]);
        s_back[r] = static_cast<int>(sum[2]);
        s_len[r] = s.L;
        sum[0] += s.n;
        sum[1] += s.np_new - s.np_old;
        sum[2] += s.back();
      }
    }
  }
  if (tid == 0 && status == 0) {
    s_cu[p.R] = static_cast<int>(all[0]);
    s_need[p.R] = static_cast<int>(all[1]);
    s_back[p.R] = static_cast<int>(all[2]);
  }
  __syncthreads();
  if (status == 0) {
    for (int i = tid; i < static_cast<int>(all[2]); i += kPlanThreads) {
      const int r = prefix_owner<int>(s_back, p.R, i);
      const PlanSeq s = plan_seq(p, r);
      const int k = i - s_back[r];
      const int j = k < s.sink_back ? k : s.back_lo + (k - s.sink_back);
      p.free_pages[free0 + i] = p.table[static_cast<int64_t>(r) * p.max_pages + j];
    }
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kKeep; ++k) {
    const int r = r0 + k;
    if (r < r1) {
      p.lens_out[r] = keep_len[k];
      p.held_out[r] = keep_held[k];
    }
  }
  for (int r = tid; r <= p.R; r += kPlanThreads) p.cu[r] = status ? 0 : s_cu[r];
  if (tid == 0) {
    *p.free_count_out = static_cast<int>(status ? free0 : free0 + all[2] - all[1]);
    *p.status = status;
  }
  if constexpr (kSlots) {
    const int tokens = status ? 0 : static_cast<int>(all[0]);
    const int top = static_cast<int>(free0 + all[2]) - 1;
    for (int q = tid; q < (p.tokens + 3) >> 2; q += kPlanThreads)
      plan_slots(p, q, tokens, s_cu, s_need, top, [&](int r) { return s_len[r]; });
  }
}

// The slots of many tokens, over the whole GPU, from what the plan kernel wrote:
// every CTA sums the new pages for itself (a few KB from L2).
constexpr int kSlotThreads = 512;

__global__ void __launch_bounds__(kSlotThreads) gla_cache_slots_kernel(const PlanParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  extern __shared__ int slot_smem[];
  __shared__ long long scratch[33];
  int* s_cu = slot_smem;           // [R + 1]
  int* s_need = s_cu + p.R + 1;    // [R + 1]
  int* s_len = s_need + p.R + 1;   // [R]
  const int tid = threadIdx.x;
  const int status = *p.status;
  const int per = (p.R + kSlotThreads - 1) / kSlotThreads;
  const int r0 = min(p.R, tid * per), r1 = min(p.R, r0 + per);
  long long sum = 0, all;
  if (status == 0) {
    for (int r = r0; r < r1; ++r) {
      const int c = p.cu[r], n = p.cu[r + 1] - c, L = p.lens_out[r] - n;
      s_cu[r] = c;
      s_len[r] = L;
      s_need[r] = n > 0 ? pages_of(static_cast<int64_t>(L) + n, p.p_shift) - pages_of(L, p.p_shift)
                        : 0;
      sum += s_need[r];
    }
  }
  sum = block_exclusive_scan<long long>(sum, scratch, all);
  int tokens = 0;
  if (status == 0) {
    for (int r = r0; r < r1; ++r) {
      const int n = s_need[r];
      s_need[r] = static_cast<int>(sum);
      sum += n;
    }
    tokens = p.cu[p.R];
    if (tid == 0) s_cu[p.R] = tokens;
  }
  __syncthreads();
  const int top = *p.free_count_out + static_cast<int>(all) - 1;
  for (int q = blockIdx.x * kSlotThreads + tid; q < (p.tokens + 3) >> 2;
       q += gridDim.x * kSlotThreads)
    plan_slots(p, q, tokens, s_cu, s_need, top, [&](int r) { return s_len[r]; });
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
// head and one of K and V (small pages: both): at most P rows of d values, read once into
// registers (the maximum needs all of them before the first code), coded and
// written once.  Items are dealt out with the heads fastest, so that CTAs of
// neighbouring items read whole token rows together.  128 threads keep P d / 8
// / 128 16-byte loads each in flight and several CTAs share an SM; where the
// next item lies is looked up while this one's loads are on their way.
// Bound by HBM: 2 bytes in and 1 byte out for each value (29440 tokens x 24 heads
// x 128, K and V: 543 MB in 93 us, 5.8 TB/s); the arithmetic stays packed, two
// bf16 an instruction, or the ALUs bind (154 us before).
template <int D, int P>
struct StoreCfg {
  static constexpr int kRowChunks = D / 8;  // 16-byte chunks of a token row
  static constexpr int kRowsPerPass = kStoreThreads / kRowChunks;
  static constexpr int kPasses = P / kRowsPerPass;
  // tensors of an item: with few loads in one, both, so that enough are in flight
  // (frames of 1560 tokens, pages of 16: 18.4 -> 16.4 us)
  static constexpr int kTensors = kPasses <= 4 ? 2 : 1;
  // CTAs of an SM: their loads together cover HBM's latency
  static constexpr int kPerSm = kPasses >= 16 ? 4 : (kPasses >= 8 ? 6 : (kPasses >= 4 ? 8 : 12));
};

template <int D, int P>
__global__ void __launch_bounds__(kStoreThreads, (StoreCfg<D, P>::kPerSm))
    gla_cache_store_kernel(const StoreParams p) {
  using C = StoreCfg<D, P>;
  constexpr int kPasses = C::kPasses, kRowsPerPass = C::kRowsPerPass;
  extern __shared__ int s_items[];  // [R + 1] prefix sums of the pages each sequence writes
  int* s_c0 = s_items + p.R + 1;    // [R + 1] first packed row of each sequence
  int* s_old = s_c0 + p.R + 1;      // [R] tokens it held before
  __shared__ long long scratch[33];
  constexpr int kTensors = C::kTensors;
  __shared__ uint32_t s_max[2][kTensors][kStoreThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int col = tid % C::kRowChunks, row0 = tid / C::kRowChunks;
  {
    const int per = (p.R + kStoreThreads - 1) / kStoreThreads;
    const int r0 = min(p.R, tid * per), r1 = min(p.R, r0 + per);
    long long sum = 0, all;
    for (int r = r0; r < r1; ++r) {
      const int c0 = min(max(p.cu[r], 0), p.tokens);
      const int n = max(min(p.cu[r + 1], p.tokens) - c0, 0);
      const int old = max(p.lens[r] - n, 0);
      s_c0[r] = c0;
      s_old[r] = old;
      s_items[r] = n > 0 ? static_cast<int>((static_cast<int64_t>(old) + n + P - 1) / P - old / P)
                         : 0;
      sum += s_items[r];
    }
    if (r1 == p.R && r0 < p.R) s_c0[p.R] = min(max(p.cu[p.R], 0), p.tokens);
    sum = block_exclusive_scan<long long>(sum, scratch, all);
    for (int r = r0; r < r1; ++r) {
      const int n = s_items[r];
      s_items[r] = static_cast<int>(sum);
      sum += n;
    }
    // more runs than tokens: the rows descend or overlap, and there is no work
    if (tid == 0) s_items[p.R] = all > p.tokens ? 0 : static_cast<int>(all);
    __syncthreads();
  }
  // an item: its first token, its rows, the head and tensor, and the slot of
  // its first token (the load is left in flight)
  struct Item {
    int t0, m, h, slot;
    bool is_v;
  };
  const unsigned heads2 = (kTensors == 2 ? 1u : 2u) * p.H;  // items of a page
  auto locate = [&](int64_t it) {
    Item x;
    const int run = static_cast<int>(static_cast<uint64_t>(it) / heads2);
    const int rest = static_cast<int>(it - static_cast<int64_t>(run) * heads2);
    x.is_v = rest >= p.H;
    x.h = x.is_v ? rest - p.H : rest;
    const int r = prefix_owner<int>(s_items, p.R, run);
    const int old = s_old[r], c0 = s_c0[r], n = max(s_c0[r + 1] - c0, 0);
    const int j = old / P + (run - s_items[r]);  // page of the sequence
    const int64_t p0 = max(static_cast<int64_t>(j) * P, static_cast<int64_t>(old));
    x.t0 = c0 + static_cast<int>(p0 - old);
    x.m = static_cast<int>(
        min(static_cast<int64_t>(j + 1) * P, static_cast<int64_t>(old) + n) - p0);
    x.slot = __ldg(p.slots + x.t0);
    return x;
  };
  const int64_t items = static_cast<int64_t>(s_items[p.R]) * heads2;
  int bad = 0;
  int flip = 0;
  Item next{};
  if (blockIdx.x < items) next = locate(blockIdx.x);
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x, flip ^= 1) {
    const Item cur = next;
    const int h = cur.h;
    const int page = cur.slot >= 0 ? cur.slot / P : p.pages;
    const int at = cur.slot >= 0 ? cur.slot % P : 0;
    // a slot outside the cache: nothing to write
    const int m = page < p.pages ? min(cur.m, P - at) : 0;
    auto is_v = [&](int w) { return kTensors == 2 ? w == 1 : cur.is_v; };

    const int64_t from = (static_cast<int64_t>(cur.t0) * p.H + h) * D + col * 8;
    uint4 x[kTensors][kPasses];
#pragma unroll
    for (int w = 0; w < kTensors; ++w) {
      const __nv_bfloat16* src = (is_v(w) ? p.v : p.k) + from;
#pragma unroll
      for (int i = 0; i < kPasses; ++i) {
        const int row = row0 + i * kRowsPerPass;
        x[w][i] = make_uint4(0, 0, 0, 0);
        if (row < m)
          x[w][i] =
              __ldcs(reinterpret_cast<const uint4*>(src + static_cast<int64_t>(row) * p.H * D));
      }
    }
    if (it + gridDim.x < items) next = locate(it + gridDim.x);
    const int64_t blk = static_cast<int64_t>(m > 0 ? page : 0) * p.H + h;
    float was[kTensors];
#pragma unroll
    for (int w = 0; w < kTensors; ++w)
      was[w] = at > 0 && m > 0 ? (is_v(w) ? p.vs : p.ks)[blk] : 0.f;
#pragma unroll
    for (int w = 0; w < kTensors; ++w) {
      // largest magnitude (packed 16-bit maxima of the bf16 bits)
      uint32_t mx = 0;
#pragma unroll
      for (int i = 0; i < kPasses; ++i) {
        const uint4& y = x[w][i];
        mx = __vmaxu2(mx, __vmaxu2(__vmaxu2(y.x & 0x7FFF7FFFu, y.y & 0x7FFF7FFFu),
                                   __vmaxu2(y.z & 0x7FFF7FFFu, y.w & 0x7FFF7FFFu)));
      }
      mx = max(mx & 0xFFFFu, mx >> 16);
      if (mx >= 0x7F80u) {
        // some are not finite: they do not count for the scale; NaN becomes 0,
        // infinities stay for the saturating conversion
        mx = 0;
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
          uint32_t* y = reinterpret_cast<uint32_t*>(&x[w][i]);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t lo = y[e] & 0x7FFFu, hi = (y[e] >> 16) & 0x7FFFu;
            bad += (lo >= 0x7F80u) + (hi >= 0x7F80u);
            if (lo > 0x7F80u) y[e] &= 0xFFFF0000u;
            if (hi > 0x7F80u) y[e] &= 0x0000FFFFu;
            mx = max(mx, max(lo < 0x7F80u ? lo : 0u, hi < 0x7F80u ? hi : 0u));
          }
        }
      }
      mx = __reduce_max_sync(0xffffffffu, mx);
      if (lane == 0) s_max[flip][w][warp] = mx;
    }
    __syncthreads();  // the other half of s_max is free again after this barrier
    if (m <= 0) continue;  // uniform over the block
    float scale[kTensors];
#pragma unroll
    for (int w = 0; w < kTensors; ++w) {
      const uint32_t* sm = s_max[flip][w];
      const uint32_t mx = max(max(sm[0], sm[1]), max(sm[2], sm[3]));
      scale[w] = exp2_int(scale_exponent(mx));
      if (at > 0) scale[w] = fmaxf(scale[w], was[w]);
      uint8_t* dst = (is_v(w) ? p.v8 : p.k8) + blk * (P * D);
      // both powers of two: the products below are exact in bf16
      const __nv_bfloat162 inv = __float2bfloat162_rn(1.0f / scale[w]);
#pragma unroll
      for (int i = 0; i < kPasses; ++i) {
        const int row = row0 + i * kRowsPerPass;
        const uint32_t y[4] = {x[w][i].x, x[w][i].y, x[w][i].z, x[w][i].w};
        uint32_t c[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const __nv_bfloat162 z = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&y[e]), inv);
          const uint32_t v = *reinterpret_cast<const uint32_t*>(&z);
          c[e] = pack_e4m3x2(bf16lo_to_f32(v), bf16hi_to_f32(v));
        }
        if (row < m)
          *reinterpret_cast<uint2*>(dst + (at + row) * D + col * 8) =
              make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
      }
      if (at > 0 && scale[w] != was[w]) {  // the scale grew: earlier tokens are coded again
        const float ratio = was[w] / scale[w];
        for (int i = tid; i < at * (D / 4); i += kStoreThreads) {
          uint32_t* y = reinterpret_cast<uint32_t*>(dst) + i;
          const uint32_t q = *y;
          const uint32_t f0 = e4m3x2_to_f16x2(q & 0xFFFFu), f1 = e4m3x2_to_f16x2(q >> 16);
          const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&f0));
          const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&f1));
          *y = pack_e4m3x2(a.x * ratio, a.y * ratio) |
               (pack_e4m3x2(b.x * ratio, b.y * ratio) << 16);
        }
      }
    }
    // every thread has read the old scale before one replaces it
    if (at > 0) __syncthreads();
    if (tid == 0) {
#pragma unroll
      for (int w = 0; w < kTensors; ++w) (is_v(w) ? p.vs : p.ks)[blk] = scale[w];
    }
  }
  if (p.nonfinite != nullptr) {
    bad = __reduce_add_sync(0xffffffffu, bad);
    if (lane == 0 && bad) atomicAdd(p.nonfinite, bad);
  }
}

}  // namespace gla
