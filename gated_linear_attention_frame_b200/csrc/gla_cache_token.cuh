// gla_cache_token.cuh -- attention of a few queries a sequence (single tokens
// and short runs) over the paged 8-bit cache.
//
// A query at position p of its sequence sees the keys s < min(len, (p / F + 1)
// F) with s >= (p / F - W + 1) F or s < n_sink (W = 0: no lower bound), F the
// frame in tokens: F = 1 is the causal form, F = tokens of a frame the anchor
// layer's.  out = sigmoid(z) sum_s softmax_s(q . k_s scale ks) (v_s vs), ks and
// vs the scales of the key's page.  A row that sees no key gives 0.
//
// With few query rows a call is bound by reading the codes once from HBM: 2 d
// bytes a key and head.  One work unit = 8 or 16 query rows (tokens x the heads
// that share a key/value head, padded; 8 where all rows of a sequence fit) of one
// sequence and key/value head; its
// visible keys are cut into blocks of 32.  All blocks of all units are laid
// end to end and dealt out evenly to the CTAs, so a long sequence is split as
// finely as the GPU is wide whatever the mix of lengths; a unit that ends up
// in several CTAs leaves one partial (O, m, l) in each, joined in the order of
// the keys by gla_cache_combine_kernel.
//
// The four warps of a CTA take every fourth block, each through its own ring
// of cp.async stages (nothing between warps waits until a unit ends).  The
// products run on mma.sync (m16n8k16, fp16 in, fp32 out): 16 rows would leave
// 7/8 of a 128-row tcgen05 tile empty, and the codes reach the B fragments
// straight from the ring, converted in registers (every e4m3 value is an fp16
// value), with no second trip through shared memory.  The order of d inside a
// fragment is free as long as Q uses the same one, so each thread reads 16
// neighbouring bytes of a key; V's fragments pair two keys of one d by a byte
// permutation.
// Queries are scaled by a power of two per row into the top of the fp16 range
// (exact but for elements 2^29 below the row's largest).  The value scale is
// folded into the exponent, P' = 2^(x + log2 vs - m + kBias), and taken out
// of the row sum again block by block.
// Measured (d = 128): 64 sequences x 8 key/value heads x 8 queries, 1.96 GB of
// codes, 367-393 us (5.0-5.3 TB/s); 2 sequences of 200 thousand keys x 24 heads,
// 2.28 GB, 393-425 us (5.4-5.8 TB/s); ranges over several GPUs.  Small calls are
// bound by the start: sums over the lengths, table, codes, one after the other.
#pragma once

#include <cuda_fp16.h>

#include "gla_cache.cuh"
#include "sm100_ptx.cuh"

namespace gla {

// Division of 0 <= n < 2^31 by d >= 1 as a multiplication and a shift (division by
// invariant integers, Granlund and Montgomery 1994: m = 2^32
// (2^s - d) / d + 1, s = ceil(log2 d); exact for every 32-bit n): the kernels
// divide by the frame and the tile in many places, and a division is 25
// instructions.
struct FastDiv {
  uint32_t m, s;
  __host__ static FastDiv make(uint32_t d) {
    FastDiv f{0, 0};
    while ((uint64_t(1) << f.s) < d) ++f.s;
    f.m = static_cast<uint32_t>((((uint64_t(1) << f.s) - d) << 32) / d + 1);
    return f;
  }
  __host__ __device__ __forceinline__ int div(int n) const {
#ifdef __CUDA_ARCH__
    return static_cast<int>((__umulhi(static_cast<uint32_t>(n), m) + static_cast<uint32_t>(n)) >> s);
#else
    return static_cast<int>(((static_cast<uint64_t>(static_cast<uint32_t>(n)) * m >> 32) +
                             static_cast<uint32_t>(n)) >> s);
#endif
  }
};

struct CacheAttnParams {
  const __nv_bfloat16* q;
  const uint8_t *k8, *v8;
  const float *ks, *vs;
  const int *table, *lens, *cu;
  const __nv_bfloat16* z;
  __nv_bfloat16* out;
  int R, tokens, H, Hkv, G;  // G = H / Hkv query heads share a key/value head
  int pages, max_pages, p_shift;  // P = 1 << p_shift
  int F, W, n_sink;
  float sl2;  // scale * log2(e)
  // token kernel: a tile of R = 8 or 16 rows holds `tile_t` tokens (all G heads of
  // each), or, where G > R, one of `tile_c` parts of one token's heads
  int tile_t, tile_c;
  FastDiv by_f, by_tile;  // by F; by tile_t, or tile_c where that is not 1
  // split units: per CTA two partials of a unit's rows (fp32 O, then m, l: TokenCfg's
  // and FrameCfg's kPartFloats)
  // and one descriptor
  float* part;
  int* desc;
};

// Exponent offset of P': the largest P' of a row is about 2^kBias when its
// reference maximum is set and may grow by 2^kLazy before the row is rescaled
// (2^15 < 65504, the largest fp16); smaller ones keep full fp16 precision
// down to 2^-22 of it.
constexpr float kCacheBias = 8.0f, kCacheLazy = 7.0f;

// The keys that the queries t_lo .. t_hi of one sequence see between them, as a
// list of blocks of BK keys: the blocks of the sinks below the window, then
// the blocks of the window.
struct CacheSpan {
  int lo, hi, sink;   // visible keys: [0, sink) and [lo, hi)
  int sb, wb0, nb;    // sink blocks, first window block, blocks (at least 1)
  __device__ __forceinline__ int pos(int k, int bk) const {
    return (k < sb ? k : wb0 + (k - sb)) * bk;
  }
  __device__ __forceinline__ bool sees(int key) const {
    return key < hi && (key >= lo || key < sink);
  }
};

struct CacheSeq {
  int c0, n, len;  // first packed row, new tokens, keys
  int p0;          // position of the first new token
};

__device__ __forceinline__ CacheSeq cache_seq(const CacheAttnParams& p, int r) {
  CacheSeq s;
  s.c0 = min(max(p.cu[r], 0), p.tokens);
  s.n = max(min(p.cu[r + 1], p.tokens) - s.c0, 0);
  const int raw = max(p.lens[r], 0);
  s.len = min(raw, p.max_pages << p.p_shift);
  s.p0 = raw - s.n;
  return s;
}

// Upper and lower end of the keys of a query at position pos (negative: none).
__device__ __forceinline__ int key_hi(const CacheAttnParams& p, const CacheSeq& s, int pos) {
  if (pos < 0) return 0;
  const int rest = pos - p.by_f.div(pos) * p.F;  // within the frame
  const uint32_t e = static_cast<uint32_t>(pos) + static_cast<uint32_t>(p.F - rest);  // < 2^32
  return static_cast<int>(min(e, static_cast<uint32_t>(s.len)));
}
__device__ __forceinline__ int key_lo(const CacheAttnParams& p, int pos) {
  if (p.W == 0 || pos < 0) return 0;
  const int q = p.by_f.div(pos);
  return q < p.W ? 0 : (q - p.W + 1) * p.F;  // at most pos
}

template <int BK>
__device__ __forceinline__ CacheSpan cache_span(const CacheAttnParams& p, const CacheSeq& s,
                                                int t_lo, int t_hi) {
  CacheSpan v;
  v.hi = key_hi(p, s, s.p0 + t_hi);
  v.lo = min(key_lo(p, s.p0 + t_lo), v.hi);
  v.sink = p.W > 0 ? min(p.n_sink, v.lo) : 0;
  v.sb = (v.sink + BK - 1) / BK;
  v.wb0 = max(v.lo / BK, v.sb);
  v.nb = max(1, v.sb + max(0, (v.hi + BK - 1) / BK - v.wb0));
  return v;
}

// Contiguous share of CTA c of `total` blocks dealt out over `ctas` CTAs.
// (total * ctas < 2^63: blocks are counted in pages of 32-bit slots.)
__device__ __forceinline__ int64_t share_lo(int64_t total, int ctas, int c) {
  return static_cast<int64_t>(static_cast<uint64_t>(total) * static_cast<uint32_t>(c) /
                              static_cast<uint32_t>(ctas));
}

// The CTA whose share holds block x.
__device__ __forceinline__ int share_owner(int64_t total, int ctas, int64_t x) {
  return static_cast<int>(((x + 1) * ctas - 1) / total);
}

// A query row is multiplied by 2^row_exponent before it becomes fp16: 14 - E for
// a largest magnitude of bf16 exponent E (0 for zero and non-finite rows).
__device__ __forceinline__ int row_exponent(uint32_t amax_bits) {
  const int e = static_cast<int>(amax_bits >> 7);
  const int up = (e == 0 || e == 255) ? 0 : 14 - (e - 127);  // in [-113, 140]
  return up > 126 ? 126 : up;
}

// i / G for 0 <= i < 256 and 1 <= G <= 128, with m = (65536 + G - 1) / G (checked
// for every i and G).
__device__ __forceinline__ int small_div(int i, int m) { return (i * m) >> 16; }

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ float lg2_approx(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool ok) {
  const int n = ok ? 16 : 0;  // 0: the 16 bytes become zero
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
               : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, bool ok) {
  const int n = ok ? 4 : 0;
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(n)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// D (16 x 8 fp32) += A (16 x 16 fp16) B (16 x 8 fp16).
__device__ __forceinline__ void mma_f16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                              uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// R: query rows of a tile, 16 or 8.  Rows of 16 are the M side of the products,
// rows of 8 the N side (S^T = K Q^T, O^T = V^T P^T): half the products, half
// the exponentials and half the accumulators, so that 12 warps fit on an SM
// instead of 8.
template <int D, int R>
struct TokenCfg {
  static_assert(R == 16 || R == 8, "rows of a tile");
  static constexpr int kThreads = 128;
  static constexpr int kWarps = 4;
  static constexpr int kRows = R;
  static constexpr int BK = 32;           // keys of a block
  static constexpr int kStages = D == 64 ? 4 : (R == 16 ? 3 : 2);
  static constexpr int kTensorBytes = BK * D;            // K or V codes of a block
  static constexpr int kStageBytes = 2 * kTensorBytes + 16;  // + ks, vs of its two key halves
  static constexpr int kRingBytes = kWarps * kStages * kStageBytes;
  static constexpr int kMergeBytes = 2 * 8 * D * 4;  // two warps' rows, eight at a time
  static constexpr int kStatBytes = kWarps * 16 * 8;
  static constexpr int kFixedBytes = kRingBytes + kMergeBytes + kStatBytes;
  static constexpr int kPartFloats = kRows * D + 2 * kRows;
  static constexpr int kCtasPerSm = R == 16 ? 2 : 3;
  static constexpr int kMinBlocks = 8;    // least blocks of a CTA
  static constexpr int kChunks = D / 16;  // 16-byte chunks of a key
};

// The same, A by value.
__device__ __forceinline__ void mma_f16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                              uint32_t a3, uint32_t b0, uint32_t b1) {
  const uint32_t a[4] = {a0, a1, a2, a3};
  mma_f16_16816(d, a, b0, b1);
}

// Transpose of an 8 x 8 matrix of 16-bit values held as a fragment (lane 4 r + c:
// row r, columns 2 c and 2 c + 1).
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

// Four codes of two neighbouring keys (a, b) -> their fp16 pairs (key a in the
// low half), code by code.
__device__ __forceinline__ void pair_keys(uint32_t a, uint32_t b, uint32_t (&y)[4]) {
  const uint32_t lo = __byte_perm(a, b, 0x5140), hi = __byte_perm(a, b, 0x7362);
  y[0] = e4m3x2_to_f16x2(lo & 0xFFFFu);
  y[1] = e4m3x2_to_f16x2(lo >> 16);
  y[2] = e4m3x2_to_f16x2(hi & 0xFFFFu);
  y[3] = e4m3x2_to_f16x2(hi >> 16);
}

template <int D, int R>
__global__ void __launch_bounds__(128, (TokenCfg<D, R>::kCtasPerSm))
    gla_cache_token_kernel(const CacheAttnParams p) {
  using C = TokenCfg<D, R>;
  constexpr int BK = C::BK;
  constexpr int KI = D / 64;   // 16-byte chunks of a key that one thread reads
  constexpr int NT = D / 8;    // n-tiles of the output
  extern __shared__ __align__(16) uint8_t smem[];
  float* s_o = reinterpret_cast<float*>(smem + C::kRingBytes);
  float2* s_ml = reinterpret_cast<float2*>(smem + C::kRingBytes + C::kMergeBytes);
  long long* s_pre = reinterpret_cast<long long*>(smem + C::kFixedBytes);  // [R + 1]
  __shared__ long long scratch[33];
  __shared__ float2 s_row[8];  // (m, l) of the rows on their way out
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t4 = lane & 3;
  const int P = 1 << p.p_shift;

  // query tiles of a sequence, and the keys one of them sees
  const int gm = (65536 + p.G - 1) / p.G;  // see small_div
  auto tiles_of = [&](const CacheSeq& s) {
    return p.tile_c > 1 ? s.n * p.tile_c : p.by_tile.div(s.n + p.tile_t - 1);
  };
  auto first_token = [&](int tile) {
    return p.tile_c > 1 ? p.by_tile.div(tile) : tile * p.tile_t;
  };
  auto span_of = [&](const CacheSeq& s, int tile) {
    const int t = first_token(tile);
    return cache_span<BK>(p, s, t, min(t + p.tile_t, s.n) - 1);
  };
  auto blocks_of = [&](int r) -> long long {
    const CacheSeq s = cache_seq(p, r);
    long long b = 0;
    for (int i = 0, n = tiles_of(s); i < n; ++i) b += span_of(s, i).nb;
    return b * p.Hkv;
  };
  long long total;
  {
    const int per = (p.R + C::kThreads - 1) / C::kThreads;
    const int r0 = min(p.R, tid * per), r1 = min(p.R, r0 + per);
    long long sum = 0;
    for (int r = r0; r < r1; ++r) {
      const long long b = blocks_of(r);
      s_pre[r] = b;
      sum += b;
    }
    long long at = block_exclusive_scan<long long>(sum, scratch, total);
    for (int r = r0; r < r1; ++r) {
      const long long b = s_pre[r];
      s_pre[r] = at;
      at += b;
    }
    if (tid == 0) s_pre[p.R] = total;
    __syncthreads();
  }
  int* desc = p.desc + 8 * blockIdx.x;
  const long long want = (total + C::kMinBlocks - 1) / C::kMinBlocks;
  const int ctas = static_cast<int>(want < gridDim.x ? want : gridDim.x);
  if (tid == 0) desc[0] = 0;  // nothing to join unless a unit goes on past this CTA
  if (static_cast<int>(blockIdx.x) >= ctas) return;
  long long x0 = 0, x1 = 0;
#pragma unroll 1
  for (int c = 0; c < 2; ++c) {  // one copy of the division
    x0 = x1;
    x1 = share_lo(total, ctas, blockIdx.x + c);
  }

  // A unit, and this warp's place in the part [k, k_end) of its blocks that
  // belongs to this CTA.
  struct Cursor {
    CacheSeq s;
    CacheSpan v;
    int r, tile, tiles, h;
    long long x_unit;  // block number of the unit's first block
    int k, k0, k_end;
    bool live;
  };
  auto open = [&](Cursor& c) {  // the unit's part of this CTA
    c.v = span_of(c.s, c.tile);
    c.k0 = c.x_unit < x0 ? static_cast<int>(x0 - c.x_unit) : 0;
    c.k_end = c.x_unit + c.v.nb > x1 ? static_cast<int>(x1 - c.x_unit) : c.v.nb;
    c.k = c.k0 + warp;
  };
  auto next_unit = [&](Cursor& c) {
    c.x_unit += c.v.nb;
    if (c.x_unit >= x1) {
      c.live = false;
      return;
    }
    if (++c.h == p.Hkv) {
      c.h = 0;
      if (++c.tile == c.tiles) {
        c.tile = 0;
        do {
          ++c.r;
          c.s = cache_seq(p, c.r);
          c.tiles = tiles_of(c.s);
        } while (c.tiles == 0);  // ends: blocks are left, so a sequence with rows follows
      }
    }
    open(c);
  };
  Cursor cur;
  {
    cur.r = prefix_owner<long long>(s_pre, p.R, x0);
    cur.s = cache_seq(p, cur.r);
    cur.tiles = tiles_of(cur.s);
    cur.x_unit = s_pre[cur.r];
    cur.tile = 0;
    for (;; ++cur.tile) {  // tiles are few: a sequence of this kernel has few rows
      const int nb = span_of(cur.s, cur.tile).nb;
      const long long all = static_cast<long long>(nb) * p.Hkv;
      if (cur.x_unit + all > x0 || cur.tile + 1 == cur.tiles) {
        cur.h = static_cast<int>((x0 - cur.x_unit) / nb);
        cur.x_unit += static_cast<long long>(cur.h) * nb;
        break;
      }
      cur.x_unit += all;
    }
    cur.live = true;
    open(cur);
  }
  Cursor ld = cur;  // runs ahead: the block loaded next

  const uint32_t ring = smem_u32(smem) + warp * C::kStages * C::kStageBytes;
  const int64_t page_stride = static_cast<int64_t>(p.Hkv) << p.p_shift;  // rows of a page

  constexpr int kRowsPerPass = 32 / C::kChunks;  // 4 (d = 128) or 8
  const int ch = lane % C::kChunks, rr = lane / C::kChunks;
  // where this lane's chunk goes in a stage: swizzled so that the fragment
  // reads below hit all banks (V: every other pass flips one more bit at d = 128)
  const uint32_t to_k = rr * D + (D == 128 ? (ch ^ ((rr & 1) << 2)) : ch) * 16;
  const uint32_t to_v = rr * D + (D == 128 ? (ch ^ ((rr >> 1) << 1)) : (ch ^ ((rr >> 1) & 3))) * 16;

  // Start the copies of this warp's next block into stage `st`.
  auto issue = [&](int st) {
    while (ld.live && ld.k >= ld.k_end) next_unit(ld);
    if (ld.live) {
      const int base = ld.v.pos(ld.k, BK);
      const int* row = p.table + static_cast<int64_t>(ld.r) * p.max_pages;
      const uint32_t dst = ring + st * C::kStageBytes;
      // a block lies in one page, or (P = 16) each half of it in one
      const int j0 = base >> p.p_shift, j1 = (base + 16) >> p.p_shift;
      int page[2];
      page[0] = j0 < p.max_pages ? row[j0] : -1;
      page[1] = j1 == j0 ? page[0] : (j1 < p.max_pages ? row[j1] : -1);
      const uint8_t *ks[2], *vs[2];
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        if (page[hf] >= p.pages) page[hf] = -1;
        const int64_t off = (max(page[hf], 0) * page_stride +
                             (static_cast<int64_t>(ld.h) << p.p_shift) +
                             ((base + hf * 16 + rr) & (P - 1))) * D + ch * 16;
        ks[hf] = p.k8 + off;
        vs[hf] = p.v8 + off;
      }
      const bool all = base >= ld.v.lo && base + BK <= ld.v.hi && page[0] >= 0 && page[1] >= 0;
#pragma unroll
      for (int i = 0; i < BK / kRowsPerPass; ++i) {
        constexpr int kHalf = 16 / kRowsPerPass;  // passes of one half
        const int hf = i / kHalf;
        const bool ok =
            all || (page[hf] >= 0 && ld.v.sees(base + i * kRowsPerPass + rr));
        const int step = (i % kHalf) * kRowsPerPass * D;
        cp_async16(dst + to_k + i * kRowsPerPass * D, ks[hf] + step, ok);
        cp_async16(dst + C::kTensorBytes + (to_v ^ (D == 128 ? (i & 1) << 6 : 0)) +
                       i * kRowsPerPass * D,
                   vs[hf] + step, ok);
      }
      if (lane < 4) {
        const int hf = lane & 1;
        const int a = base + hf * 16;  // a half that shows no key has scale 0
        const bool any = page[hf] >= 0 && a < ld.v.hi && (a + 16 > ld.v.lo || a < ld.v.sink);
        const float* sc = (lane < 2 ? p.ks : p.vs) +
                          (any ? static_cast<int64_t>(page[hf]) * p.Hkv + ld.h : 0);
        cp_async4(dst + 2 * C::kTensorBytes + lane * 4, sc, any);
      }
      ld.k += C::kWarps;
    }
    cp_async_commit();
  };
  int ahead = 0;               // blocks in the ring
  int st_in = 0, st = 0;       // stages filled and used next

  for (; cur.live; next_unit(cur)) {
    // rows of the tile: token t0 + row / G, head g0 + row % G of the group
    const int t0 = first_token(cur.tile);
    const int g0 = p.tile_c > 1 ? (cur.tile - t0 * p.tile_c) * R : 0;
    const int rows = p.tile_c > 1 ? min(R, p.G - g0) : min(p.tile_t, cur.s.n - t0) * p.G;
    const int64_t row0 =
        (static_cast<int64_t>(cur.s.c0) + t0) * p.H + cur.h * p.G + g0;  // of q and out
    auto row_token = [&](int rho) { return p.tile_c > 1 ? 0 : small_div(rho, gm); };
    // ---- query fragments: rows g (and g + 8) of the tile
    constexpr int E = R / 8;     // rows of a lane's fragment
    uint32_t qa[D / 16][2 * E];
    float rq[E];                 // undoes the row scale, times scale log2(e)
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int rho = g + 8 * e;
      const bool have = rho < rows;
      const int rt = have ? row_token(rho) : 0;
      const __nv_bfloat16* qp =
          p.q + (row0 + static_cast<int64_t>(rt) * p.H + (have ? rho - rt * p.G : 0)) * D;
      uint4 w[KI][2];
      uint32_t mx = 0;
#pragma unroll
      for (int i = 0; i < KI; ++i)
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          w[i][f] = make_uint4(0, 0, 0, 0);
          if (have)
            w[i][f] = *reinterpret_cast<const uint4*>(qp + i * 64 + t4 * 16 + f * 8);
          mx = __vmaxu2(mx, __vmaxu2(__vmaxu2(w[i][f].x & 0x7FFF7FFFu, w[i][f].y & 0x7FFF7FFFu),
                                     __vmaxu2(w[i][f].z & 0x7FFF7FFFu, w[i][f].w & 0x7FFF7FFFu)));
        }
      mx = max(mx & 0xFFFFu, mx >> 16);
      mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const int up = row_exponent(mx);
      const float f = exp2_int(up);
      rq[e] = exp2_int(-up) * p.sl2;
#pragma unroll
      for (int i = 0; i < KI; ++i)
#pragma unroll
        for (int jj = 0; jj < 4; ++jj) {
          const uint4& x = w[i][jj >> 1];
          const uint32_t w0 = (jj & 1) ? x.z : x.x, w1 = (jj & 1) ? x.w : x.y;
          qa[i * 4 + jj][e] = pack_f16x2(bf16lo_to_f32(w0) * f, bf16hi_to_f32(w0) * f);
          qa[i * 4 + jj][E + e] = pack_f16x2(bf16lo_to_f32(w1) * f, bf16hi_to_f32(w1) * f);
        }
    }
    // the rows of this lane's scores: g and g + 8, or (8 rows) 2 t4 and 2 t4 + 1
    float rs[2];
    int hi[2], lo[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int rho = R == 16 ? g + 8 * e : 2 * t4 + e;
      rs[e] = R == 16 ? rq[e % E] : __shfl_sync(0xffffffffu, rq[0], rho * 4);
      const bool have = rho < rows;
      const int pos = cur.s.p0 + t0 + (have ? row_token(rho) : 0);
      hi[e] = have ? key_hi(p, cur.s, pos) : 0;
      lo[e] = key_lo(p, pos);
    }
    // accumulators: 16 rows: n-tile n, [row g: x = 0, 1; row g + 8: x = 2, 3];
    // 8 rows: m-tile n, [d 2 n of the lane's: rows 2 t4, 2 t4 + 1; d 2 n + 1: the same]
    constexpr int NO = R == 16 ? NT : D / 16;
    float o[NO][4];
#pragma unroll
    for (int n = 0; n < NO; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    // every row sees every key of a block inside [all_lo, all_hi)
    const int all_hi = key_hi(p, cur.s, cur.s.p0 + t0);
    const int all_lo = key_lo(p, cur.s.p0 + t0 + row_token(rows - 1));

    for (;; cur.k += C::kWarps) {
#pragma unroll 1
      for (; ahead < C::kStages; ++ahead) {  // all of them at first, then one a block
        issue(st_in);
        st_in = st_in + 1 == C::kStages ? 0 : st_in + 1;
      }
      if (cur.k >= cur.k_end) break;
      cp_async_wait<C::kStages - 1>();
      __syncwarp();
      const uint32_t kb = ring + st * C::kStageBytes, vb = kb + C::kTensorBytes;
      const uint4 sc = ld_shared_v4(vb + C::kTensorBytes);
      const float ksc[2] = {__uint_as_float(sc.x), __uint_as_float(sc.y)};
      const float vsc[2] = {__uint_as_float(sc.z), __uint_as_float(sc.w)};
      // ---- S: 16 scores of 16 rows (n-tile j: keys 8 j ..), or 8 of 8 rows (m-tile
      // j: keys 16 j ..) for each lane
      constexpr int NS = R == 16 ? 4 : 2;
      float s[NS][4];
#pragma unroll
      for (int j = 0; j < NS; ++j) {
        s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.f;
#pragma unroll
        for (int i = 0; i < KI; ++i) {
          const int c = i * 4 + t4;
          auto chunk = [&](int kr) {
            return ld_shared_v4(kb + kr * D + (D == 128 ? (c ^ ((kr & 1) << 2)) : c) * 16);
          };
          if constexpr (R == 16) {
            const uint4 w = chunk(j * 8 + g);
            const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int jj = 0; jj < 4; ++jj)
              mma_f16_16816(s[j], qa[i * 4 + jj], e4m3x2_to_f16x2(ww[jj] & 0xFFFFu),
                            e4m3x2_to_f16x2(ww[jj] >> 16));
          } else {
            const uint4 w = chunk(j * 16 + g), v = chunk(j * 16 + 8 + g);
            const uint32_t ww[4] = {w.x, w.y, w.z, w.w}, vv[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int jj = 0; jj < 4; ++jj)
              mma_f16_16816(s[j], e4m3x2_to_f16x2(ww[jj] & 0xFFFFu),
                            e4m3x2_to_f16x2(vv[jj] & 0xFFFFu), e4m3x2_to_f16x2(ww[jj] >> 16),
                            e4m3x2_to_f16x2(vv[jj] >> 16), qa[i * 4 + jj][0], qa[i * 4 + jj][1]);
          }
        }
      }
      const int base = cur.v.pos(cur.k, BK);
      float lv[2], iv[2];
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        lv[hf] = lg2_approx(vsc[hf]);  // scale 0 (nothing visible): -inf
        iv[hf] = vsc[hf] > 0.f ? ex2_approx(-lv[hf]) : 0.f;
      }
      const bool whole = base >= all_lo && base + BK <= all_hi;  // uniform
      // score (j, x) belongs to row e = row_of(x), in key half half_of(j)
      auto row_of = [](int x) { return R == 16 ? x >> 1 : x & 1; };
      auto half_of = [](int j) { return R == 16 ? j >> 1 : j; };
#pragma unroll
      for (int j = 0; j < NS; ++j)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int e = row_of(x);
          s[j][x] = fmaf(s[j][x], rs[e] * ksc[half_of(j)], lv[half_of(j)]);
          if (!whole) {
            const int key =
                base + (R == 16 ? j * 8 + t4 * 2 + (x & 1) : j * 16 + g + (x >> 1) * 8);
            if (!(key < hi[e] && (key >= lo[e] || key < p.n_sink))) s[j][x] = -INFINITY;
          }
        }
      bool grow = false;
      float mt[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float a = -INFINITY;
#pragma unroll
        for (int j = 0; j < NS; ++j)
          a = R == 16 ? fmax3(a, s[j][2 * e], s[j][2 * e + 1]) : fmax3(a, s[j][e], s[j][2 + e]);
        if (R == 16) {  // over the lanes of a row
          a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
          a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 2));
        } else {
          a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 4));
          a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 8));
          a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 16));
        }
        mt[e] = a;
        grow |= a > m[e] + kCacheLazy;  // also the first visible key: m = -inf
      }
      if (__any_sync(0xffffffffu, grow)) {
        float f[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float mn = fmaxf(m[e], mt[e]);
          f[e] = m[e] == -INFINITY ? 0.f : ex2_approx(m[e] - mn);
          m[e] = mn;
          l[e] *= f[e];
        }
#pragma unroll
        for (int n = 0; n < NO; ++n)
#pragma unroll
          for (int x = 0; x < 4; ++x) o[n][x] *= f[row_of(x)];
      }
      // ---- P' and the row sums (the value scale leaves the sums again)
      const float sh[2] = {m[0] == -INFINITY ? 0.f : kCacheBias - m[0],
                           m[1] == -INFINITY ? 0.f : kCacheBias - m[1]};
      uint32_t pa[2][4];  // 16 rows: A fragment of each key half; 8 rows: B fragment in [0], [1]
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        if constexpr (R == 16) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float x[4];
#pragma unroll
            for (int y = 0; y < 4; ++y)
              x[y] = ex2_approx(s[hf * 2 + (y >> 1)][2 * e + (y & 1)] + sh[e]);
            l[e] = fmaf((x[0] + x[1]) + (x[2] + x[3]), iv[hf], l[e]);
            pa[hf][e] = pack_f16x2(x[0], x[1]);
            pa[hf][2 + e] = pack_f16x2(x[2], x[3]);
          }
        } else {
          float x[4];
#pragma unroll
          for (int y = 0; y < 4; ++y) x[y] = ex2_approx(s[hf][y] + sh[y & 1]);
          l[0] = fmaf(x[0] + x[2], iv[hf], l[0]);
          l[1] = fmaf(x[1] + x[3], iv[hf], l[1]);
          pa[hf][0] = movmatrix_trans(pack_f16x2(x[0], x[1]));  // keys 0 .. 7 of the half
          pa[hf][1] = movmatrix_trans(pack_f16x2(x[2], x[3]));  // keys 8 .. 15
        }
      }
      // ---- O += P' V.  Lane (g, t4) reads the bytes of d = D / 8 g .. of the keys
      // 2 t4, 2 t4 + 1 and those plus 8
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        constexpr int NW = D / 32;  // words of a lane's piece of a key
        uint32_t w[4][NW];
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const int kr = hf * 16 + t4 * 2 + (y & 1) + (y >> 1) * 8;
          if constexpr (D == 128) {
            const uint4 v = ld_shared_v4(vb + kr * D + ((g ^ (((kr >> 1) & 3) << 1))) * 16);
            w[y][0] = v.x;
            w[y][1] = v.y;
            w[y][2] = v.z;
            w[y][3] = v.w;
          } else {
            const uint32_t ad = vb + kr * D + (((g >> 1) ^ ((kr >> 1) & 3)) * 16) + (g & 1) * 8;
            asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];"
                         : "=r"(w[y][0]), "=r"(w[y][1])
                         : "r"(ad)
                         : "memory");
          }
        }
#pragma unroll
        for (int q = 0; q < NW; ++q) {
          uint32_t a[4], b[4];  // codes 4 q .. 4 q + 3 of the piece: keys 2 t4 .., and plus 8
          pair_keys(w[0][q], w[1][q], a);
          pair_keys(w[2][q], w[3][q], b);
          if constexpr (R == 16) {
#pragma unroll
            for (int y = 0; y < 4; ++y) mma_f16_16816(o[q * 4 + y], pa[hf], a[y], b[y]);
          } else {
#pragma unroll
            for (int y = 0; y < 2; ++y)
              mma_f16_16816(o[q * 2 + y], a[2 * y], a[2 * y + 1], b[2 * y], b[2 * y + 1],
                            pa[hf][0], pa[hf][1]);
          }
        }
      }
      __syncwarp();  // the stage is read by every lane before it is loaded again
      st = st + 1 == C::kStages ? 0 : st + 1;
      --ahead;
    }

    // ---- join the four warps
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if (R == 16) {
        l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
        l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
        if (t4 == 0) s_ml[warp * 16 + g + 8 * e] = make_float2(m[e], l[e]);
      } else {
        l[e] += __shfl_xor_sync(0xffffffffu, l[e], 4);
        l[e] += __shfl_xor_sync(0xffffffffu, l[e], 8);
        l[e] += __shfl_xor_sync(0xffffffffu, l[e], 16);
        if (g == 0) s_ml[warp * 16 + 2 * t4 + e] = make_float2(m[e], l[e]);
      }
    }
    __syncthreads();
    float mm[2], ll[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int rho = R == 16 ? g + 8 * e : 2 * t4 + e;
      float2 a[C::kWarps];
      mm[e] = -INFINITY;
#pragma unroll
      for (int w = 0; w < C::kWarps; ++w) {
        a[w] = s_ml[w * 16 + rho];
        mm[e] = fmaxf(mm[e], a[w].x);
      }
      ll[e] = 0.f;
#pragma unroll
      for (int w = 0; w < C::kWarps; ++w)
        // (m = -inf: l is 0, or NaN for a row that is not finite: it goes on)
        ll[e] += a[w].x == -INFINITY ? a[w].y : a[w].y * ex2_approx(a[w].x - mm[e]);
      const float f = m[e] == -INFINITY ? 0.f : ex2_approx(m[e] - mm[e]);
#pragma unroll
      for (int n = 0; n < NO; ++n)
#pragma unroll
        for (int x = 0; x < 4; ++x)
          if ((R == 16 ? x >> 1 : x & 1) == e) o[n][x] *= f;
    }
    // eight rows at a time: 2 NT floats a lane
    auto piece = [&](int e, int i) -> float& {
      if constexpr (R == 16)
        return o[i >> 1][2 * e + (i & 1)];
      else
        return o[i >> 2][i & 3];
    };
    const bool low = rows > 8;  // rows g + 8 hold something (uniform)
    const bool starts = cur.k0 == 0, ends = cur.k_end == cur.v.nb, whole = starts && ends;
    // the CTA's first part of a unit begun before it goes to its partial 0, a
    // unit that goes on after it to partial 1
    float* part = p.part + (2ll * blockIdx.x + (starts ? 1 : 0)) * C::kPartFloats;
    auto slot = [&](int buf, int i) -> float& { return s_o[(buf * 2 * NT + i) * 32 + lane]; };
#pragma unroll
    for (int e = 0; e < R / 8; ++e) {  // rows g, then rows g + 8
      if (e == 1) {
        if (!low) break;
        __syncthreads();  // the buffers are read
      }
#pragma unroll
      for (int half = 2; half >= 1; half >>= 1) {  // warps half .. 2 half - 1 give, the others take
        if (warp >= half && warp < 2 * half) {
          const int buf = half == 2 ? warp - 2 : 1;
#pragma unroll
          for (int i = 0; i < 2 * NT; ++i) slot(buf, i) = piece(e, i);
        }
        __syncthreads();
        if (warp < half) {
          const int buf = half == 2 ? warp : 1;
#pragma unroll
          for (int i = 0; i < 2 * NT; ++i) piece(e, i) += slot(buf, i);
        }
      }
      // warp 0 holds the sums: through shared memory once more, so that all
      // threads write whole row pieces of 8 columns
      if (warp == 0) {
#pragma unroll
        for (int i = 0; i < 2 * NT; ++i) slot(0, i) = piece(e, i);
        if (R == 16) {
          if (t4 == 0) s_row[g] = make_float2(mm[e], ll[e]);
        } else if (g == 0) {
          s_row[2 * t4] = make_float2(mm[0], ll[0]);
          s_row[2 * t4 + 1] = make_float2(mm[1], ll[1]);
        }
      }
      __syncthreads();
      constexpr int kPieces = D / 8;  // of a row
#pragma unroll 1
      for (int i = tid; i < 8 * kPieces; i += C::kThreads) {
        const int r8 = i / kPieces, c = i % kPieces, rho = r8 + 8 * e;
        if (rho >= rows) continue;
        // column 8 c + y: with 16 rows lane (r8, col / (D / 4)) holds it in n-tile
        // col % NT, x = (col / NT) & 1; with 8 rows lane (col / (D / 8), r8 / 2) in
        // m-tile (col % (D / 8)) / 2, x = 2 (col & 1) + (r8 & 1)
        float v[8];
#pragma unroll
        for (int y = 0; y < 8; ++y) {
          const int col = c * 8 + y;
          if constexpr (R == 16)
            v[y] = s_o[((col % NT) * 2 + ((col / NT) & 1)) * 32 + r8 * 4 + col / (D / 4)];
          else
            v[y] = s_o[(((col % (D / 8)) >> 1) * 4 + (col & 1) * 2 + (r8 & 1)) * 32 +
                       (col / (D / 8)) * 4 + (r8 >> 1)];
        }
        const float2 ml = s_row[r8];
        if (whole) {
          const int rt = row_token(rho);
          const int64_t at =
              (row0 + static_cast<int64_t>(rt) * p.H + (rho - rt * p.G)) * D + c * 8;
          const float rl = ml.x == -INFINITY ? 0.f : 1.0f / ml.y;
          uint4 zw = make_uint4(0, 0, 0, 0);
          if (p.z != nullptr) zw = *reinterpret_cast<const uint4*>(p.z + at);
          const uint32_t zz[4] = {zw.x, zw.y, zw.z, zw.w};
          uint32_t w[4];
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            float a = v[2 * y] * rl, b = v[2 * y + 1] * rl;
            if (p.z != nullptr) {
              a = __fdividef(a, 1.0f + __expf(-bf16lo_to_f32(zz[y])));
              b = __fdividef(b, 1.0f + __expf(-bf16hi_to_f32(zz[y])));
            }
            w[y] = pack_bf16x2(a, b);
          }
          *reinterpret_cast<uint4*>(p.out + at) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
          float4* dst = reinterpret_cast<float4*>(part + rho * D + c * 8);
          dst[0] = make_float4(v[0], v[1], v[2], v[3]);
          dst[1] = make_float4(v[4], v[5], v[6], v[7]);
          if (c == 0) *reinterpret_cast<float2*>(part + R * D + 2 * rho) = ml;
        }
      }
    }
    if (tid == 0 && starts && !ends) {
      const int parts = share_owner(total, ctas, cur.x_unit + cur.v.nb - 1) - blockIdx.x + 1;
      desc[1] = cur.s.c0 + t0;
      desc[2] = g0;
      desc[3] = cur.h;
      desc[4] = rows;
      desc[0] = parts;
    }
  }
  cp_async_wait<0>();
}

// Joins the partials of a unit that several CTAs share: CTA x of the grid takes
// the unit (if any) that begins in CTA x of the attention kernel and goes on
// after it; its parts are partial 1 of that CTA and partial 0 of the next
// ones.  blockIdx.y: a query row.  Warp w takes parts w, w + 4, ..: 32 (m, l) at
// a time, one a lane, then their O rows, eight loads in flight; the four warps
// are joined in a fixed order.
template <int D, int R>
__global__ void __launch_bounds__(128) gla_cache_combine_kernel(const CacheAttnParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int kFloats = TokenCfg<D, R>::kPartFloats;
  constexpr int V = D / 32;  // columns of a lane
  __shared__ float s_acc[4][D];
  __shared__ float2 s_ml[4];
  // (the partials are read past L1: this grid may have started before they were
  // written)
  const int4 d0 = __ldcg(reinterpret_cast<const int4*>(p.desc + 8 * blockIdx.x));
  const int rows = __ldcg(p.desc + 8 * blockIdx.x + 4);
  const int parts = d0.x, rho = blockIdx.y;
  if (parts == 0 || rho >= rows) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto part_of = [&](int i) {
    return p.part + (i == 0 ? 2ll * blockIdx.x + 1 : 2ll * (blockIdx.x + i)) * kFloats;
  };
  float m = -INFINITY, l = 0.f, acc[V] = {};
  for (int i0 = warp; i0 < parts; i0 += 128) {
    const int mine = i0 + 4 * lane;  // this lane's part
    float2 ml = make_float2(-INFINITY, 0.f);
    if (mine < parts) ml = __ldcg(reinterpret_cast<const float2*>(part_of(mine) + R * D + 2 * rho));
    float mn = fmaxf(m, ml.x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
    // nothing visible in these parts, unless the row is NaN (l is, and w below)
    if (mn == -INFINITY && !__any_sync(0xffffffffu, ml.y != ml.y)) continue;
    const float f = m == -INFINITY ? 0.f : exp2f(m - mn);
    const float w = ml.x == -INFINITY ? ml.y : exp2f(ml.x - mn);
    float ls = ml.y * w;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ls += __shfl_xor_sync(0xffffffffu, ls, o);
    m = mn;
    l = l * f + ls;
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] *= f;
    const int n = min(32, (parts - i0 + 3) / 4);
#pragma unroll 8
    for (int i = 0; i < n; ++i) {
      const float wi = __shfl_sync(0xffffffffu, w, i);
      const float* x = part_of(i0 + 4 * i) + rho * D + lane * V;
      if constexpr (V == 4) {
        const float4 o = __ldcg(reinterpret_cast<const float4*>(x));
        acc[0] = fmaf(o.x, wi, acc[0]);
        acc[1] = fmaf(o.y, wi, acc[1]);
        acc[2] = fmaf(o.z, wi, acc[2]);
        acc[3] = fmaf(o.w, wi, acc[3]);
      } else {
        const float2 o = __ldcg(reinterpret_cast<const float2*>(x));
        acc[0] = fmaf(o.x, wi, acc[0]);
        acc[1] = fmaf(o.y, wi, acc[1]);
      }
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) s_acc[warp][lane * V + v] = acc[v];
  if (lane == 0) s_ml[warp] = make_float2(m, l);
  __syncthreads();
  const int col = threadIdx.x * 2;
  if (col >= D) return;
  float mm = -INFINITY;
#pragma unroll
  for (int w = 0; w < 4; ++w) mm = fmaxf(mm, s_ml[w].x);
  float x0 = 0.f, x1 = 0.f, ls = 0.f;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const float f = s_ml[w].x == -INFINITY ? s_ml[w].y : exp2f(s_ml[w].x - mm);
    ls += s_ml[w].y * f;
    x0 += s_acc[w][col] * f;
    x1 += s_acc[w][col + 1] * f;
  }
  const float rl = mm == -INFINITY ? 0.f : 1.0f / ls;
  x0 *= rl;
  x1 *= rl;
  const int g = d0.z + rho, rt = g / p.G;  // d0.z = 0 unless a token has several tiles
  const int64_t off =
      ((static_cast<int64_t>(d0.y) + rt) * p.H + d0.w * p.G + (g - rt * p.G)) * D + col;
  if (p.z != nullptr) {
    const uint32_t z = *reinterpret_cast<const uint32_t*>(p.z + off);
    x0 *= 1.0f / (1.0f + __expf(-bf16lo_to_f32(z)));
    x1 *= 1.0f / (1.0f + __expf(-bf16hi_to_f32(z)));
  }
  *reinterpret_cast<uint32_t*>(p.out + off) = pack_bf16x2(x0, x1);
}

}  // namespace gla
