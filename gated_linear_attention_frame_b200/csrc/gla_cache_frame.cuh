// gla_cache_frame.cuh -- attention of many queries a sequence (frames, prompts)
// over the paged 8-bit cache, on tcgen05.  The definition is that of
// gla_cache_token.cuh.
//
// With many query rows a call is bound by the tensor cores: 4 d flops for each
// query, visible key and head.  One work unit = 256 query rows (tokens x the
// heads that share a key/value head) of one sequence and key/value head, held
// as two halves of 128 rows; its visible keys are cut into tiles of 128.  The
// tiles of all units are laid end to end and dealt out evenly to one CTA per
// SM (gla_cache_schedule_kernel finds where each CTA begins); a unit that ends
// up in several CTAs leaves a partial (O, m, l) in each, joined by
// gla_cache_combine_kernel.
//
// Both halves of a unit share each key/value tile, because every tile has to
// be converted first: tcgen05 wants both operands of a product in one type,
// and q in 8 bits would cost its precision.  Four converter warps read the
// codes from global memory straight into registers (one tile ahead), turn
// them into fp16 (exact) and write them in the swizzled operand layout; the
// mask's outer ends are handled there too (keys that no row of the unit sees
// become zeros), so stray pages and NaN codes never reach a product.
//   S_h = Q_h K^T   A = Q half [128 x d] K-major, B = K tile [128 keys] K-major
//   O_h += P_h V    A = P_h in TMEM (fp16, over the columns of S_h),
//                   B = V tile [128 keys x d] MN-major
// TMEM: S_0, S_1 (128 columns each), O_0, O_1 (d columns each).  One issuing
// warp per half: P V of tile j, then S of tile j + 1 into the same columns
// (the tensor core runs one thread's products in order), while the other
// half's softmax runs; so the two halves alternate between the tensor core and
// the exponentials.
// Softmax: one thread per row.  x = S f_g + lv_g for the keys of 16-key group
// g (f_g: key scale x row scale x softmax scale x log2 e, lv_g: log2 of the
// value scale), P' = 2^(x - m + kCacheBias); the row's reference maximum m
// moves only when a tile exceeds it by 2^kCacheLazy, and O is rescaled then.
// One pair of exponentials in four runs on the FMA pipe (exp2_poly3_x2).
// Warp roles: 0-3 / 4-7 softmax and epilogue of half 0 / 1, 8-11 converters,
// 12 / 13 MMA issuers of half 0 / 1 (14, 15 idle: they complete a register
// group).
#pragma once

#include "gla_cache_token.cuh"
#include "gla_increment.cuh"  // warp_wait
#include "gla_softmax_anchor.cuh"  // exp2_poly3_x2

namespace gla {

// kind::f16 with fp16 A and B and fp32 D (idesc_bf16_f32 without the two
// bf16 format bits).
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, bool b_mn_major) {
  return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

template <int N>
__device__ __forceinline__ void reg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void reg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

template <int D>
struct FrameCfg {
  using G = Geo<D>;
  static constexpr int kThreads = 512;
  static constexpr int BK = 128;
  static constexpr int kRows = 256;
  static constexpr int kTileBytes = G::kTileBytes;  // [128 x D] in fp16
  static constexpr int kSlots = 2;                  // K tiles and V tiles held each
  static constexpr int kScaleSlots = 4;
  static constexpr int kAccO = 256;
  static constexpr int kBarCount = 4 * kSlots + 11;
  static constexpr int kOffK = 2 * kTileBytes;
  static constexpr int kOffV = kOffK + kSlots * kTileBytes;
  static constexpr int kOffRs = kOffV + kSlots * kTileBytes;       // [2][256] row scales
  static constexpr int kOffSc = kOffRs + 2 * kRows * 4;            // [kScaleSlots][8] float4
  static constexpr int kOffBar = kOffSc + kScaleSlots * 8 * 16;
  static constexpr int kSmemBytes = 1024 + kOffBar + kBarCount * 8 + 16;
  static_assert(kSmemBytes <= 227 * 1024, "shared memory per CTA");
  static constexpr int kPartFloats = kRows * D + 2 * kRows;
  static constexpr int kMinTiles = 4;  // least tiles of a CTA
  // registers a thread: 128 at launch (512 threads); 256 softmax threads, 128
  // converters, 128 issuers
  static constexpr int kSoftmaxRegs = 168, kConverterRegs = 112, kIssuerRegs = 64;
  static_assert(256 * kSoftmaxRegs + 128 * (kConverterRegs + kIssuerRegs) <= 512 * 128,
                "register shares beyond the launch's total would wait forever");
};

// Where the schedule goes: starts[c] = {sequence, kv head, unit, tile} of the
// first tile of CTA c and n[c] its number of tiles.
struct FrameSchedule {
  int4* starts;
  int* n;
  long long* prefix;  // used when the entries do not fit in shared memory
  int entries_max;    // host bound of the entries (units of one kv head)
  int use_smem;
  int ctas;           // CTAs of the attention kernel
  int TQ;             // tokens of a half: 128 / G
};

// One CTA.  Entry e = unit i of sequence r (all kv heads alike); prefix sums
// of the tiles over the entries, then CTA c's first tile is found by two
// searches.  Order of the tiles: sequence, kv head, unit, tile.
template <int D>
__global__ void __launch_bounds__(1024, 1)
    gla_cache_schedule_kernel(const CacheAttnParams p, const FrameSchedule fs) {
  extern __shared__ __align__(16) uint8_t sch_smem[];
  __shared__ long long scratch[33];
  int* e0 = reinterpret_cast<int*>(sch_smem);  // [R + 1] first entry of each sequence
  long long* pre = fs.use_smem
                       ? reinterpret_cast<long long*>(sch_smem + ((p.R + 1) * 4 + 15) / 16 * 16)
                       : fs.prefix;  // [entries + 1]
  const int tid = threadIdx.x;
  const int TU = 2 * fs.TQ;
  int entries;
  {
    const int per = (p.R + 1023) / 1024;
    const int r0 = min(p.R, tid * per), r1 = min(p.R, r0 + per);
    long long sum = 0, all;
    for (int r = r0; r < r1; ++r) sum += (cache_seq(p, r).n + TU - 1) / TU;
    sum = block_exclusive_scan<long long>(sum, scratch, all);
    for (int r = r0; r < r1; ++r) {
      e0[r] = static_cast<int>(sum);
      sum += (cache_seq(p, r).n + TU - 1) / TU;
    }
    if (tid == 0) e0[p.R] = static_cast<int>(all);
    __syncthreads();
    entries = static_cast<int>(all);
  }
  long long total;
  {
    const int per = (entries + 1023) / 1024;
    const int a = min(entries, tid * per), b = min(entries, a + per);
    long long sum = 0;
    if (a < b) {
      int r = prefix_owner<int>(e0, p.R, a);
      CacheSeq s = cache_seq(p, r);
      for (int e = a; e < b; ++e) {
        while (e >= e0[r + 1]) s = cache_seq(p, ++r);
        const int t = (e - e0[r]) * TU;
        const int nb = cache_span<128>(p, s, t, min(t + TU, s.n) - 1).nb;
        pre[e] = sum;
        sum += nb;
      }
    }
    const long long base = block_exclusive_scan<long long>(sum, scratch, total);
    for (int e = a; e < b; ++e) pre[e] += base;
    if (tid == 0) pre[entries] = total;
    __syncthreads();
  }
  const long long tiles = total * p.Hkv;
  const long long want = (tiles + FrameCfg<D>::kMinTiles - 1) / FrameCfg<D>::kMinTiles;
  const int ctas = static_cast<int>(want < fs.ctas ? want : fs.ctas);
  for (int c = tid; c < fs.ctas; c += 1024) {
    int4 st = make_int4(0, 0, 0, 0);
    int n = 0;
    if (c < ctas) {
      const long long x0 = share_lo(tiles, ctas, c);
      n = static_cast<int>(share_lo(tiles, ctas, c + 1) - x0);
      int lo = 0, hi = p.R;  // sequence: tiles before lo <= x0 < tiles before hi
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (pre[e0[mid]] * p.Hkv <= x0)
          lo = mid;
        else
          hi = mid;
      }
      const long long base = pre[e0[lo]];
      const long long one = pre[e0[lo + 1]] - base;  // tiles of one kv head
      long long x = x0 - base * p.Hkv;
      st.x = lo;
      st.y = static_cast<int>(x / one);
      x = x % one + base;
      const int nu = e0[lo + 1] - e0[lo];
      st.z = prefix_owner<long long>(pre + e0[lo], nu, x);
      st.w = static_cast<int>(x - pre[e0[lo] + st.z]);
    }
    fs.starts[c] = st;
    fs.n[c] = n;
  }
}

// One CTA's walk over its part of the tiles, segment by segment (a segment =
// its tiles of one unit).
struct FrameCursor {
  CacheSeq s;
  CacheSpan v;
  int r, h, i, units;
  int t0, t1;  // tiles [t0, t1) of the unit
  int left;    // tiles of this CTA from t0 on
  bool live;

  __device__ void init(const CacheAttnParams& p, const FrameSchedule& fs) {
    const int4 st = fs.starts[blockIdx.x];
    left = fs.n[blockIdx.x];
    r = st.x;
    h = st.y;
    i = st.z;
    t0 = st.w;
    live = left > 0;
    if (live) {
      seq(p, fs);
      open(p, fs);
    }
  }
  __device__ void seq(const CacheAttnParams& p, const FrameSchedule& fs) {
    s = cache_seq(p, r);
    units = (s.n + 2 * fs.TQ - 1) / (2 * fs.TQ);
  }
  __device__ void open(const CacheAttnParams& p, const FrameSchedule& fs) {
    const int t = i * 2 * fs.TQ;
    v = cache_span<128>(p, s, t, min(t + 2 * fs.TQ, s.n) - 1);
    t1 = min(v.nb, t0 + left);
  }
  __device__ void next(const CacheAttnParams& p, const FrameSchedule& fs) {
    left -= t1 - t0;
    if (left <= 0) {
      live = false;
      return;
    }
    t0 = 0;
    if (++i == units) {
      i = 0;
      if (++h == p.Hkv) {
        h = 0;
        do {
          ++r;
          seq(p, fs);
        } while (units == 0);  // tiles are left, so a sequence with rows follows
      }
    }
    open(p, fs);
  }
};

template <int D>
__global__ void __launch_bounds__(512, 1)
    gla_cache_frame_kernel(const CacheAttnParams p, const FrameSchedule fs) {
  using G = Geo<D>;
  using C = FrameCfg<D>;
  constexpr unsigned kCode = 256u;
  constexpr int KPA = G::kAtomElems / 16;  // K steps of 16 in one swizzle atom
  constexpr int kRowChunks = D / 16;       // 16-byte code chunks of a key
  constexpr int kRowsPerPass = 128 / kRowChunks;
  constexpr int kPasses = 128 / kRowsPerPass;  // 8 (d = 128) or 4 loads a thread and tile

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  auto qbuf = [&](int h) { return sbase + h * C::kTileBytes; };
  auto kbuf = [&](int s) { return sbase + C::kOffK + s * C::kTileBytes; };
  auto vbuf = [&](int s) { return sbase + C::kOffV + s * C::kTileBytes; };
  float* s_rs = reinterpret_cast<float*>(smem + C::kOffRs);
  const uint32_t s_sc = sbase + C::kOffSc;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  const uint32_t bar0 = smem_u32(bars);
  constexpr int S = C::kSlots;
  auto kfull = [&](int s) { return bar0 + 8u * s; };
  auto kempty = [&](int s) { return bar0 + 8u * (S + s); };
  auto vfull = [&](int s) { return bar0 + 8u * (2 * S + s); };
  auto vempty = [&](int s) { return bar0 + 8u * (3 * S + s); };
  const uint32_t qfull = bar0 + 8u * (4 * S);
  const uint32_t qempty = bar0 + 8u * (4 * S + 1);
  auto sfull = [&](int h) { return bar0 + 8u * (4 * S + 2 + h); };  // S_h landed
  auto pfull = [&](int h) { return bar0 + 8u * (4 * S + 4 + h); };  // P_h written, O_h scaled
  auto ofull = [&](int h) { return bar0 + 8u * (4 * S + 6 + h); };  // O_h of the segment done
  auto ofree = [&](int h) { return bar0 + 8u * (4 * S + 8 + h); };  // O_h read
  const uint32_t done_bar = bar0 + 8u * (4 * S + 10);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::kBarCount);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(kfull(s), 4);
      mbar_init(kempty(s), 2);
      mbar_init(vfull(s), 4);
      mbar_init(vempty(s), 2);
    }
    mbar_init(qfull, 4);
    mbar_init(qempty, 2);
    for (int h = 0; h < 2; ++h) {
      mbar_init(sfull(h), 1);
      mbar_init(pfull(h), 4);
      mbar_init(ofull(h), 1);
      mbar_init(ofree(h), 4);
    }
    mbar_init(done_bar, 2);
    *abort = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the schedule is written
  if (threadIdx.x == 0) p.desc[8 * blockIdx.x] = 0;   // nothing to join, unless set below

  const int used = fs.TQ * p.G;  // rows of a half in use
  if (warp >= 12) {
    // ------------------------------------------------------------ MMA issuers
    reg_dec<C::kIssuerRegs>();
    const int me = warp - 12;
    if (me < 2 && lane == 0) {
      constexpr uint32_t idesc_s = idesc_f16_f32(128, 128, false);
      constexpr uint32_t idesc_o = idesc_f16_f32(128, D, true);
      constexpr uint64_t kStep = C::kTileBytes >> 4;  // next buffer, in the address field
      const uint64_t qd = smem_desc(qbuf(me), 16, G::kGroupBytes, G::kLayout);
      const uint64_t kd = smem_desc(kbuf(0), 16, G::kGroupBytes, G::kLayout);
      const uint64_t vd = smem_desc(vbuf(0), G::kAtomTileBytes, G::kGroupBytes, G::kLayout);
      const uint32_t ts = tmem + me * 128, to = tmem + C::kAccO + me * D;
      uint32_t n = 0, seg = 0;  // tiles and segments so far
      FrameCursor cur;
      cur.init(p, fs);
      bool ok = true;
      for (; cur.live && ok; cur.next(p, fs), ++seg) {
        ok = mbar_wait(qfull, seg & 1u, abort, kCode);
        auto issue_s = [&](uint32_t k) {  // S of tile k of this CTA
          if (!mbar_wait(kfull(k & 1u), (k >> 1) & 1u, abort, kCode)) return false;
          tc_fence_after();
          const uint64_t b0 = kd + (k & 1u) * kStep;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint64_t off =
                static_cast<uint64_t>(((kk / KPA) * G::kAtomTileBytes + (kk % KPA) * 32) >> 4);
            mma_bf16(ts, qd + off, b0 + off, idesc_s, kk > 0 ? 1u : 0u);
          }
          mma_commit(sfull(me));
          mma_commit(kempty(k & 1u));
          return true;
        };
        if (ok) ok = issue_s(n);
        for (int t = cur.t0; t < cur.t1 && ok; ++t, ++n) {
          const bool first = t == cur.t0, last = t + 1 == cur.t1;
          if (last) mma_commit(qempty);  // every S of the segment has been issued
          if (first && !mbar_wait(ofree(me), (seg & 1u) ^ 1u, abort, kCode)) ok = false;
          if (!ok || !mbar_wait(vfull(n & 1u), (n >> 1) & 1u, abort, kCode) ||
              !mbar_wait(pfull(me), n & 1u, abort, kCode)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t b0 = vd + (n & 1u) * kStep;
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)  // 16 keys = 8 columns of P
            mma_bf16_ts(to, ts + kk * 8, b0 + static_cast<uint64_t>((kk * 2 * G::kGroupBytes) >> 4),
                        idesc_o, (first && kk == 0) ? 0u : 1u);
          mma_commit(vempty(n & 1u));
          if (last)
            mma_commit(ofull(me));
          else
            ok = issue_s(n + 1);
        }
      }
      mma_commit(done_bar);
      mbar_wait_drain(done_bar, 0);
    }
  } else if (warp >= 8) {
    // ------------------------------------------------------------- converters
    reg_dec<C::kConverterRegs>();
    const int cw = warp - 8, ct = threadIdx.x - 256;
    const int ch = ct % kRowChunks, row0 = ct / kRowChunks;
    const int P = 1 << p.p_shift;
    const int64_t page_rows = static_cast<int64_t>(p.Hkv) << p.p_shift;
    uint4 ka[kPasses], va[kPasses];
    float ksc = 1.f, vsc = 0.f;  // lanes 0 .. 7 of every warp: scales of 16-key group `lane`
    FrameCursor ld;              // the tile loaded next
    ld.init(p, fs);
    int lt = ld.t0;
    int page_of[8];              // pages of the tile's 16-key groups (-1: nothing visible there)
    int64_t off[kPasses];        // byte offset of this thread's chunk in every pass (-1: zeros)
    auto locate = [&]() {        // pages and offsets of tile lt of ld
      const int base = ld.v.pos(lt, C::BK);
      const int* row = p.table + static_cast<int64_t>(ld.r) * p.max_pages;
      const int a = base + 16 * (lane & 7);
      const int j = a >> p.p_shift;
      int pg = -1;
      if (j < p.max_pages && a < ld.v.hi && (a + 16 > ld.v.lo || a < ld.v.sink)) pg = row[j];
      if (pg >= p.pages) pg = -1;
      ksc = 1.f;
      vsc = 0.f;
      if (pg >= 0 && cw == 0 && lane < 8) {
        const int64_t x = static_cast<int64_t>(pg) * p.Hkv + ld.h;
        ksc = p.ks[x];
        vsc = p.vs[x];
      }
#pragma unroll
      for (int g = 0; g < 8; ++g) page_of[g] = __shfl_sync(0xffffffffu, pg, g);
#pragma unroll
      for (int i = 0; i < kPasses; ++i) {
        const int kr = i * kRowsPerPass + row0;
        const int key = base + kr;
        int pgk = page_of[i * kRowsPerPass / 16];
        if (kRowsPerPass > 16 && row0 >= 16) pgk = page_of[i * kRowsPerPass / 16 + 1];
        off[i] = pgk >= 0 && ld.v.sees(key)
                     ? (pgk * page_rows + (static_cast<int64_t>(ld.h) << p.p_shift) +
                        (key & (P - 1))) * D + ch * 16
                     : -1;
      }
    };
    auto load = [&](uint4 (&x)[kPasses], const uint8_t* src) {
#pragma unroll
      for (int i = 0; i < kPasses; ++i) {
        x[i] = make_uint4(0, 0, 0, 0);
        if (off[i] >= 0) x[i] = __ldg(reinterpret_cast<const uint4*>(src + off[i]));
      }
    };
    auto advance = [&]() {
      if (++lt >= ld.t1) {
        ld.next(p, fs);
        lt = ld.t0;
      }
    };
    // 16 codes -> 32 bytes of fp16 in the swizzled row; the odd half of the
    // lanes writes its two chunks in the other order (bank conflicts)
    auto convert = [&](const uint4 (&x)[kPasses], uint32_t buf) {
      const int c2 = (ch * 2) & 7;  // first 16-byte chunk within its 128-byte atom row
      const uint32_t atom = static_cast<uint32_t>(ch * 2 / 8) * G::kAtomTileBytes;
      const bool swap = (ch & 4) != 0;
#pragma unroll
      for (int i = 0; i < kPasses; ++i) {
        const int kr = i * kRowsPerPass + row0;
        const uint32_t rowp = buf + atom + kr * 128;
        uint4 a, b;
        a.x = e4m3x2_to_f16x2(x[i].x & 0xFFFFu);
        a.y = e4m3x2_to_f16x2(x[i].x >> 16);
        a.z = e4m3x2_to_f16x2(x[i].y & 0xFFFFu);
        a.w = e4m3x2_to_f16x2(x[i].y >> 16);
        b.x = e4m3x2_to_f16x2(x[i].z & 0xFFFFu);
        b.y = e4m3x2_to_f16x2(x[i].z >> 16);
        b.z = e4m3x2_to_f16x2(x[i].w & 0xFFFFu);
        b.w = e4m3x2_to_f16x2(x[i].w >> 16);
        const uint32_t pa = rowp + ((c2 ^ (kr & 7)) << 4);
        const uint32_t pb = rowp + (((c2 + 1) ^ (kr & 7)) << 4);
        st_shared_v4(swap ? pb : pa, swap ? b : a);
        st_shared_v4(swap ? pa : pb, swap ? a : b);
      }
      fence_proxy_async_smem();
      __syncwarp();
    };
    if (ld.live) {
      locate();
      load(ka, p.k8);
      load(va, p.v8);
    }
    FrameCursor cur;
    cur.init(p, fs);
    uint32_t n = 0, seg = 0;
    bool ok = true;
    for (; cur.live && ok; cur.next(p, fs), ++seg) {
      // ---- queries: bf16 -> fp16, scaled per row
      constexpr int kQChunks = D / 8, kQRows = 128 / kQChunks, kBatch = 8;
      if (!warp_wait(qempty, (seg & 1u) ^ 1u, abort, kCode)) break;
      const int qc = ct % kQChunks, qr0 = ct / kQChunks;
      const int t_unit = cur.i * 2 * fs.TQ;
#pragma unroll 1
      for (int pass = 0; pass < 256 / kQRows; pass += kBatch) {
        uint4 x[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int row = (pass + i) * kQRows + qr0;
          const int lr = row & 127;
          const int t = t_unit + (row >> 7) * fs.TQ + lr / p.G;
          x[i] = make_uint4(0, 0, 0, 0);
          if (lr < used && t < cur.s.n)
            x[i] = __ldg(reinterpret_cast<const uint4*>(
                p.q + ((static_cast<int64_t>(cur.s.c0) + t) * p.H + cur.h * p.G + lr % p.G) * D +
                qc * 8));
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int row = (pass + i) * kQRows + qr0;
          uint32_t mx = __vmaxu2(__vmaxu2(x[i].x & 0x7FFF7FFFu, x[i].y & 0x7FFF7FFFu),
                                 __vmaxu2(x[i].z & 0x7FFF7FFFu, x[i].w & 0x7FFF7FFFu));
          mx = max(mx & 0xFFFFu, mx >> 16);
#pragma unroll
          for (int o = kQChunks / 2; o > 0; o >>= 1)
            mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
          float f, inv;
          row_scale(mx, f, inv);
          uint4 w;
          w.x = pack_f16x2(bf16lo_to_f32(x[i].x) * f, bf16hi_to_f32(x[i].x) * f);
          w.y = pack_f16x2(bf16lo_to_f32(x[i].y) * f, bf16hi_to_f32(x[i].y) * f);
          w.z = pack_f16x2(bf16lo_to_f32(x[i].z) * f, bf16hi_to_f32(x[i].z) * f);
          w.w = pack_f16x2(bf16lo_to_f32(x[i].w) * f, bf16hi_to_f32(x[i].w) * f);
          const int lr = row & 127;
          st_shared_v4(qbuf(row >> 7) + (qc >> 3) * G::kAtomTileBytes + lr * 128 +
                           (((qc & 7) ^ (lr & 7)) << 4),
                       w);
          if (qc == 0) s_rs[(seg & 1u) * C::kRows + row] = inv * p.sl2;
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(qfull);
      // ---- key / value tiles
      for (int t = cur.t0; t < cur.t1; ++t, ++n) {
        const int sl = n & 1u;
        const uint32_t ph = ((n >> 1) & 1u) ^ 1u;
        if (!warp_wait(kempty(sl), ph, abort, kCode)) {
          ok = false;
          break;
        }
        convert(ka, kbuf(sl));
        if (cw == 0 && lane < 8) {
          // scale slot n % 4: its last reader finished tile n - 4 before S of
          // tile n - 2 was issued, which the wait above has seen complete
          const float lv = lg2_approx(vsc);  // -inf where nothing is visible
          const float iv = vsc > 0.f ? ex2_approx(-lv) : 0.f;
          st_shared_v4(s_sc + (n & 3u) * 128 + lane * 16,
                       make_uint4(__float_as_uint(ksc), __float_as_uint(lv), __float_as_uint(iv),
                                  0u));
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(kfull(sl));
        advance();
        const bool more = ld.live;
        if (!warp_wait(vempty(sl), ph, abort, kCode)) {
          ok = false;
          break;
        }
        if (more) {
          locate();
          load(ka, p.k8);
        }
        convert(va, vbuf(sl));
        if (lane == 0) mbar_arrive(vfull(sl));
        if (more) load(va, p.v8);
      }
    }
  } else {
    // -------------------------------------------------- softmax and epilogue
    reg_inc<C::kSoftmaxRegs>();
    const int half = warp >> 2, q4 = warp & 3;
    const int row = q4 * 32 + lane;  // row of the half
    const uint32_t lane_base = static_cast<uint32_t>(q4 * 32) << 16;
    const uint32_t ts = tmem + lane_base + half * 128;
    const uint32_t to = tmem + lane_base + C::kAccO + half * D;
    uint32_t n = 0, seg = 0;
    FrameCursor cur;
    cur.init(p, fs);
    for (; cur.live; cur.next(p, fs), ++seg) {
      const int t = cur.i * 2 * fs.TQ + half * fs.TQ + row / p.G;
      const bool have = row < used && t < cur.s.n;
      // rows that hold no query see everything: they cost no mask
      const int hi = have ? key_hi(p, cur.s, cur.s.p0 + t) : INT32_MAX;
      const int lo = have ? key_lo(p, cur.s.p0 + t) : 0;
      bool ok = true;
      float rs = 0.f, m = -INFINITY, l = 0.f;
      for (int tile = cur.t0; tile < cur.t1 && ok; ++tile, ++n) {
        const int base = cur.v.pos(tile, C::BK);
        if (!warp_wait_fast(sfull(half), n & 1u, abort, kCode)) {
          ok = false;
          break;
        }
        tc_fence_after();
        // the row scales of segment seg are written before its first S and
        // replaced after the last P of segment seg + 1
        if (tile == cur.t0) rs = s_rs[(seg & 1u) * C::kRows + half * 128 + row];
        uint32_t s[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld_32cols(ts + c * 32, s[c]);
        tmem_wait_ld();
        const bool whole = base >= lo && base + C::BK <= hi;
        if (!__all_sync(0xffffffffu, whole)) {
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const int key = base + c * 32 + e;
              if (!(key < hi && (key >= lo || key < p.n_sink)))
                s[c][e] = __float_as_uint(-INFINITY);
            }
        }
        const uint32_t sc = s_sc + (n & 3u) * 128;
        float mt = -INFINITY;
#pragma unroll
        for (int g = 0; g < 8; ++g) {
          const uint32_t* x = &s[g >> 1][(g & 1) * 16];
          float a = fmax3(__uint_as_float(x[0]), __uint_as_float(x[1]), __uint_as_float(x[2]));
          float b = fmax3(__uint_as_float(x[3]), __uint_as_float(x[4]), __uint_as_float(x[5]));
          a = fmax3(a, __uint_as_float(x[6]), __uint_as_float(x[7]));
          b = fmax3(b, __uint_as_float(x[8]), __uint_as_float(x[9]));
          a = fmax3(a, __uint_as_float(x[10]), __uint_as_float(x[11]));
          b = fmax3(b, __uint_as_float(x[12]), __uint_as_float(x[13]));
          a = fmax3(a, __uint_as_float(x[14]), __uint_as_float(x[15]));
          const float4 k = ld_shared_f4(sc + g * 16);
          mt = fmaxf(mt, fmaf(fmaxf(a, b), rs * k.x, k.y));
        }
        const bool grow = mt > m + kCacheLazy;  // also the first visible key: m = -inf
        if (__any_sync(0xffffffffu, grow && tile != cur.t0)) {
          // O of the previous tiles is complete: S of this tile was issued
          // after the last P V by the same thread
          const float f = grow ? (m == -INFINITY ? 0.f : ex2_approx(m - mt)) : 1.0f;
          if (grow) {
            l *= f;
            m = mt;
          }
#pragma unroll 1
          for (int c = 0; c < D / 16; ++c) {
            uint32_t o[16];
            tmem_ld_16cols(to + c * 16, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            tmem_st_16cols(to + c * 16, o);
          }
          tmem_wait_st();
        } else if (grow) {
          m = mt;
        }
        const float sh = m == -INFINITY ? 0.f : kCacheBias - m;
#pragma unroll
        for (int hb = 0; hb < 2; ++hb) {
          uint32_t pw[32];
#pragma unroll
          for (int gg = 0; gg < 4; ++gg) {
            const int g = hb * 4 + gg;
            const float4 k = ld_shared_f4(sc + g * 16);
            const float fg = rs * k.x, sg = k.y + sh;
            const uint64_t f2 = f2_pack(fg, fg), s2 = f2_pack(sg, sg);
            uint64_t sum = f2_pack(0.f, 0.f);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const uint32_t* x = &s[g >> 1][(g & 1) * 16 + 2 * e];
              float a0, a1, y0, y1;
              f2_unpack(f2_fma(f2_pack(__uint_as_float(x[0]), __uint_as_float(x[1])), f2, s2), a0,
                        a1);
              if ((e & 3) == 0) {
                exp2_poly3_x2(a0, a1, y0, y1);
              } else {
                y0 = ex2_approx(a0);
                y1 = ex2_approx(a1);
              }
              sum = f2_add(sum, f2_pack(y0, y1));
              pw[gg * 8 + e] = pack_f16x2(y0, y1);
            }
            float l0, l1;
            f2_unpack(sum, l0, l1);
            l = fmaf(l0 + l1, k.z, l);
          }
          tmem_st_32cols(ts + hb * 32, pw);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(pfull(half));
      }
      if (!ok || !warp_wait(ofull(half), seg & 1u, abort, kCode)) break;
      tc_fence_after();
      // ---- the segment's result: out, or a partial when the unit goes on elsewhere
      const bool starts = cur.t0 == 0, ends = cur.t1 == cur.v.nb;
      const int64_t at = have ? ((static_cast<int64_t>(cur.s.c0) + t) * p.H + cur.h * p.G +
                                 row % p.G) * D
                              : 0;
      const float rl = m == -INFINITY ? 0.f : 1.0f / l;
      float* part = p.part + (2ll * blockIdx.x + (starts ? 1 : 0)) * C::kPartFloats;
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        tmem_ld_32cols(to + c * 32, o);
        tmem_wait_ld();
        if (!have) continue;
        if (starts && ends) {
          const uint4* zp = reinterpret_cast<const uint4*>(p.z + at + c * 32);
          uint4* op = reinterpret_cast<uint4*>(p.out + at + c * 32);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            float x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = __uint_as_float(o[q * 8 + e]) * rl;
            if (p.z != nullptr) {
              const uint4 zw = __ldg(zp + q);
              const uint32_t zz[4] = {zw.x, zw.y, zw.z, zw.w};
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float zf = (e & 1) ? bf16hi_to_f32(zz[e >> 1]) : bf16lo_to_f32(zz[e >> 1]);
                x[e] *= 1.0f / (1.0f + __expf(-zf));
              }
            }
            op[q] = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                               pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
          }
        } else {
          float4* dst = reinterpret_cast<float4*>(part + (half * 128 + row) * D + c * 32);
          // rows that saw no key in this part hold zeros in O already
#pragma unroll
          for (int q = 0; q < 8; ++q)
            dst[q] = make_float4(__uint_as_float(o[4 * q]), __uint_as_float(o[4 * q + 1]),
                                 __uint_as_float(o[4 * q + 2]), __uint_as_float(o[4 * q + 3]));
        }
      }
      if (!(starts && ends))
        *reinterpret_cast<float2*>(part + C::kRows * D + 2 * (half * 128 + row)) =
            make_float2(m, l);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(ofree(half));
      if (threadIdx.x == 0 && starts && !ends) {
        // this unit's parts: this CTA, then every one up to the last tile
        int parts = 1, rest = cur.v.nb - cur.t1;
        for (int c = blockIdx.x + 1; rest > 0 && c < static_cast<int>(gridDim.x); ++c) {
          ++parts;
          rest -= fs.n[c];
        }
        int* desc = p.desc + 8 * blockIdx.x;
        desc[1] = cur.s.c0;
        desc[2] = cur.i * 2 * fs.TQ * p.G;
        desc[3] = cur.h;
        desc[4] = min(2 * fs.TQ, cur.s.n - cur.i * 2 * fs.TQ) * p.G;
        desc[0] = parts;
      }
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace gla
