// gla_cache_frame.cuh -- attention of many queries a sequence (frames, prompts)
// over the paged 8-bit cache, on tcgen05.  The definition is that of
// gla_cache_token.cuh.
//
// With many query rows a call is bound by the tensor cores: 4 d flops for each
// query, visible key and head.  One work unit = 256 query rows (tokens x the
// heads that share a key/value head) of one sequence and key/value head, held
// as two halves of 128 rows; its visible keys are cut into tiles of 128.  The
// tiles of all units, and a fixed cost before each unit, are laid end to end and
// dealt out evenly to one CTA per SM (gla_cache_schedule_kernel finds where each
// CTA begins); a unit that ends up in several CTAs leaves a partial (O, m, l) in
// each, joined by gla_cache_join_kernel.
//
// Both halves of a unit share each key/value tile, because every tile has to
// be converted first: tcgen05 wants both operands of a product in one type,
// and q in 8 bits would cost its precision.  A producer warp brings the codes
// in by bulk copies (a page of one head is contiguous), four converter warps
// turn them into fp16 and write them in the swizzled operand layout.  All 128
// keys of a tile take one key scale and one value scale, the largest of its
// pages': the converters multiply the codes of the other pages by the ratio, a
// power of two (exact while it is at least 2^-15; a page 2^25 or more below
// another of its tile counts as zeros).  Keys that no row of the unit sees become zeros there, so
// stray pages and NaN codes never reach a product.
//   S_h = Q_h K^T   A = Q half [128 x d] K-major, B = K tile [128 keys] K-major
//   O_h += P_h V    A = P_h in TMEM (fp16, over the columns of S_h),
//                   B = V tile [128 keys x d] MN-major
// Each half's queries have their own buffer and barriers: half 0 takes the next
// unit's while half 1 still works on the old one.
// TMEM: S_0, S_1 (128 columns each), O_0, O_1 (d columns each).  One issuing
// warp per half: P V of tile j (in two steps of 64 keys, as P is written), then
// S of tile j + 1 into the same columns (the tensor core runs one thread's
// products in order), while the other half's softmax runs.
// Softmax: one thread per row.  P' = 2^(S f + lv - m + kCacheBias), f = key scale
// x row scale x softmax scale x log2 e, lv = log2 of the value scale (taken out
// of the row sum again).  The maximum of a tile is not taken as a rule: the
// row's reference m stays while the sum of P' over 64 keys stays below 2^15
// (then no P' leaves the fp16 range); otherwise, and on the first keys that a
// row sees, they are read again, m becomes their maximum, and O is rescaled.
// (At d = 64 one pair of exponentials in four runs on the FMA pipe, exp2_poly3_x2.)
// Warp roles: 0-3 / 4-7 softmax and epilogue of half 0 / 1, 8-11 converters,
// 12 / 13 MMA issuers of half 0 / 1, 14 producer (15 idle: it completes the
// register group).
// Measured (d = 128): 3680 queries x 14976 visible keys x 24 heads in 792-809 us,
// 0.84-0.86 PFLOP/s, 0.60 of the sustained bf16 rate (0.50 of the burst rate, which
// the clock of so short a run is nearer to).  A tile takes about 4700 cycles
// of 2048 on the tensor core, a unit 3 (d = 64) to 6 tiles more; the rest is the chain scores -> exponentials ->
// P V -> next scores of two halves, one warp a scheduler each.  The roles share
// the instruction cache: code size is time here (156 KB of code ran 1.3 times as
// long as 97 KB), hence the rolled loops and cold passes.
#pragma once

#include "gla_cache_token.cuh"
#include "gla_common.cuh"
#include "gla_softmax_anchor.cuh"  // exp2_poly3_parts_x2

namespace gla {

// kind::f16 with fp16 A and B and fp32 D (idesc_bf16_f32 without the two
// bf16 format bits).
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, bool b_mn_major) {
  return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

// One lane of a converged warp, the same one at every call.
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(ok));
  return ok != 0;
}

template <int N>
__device__ __forceinline__ void reg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void reg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// mbar_wait with a suspend hint: a waiting warp leaves the issue slots to the
// others for up to 20 us at a time instead of polling.
__device__ __forceinline__ bool mbar_wait_idle(uint32_t bar, uint32_t parity, volatile int* abort,
                                               unsigned int code) {
  uint64_t t0 = 0;
  for (;;) {
    uint32_t ok;  // up to 16 tries
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .u32 c;\n\t"
        "mov.u32 c, 0;\n\t"
        "TRY_%=:\n\t"
        "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "@p bra DONE_%=;\n\t"
        "add.u32 c, c, 1;\n\t"
        "setp.lt.u32 q, c, 16;\n\t"
        "@q bra TRY_%=;\n\t"
        "DONE_%=:\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(20000u)
        : "memory");
    if (ok) return true;
    if (*abort) return false;
    const uint64_t now = global_timer_ns();
    if (t0 == 0) {
      t0 = now;
    } else if (now - t0 > g_gla_wait_limit_ns) {
      *abort = 1;
      atomicOr(&g_gla_fault, code);
      return false;
    }
  }
}

// The same for every lane of a warp (each lane acquires by its own wait).
__device__ __forceinline__ bool warp_wait_idle(uint32_t bar, uint32_t parity, volatile int* abort,
                                               unsigned int code) {
  const bool ok = mbar_wait_idle(bar, parity, abort, code);
  return __all_sync(0xffffffffu, ok);
}

// tcgen05.wait::ld that the registers of the load depend on: nothing that uses
// them can be moved before it.
__device__ __forceinline__ void tmem_wait_ld_of(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]),
                 "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}

__device__ __forceinline__ void tmem_wait_ld_of(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}

// 32-byte global accesses, a whole sector for each lane.
__device__ __forceinline__ void st_global_v8(void* p, const uint32_t (&v)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// exp2_poly3_x2 for any argument.  The weights of 64 keys are computed before
// their maximum is known, and from 129 on the exponent field would run into the
// sign: from kExp2Top on the result is 2^kExp2Top, beyond every sum that passes for
// right.  A NaN stays one (a row that is not finite must not come out as 0): the
// bounds hand it on, and 2^n is multiplied in, where an integer added to the
// exponent field would make a number of it.
constexpr float kExp2Top = 127.0f;

__device__ __forceinline__ float clamp_nan(float x, float lo, float hi) {
  float y;
  asm("{\n\t.reg .f32 t;\n\t"
      "min.NaN.f32 t, %1, %3;\n\t"
      "max.NaN.f32 %0, t, %2;\n\t}\n"
      : "=f"(y)
      : "f"(x), "f"(lo), "f"(hi));
  return y;
}

__device__ __forceinline__ void exp2_poly3_any_x2(float a0, float a1, float& x0, float& x1) {
  float t0, t1;
  uint64_t t;
  const uint64_t p = exp2_poly3_parts_x2(
      f2_pack(clamp_nan(a0, -126.0f, kExp2Top), clamp_nan(a1, -126.0f, kExp2Top)), t);
  f2_unpack(t, t0, t1);
  // bits of t << 23: n in the exponent field; with the field of 1.0: 2^n
  const uint64_t e = f2_pack(__int_as_float((__float_as_int(t0) << 23) + 0x3F800000),
                             __int_as_float((__float_as_int(t1) << 23) + 0x3F800000));
  f2_unpack(f2_mul(p, e), x0, x1);
}

// Bits 0 .. n - 1 (none for n <= 0, all for n >= 32).
__device__ __forceinline__ uint32_t bits_below(int n) {
  return n >= 32 ? 0xFFFFFFFFu : (n <= 0 ? 0u : (1u << n) - 1u);
}

// Which of the 32 keys from `key` on a row sees: [lo, hi) and the sinks.
__device__ __forceinline__ uint32_t visible_bits(int key, int lo, int hi, int n_sink) {
  return bits_below(hi - key) & (~bits_below(lo - key) | bits_below(n_sink - key));
}

// What the producer leaves about a tile and about a segment (a CTA's tiles of
// one unit), so that no other warp has to walk the schedule: registers are what
// the softmax and the converters have least of, and a spilled one costs a trip
// to L2 here (shared memory takes nearly all of L1).
struct TileInfo {
  uint32_t kfac[8], vfac[8];  // fp16 pair: scale of each 16-key group over the tile's
  float ks, lv, iv;           // key scale; log2 of the value scale and 2^-lv
  uint32_t flags;
  int base;                   // position of the first key
  uint32_t pad[3];
};
static_assert(sizeof(TileInfo) == 96, "one slot of the info ring");
enum : uint32_t {
  kTileBad = 255u,     // bit g: 16-key group g has no page
  kTileAll = 256u,     // every key of the tile is visible to some row
  kTileScaleK = 512u,  // the factors of K (V) are not all 1
  kTileScaleV = 1024u,
  kTileFirst = 2048u,  // first, last tile of its segment
  kTileLast = 4096u,
};
struct SegInfo {
  long long row0;    // (first token of the unit) * H + (first query head): row of q and out
  int tokens;        // tokens of the unit (at most 2 TQ count)
  int p0;            // position of its first token
  int len;           // keys of the sequence
  int lo, hi, sink;  // visible keys, as in CacheSpan
  int whole, starts; // the segment is the unit; it holds the unit's first tile
  int c0, t_unit, h;  // for the join: packed row and token of the unit's start, head
  int pad;
};
static_assert(sizeof(SegInfo) == 56, "one slot of the segment ring");

template <int D>
struct FrameCfg {
  using G = Geo<D>;
  static constexpr int kThreads = 512;
  static constexpr int BK = 128;
  static constexpr int kRows = 256;
  static constexpr int kTileBytes = G::kTileBytes;  // [128 x D] in fp16
  static constexpr int kSlots = 2;                  // K tiles and V tiles held each
  static constexpr int kInfoSlots = 8;
  static constexpr int kAccO = 256;
  static constexpr int kBarCount = 4 * kSlots + 29;
  static constexpr int kOffK = 2 * kTileBytes;
  static constexpr int kOffV = kOffK + kSlots * kTileBytes;
  static constexpr int kOffRs = kOffV + kSlots * kTileBytes;       // [2][256] row exponents
  static constexpr int kOffInfo = kOffRs + 2 * kRows;              // [kInfoSlots] TileInfo
  static constexpr int kOffSeg = kOffInfo + kInfoSlots * 96;      // [kInfoSlots] SegInfo
  static constexpr int kOffRaw = kOffSeg + kInfoSlots * 56;        // codes of one K, one V tile
  static constexpr int kRawBytes = 128 * D;
  static constexpr int kOffBar = kOffRaw + 2 * kRawBytes;
  static constexpr int kSmemBytes = 1024 + kOffBar + kBarCount * 8 + 16;
  static_assert(kSmemBytes <= 227 * 1024, "shared memory per CTA");
  static constexpr int kPartFloats = kRows * D + 2 * kRows;
  static constexpr int kMinTiles = 4;  // least tiles of a CTA
  // what a unit costs beyond its tiles (queries, first and masked tiles, result), in
  // tiles.  Ragged prompts of up to 2048 tokens on up to 4096 keys, shares by tiles
  // alone / with 2, 3, 4, 5, 6, 8 for a unit: d = 64 343 / 298, 287, 289, 290, 293,
  // 302 us; d = 128 465 / -, 375, 359, 355, 347, 350 us.
  static constexpr int kUnitTiles = D == 128 ? 6 : 3;
  // The two halves' softmax warps of one scheduler take turns (d = 128) or run
  // as they come (d = 64).  Left alone, the halves fall into step: both in the
  // softmax, then both on the tensor core.  Taking turns keeps one on each; a
  // lone warp is then bound by its instructions, not by the exponential unit,
  // so all exponentials go there.  Measured, turns / as they come with one pair
  // of exponentials in four on the FMA pipe (before units had their cost in the
  // schedule): 801 / about 880 us (d = 128, 3680 queries, 14720 keys, 24 heads),
  // 365 / 348 us (d = 64 ragged prompts: half the tensor work, little to hide
  // behind; the bounds on the polynomial's argument add 2%).
  static constexpr bool kTurns = D == 128;
  // registers a thread: 128 at launch (512 threads); 256 softmax threads, 128
  // converters, 128 issuers and producer
  static constexpr int kSoftmaxRegs = 160, kConverterRegs = 96, kIssuerRegs = 96;
  static_assert(256 * kSoftmaxRegs + 128 * (kConverterRegs + kIssuerRegs) <= 512 * 128,
                "register shares beyond the launch's total would wait forever");
};

constexpr int kMaxScheduleCtas = 1024;
constexpr int kJoinTiles = 6;  // what writing and joining partials costs, in tiles (measured at
                               // d = 128: about 17 us and 2.9 us)

// Where the schedule goes: starts[c] = {sequence, kv head, unit, tile} of the
// first tile of CTA c and n[c] its number of tiles (and see there).
struct FrameSchedule {
  int4* starts;
  int2* n;            // tiles, CTAs that share the unit which begins here and goes on
  long long* prefix;  // used when the entries do not fit in shared memory
  int entries_max;    // host bound of the entries (units of one kv head)
  int use_smem;
  int ctas;           // CTAs of the attention kernel
  int TQ;             // tokens of a half: 128 / G
};

// One CTA.  Entry e = unit i of sequence r (all kv heads alike); prefix sums
// of their cost over the entries, then CTA c's first tile is found by two
// searches.  A unit costs its tiles and kUnitTiles for its queries and its result,
// which lie before its first tile.  Order: sequence, kv head, unit, tile.
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
  constexpr int kUnitTiles = FrameCfg<D>::kUnitTiles;
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
    // rows that descend or overlap can ask for more entries than there is room
    // for: then there is no work
    if (all > fs.entries_max) all = 0;
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
        sum += nb + kUnitTiles;
      }
    }
    const long long base = block_exclusive_scan<long long>(sum, scratch, total);
    for (int e = a; e < b; ++e) pre[e] += base;
    if (tid == 0) pre[entries] = total;
    __syncthreads();
  }
  const long long cost = total * p.Hkv;
  const long long tiles = cost - static_cast<long long>(entries) * p.Hkv * kUnitTiles;
  struct Place {
    int4 st;            // sequence, kv head, unit, tile
    int off, w, nt;     // cost since the unit's start, of the unit; tiles of the unit
    long long before;   // tiles before this one
  };
  auto find = [&](long long x0) {  // 0 <= x0 < cost
    int lo = 0, hi = p.R;  // sequence: cost before lo <= x0 < cost before hi
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (pre[e0[mid]] * p.Hkv <= x0)
        lo = mid;
      else
        hi = mid;
    }
    const int units = e0[lo + 1] - e0[lo];
    const long long base = pre[e0[lo]];
    const long long one = pre[e0[lo + 1]] - base;  // of one kv head
    const long long x = x0 - base * p.Hkv;
    Place f;
    f.st.x = lo;
    f.st.y = static_cast<int>(x / one);
    const long long in_head = x % one + base;
    f.st.z = prefix_owner<long long>(pre + e0[lo], units, in_head);
    const long long start = pre[e0[lo] + f.st.z];
    f.off = static_cast<int>(in_head - start);
    f.w = static_cast<int>(pre[e0[lo] + f.st.z + 1] - start);
    f.nt = f.w - kUnitTiles;
    f.st.w = max(f.off - kUnitTiles, 0);
    const long long units_before = static_cast<long long>(e0[lo]) * p.Hkv +
                                   static_cast<long long>(f.st.y) * units + f.st.z;
    f.before = x0 - f.off - units_before * kUnitTiles + f.st.w;
    return f;
  };
  // Equal shares over as many CTAs as there are tiles, cut at the nearest unit
  // (no partials, no join), where that costs no CTA more than kJoinTiles tiles;
  // otherwise cut anywhere, kMinTiles tiles a CTA at least.
  __shared__ long long s_cut[kMaxScheduleCtas + 1];
  int ctas = 0;
  bool cut = true;
#pragma unroll 1
  for (int least = 1; cut && least <= FrameCfg<D>::kMinTiles; least += FrameCfg<D>::kMinTiles - 1) {
    const long long want = (tiles + least - 1) / least;
    ctas = static_cast<int>(want < fs.ctas ? want : fs.ctas);
    for (int c = tid; c <= ctas; c += 1024) {
      long long x = share_lo(cost, max(ctas, 1), c);
      if (c > 0 && c < ctas) {
        const Place f = find(x);
        x += 2 * f.off >= f.w ? f.w - f.off : -f.off;
      }
      s_cut[c] = x;
    }
    __syncthreads();
    const long long share = ctas > 0 ? (cost + ctas - 1) / ctas : 0;
    int over = 0;
    for (int c = tid; c < ctas; c += 1024) over |= s_cut[c + 1] - s_cut[c] > share + kJoinTiles;
    cut = __syncthreads_or(over);
  }
  // the cuts in tiles, and the end of the unit that each cut splits
  __shared__ long long s_end[kMaxScheduleCtas + 1];
  for (int c = tid; c <= ctas; c += 1024) {
    const long long x = cut && ctas > 0 ? share_lo(cost, ctas, c) : s_cut[c];
    long long before = tiles, end = tiles;
    if (x < cost) {
      const Place f = find(x);
      before = f.before;
      end = f.st.w > 0 ? before - f.st.w + f.nt : before;
      if (c < ctas) fs.starts[c] = f.st;
    }
    s_cut[c] = before;
    s_end[c] = end;
  }
  __syncthreads();
  for (int c = tid; c < fs.ctas; c += 1024) {
    int n = 0, last = c;
    if (c < ctas) {
      n = static_cast<int>(s_cut[c + 1] - s_cut[c]);
      int hi = ctas - 1;  // first CTA from c on whose tiles reach the unit's end
      while (last < hi) {
        const int mid = (last + hi) >> 1;
        if (s_cut[mid + 1] >= s_end[c + 1])
          hi = mid;
        else
          last = mid + 1;
      }
    }
    fs.n[c] = make_int2(n, last - c + 1);
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
    left = fs.n[blockIdx.x].x;
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
  constexpr int kPasses = 128 / kRowsPerPass;  // 8 (d = 128) or 4 chunks a thread and tile

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  auto qbuf = [&](int h) { return sbase + h * C::kTileBytes; };
  auto kbuf = [&](int s) { return sbase + C::kOffK + s * C::kTileBytes; };
  auto vbuf = [&](int s) { return sbase + C::kOffV + s * C::kTileBytes; };
  int8_t* s_rs = reinterpret_cast<int8_t*>(smem + C::kOffRs);
  TileInfo* s_info = reinterpret_cast<TileInfo*>(smem + C::kOffInfo);
  SegInfo* s_seg = reinterpret_cast<SegInfo*>(smem + C::kOffSeg);
  constexpr uint32_t kRing = C::kInfoSlots - 1;
  const uint32_t kraw = sbase + C::kOffRaw, vraw = kraw + C::kRawBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  const uint32_t bar0 = smem_u32(bars);
  constexpr int S = C::kSlots;
  auto kfull = [&](int s) { return bar0 + 8u * s; };
  auto kempty = [&](int s) { return bar0 + 8u * (S + s); };
  auto vfull = [&](int s) { return bar0 + 8u * (2 * S + s); };
  auto vempty = [&](int s) { return bar0 + 8u * (3 * S + s); };
  // the queries of half h are in place; every S_h of the segment is done
  auto qfull = [&](int h) { return bar0 + 8u * (h ? 4 * S + 27 : 4 * S); };
  auto qempty = [&](int h) { return bar0 + 8u * (h ? 4 * S + 28 : 4 * S + 1); };
  auto sfull = [&](int h) { return bar0 + 8u * (4 * S + 2 + h); };  // S_h landed
  // the first (second) 64 keys of P_h are written; P V of the first 64 is done
  auto pfull = [&](int h, int part) { return bar0 + 8u * (4 * S + (part ? 15 : 4) + h); };
  auto pvdone = [&](int h) { return bar0 + 8u * (4 * S + 17 + h); };
  auto ofull = [&](int h) { return bar0 + 8u * (4 * S + 6 + h); };  // O_h of the segment done
  auto ofree = [&](int h) { return bar0 + 8u * (4 * S + 8 + h); };  // O_h read
  // codes of a tile landed / read; t = 0: K, 1: V
  auto rfull = [&](int t) { return bar0 + 8u * (4 * S + 10 + t); };
  auto rempty = [&](int t) { return bar0 + 8u * (4 * S + 12 + t); };
  const uint32_t done_bar = bar0 + 8u * (4 * S + 14);
  // whose turn it is: softmax warps q4 of the two halves (they share a scheduler)
  auto turn = [&](int h, int q4) { return bar0 + 8u * (4 * S + 19 + 4 * h + q4); };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::kBarCount);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 8; ++i) mbar_init(turn(i >> 2, i & 3), 1);
    for (int s = 0; s < S; ++s) {
      mbar_init(kfull(s), 4);
      mbar_init(kempty(s), 2);
      mbar_init(vfull(s), 4);
      mbar_init(vempty(s), 2);
    }
    for (int h = 0; h < 2; ++h) {
      mbar_init(qfull(h), 4);
      mbar_init(qempty(h), 1);
      mbar_init(sfull(h), 1);
      mbar_init(pfull(h, 0), 4);
      mbar_init(pfull(h, 1), 4);
      mbar_init(pvdone(h), 1);
      mbar_init(ofull(h), 1);
      mbar_init(ofree(h), 4);
      mbar_init(rfull(h), 1);
      mbar_init(rempty(h), 4);
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
  const uint32_t total = fs.n[blockIdx.x].x;  // tiles of this CTA
  const int gm = (65536 + p.G - 1) / p.G;
  if (warp >= 12) {
    reg_dec<C::kIssuerRegs>();
    const int me = warp - 12;
    if (me < 2) {
      // ---------------------------------------------------------- MMA issuers
      // The whole warp walks the tiles, so that addresses and descriptors stay
      // in uniform registers; one lane issues and commits.  A wait that runs out
      // ends the loop for all lanes at once (warp_wait_idle): lanes that went
      // apart would meet at different barriers.
      constexpr uint32_t idesc_s = idesc_f16_f32(128, 128, false);
      constexpr uint32_t idesc_o = idesc_f16_f32(128, D, true);
      constexpr uint64_t kStep = C::kTileBytes >> 4;  // next buffer, in the address field
      const uint64_t qd = smem_desc(qbuf(me), 16, G::kGroupBytes, G::kLayout);
      const uint64_t kd = smem_desc(kbuf(0), 16, G::kGroupBytes, G::kLayout);
      const uint64_t vd = smem_desc(vbuf(0), G::kAtomTileBytes, G::kGroupBytes, G::kLayout);
      const uint32_t ts = tmem + me * 128, to = tmem + C::kAccO + me * D;
      const bool lead = elect_one();
      uint32_t seg = 0, flags = 0;
      auto issue_s = [&](uint32_t k) {  // S of tile k of this CTA
        if (!warp_wait_idle(kfull(k & 1u), (k >> 1) & 1u, abort, kCode)) return false;
        flags = *reinterpret_cast<volatile uint32_t*>(&s_info[k & kRing].flags);
        if ((flags & kTileFirst) && !warp_wait_idle(qfull(me), seg & 1u, abort, kCode)) return false;
        tc_fence_after();
        const uint64_t b0 = kd + (k & 1u) * kStep;
        if (lead) {
#pragma unroll
          for (uint32_t kk = 0; kk < D / 16; ++kk) {
            const uint64_t off = ((kk / KPA) * G::kAtomTileBytes + (kk % KPA) * 32) >> 4;
            mma_bf16(ts, qd + off, b0 + off, idesc_s, kk);
          }
          mma_commit(sfull(me));
          mma_commit(kempty(k & 1u));
          if (flags & kTileLast) mma_commit(qempty(me));  // every S of the segment has been issued
        }
        __syncwarp();
        return true;
      };
      bool ok = total > 0 && issue_s(0);
      for (uint32_t n = 0; n < total && ok; ++n) {
        const uint32_t now = flags;  // of tile n
        if (((now & kTileFirst) && !warp_wait_idle(ofree(me), (seg & 1u) ^ 1u, abort, kCode)) ||
            !warp_wait_idle(vfull(n & 1u), (n >> 1) & 1u, abort, kCode) ||
            !warp_wait_idle(pfull(me, 0), n & 1u, abort, kCode))
          break;
        tc_fence_after();
        const uint64_t b0 = vd + (n & 1u) * kStep;
        const uint32_t keep = (now & kTileFirst) ? 0u : 1u;  // add to O, or begin it
        if (lead) {
#pragma unroll
          for (uint32_t kk = 0; kk < 4; ++kk)  // 16 keys = 8 columns of P
            mma_bf16_ts(to, ts + kk * 8, b0 + kk * (2 * G::kGroupBytes >> 4), idesc_o, kk | keep);
          mma_commit(pvdone(me));
        }
        __syncwarp();
        if (!warp_wait_idle(pfull(me, 1), n & 1u, abort, kCode)) break;
        tc_fence_after();
        if (lead) {
#pragma unroll
          for (uint32_t kk = 4; kk < 8; ++kk)
            mma_bf16_ts(to, ts + kk * 8, b0 + kk * (2 * G::kGroupBytes >> 4), idesc_o, 1u);
          mma_commit(vempty(n & 1u));
          if (now & kTileLast) mma_commit(ofull(me));
        }
        __syncwarp();
        if (now & kTileLast) ++seg;
        if (n + 1 < total) ok = issue_s(n + 1);
      }
      __syncwarp();
      if (lead) mma_commit(done_bar);
      mbar_wait_drain(done_bar, 0);
    } else if (me == 2) {
      // ------------------------------------------------------------- producer
      const int P = 1 << p.p_shift;
      const int64_t page_bytes = (static_cast<int64_t>(p.Hkv) << p.p_shift) * D;
      const uint32_t chunk = static_cast<uint32_t>(D) << p.p_shift;  // one page of one head
      const int copies = 128 >> p.p_shift, per = P >> 4;  // pages of a tile, groups of a page
      uint32_t n = 0, seg = 0, issued = 0;  // copies of K and V tiles begun
      // gla_inject_stall (testing): CTA 0 withholds one tile, once
      long long stall = -1;
      if (blockIdx.x == 0) {
        stall = *const_cast<volatile long long*>(&g_gla_stall_tile);
        __syncwarp();
        if (lane == 0 && stall >= 0) g_gla_stall_tile = -1;
      }
      bool ok = true;
      FrameCursor cur;
      for (cur.init(p, fs); cur.live && ok; cur.next(p, fs), ++seg) {
        const int* row = p.table + static_cast<int64_t>(cur.r) * p.max_pages;
        for (int t = cur.t0; t < cur.t1 && ok; ++t, ++n) {
          const int base = cur.v.pos(t, C::BK);
          const int a = base + 16 * (lane & 7);  // lanes 8 .. repeat lanes 0 .. 7
          const int j = a >> p.p_shift;
          const bool vis = a < cur.v.hi && (a + 16 > cur.v.lo || a < cur.v.sink);
          int pg = vis && j < p.max_pages ? row[j] : -1;
          if (pg >= p.pages) pg = -1;
          float ks = 0.f, vs = 0.f;
          if (pg >= 0) {
            const int64_t x = static_cast<int64_t>(pg) * p.Hkv + cur.h;
            ks = p.ks[x];
            vs = p.vs[x];
          }
          // positive floats order like their bits
          float kt = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(ks)));
          float vt = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(vs)));
          if (!(kt > 0.f)) kt = 1.f;
          if (!(vt > 0.f)) vt = 1.f;
          const uint32_t bad = __ballot_sync(0xffffffffu, vis && pg < 0) & 255u;
          const uint32_t scale_k = __any_sync(0xffffffffu, pg >= 0 && ks != kt) ? kTileScaleK : 0u;
          const uint32_t scale_v = __any_sync(0xffffffffu, pg >= 0 && vs != vt) ? kTileScaleV : 0u;
          const bool all = base + C::BK <= cur.v.sink ||
                           (base >= cur.v.lo && base + C::BK <= cur.v.hi);
          // Safe to write: raw codes of tile n - 2 have been read, after the
          // converters saw S of tile n - 4 complete; so every softmax warp is
          // past tile n - 5 (and past the segments that ended there).
          TileInfo& info = s_info[n & kRing];
          if (t == cur.t0 && lane == 0) {
            const int t_unit = cur.i * 2 * fs.TQ;
            SegInfo& si = s_seg[seg & kRing];
            si.row0 = (static_cast<long long>(cur.s.c0) + t_unit) * p.H + cur.h * p.G;
            si.tokens = cur.s.n - t_unit;
            si.p0 = cur.s.p0 + t_unit;
            si.len = cur.s.len;
            si.lo = cur.v.lo;
            si.hi = cur.v.hi;
            si.sink = cur.v.sink;
            si.whole = cur.t0 == 0 && cur.t1 == cur.v.nb;
            si.starts = cur.t0 == 0;
            si.c0 = cur.s.c0;
            si.t_unit = t_unit;
            si.h = cur.h;
          }
          // one page's share of the tile, by lane: the page of its first visible group
          const uint32_t groups =
              __ballot_sync(0xffffffffu, pg >= 0) & 255u & (((1u << per) - 1u) << (lane * per & 31));
          const int use = __shfl_sync(0xffffffffu, pg, groups ? __ffs(groups) - 1 : 0);
          const bool mine = lane < copies && groups != 0;
          const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, mine)) * chunk;
          if (lane < 8) {
            const __half2 kf = __float2half2_rn(ks * (1.0f / kt)), vf = __float2half2_rn(vs * (1.0f / vt));
            info.kfac[lane] = *reinterpret_cast<const uint32_t*>(&kf);
            info.vfac[lane] = *reinterpret_cast<const uint32_t*>(&vf);
            if (lane == 0) {
              const float lv = lg2_approx(vt);
              info.ks = kt;
              info.lv = lv;
              info.iv = ex2_approx(-lv);
              info.flags = bad | (all ? kTileAll : 0u) | scale_k | scale_v |
                           (t == cur.t0 ? kTileFirst : 0u) | (t + 1 == cur.t1 ? kTileLast : 0u);
              info.base = base;
            }
          }
          __syncwarp();
          const int64_t off = (mine ? use : 0) * page_bytes + static_cast<int64_t>(cur.h) * chunk;
#pragma unroll 1
          for (int w = 0; w < 2; ++w) {
            if (!warp_wait_idle(rempty(w), (n & 1u) ^ 1u, abort, kCode)) {
              ok = false;
              break;
            }
            if (n == stall) continue;  // nothing arrives on rfull for this tile
            if (lane == 0) mbar_arrive_expect_tx(rfull(w), bytes);
            __syncwarp();
            ++issued;
            if (mine)
              bulk_load((w ? vraw : kraw) + lane * chunk, (w ? p.v8 : p.k8) + off, chunk,
                        rfull(w));
          }
        }
      }
      // copies in flight land before the CTA ends
      if (issued > 0) mbar_wait_drain(rfull(0), ((issued + 1) / 2 - 1) & 1u);
      if (issued > 1) mbar_wait_drain(rfull(1), (issued / 2 - 1) & 1u);
    }
  } else if (warp >= 8) {
    // ------------------------------------------------------------- converters
    reg_dec<C::kConverterRegs>();
    const int ct = threadIdx.x - 256;
    const int ch = ct % kRowChunks, row0 = ct / kRowChunks;
    const int c2 = (ch * 2) & 7;  // first 16-byte fp16 chunk within its 128-byte atom row
    const uint32_t atom = static_cast<uint32_t>(ch * 2 / 8) * G::kAtomTileBytes;
    const bool swap = (ch & 4) != 0;  // these lanes write their two chunks in the other order
                                      // (bank conflicts)
    // ---- queries of segment `seg`: all rows are copied to their places as bf16
    // at once, then each thread turns its own chunks into fp16 in place, scaled
    // per row.  The scores of the unit wait for this: four copies and kBatch rows
    // are in work at a time (row by row it took 17 thousand cycles at d = 128).
    auto convert_q = [&](uint32_t seg, int hf) {
      constexpr int kQChunks = D / 8, kQRows = 128 / kQChunks;
      constexpr int kPerHalf = 128 / kQRows, kBatch = 8;
      static_assert(kQRows % 8 == 0 && kPerHalf % kBatch == 0, "one swizzle for all rows of a thread");
      if (!warp_wait_idle(qempty(hf), (seg & 1u) ^ 1u, abort, kCode)) return false;
      const SegInfo& si = s_seg[seg & kRing];
      const int qc = ct % kQChunks, qr0 = ct / kQChunks;
      const __nv_bfloat16* qp = p.q + si.row0 * D + qc * 8;
      const int tokens = si.tokens;
      const uint32_t place = qbuf(hf) + (qc >> 3) * G::kAtomTileBytes + qr0 * 128 +
                             (((qc & 7) ^ (qr0 & 7)) << 4);
#pragma unroll 4
      for (int i = 0; i < kPerHalf; ++i) {
        const int lr = qr0 + i * kQRows;
        const int lt = small_div(lr, gm);
        const int t = hf * fs.TQ + lt;
        const bool have = lr < used && t < tokens;
        const int at = have ? t * p.H + (lr - lt * p.G) : 0;  // below 2^25
        cp_async16(place + i * (kQRows * 128), qp + static_cast<int64_t>(at) * D, have);
      }
      cp_async_commit();
      cp_async_wait<0>();
#pragma unroll 1
      for (int i = 0; i < kPerHalf; i += kBatch) {
        const uint32_t at = place + i * (kQRows * 128);
        uint4 x[kBatch];
        uint32_t mx[kBatch];
#pragma unroll
        for (int e = 0; e < kBatch; ++e) x[e] = ld_shared_v4(at + e * (kQRows * 128));
#pragma unroll
        for (int e = 0; e < kBatch; ++e) {
          mx[e] = __vmaxu2(__vmaxu2(x[e].x & 0x7FFF7FFFu, x[e].y & 0x7FFF7FFFu),
                           __vmaxu2(x[e].z & 0x7FFF7FFFu, x[e].w & 0x7FFF7FFFu));
        }
#pragma unroll
        for (int o = kQChunks / 2; o > 0; o >>= 1)
#pragma unroll
          for (int e = 0; e < kBatch; ++e)
            mx[e] = __vmaxu2(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], o));
#pragma unroll
        for (int e = 0; e < kBatch; ++e) {
          const int up = row_exponent(max(mx[e] & 0xFFFFu, mx[e] >> 16));
          const float f = exp2_int(up);
          uint4 w;
          w.x = pack_f16x2(bf16lo_to_f32(x[e].x) * f, bf16hi_to_f32(x[e].x) * f);
          w.y = pack_f16x2(bf16lo_to_f32(x[e].y) * f, bf16hi_to_f32(x[e].y) * f);
          w.z = pack_f16x2(bf16lo_to_f32(x[e].z) * f, bf16hi_to_f32(x[e].z) * f);
          w.w = pack_f16x2(bf16lo_to_f32(x[e].w) * f, bf16hi_to_f32(x[e].w) * f);
          st_shared_v4(at + e * (kQRows * 128), w);
          if (qc == 0)
            s_rs[(seg & 1u) * C::kRows + hf * 128 + qr0 + (i + e) * kQRows] = static_cast<int8_t>(up);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(qfull(hf));
      return true;
    };
    uint32_t seg = 0;
    bool ok = true;
    for (uint32_t n = 0; n < total && ok; ++n) {
      const int sl = n & 1u;
      const TileInfo& info = s_info[n & kRing];
      // queries of half 0, K, V, queries of half 1 (whose scores come later): one
      // copy of the code
#pragma unroll 1
      for (int w = 0; w < 3; ++w) {
        if (w < 2 && !warp_wait_idle(rfull(w), n & 1u, abort, kCode)) {
          ok = false;
          break;
        }
        const uint32_t flags = *const_cast<volatile const uint32_t*>(&info.flags);
        if (w != 1 && (flags & kTileFirst) && !convert_q(seg, w >> 1)) {
          ok = false;
          break;
        }
        if (w == 2) {
          if (flags & kTileLast) ++seg;
          break;
        }
        uint4 x[kPasses];
        const uint32_t raw = (w ? vraw : kraw) + ct * 16;
#pragma unroll
        for (int i = 0; i < kPasses; ++i) x[i] = ld_shared_v4(raw + i * 2048);
        if ((flags & (kTileBad | kTileAll)) != kTileAll) {
          // uniform: keys that no row sees, or whose page is missing
          const SegInfo& si = s_seg[seg & kRing];
          const int key0 = info.base + row0, lo = si.lo, hi = si.hi, sink = si.sink;
#pragma unroll
          for (int i = 0; i < kPasses; ++i)
            if (!(key0 + i * kRowsPerPass < hi &&
                  (key0 + i * kRowsPerPass >= lo || key0 + i * kRowsPerPass < sink)) ||
                (flags >> (kRowsPerPass > 16 ? 2 * i + (row0 >> 4) : i) & 1))
              x[i] = make_uint4(0, 0, 0, 0);
        }
        if (!warp_wait_idle(w ? vempty(sl) : kempty(sl), ((n >> 1) & 1u) ^ 1u, abort, kCode)) {
          ok = false;
          break;
        }
        const uint32_t buf = (w ? vbuf(sl) : kbuf(sl)) + atom;
        const bool scaled = flags & (w ? kTileScaleV : kTileScaleK);  // uniform
        const uint32_t* fac = w ? info.vfac : info.kfac;
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
          const int kr = i * kRowsPerPass + row0;
          uint32_t y[8];
          const uint32_t c[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
          for (int e = 0; e < 8; ++e)
            y[e] = e4m3x2_to_f16x2((e & 1) ? c[e >> 1] >> 16 : c[e >> 1] & 0xFFFFu);
          if (scaled) {
            const uint32_t fw = fac[kRowsPerPass > 16 ? 2 * i + (row0 >> 4) : i];
            const __half2 f = *reinterpret_cast<const __half2*>(&fw);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const __half2 v = __hmul2(*reinterpret_cast<const __half2*>(&y[e]), f);
              y[e] = *reinterpret_cast<const uint32_t*>(&v);
            }
          }
          const uint32_t pa = buf + kr * 128 + ((c2 ^ (kr & 7)) << 4);
          const uint32_t pb = buf + kr * 128 + (((c2 + 1) ^ (kr & 7)) << 4);
          const uint4 lo = make_uint4(y[0], y[1], y[2], y[3]);
          const uint4 hi = make_uint4(y[4], y[5], y[6], y[7]);
          st_shared_v4(swap ? pb : pa, swap ? hi : lo);
          st_shared_v4(swap ? pa : pb, swap ? lo : hi);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(w ? vfull(sl) : kfull(sl));
          mbar_arrive(rempty(w));  // every code has been used: no load of one is outstanding
        }
      }
    }
  } else {
    // -------------------------------------------------- softmax and epilogue
    reg_inc<C::kSoftmaxRegs>();
    const int half = warp >> 2, q4 = warp & 3;
    const int row = q4 * 32 + lane;  // row of the half
    const int row_t = small_div(row, gm), row_g = row - row_t * p.G;
    const uint32_t lane_base = static_cast<uint32_t>(q4 * 32) << 16;
    const uint32_t ts = tmem + lane_base + half * 128;
    const uint32_t to = tmem + lane_base + C::kAccO + half * D;
    uint32_t seg = 0;
    int hi = 0, lo = 0;
    float rs = 0.f, m = -INFINITY, l = 0.f;
    bool unset = true;  // some row of the warp has no reference yet
    for (uint32_t n = 0; n < total; ++n) {
      if (!warp_wait_idle(sfull(half), n & 1u, abort, kCode)) break;
      tc_fence_after();
      uint32_t s[2][32];  // 32 keys in work, the next 32 on their way
      tmem_ld_32cols(ts, s[0]);
      const float4 info = ld_shared_f4(smem_u32(&s_info[n & kRing].ks));
      const int base = *const_cast<volatile int*>(&s_info[n & kRing].base);
      const uint32_t flags = __float_as_uint(info.w);
      {
        if (flags & kTileFirst) {
          const SegInfo& si = s_seg[seg & kRing];
          const int t = half * fs.TQ + row_t;
          const bool have = row < used && t < si.tokens;
          CacheSeq s;
          s.len = si.len;
          // rows that hold no query see everything: they cost no mask
          hi = have ? key_hi(p, s, si.p0 + t) : INT32_MAX;
          lo = have ? key_lo(p, si.p0 + t) : 0;
          // the row scales of segment seg are written before its first S and
          // replaced after the last P of segment seg + 1
          rs = exp2_int(-s_rs[(seg & 1u) * C::kRows + half * 128 + row]) * p.sl2;
          m = -INFINITY;
          l = 0.f;
          unset = true;
        }
        const uint32_t bad = flags & kTileBad;
        if (!__all_sync(0xffffffffu, base >= lo && base + C::BK <= hi && bad == 0)) {
          // hidden keys: S = -inf, written back, in a pass of its own (few tiles
          // need it, and inside the loops below its code would be fetched with
          // theirs); 32 keys that all rows see are left alone
          tmem_wait_ld_of(s[0]);  // the load on its way is taken again below
#pragma unroll 1
          for (int g = 0; g < 4; ++g) {
            uint32_t w = visible_bits(base + g * 32, lo, hi, p.n_sink);
            if (bad >> (2 * g) & 1u) w &= 0xFFFF0000u;
            if (bad >> (2 * g) & 2u) w &= 0x0000FFFFu;
            if (__all_sync(0xffffffffu, w == 0xFFFFFFFFu)) continue;
            if (__any_sync(0xffffffffu, w != 0)) {
              tmem_ld_32cols(ts + g * 32, s[0]);
              tmem_wait_ld_of(s[0]);
            }
#pragma unroll
            for (int e = 0; e < 32; ++e)
              s[0][e] = (w >> e & 1u) ? s[0][e] : __float_as_uint(-INFINITY);
            tmem_st_32cols(ts + g * 32, s[0]);
          }
          tmem_wait_st();
          tmem_ld_32cols(ts, s[0]);
        }
        // never 0, for the mask's -inf: a tiny row on keys that are all 0 (2^-126 of
        // a score is nothing either way)
        const float fg = fmaxf(rs * info.x, 1.1754944e-38f);
        const uint64_t f2 = f2_pack(fg, fg);
        float tsum = 0.f;
        bool gave_up = C::kTurns && !warp_wait_idle(turn(half, q4), half == 0 ? (n & 1u) ^ 1u : n & 1u,
                                                    abort, kCode);
        if (gave_up) break;
#pragma unroll 1
        for (int hb = 0; hb < 2; ++hb) {  // 64 keys at a time: their P' stays in 32 registers
          bool need = unset;  // take the maximum first
          uint32_t pw[32];
          float hsum;
          bool passed = false;
          for (;;) {
            if (need) {
              tmem_wait_ld_of(s[0]);  // the load on its way is taken again below
              float mt = -INFINITY;
#pragma unroll 1
              for (int c = 2 * hb; c < 2 * hb + 2; ++c) {
                tmem_ld_32cols(ts + c * 32, s[0]);
                tmem_wait_ld_of(s[0]);
                float mx[4] = {mt, mt, mt, mt};
#pragma unroll
                for (int e = 0; e < 32; e += 2)
                  mx[(e >> 1) & 3] = fmax3(mx[(e >> 1) & 3], __uint_as_float(s[0][e]),
                                           __uint_as_float(s[0][e + 1]));
                mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
              }
              const float x = fmaf(mt, fg, info.y);
              // whole steps: the factor is a power of two, exact for O
              const float mn = m == -INFINITY ? x : m + ceilf(fmaxf(x - m, 0.f));
              const float f = m == -INFINITY ? 0.f : ex2_approx(m - mn);
              l *= f;
              tsum *= f;
              m = mn;
              unset = __any_sync(0xffffffffu, m == -INFINITY);
              // O of the previous tiles is complete: S of this tile was issued
              // after the last P V by the same thread; the first 64 keys of
              // this tile may be in work still
              if (hb == 1 && !warp_wait_idle(pvdone(half), n & 1u, abort, kCode)) {
                gave_up = true;
                break;
              }
              if (hb == 1 || !(flags & kTileFirst)) {
                tc_fence_after();
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                  tmem_ld_32cols(to + c * 32, s[0]);
                  tmem_wait_ld_of(s[0]);
#pragma unroll
                  for (int e = 0; e < 32; ++e)
                    s[0][e] = __float_as_uint(__uint_as_float(s[0][e]) * f);
                  tmem_st_32cols(to + c * 32, s[0]);
                }
                tmem_wait_st();
              }
              tmem_ld_32cols(ts + hb * 64, s[0]);
            }
            const float sg = m == -INFINITY ? 0.f : info.y + (kCacheBias - m);
            const uint64_t s2 = f2_pack(sg, sg);
            uint64_t sum[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[e] = f2_pack(0.f, 0.f);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              tmem_wait_ld_of(s[c]);
              if (c == 0)
                tmem_ld_32cols(ts + hb * 64 + 32, s[1]);
              else if (hb == 0)
                tmem_ld_32cols(ts + 64, s[0]);
              if (C::kTurns && c == 1 && hb == 1 && !passed) {
                // the last 32 keys: the other half may begin (measured 2% better
                // than at the end)
                passed = true;
                if (lane == 0) mbar_arrive(turn(half ^ 1, q4));
              }
              uint32_t(&x)[32] = s[c];
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                float a0, a1, y0, y1;
                f2_unpack(f2_fma(f2_pack(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])),
                                 f2, s2),
                          a0, a1);
                if (!C::kTurns && (e & 3) == 0) {
                  exp2_poly3_any_x2(a0, a1, y0, y1);
                } else {
                  y0 = ex2_approx(a0);
                  y1 = ex2_approx(a1);
                }
                sum[e & 3] = f2_add(sum[e & 3], f2_pack(y0, y1));
                pw[c * 16 + e] = pack_f16x2(y0, y1);
              }
            }
            float l0, l1;
            f2_unpack(f2_add(f2_add(sum[0], sum[1]), f2_add(sum[2], sum[3])), l0, l1);
            hsum = l0 + l1;
            // every P' is at most the sum: below 2^15 all of them are fp16 numbers
            if (need || __all_sync(0xffffffffu, hsum < 32768.0f)) break;
            need = true;  // once: then P' is at most 2^kCacheBias
          }
          if (gave_up) break;
          tmem_st_32cols(ts + hb * 32, pw);
          tsum += hsum;
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(pfull(half, hb));
        }
        if (gave_up) break;
        l = fmaf(tsum, info.z, l);
      }
      if (!(flags & kTileLast)) continue;
      // ---- the segment's result: out, or a partial when the unit goes on elsewhere
      const SegInfo& si = s_seg[seg & kRing];
      const int t = half * fs.TQ + row_t;
      const bool have = row < used && t < si.tokens;
      const bool whole = si.whole;
      const int64_t at = have ? (si.row0 + static_cast<int64_t>(t) * p.H + row_g) * D : 0;
      const bool gate = have && whole && p.z != nullptr;
      const uint4* zp = reinterpret_cast<const uint4*>(p.z + at);
      if (!warp_wait_idle(ofull(half), seg & 1u, abort, kCode)) break;
      tc_fence_after();
      const float rl = m == -INFINITY ? 0.f : 1.0f / l;
      float* part = p.part + (2ll * blockIdx.x + (si.starts ? 1 : 0)) * C::kPartFloats;
#pragma unroll 1
      for (int c = 0; c < D / 16; ++c) {
        uint32_t zz[8];
        if (gate) {
          const uint4 z0 = __ldg(zp + c * 2), z1 = __ldg(zp + c * 2 + 1);
          zz[0] = z0.x, zz[1] = z0.y, zz[2] = z0.z, zz[3] = z0.w;
          zz[4] = z1.x, zz[5] = z1.y, zz[6] = z1.z, zz[7] = z1.w;
        }
        uint32_t o[16];
        tmem_ld_16cols(to + c * 16, o);
        tmem_wait_ld_of(o);
        if (whole) {
          uint32_t w[8];
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            float x0 = __uint_as_float(o[2 * q]) * rl, x1 = __uint_as_float(o[2 * q + 1]) * rl;
            if (gate) {
              x0 = __fdividef(x0, 1.0f + __expf(-bf16lo_to_f32(zz[q])));
              x1 = __fdividef(x1, 1.0f + __expf(-bf16hi_to_f32(zz[q])));
            }
            w[q] = pack_bf16x2(x0, x1);
          }
          if (have) {  // rows are 16-byte aligned, not always 32
            uint4* op = reinterpret_cast<uint4*>(p.out + at + c * 16);
            if ((reinterpret_cast<uintptr_t>(op) & 31) == 0) {
              st_global_v8(op, w);
            } else {
              op[0] = make_uint4(w[0], w[1], w[2], w[3]);
              op[1] = make_uint4(w[4], w[5], w[6], w[7]);
            }
          }
        } else if (have) {
          // (rows that saw no key in this part hold zeros)
          float* dst = part + (half * 128 + row) * D + c * 16;
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const uint32_t v[8] = {o[8 * q],     o[8 * q + 1], o[8 * q + 2], o[8 * q + 3],
                                   o[8 * q + 4], o[8 * q + 5], o[8 * q + 6], o[8 * q + 7]};
            st_global_v8(dst + q * 8, v);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(ofree(half));
      if (!whole)
        *reinterpret_cast<float2*>(part + C::kRows * D + 2 * (half * 128 + row)) =
            make_float2(m, l);
      if (threadIdx.x == 0 && si.starts && !whole) {
        // this unit's parts: this CTA, then every one up to the last tile
        int* desc = p.desc + 8 * blockIdx.x;
        desc[1] = si.c0;
        desc[2] = si.t_unit;
        desc[3] = si.h;
        desc[4] = min(2 * fs.TQ, si.tokens) * p.G;
        desc[0] = fs.n[blockIdx.x].y;
      }
      ++seg;
    }
    __syncwarp();
    tmem_wait_ld();  // a load on its way when a wait ran out
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the partials of a unit that several CTAs share, one warp a row: unit and
// parts as in gla_cache_combine_kernel, which spends a block on a row (measured
// over 148 split units of 256 rows: 33 us).  32 parts at a time: each lane takes
// one part's (m, l), the weights go round by shuffle.
constexpr int kJoinBlocks = 16;  // blocks a unit, four warps each

template <int D>
__global__ void __launch_bounds__(128)
    gla_cache_join_kernel(const CacheAttnParams p, int used) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  using C = FrameCfg<D>;
  constexpr int V = D / 32;  // columns of a lane
  // (the partials are read past L1: this grid may have started before they were
  // written)
  const int4 d0 = __ldcg(reinterpret_cast<const int4*>(p.desc + 8 * blockIdx.x));
  const int parts = d0.x, c0 = d0.y, t_unit = d0.z, h = d0.w;
  if (parts == 0) return;
  const int rows = __ldcg(p.desc + 8 * blockIdx.x + 4);
  const int lane = threadIdx.x & 31;
  const int first = blockIdx.y * 4 + (threadIdx.x >> 5);
  auto part_of = [&](int i) {
    return p.part +
           (i == 0 ? 2ll * blockIdx.x + 1 : 2ll * (blockIdx.x + i)) * C::kPartFloats;
  };
  for (int r = first; r < rows; r += kJoinBlocks * 4) {
    const int rho = r < used ? r : 128 + (r - used);  // row of the partial
    float m = -INFINITY, l = 0.f, acc[V] = {};
    for (int i0 = 0; i0 < parts; i0 += 32) {
      float2 ml = make_float2(-INFINITY, 0.f);
      if (i0 + lane < parts)
        ml = __ldcg(reinterpret_cast<const float2*>(part_of(i0 + lane) + C::kRows * D + 2 * rho));
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
      const int n = min(32, parts - i0);
#pragma unroll 4
      for (int i = 0; i < n; ++i) {
        const float wi = __shfl_sync(0xffffffffu, w, i);
        const float* x = part_of(i0 + i) + rho * D + lane * V;
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
    const float rl = m == -INFINITY ? 0.f : 1.0f / l;
    const int64_t off =
        ((static_cast<int64_t>(c0) + t_unit + r / p.G) * p.H + h * p.G + r % p.G) * D + lane * V;
#pragma unroll
    for (int v = 0; v < V; v += 2) {
      float x0 = acc[v] * rl, x1 = acc[v + 1] * rl;
      if (p.z != nullptr) {
        const uint32_t z = *reinterpret_cast<const uint32_t*>(p.z + off + v);
        x0 *= 1.0f / (1.0f + __expf(-bf16lo_to_f32(z)));
        x1 *= 1.0f / (1.0f + __expf(-bf16hi_to_f32(z)));
      }
      *reinterpret_cast<uint32_t*>(p.out + off + v) = pack_bf16x2(x0, x1);
    }
  }
}

}  // namespace gla
