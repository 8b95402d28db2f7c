// Paged attention of many query rows a KV head (chunks, prompts, drafts of
// wide groups) on the tcgen05 tensor cores: D 64 or 128, groups of 32, 4- or
// 8-bit codes, bf16 rows.
//
// An item (paged.cuh) is up to two tiles of 128 query rows of one sequence,
// token-major with the KV head's G query heads side by side: a tile holds
// floor(128 / G) tokens, fetched by one 4-D TMA copy per 64 features (feature,
// head of the group, KV head, token).  Per block of 128 keys the packed bytes
// come page by page, are decoded -- (code - qmax) * scale, rounded once to
// fp16 -- into shared-memory tiles, S = Q K^T goes to tensor memory (TMEM),
// the softmax turns S into P (fp16) in place and O += P V accumulates in TMEM.
//
// fp16, not bf16: rounding K to eight bits moved the scores of long contexts so
// far that the rows were 0.8 % of their norm off; with eleven they are 0.19 %,
// nearly all of it the output's own bf16 rounding.  Its range is the price: a
// kernel before this one finds the largest and the smallest K and V scale of each
// sequence and KV head and turns the query rows to fp16 (powers of two below), 6
// to 18 us.
//
// What bounds it: at 128 rows a block costs 4 * 128 * D * 128 FLOPs for 160
// (288) bytes a key at D = 128, so the tensor pipe and not memory; 4 x 64 rows
// of 4 heads over 16384 keys take 108 us, 635 TFLOP/s, 40 % of the measured bf16
// rate.  The MMAs alone would take 2.6k cycles a block of two tiles.  A block
// takes about 4.9k: V is decoded (2.0 to 2.5k), then P V of the first tile, Q K of
// its next block and P V of the second run before V's tile is free again, while
// the two softmaxes (3k each) and K's decode run beside that chain.  So two row
// tiles are in flight, and a lone tile has its scores twice: the next block's are
// there before this one's values (24 x 40 rows: 133 -> 119 us at the time, 120 now).
//
// The kernel's size counts as well: roles that run side by side share the
// instruction cache, and at 130 KB of code instead of 70 everything took a
// quarter longer.  Each step has one site; waits and segment changes are short.
//
// Causal rows: a column past a row's position takes no part in its maximum and
// its p is zero.  A *value* that is not finite would still reach such a row
// through 0 * inf, so its scale is taken as zero in the tile and the token is
// remembered with the scale's 32 features: there, rows that do see it become NaN at
// the segment's end.
//
// The softmax reads S twice (its maximum, then p): a read of 32 columns takes
// about 70 cycles, a vote and a branch per 32 columns in a single pass took four
// times that.  Its reference maximum is lazy: it moves, and O and z are rescaled,
// only when a block's maximum outruns it by more than 8 in log2 units.  Any
// reference that never falls more than that below the running maximum gives
// the same u / z in exact arithmetic.
//
// Warp roles (20 warps, 96 registers each):
//   0        producer: two lanes copy 32 keys each (codes and scales) of half a
//            K or V block into a ring; order K(0), K(1), V(0), K(2), ...
//   1        MMA issuer (the warp runs converged, one lane issues) and TMEM owner
//   2        Q loader; leaves a segment's powers to the others
//   3        finds the CTA's form, which says what bodies 4..19 run
//   4..7     softmax of tile 0 (a thread a row), 8..11 of tile 1
//   12..19   decode: warp w converts 16 keys of each block, warps 12..15 from
//            its first half-unit, 16..19 from its second
// K tiles are double, V has one: a second V tile leaves 27 KB for the ring, and
// the copies' latency then costs more than the wait for V's turn (in bf16, ring of
// 59 KB and one V tile: 104 us for 4 x 64 rows over 16384 keys; 27 KB and two:
// 107; at 8 bits, prompts: 348 against 369 us).  63 KB are no faster than 55.
// TMEM columns: S/P of tile t at [128 t, +128), O at [256 + 128 t, +D).
// Shared-memory tiles use the 128-byte-swizzled UMMA layout of tc_common.cuh.
#include <cuda.h>

#include <algorithm>
#include <type_traits>

#include "f32x2.cuh"
#include "paged.cuh"
#include "tc_common.cuh"

namespace kvq {
namespace paged {
namespace {

using namespace tc;

constexpr int kBT = 128;
constexpr int kThreads = 640;
constexpr int kDecodeWarps = 8;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLazy = 8.f;
constexpr int kTileHalf = kBT * 128;              // 16 KB: 128 rows x 64 fp16
constexpr int kMaxUnits = 12;                    // half-units of the ring

// Powers of two that keep the fp16 tiles in range.  A query row is multiplied by
// 2^(kTopQ - e) of its own, e the exponent of its largest element.  For K and V
// there are two forms, chosen for a segment by its sequence's and KV head's scales:
//
//   narrow  the largest K (V) scale is at most 2^kSpread times the smallest: the
//           tiles hold (code - qmax) * scale * 2^(kTop - e), e the exponent of the
//           largest.  That is below 2^15 (the scale is below 2^(e + 1), the code
//           at most 2^7 away from zero), and a code of one times the smallest scale
//           is a normal fp16 number, so nothing but the power depends on it.
//   wide    a key's row of K (of V) is multiplied by 2^(kTopQ - e_t) of its own
//           largest value, as query rows are.  The decode warps leave the powers in
//           shared memory; a column's score is multiplied by K's, and V's exponent
//           joins the weight: with w_t = (s_t - m) + e_t (log2 units, m the score's
//           reference), p'_t = 2^(w_t - R) for a row's own lazy reference R of w
//           (it follows m), z sums p_t = 2^(s_t - m) as always, and O = sum p'_t
//           (v_t 2^(kTopQ - e_t)) 2^(R - kTopQ) / z.
//           So a key that a row does not see changes nothing of the row's, a group
//           of zeros (whose scale is 1) is a group of zeros, and what is lost is
//           what float32 sums lose too: contributions below 2^-21 of the largest.
//           Its softmax waits for V's tile and takes S apart three times: 24 x 40
//           rows 126 -> 395 us, prompts 387 -> 560, for data that is rarely met.
constexpr int kTop = 7, kTopQ = 14;
constexpr float kTopP = 7.f;                     // p <= 2^(kTopP + kLazy) = 2^15
constexpr int kExpMin = -100, kExpMax = 127;
constexpr int kSpread = 21;                      // 2^kTop * 2^-kSpread = 2^-14, the smallest normal fp16 number
constexpr int kWide = 1 << 10;                   // in place of an exponent: the segment's form is wide
constexpr int kParts = 16;                       // of a sequence's groups, at most, each with extremes of its own
constexpr uint32_t kInfBits = 0x7f800000u;

__device__ __forceinline__ float exp2i(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }
// Whether scales from `least` to `most` (bits; most 0: none that is finite) are too
// far apart for the narrow form.
__device__ __forceinline__ bool spread_wide(uint32_t most, uint32_t least) {
  return most > 0u && (static_cast<int>(most >> 23) - static_cast<int>(least >> 23) > kSpread ||
                       static_cast<int>(least >> 23) - 127 < kExpMin - kSpread);
}
// exponent of a value given by its bits
__device__ __forceinline__ int exponent(uint32_t bits) {
  return min(max(static_cast<int>(bits >> 23) - 127, kExpMin), kExpMax);
}

template <int D>
struct Smem {
  static constexpr int kTile = D / 64 * kTileHalf;
  static constexpr int kQ = 0;                     // two row tiles
  static constexpr int kK = 2 * kTile;             // two K tiles
  static constexpr int kV = kK + 2 * kTile;        // one V tile
  static constexpr int kRing = kV + kTile;
  static constexpr int kRingBytes = 55 * 1024;
  static constexpr int kBar = kRing + kRingBytes;
  static constexpr int kMisc = kBar + 58 * 8;      // TMEM base, abort flag, the CTA's form
  static constexpr int kBad = kMisc + 16;          // uint64 [8][4]: a segment's non-finite tokens, per 32 features
  static constexpr int kPow = kBad + 8 * 4 * 8;    // int2 [4]: a segment's exponents (K, V), or kWide
  static constexpr int kKeyPow = kPow + 32;         // float [4][kBT]: powers of the keys of four K tiles (wide form)
  static constexpr int kValExp = kKeyPow + 4 * kBT * 4;   // float [kBT]: exponents of V's rows (wide form)
  static constexpr int kPre = kValExp + kBT * 4;    // int64 pre[S + 1] (inline plan)
};

enum Bar {
  RING_FULL = 0,                 // [kMaxUnits][2 halves]
  RING_EMPTY = 24,               // [kMaxUnits]
  K_READY = 36,                  // [2]
  K_FREE = 38,                   // [2]
  V_READY = 40,
  V_FREE = 41,
  S_FULL = 42,                   // [3]: tile 0, tile 1, a lone tile's other S / P
  P_FULL = 45,                   // [3]
  PV_DONE = 48,                  // [3]
  Q_READY = 51,
  Q_FREE = 52,
  POWERS = 53,                   // [4]
  FORM = 57,                     // the CTA's form is known
};

struct Params {
  Batch t;
  PlanMem plan;
  const uint8_t* k_codes;
  const float* k_scales;
  const uint8_t* v_codes;
  const float* v_scales;
  const uint32_t* tops;          // [S][H][4][kParts]: bits of the largest K and V scales, kInfBits less the smallest's
  int parts;                     // of them in use
  const float* q_pow;            // [T][H_q]: 2^(e - kTopQ) of a query row
  float qscale;                  // scale * log2(e)
  __nv_bfloat16* O;
  float* partials;               // [2 ctas][8][D + 2][32]
  int ctas, RI, TT;              // rows of an item, tokens of a row tile
  unsigned int* err;
};

// ---------------------------------------------------------------------------
// a CTA's blocks
// ---------------------------------------------------------------------------
struct Place {
  int i, h, j, nb;
  int left;                      // blocks from here to the CTA's end (2^31 would take it an hour)
  Item it;
  SeqView s;
  bool start;                    // first block of a segment
};
struct Walk {
  const Params& p;
  PlanView v;
  __device__ __forceinline__ void enter(Place& a) const {
    a.it = plan_item(v, a.i);
    a.s = seq_view(p.t, a.it.b);
    a.nb = v.blocks(a.i);
  }
  __device__ __forceinline__ Place begin(const Range& r) const {
    Place a;
    a.left = static_cast<int>(r.g1 - r.g0);
    a.start = true;
    if (a.left <= 0) return a;
    a.i = find_item(v, p.t.H, r.g0);
    enter(a);
    const long long off = r.g0 - static_cast<long long>(p.t.H) * v.pre[a.i];
    a.h = static_cast<int>(off / a.nb);
    a.j = static_cast<int>(off % a.nb);
    return a;
  }
  __device__ __forceinline__ void next(Place& a) const {
    if (--a.left <= 0) return;
    a.start = false;
    if (++a.j < a.nb) return;
    a.start = true;
    a.j = 0;
    if (++a.h == p.t.H) {
      a.h = 0;
      do ++a.i;
      while (v.blocks(a.i) == 0);
      enter(a);
    }
  }
  // last block of a segment
  __device__ __forceinline__ bool last(const Place& a) const { return a.left == 1 || a.j + 1 == a.nb; }
  // row tiles of the place's item
  __device__ __forceinline__ int tiles(const Place& a) const {
    return a.s.n * p.t.G - a.it.r0 > p.TT * p.t.G && p.RI > p.TT * p.t.G ? 2 : 1;
  }
};

// ---------------------------------------------------------------------------
// decode of a unit's 16 keys to fp16 values in a swizzled tile
// ---------------------------------------------------------------------------
// A lane takes 16 features (two 16-byte chunks of the tile) of a token; at D =
// 128 a quarter warp is one token, and lanes q and q + 4 store their chunks in
// opposite order, so the quarter warp meets eight bank groups; at D = 64 it is
// two tokens, whose rows swizzle differently.
// kWideForm: the values' power is the key's own and goes to s_key[t]: K's inverse
// power, V's exponent.
template <int BITS, int D, bool kV, bool kWideForm>
__device__ __forceinline__ void decode_unit(const unsigned char* u, unsigned char* dst, int wk, int lane, int nv,
                                            float power, int t_base, unsigned long long seg_key,
                                            unsigned long long* s_bad, float* s_key) {
  constexpr int kCb = D * BITS / 8, QN = D / 16, TPP = 32 / QN;
  const int q = lane % QN, tt = lane / QN;
  const bool swap = D == 128 && (q & 4) != 0;
  const int w4 = wk & 3;                            // the warp's 16 keys within the half-unit
  const float* sc = reinterpret_cast<const float*>(u + kBT / 2 * kCb);
  u64 ks[8];                                       // slot 4 i + r: pair r of 8-feature half i ^ swap
  if (!kV) {
    if (16 * wk < nv) {
      const float4* s4 = reinterpret_cast<const float4*>(sc + (w4 >> 1) * D + 16 * q);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int ci = i ^ (swap ? 1 : 0);
        const float4 v0 = s4[2 * ci], v1 = s4[2 * ci + 1];
        ks[4 * i] = pack2(v0.x, v0.y);
        ks[4 * i + 1] = pack2(v0.z, v0.w);
        ks[4 * i + 2] = pack2(v1.x, v1.y);
        ks[4 * i + 3] = pack2(v1.z, v1.w);
      }
      if (!kWideForm) {
#pragma unroll
        for (int i = 0; i < 8; ++i) ks[i] = mul2(ks[i], pack2(power, power));
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) ks[i] = 0ull;
    }
  }
  const u64 mul = pack2(256.f, 16.f), add = pack2(-263.f, -23.f), sub = pack2(-8388735.f, -8388735.f);
#pragma unroll 1
  for (int it = 0; it < 16 / TPP; ++it) {
    const int t = 16 * wk + TPP * it + tt, tu = 16 * w4 + TPP * it + tt;
    uint4 o[2];
    u64 own[8];                                    // wide form: the values, then times the key's power
    if (kWideForm) {
#pragma unroll
      for (int i = 0; i < 8; ++i) own[i] = 0ull;
    }
    if (t < nv) {
      u64 s2 = 0ull;
      if (kV) {
        float s = sc[D / 32 * tu + (q >> 1)];
        if (!(fabsf(s) < INFINITY)) {              // remembered: rows that see the token become NaN there
          atomicMax(s_bad + (q >> 1), seg_key | static_cast<unsigned>(0x7fffffff - (t_base + t)));
          s = 0.f;
        }
        if (!kWideForm) s *= power;
        s2 = pack2(s, s);
      }
      uint32_t h[8];
      if (BITS == 4) {
        const uint2 w2 = *reinterpret_cast<const uint2*>(u + tu * kCb + 8 * q);
        const uint32_t w[2] = {swap ? w2.y : w2.x, swap ? w2.x : w2.y};
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const u64 f = fma2(nibble_pair(byte_at15(w[i], r)), mul, add);
            const u64 x = mul2(f, kV ? s2 : ks[4 * i + r]);
            if (kWideForm) own[4 * i + r] = x;
            else h[4 * i + r] = pack_f16(lo_f(x), hi_f(x));
          }
      } else {
        const uint4 w4 = *reinterpret_cast<const uint4*>(u + tu * kCb + 16 * q);
        const uint32_t w[4] = {swap ? w4.z : w4.x, swap ? w4.w : w4.y, swap ? w4.x : w4.z, swap ? w4.y : w4.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int r = 0; r < 4; r += 2) {
            const u64 f = add2(byte_pair(w[i], r), sub);
            const u64 x = mul2(f, kV ? s2 : ks[2 * i + r / 2]);
            if (kWideForm) own[2 * i + r / 2] = x;
            else h[2 * i + r / 2] = pack_f16(lo_f(x), hi_f(x));
          }
      }
      if (!kWideForm) {
        o[0] = make_uint4(h[0], h[1], h[2], h[3]);
        o[1] = make_uint4(h[4], h[5], h[6], h[7]);
      }
    } else {
      o[0] = make_uint4(0u, 0u, 0u, 0u);
      o[1] = o[0];
    }
    if (kWideForm) {
      uint32_t m = 0u;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        m = max(m, max(static_cast<uint32_t>(own[i]) & 0x7fffffffu, static_cast<uint32_t>(own[i] >> 32) & 0x7fffffffu));
#pragma unroll
      for (int x = 1; x < QN; x <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, x));
      const int e = exponent(m);
      const float f = exp2i(kTopQ - e);
      uint32_t h[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) h[i] = pack_f16(lo_f(own[i]) * f, hi_f(own[i]) * f);
      o[0] = make_uint4(h[0], h[1], h[2], h[3]);
      o[1] = make_uint4(h[4], h[5], h[6], h[7]);
      if (q == 0) s_key[t] = kV ? static_cast<float>(e) : exp2i(e - kTopQ);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int ch = 2 * q + (i ^ (swap ? 1 : 0));
      *reinterpret_cast<uint4*>(dst + (ch >> 3) * kTileHalf + swz(t, ch & 7)) = o[i];
    }
  }
}

// Maximum of 64 raw scores held in registers, as eight independent chains of
// three-input operations.
__device__ __forceinline__ float row_max(const uint32_t (&sr)[64]) {
  auto f = [](uint32_t x) { return __uint_as_float(x); };
  float acc[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    acc[j] = max3(f(sr[j]), f(sr[8 + j]), f(sr[16 + j]));
    acc[j] = max3(acc[j], f(sr[24 + j]), f(sr[32 + j]));
    acc[j] = max3(acc[j], f(sr[40 + j]), f(sr[48 + j]));
    acc[j] = fmaxf(acc[j], f(sr[56 + j]));
  }
  return max3(max3(acc[0], acc[1], acc[2]), max3(acc[3], acc[4], acc[5]), fmaxf(acc[6], acc[7]));
}

// Bounded wait: after about two seconds raises the CTA's abort flag and goes on;
// once the flag is up every later wait gives up too, and the CTA records
// KVQ_ERR_TIMEOUT as it ends.
__device__ __forceinline__ void wait(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  if (mbar_try(bar, parity)) return;
  const uint32_t t0 = static_cast<uint32_t>(globaltimer());
  uint32_t it = 0;
  while (!mbar_try(bar, parity))
    if ((++it & 15u) == 0) {
      if (*abort_flag) return;
      if (static_cast<uint32_t>(globaltimer()) - t0 > 2000000000u) *abort_flag = 1;
    }
}

// After a time-out: waits (100 ms at most) for a copy that is still in flight.
__device__ __forceinline__ void drain(uint32_t bar, uint32_t parity) {
  const uint64_t t0 = globaltimer();
  while (!mbar_try(bar, parity) && globaltimer() - t0 < 100000000ull) {
  }
}

// A block's softmax in the wide form, for a warp's rows: the references and z
// move, O (D columns at o_col) is rescaled where they do, and P replaces S at s_col.
// nv: columns the row sees; s_key, s_val: the block's powers and exponents.  O may be
// rescaled once pv_bar's phase is over (0: it is).
struct WideRow {
  float m, z, r;                  // the score's reference; sum of the weights; the reference of weight + exponent
};
template <int D>
__device__ __forceinline__ WideRow softmax_wide(WideRow w, uint32_t s_col, uint32_t o_col, float qs, int nv,
                                             const float* s_key, const float* s_val, uint32_t v_bar, uint32_t v_parity,
                                             bool first, uint32_t pv_bar, uint32_t pv_parity,
                                             volatile int* abort_flag) {
  const int seen = __reduce_max_sync(0xffffffffu, nv);
  // scores of 16 columns, each less `less`
  auto scores = [&](float (&x)[16], int cc, float less) {
    uint32_t sr[16];
    KVQ_LD16(sr, s_col + 16u * cc);
    tmem_wait_ld();
#pragma unroll
    for (int e = 0; e < 16; ++e) x[e] = __fmul_rn(__uint_as_float(sr[e]), qs * s_key[16 * cc + e]) - less;
  };
  float x[16];
  float top = -INFINITY;
#pragma unroll 1
  for (int cc = 0; 16 * cc < seen; ++cc) {
    scores(x, cc, 0.f);
#pragma unroll
    for (int e = 0; e < 16; ++e)
      if (16 * cc + e < nv) top = fmaxf(top, x[e]);
  }
  if (top > w.m + kLazy) {
    w.z *= ex2(w.m - top);                               // 0 where the row had no key
    w.r += w.m - top;
    w.m = top;
  }
  // V's exponents come with its tile.  (The phase before this one is over: this
  // row's tile waited for it, or, where a segment begins, the MMA issuer did before
  // the scores.)
  wait(v_bar, v_parity, abort_flag);
  top = -INFINITY;
#pragma unroll 1
  for (int cc = 0; 16 * cc < seen; ++cc) {
    scores(x, cc, w.m);
#pragma unroll
    for (int e = 0; e < 16; ++e)
      if (16 * cc + e < nv) top = fmaxf(top, x[e] + s_val[16 * cc + e]);
  }
  const bool need = top > w.r + kLazy;
  if (__any_sync(0xffffffffu, need)) {
    const float a = need ? ex2(w.r - top) : 1.f;
    if (need) w.r = top;
    if (!first) {
      if (pv_bar) {
        wait(pv_bar, pv_parity, abort_flag);
        tc_fence_after();
      }
#pragma unroll 1
      for (int oc = 0; oc < D / 16; ++oc) {
        uint32_t orr[16];
        KVQ_LD16(orr, o_col + 16u * oc);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 16; ++e) orr[e] = __float_as_uint(__uint_as_float(orr[e]) * a);
        KVQ_ST16(o_col + 16u * oc, orr);
      }
    }
  }
#pragma unroll 1
  for (int cc = 0; cc < 8; ++cc) {
    const int left = nv - 16 * cc;
    uint32_t pk[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
    if (16 * cc < seen) {
      scores(x, cc, w.m);
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        if (e < left) w.z += ex2(x[e] + kTopP);
        x[e] = e < left ? ex2(x[e] + (s_val[16 * cc + e] - w.r) + kTopP) : 0.f;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) pk[e] = pack_f16(x[2 * e], x[2 * e + 1]);
    }
    KVQ_ST8(s_col + 8u * cc, pk);
  }
  return w;
}

// What the attention needs beforehand.  The first S * H * parts CTAs find the
// largest and smallest K and V scales of a sequence and KV head, in parts of its
// groups of 32 tokens, a warp a group: they read the scales alone (32 of 160 bytes a token at D
// = 128 and 4 bits), and the attention finds them in the L2 afterwards.  The
// others turn the query rows to fp16, D / 8 lanes a row.  (Turned in shared memory
// by the softmax, at a segment's start, prompts took 419 us instead of 397.)
constexpr int kPrepareWarps = 8, kRowsPerLane = 4;
template <int D>
__global__ void __launch_bounds__(32 * kPrepareWarps)
    paged_prepare_kernel(Batch t, const float* k_scales, const float* v_scales, uint32_t* tops, int parts,
                         const uint4* Q, uint4* Qh, float* q_pow, long long rows, int beside, unsigned int* err) {
  // beside: the kernel before is the plan's, which has waited for every other
  // and writes what this one does not touch.  (All that is read may just have been
  // written by such a grid, of the library too: through the L2.)
  if (beside) griddep_release();
  else griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long scans = static_cast<long long>(t.S) * t.H * parts;
  if (blockIdx.x >= scans) {
    constexpr int L = D / 8, PASS = 32 * kPrepareWarps / L;
    const long long first = (blockIdx.x - scans) * (PASS * kRowsPerLane) + threadIdx.x / L;
    const int l = threadIdx.x % L;
    uint4 x[kRowsPerLane];
#pragma unroll
    for (int i = 0; i < kRowsPerLane; ++i) {
      const long long row = first + i * PASS;
      x[i] = make_uint4(0u, 0u, 0u, 0u);
      if (row < rows) x[i] = __ldcg(Q + row * L + l);
    }
#pragma unroll
    for (int i = 0; i < kRowsPerLane; ++i) {
      const long long row = first + i * PASS;
      uint32_t m = __vmaxu2(__vmaxu2(x[i].x & 0x7fff7fffu, x[i].y & 0x7fff7fffu),
                            __vmaxu2(x[i].z & 0x7fff7fffu, x[i].w & 0x7fff7fffu));   // (magnitudes order as their bits do)
      m = max(m & 0xffffu, m >> 16);
#pragma unroll
      for (int o = 1; o < L; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
      const int e = exponent(m << 16);
      const float f = exp2i(kTopQ - e);
      auto turn = [&](uint32_t v) {
        return pack_f16(__uint_as_float(v << 16) * f, __uint_as_float(v & 0xffff0000u) * f);
      };
      if (row < rows) {
        Qh[row * L + l] = make_uint4(turn(x[i].x), turn(x[i].y), turn(x[i].z), turn(x[i].w));
        if (l == 0) q_pow[row] = exp2i(e - kTopQ);
      }
    }
    if (beside) griddep_join();
    return;
  }
  const int part = static_cast<int>(blockIdx.x % parts), bh = static_cast<int>(blockIdx.x / parts);
  const int b = bh / t.H, h = bh % t.H;
  const SeqView s = seq_view(t, b);
  const int32_t* table = t.table + static_cast<long long>(b) * t.max_pages;
  uint32_t top[4] = {0u, 0u, 0u, 0u};                     // K's and V's largest, kInfBits less the smallest
  // lane i looks up the page of the warp's i-th group, 32 at a time; then the
  // scales of four groups are on their way together
  const int stride = parts * kPrepareWarps, groups = s.n > 0 ? (s.len + 31) >> 5 : 0;
  for (int g0 = part * kPrepareWarps + warp; g0 < groups; g0 += 32 * stride) {
    const int g = g0 + lane * stride;
    long long own = 0;
    if (g < groups) {
      const int pi = 32 * g / t.P;
      own = (static_cast<long long>(read_page(__ldcg(table + pi), t.pages, err)) * t.H + h) * t.P + 32 * g - pi * t.P;
    }
    const int n = min(32, (groups - g0 + stride - 1) / stride);
    for (int i0 = 0; i0 < n; i0 += 4) {
      using Vec = typename std::conditional<D == 128, uint4, uint2>::type;
      Vec x[4][2];
#pragma unroll
      for (int i = 0; i < 4; ++i) {                       // (past the last one: the last one again)
        const long long tok = __shfl_sync(0xffffffffu, own, min(i0 + i, n - 1));
        x[i][0] = __ldcg(reinterpret_cast<const Vec*>(k_scales + (tok >> 5) * D) + lane);
        x[i][1] = __ldcg(reinterpret_cast<const Vec*>(v_scales + tok * (D / 32)) + lane);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool live = 32 * (g0 + min(i0 + i, n - 1) * stride) + lane < s.len;   // the lane's token
#pragma unroll
        for (int e = 0; e < 2 * D / 32; ++e) {            // (zero, and what is not finite, stays that whatever the power)
          const uint32_t v = reinterpret_cast<const uint32_t*>(&x[i][e / (D / 32)])[e % (D / 32)] & 0x7fffffffu;
          if (v - 1u < kInfBits - 1u && (e < D / 32 || live)) {
            top[e / (D / 32)] = max(top[e / (D / 32)], v);
            top[2 + e / (D / 32)] = max(top[2 + e / (D / 32)], kInfBits - v);
          }
        }
      }
    }
  }
  __shared__ uint32_t s_top[4][kPrepareWarps];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t m = __reduce_max_sync(0xffffffffu, top[i]);
    if (lane == 0) s_top[i][warp] = m;
  }
  __syncthreads();
  if (threadIdx.x < 4) {
    uint32_t m = 0u;
    for (int w = 0; w < kPrepareWarps; ++w) m = max(m, s_top[threadIdx.x][w]);
    tops[(static_cast<long long>(bh) * 4 + threadIdx.x) * kParts + part] = m;
  }
  if (beside) griddep_join();
}

// ---------------------------------------------------------------------------
// the decode and softmax roles
// ---------------------------------------------------------------------------
// What they need of their CTA.
template <int BITS, int D>
struct Cta {
  using M = Smem<D>;
  static constexpr int kCodes = D * BITS / 8;             // code bytes of a key
  static constexpr int kScales = D * 8;                   // scale bytes of a half-unit (K: 2 groups x D; V: 64 x D / 32)
  static constexpr int kUnit = kBT / 2 * kCodes + kScales;
  static constexpr uint32_t kUnits = M::kRingBytes / kUnit < kMaxUnits ? M::kRingBytes / kUnit : kMaxUnits;
  const Params& p;
  Walk walk;
  Range wr;
  unsigned char* sm;
  uint32_t base, tmem;
  __device__ __forceinline__ uint32_t bar(int i) const { return base + M::kBar + 8u * static_cast<uint32_t>(i); }
};

// kWideToo: a segment may have the wide form.
template <int BITS, int D, bool kWideToo>
__device__ __forceinline__ void decode_role(const Cta<BITS, D>& cta) {
  using M = Smem<D>;
  const Params& p = cta.p;
  const Walk& walk = cta.walk;
  const Range& wr = cta.wr;
  unsigned char* const sm = cta.sm;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto bar = [&](int i) { return cta.bar(i); };
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(sm + M::kMisc + 4);
  unsigned long long* const s_bad = reinterpret_cast<unsigned long long*>(sm + M::kBad);
  const int2* const s_pow = reinterpret_cast<const int2*>(sm + M::kPow);
  float* const s_key = reinterpret_cast<float*>(sm + M::kKeyPow);
  float* const s_val = reinterpret_cast<float*>(sm + M::kValExp);
  constexpr uint32_t nu = Cta<BITS, D>::kUnits;
  constexpr int unit_bytes = Cta<BITS, D>::kUnit;
  const int wk = warp - 12;
  const int half = wk >> 2;
  uint32_t slot = half, wraps = 0, kb = 0, seg = 0;    // kb: K blocks decoded; V's are one behind
  Place c = walk.begin(wr);
  int t0 = 0, nv = 0;                                 // V's block
  bool start = false;
  uint32_t segs = 0;                                  // segments begun
  int2 pw = make_int2(0, 0);                          // K's and V's block's
  int ev = 0;
  auto arrived = [&]() {
    wait(bar(RING_FULL + 2 * slot + half), wraps >> (nu & 1u) & 1u, abort_flag);
    return sm + M::kRing + slot * unit_bytes;
  };
  auto finished = [&](uint32_t ready) {
    fence_proxy_async();
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(ready);
      mbar_arrive(bar(RING_EMPTY + slot));
    }
    slot += 2;
    if (slot >= nu) {
      slot -= nu;
      ++wraps;
    }
  };
#pragma unroll 1
  for (;; ++kb) {                                     // K(kb), then V(kb - 1)
    const int t0_k = c.j * kBT, nv_k = c.s.len - t0_k;
    const bool more = c.left > 0, start_k = c.start;
    if (more) {
      const uint32_t buf = kb & 1u;
      if (start_k) {
        wait(bar(POWERS + (segs & 3u)), segs >> 2 & 1u, abort_flag);
        pw = s_pow[segs & 3u];
        ++segs;
      }
      const unsigned char* u = arrived();
      if (kb >= 2) wait(bar(K_FREE + buf), ((kb >> 1) - 1) & 1u, abort_flag);
      // (a key's powers are read by the softmax, after the tile's buffer is free
      // again: four of them)
      if (kWideToo && pw.x == kWide)
        decode_unit<BITS, D, false, true>(u, sm + M::kK + buf * M::kTile, wk, lane, min(kBT, nv_k), 0.f, 0, 0, nullptr,
                                         s_key + (kb & 3u) * kBT);
      else
        decode_unit<BITS, D, false, false>(u, sm + M::kK + buf * M::kTile, wk, lane, min(kBT, nv_k),
                                           exp2i(kTop - pw.x), 0, 0, nullptr, nullptr);
      finished(bar(K_READY + buf));
      walk.next(c);
    }
    if (kb > 0) {
      const uint32_t v = kb - 1;
      const unsigned char* u = arrived();
      if (v >= 1) wait(bar(V_FREE), (v - 1) & 1u, abort_flag);
      if (start) ++seg;
      const unsigned long long key = static_cast<unsigned long long>(seg) << 32;
      if (kWideToo && ev == kWide)
        decode_unit<BITS, D, true, true>(u, sm + M::kV, wk, lane, min(kBT, nv), 0.f, t0, key,
                                         s_bad + 4 * (seg & 7u), s_val);
      else
        decode_unit<BITS, D, true, false>(u, sm + M::kV, wk, lane, min(kBT, nv), exp2i(kTop - ev), t0, key,
                                          s_bad + 4 * (seg & 7u), nullptr);
      finished(bar(V_READY));
    }
    if (!more) break;
    t0 = t0_k;
    nv = nv_k;
    start = start_k;
    ev = pw.y;
  }
}

// One query row a thread.
template <int BITS, int D, bool kWideToo>
__device__ __forceinline__ void softmax_role(const Cta<BITS, D>& cta) {
  using M = Smem<D>;
  const Params& p = cta.p;
  const Walk& walk = cta.walk;
  const Range& wr = cta.wr;
  unsigned char* const sm = cta.sm;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto bar = [&](int i) { return cta.bar(i); };
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(sm + M::kMisc + 4);
  unsigned long long* const s_bad = reinterpret_cast<unsigned long long*>(sm + M::kBad);
  const int2* const s_pow = reinterpret_cast<const int2*>(sm + M::kPow);
  float* const s_key = reinterpret_cast<float*>(sm + M::kKeyPow);
  float* const s_val = reinterpret_cast<float*>(sm + M::kValExp);
  const int H = p.t.H, G = p.t.G, TR = p.TT * G;
  const uint32_t tmem = cta.tmem;
  const int tile = (warp - 4) >> 2;
  const int r = ((warp & 3) << 5) + lane;            // TMEM lane = row within the tile
  const uint32_t lane_addr = static_cast<uint32_t>((warp & 3) * 32) << 16;
  const uint32_t o_col = tmem + lane_addr + 256u + 128u * tile;
  const bool neg = p.qscale < 0.f;
  float m_ref = -INFINITY, z = 0.f;
  float qs = 0.f, ov = 0.f;                           // what the row's scores and its O are multiplied by;
                                                      // wide form: ov is R, the reference of weight + exponent
  uint32_t k[2] = {0, 0}, seg = 0;                    // blocks of the tile's S and of its other one (tile 1: and
                                                      // those it has no part in); segments of the CTA
  bool other = true;
  long long row = 0;                                  // of Q and O
  int lim = 0;                                        // keys the row sees
  bool real = false;                                  // the row exists
  bool first_seg = true, seg_is_first = true, from_zero = false;
#pragma unroll 1
  for (Place c = walk.begin(wr); c.left > 0; walk.next(c)) {
    if (c.start) {
      ++seg;
      seg_is_first = first_seg;
      first_seg = false;
      from_zero = c.j == 0;
      const int rr = c.it.r0 + tile * TR + r;
      real = r < TR && rr < c.s.n * G;
      lim = real ? row_limit(p.t, c.s, rr) : c.s.len;  // rows that do not exist take the unmasked path
      row = static_cast<long long>(c.s.q0 + rr / G) * (H * G) + c.h * G + rr % G;
      m_ref = -INFINITY;
      z = 0.f;
      qs = real ? __ldcg(p.q_pow + row) : 0.f;        // (no row: equal scores, never a new reference)
    }
    const bool lone = walk.tiles(c) == 1;
    if (lone && tile) {
      if (kWideToo) ++k[1];
      continue;
    }
    other = lone && !c.start && !other;               // a lone tile takes its two in turn
    const int u = other ? 2 : tile;
    const uint32_t s_col = tmem + lane_addr + (u > 0 ? 128u : 0u), nth = other ? k[1] : k[0];
    wait(bar(S_FULL + u), nth & 1u, abort_flag);
    const int2 pw = s_pow[(seg - 1) & 3u];            // (written before the query rows were asked for)
    const bool wide = kWideToo && pw.x == kWide;
    if (c.start) {
      qs = p.qscale * qs * (wide ? 1.f : exp2i(pw.x - kTop));
      ov = wide ? -INFINITY : exp2i(pw.y - kTop);
    }
    tc_fence_after();
    const int nv = min(kBT, lim - c.j * kBT);       // columns the row sees
    if (wide) {
      const uint32_t blk = k[0] + k[1];               // blocks of the CTA before this one
      const WideRow w = softmax_wide<D>(WideRow{m_ref, z, ov}, s_col, o_col, qs, nv, s_key + (blk & 3u) * kBT, s_val,
                                        bar(V_READY), blk & 1u, c.start, lone ? bar(PV_DONE + 2 - u) : 0u,
                                        ((other ? k[0] : k[1]) - 1) & 1u, abort_flag);
      m_ref = w.m;
      z = w.z;
      ov = w.r;
    } else {
      const bool plain = !neg && __all_sync(0xffffffffu, nv >= kBT);
      const int seen = plain ? kBT : __reduce_max_sync(0xffffffffu, nv);   // columns that a row of the warp sees
      // the row's largest score over the columns it sees (none: never a new reference)
      float mb = -INFINITY;
      if (plain) {
#pragma unroll 1
        for (int hh = 0; hh < 2; ++hh) {
          uint32_t sr[64];
          KVQ_LD32_AT(sr, 0, s_col + 64u * hh);
          KVQ_LD32_AT(sr, 32, s_col + 64u * hh + 32u);
          tmem_wait_ld();
          mb = fmaxf(mb, row_max(sr));
        }
        mb *= qs;
      } else {
#pragma unroll 1
        for (int cc = 0; 16 * cc < seen; ++cc) {
          uint32_t sr[16];
          KVQ_LD16(sr, s_col + 16u * cc);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (16 * cc + e < nv) mb = fmaxf(mb, __uint_as_float(sr[e]) * qs);
        }
      }
      const bool need = mb > m_ref + kLazy;
      if (__any_sync(0xffffffffu, need)) {
        const float a = need ? ex2(m_ref - mb) : 1.f;    // 0 where the row had no key
        if (need) m_ref = mb;
        z *= a;
        if (!c.start) {
          if (lone) {                                   // (its S did not wait for the last product)
            wait(bar(PV_DONE + 2 - u), ((other ? k[0] : k[1]) - 1) & 1u, abort_flag);
            tc_fence_after();
          }
#pragma unroll 1
          for (int oc = 0; oc < D / 16; ++oc) {
            uint32_t orr[16];
            KVQ_LD16(orr, o_col + 16u * oc);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) orr[e] = __float_as_uint(__uint_as_float(orr[e]) * a);
            KVQ_ST16(o_col + 16u * oc, orr);
          }
        }
      }
      // p = exp2(s * qs - m_ref + kTopP) as fp16 over the columns already read,
      // 16 at a time, the next ones on their way.  (m_ref is a product's rounding and
      // the fused product is not rounded: the largest p is off by half an ulp of
      // m_ref in its exponent, the same for all of a row's.  That is 1/8 below 2^22;
      // beyond, the other body rounds the products too, or p could leave fp16.)
      const float m_top = kTopP - m_ref;
      u64 z2 = 0ull;
      const bool far = __any_sync(0xffffffffu, fabsf(m_ref) > 4194304.f);
      if (plain && !far) {
        uint32_t s0[16], s1[16];
        const u64 f2 = pack2(qs, qs), c2 = pack2(m_top, m_top);
        auto columns = [&](const uint32_t (&sr)[16], int cc) {
          uint32_t pk[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const u64 x = fma2(pack2(__uint_as_float(sr[2 * e]), __uint_as_float(sr[2 * e + 1])), f2, c2);
            const float p0 = ex2(lo_f(x)), p1 = ex2(hi_f(x));
            z2 = add2(z2, pack2(p0, p1));
            pk[e] = pack_f16(p0, p1);
          }
          KVQ_ST8(s_col + 8u * cc, pk);
        };
        KVQ_LD16(s0, s_col);
#pragma unroll 1
        for (int cc = 0; cc < 8; cc += 2) {
          tmem_wait_ld();
          KVQ_LD16(s1, s_col + 16u * cc + 16u);
          columns(s0, cc);
          tmem_wait_ld();
          if (cc < 6) KVQ_LD16(s0, s_col + 16u * cc + 32u);
          columns(s1, cc + 1);
        }
      } else {
#pragma unroll 1
        for (int cc = 0; cc < 8; ++cc) {
          const int left = nv - 16 * cc;
          uint32_t pk[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
          if (16 * cc < seen) {
            uint32_t sr[16];
            KVQ_LD16(sr, s_col + 16u * cc);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
              const float y0 = __uint_as_float(sr[e]), y1 = __uint_as_float(sr[e + 1]);
              const float x0 = far ? __fmul_rn(y0, qs) - m_ref + kTopP : fmaf(y0, qs, m_top);
              const float x1 = far ? __fmul_rn(y1, qs) - m_ref + kTopP : fmaf(y1, qs, m_top);
              const float p0 = e < left ? ex2(x0) : 0.f;
              const float p1 = e + 1 < left ? ex2(x1) : 0.f;
              z2 = add2(z2, pack2(p0, p1));
              pk[e >> 1] = pack_f16(p0, p1);
            }
          }
          KVQ_ST8(s_col + 8u * cc, pk);
        }
      }
      z += lo_f(z2) + hi_f(z2);
    }
    tmem_wait_st();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(P_FULL + u));
    if (other) ++k[1]; else ++k[0];
    if (walk.last(c)) {
      // the segment's last P V product must be done before O is read
      wait(bar(PV_DONE + u), nth & 1u, abort_flag);
      tc_fence_after();
      const bool whole = from_zero && c.j + 1 == c.nb;
      if (wide) ov = z == 0.f ? 0.f : ex2(ov - static_cast<float>(kTopQ));
      const int pr = tile * 128 + r;
      float* part = p.partials + (2 * static_cast<long long>(blockIdx.x) + (seg_is_first ? 0 : 1)) * 256 * (D + 2) +
                    static_cast<long long>(pr >> 5) * (D + 2) * 32 + (pr & 31);
      if (!whole) {
        part[0] = m_ref;
        part[32] = z;
      }
      // z = 0: a row without a key
      const float inv = z == 0.f ? 0.f : ov / z;
      uint32_t bad_mask = 0u;                           // feature groups with a non-finite scale that the row sees
#pragma unroll
      for (int cc = 0; cc < D / 32; ++cc) {
        const unsigned long long bad = *reinterpret_cast<volatile unsigned long long*>(s_bad + 4 * (seg & 7u) + cc);
        if ((bad >> 32) == seg && 0x7fffffff - static_cast<int>(bad & 0xffffffffu) < lim) bad_mask |= 1u << cc;
      }
#pragma unroll 1
      for (int cc = 0; cc < D / 32; ++cc) {
        const float by = (bad_mask >> cc & 1u) ? __uint_as_float(0x7fc00000u) : (whole ? inv : ov);
        uint32_t orr[32];
        KVQ_LD32(orr, o_col + 32u * cc);
        tmem_wait_ld();
        if (whole) {
          uint32_t ob[16];
#pragma unroll
          for (int e = 0; e < 16; ++e)
            ob[e] = pack_bf16(__uint_as_float(orr[2 * e]) * by, __uint_as_float(orr[2 * e + 1]) * by);
          if (real) {
            uint4* dst = reinterpret_cast<uint4*>(p.O + row * D + 32 * cc);
#pragma unroll
            for (int qq = 0; qq < 4; ++qq)
              dst[qq] = make_uint4(ob[4 * qq], ob[4 * qq + 1], ob[4 * qq + 2], ob[4 * qq + 3]);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) part[(2 + 32 * cc + e) * 32] = __uint_as_float(orr[e]) * by;
        }
      }
      tc_fence_before();
    }
  }
}
// Both, for a CTA with such segments.  Out of line: side by side in the narrow
// form's loops these steps cost it 4 % (drafts 119 -> 125, prompts 379 -> 395 us).
template <int BITS, int D>
__device__ __noinline__ void wide_roles(Cta<BITS, D> cta) {
  if (threadIdx.x >= 12 * 32) decode_role<BITS, D, true>(cta);
  else softmax_role<BITS, D, true>(cta);
}

template <int BITS, int D>
__global__ void __launch_bounds__(kThreads, 1) paged_chunk_kernel(const __grid_constant__ CUtensorMap qmap,
                                                                  const __grid_constant__ Params p) {
  using M = Smem<D>;
  griddep_wait();
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  const uint32_t raw_addr = su(smem_raw);
  const uint32_t base = (raw_addr + 1023u) & ~1023u;
  unsigned char* sm = smem_raw + (base - raw_addr);
  long long* s_pre = reinterpret_cast<long long*>(sm + M::kPre);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + M::kMisc + 4);
  int2* s_pow = reinterpret_cast<int2*>(sm + M::kPow);
  unsigned long long* s_bad = reinterpret_cast<unsigned long long*>(sm + M::kBad);
  const uint32_t bar0 = base + M::kBar;
  auto bar = [&](int i) { return bar0 + 8u * static_cast<uint32_t>(i); };

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int H = p.t.H, G = p.t.G, TR = p.TT * G;
  constexpr int cb = Cta<BITS, D>::kCodes, kScales = Cta<BITS, D>::kScales, unit_bytes = Cta<BITS, D>::kUnit;
  constexpr uint32_t nu = Cta<BITS, D>::kUnits;

  if (!p.plan.count && warp == 0) warp_prefix(p.t, p.RI, kBT, s_pre);
  if (threadIdx.x == 32) {
    *abort_flag = 0;
    for (int i = 0; i < 8 * 4; ++i) s_bad[i] = 0;
    for (uint32_t u = 0; u < nu; ++u) {
      mbar_init(bar(RING_FULL + 2 * u), 1);
      mbar_init(bar(RING_FULL + 2 * u + 1), 1);
      mbar_init(bar(RING_EMPTY + u), kDecodeWarps / 2);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(K_READY + i), kDecodeWarps);
      mbar_init(bar(K_FREE + i), 1);
    }
    for (int i = 0; i < 3; ++i) {
      mbar_init(bar(S_FULL + i), 1);
      mbar_init(bar(P_FULL + i), 4);
      mbar_init(bar(PV_DONE + i), 1);
    }
    for (int i = 0; i < 4; ++i) mbar_init(bar(POWERS + i), 1);
    mbar_init(bar(FORM), 1);
    mbar_init(bar(V_READY), kDecodeWarps);
    mbar_init(bar(V_FREE), 1);
    mbar_init(bar(Q_READY), 1);
    mbar_init(bar(Q_FREE), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(base + M::kMisc),
                 "r"(512));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(sm + M::kMisc);

  const Walk walk{p, plan_view(p.plan, s_pre, p.t.S)};
  const Range wr = worker_range(walk.v, H, p.ctas, blockIdx.x);
  if (wr.g0 < wr.g1) {
    if (warp == 0) {
      // ======================= producer =======================
      // Lane i < 4 brings keys 32 i .. 32 i + 31 of a block (32 keys lie in one
      // page); lanes 0, 1 fill the first half-unit, 2, 3 the second.  What the
      // loop needs of a block is carried along from the one before: this one warp
      // has to be through with four half-units in less time than a block takes
      // (with divisions and 64-bit products per half it took 3.2k cycles itself).
      const int half = (lane >> 1) & 1, P = p.t.P;
      const int step_pages = kBT / P, step_rows = kBT % P;
      const long long head_tokens = P, page_tokens = static_cast<long long>(H) * P;
      Place kc = walk.begin(wr);
      int pi = 0, at = 0, page = 0, left = 0;             // this lane's page index, row, page; keys from its first on
      const int32_t* table = p.t.table;
      auto look = [&]() {                                 // page of block kc for this lane
        if (kc.left <= 0) return;
        if (kc.start) {
          const int t = kc.j * kBT + 32 * lane;
          pi = t / P;
          at = t - pi * P;
          left = kc.s.len - t;
          table = p.t.table + static_cast<long long>(kc.it.b) * p.t.max_pages;
        } else {
          pi += step_pages;
          at += step_rows;
          if (at >= P) {
            at -= P;
            ++pi;
          }
          left -= kBT;
        }
        page = lane < 4 && left > 0 ? __ldg(table + pi) : 0;
      };
      look();
      uint32_t n = 0, slot = half, wraps = 0;             // half-units issued; this half's slot and its rounds
      auto unit = [&](bool is_v, long long tok, int groups) {
        if (lane < 4 && wraps > 0) wait(bar(RING_EMPTY + slot), (wraps - 1) & 1u, abort_flag);
        if (__any_sync(0xffffffffu, *abort_flag)) return;   // after a time-out nothing more is copied
        const uint32_t fb = bar(RING_FULL + 2 * slot + half);
        if ((lane & ~2) == 0)                             // (a half past the end brings nothing)
          mbar_expect_tx(fb, static_cast<uint32_t>(min(max(groups - lane, 0), 2) * (32 * cb + kScales / 2)));
        __syncwarp();
        if (lane < groups) {
          const uint32_t dst = base + M::kRing + slot * unit_bytes, i = lane & 1;
          const uint8_t* codes = (is_v ? p.v_codes : p.k_codes) + tok * cb;
          const float* scales = is_v ? p.v_scales + tok * (D / 32) : p.k_scales + (tok >> 5) * D;
          bulk_g2s(dst + i * 32 * cb, codes, 32 * cb, fb);
          bulk_g2s(dst + kBT / 2 * cb + i * (kScales / 2), scales, kScales / 2, fb);
        }
        n += 2;
        slot += 2;
        if (slot >= nu) {
          slot -= nu;
          ++wraps;
        }
      };
      long long tok_v = 0, tok = 0;
      int groups_v = 0, groups = 0;
      const int blocks = static_cast<int>(wr.g1 - wr.g0);
#pragma unroll 1
      for (int i = 0; i <= blocks; ++i) {
#pragma unroll 1
        for (int is_v = i == blocks; is_v < 2; ++is_v) {  // K(i), then V(i - 1)
          if (!is_v) {
            tok_v = tok;
            groups_v = groups;
            tok = read_page(page, p.t.pages, p.err) * page_tokens + kc.h * head_tokens + at;
            groups = (min(kBT, __shfl_sync(0xffffffffu, left, 0)) + 31) >> 5;
            walk.next(kc);
            look();
          } else if (i == 0) {
            break;
          } else if (i == blocks) {
            tok_v = tok;
            groups_v = groups;
          }
          unit(is_v, is_v ? tok_v : tok, is_v ? groups_v : groups);
        }
      }
      // The decode warps took every copy before they ended, unless a wait ran
      // out: then the last ones in flight are waited for here (again bounded),
      // so that none writes into shared memory after the CTA has left it.
      if (*abort_flag && lane == 0)
        for (uint32_t i = n > nu ? n - nu : 0; i < n; ++i) {
          const uint32_t b = bar(RING_FULL + 2 * (i % nu) + (i & 1u)), ph = (i / nu) >> (nu & 1u) & 1u;
          drain(b, ph);
        }
      __syncwarp();
    } else if (warp == 1) {
      // ======================= MMA issuer =======================
      // The whole warp runs this loop, on values that are the same in every
      // lane (broadcast where they come from memory), and one lane issues: the
      // operands of tcgen05.mma then sit in uniform registers.  With the loop
      // in one lane's branch each instruction had to move its eight operands
      // there first, and 32 of them a block took longer than their execution.
      const uint32_t lead = elect_one();
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      const uint32_t idesc_qk = instr_desc_f16(kBT, false);
      const uint32_t idesc_pv = instr_desc_f16(D, true);
      // descriptors: the address field counts 16-byte units, so a step adds to the low word
      const uint64_t dq = smem_desc(base + M::kQ, 16, 1024), dk = smem_desc(base + M::kK, 16, 1024),
                     dv = smem_desc(base + M::kV, kTileHalf, 1024);
      // u: 0 and 1, the tiles; 2, a lone tile's other S / P (in tile 1's columns)
      auto qk = [&](int u, uint32_t k) {
        const uint64_t q0 = dq + static_cast<uint64_t>((u & 1) * (M::kTile >> 4)),
                       k0 = dk + static_cast<uint64_t>((k & 1u) * (M::kTile >> 4));
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const uint64_t step = static_cast<uint64_t>(((i >> 2) * kTileHalf + (i & 3) * 32) >> 4);
          mma_ss_if(lead, tm + (u > 0 ? 128u : 0u), q0 + step, k0 + step, idesc_qk, i > 0);
        }
        mma_commit_if(lead, bar(S_FULL + u));
      };
      uint32_t done[3] = {0, 0, 0};                       // P V products issued
      auto pv = [&](int u, bool first) {
        wait(bar(P_FULL + u), done[u] & 1u, abort_flag);
        tc_fence_after();
#pragma unroll
        for (int i = 0; i < kBT / 16; ++i)
          mma_ts_if(lead, tm + 256u + 128u * (u & 1), tm + (u > 0 ? 128u : 0u) + 8u * i,
                    dv + static_cast<uint64_t>(i * 128), idesc_pv, (!first) || (i > 0));
        mma_commit_if(lead, bar(PV_DONE + u));
        ++done[u];
      };
      // an S overwrites the P there: the last P V product must be done
      auto pv_done = [&](int u) {
        if (done[u] > 0) {
          wait(bar(PV_DONE + u), (done[u] - 1) & 1u, abort_flag);
          tc_fence_after();
        }
      };
      // what the loop asks about a block, in one word
      enum : uint32_t { kMore = 1, kStart = 2, kTwo = 4, kLast = 8 };
      Place c = walk.begin(wr);
      auto flags = [&]() {
        const uint32_t f = c.left > 0 ? kMore | (c.start ? kStart : 0u) | (walk.tiles(c) == 2 ? kTwo : 0u) |
                                            (walk.last(c) ? kLast : 0u)
                                      : 0u;
        walk.next(c);
        return __shfl_sync(0xffffffffu, f, 0);
      };
      uint32_t sq = 0;                                    // segments begun
      bool other = false, other_next = false;             // the current block's S is a lone tile's other one
      uint32_t fc = 0, fn = 0;                            // the current block's (k) and the next one's
#pragma unroll 1
      for (uint32_t k = ~0u - 1u;; ++k) {                 // (the first rounds have no current block, no next one)
        const bool have = fc & kMore, more = fn & kMore, boundary = more && (fn & kStart);
        // a lone tile has its S twice: the next block's scores are there before
        // this one's values are
        const bool lone = have && more && !boundary && !(fn & kTwo);
        if (boundary) other_next = false;
        else other_next = !other && !(fn & kTwo);
        if (lone) {
          wait(bar(K_READY + ((k + 1) & 1u)), ((k + 1) >> 1) & 1u, abort_flag);
          if (other_next) {
            pv_done(1);
            pv_done(2);
            tc_fence_after();
            qk(2, k + 1);
          } else {
            pv_done(0);
            tc_fence_after();
            qk(0, k + 1);
          }
          mma_commit_if(lead, bar(K_FREE + ((k + 1) & 1u)));
          if (fn & kLast) mma_commit_if(lead, bar(Q_FREE));
        }
        if (have) {
          wait(bar(V_READY), k & 1u, abort_flag);
          tc_fence_after();
          if (other) pv(2, fc & kStart);
          else pv(0, fc & kStart);
        }
        const uint32_t fnn = flags();                     // while the product runs
        // Q K of the next block's first tile, then P V of this one's second; the
        // other way round where the query rows change
#pragma unroll 1
        for (int step = 0; step < 2; ++step) {
          if (step == boundary) {
            if (more && !lone) {
              if (boundary) wait(bar(Q_READY), sq++ & 1u, abort_flag);
              wait(bar(K_READY + ((k + 1) & 1u)), ((k + 1) >> 1) & 1u, abort_flag);
              pv_done(0);
              tc_fence_after();
              qk(0, k + 1);
            }
          } else if (have) {
            if (fc & kTwo) pv(1, fc & kStart);
            mma_commit_if(lead, bar(V_FREE));
          }
        }
        if (more && !lone) {
          if (fn & kTwo) {
            pv_done(1);
            pv_done(2);
            tc_fence_after();
            qk(1, k + 1);
          }
          mma_commit_if(lead, bar(K_FREE + ((k + 1) & 1u)));
          if (fn & kLast) mma_commit_if(lead, bar(Q_FREE));
        }
        fc = fn;
        fn = fnn;
        other = other_next;
        if (!(fc | fn)) break;
      }
      __syncwarp();
    } else if (warp == 2) {
      // ======================= Q loader, and the segments' powers =======================
      // (a segment's are read before the last one's query rows are free: the decode
      // warps are ahead of the MMAs)
      uint32_t s = 0;                                     // segments
#pragma unroll 1
      for (Place c = walk.begin(wr); c.left > 0; walk.next(c)) {
        if (!c.start) continue;
        const uint32_t* tops = p.tops + (static_cast<long long>(c.it.b) * H + c.h) * (4 * kParts) + lane;
        const bool live = lane % kParts < p.parts;
        const uint32_t x = live ? __ldcg(tops) : 0u, y = live ? __ldcg(tops + 2 * kParts) : 0u;
        const uint32_t ke = __reduce_max_sync(0xffffffffu, lane < kParts ? x : 0u);
        const uint32_t ve = __reduce_max_sync(0xffffffffu, lane < kParts ? 0u : x);
        const uint32_t kl = kInfBits - __reduce_max_sync(0xffffffffu, lane < kParts ? y : 0u);
        const uint32_t vl = kInfBits - __reduce_max_sync(0xffffffffu, lane < kParts ? 0u : y);
        if (lane == 0) {
          s_pow[s & 3u] = spread_wide(ke, kl) || spread_wide(ve, vl) ? make_int2(kWide, kWide)
                                                                     : make_int2(exponent(ke), exponent(ve));
          mbar_arrive(bar(POWERS + (s & 3u)));
        }
        if (s > 0) wait(bar(Q_FREE), (s - 1) & 1u, abort_flag);
        if (__any_sync(0xffffffffu, *abort_flag)) break;
        ++s;
        const int nt = walk.tiles(c), tok = c.s.q0 + c.it.r0 / G;
        if (lane == 0) {
          mbar_expect_tx(bar(Q_READY), static_cast<uint32_t>(nt * (D / 64) * TR * 128));
#pragma unroll 1
          for (int i = 0; i < nt * (D / 64); ++i) {
            const int t = i / (D / 64), half = i % (D / 64);
            tma_load_4d(base + M::kQ + t * M::kTile + half * kTileHalf, &qmap, 64 * half, 0, c.h, tok + t * p.TT,
                        bar(Q_READY));
          }
        }
      }
      if (*abort_flag && lane == 0 && s > 0) drain(bar(Q_READY), (s - 1) & 1u);
    } else if (warp == 3) {
      // ======================= the CTA's form =======================
      // The largest and smallest scales over its sequences (of any head) say whether
      // a segment can be wide: only then do the decode and softmax warps run the
      // bodies that know that form.
      const int b0 = plan_item(walk.v, find_item(walk.v, H, wr.g0)).b,
                b1 = plan_item(walk.v, find_item(walk.v, H, wr.g1 - 1)).b;
      const uint32_t* tops = p.tops + static_cast<long long>(b0) * H * (4 * kParts);
      uint32_t most = 0u, least = 0u;                     // of lanes below kParts K's, of the others V's
      const int n = lane % kParts < p.parts ? (b1 - b0 + 1) * H : 0;
#pragma unroll 1
      for (int i = 0; i < n; i += 8) {                    // (past the last one: the last one again)
        uint32_t x[8], y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t* at = tops + static_cast<long long>(min(i + e, n - 1)) * (4 * kParts) + lane;
          x[e] = __ldcg(at);
          y[e] = __ldcg(at + 2 * kParts);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          most = max(most, x[e]);
          least = max(least, y[e]);
        }
      }
      __syncwarp();
      bool wide = false;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const bool mine = lane / kParts == i;
        wide |= spread_wide(__reduce_max_sync(0xffffffffu, mine ? most : 0u),
                            kInfBits - __reduce_max_sync(0xffffffffu, mine ? least : 0u));
      }
      if (lane == 0) {
        *reinterpret_cast<volatile int*>(sm + M::kMisc + 8) = wide;
        mbar_arrive(bar(FORM));
      }
    } else if (warp >= 4) {
      const Cta<BITS, D> cta{p, walk, wr, sm, base, tmem};
      wait(bar(FORM), 0u, abort_flag);
      const bool wide = *reinterpret_cast<volatile int*>(sm + M::kMisc + 8) != 0;
      if (wide) wide_roles<BITS, D>(cta);
      else if (warp >= 12) decode_role<BITS, D, false>(cta);
      else softmax_role<BITS, D, false>(cta);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && *abort_flag) record_error(p.err, KVQ_ERR_TIMEOUT);
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
int tile_tokens(const AttendArgs& a) { return 128 / a.G; }
// Rows of an item: one tile where no sequence has more, else two.
int item_rows(const AttendArgs& a) {
  const int tr = tile_tokens(a) * a.G;
  return static_cast<long long>(a.max_q) * a.G > tr ? 2 * tr : tr;
}
template <int D>
size_t smem_bytes(const AttendArgs& a) {
  return 1024 + Smem<D>::kPre + (plan_inline(a, item_rows(a)) ? sizeof(long long) * (a.S + 1) : 0);
}
size_t smem_of(const AttendArgs& a) { return a.g.D == 64 ? smem_bytes<64>(a) : smem_bytes<128>(a); }

int ctas(const AttendArgs& a) { return a.splits > 0 ? a.splits : (sm_count() > 0 ? sm_count() : 148); }

// Below these rows a KV head the rows kernel is faster (16 sequences of 4096 keys,
// D = 128, us: rows / this one): 4 bits 8 rows 43 / 88, 16 rows 81 / 89, 20 rows
// 110 / 89; 8 bits 8 rows 59 / 87, 9 rows 106 / 87 (the rows kernel's second tile).
bool applies(const AttendArgs& a) {
  return a.g.group == 32 && (a.g.D == 64 || a.g.D == 128) && a.q_dtype == KVQ_BF16 && a.G <= 128 &&
         static_cast<long long>(a.max_q) * a.G > (a.g.bits == 4 ? 16 : 8) && smem_of(a) <= 227 * 1024;
}
size_t partials_bytes(const AttendArgs& a) {
  return 2 * static_cast<size_t>(ctas(a)) * 256 * (a.g.D + 2) * sizeof(float);
}
// workspace: the plan, partial results, fp16 query rows and their powers, largest and smallest scales
struct Layout {
  size_t partials, rows, powers, tops, bytes;
};
Layout layout(const AttendArgs& a) {
  auto up = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
  const size_t rows = static_cast<size_t>(a.T) * a.H_q;
  Layout l;
  l.partials = up(plan_bytes(a, item_rows(a)));
  l.rows = l.partials + up(partials_bytes(a));
  l.powers = l.rows + up(rows * a.g.D * 2);
  l.tops = l.powers + up(rows * sizeof(float));
  l.bytes = l.tops + 4 * sizeof(uint32_t) * kParts * a.S * a.g.H_kv;
  return l;
}
size_t workspace(const AttendArgs& a) { return layout(a).bytes; }

// cuTensorMapEncodeTiled through the runtime's driver entry point (no libcuda link)
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiled encode_tiled() {
  static EncodeTiled fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q{};
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return static_cast<EncodeTiled>(nullptr);
    return reinterpret_cast<EncodeTiled>(f);
  }();
  return fn;
}

// Q as (feature, head of the group, KV head, token); a box is a row tile's
// half: 64 features x G heads x 1 x TT tokens, rows token-major in shared
// memory with the 128-byte swizzle the UMMA descriptors expect.  Tokens past T
// read as zero.
bool make_q_map(const AttendArgs& a, void* rows, CUtensorMap* map) {
  const EncodeTiled enc = encode_tiled();
  if (!enc) return false;
  const cuuint64_t D = static_cast<cuuint64_t>(a.g.D), G = static_cast<cuuint64_t>(a.G),
                   H = static_cast<cuuint64_t>(a.g.H_kv);
  const cuuint64_t dims[4] = {D, G, H, static_cast<cuuint64_t>(a.T)};
  const cuuint64_t strides[3] = {D * 2, G * D * 2, H * G * D * 2};
  const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(a.G), 1, static_cast<cuuint32_t>(tile_tokens(a))};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, rows, dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

kvq_status launch(const AttendArgs& a, cudaStream_t s) {
  const int RI = item_rows(a);
  CUtensorMap qmap;
  const Layout l = layout(a);
  char* ws = static_cast<char*>(a.workspace);
  if (!make_q_map(a, ws + l.rows, &qmap)) return KVQ_ERR_CUDA;
  Params p{};
  p.t = make_batch(a);
  p.plan = plan_mem(a, RI, a.workspace);
  p.k_codes = a.k_codes;
  p.k_scales = a.k_scales;
  p.v_codes = a.v_codes;
  p.v_scales = a.v_scales;
  p.qscale = a.scale * kLog2e;
  p.O = static_cast<__nv_bfloat16*>(a.O);
  p.partials = reinterpret_cast<float*>(ws + l.partials);
  float* q_pow = reinterpret_cast<float*>(ws + l.powers);
  uint32_t* tops = reinterpret_cast<uint32_t*>(ws + l.tops);
  // four CTAs an SM where the sequences and heads alone are fewer (two: the same
  // within 1 us)
  const long long bh = static_cast<long long>(a.S) * a.g.H_kv;
  const int parts = static_cast<int>(std::min<long long>(kParts, std::max<long long>(1, (4 * 148 + bh - 1) / bh)));
  p.tops = tops;
  p.parts = parts;
  p.q_pow = q_pow;
  p.ctas = ctas(a);
  p.RI = RI;
  p.TT = tile_tokens(a);
  p.err = error_word();
  if (!p.err) return KVQ_ERR_CUDA;
  if (p.plan.count) {
    const kvq_status st = launch_plan(a, p.plan, RI, kBT, s);
    if (st != KVQ_OK) return st;
  }
  const long long rows = static_cast<long long>(a.T) * a.H_q;
  const int row_pass = 32 * kPrepareWarps / (a.g.D / 8) * kRowsPerLane;
  const long long blocks = bh * parts + (rows + row_pass - 1) / row_pass;
  if (blocks > 0x7fffffffLL) return KVQ_ERR_UNSUPPORTED;
  if (launch_pdl(a.g.D == 64 ? paged_prepare_kernel<64> : paged_prepare_kernel<128>,
                 dim3(static_cast<unsigned>(blocks)), dim3(32 * kPrepareWarps), 0, s, p.t, p.k_scales, p.v_scales, tops,
                 parts, static_cast<const uint4*>(a.Q), reinterpret_cast<uint4*>(ws + l.rows), q_pow, rows, p.plan.count != nullptr,
                 p.err) !=
      cudaSuccess)
    return KVQ_ERR_CUDA;
  count_launch();
  const size_t smem = smem_of(a);
  auto kernel = a.g.D == 64 ? (a.g.bits == 4 ? paged_chunk_kernel<4, 64> : paged_chunk_kernel<8, 64>)
                            : (a.g.bits == 4 ? paged_chunk_kernel<4, 128> : paged_chunk_kernel<8, 128>);
  if (!ensure_dynamic_smem(reinterpret_cast<const void*>(kernel), smem)) return KVQ_ERR_CUDA;
  if (launch_pdl(kernel, dim3(p.ctas), dim3(kThreads), smem, s, qmap, p) != cudaSuccess) return KVQ_ERR_CUDA;
  count_launch();
  MergeCall m{};
  m.t = p.t;
  m.plan = p.plan;
  m.items = plan_items(a, RI);
  m.RI = RI;
  m.BT = kBT;
  m.workers = p.ctas;
  m.D = a.g.D;
  m.partials = p.partials;
  m.O = a.O;
  m.o_dtype = a.q_dtype;
  m.tile_rows = p.TT * a.G;
  return launch_merge(m, s);
}

const AttendImpl kChunk{"paged_chunk_tcgen05", applies, workspace, launch};

}  // namespace

const AttendImpl& chunk_impl() { return kChunk; }

}  // namespace paged
}  // namespace kvq
