// Paged cache: append of a ragged batch of new tokens, and reading tokens back.
//
// Append.  A key row is rotated by its position -- each product and each sum
// rounded to float32, so that the bytes do not depend on who computes them --
// and packed with its K group ("KV分组打包：4-bit到底省了多少？",
// huhohoo.com/docs/llm/kv-packed-groups, sections "一个字节里到底装了什么" and
// "为什么分组要同时看方向与长度"; the quantization is quant.cuh's, the same as
// kvq_pack's).  K scales run along tokens: a group that is not full when a
// call ends is packed as if zeros followed, and its float32 rows stay in the
// sequence's tail slot for the call that brings the next token.
//
// One CTA per (touched K group, KV head): it holds the group's g x D rows in
// shared memory, so each new K and V element is read once.  The group that a
// call begins in reads the tail slot and the group that it ends in writes it;
// where these are two groups and both are unfinished, one CTA does them one
// after the other, so the slot's rows are read before they are replaced.  The
// vector form (features in eights, groups a power of two) gives K and V a CTA
// each, eight features a lane; a call of one token a sequence has V in K's.
//
// Bound by latency and issue.  8 thousand new tokens of 8 heads, D = 128, and
// reading 8 thousand back: 140 MB in 63.5 us (2.2 TB/s), captured alone 44 us the
// append (issue 47 %) and 24 the read-back (52 %).  One token of each of 64
// sequences, and their groups read back: 14.8 us, of which two launches are 10
// (groups of 8 of 9 sequences take that); captured cold, the append's 512 CTAs wait
// for instructions more than for loads (12.4 us; the read-back 9.1).  In the scalar
// form the two take 130 and 26 us; it serves the other shapes, groups of 64 among
// them (8 thousand tokens with the read-back: 184 us).
#include "f32x2.cuh"
#include "paged.cuh"
#include "quant.cuh"

namespace kvq {
namespace paged {
namespace {

constexpr int kThreads = 128;

// Unit u of a launch belongs to the sequence b with base(b) <= u < base(b + 1):
// base(b) = cu[b] / g + 2 b is an upper bound of the groups that the sequences
// before b touch (a sequence of n tokens touches at most n / g + 2, and
// floor((c + n) / g) - floor(c / g) >= floor(n / g)), which needs no sum over
// the sequences.  With at most one token a sequence, base(b) = b.
struct GroupSize {
  int g, lg;                       // lg: its logarithm where it is a power of two, else -1
  __device__ __forceinline__ int div(int x) const { return lg >= 0 ? x >> lg : x / g; }
};
__device__ __forceinline__ long long unit_base(int c, int b, int T, const GroupSize& gs) {
  return gs.div(min(max(c, 0), T)) + 2LL * b;
}
// The same for rows: base(b) = cu[b].
__device__ __forceinline__ long long row_base(int c, int T) { return min(max(c, 0), T); }

// The sequence of unit u: the largest b in [0, S) with base(cu[b], b) <= u (0
// if none), with cu[b] and cu[b + 1], by one warp.  Up to 127 sequences take one
// round of loads, four entries a lane; more take one per factor of 32.
struct Found {
  int b, c0, c1;
};
template <typename Base>
__device__ __forceinline__ Found warp_find(const int32_t* cu, int S, long long u, Base base) {
  const int lane = threadIdx.x & 31;
  Found f;
  if (S < 128) {
    int c[4], count = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = lane + 32 * k;
      c[k] = i <= S ? __ldcg(cu + i) : 0;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = lane + 32 * k;
      count += __popc(__ballot_sync(0xffffffffu, i < S && base(c[k], i) <= u));
    }
    f.b = max(count - 1, 0);
    auto entry = [&](int i) {
      const int k = i >> 5;
      return __shfl_sync(0xffffffffu, k == 0 ? c[0] : k == 1 ? c[1] : k == 2 ? c[2] : c[3], i & 31);
    };
    f.c0 = entry(f.b);
    f.c1 = entry(f.b + 1);
    return f;
  }
  int lo = 0, n = S;
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int at = lane * step;
    const bool le = at < n && base(__ldcg(cu + lo + at), lo + at) <= u;
    const int k = __popc(__ballot_sync(0xffffffffu, le));
    if (k == 0) break;
    lo += (k - 1) * step;
    n = min(step, n - (k - 1) * step);
  }
  f.b = lo;
  f.c0 = __ldcg(cu + lo);
  f.c1 = __ldcg(cu + lo + 1);
  return f;
}

struct AppendParams {
  const void* K;
  const void* V;
  long long k_stride, v_stride;
  int dtype;
  const int32_t* table;
  int max_pages;
  const int32_t* lengths;
  const int32_t* cu;
  const int32_t* slots;
  int S, T, max_new;
  const float* rope;               // [n_pos][rot]
  int n_pos, rot, interleaved;
  int bits, group, lg, D, Dp, H, P, pages, cap;    // lg: log2 of the group, or -1
  long long k_codes_head, k_scales_head, v_codes_head, v_scales_head;
  uint8_t* k_codes;
  float* k_scales;
  uint8_t* v_codes;
  float* v_scales;
  float* tail;
  int tail_slots;
  unsigned int* err;
};

template <bool kBf16>
__device__ __forceinline__ float load1(const void* p, long long i) {
  if (kBf16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  return static_cast<const float*>(p)[i];
}

// One group of one head: tokens [tok0, tok0 + g) of a sequence whose tokens
// [first, len) are new (rows row0 + token - first).
template <bool kBf16>
__device__ __forceinline__ void append_group(const AppendParams& p, float* s_x, int h, int tok0, int first, int len,
                                             int row0, int page, float* tail) {
  const int g = p.group, D = p.D;
  const int qmax = p.bits == 4 ? 7 : 127;
  const int live = min(g, len - tok0);              // rows of the group that exist
  const int kept = max(0, first - tok0);            // of these, rows from the tail slot
  for (int i = threadIdx.x; i < kept * D; i += kThreads) s_x[i] = tail[i];
  for (int i = live * D + threadIdx.x; i < g * D; i += kThreads) s_x[i] = 0.f;
  // new rows: the rotated pairs, then the features beyond the rotation
  const int half = p.rot / 2, rest = D - p.rot;
  for (int i = threadIdx.x; i < (live - kept) * half; i += kThreads) {
    const int r = kept + i / half, e = i % half;
    const int pos = tok0 + r;
    const int a = p.interleaved ? 2 * e : e, b = p.interleaved ? 2 * e + 1 : e + half;
    const long long src = static_cast<long long>(row0 + pos - first) * p.k_stride + static_cast<long long>(h) * D;
    const float x = load1<kBf16>(p.K, src + a), y = load1<kBf16>(p.K, src + b);
    float xr = x, yr = y;
    if (pos < p.n_pos) {
      const float* cs = p.rope + static_cast<long long>(pos) * p.rot;
      const float c = __ldg(cs + e), s = __ldg(cs + half + e);
      xr = __fsub_rn(__fmul_rn(x, c), __fmul_rn(y, s));
      yr = __fadd_rn(__fmul_rn(y, c), __fmul_rn(x, s));
    } else if (e == 0 && h == 0) {
      record_error(p.err, KVQ_ERR_INDEX);
    }
    s_x[r * D + a] = xr;
    s_x[r * D + b] = yr;
  }
  for (int i = threadIdx.x; i < (live - kept) * rest; i += kThreads) {
    const int r = kept + i / rest, d = p.rot + i % rest;
    s_x[r * D + d] = load1<kBf16>(
        p.K, static_cast<long long>(row0 + tok0 + r - first) * p.k_stride + static_cast<long long>(h) * D + d);
  }
  __syncthreads();
  if (live < g) {                                   // an unfinished group: its new rows are kept
    for (int i = kept * D + threadIdx.x; i < live * D; i += kThreads) tail[i] = s_x[i];
  }
  if (page >= 0) {
    const long long head = static_cast<long long>(page) * p.H + h;
    const int in_page = tok0 % p.P;
    float* s_scale = s_x + g * D;
    for (int d = threadIdx.x; d < D; d += kThreads) {
      float amax = 0.f;
      for (int t = 0; t < g; ++t) amax = fmaxf(amax, fabsf(s_x[t * D + d]));
      const float sc = group_scale(amax, qmax);
      s_scale[d] = sc;
      s_scale[D + d] = __frcp_rn(sc);
      p.k_scales[head * p.k_scales_head + static_cast<long long>(in_page / g) * D + d] = sc;
    }
    __syncthreads();
    uint8_t* out = p.k_codes + head * p.k_codes_head + static_cast<long long>(in_page) * D * p.bits / 8;
    if (p.bits == 4) {
      for (int jb = threadIdx.x; jb < g * D / 2; jb += kThreads) {
        const int f = 2 * jb, d0 = f % D, d1 = (f + 1) % D;
        const unsigned lo = quant_code(s_x[f], s_scale[d0], s_scale[D + d0], qmax);
        const unsigned hi = quant_code(s_x[f + 1], s_scale[d1], s_scale[D + d1], qmax);
        out[jb] = static_cast<uint8_t>(lo | (hi << 4));
      }
    } else {
      for (int f = threadIdx.x; f < g * D; f += kThreads)
        out[f] = static_cast<uint8_t>(quant_code(s_x[f], s_scale[f % D], s_scale[D + f % D], qmax));
    }
    // V of the group's new rows: a thread per (row, group of g features)
    const int ng = p.Dp / g;
    for (int i = threadIdx.x; i < (live - kept) * ng; i += kThreads) {
      const int r = kept + i / ng, gj = i % ng, d0 = gj * g;
      const long long src = static_cast<long long>(row0 + tok0 + r - first) * p.v_stride + static_cast<long long>(h) * D;
      float amax = 0.f;
      for (int e = 0; e < g; ++e)
        if (d0 + e < D) amax = fmaxf(amax, fabsf(load1<kBf16>(p.V, src + d0 + e)));
      const float sc = group_scale(amax, qmax), rs = __frcp_rn(sc);
      const long long tok = in_page + r;
      p.v_scales[head * p.v_scales_head + tok * ng + gj] = sc;
      uint8_t* vo = p.v_codes + head * p.v_codes_head + (tok * p.Dp + d0) * p.bits / 8;
      for (int e = 0; e < g; e += 2) {
        const float x0 = d0 + e < D ? load1<kBf16>(p.V, src + d0 + e) : 0.f;
        const float x1 = d0 + e + 1 < D ? load1<kBf16>(p.V, src + d0 + e + 1) : 0.f;
        const unsigned c0 = quant_code(x0, sc, rs, qmax), c1 = quant_code(x1, sc, rs, qmax);
        if (p.bits == 4) {
          vo[e / 2] = static_cast<uint8_t>(c0 | (c1 << 4));
        } else {
          vo[e] = static_cast<uint8_t>(c0);
          vo[e + 1] = static_cast<uint8_t>(c1);
        }
      }
    }
  }
  __syncthreads();
}

// ---------------------------------------------------------------------------
// vector form
// ---------------------------------------------------------------------------
// Eight features a thread: LPR lanes (a power of two, D / 8 of them used) hold
// a row, so a row comes with one 16-byte load a lane (two for f32), the partner
// of a rotation pair is a shuffle away, and a lane's eight codes leave as one
// word or two.  K and V have CTAs of their own (blockIdx.z): half the
// registers, twice the loads in flight.  A K CTA holds the group's rows in
// registers, PASS rows a thread; a channel's maximum goes over the thread's
// rows, the warp's and (through shared memory) the four warps'.  Arithmetic is
// on pairs (f32x2).  Needs D and the pairs' distance in whole vectors, aligned rows,
// and groups of 8 or 32, or of 16 where D is at most 128, that divide D (what
// pick_append has an instance for); append_group above takes the rest.
constexpr float kRound = 12582912.f;               // 1.5 * 2^23: x + kRound has rint(x) in its low bits

// Eight floats as four pairs.
struct Eight {
  u64 v[4];
  __device__ __forceinline__ float at(int k) const { return k & 1 ? hi_f(v[k >> 1]) : lo_f(v[k >> 1]); }
};
__device__ __forceinline__ Eight zero8() { return Eight{{0ull, 0ull, 0ull, 0ull}}; }
__device__ __forceinline__ Eight load8f(const float* p) {
  const ulonglong2 a = *reinterpret_cast<const ulonglong2*>(p), b = *reinterpret_cast<const ulonglong2*>(p + 4);
  return Eight{{a.x, a.y, b.x, b.y}};
}
__device__ __forceinline__ void store8f(float* p, const Eight& x) {
  *reinterpret_cast<ulonglong2*>(p) = make_ulonglong2(x.v[0], x.v[1]);
  *reinterpret_cast<ulonglong2*>(p + 4) = make_ulonglong2(x.v[2], x.v[3]);
}
template <bool kBf16>
__device__ __forceinline__ Eight load8(const void* p, long long i) {
  if (!kBf16) return load8f(static_cast<const float*>(p) + i);
  const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + i);
  const unsigned w[4] = {v.x, v.y, v.z, v.w};
  Eight x;
#pragma unroll
  for (int k = 0; k < 4; ++k) x.v[k] = pack2(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xFFFF0000u));
  return x;
}
__device__ __forceinline__ u64 neg2(u64 a) { return a ^ 0x8000000080000000ull; }

// Whether quantize8's fast form holds for a scale: 1 / s, and the residuals of
// quotients up to 127, stay clear of overflow and of denormals.
__device__ __forceinline__ bool plain_scale(float s) { return s > 1e-28f && s < 1e28f; }

// Quantizes eight values (scale s, reciprocal rs = 1 / s rounded to nearest)
// and stores their codes at flat code index i, a multiple of 8.
// The codes are rint of the quotient rounded to f32 (quant.cuh).  That quotient
// comes without a division from Markstein's theorem (P. Markstein, "Computation
// of elementary functions on the IBM RISC System/6000 processor", 1990): if q is
// within an ulp of x / s and r = x - q s is exact, q + r rs rounds to the
// rounded quotient; x rs is within two ulps, the first correction brings it
// within one.  Adding kRound leaves rint in the sum's low bits, so the codes of
// a word add up as integers: sum over k of bits_k * 2^(bits k), corrected by
// one constant.  Values that are not finite, and scales outside plain_scale,
// take quant_code.
__device__ __forceinline__ void quantize8(uint8_t* out, long long i, const Eight& x, const Eight& s, const Eight& rs,
                                          int bits, bool plain) {
  const u64 r2 = pack2(kRound, kRound);
  unsigned b[8];
  if (plain) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const u64 ms = neg2(s.v[k]);
      u64 q = mul2(x.v[k], rs.v[k]);
      q = fma2(fma2(q, ms, x.v[k]), rs.v[k], q);
      q = fma2(fma2(q, ms, x.v[k]), rs.v[k], q);
      const u64 t = add2(q, r2);
      b[2 * k] = static_cast<unsigned>(t);
      b[2 * k + 1] = static_cast<unsigned>(t >> 32);
    }
  } else {
    const int qmax = bits == 4 ? 7 : 127;
#pragma unroll
    for (int k = 0; k < 8; ++k) b[k] = 0x4B400000u + quant_code(x.at(k), s.at(k), __frcp_rn(s.at(k)), qmax) - qmax;
  }
  if (bits == 4) {
    unsigned w = 0x77777777u - 0x4B400000u * 0x11111111u;
#pragma unroll
    for (int k = 0; k < 8; ++k) w += b[k] << (4 * k);
    *reinterpret_cast<unsigned*>(out + i / 2) = w;
  } else {
    unsigned w[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      w[j] = 0x7F7F7F7Fu - 0x4B400000u * 0x01010101u;
#pragma unroll
      for (int k = 0; k < 4; ++k) w[j] += b[4 * j + k] << (8 * k);
    }
    *reinterpret_cast<uint2*>(out + i) = make_uint2(w[0], w[1]);
  }
}
// Whether the sum of eight values is finite (so each of them is).
__device__ __forceinline__ u64 sum4(const Eight& x) { return add2(add2(x.v[0], x.v[1]), add2(x.v[2], x.v[3])); }
__device__ __forceinline__ bool finite2(u64 a) { return fabsf(lo_f(a)) < INFINITY && fabsf(hi_f(a)) < INFINITY; }

// A group's place in the pages and in the call.
struct GroupAt {
  int tok0, first, len, row0;
};

// A lane's eight features of a V row, given its group's maximum, or its scale.
__device__ __forceinline__ void store_v_scaled(const AppendParams& p, long long head, long long tok, int d0,
                                               const Eight& x, float sc) {
  const float rs = __frcp_rn(sc);
  if ((d0 & (p.group - 1)) == 0) p.v_scales[head * p.v_scales_head + tok * (p.D >> p.lg) + (d0 >> p.lg)] = sc;
  Eight s8, r8;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    s8.v[k] = pack2(sc, sc);
    r8.v[k] = pack2(rs, rs);
  }
  quantize8(p.v_codes + head * p.v_codes_head, tok * p.D + d0, x, s8, r8, p.bits,
            plain_scale(sc) && finite2(sum4(x)));
}
__device__ __forceinline__ void store_v_row(const AppendParams& p, long long head, long long tok, int d0,
                                            const Eight& x, float top) {
  store_v_scaled(p, head, tok, d0, x, group_scale(top, p.bits == 4 ? 7 : 127));
}

template <bool kBf16, int LPR, int PASS>
__device__ __forceinline__ void append_k_vec(const AppendParams& p, float* s_max, int h, const GroupAt& a,
                                             const int32_t* table, float* tail, bool with_v) {
  constexpr int RPP = kThreads / LPR;              // rows of a pass
  const int g = p.group, D = p.D;
  const int qmax = p.bits == 4 ? 7 : 127;
  const int warp = threadIdx.x >> 5;
  const int l = threadIdx.x % LPR, slot = threadIdx.x / LPR, d0 = 8 * l;
  const bool on = l < D / 8;
  const int live = min(g, a.len - a.tok0), kept = max(0, a.first - a.tok0);
  int page = __ldg(table + a.tok0 / p.P);
  Eight x[PASS];
#pragma unroll
  for (int q = 0; q < PASS; ++q) {
    const int r = q * RPP + slot;
    x[q] = zero8();
    if (on && r < live) {
      if (r < kept) x[q] = load8f(tail + r * D + d0);
      else x[q] = load8<kBf16>(p.K, (a.row0 + a.tok0 + r - a.first) * p.k_stride + static_cast<long long>(h) * D + d0);
    }
  }
  // a call of one token a sequence: its V row is the same CTA's
  const bool v_on = with_v && on && slot == 0;
  Eight v = zero8();
  if (v_on) v = load8<kBf16>(p.V, (a.row0 + a.tok0 + kept - a.first) * p.v_stride + static_cast<long long>(h) * D + d0);
  if (p.rot > 0) {
    const int half = p.rot / 2;
    const bool turns = on && d0 < p.rot, upper = !p.interleaved && d0 >= half;
    const int lane = threadIdx.x & 31;
    const int partner = p.interleaved || !turns ? lane : (upper ? lane - half / 8 : lane + half / 8);
    // a pair's first feature becomes x c - y s, its second y c + x s
    Eight c, s;
    auto angles = [&](int pos) {
      const float* tab = p.rope + static_cast<long long>(pos) * p.rot;
      if (p.interleaved) {
        const float4 cv = __ldg(reinterpret_cast<const float4*>(tab + d0 / 2));
        const float4 sv = __ldg(reinterpret_cast<const float4*>(tab + half + d0 / 2));
        const float cc[4] = {cv.x, cv.y, cv.z, cv.w}, ss[4] = {sv.x, sv.y, sv.z, sv.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          c.v[k] = pack2(cc[k], cc[k]);
          s.v[k] = pack2(ss[k], ss[k]);
        }
      } else {
        const int e = upper ? d0 - half : d0;
        c = load8f(tab + e);
        s = load8f(tab + half + e);
      }
    };
    // the thread's first new row's are asked for before its rows are waited for
    const int q_first = max(0, (kept - slot + RPP - 1) / RPP);
    if (turns && a.tok0 + q_first * RPP + slot < min(a.len, p.n_pos)) angles(a.tok0 + q_first * RPP + slot);
#pragma unroll
    for (int q = 0; q < PASS; ++q) {
      const int r = q * RPP + slot, pos = a.tok0 + r;
      const bool fresh = r >= kept && r < live, turn = turns && fresh && pos < p.n_pos;
      if (fresh && pos >= p.n_pos && l == 0 && h == 0) record_error(p.err, KVQ_ERR_INDEX);
      Eight o;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        o.v[k] = p.interleaved ? (x[q].v[k] << 32 | x[q].v[k] >> 32) : __shfl_sync(0xffffffffu, x[q].v[k], partner);
      if (turn) {
        if (q != q_first) angles(pos);
        const u64 flip = p.interleaved ? 0x0000000080000000ull : (upper ? 0ull : 0x8000000080000000ull);
        // (-s) y added is s y subtracted, bit for bit; scalar operations, since
        // a packed product and sum may become one rounding
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const u64 sk = s.v[k] ^ flip;
          x[q].v[k] = pack2(__fadd_rn(__fmul_rn(x[q].at(2 * k), c.at(2 * k)), __fmul_rn(o.at(2 * k), lo_f(sk))),
                            __fadd_rn(__fmul_rn(x[q].at(2 * k + 1), c.at(2 * k + 1)),
                                      __fmul_rn(o.at(2 * k + 1), hi_f(sk))));
        }
      }
    }
  }
  if (live < g) {                                  // an unfinished group: its new rows are kept
#pragma unroll
    for (int q = 0; q < PASS; ++q) {
      const int r = q * RPP + slot;
      if (on && r >= kept && r < live) store8f(tail + r * D + d0, x[q]);
    }
  }
  if (static_cast<unsigned>(page) >= static_cast<unsigned>(p.pages)) {
    if (threadIdx.x == 0) record_error(p.err, KVQ_ERR_INDEX);
    return;
  }
  const long long head = static_cast<long long>(page) * p.H + h;
  const int in_page = a.tok0 % p.P;
  if (with_v && threadIdx.x < 32) {                // (the row's lanes are the warp's first)
    float m = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) m = fmaxf(m, fabsf(v.at(k)));
    for (int o = 1; o < g >> 3; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (v_on) store_v_row(p, head, in_page + kept, d0, v, m);
  }
  // a channel's maximum over the group's rows
  float top[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    top[k] = 0.f;
#pragma unroll
    for (int q = 0; q < PASS; ++q) top[k] = fmaxf(top[k], fabsf(x[q].at(k)));
#pragma unroll
    for (int o = LPR; o < 32; o <<= 1) top[k] = fmaxf(top[k], __shfl_xor_sync(0xffffffffu, top[k], o));
  }
  if (on && (threadIdx.x & 31) < LPR) {
    *reinterpret_cast<float4*>(s_max + warp * D + d0) = make_float4(top[0], top[1], top[2], top[3]);
    *reinterpret_cast<float4*>(s_max + warp * D + d0 + 4) = make_float4(top[4], top[5], top[6], top[7]);
  }
  __syncthreads();
  // a thread turns one channel's maximum into its scale (D <= 256: two a thread)
  float* s_scale = s_max + 4 * D;                  // [D], then the reciprocals
  for (int d = threadIdx.x; d < D; d += kThreads) {
    const float m = fmaxf(fmaxf(s_max[d], s_max[D + d]), fmaxf(s_max[2 * D + d], s_max[3 * D + d]));
    const float sc = group_scale(m, qmax);
    s_scale[d] = sc;
    s_scale[D + d] = __frcp_rn(sc);
    p.k_scales[head * p.k_scales_head + static_cast<long long>(in_page >> p.lg) * D + d] = sc;
  }
  __syncthreads();
  if (!on) return;
  const Eight sc = load8f(s_scale + d0), rs = load8f(s_scale + D + d0);
  u64 sum = sum4(x[0]);
#pragma unroll
  for (int q = 1; q < PASS; ++q) sum = add2(sum, sum4(x[q]));
  bool plain = finite2(sum);
#pragma unroll
  for (int k = 0; k < 8; ++k) plain = plain && plain_scale(sc.at(k));
  uint8_t* out = p.k_codes + head * p.k_codes_head;
  const long long at = static_cast<long long>(in_page) * D + d0;
#pragma unroll
  for (int q = 0; q < PASS; ++q) {
    const int r = q * RPP + slot;
    if (r < g) quantize8(out, at + r * D, x[q], sc, rs, p.bits, plain);
  }
}

// V rows of the group's new tokens: a group of g features is g / 8 neighbouring
// lanes of the row.
template <bool kBf16, int LPR, int PASS>
__device__ __forceinline__ void append_v_vec(const AppendParams& p, int h, const GroupAt& a, const int32_t* table) {
  constexpr int RPP = kThreads / LPR;
  const int g = p.group, D = p.D;
  const int qmax = p.bits == 4 ? 7 : 127;
  const int l = threadIdx.x % LPR, slot = threadIdx.x / LPR, d0 = 8 * l;
  const bool on = l < D / 8;
  const int live = min(g, a.len - a.tok0), kept = max(0, a.first - a.tok0);
  const int page = __ldg(table + a.tok0 / p.P);
  Eight x[PASS];
#pragma unroll
  for (int q = 0; q < PASS; ++q) {
    const int r = q * RPP + slot;
    x[q] = zero8();
    if (on && r >= kept && r < live)
      x[q] = load8<kBf16>(p.V, (a.row0 + a.tok0 + r - a.first) * p.v_stride + static_cast<long long>(h) * D + d0);
  }
  if (static_cast<unsigned>(page) >= static_cast<unsigned>(p.pages)) return;   // the K CTA records it
  const long long head = static_cast<long long>(page) * p.H + h;
  const int in_page = a.tok0 % p.P;
  // a group's lanes divide its rows' scales: lane q the one of pass q
  const int lanes = g >> 3, own = l & (lanes - 1);
  float mx[PASS], top = 0.f;
#pragma unroll
  for (int q = 0; q < PASS; ++q) {
    float m = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) m = fmaxf(m, fabsf(x[q].at(k)));
    for (int o = 1; o < lanes; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    mx[q] = m;
    if (q == own) top = m;
  }
  const float scale = group_scale(top, qmax);
#pragma unroll
  for (int q = 0; q < PASS; ++q) {
    const int r = q * RPP + slot;
    const float sc = lanes >= PASS ? __shfl_sync(0xffffffffu, scale, (threadIdx.x & 31) - own + q)
                                   : group_scale(mx[q], qmax);
    if (on && r >= kept && r < live) store_v_scaled(p, head, in_page + r, d0, x[q], sc);
  }
}

template <bool kBf16, int LPR, int PASS>
__global__ void __launch_bounds__(kThreads, LPR == 0 || PASS == 8 ? 3 : 6) paged_append_kernel(AppendParams p) {
  griddep_wait();
  // LPR = 0: append_group's [g][D], scale[D], 1/scale[D]; else [4 warps][D]
  // maxima, scale[D], 1/scale[D]
  extern __shared__ __align__(16) float s_x[];
  const long long u = blockIdx.x;
  const int h = blockIdx.y, g = p.group;
  const bool v_part = blockIdx.z != 0;              // K has a CTA of its own (LPR > 0)
  const GroupSize gs{g, LPR > 0 ? max(p.lg, 0) : p.lg};       // (the vector form's groups are powers of two)
  const bool single = p.max_new == 1;
  Found f{static_cast<int>(u), 0, 0};
  if (single) {
    f.c0 = __ldcg(p.cu + f.b);
    f.c1 = __ldcg(p.cu + f.b + 1);
  } else {
    f = warp_find(p.cu, p.S, u, [&](int c, int i) { return unit_base(c, i, p.T, gs); });
  }
  const int b = f.b;
  const int len = __ldg(p.lengths + b), slot = p.slots ? __ldg(p.slots + b) : b;
  const RowRange rr = row_range(f.c0, f.c1, p.T, p.max_new);
  const int j = single ? 0 : static_cast<int>(u - unit_base(f.c0, b, p.T, gs));
  if (j < 0) return;                                // before the first sequence's rows
  const bool report = threadIdx.x == 0 && j == 0 && h == 0 && !v_part;
  if (rr.bad && report) record_error(p.err, KVQ_ERR_LENGTH);
  if (rr.n == 0) return;
  if (len < rr.n || len > p.cap) {
    if (report) record_error(p.err, KVQ_ERR_LENGTH);
    return;
  }
  if (static_cast<unsigned>(slot) >= static_cast<unsigned>(p.tail_slots)) {
    if (report) record_error(p.err, KVQ_ERR_INDEX);
    return;
  }
  const int first = len - rr.n;
  const int j0 = gs.div(first), last = gs.div(len - 1) - j0;
  if (j > last) return;
  const int32_t* table = p.table + static_cast<long long>(b) * p.max_pages;
  if constexpr (LPR > 0) {
    if (v_part) {
      append_v_vec<kBf16, LPR, PASS>(p, h, GroupAt{(j0 + j) * g, first, len, rr.r0}, table);
      return;
    }
  }
  // both ends unfinished: the CTA of the first group does the last one too
  const bool joined = last > 0 && j0 * g != first && gs.div(len) * g != len;
  if (joined && j == last) return;
  float* tail = p.tail + (static_cast<long long>(slot) * p.H + h) * g * p.D;
  for (int k = j; k <= last; k += joined && j == 0 ? last : last + 1) {
    const GroupAt at{(j0 + k) * g, first, len, rr.r0};
    if constexpr (LPR == 0) {
      int page = __ldg(table + at.tok0 / p.P);
      if (static_cast<unsigned>(page) >= static_cast<unsigned>(p.pages)) {
        if (threadIdx.x == 0) record_error(p.err, KVQ_ERR_INDEX);
        page = -1;
      }
      append_group<kBf16>(p, s_x, h, at.tok0, first, len, rr.r0, page, tail);
    } else {
      append_k_vec<kBf16, LPR, PASS>(p, s_x, h, at, table, tail, single);
      __syncthreads();                              // the tail rows were read, the shared maxima too
    }
  }
}

// ---------------------------------------------------------------------------
// gather
// ---------------------------------------------------------------------------
struct GatherParams {
  const int32_t* table;
  int max_pages;
  const int32_t* starts;
  const int32_t* cu;
  int S, T, max_rows;
  int bits, group, D, Dp, H, P, pages, cap;
  long long k_codes_head, k_scales_head, v_codes_head, v_scales_head;
  const uint8_t* k_codes;
  const float* k_scales;
  const uint8_t* v_codes;
  const float* v_scales;
  void* K;
  void* V;
  int dtype;
  unsigned int* err;
};

__device__ __forceinline__ float value_at(const uint8_t* codes, long long flat, int bits, float scale) {
  const int c = bits == 8 ? codes[flat] - 127 : ((codes[flat >> 1] >> ((flat & 1) * 4)) & 15) - 7;
  return __fmul_rn(static_cast<float>(c), scale);
}

// W (8 or 4) consecutive codes from flat index i, a multiple of W, as they lie in memory.
template <int W>
__device__ __forceinline__ uint2 load_codes(const uint8_t* codes, long long i, int bits) {
  if (bits == 8) {
    if (W == 8) return __ldg(reinterpret_cast<const uint2*>(codes + i));
    return make_uint2(__ldg(reinterpret_cast<const unsigned*>(codes + i)), 0u);
  }
  if (W == 8) return make_uint2(__ldg(reinterpret_cast<const unsigned*>(codes + i / 2)), 0u);
  return make_uint2(__ldg(reinterpret_cast<const unsigned short*>(codes + i / 2)), 0u);
}
// Code k of them, less qmax.
__device__ __forceinline__ float code_at(const uint2& w, int k, int bits) {
  if (bits == 8) return static_cast<float>(static_cast<int>(((k < 4 ? w.x : w.y) >> (8 * (k & 3))) & 255u) - 127);
  return static_cast<float>(static_cast<int>((w.x >> (4 * k)) & 15u) - 7);
}
template <int W>
__device__ __forceinline__ void store_values(void* p, long long i, const float (&x)[W], int dtype) {
  if (dtype == KVQ_F32) {
#pragma unroll
    for (int k = 0; k < W; k += 4)
      *reinterpret_cast<float4*>(static_cast<float*>(p) + i + k) = make_float4(x[k], x[k + 1], x[k + 2], x[k + 3]);
    return;
  }
  unsigned u[W / 2];
#pragma unroll
  for (int k = 0; k < W; k += 2) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(x[k], x[k + 1]);
    u[k / 2] = *reinterpret_cast<const unsigned*>(&a);
  }
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p) + i;
  if constexpr (W == 8) *reinterpret_cast<uint4*>(out) = make_uint4(u[0], u[1], u[2], u[3]);
  else *reinterpret_cast<uint2*>(out) = make_uint2(u[0], u[1]);
}

// A CTA takes kGatherRows rows: a warp finds each row's page, then a thread
// takes W features (8, 4 or 1) of one head of all the rows: first every row's
// loads, then the values and stores, so that no load waits for another's row.
// (Append and read-back of 8 thousand tokens: 68 us with four rows, 63 with two, 65
// with one.)
constexpr int kGatherRows = 2, kGatherThreads = 128;
template <int W>
__global__ void __launch_bounds__(kGatherThreads, 8) paged_gather_kernel(GatherParams p) {
  griddep_wait();
  __shared__ int s_page[kGatherRows], s_at[kGatherRows], s_group[kGatherRows];
  const long long row0 = static_cast<long long>(blockIdx.x) * kGatherRows;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp < kGatherRows) {
    const long long row = row0 + warp;
    int page = -1, at = -1;                         // at < 0: a zero row; page < 0: no sequence's row
    if (row < p.T) {
      const Found f = warp_find(p.cu, p.S, row, [&](int c, int) { return row_base(c, p.T); });
      const int b = f.b;
      const RowRange rr = row_range(f.c0, f.c1, p.T, p.max_rows);
      if (lane == 0 && rr.bad) record_error(p.err, KVQ_ERR_LENGTH);
      if (row >= rr.r0 && row < rr.r0 + rr.n) {
        const int start = __ldg(p.starts + b);
        const long long tok = static_cast<long long>(start) + (row - rr.r0);
        page = 0;
        if (start >= 0 && tok < p.cap) {
          page = read_page(__ldg(p.table + static_cast<long long>(b) * p.max_pages + tok / p.P), p.pages, p.err);
          at = static_cast<int>(tok % p.P);
        } else if (lane == 0) {
          record_error(p.err, KVQ_ERR_LENGTH);
        }
      }
    }
    if (lane == 0) {
      s_page[warp] = page;
      s_at[warp] = at;
      s_group[warp] = max(at, 0) / p.group;
    }
  }
  __syncthreads();
  const int per_head = p.D / W, width = p.H * p.D, vgs = p.Dp / p.group;
  for (int i = threadIdx.x; i < p.H * per_head; i += kGatherThreads) {
    const int h = i / per_head, d = (i - h * per_head) * W, vg = d / p.group;
    if constexpr (W > 1) {
      uint2 kc[kGatherRows], vc[kGatherRows];
      float4 ks[kGatherRows][W / 4];
      float vs[kGatherRows];
#pragma unroll
      for (int k = 0; k < kGatherRows; ++k) {
        const long long head = static_cast<long long>(max(s_page[k], 0)) * p.H + h, t = max(s_at[k], 0);
        if (s_page[k] < 0) continue;
        if (p.K) {
          kc[k] = load_codes<W>(p.k_codes + head * p.k_codes_head, t * p.D + d, p.bits);
          const float* at = p.k_scales + head * p.k_scales_head + static_cast<long long>(s_group[k]) * p.D + d;
#pragma unroll
          for (int e = 0; e < W / 4; ++e) ks[k][e] = __ldg(reinterpret_cast<const float4*>(at) + e);
        }
        if (p.V) {
          vc[k] = load_codes<W>(p.v_codes + head * p.v_codes_head, t * p.Dp + d, p.bits);
          vs[k] = __ldg(p.v_scales + head * p.v_scales_head + t * vgs + vg);
        }
      }
#pragma unroll
      for (int k = 0; k < kGatherRows; ++k) {
        if (s_page[k] < 0) continue;
        const long long o = (row0 + k) * width + h * p.D + d;
        const bool zero = s_at[k] < 0;
        float x[W];
        if (p.K) {
#pragma unroll
          for (int e = 0; e < W; ++e) {
            const float4& s4 = ks[k][e / 4];
            const float sc = (e & 3) == 0 ? s4.x : (e & 3) == 1 ? s4.y : (e & 3) == 2 ? s4.z : s4.w;
            x[e] = zero ? 0.f : __fmul_rn(code_at(kc[k], e, p.bits), sc);
          }
          store_values<W>(p.K, o, x, p.dtype);
        }
        if (p.V) {
#pragma unroll
          for (int e = 0; e < W; ++e) x[e] = zero ? 0.f : __fmul_rn(code_at(vc[k], e, p.bits), vs[k]);
          store_values<W>(p.V, o, x, p.dtype);
        }
      }
    } else {
#pragma unroll
      for (int k = 0; k < kGatherRows; ++k) {
        const int page = s_page[k], at = s_at[k];
        if (page < 0) continue;
        const long long head = static_cast<long long>(page) * p.H + h, t = max(at, 0);
        const long long o = (row0 + k) * width + h * p.D + d;
        const float kv = value_at(p.k_codes + head * p.k_codes_head, t * p.D + d, p.bits,
                                  p.k_scales[head * p.k_scales_head + static_cast<long long>(s_group[k]) * p.D + d]);
        const float vv = value_at(p.v_codes + head * p.v_codes_head, t * p.Dp + d, p.bits,
                                  p.v_scales[head * p.v_scales_head + t * vgs + vg]);
        if (p.K) store_from_f32(p.K, o, at >= 0 ? kv : 0.f, p.dtype);
        if (p.V) store_from_f32(p.V, o, at >= 0 ? vv : 0.f, p.dtype);
      }
    }
  }
}

template <typename P>
void fill_geometry(const Geometry& g, int max_pages, P* p) {
  p->max_pages = max_pages;
  p->bits = g.bits;
  p->group = g.group;
  p->D = g.D;
  p->Dp = g.Dp;
  p->H = g.H_kv;
  p->P = g.N_cap;
  p->pages = g.B;
  p->cap = max_pages * g.N_cap;
  p->k_codes_head = static_cast<long long>(g.k_codes_head);
  p->k_scales_head = static_cast<long long>(g.k_scales_head);
  p->v_codes_head = static_cast<long long>(g.v_codes_head);
  p->v_scales_head = static_cast<long long>(g.v_scales_head);
}

// Whether the vector form's conditions hold but for the group's size, which
// pick_append knows (figures of both forms at the top).
bool vector_form(const AppendCall& a) {
  const int D = a.g.D, g = a.g.group;
  const size_t es = a.in_dtype == KVQ_BF16 ? 2 : 4;
  auto aligned = [&](const void* p, long long stride) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && static_cast<size_t>(stride) * es % 16 == 0;
  };
  if (D % 8 != 0 || D < 8 || D > 256 || g < 8 || (g & (g - 1)) != 0 || D % g != 0) return false;
  if (!aligned(a.K, a.k_stride) || !aligned(a.V, a.v_stride)) return false;
  if (!a.rope.table) return true;
  // whole vectors of pairs, and 16-byte rows of the table
  return a.rope.rot_dim % (a.rope.interleaved ? 8 : 16) == 0 && reinterpret_cast<uintptr_t>(a.rope.table) % 16 == 0;
}

template <bool kBf16>
auto pick_append(int lpr, int pass) -> void (*)(AppendParams) {
  if (pass == 1 && lpr == 8) return paged_append_kernel<kBf16, 8, 1>;
  if (pass == 1 && lpr == 16) return paged_append_kernel<kBf16, 16, 1>;
  if (pass == 2 && lpr == 8) return paged_append_kernel<kBf16, 8, 2>;
  if (pass == 2 && lpr == 16) return paged_append_kernel<kBf16, 16, 2>;
  if (pass == 2 && lpr == 32) return paged_append_kernel<kBf16, 32, 2>;
  if (pass == 4 && lpr == 16) return paged_append_kernel<kBf16, 16, 4>;
  if (pass == 8 && lpr == 32) return paged_append_kernel<kBf16, 32, 8>;
  return nullptr;
}

}  // namespace

kvq_status launch_append(const AppendCall& a, cudaStream_t s) {
  AppendParams p{};
  fill_geometry(a.g, a.max_pages, &p);
  p.K = a.K;
  p.V = a.V;
  p.k_stride = a.k_stride;
  p.v_stride = a.v_stride;
  p.dtype = a.in_dtype;
  p.table = a.table;
  p.lengths = a.lengths;
  p.cu = a.cu;
  p.slots = a.slots;
  p.S = a.S;
  p.T = a.T;
  p.max_new = a.max_new;
  p.rope = a.rope.table;
  p.n_pos = a.rope.n_pos;
  p.rot = a.rope.table ? a.rope.rot_dim : 0;
  p.interleaved = a.rope.interleaved;
  p.lg = -1;
  for (int k = 0; k < 31; ++k)
    if (a.g.group == 1 << k) p.lg = k;
  p.k_codes = a.cache->pages.k_codes;
  p.k_scales = a.cache->pages.k_scales;
  p.v_codes = a.cache->pages.v_codes;
  p.v_scales = a.cache->pages.v_scales;
  p.tail = a.cache->k_tail;
  p.tail_slots = a.cache->tail_slots;
  p.err = error_word();
  if (!p.err) return KVQ_ERR_CUDA;
  const long long units = a.max_new == 1 ? a.S : static_cast<long long>(a.T) / a.g.group + 2LL * a.S;
  if (units > 0x7fffffffLL) return KVQ_ERR_UNSUPPORTED;
  void (*kernel)(AppendParams) = nullptr;
  size_t smem = 6 * static_cast<size_t>(a.g.D) * sizeof(float);
  unsigned parts = a.max_new == 1 ? 1 : 2;          // K and V, or (one token a sequence) both in one CTA
  int pass = 0, lpr = 8;
  if (vector_form(a)) {
    while (8 * lpr < a.g.D) lpr *= 2;
    pass = (a.g.group + kThreads / lpr - 1) / (kThreads / lpr);
  }
  if (a.in_dtype == KVQ_BF16) kernel = pick_append<true>(lpr, pass);
  else kernel = pick_append<false>(lpr, pass);
  if (!kernel) {
    kernel = a.in_dtype == KVQ_BF16 ? paged_append_kernel<true, 0, 0> : paged_append_kernel<false, 0, 0>;
    smem = (static_cast<size_t>(a.g.group) * a.g.D + 2 * a.g.D) * sizeof(float);
    parts = 1;
  }
  if (!ensure_dynamic_smem(reinterpret_cast<const void*>(kernel), smem)) return KVQ_ERR_CUDA;
  if (launch_pdl(kernel, dim3(static_cast<unsigned>(units), a.g.H_kv, parts), dim3(kThreads), smem, s, p) != cudaSuccess)
    return KVQ_ERR_CUDA;
  count_launch();
  return KVQ_OK;
}

kvq_status launch_gather(const GatherCall& a, cudaStream_t s) {
  GatherParams p{};
  fill_geometry(a.g, a.max_pages, &p);
  p.table = a.table;
  p.starts = a.starts;
  p.cu = a.cu;
  p.S = a.S;
  p.T = a.T;
  p.max_rows = a.max_rows;
  p.k_codes = a.cache->pages.k_codes;
  p.k_scales = a.cache->pages.k_scales;
  p.v_codes = a.cache->pages.v_codes;
  p.v_scales = a.cache->pages.v_scales;
  p.K = a.K;
  p.V = a.V;
  p.dtype = a.out_dtype;
  p.err = error_word();
  if (!p.err) return KVQ_ERR_CUDA;
  // eight or four features together: codes in one load, one V scale
  const int both = a.g.D | a.g.group;
  auto kernel = both % 8 == 0 ? paged_gather_kernel<8> : both % 4 == 0 ? paged_gather_kernel<4> : paged_gather_kernel<1>;
  if (launch_pdl(kernel, dim3((a.T + kGatherRows - 1) / kGatherRows), dim3(kGatherThreads), 0, s, p) != cudaSuccess)
    return KVQ_ERR_CUDA;
  count_launch();
  return KVQ_OK;
}

}  // namespace paged
}  // namespace kvq
