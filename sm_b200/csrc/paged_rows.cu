// Paged attention of few query rows a KV head (decode, drafted tokens): D 64
// or 128, groups of 32, 4- or 8-bit codes, bf16 or f32 rows.
//
// Both contractions run on the tensor cores (mma.sync m16n8k16, bf16 in, f32
// out) with the *codes* as the 16-row operand: integers of at most eight bits
// are exact in bf16, so no decoded value is ever formed or rounded.
//   S^T[token][row]   = sum_d (code_K[token][d] - qmax) * (q[row][d] ks[d])
//   O^T[feature][row] = sum_t (code_V[t][feature] - qmax) * (p[row][t] vs[t])
// The scales go to the other operand: K scales are one per channel of a
// 32-token group, so a group's q' = q ks is formed once for its 32 tokens; V
// scales are one per token and 32 features, so p' = p vs is formed per token
// for each 32-feature slice.  q' and p' are f32 values split into two bf16
// terms (three for f32 rows) that take neighbouring columns of the 8-column
// operand: four query rows fill a tile, and the result has the precision of
// 16 (24) bits.  The tensor cores cut their sums off instead of rounding them:
// f32 rows add them up outside (without that, rows over long contexts were 1.7e-6
// of their norm off instead of 4e-7, for 0.7 us of 16 at the time).
//
// What bounds it: at four rows a KV head a 4-bit token costs 160 bytes, 7
// cycles of one SM's share of the measured memory bandwidth, and about 27 warp
// instructions, 7 cycles at full issue; half of these take the codes apart (a
// shift and one three-input logic operation make two bf16 integers of a
// word's nibbles 16 bits apart).  Issue is 59 % busy, the integer pipe 53 %: 32
// x 4096 keys of 8 KV heads (168 MB) take 52.5 us, 3.2 TB/s; at 8 bits, where a
// byte costs fewer instructions, 455 MB take 122 us, 3.7 TB/s, 56 % of the
// measured copy rate.  Small calls (one sequence, 10.5 us) are two launches and the
// latency of a few dependent loads each.  Many f32 rows come here too, eight a pass
// over the keys: 4 x 64 rows of 32 heads over 4096 keys take 397 us.  A 32-token block of one page -- codes and
// scales -- is fetched by the warp that uses it with 16-byte asynchronous
// copies (two blocks in flight a warp), placed so that every later
// shared-memory read is free of bank conflicts.  A warp is a worker of the
// plan (paged.cuh): no barrier spans more than a warp.
//
// Softmax as in attend_chunk.cu: log2 units, a row's reference maximum moves
// only when a block outruns it by more than 8.  The running state follows
// "Block KV decoding: less workspace, more time"
// (huhohoo.com/en/docs/llm/kv-block-decode-cost, section "Do not average
// independently normalized blocks").
#include <algorithm>
#include <type_traits>

#include "f32x2.cuh"
#include "paged.cuh"

namespace kvq {
namespace paged {
namespace {

constexpr int kBT = 32;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLazy = 8.f;

struct Params {
  Batch t;
  PlanMem plan;
  const void* Q;
  const uint8_t* k_codes;
  const float* k_scales;
  const uint8_t* v_codes;
  const float* v_scales;
  float qscale;                  // scale * log2(e)
  void* O;
  float* partials;
  int workers;
  float spread;
  unsigned int* err;
};

// ---------------------------------------------------------------------------
// instructions
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// two floats to bf16, rounded toward zero / to nearest; lo in the low half
__device__ __forceinline__ uint32_t bf16_rz(float lo, float hi) {
  uint32_t r;
  asm("cvt.rz.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t bf16_rn(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t add_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ float top16(float x) { return __uint_as_float(__float_as_uint(x) & 0xFFFF0000u); }

// Nibble i of each 16-bit half of w as a bf16 pair 16 + n: the four bits land
// on mantissa bits 3..6 of 16.0 (0x4180); with 256.0 (0x4380) the pair is
// 256 + 16 n.
template <int I, bool kHigh>
__device__ __forceinline__ uint32_t nibbles(uint32_t w) {
  constexpr uint32_t magic = kHigh ? 0x43804380u : 0x41804180u;
  const uint32_t s = I == 0 ? w << 3 : w >> (4 * I - 3);
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(s), "n"(0x00780078u), "n"(magic));   // (s & mask) | magic
  return r;
}

// Nibble 0 of each half without a shift, as 128 + n.
__device__ __forceinline__ uint32_t nibbles_low(uint32_t w) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w), "n"(0x000F000Fu), "n"(0x43004300u));
  return r;
}

// ---------------------------------------------------------------------------
// layout of one warp's shared memory
// ---------------------------------------------------------------------------
// NT tiles of four query rows; NS bf16 terms of q' and p'.
template <int BITS, int D, int NT, int NS>
struct Cfg {
  static constexpr int RI = 4 * NT;                       // rows of an item
  static constexpr int RB = D * BITS / 8;                 // code bytes of a token
  static constexpr int CH = RB / 16;                      // 16-byte chunks of a token's codes
  static constexpr int FPC = 128 / BITS;                  // features of a chunk
  static constexpr int KW = RB / 16;                      // words of a token a lane holds (four lanes share a token)
  static constexpr int FL = D / 4;                        // features of a lane
  static constexpr int VG = D / 32;                       // V scale groups
  static constexpr int kOffV = 32 * RB, kOffKS = 64 * RB, kOffVS = kOffKS + 4 * D;
  static constexpr int kStage = kOffVS + 32 * VG * 4;
  static constexpr int kStages = 2;
  static constexpr int kQ = RI * D * 4;                   // the segment's q, f32
  static constexpr int kWarp = kStages * kStage + kQ;
  static constexpr int MT = D / 16;                       // 16-feature tiles of O^T
  static constexpr int SETS = NS == 3 ? 2 : 1;            // B operands: (hi, mid) and (lo, 0)
  // warps of a CTA, two CTAs to an SM where shared memory and registers allow
  static constexpr int kCtas = (NT == 1 && NS == 2 && D <= 128) ? 2 : 1;
  static constexpr int kFit = (kCtas == 2 ? 110 : 220) * 1024 / kWarp;
  static constexpr int kMost = kCtas == 2 ? 8 : (NT == 1 ? 12 : 8);
  static constexpr int kWarps = kFit < kMost ? kFit : kMost;
};

// Position of a 16-byte chunk of token t's codes within the block's 32 rows.
// K: the eight lanes of a quarter warp read two neighbouring tokens, four
// chunks each.  V: ldmatrix reads one chunk of eight consecutive tokens.
template <int CH>
__device__ __forceinline__ int k_slot(int t, int ch) {
  return CH <= 4 ? t * CH + ch : t * CH + (ch ^ ((t & 1) << 2));
}
template <int CH>
__device__ __forceinline__ int v_slot(int t, int ch) {
  if (CH == 2) return t * 2 + (ch ^ ((t >> 2) & 1));
  if (CH == 4) return t * 4 + (ch ^ ((t >> 1) & 3));
  return t * CH + (ch ^ (t & 7));
}

template <int BITS, int D, int NT, int NS>
struct Pos {
  // a place in the worker's list of blocks
  int i, h, j, nb;
  int pi, at;                     // its page's index in the sequence, its first row there
  long long left;                 // blocks from here to the worker's end
  Item it;
  SeqView s;
};

template <int BITS, int D, int NT, int NS>
__global__ void __launch_bounds__(32 * Cfg<BITS, D, NT, NS>::kWarps, Cfg<BITS, D, NT, NS>::kCtas)
    paged_rows_kernel(Params p) {
  using C = Cfg<BITS, D, NT, NS>;
  griddep_wait();
  extern __shared__ __align__(128) unsigned char smem[];
  long long* s_pre = reinterpret_cast<long long*>(smem + C::kWarps * C::kWarp);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  if (!p.plan.count) {
    if (warp == 0) warp_prefix(p.t, C::RI, kBT, s_pre);
    __syncthreads();
  }
  const PlanView v = plan_view(p.plan, s_pre, p.t.S);
  const int H = p.t.H, G = p.t.G, H_q = H * G, P = p.t.P;
  // neighbouring workers sit in different CTAs: a short list still uses every SM
  const long long w = static_cast<long long>(warp) * gridDim.x + blockIdx.x;
  const Range wr = worker_range(v, H, p.workers, w, p.spread);
  if (wr.g0 >= wr.g1) return;

  unsigned char* base = smem + warp * C::kWarp;
  float* s_q = reinterpret_cast<float*>(base + C::kStages * C::kStage);
  const uint32_t base_u = smem_u32(base);

  using Place = Pos<BITS, D, NT, NS>;
  auto enter = [&](Place& a) {                 // the item of place a
    a.it = plan_item(v, a.i);
    a.s = seq_view(p.t, a.it.b);
    a.nb = v.blocks(a.i);
  };
  auto advance = [&](Place& a) {               // the next block; true where a new segment begins
    if (--a.left == 0) return false;
    if (++a.j < a.nb) {
      if ((a.at += kBT) == P) {                // (a page holds whole blocks)
        a.at = 0;
        ++a.pi;
      }
      return false;
    }
    a.j = a.pi = a.at = 0;
    if (++a.h == H) {
      a.h = 0;
      do ++a.i;
      while (v.blocks(a.i) == 0);
      enter(a);
    }
    return true;
  };
  Place cur;
  cur.i = find_item(v, H, wr.g0);
  enter(cur);
  {
    const long long off = wr.g0 - static_cast<long long>(H) * v.pre[cur.i];
    cur.h = static_cast<int>(off / cur.nb);
    cur.j = static_cast<int>(off % cur.nb);
    cur.left = wr.g1 - wr.g0;
    cur.pi = cur.j * kBT / P;
    cur.at = cur.j * kBT - cur.pi * P;
  }

  // ---- block copies -------------------------------------------------------
  // a lane's destination offsets are the same for every block
  auto page_of = [&](const Place& a) {
    return __ldg(p.t.table + static_cast<long long>(a.it.b) * p.t.max_pages + a.pi);
  };
  auto copy = [&](const Place& a, int page, uint32_t dst) {
    page = read_page(page, p.t.pages, p.err);
    const long long head = static_cast<long long>(page) * H + a.h;
    const long long tok = head * P + a.at;                     // the page's arrays are dense: token rows of all heads
    const uint8_t* kc = p.k_codes + tok * C::RB + lane * 16;
    const uint8_t* vc = p.v_codes + tok * C::RB + lane * 16;
#pragma unroll
    for (int m = 0; m < C::CH; ++m) {
      const int x = m * 32 + lane, t = x / C::CH, ch = x % C::CH;
      cp16(dst + 16 * k_slot<C::CH>(t, ch), kc + m * 512);
      cp16(dst + C::kOffV + 16 * v_slot<C::CH>(t, ch), vc + m * 512);
    }
    // K scales: the lane that owns a feature finds it at [its j-th four][lane]
    const uint8_t* ks = reinterpret_cast<const uint8_t*>(p.k_scales + tok / 32 * D) + lane * 16;
#pragma unroll
    for (int m = 0; m < (D + 127) / 128; ++m) {
      const int x = m * 32 + lane;                           // features 4 x .. 4 x + 3
      int cc, jj;
      if (C::RB >= 64) {
        const int ch = 4 * x / C::FPC;
        cc = ch & 3;
        jj = (ch >> 2) * (C::FPC / 4) + x % (C::FPC / 4);
      } else {
        cc = x / (C::FL / 4);
        jj = x % (C::FL / 4);
      }
      if (x < D / 4) cp16(dst + C::kOffKS + 16 * (jj * 4 + cc), ks + m * 512);
    }
    const uint8_t* vs = reinterpret_cast<const uint8_t*>(p.v_scales + tok * C::VG) + lane * 16;
#pragma unroll
    for (int m = 0; m < (32 * C::VG + 127) / 128; ++m)
      if (m * 32 + lane < 8 * C::VG) cp16(dst + C::kOffVS + m * 512 + lane * 16, vs + m * 512);
  };

  Place ahead = cur;                            // the block to copy next
  copy(ahead, page_of(ahead), base_u);
  cp_commit();
  advance(ahead);
  int page_next = ahead.left > 0 ? page_of(ahead) : 0;

  // ---- state of a segment --------------------------------------------------
  float u[NT][C::MT][4];
  float m_ref[NT], z[NT];
  int lim[NT];                                  // keys the lane's row of each tile sees
  int full = 0;                                 // keys that every row of the item sees
  int rows = 0;
  bool first_block = true, seg_first = true;
  const bool part_b = (g & 1) != 0;
  const uint32_t split_mask = part_b ? 0xFFFF0000u : 0u;

  int stage = 0;
  for (;;) {
    if (ahead.left > 0) {
      copy(ahead, page_next, base_u + (stage ^ 1) * C::kStage);
      cp_commit();
      advance(ahead);
      if (ahead.left > 0) page_next = page_of(ahead);
    } else {
      cp_commit();                              // an empty group keeps the count
    }
    if (first_block) {
      first_block = false;
      rows = min(C::RI, cur.s.n * G - cur.it.r0);
      full = row_limit(p.t, cur.s, cur.it.r0);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int r = 4 * n + c;
        lim[n] = r < rows ? row_limit(p.t, cur.s, cur.it.r0 + r) : 0;
        m_ref[n] = -INFINITY;
        z[n] = 0.f;
#pragma unroll
        for (int m = 0; m < C::MT; ++m)
#pragma unroll
          for (int e = 0; e < 4; ++e) u[n][m][e] = 0.f;
      }
      // q of the item's rows: [tile][j][row of the tile][owner lane c][4 features]
      __syncwarp();
      for (int x = lane; x < C::RI * (D / 4); x += 32) {
        const int r = x / (D / 4), f4 = x % (D / 4);          // features 4 f4 ..
        int cc, jj;
        if (C::RB >= 64) {
          const int ch = 4 * f4 / C::FPC;
          cc = ch & 3;
          jj = (ch >> 2) * (C::FPC / 4) + f4 % (C::FPC / 4);
        } else {
          cc = f4 / (C::FL / 4);
          jj = f4 % (C::FL / 4);
        }
        float4 q = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < rows) {
          const int rr = cur.it.r0 + r;
          const long long o = (static_cast<long long>(cur.s.q0 + rr / G) * H_q + cur.h * G + rr % G) * D + 4 * f4;
          if (NS == 3) {
            q = *reinterpret_cast<const float4*>(static_cast<const float*>(p.Q) + o);
          } else {
            const uint2 b = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p.Q) + o);
            q = make_float4(__uint_as_float(b.x << 16), __uint_as_float(b.x & 0xFFFF0000u),
                            __uint_as_float(b.y << 16), __uint_as_float(b.y & 0xFFFF0000u));
          }
          q.x *= p.qscale;
          q.y *= p.qscale;
          q.z *= p.qscale;
          q.w *= p.qscale;
        }
        reinterpret_cast<float4*>(s_q)[((r >> 2) * (C::FL / 4) + jj) * 16 + (r & 3) * 4 + cc] = q;
      }
    }
    cp_wait<1>();
    __syncwarp();

    const unsigned char* st = base + stage * C::kStage;
    const uint32_t st_u = base_u + stage * C::kStage;
    const int t0 = cur.j * kBT;

    // ---- q' = q ks of this group, split over the two columns of the row ----
    uint32_t bq[NT][C::SETS][D / 8];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const float4* sq = reinterpret_cast<const float4*>(s_q) + n * (C::FL / 4) * 16 + (g >> 1) * 4 + c;
      const float4* sk = reinterpret_cast<const float4*>(st + C::kOffKS) + c;
      // one word of codes: 8 (4-bit) or 4 (8-bit) features
      constexpr int FW = 32 / BITS;
#pragma unroll
      for (int x = 0; x < C::KW; ++x) {
        float y[FW], lo[FW];
#pragma unroll
        for (int e = 0; e < FW; e += 4) {
          const int j = (x * FW + e) / 4;
          const float4 q = sq[j * 16], s = sk[j * 4];
          const u64 a0 = mul2(pack2(q.x, q.y), pack2(s.x, s.y)), a1 = mul2(pack2(q.z, q.w), pack2(s.z, s.w));
          if (NS == 2) {
            const u64 h0 = pack2(__uint_as_float(__float_as_uint(lo_f(a0)) & split_mask),
                                 __uint_as_float(__float_as_uint(hi_f(a0)) & split_mask));
            const u64 h1 = pack2(__uint_as_float(__float_as_uint(lo_f(a1)) & split_mask),
                                 __uint_as_float(__float_as_uint(hi_f(a1)) & split_mask));
            const u64 m1 = pack2(-1.f, -1.f);
            const u64 d0 = fma2(h0, m1, a0), d1 = fma2(h1, m1, a1);
            y[e] = lo_f(d0);
            y[e + 1] = hi_f(d0);
            y[e + 2] = lo_f(d1);
            y[e + 3] = hi_f(d1);
          } else {
            const float xs[4] = {lo_f(a0), hi_f(a0), lo_f(a1), hi_f(a1)};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float hi = top16(xs[k]), r1 = xs[k] - hi, mid = top16(r1);
              y[e + k] = part_b ? mid : hi;
              lo[e + k] = part_b ? 0.f : r1 - mid;
            }
          }
        }
        if (BITS == 4) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            bq[n][0][4 * x + k] = bf16_rz(y[k], y[k + FW / 2]);
            if (NS == 3) bq[n][C::SETS - 1][4 * x + k] = bf16_rz(lo[k], lo[k + FW / 2]);
          }
        } else {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            bq[n][0][2 * x + k] = bf16_rz(y[k], y[k + 2]);
            if (NS == 3) bq[n][C::SETS - 1][2 * x + k] = bf16_rz(lo[k], lo[k + 2]);
          }
        }
      }
    }

    // ---- scores of the block: lane = row c of each tile, tokens g + 8 i ------
    // The codes' offset (the operand holds 16 + n, or 256 + 16 n) is taken from the
    // operand: taken from the score instead, as that constant times the sum of q', it
    // cost a score the precision of the largest q', though its code may be zero (a
    // channel of zeros has the scale 1, one with an outlier the outlier's).
    // The tensor cores' sums are cut off, not rounded: f32 rows add them up
    // outside, rounded, a word's at a time, or the loss grows with D (and, below,
    // with the length).
    auto products = [](float (&acc)[4], const uint32_t (&a0)[4], const uint32_t (&a1)[4],
                       const uint32_t (&b)[C::SETS][D / 8], int j0, int j1) {
      if (NS == 2) {
        mma(acc, a0, b[0][j0], b[0][j0 + 1]);
        mma(acc, a1, b[0][j1], b[0][j1 + 1]);
      } else {
        float x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int set = C::SETS - 1; set >= 0; --set) {
          mma(x, a0, b[set][j0], b[set][j0 + 1]);
          mma(x, a1, b[set][j1], b[set][j1 + 1]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[e] += x[e];
      }
    };
    float sc[NT][4];
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      float acc[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[n][e] = 0.f;
      const int ta = 16 * hh + g, tb = ta + 8;
      constexpr int STEP = C::KW < 4 ? C::KW : 4;             // words of one load
#pragma unroll
      for (int x0 = 0; x0 < C::KW; x0 += STEP) {
        uint32_t wa[STEP], wb[STEP];
        if (STEP == 4) {
          const uint4 a = *reinterpret_cast<const uint4*>(st + 16 * k_slot<C::CH>(ta, c + x0));
          const uint4 b = *reinterpret_cast<const uint4*>(st + 16 * k_slot<C::CH>(tb, c + x0));
          wa[0] = a.x; wa[1] = a.y; wa[STEP - 2] = a.z; wa[STEP - 1] = a.w;
          wb[0] = b.x; wb[1] = b.y; wb[STEP - 2] = b.z; wb[STEP - 1] = b.w;
        } else {
          const uint2 a = *reinterpret_cast<const uint2*>(st + ta * C::RB + 8 * c);
          const uint2 b = *reinterpret_cast<const uint2*>(st + tb * C::RB + 8 * c);
          wa[0] = a.x; wa[STEP - 1] = a.y;
          wb[0] = b.x; wb[STEP - 1] = b.y;
        }
#pragma unroll
        for (int k = 0; k < STEP; ++k) {
          const int x = x0 + k;
          if (BITS == 4) {
            uint32_t a0[4] = {nibbles<0, false>(wa[k]), nibbles<0, false>(wb[k]), nibbles<1, false>(wa[k]),
                              nibbles<1, false>(wb[k])};
            uint32_t a1[4] = {nibbles<2, false>(wa[k]), nibbles<2, false>(wb[k]), nibbles<3, false>(wa[k]),
                              nibbles<3, false>(wb[k])};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              a0[e] = add_bf16x2(a0[e], 0xC1B8C1B8u);         // -23
              a1[e] = add_bf16x2(a1[e], 0xC1B8C1B8u);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) products(acc[n], a0, a1, bq[n], 4 * x, 4 * x + 2);
          } else {
            uint32_t a0[4] = {nibbles<0, false>(wa[k]), nibbles<0, false>(wb[k]), nibbles<2, false>(wa[k]),
                              nibbles<2, false>(wb[k])};
            uint32_t a1[4] = {nibbles<1, true>(wa[k]), nibbles<1, true>(wb[k]), nibbles<3, true>(wa[k]),
                              nibbles<3, true>(wb[k])};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              a0[e] = add_bf16x2(a0[e], 0xC1F8C1F8u);         // -31
              a1[e] = add_bf16x2(a1[e], 0xC3B8C3B8u);         // -368
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) products(acc[n], a0, a1, bq[n], 2 * x, 2 * x);
          }
        }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        sc[n][2 * hh] = acc[n][0] + acc[n][1];
        sc[n][2 * hh + 1] = acc[n][2] + acc[n][3];
      }
    }

    // ---- softmax --------------------------------------------------------------
    // (two bodies: only an item's last blocks pay for the selections)
    auto softmax_pv = [&](auto masked_c) {
    constexpr bool masked = decltype(masked_c)::value;
    bool need = false;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      if (masked) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (t0 + g + 8 * i >= lim[n]) sc[n][i] = -INFINITY;
      }
      const float mx = fmaxf(fmaxf(sc[n][0], sc[n][1]), fmaxf(sc[n][2], sc[n][3]));
      need |= mx > m_ref[n] + kLazy;
    }
    if (__any_sync(0xffffffffu, need)) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float mx = fmaxf(fmaxf(sc[n][0], sc[n][1]), fmaxf(sc[n][2], sc[n][3]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
        if (mx > m_ref[n] + kLazy) {
          const float a = ex2(m_ref[n] - mx);            // 0 where the row had no key
          m_ref[n] = mx;
          z[n] *= a;
#pragma unroll
          for (int m = 0; m < C::MT; ++m)
#pragma unroll
            for (int e = 0; e < 4; ++e) u[n][m][e] *= a;
        }
      }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool seen = !masked || t0 + g + 8 * i < lim[n];
        sc[n][i] = seen ? ex2(sc[n][i] - m_ref[n]) : 0.f;
        z[n] += sc[n][i];
      }

    // ---- O^T += V^T p', 16 tokens at a time -----------------------------------
    auto weigh = [](float (&acc)[4], const uint32_t (&a)[4], const uint32_t (&b)[C::SETS][2]) {
      if (NS == 2) {
        mma(acc, a, b[0][0], b[0][1]);
      } else {
        float x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int set = C::SETS - 1; set >= 0; --set) mma(x, a, b[set][0], b[set][1]);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[e] += x[e];
      }
    };
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      const int ta = 16 * hh + g, tb = ta + 8;
      const float* va = reinterpret_cast<const float*>(st + C::kOffVS) + ta * C::VG;
      const float* vb = va + 8 * C::VG;
#pragma unroll
      for (int fg = 0; fg < C::VG; ++fg) {
        const float sa = va[fg], sb = vb[fg];
        uint32_t bp[NT][C::SETS][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float xa = sc[n][2 * hh] * sa, xb = sc[n][2 * hh + 1] * sb;
          if (masked) {                                      // a scale past a row's keys may be anything
            if (t0 + ta >= lim[n]) xa = 0.f;
            if (t0 + tb >= lim[n]) xb = 0.f;
          }
          const float ha = top16(xa), hb = top16(xb);
          const float ra = xa - ha, rb = xb - hb;
          if (NS == 2) {
            bp[n][0][0] = transpose8(bf16_rn(ha, ra));
            bp[n][0][1] = transpose8(bf16_rn(hb, rb));
          } else {
            const float ma = top16(ra), mb = top16(rb);
            bp[n][0][0] = transpose8(bf16_rn(ha, ma));
            bp[n][0][1] = transpose8(bf16_rn(hb, mb));
            bp[n][C::SETS - 1][0] = transpose8(bf16_rn(ra - ma, 0.f));
            bp[n][C::SETS - 1][1] = transpose8(bf16_rn(rb - mb, 0.f));
          }
        }
        // the 32 features of this group: one chunk (4-bit) or two (8-bit)
        const int tr = 16 * hh + (lane & 15);
        uint32_t xr[4];
        if (BITS == 4) {
          // one chunk: tokens 0-7 and 8-15 of the half
          asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0,%1}, [%2];"
                       : "=r"(xr[0]), "=r"(xr[1])
                       : "r"(st_u + C::kOffV + 16 * v_slot<C::CH>(tr, fg))
                       : "memory");
          const uint32_t off = 0xC1B8C1B8u, off0 = 0xC307C307u;   // -23, -135
          const uint32_t a0[4] = {add_bf16x2(nibbles_low(xr[0]), off0), add_bf16x2(nibbles<1, false>(xr[0]), off),
                                  add_bf16x2(nibbles_low(xr[1]), off0), add_bf16x2(nibbles<1, false>(xr[1]), off)};
          const uint32_t a1[4] = {add_bf16x2(nibbles<2, false>(xr[0]), off), add_bf16x2(nibbles<3, false>(xr[0]), off),
                                  add_bf16x2(nibbles<2, false>(xr[1]), off), add_bf16x2(nibbles<3, false>(xr[1]), off)};
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            weigh(u[n][2 * fg], a0, bp[n]);
            weigh(u[n][2 * fg + 1], a1, bp[n]);
          }
        } else {
          ldsm4t(xr, st_u + C::kOffV + 16 * v_slot<C::CH>(tr, 2 * fg + (lane >> 4)));
          const uint32_t ol = 0xC1F8C1F8u, ol0 = 0xC30FC30Fu, oh = 0xC3B8C3B8u;   // -31, -143, -368
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint32_t xa = xr[2 * k], xb = xr[2 * k + 1];
            const uint32_t a0[4] = {add_bf16x2(nibbles_low(xa), ol0), add_bf16x2(nibbles<2, false>(xa), ol),
                                    add_bf16x2(nibbles_low(xb), ol0), add_bf16x2(nibbles<2, false>(xb), ol)};
            const uint32_t a1[4] = {add_bf16x2(nibbles<1, true>(xa), oh), add_bf16x2(nibbles<3, true>(xa), oh),
                                    add_bf16x2(nibbles<1, true>(xb), oh), add_bf16x2(nibbles<3, true>(xb), oh)};
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              weigh(u[n][2 * fg + k], a0, bp[n]);
              weigh(u[n][2 * fg + k], a1, bp[n]);
            }
          }
        }
      }
    }
    };
    if (t0 + kBT > full) softmax_pv(std::true_type{});
    else softmax_pv(std::false_type{});
    __syncwarp();                               // the stage may be overwritten

    // ---- end of a segment -------------------------------------------------------
    const Place done = cur;
    const bool last = cur.left == 1;
    const bool seg_end = advance(cur) || last;
    if (seg_end) {
      // the segment covers the (item, head) whole if it began at block 0 and ended at the last
      const bool whole = done.j == done.nb - 1 && (!seg_first || wr.g0 == static_cast<long long>(H) * v.pre[done.i] +
                                                                          static_cast<long long>(done.h) * done.nb);
      const long long slot = 2 * w + (seg_first ? 0 : 1);
      float* part = p.partials + slot * C::RI * (D + 2);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float zt = z[n];
        zt += __shfl_xor_sync(0xffffffffu, zt, 4);
        zt += __shfl_xor_sync(0xffffffffu, zt, 8);
        zt += __shfl_xor_sync(0xffffffffu, zt, 16);
        const int r = 4 * n + c;
        if (r < rows) {
          const int rr = done.it.r0 + r;
          const float inv = zt == 0.f ? 0.f : 1.f / zt;
          const long long o = (static_cast<long long>(done.s.q0 + rr / G) * H_q + done.h * G + rr % G) * D;
          if (!whole && g == 0) *reinterpret_cast<float2*>(part + C::RI * D + 2 * r) = make_float2(m_ref[n], zt);
          // 4-bit: features 32 ch + 4 g + 0..3; 8-bit: 16 ch + 2 g + 0..1
          constexpr int TPC = BITS == 4 ? 2 : 1, FV = 2 * TPC;
#pragma unroll
          for (int ch = 0; ch < C::MT / TPC; ++ch) {
            float x[FV];
#pragma unroll
            for (int k = 0; k < TPC; ++k) {
              const float(&uu)[4] = u[n][ch * TPC + k];
              x[2 * k] = uu[0] + uu[1];
              x[2 * k + 1] = uu[2] + uu[3];
            }
            const int f = ch * 8 * FV + FV * g;
            if (!whole) {
              if (FV == 4) *reinterpret_cast<float4*>(part + r * D + f) = make_float4(x[0], x[1], x[FV - 2], x[FV - 1]);
              else *reinterpret_cast<float2*>(part + r * D + f) = make_float2(x[0], x[1]);
            } else if (NS == 3) {
              float* out = static_cast<float*>(p.O) + o + f;
              if (FV == 4)
                *reinterpret_cast<float4*>(out) = make_float4(x[0] * inv, x[1] * inv, x[FV - 2] * inv, x[FV - 1] * inv);
              else *reinterpret_cast<float2*>(out) = make_float2(x[0] * inv, x[1] * inv);
            } else {
              __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.O) + o + f;
              if (FV == 4)
                *reinterpret_cast<uint2*>(out) =
                    make_uint2(bf16_rn(x[0] * inv, x[1] * inv), bf16_rn(x[FV - 2] * inv, x[FV - 1] * inv));
              else *reinterpret_cast<uint32_t*>(out) = bf16_rn(x[0] * inv, x[1] * inv);
            }
          }
        }
      }
      seg_first = false;
      first_block = true;
    }
    if (last) break;
    stage ^= 1;
  }
  cp_wait<0>();
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
template <int BITS, int D, int NT, int NS>
struct Run {
  using C = Cfg<BITS, D, NT, NS>;
  static int ctas(const AttendArgs& a) {
    return a.splits > 0 ? a.splits : C::kCtas * (sm_count() > 0 ? sm_count() : 148);
  }
  static size_t workspace(const AttendArgs& a) {
    return plan_bytes(a, C::RI) +
           2 * static_cast<size_t>(ctas(a)) * C::kWarps * C::RI * (D + 2) * sizeof(float);
  }
  static kvq_status launch(const AttendArgs& a, cudaStream_t s) {
    Params p{};
    p.t = make_batch(a);
    p.plan = plan_mem(a, C::RI, a.workspace);
    p.Q = a.Q;
    p.k_codes = a.k_codes;
    p.k_scales = a.k_scales;
    p.v_codes = a.v_codes;
    p.v_scales = a.v_scales;
    p.qscale = a.scale * kLog2e;
    p.O = a.O;
    p.partials = reinterpret_cast<float*>(static_cast<char*>(a.workspace) + plan_bytes(a, C::RI));
    // no more CTAs than a fourth of the blocks that the tables could hold (one
    // sequence of 1000 keys, 8 heads: 11.1 us with 296 CTAs, 10.6 with 64)
    const long long most = plan_items(a, C::RI) * a.g.H_kv * ((static_cast<long long>(p.t.cap) + kBT - 1) / kBT);
    const int n = a.splits > 0 ? a.splits : static_cast<int>(std::min<long long>(ctas(a), (most + 3) / 4));
    p.workers = n * C::kWarps;
    // a block of 32 keys takes about 12 times as long as joining a part (one
    // sequence of 16384 keys, 8 heads: 34 us with a worker for every two blocks, 27
    // so); the caller's own splits are as given
    p.spread = a.splits > 0 ? 0.f : 1.f / 12.f;
    p.err = error_word();
    if (!p.err) return KVQ_ERR_CUDA;
    if (p.plan.count) {
      const kvq_status st = launch_plan(a, p.plan, C::RI, kBT, s);
      if (st != KVQ_OK) return st;
    }
    const size_t smem = C::kWarps * C::kWarp + (p.plan.count ? 0 : (a.S + 1) * sizeof(long long));
    auto kernel = paged_rows_kernel<BITS, D, NT, NS>;
    if (!ensure_dynamic_smem(reinterpret_cast<const void*>(kernel), smem)) return KVQ_ERR_CUDA;
    if (launch_pdl(kernel, dim3(n), dim3(32 * C::kWarps), smem, s, p) != cudaSuccess) return KVQ_ERR_CUDA;
    count_launch();
    MergeCall m{};
    m.t = p.t;
    m.plan = p.plan;
    m.items = plan_items(a, C::RI);
    m.RI = C::RI;
    m.BT = kBT;
    m.workers = p.workers;
    m.spread = p.spread;
    m.D = D;
    m.partials = p.partials;
    m.O = a.O;
    m.o_dtype = a.q_dtype;
    return launch_merge(m, s);
  }
};

struct Entry {
  size_t (*workspace)(const AttendArgs&);
  kvq_status (*launch)(const AttendArgs&, cudaStream_t);
};
template <int BITS, int D, int NT, int NS>
constexpr Entry entry() {
  return Entry{Run<BITS, D, NT, NS>::workspace, Run<BITS, D, NT, NS>::launch};
}
template <int BITS, int D>
Entry by_rows(const AttendArgs& a) {
  const bool two = static_cast<long long>(a.max_q) * a.G > 4;
  if (a.q_dtype == KVQ_F32) return two ? entry<BITS, D, 2, 3>() : entry<BITS, D, 1, 3>();
  return two ? entry<BITS, D, 2, 2>() : entry<BITS, D, 1, 2>();
}
Entry pick(const AttendArgs& a) {
  if (a.g.bits == 4) return a.g.D == 64 ? by_rows<4, 64>(a) : by_rows<4, 128>(a);
  return a.g.D == 64 ? by_rows<8, 64>(a) : by_rows<8, 128>(a);
}

bool applies(const AttendArgs& a) {
  // a page holds whole 32-token blocks, and a block lies in one page
  return a.g.group == 32 && (a.g.D == 64 || a.g.D == 128);
}
size_t workspace(const AttendArgs& a) { return pick(a).workspace(a); }
kvq_status launch(const AttendArgs& a, cudaStream_t s) { return pick(a).launch(a, s); }

const AttendImpl kRows{"paged_rows", applies, workspace, launch};

}  // namespace

const AttendImpl& rows_impl() { return kRows; }

}  // namespace paged
}  // namespace kvq
