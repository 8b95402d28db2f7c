// RMS norm of each query and key head and the position rotation, one pass:
//   y_d = x_d * w_d / sqrt(mean_d(x^2) + eps),
//   (y_a, y_b) -> (y_a c - y_b s, y_b c + y_a s) per pair of the rotation,
// in float32 throughout, rounded once to the output's type.
//
// The bound is memory: every element is read and written once.  A row of D
// features is held by a few lanes, 16 bytes each, so one load brings a row's
// part, shuffles give the sum of squares and (pairs D/2 apart) the partner,
// and a warp takes several heads of one token, whose angles it loads once.
// 172 MB (8 thousand tokens of 32 + 8 heads, D = 128) take 36 us, 4.7 TB/s, 72 %
// of the measured copy rate; forms with fewer registers and more warps took 40 to
// 43.  A step of 64 tokens takes 5 us, a launch.
#include <type_traits>

#include "f32x2.cuh"
#include "kvq_internal.cuh"

namespace kvq {
namespace {

constexpr int kThreads = 128;

struct Params {
  const void* Q;
  const void* K;
  long long q_stride, k_stride;
  int T, H_q, H_kv, D;
  const void* q_weight;
  const void* k_weight;
  float eps;
  const int32_t* positions;
  const float* rope;
  int n_pos, rot, interleaved;
  void* Q_out;
  void* K_out;
  float inv_d;
  int chunks;                    // vector path: chunks of a token that a warp takes
  unsigned int* err;
};

__device__ __forceinline__ int rope_position(const Params& p, int t, bool report) {
  if (p.rot == 0) return -1;
  const int pos = __ldg(p.positions + t);
  if (static_cast<unsigned>(pos) < static_cast<unsigned>(p.n_pos)) return pos;
  if (report) record_error(p.err, KVQ_ERR_INDEX);
  return -1;
}

// 16 bytes of T as pairs of floats.
template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void widen(const uint4& v, u64 (&x)[2]) {
    x[0] = pack2(__uint_as_float(v.x), __uint_as_float(v.y));
    x[1] = pack2(__uint_as_float(v.z), __uint_as_float(v.w));
  }
  // the features of each pair exchanged
  static __device__ __forceinline__ uint4 exchange(const uint4& v) { return make_uint4(v.y, v.x, v.w, v.z); }
  static __device__ __forceinline__ void store(void* p, long long i, const u64 (&x)[2]) {
    *reinterpret_cast<ulonglong2*>(static_cast<float*>(p) + i) = make_ulonglong2(x[0], x[1]);
  }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void widen(const uint4& v, u64 (&x)[4]) {
    const unsigned w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = pack2(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xFFFF0000u));
  }
  static __device__ __forceinline__ uint4 exchange(const uint4& v) {
    return make_uint4(__byte_perm(v.x, 0, 0x1032), __byte_perm(v.y, 0, 0x1032), __byte_perm(v.z, 0, 0x1032),
                      __byte_perm(v.w, 0, 0x1032));
  }
  static __device__ __forceinline__ void store(void* p, long long i, const u64 (&x)[4]) {
    unsigned w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(lo_f(x[k]), hi_f(x[k]));
      w[k] = *reinterpret_cast<const unsigned*>(&b);
    }
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p) + i) = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <typename T>
__device__ __forceinline__ uint4 load16(const void* p, long long i) {
  return *reinterpret_cast<const uint4*>(static_cast<const T*>(p) + i);
}

// Vector path: LPR lanes hold a row (a power of two; D = LPR * N); the pairs
// of the rotation lie within a lane (kInter) or whole lanes apart.  A chunk is
// U * 32 / LPR heads of one token, all of Q or all of K; a warp takes
// p.chunks of a token's chunks one after the other, the next one's loads in
// flight while it works.  Weight times angle is formed once a token and side,
// so a feature costs y = r (x wc + partner ws): two products and a fused sum,
// on pairs.
template <typename T, int LPR, int U, bool kInter>
__global__ void __launch_bounds__(kThreads) qk_vec_kernel(Params p) {
  griddep_wait();
  constexpr int N = Vec<T>::N, RPW = 32 / LPR, HEADS = RPW * U;   // rows a warp loads at once; a chunk's heads
  const int lane = threadIdx.x & 31, sub = lane / LPR, l = lane % LPR;
  const int q_chunks = (p.H_q + HEADS - 1) / HEADS, chunks = q_chunks + (p.H_kv + HEADS - 1) / HEADS;
  const int per_token = (chunks + p.chunks - 1) / p.chunks;
  const unsigned unit = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const int t = static_cast<int>(unit / per_token);
  if (t >= p.T) return;
  int ch = static_cast<int>(unit - static_cast<unsigned>(t) * per_token) * p.chunks;
  const int ch_end = min(chunks, ch + p.chunks);
  const int half = p.rot / 2, d0 = l * N;
  const T* q_row = static_cast<const T*>(p.Q) + t * p.q_stride + sub * p.D + d0;
  const T* k_row = static_cast<const T*>(p.K) + t * p.k_stride + sub * p.D + d0;
  auto load = [&](int c, uint4 (&raw)[U]) {
    const bool is_k = c >= q_chunks;
    const int h = (is_k ? c - q_chunks : c) * HEADS, left = (is_k ? p.H_kv : p.H_q) - h - sub;
    const T* src = (is_k ? k_row : q_row) + h * p.D;
#pragma unroll
    for (int u = 0; u < U; ++u)
      raw[u] = u * RPW < left ? load16<T>(src, u * RPW * p.D) : make_uint4(0u, 0u, 0u, 0u);
  };
  uint4 raw[U];
  load(ch, raw);
  const int pos = rope_position(p, t, lane == 0 && ch == 0);
  const bool turns = pos >= 0 && d0 < p.rot;
  const bool upper = !kInter && d0 >= half;
  const int shift = turns && !kInter ? (upper ? -half / N : half / N) : 0;   // the partner lane's distance
  // the angles; the sign of s makes both features of a pair x c + partner s
  u64 c2[N / 2], s2[N / 2];
#pragma unroll
  for (int k = 0; k < N / 2; ++k) {
    c2[k] = pack2(1.f, 1.f);
    s2[k] = 0ull;
  }
  if (turns) {
    const float* tab = p.rope + static_cast<long long>(pos) * p.rot;
    if (kInter) {
#pragma unroll
      for (int k = 0; k < N / 2; ++k) {
        const float c = __ldg(tab + d0 / 2 + k), s = __ldg(tab + half + d0 / 2 + k);
        c2[k] = pack2(c, c);
        s2[k] = pack2(-s, s);
      }
    } else {
      const int e = upper ? d0 - half : d0;
      const u64 flip = upper ? 0ull : 0x8000000080000000ull;
#pragma unroll
      for (int k = 0; k < N / 2; k += 2) {
        const ulonglong2 c = *reinterpret_cast<const ulonglong2*>(tab + e + 2 * k);
        const ulonglong2 s = *reinterpret_cast<const ulonglong2*>(tab + half + e + 2 * k);
        c2[k] = c.x;
        c2[k + 1] = c.y;
        s2[k] = s.x ^ flip;
        s2[k + 1] = s.y ^ flip;
      }
    }
  }
  const unsigned mask = turns ? 0xFFFFFFFFu : 0u;      // a lane that does not turn has no partner: inf * 0 stays out
  u64 wc[N / 2], ws[N / 2];
  const void* w = nullptr;
  int side = -1;
  for (; ch < ch_end; ++ch) {
    const bool is_k = ch >= q_chunks;
    if (side != static_cast<int>(is_k)) {
      side = is_k;
      w = is_k ? p.k_weight : p.q_weight;
#pragma unroll
      for (int k = 0; k < N / 2; ++k) {
        wc[k] = c2[k];
        ws[k] = s2[k];
      }
      if (w) {
        const uint4 own = load16<T>(w, d0), other = kInter ? Vec<T>::exchange(own) : load16<T>(w, d0 + shift * N);
        u64 wv[N / 2];
        Vec<T>::widen(own, wv);
#pragma unroll
        for (int k = 0; k < N / 2; ++k) wc[k] = mul2(wc[k], wv[k]);
        Vec<T>::widen(other, wv);
#pragma unroll
        for (int k = 0; k < N / 2; ++k) ws[k] = mul2(ws[k], wv[k]);
      }
    }
    uint4 next[U];
    if (ch + 1 < ch_end) load(ch + 1, next);
    const int h = (is_k ? ch - q_chunks : ch) * HEADS + sub, heads = is_k ? p.H_kv : p.H_q;
    T* dst = static_cast<T*>(is_k ? p.K_out : p.Q_out) + (static_cast<long long>(t) * heads + h) * p.D + d0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      u64 x[N / 2], o[N / 2], y[N / 2];
      Vec<T>::widen(raw[u], x);
      uint4 b;
      if (kInter) {
        b = Vec<T>::exchange(raw[u]);
      } else {
        b.x = __shfl_sync(0xffffffffu, raw[u].x, lane + shift);
        b.y = __shfl_sync(0xffffffffu, raw[u].y, lane + shift);
        b.z = __shfl_sync(0xffffffffu, raw[u].z, lane + shift);
        b.w = __shfl_sync(0xffffffffu, raw[u].w, lane + shift);
      }
      Vec<T>::widen(make_uint4(b.x & mask, b.y & mask, b.z & mask, b.w & mask), o);
#pragma unroll
      for (int k = 0; k < N / 2; ++k) y[k] = fma2(o[k], ws[k], mul2(x[k], wc[k]));
      if (w) {
        u64 sq = mul2(x[0], x[0]);
#pragma unroll
        for (int k = 1; k < N / 2; ++k) sq = fma2(x[k], x[k], sq);
        float sum = lo_f(sq) + hi_f(sq);
#pragma unroll
        for (int d = LPR / 2; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        const float r = rsqrtf(fmaf(sum, p.inv_d, p.eps));
        const u64 r2 = pack2(r, r);
#pragma unroll
        for (int k = 0; k < N / 2; ++k) y[k] = mul2(y[k], r2);
      }
      if (h + u * RPW < heads) Vec<T>::store(dst, u * RPW * p.D, y);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) raw[u] = next[u];
  }
}

// Any width, alignment and rotation: a warp per row, the row in shared memory
// (so a row may be written where it was read).  An element a lane and load: 8
// thousand tokens of 32 + 8 heads at D = 80 or 96 take 159 us.
template <typename T>
__global__ void __launch_bounds__(kThreads) qk_any_kernel(Params p) {
  griddep_wait();
  extern __shared__ float s_row[];              // [warps][D]
  constexpr int dt = sizeof(T) == 4 ? KVQ_F32 : KVQ_BF16;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int heads = p.H_q + (p.K ? p.H_kv : 0);
  const long long row = static_cast<long long>(blockIdx.x) * (kThreads / 32) + warp;
  if (row >= static_cast<long long>(p.T) * heads) return;
  const int t = static_cast<int>(row / heads), h = static_cast<int>(row % heads);
  const bool is_k = h >= p.H_q;
  const int pos = rope_position(p, t, lane == 0 && h == 0);
  const void* src = is_k ? p.K : p.Q;
  const long long in = is_k ? t * p.k_stride + static_cast<long long>(h - p.H_q) * p.D
                            : t * p.q_stride + static_cast<long long>(h) * p.D;
  const long long out = is_k ? (static_cast<long long>(t) * p.H_kv + h - p.H_q) * p.D
                             : (static_cast<long long>(t) * p.H_q + h) * p.D;
  void* dst = is_k ? p.K_out : p.Q_out;
  const void* w = is_k ? p.k_weight : p.q_weight;
  float* x = s_row + warp * p.D;
  float sum = 0.f;
  for (int d = lane; d < p.D; d += 32) {
    const float v = load_as_f32(src, in + d, dt);
    x[d] = v;
    sum = fmaf(v, v, sum);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (w) {
    const float r = rsqrtf(sum / static_cast<float>(p.D) + p.eps);
    for (int d = lane; d < p.D; d += 32) x[d] = x[d] * r * load_as_f32(w, d, dt);
  }
  __syncwarp();
  const int half = p.rot / 2;
  const float* tab = p.rope + static_cast<long long>(pos) * p.rot;
  for (int d = lane; d < p.D; d += 32) {
    float y = x[d];
    if (pos >= 0 && d < p.rot) {
      const int e = p.interleaved ? d / 2 : d % half;
      const bool second = p.interleaved ? (d & 1) != 0 : d >= half;
      const float c = tab[e], s = tab[half + e];
      const float o = x[p.interleaved ? d ^ 1 : (second ? d - half : d + half)];
      y = fmaf(o, second ? s : -s, y * c);
    }
    store_from_f32(dst, out + d, y, dt);
  }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

template <typename T>
kvq_status launch(Params p, cudaStream_t s) {
  constexpr int N = Vec<T>::N;
  const int heads = p.H_q + (p.K ? p.H_kv : 0), warps = kThreads / 32;
  const int lpr = p.D / N;
  const bool vec = p.D % N == 0 && lpr <= 32 && (lpr & (lpr - 1)) == 0 && aligned16(p.Q) && aligned16(p.Q_out) &&
                   p.q_stride % N == 0 &&
                   (!p.K || (aligned16(p.K) && aligned16(p.K_out) && p.k_stride % N == 0)) &&
                   aligned16(p.q_weight) && aligned16(p.k_weight) &&
                   (p.rot == 0 || (p.interleaved ? p.rot % N == 0
                                                 : p.rot % (2 * N) == 0 && aligned16(p.rope)));
  if (vec) {
    // A warp takes as many of a token's heads as still leaves 148 SMs 24 warps
    // each: the angles and the weights are then formed for all of them.  Where
    // even one chunk of four loads a warp leaves fewer, the step is latency and
    // one load a warp finishes soonest.
    const int rpw = 32 / lpr;
    auto chunks_of = [&](int heads_of) { return (p.H_q + heads_of - 1) / heads_of + (p.H_kv + heads_of - 1) / heads_of; };
    const bool many = static_cast<long long>(p.T) * chunks_of(4 * rpw) >= 148 * 24;
    const int chunks = chunks_of(many ? 4 * rpw : rpw);
    p.chunks = 1;
    while (many && p.chunks < chunks &&
           static_cast<long long>(p.T) * ((chunks + p.chunks) / (p.chunks + 1)) >= 148 * 24)
      ++p.chunks;
    const long long grid = (static_cast<long long>(p.T) * ((chunks + p.chunks - 1) / p.chunks) + warps - 1) / warps;
    if (grid > 0x3fffffffLL) return KVQ_ERR_UNSUPPORTED;
    cudaError_t e = cudaErrorInvalidValue;
    const dim3 g(static_cast<unsigned>(grid)), b(kThreads);
    auto run = [&](auto lpr_c) {
      constexpr int L = decltype(lpr_c)::value;
      e = p.interleaved ? (many ? launch_pdl(qk_vec_kernel<T, L, 4, true>, g, b, 0, s, p)
                                : launch_pdl(qk_vec_kernel<T, L, 1, true>, g, b, 0, s, p))
                        : (many ? launch_pdl(qk_vec_kernel<T, L, 4, false>, g, b, 0, s, p)
                                : launch_pdl(qk_vec_kernel<T, L, 1, false>, g, b, 0, s, p));
    };
    switch (lpr) {
      case 1: run(std::integral_constant<int, 1>{}); break;
      case 2: run(std::integral_constant<int, 2>{}); break;
      case 4: run(std::integral_constant<int, 4>{}); break;
      case 8: run(std::integral_constant<int, 8>{}); break;
      case 16: run(std::integral_constant<int, 16>{}); break;
      case 32: run(std::integral_constant<int, 32>{}); break;
    }
    if (e != cudaSuccess) return KVQ_ERR_CUDA;
  } else {
    const long long grid = (static_cast<long long>(p.T) * heads + warps - 1) / warps;
    if (grid > 0x7fffffffLL) return KVQ_ERR_UNSUPPORTED;
    if (launch_pdl(qk_any_kernel<T>, dim3(static_cast<unsigned>(grid)), dim3(kThreads),
                   static_cast<size_t>(warps) * p.D * sizeof(float), s, p) != cudaSuccess)
      return KVQ_ERR_CUDA;
  }
  count_launch();
  return KVQ_OK;
}

}  // namespace
}  // namespace kvq

using namespace kvq;

extern "C" kvq_status kvq_qk_norm_rope(const void* Q, int64_t q_stride, const void* K, int64_t k_stride,
                                       kvq_dtype dtype, int32_t T, int32_t H_q, int32_t H_kv, int32_t D,
                                       const void* q_weight, const void* k_weight, float eps,
                                       const int32_t* positions, const kvq_rope* rope, void* Q_out, void* K_out,
                                       void* stream) {
  if (dtype != KVQ_F32 && dtype != KVQ_BF16) return KVQ_ERR_ARG;
  if (!Q || !Q_out || (K != nullptr) != (K_out != nullptr)) return KVQ_ERR_ARG;
  if (T < 1 || H_q < 1 || D < 1 || (K && H_kv < 1)) return KVQ_ERR_ARG;
  if (q_stride < static_cast<int64_t>(H_q) * D || (K && k_stride < static_cast<int64_t>(H_kv) * D)) return KVQ_ERR_ARG;
  if (!(eps >= 0.f)) return KVQ_ERR_ARG;
  const bool turn = rope && rope->table;
  if (turn && (rope->rot_dim < 2 || (rope->rot_dim & 1) || rope->rot_dim > D || rope->n_pos < 1 || !positions))
    return KVQ_ERR_ARG;
  if (D > 1024) return KVQ_ERR_UNSUPPORTED;
  const size_t esz = dtype == KVQ_F32 ? 4 : 2;
  if ((reinterpret_cast<uintptr_t>(Q) | reinterpret_cast<uintptr_t>(K) | reinterpret_cast<uintptr_t>(Q_out) |
       reinterpret_cast<uintptr_t>(K_out) | reinterpret_cast<uintptr_t>(q_weight) |
       reinterpret_cast<uintptr_t>(k_weight)) % esz)
    return KVQ_ERR_ALIGN;
  if (turn && (reinterpret_cast<uintptr_t>(positions) | reinterpret_cast<uintptr_t>(rope->table)) % 4)
    return KVQ_ERR_ALIGN;
  Params p{};
  p.Q = Q;
  p.K = K;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.T = T;
  p.H_q = H_q;
  p.H_kv = K ? H_kv : 0;
  p.D = D;
  p.q_weight = q_weight;
  p.k_weight = k_weight;
  p.eps = eps;
  p.inv_d = 1.f / static_cast<float>(D);
  p.positions = positions;
  p.rope = turn ? rope->table : nullptr;
  p.n_pos = turn ? rope->n_pos : 0;
  p.rot = turn ? rope->rot_dim : 0;
  p.interleaved = turn && rope->interleaved;
  p.Q_out = Q_out;
  p.K_out = K_out;
  p.err = error_word();
  if (!p.err) return KVQ_ERR_CUDA;
  return dtype == KVQ_BF16 ? launch<__nv_bfloat16>(p, static_cast<cudaStream_t>(stream))
                           : launch<float>(p, static_cast<cudaStream_t>(stream));
}
