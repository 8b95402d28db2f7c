// RMS norm of each query and key head and the position rotation, one pass:
//   y_d = x_d * w_d / sqrt(mean_d(x^2) + eps),
//   (y_a, y_b) -> (y_a c - y_b s, y_b c + y_a s) per pair of the rotation,
// in float32 throughout, rounded once to the output's type.
//
// The bound is memory: every element is read and written once.  A row of D
// features is held by a few lanes, 16 bytes each, so one load brings a row's
// part, shuffles give the sum of squares and (pairs D/2 apart) the partner,
// and a warp takes several heads of one token, whose angles it loads once.
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
  unsigned int* err;
};

__device__ __forceinline__ int rope_position(const Params& p, int t, bool report) {
  if (p.rot == 0) return -1;
  const int pos = __ldg(p.positions + t);
  if (static_cast<unsigned>(pos) < static_cast<unsigned>(p.n_pos)) return pos;
  if (report) record_error(p.err, KVQ_ERR_INDEX);
  return -1;
}

template <typename T>
struct Vec;                                    // 16 bytes of T
template <>
struct Vec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ uint4 load(const void* p, long long i) {
    return *reinterpret_cast<const uint4*>(static_cast<const float*>(p) + i);
  }
  static __device__ __forceinline__ void widen(const uint4& v, float (&x)[4]) {
    x[0] = __uint_as_float(v.x); x[1] = __uint_as_float(v.y); x[2] = __uint_as_float(v.z); x[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ void store(void* p, long long i, const float (&x)[4]) {
    *reinterpret_cast<float4*>(static_cast<float*>(p) + i) = make_float4(x[0], x[1], x[2], x[3]);
  }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ uint4 load(const void* p, long long i) {
    return *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + i);
  }
  static __device__ __forceinline__ void widen(const uint4& v, float (&x)[8]) {
    const unsigned w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      x[2 * k] = __uint_as_float(w[k] << 16);
      x[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ void store(void* p, long long i, const float (&x)[8]) {
    unsigned w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * k], x[2 * k + 1]);
      w[k] = *reinterpret_cast<const unsigned*>(&b);
    }
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p) + i) = make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// Vector path: LPR lanes hold a row (a power of two; D = LPR * N); the pairs
// of the rotation lie within a lane (interleaved) or whole lanes apart.  A
// warp takes U * 32 / LPR heads of one token: all their loads go out before
// the position's and the table's answer comes back.
template <typename T, int LPR, int U>
__global__ void __launch_bounds__(kThreads) qk_vec_kernel(Params p) {
  griddep_wait();
  constexpr int N = Vec<T>::N, RPW = 32 / LPR, HEADS = RPW * U;   // rows a warp loads at once; its heads
  const int lane = threadIdx.x & 31, sub = lane / LPR, l = lane % LPR;
  const int heads = p.H_q + p.H_kv;
  const int per_token = (heads + HEADS - 1) / HEADS;
  const long long unit = static_cast<long long>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  if (unit >= static_cast<long long>(p.T) * per_token) return;
  const int t = static_cast<int>(unit / per_token), h0 = static_cast<int>(unit - static_cast<long long>(t) * per_token) * HEADS;
  const int half = p.rot / 2, d0 = l * N;
  uint4 raw[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int h = h0 + u * RPW + sub;
    raw[u] = make_uint4(0u, 0u, 0u, 0u);
    if (h < heads)
      raw[u] = h < p.H_q ? Vec<T>::load(p.Q, t * p.q_stride + static_cast<long long>(h) * p.D + d0)
                         : Vec<T>::load(p.K, t * p.k_stride + static_cast<long long>(h - p.H_q) * p.D + d0);
  }
  const int pos = rope_position(p, t, lane == 0 && h0 == 0);
  // this lane's angles; the sign of s makes both features of a pair x c + partner s
  float c[N], s[N];
  int partner = lane;
  const bool turns = pos >= 0 && d0 < p.rot;
#pragma unroll
  for (int k = 0; k < N; ++k) {
    c[k] = 1.f;
    s[k] = 0.f;
  }
  if (turns) {
    const float* tab = p.rope + static_cast<long long>(pos) * p.rot;
    if (p.interleaved) {
#pragma unroll
      for (int k = 0; k < N; k += 2) {
        c[k] = c[k + 1] = __ldg(tab + d0 / 2 + k / 2);
        s[k + 1] = __ldg(tab + half + d0 / 2 + k / 2);
        s[k] = -s[k + 1];
      }
    } else {
      const bool upper = d0 >= half;
      const int e = upper ? d0 - half : d0;
      partner = upper ? lane - half / N : lane + half / N;
#pragma unroll
      for (int k = 0; k < N; k += 4) {
        const float4 cv = __ldg(reinterpret_cast<const float4*>(tab + e + k));
        const float4 sv = __ldg(reinterpret_cast<const float4*>(tab + half + e + k));
        c[k] = cv.x; c[k + 1] = cv.y; c[k + 2] = cv.z; c[k + 3] = cv.w;
        s[k] = sv.x; s[k + 1] = sv.y; s[k + 2] = sv.z; s[k + 3] = sv.w;
      }
      if (!upper) {
#pragma unroll
        for (int k = 0; k < N; ++k) s[k] = -s[k];
      }
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int h = h0 + u * RPW + sub;
    const bool on = h < heads, is_k = h >= p.H_q;
    float x[N];
    Vec<T>::widen(raw[u], x);
    const void* w = is_k ? p.k_weight : p.q_weight;
    if (p.k_weight || p.q_weight) {
      float sum = 0.f;
#pragma unroll
      for (int k = 0; k < N; ++k) sum = fmaf(x[k], x[k], sum);
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (on && w) {
        float wv[N];
        Vec<T>::widen(Vec<T>::load(w, d0), wv);
        const float r = rsqrtf(fmaf(sum, p.inv_d, p.eps));
#pragma unroll
        for (int k = 0; k < N; ++k) x[k] = x[k] * r * wv[k];
      }
    }
    float y[N];
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const float o = p.interleaved ? x[k ^ 1] : __shfl_sync(0xffffffffu, x[k], partner);
      y[k] = turns ? fmaf(o, s[k], x[k] * c[k]) : x[k];
    }
    if (on) {
      if (is_k) Vec<T>::store(p.K_out, (static_cast<long long>(t) * p.H_kv + h - p.H_q) * p.D + d0, y);
      else Vec<T>::store(p.Q_out, (static_cast<long long>(t) * p.H_q + h) * p.D + d0, y);
    }
  }
}

// Any width, alignment and rotation: a warp per row, the row in shared memory
// (so a row may be written where it was read).
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
    // four loads a warp in flight where that leaves enough warps to fill the GPU
    // (148 SMs of 32 warps), one where it would not: at 64 tokens of 40 heads
    // the step is latency, and fewer heads a warp finish sooner
    const int rpw = 32 / lpr;
    const bool many = static_cast<long long>(p.T) * ((heads + 4 * rpw - 1) / (4 * rpw)) >= 148 * 32;
    const int rows = many ? 4 * rpw : rpw;
    const long long units = static_cast<long long>(p.T) * ((heads + rows - 1) / rows);
    const long long grid = (units + warps - 1) / warps;
    if (grid > 0x7fffffffLL) return KVQ_ERR_UNSUPPORTED;
    cudaError_t e = cudaErrorInvalidValue;
    const dim3 g(static_cast<unsigned>(grid)), b(kThreads);
    auto run = [&](auto one, auto four) { e = many ? launch_pdl(four, g, b, 0, s, p) : launch_pdl(one, g, b, 0, s, p); };
    switch (lpr) {
      case 1: run(qk_vec_kernel<T, 1, 1>, qk_vec_kernel<T, 1, 4>); break;
      case 2: run(qk_vec_kernel<T, 2, 1>, qk_vec_kernel<T, 2, 4>); break;
      case 4: run(qk_vec_kernel<T, 4, 1>, qk_vec_kernel<T, 4, 4>); break;
      case 8: run(qk_vec_kernel<T, 8, 1>, qk_vec_kernel<T, 8, 4>); break;
      case 16: run(qk_vec_kernel<T, 16, 1>, qk_vec_kernel<T, 16, 4>); break;
      case 32: run(qk_vec_kernel<T, 32, 1>, qk_vec_kernel<T, 32, 4>); break;
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
