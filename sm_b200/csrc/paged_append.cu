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
// after the other, so the slot's rows are read before they are replaced.
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
__device__ __forceinline__ long long unit_base(const int32_t* cu, int b, int T, int per) {
  return min(max(__ldcg(cu + b), 0), T) / per + 2LL * b;
}
// The same for rows: base(b) = cu[b].
__device__ __forceinline__ long long row_base(const int32_t* cu, int b, int T) {
  return min(max(__ldcg(cu + b), 0), T);
}

// Largest b in [0, S) with base(b) <= u, by one warp, 32 probes a round.
template <typename Base>
__device__ __forceinline__ int warp_find(int S, long long u, Base base) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = S;
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int at = lane * step;
    const bool le = at < n && base(lo + at) <= u;
    const int k = __popc(__ballot_sync(0xffffffffu, le));
    if (k == 0) return lo;
    lo += (k - 1) * step;
    n = min(step, n - (k - 1) * step);
  }
  return lo;
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
  int bits, group, D, Dp, H, P, pages, cap;
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

template <bool kBf16>
__global__ void __launch_bounds__(kThreads) paged_append_kernel(AppendParams p) {
  griddep_wait();
  extern __shared__ __align__(16) float s_x[];      // [g][D], scale[D], 1/scale[D]
  const long long u = blockIdx.x;
  const int h = blockIdx.y, g = p.group;
  const int b = p.max_new == 1 ? static_cast<int>(u)
                               : warp_find(p.S, u, [&](int i) { return unit_base(p.cu, i, p.T, g); });
  const int j = p.max_new == 1 ? 0 : static_cast<int>(u - unit_base(p.cu, b, p.T, g));
  if (j < 0) return;                                // before the first sequence's rows
  const RowRange rr = row_range(p.cu, b, p.T, p.max_new);
  const bool report = threadIdx.x == 0 && j == 0 && h == 0;
  if (rr.bad && report) record_error(p.err, KVQ_ERR_LENGTH);
  if (rr.n == 0) return;
  const int len = __ldg(p.lengths + b);
  if (len < rr.n || len > p.cap) {
    if (report) record_error(p.err, KVQ_ERR_LENGTH);
    return;
  }
  const int slot = p.slots ? __ldg(p.slots + b) : b;
  if (static_cast<unsigned>(slot) >= static_cast<unsigned>(p.tail_slots)) {
    if (report) record_error(p.err, KVQ_ERR_INDEX);
    return;
  }
  const int first = len - rr.n;
  const int j0 = first / g, last = (len - 1) / g - j0;
  if (j > last) return;
  // both ends unfinished: the CTA of the first group does the last one too
  const bool joined = last > 0 && first % g != 0 && len % g != 0;
  if (joined && j == last) return;
  float* tail = p.tail + (static_cast<long long>(slot) * p.H + h) * g * p.D;
  for (int k = j; k <= last; k += joined && j == 0 ? last : last + 1) {
    const int tok0 = (j0 + k) * g;
    int page = __ldg(p.table + static_cast<long long>(b) * p.max_pages + tok0 / p.P);
    if (static_cast<unsigned>(page) >= static_cast<unsigned>(p.pages)) {
      if (threadIdx.x == 0) record_error(p.err, KVQ_ERR_INDEX);
      page = -1;
    }
    append_group<kBf16>(p, s_x, h, tok0, first, len, rr.r0, page, tail);
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

// One warp per row.
__global__ void __launch_bounds__(kThreads) paged_gather_kernel(GatherParams p) {
  griddep_wait();
  const long long row = static_cast<long long>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  if (row >= p.T) return;
  const int lane = threadIdx.x & 31;
  const int b = warp_find(p.S, row, [&](int i) { return row_base(p.cu, i, p.T); });
  const RowRange rr = row_range(p.cu, b, p.T, p.max_rows);
  if (lane == 0 && rr.bad) record_error(p.err, KVQ_ERR_LENGTH);
  if (row < rr.r0 || row >= rr.r0 + rr.n) return;   // no sequence's row
  const int start = __ldg(p.starts + b);
  const long long tok = static_cast<long long>(start) + (row - rr.r0);
  const bool in = start >= 0 && tok < p.cap;
  if (!in && lane == 0) record_error(p.err, KVQ_ERR_LENGTH);
  const int page =
      in ? read_page(__ldg(p.table + static_cast<long long>(b) * p.max_pages + tok / p.P), p.pages, p.err) : 0;
  const long long at = in ? tok % p.P : 0;
  for (int i = lane; i < p.H * p.D; i += 32) {
    const int h = i / p.D, d = i % p.D;
    const long long head = static_cast<long long>(page) * p.H + h;
    const long long o = row * p.H * p.D + i;
    if (p.K) {
      const float s = p.k_scales[head * p.k_scales_head + (at / p.group) * p.D + d];
      store_from_f32(p.K, o, in ? value_at(p.k_codes + head * p.k_codes_head, at * p.D + d, p.bits, s) : 0.f, p.dtype);
    }
    if (p.V) {
      const float s = p.v_scales[head * p.v_scales_head + at * (p.Dp / p.group) + d / p.group];
      store_from_f32(p.V, o, in ? value_at(p.v_codes + head * p.v_codes_head, at * p.Dp + d, p.bits, s) : 0.f, p.dtype);
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
  const size_t smem = (static_cast<size_t>(a.g.group) * a.g.D + 2 * a.g.D) * sizeof(float);
  auto kernel = a.in_dtype == KVQ_BF16 ? paged_append_kernel<true> : paged_append_kernel<false>;
  if (!ensure_dynamic_smem(reinterpret_cast<const void*>(kernel), smem)) return KVQ_ERR_CUDA;
  if (launch_pdl(kernel, dim3(static_cast<unsigned>(units), a.g.H_kv), dim3(kThreads), smem, s, p) != cudaSuccess)
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
  const int warps = kThreads / 32;
  if (launch_pdl(paged_gather_kernel, dim3((a.T + warps - 1) / warps), dim3(kThreads), 0, s, p) != cudaSuccess)
    return KVQ_ERR_CUDA;
  count_launch();
  return KVQ_OK;
}

}  // namespace paged
}  // namespace kvq
