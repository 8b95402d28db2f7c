// Generic paged attention: any width D <= 256, 4- or 8-bit codes, any even
// group, any page size, any GQA ratio, f32 or bf16 rows.  The path of the
// shapes the tensor-core kernels do not take.
//
// Per block of 32 tokens the CTA decodes K and V into shared memory as
// float32, scores its 16 query rows against them and folds the block into the
// running (m, z, u) with the block rule ("Block KV decoding: less workspace,
// more time", huhohoo.com/en/docs/llm/kv-block-decode-cost, section "Do not
// average independently normalized blocks").  Bound by its own instructions (every
// code is decoded alone, products on the CUDA cores): 32 x 4096 keys of 8 heads in
// groups of 8 take 3.8 ms at 4 bits, 3.0 at 8.
#include "paged.cuh"

namespace kvq {
namespace paged {
namespace {

constexpr int kBT = 32;
constexpr int kRT = 16;
constexpr int kThreads = 256;
constexpr float kLog2e = 1.4426950408889634f;

struct Params {
  Batch t;
  PlanMem plan;
  const void* Q;
  int q_dtype;
  const uint8_t* k_codes;
  const float* k_scales;
  const uint8_t* v_codes;
  const float* v_scales;
  int bits, group, D, Dp;
  long long k_codes_head, k_scales_head, v_codes_head, v_scales_head;
  float qscale;                  // scale * log2(e)
  void* O;
  float* partials;
  int workers;
  unsigned int* err;
};

__device__ __forceinline__ int code_at(const uint8_t* codes, long long flat, int bits) {
  if (bits == 8) return codes[flat];
  const unsigned b = codes[flat >> 1];
  return (flat & 1) ? static_cast<int>(b >> 4) : static_cast<int>(b & 15u);
}

size_t smem_bytes(int D, int S) {
  return (static_cast<size_t>(2 * kBT * (D + 1) + 2 * kRT * D + kRT * kBT + 3 * kRT) + kRT) * sizeof(float) +
         kBT * sizeof(int) + (static_cast<size_t>(S) + 1) * sizeof(long long);
}

__global__ void __launch_bounds__(kThreads) paged_generic_kernel(Params p) {
  griddep_wait();
  extern __shared__ __align__(16) unsigned char smem_raw[];
  const int D = p.D, DS = D + 1;
  float* s_k = reinterpret_cast<float*>(smem_raw);   // [kBT][DS]
  float* s_v = s_k + kBT * DS;                        // [kBT][DS]
  float* s_q = s_v + kBT * DS;                        // [kRT][D]
  float* s_u = s_q + kRT * D;                         // [kRT][D]
  float* s_p = s_u + kRT * D;                         // [kRT][kBT]
  float* s_m = s_p + kRT * kBT;
  float* s_z = s_m + kRT;
  float* s_a = s_z + kRT;
  int* s_lim = reinterpret_cast<int*>(s_a + kRT);     // [kRT] keys each row sees
  int* s_page = s_lim + kRT;                          // [kBT] page of each token of the block
  long long* s_pre = reinterpret_cast<long long*>(s_page + kBT);   // [S + 1] (an even number of words comes before)

  if (!p.plan.count && threadIdx.x < 32) warp_prefix(p.t, kRT, kBT, s_pre);
  __syncthreads();
  const PlanView v = plan_view(p.plan, s_pre, p.t.S);
  const int H = p.t.H, H_q = H * p.t.G, qmax = p.bits == 4 ? 7 : 127, ngv = p.Dp / p.group;
  const Range wr = worker_range(v, H, p.workers, blockIdx.x);
  if (wr.g0 >= wr.g1) return;

  int i = find_item(v, H, wr.g0);
  int nb = v.blocks(i);
  const long long off = wr.g0 - static_cast<long long>(H) * v.pre[i];
  int h = static_cast<int>(off / nb), j = static_cast<int>(off % nb);
  long long g = wr.g0;
  while (g < wr.g1) {
    const Item it = plan_item(v, i);
    const SeqView s = seq_view(p.t, it.b);
    const int rows = min(kRT, s.n * p.t.G - it.r0);
    const int j0 = j, j1 = static_cast<int>(min(static_cast<long long>(nb), j + (wr.g1 - g)));
    const bool whole = j0 == 0 && j1 == nb;
    auto q_row = [&](int r) {
      const int rr = it.r0 + r;
      return static_cast<long long>(s.q0 + rr / p.t.G) * H_q + h * p.t.G + rr % p.t.G;
    };
    for (int idx = threadIdx.x; idx < rows * D; idx += kThreads)
      s_q[idx] = load_as_f32(p.Q, q_row(idx / D) * D + idx % D, p.q_dtype);
    for (int idx = threadIdx.x; idx < kRT * D; idx += kThreads) s_u[idx] = 0.f;
    if (threadIdx.x < kRT) {
      s_m[threadIdx.x] = -INFINITY;
      s_z[threadIdx.x] = 0.f;
      s_lim[threadIdx.x] = static_cast<int>(threadIdx.x) < rows ? row_limit(p.t, s, it.r0 + threadIdx.x) : 0;
    }
    for (; j < j1; ++j) {
      const int t0 = j * kBT, nt = min(kBT, s.len - t0);
      __syncthreads();                                 // the previous block's reads are done
      if (static_cast<int>(threadIdx.x) < nt)
        s_page[threadIdx.x] = read_page(
            __ldg(p.t.table + static_cast<long long>(it.b) * p.t.max_pages + (t0 + threadIdx.x) / p.t.P), p.t.pages,
            p.err);
      __syncthreads();
      for (int idx = threadIdx.x; idx < kBT * D; idx += kThreads) {
        const int t = idx / D, d = idx - t * D;
        float kv = 0.f, vv = 0.f;
        if (t < nt) {
          const long long head = static_cast<long long>(s_page[t]) * H + h;
          const int row = (t0 + t) % p.t.P;
          const long long tok = row;
          kv = __fmul_rn(static_cast<float>(code_at(p.k_codes + head * p.k_codes_head, tok * D + d, p.bits) - qmax),
                         p.k_scales[head * p.k_scales_head + (tok / p.group) * D + d]);
          vv = __fmul_rn(static_cast<float>(code_at(p.v_codes + head * p.v_codes_head, tok * p.Dp + d, p.bits) - qmax),
                         p.v_scales[head * p.v_scales_head + tok * ngv + d / p.group]);
        }
        s_k[t * DS + d] = kv;
        s_v[t * DS + d] = vv;
      }
      __syncthreads();
      for (int idx = threadIdx.x; idx < kRT * kBT; idx += kThreads) {
        const int r = idx / kBT, t = idx - r * kBT;
        float sc = -INFINITY;
        if (r < rows && t0 + t < s_lim[r]) {
          float acc = 0.f;
          for (int d = 0; d < D; ++d) acc = fmaf(s_q[r * D + d], s_k[t * DS + d], acc);
          sc = acc * p.qscale;
        }
        s_p[idx] = sc;
      }
      __syncthreads();
      static_assert(kBT == 32, "one token per lane");
      for (int r = static_cast<int>(threadIdx.x >> 5); r < rows; r += kThreads / 32) {
        const int t = static_cast<int>(threadIdx.x & 31);
        const float sc = s_p[r * kBT + t];
        float mb = sc;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mb = fmaxf(mb, __shfl_xor_sync(0xffffffffu, mb, o));
        const float mo = s_m[r], mn = fmaxf(mo, mb);
        // a masked key is -inf, and so is mn while the row has seen none; a
        // key the row sees always counts, whatever its score
        const float e = t0 + t < s_lim[r] ? exp2f(sc - mn) : 0.f;
        s_p[r * kBT + t] = e;
        float zs = e;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) zs += __shfl_xor_sync(0xffffffffu, zs, o);
        __syncwarp();
        if (t == 0) {
          const float a = mo == -INFINITY ? 0.f : exp2f(mo - mn);
          s_z[r] = a * s_z[r] + zs;
          s_m[r] = mn;
          s_a[r] = a;
        }
      }
      __syncthreads();
      for (int idx = threadIdx.x; idx < rows * D; idx += kThreads) {
        const int r = idx / D, d = idx - r * D;
        float acc = s_a[r] * s_u[idx];
        const int seen = min(nt, s_lim[r] - t0);      // a key the row does not see may hold anything
        for (int t = 0; t < seen; ++t) acc = fmaf(s_p[r * kBT + t], s_v[t * DS + d], acc);
        s_u[idx] = acc;
      }
    }
    __syncthreads();
    if (whole) {
      for (int idx = threadIdx.x; idx < rows * D; idx += kThreads) {
        const int r = idx / D;
        store_from_f32(p.O, q_row(r) * D + idx % D, s_z[r] == 0.f ? 0.f : s_u[idx] / s_z[r], p.q_dtype);
      }
    } else {
      const long long slot = 2 * static_cast<long long>(blockIdx.x) + (g == wr.g0 ? 0 : 1);
      float* part = p.partials + slot * kRT * (D + 2);
      for (int idx = threadIdx.x; idx < rows * D; idx += kThreads) part[idx] = s_u[idx];
      if (static_cast<int>(threadIdx.x) < rows) {
        part[kRT * D + 2 * threadIdx.x] = s_m[threadIdx.x];
        part[kRT * D + 2 * threadIdx.x + 1] = s_z[threadIdx.x];
      }
    }
    __syncthreads();
    g += j1 - j0;
    j = 0;
    if (g < wr.g1 && ++h == H) {
      h = 0;
      do {
        ++i;
        nb = v.blocks(i);
      } while (nb == 0);
    }
  }
}

bool applies(const AttendArgs&) { return true; }

int workers(const AttendArgs& a) {
  if (a.splits > 0) return a.splits;
  return 2 * (sm_count() > 0 ? sm_count() : 148);
}

size_t workspace(const AttendArgs& a) {
  return plan_bytes(a, kRT) + 2 * static_cast<size_t>(workers(a)) * kRT * (a.g.D + 2) * sizeof(float);
}

kvq_status launch(const AttendArgs& a, cudaStream_t s) {
  Params p{};
  p.t = make_batch(a);
  p.plan = plan_mem(a, kRT, a.workspace);
  p.Q = a.Q;
  p.q_dtype = a.q_dtype;
  p.k_codes = a.k_codes;
  p.k_scales = a.k_scales;
  p.v_codes = a.v_codes;
  p.v_scales = a.v_scales;
  p.bits = a.g.bits;
  p.group = a.g.group;
  p.D = a.g.D;
  p.Dp = a.g.Dp;
  p.k_codes_head = static_cast<long long>(a.g.k_codes_head);
  p.k_scales_head = static_cast<long long>(a.g.k_scales_head);
  p.v_codes_head = static_cast<long long>(a.g.v_codes_head);
  p.v_scales_head = static_cast<long long>(a.g.v_scales_head);
  p.qscale = a.scale * kLog2e;
  p.O = a.O;
  p.partials = reinterpret_cast<float*>(static_cast<char*>(a.workspace) + plan_bytes(a, kRT));
  p.workers = workers(a);
  p.err = error_word();
  if (!p.err) return KVQ_ERR_CUDA;
  if (p.plan.count) {
    const kvq_status st = launch_plan(a, p.plan, kRT, kBT, s);
    if (st != KVQ_OK) return st;
  }
  const size_t smem = smem_bytes(p.D, p.plan.count ? 0 : a.S);
  if (!ensure_dynamic_smem(reinterpret_cast<const void*>(paged_generic_kernel), smem)) return KVQ_ERR_CUDA;
  if (launch_pdl(paged_generic_kernel, dim3(p.workers), dim3(kThreads), smem, s, p) != cudaSuccess) return KVQ_ERR_CUDA;
  count_launch();
  MergeCall m{};
  m.t = p.t;
  m.plan = p.plan;
  m.items = plan_items(a, kRT);
  m.RI = kRT;
  m.BT = kBT;
  m.workers = p.workers;
  m.D = p.D;
  m.partials = p.partials;
  m.O = a.O;
  m.o_dtype = a.q_dtype;
  return launch_merge(m, s);
}

const AttendImpl kGeneric{"paged_generic", applies, workspace, launch};

}  // namespace

const AttendImpl& generic_impl() { return kGeneric; }

}  // namespace paged
}  // namespace kvq
