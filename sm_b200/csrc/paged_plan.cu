// Paged attention: the item list of a ragged batch, and the merge of the
// states that several workers computed for one (item, KV head).
//
// The merge is the block rule of "Block KV decoding: less workspace, more
// time" (huhohoo.com/en/docs/llm/kv-block-decode-cost, section "Do not average
// independently normalized blocks"): M = max m_c, w_c = 2^(m_c - M),
// O = sum w_c u_c / sum w_c z_c over the parts c that hold a key.  It is
// bound by latency: the m and z of up to 32 parts come in one round (lane =
// part), the u rows in a second whose loads do not depend on one another.
#include "paged.cuh"

namespace kvq {
namespace paged {
namespace {

constexpr int kPlanThreads = 1024;

// Sum of two counts, held below 2^30: a cu that is not as stated can give
// the sequences more rows than there are, and the prefix must stay ordered.
__device__ __forceinline__ int add_sat(int a, int b) { return min(a + b, 0x3fffffff); }

// Inclusive scan of one count per thread over the CTA.
__device__ __forceinline__ int block_scan(int v, int* s_warp) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int n = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v = add_sat(v, n);
  }
  if (lane == 31) s_warp[w] = v;
  __syncthreads();
  if (w == 0) {
    int x = s_warp[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int n = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x = add_sat(x, n);
    }
    s_warp[lane] = x;
  }
  __syncthreads();
  const int add = w > 0 ? s_warp[w - 1] : 0;
  __syncthreads();
  return add_sat(v, add);
}

// One CTA.  Item counts of the sequences are summed into s_first (sequences
// 1024 at a time, the prefix kept in the workspace's pre array until the
// items' own prefix replaces it: pre has room for items + 1 >= the sequences
// that have rows, so the sequences' prefix lives in shared memory instead).
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(Batch t, PlanMem m, int RI, int BT, int max_items,
                                                            unsigned int* err) {
  griddep_wait();
  extern __shared__ int s_first[];              // [S + 1] first item of each sequence
  __shared__ int s_warp[32];
  int carry = 0;
  for (int base = 0; base < t.S; base += kPlanThreads) {
    const int b = base + static_cast<int>(threadIdx.x);
    int v = 0;
    if (b < t.S) {
      const SeqView s = seq_view(t, b);
      if (s.bad) record_error(err, KVQ_ERR_LENGTH);
      v = (s.n * t.G + RI - 1) / RI;
    }
    const int inc = block_scan(v, s_warp);
    if (b < t.S) s_first[b + 1] = add_sat(carry, inc);
    __syncthreads();
    carry = s_first[min(base + kPlanThreads, t.S)];
  }
  if (threadIdx.x == 0) s_first[0] = 0;
  __syncthreads();
  const int items = min(s_first[t.S], max_items);
  int blocks = 0;
  for (int base = 0; base < items; base += kPlanThreads) {
    const int i = base + static_cast<int>(threadIdx.x);
    int v = 0;
    if (i < items) {
      int lo = 0, hi = t.S - 1;                 // largest b with s_first[b] <= i
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s_first[mid] <= i) lo = mid;
        else hi = mid - 1;
      }
      const int r0 = (i - s_first[lo]) * RI;
      v = item_blocks(t, seq_view(t, lo), r0, RI, BT);
      m.item[i] = Item{lo, r0};
    }
    const int inc = block_scan(v, s_warp);
    if (i < items) m.pre[i + 1] = add_sat(blocks, inc);
    if (threadIdx.x == kPlanThreads - 1) s_warp[0] = inc;
    __syncthreads();
    blocks = add_sat(blocks, s_warp[0]);
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    m.pre[0] = 0;
    *m.count = items;
  }
}

struct MergeParams {
  MergeCall c;
  unsigned int* err;
};

struct Parts {
  int rows;              // rows of the item
  long long out0;        // row index of the item's row 0 within O's [T, H_q]
  long long c_first;     // first worker
  int n;                 // workers (0: no key, zero rows)
  bool first_is_start;   // the first worker's range begins inside (or at) this head's blocks
};

// The workers whose ranges meet the blocks of (item, head h).
__device__ __forceinline__ Parts find_parts(const MergeCall& c, const PlanView& v, int i, const Item& it,
                                            const SeqView& s, int h) {
  Parts p{};
  p.rows = min(c.RI, s.n * c.t.G - it.r0);
  const int nb = v.pre[i + 1] - v.pre[i];
  if (nb > 0) {
    const Range r = worker_range(v, c.t.H, c.workers, 0);
    const long long S = static_cast<long long>(c.t.H) * v.pre[i] + static_cast<long long>(h) * nb;
    p.c_first = S / r.per;
    p.n = static_cast<int>((S + nb - 1) / r.per - p.c_first + 1);
    p.first_is_start = p.c_first * r.per == S;
  }
  return p;
}

// Slot of part k: every worker after the first begins inside this head's
// blocks; the first does only if its range starts exactly at them.
__device__ __forceinline__ long long part_slot(const Parts& p, int k) {
  return 2 * (p.c_first + k) + ((k > 0 || p.first_is_start) ? 0 : 1);
}

__device__ __forceinline__ float exp2_w(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Row-major partials: one CTA per (item, head); a warp per (row, 32 features).
constexpr int kMergeThreads = 256;
__global__ void __launch_bounds__(kMergeThreads) merge_rows_kernel(MergeParams p) {
  extern __shared__ int s_pre[];
  const MergeCall& c = p.c;
  const int i = blockIdx.x / c.t.H, h = blockIdx.x % c.t.H;
  // the inline plan reads only the call's inputs (through the L2), so it runs
  // while the attention kernel drains
  if (c.plan.count) griddep_wait();
  else if (threadIdx.x < 32) warp_prefix(c.t, c.RI, c.BT, s_pre);
  __syncthreads();
  const PlanView v = plan_view(c.plan, s_pre, c.t.S);
  const bool live = i < v.items;
  const Item it = live ? plan_item(v, i) : Item{0, 0};
  const SeqView s = seq_view(c.t, it.b);
  Parts q{};
  if (live) q = find_parts(c, v, i, it, s, h);
  if (!c.plan.count) griddep_wait();
  if (!live) return;
  if (!c.plan.count && h == 0 && threadIdx.x == 0 && s.bad) record_error(p.err, KVQ_ERR_LENGTH);
  if (q.n == 1) return;                        // that worker wrote the rows
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int D = c.D, slices = (D + 31) / 32;
  const long long stride = static_cast<long long>(c.RI) * (D + 2);
  const int H_q = c.t.H * c.t.G;
  for (int task = warp; task < q.rows * slices; task += kMergeThreads / 32) {
    const int r = task / slices, f = (task % slices) * 32 + lane;
    const int rr = it.r0 + r;
    const long long o = (static_cast<long long>(s.q0 + rr / c.t.G) * H_q + h * c.t.G + rr % c.t.G) * D + f;
    float M = -INFINITY, Z = 0.f, U = 0.f;
    bool nan = false;                          // a part whose sum is not a number: neither is the row
    for (int k0 = 0; k0 < q.n; k0 += 32) {
      const int k = k0 + lane;
      float m = -INFINITY, z = 0.f;
      if (k < q.n) {
        const float2 mz = *reinterpret_cast<const float2*>(c.partials + part_slot(q, k) * stride +
                                                           static_cast<long long>(c.RI) * D + 2 * r);
        z = mz.y;
        m = z > 0.f ? mz.x : -INFINITY;
      }
      nan |= __any_sync(0xffffffffu, z != z);
      float top = m;
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
      top = fmaxf(top, M);
      if (top == -INFINITY) continue;
      const float keep = exp2_w(M - top);
      const float w = exp2_w(m - top);
      float zs = w * z;
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) zs += __shfl_xor_sync(0xffffffffu, zs, x);
      M = top;
      Z = Z * keep + zs;
      U *= keep;
      const int n = min(32, q.n - k0);
#pragma unroll 8
      for (int j = 0; j < n; ++j) {
        const float wj = __shfl_sync(0xffffffffu, w, j);
        const float u = f < D ? c.partials[part_slot(q, k0 + j) * stride + static_cast<long long>(r) * D + f] : 0.f;
        if (wj > 0.f) U = fmaf(wj, u, U);      // a part without a key holds nothing
      }
    }
    if (f < D) store_from_f32(c.O, o, nan ? NAN : (Z > 0.f ? U / Z : 0.f), c.o_dtype);
  }
}

// Feature-major partials: one CTA per (item, head), 32-row chunk (blockIdx.y)
// and 32 features (blockIdx.z); lane = row, a warp takes four features, four
// parts' loads in flight.
__global__ void __launch_bounds__(256) merge_tiles_kernel(MergeParams p) {
  extern __shared__ int s_pre[];
  const MergeCall& c = p.c;
  const int i = blockIdx.x / c.t.H, h = blockIdx.x % c.t.H;
  if (c.plan.count) griddep_wait();
  else if (threadIdx.x < 32) warp_prefix(c.t, c.RI, c.BT, s_pre);
  __syncthreads();
  const PlanView v = plan_view(c.plan, s_pre, c.t.S);
  const bool live = i < v.items;
  const Item it = live ? plan_item(v, i) : Item{0, 0};
  const SeqView s = seq_view(c.t, it.b);
  Parts q{};
  if (live) q = find_parts(c, v, i, it, s, h);
  if (!c.plan.count) griddep_wait();
  if (!live) return;
  if (!c.plan.count && h == 0 && blockIdx.y == 0 && blockIdx.z == 0 && threadIdx.x == 0 && s.bad)
    record_error(p.err, KVQ_ERR_LENGTH);
  if (q.n == 1) return;
  const int lane = threadIdx.x & 31, f = 32 * blockIdx.z + 4 * (threadIdx.x >> 5);
  const int pr = 32 * blockIdx.y + lane, tile = pr >> 7;               // padded row of the slot
  const int r = tile * c.tile_rows + (pr & 127);
  const bool real = (pr & 127) < c.tile_rows && r < q.rows;
  const int D = c.D;
  const long long stride = 256LL * (D + 2);
  const float* base = c.partials + static_cast<long long>(blockIdx.y) * (D + 2) * 32 + lane;
  float M = -INFINITY, Z = 0.f, U[4] = {0.f, 0.f, 0.f, 0.f};
  constexpr int PB = 4;
  bool nan = false;
  for (int k0 = 0; k0 < q.n; k0 += PB) {
    float m[PB], z[PB], u[PB][4];
#pragma unroll
    for (int k = 0; k < PB; ++k) {
      m[k] = -INFINITY;
      z[k] = 0.f;
      if (k0 + k < q.n && real) {
        const float* part = base + part_slot(q, k0 + k) * stride;
        m[k] = part[0];
        z[k] = part[32];
#pragma unroll
        for (int e = 0; e < 4; ++e) u[k][e] = part[(2 + f + e) * 32];
      }
    }
    float top = M;
#pragma unroll
    for (int k = 0; k < PB; ++k) nan |= z[k] != z[k];
#pragma unroll
    for (int k = 0; k < PB; ++k)
      if (z[k] > 0.f) top = fmaxf(top, m[k]);
    if (top == -INFINITY) continue;
    const float keep = exp2_w(M - top);
    M = top;
    Z *= keep;
#pragma unroll
    for (int e = 0; e < 4; ++e) U[e] *= keep;
#pragma unroll
    for (int k = 0; k < PB; ++k)
      if (z[k] > 0.f) {
        const float w = exp2_w(m[k] - top);
        Z = fmaf(w, z[k], Z);
#pragma unroll
        for (int e = 0; e < 4; ++e) U[e] = fmaf(w, u[k][e], U[e]);
      }
  }
  if (real) {
    const int rr = it.r0 + r;
    const long long o =
        (static_cast<long long>(s.q0 + rr / c.t.G) * c.t.H * c.t.G + h * c.t.G + rr % c.t.G) * D + f;
    const float inv = nan ? NAN : (Z > 0.f ? 1.f / Z : 0.f);
    __nv_bfloat162 lo = __floats2bfloat162_rn(U[0] * inv, U[1] * inv), hi = __floats2bfloat162_rn(U[2] * inv, U[3] * inv);
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(c.O) + o) =
        make_uint2(*reinterpret_cast<unsigned*>(&lo), *reinterpret_cast<unsigned*>(&hi));
  }
}

}  // namespace

kvq_status launch_plan(const AttendArgs& a, const PlanMem& m, int RI, int BT, cudaStream_t s) {
  const size_t smem = (static_cast<size_t>(a.S) + 1) * sizeof(int);
  if (!ensure_dynamic_smem(reinterpret_cast<const void*>(plan_kernel), smem)) return KVQ_ERR_CUDA;
  unsigned int* err = error_word();
  if (!err) return KVQ_ERR_CUDA;
  if (launch_pdl(plan_kernel, dim3(1), dim3(kPlanThreads), smem, s, make_batch(a), m, RI, BT,
                 static_cast<int>(plan_items(a, RI)), err) != cudaSuccess)
    return KVQ_ERR_CUDA;
  count_launch();
  return KVQ_OK;
}

kvq_status launch_merge(const MergeCall& c, cudaStream_t s) {
  MergeParams p{c, error_word()};
  if (!p.err) return KVQ_ERR_CUDA;
  const long long grid = c.items * c.t.H;
  if (grid > 0x7fffffffLL) return KVQ_ERR_UNSUPPORTED;
  const size_t smem = c.plan.count ? 0 : (static_cast<size_t>(c.t.S) + 1) * sizeof(int);
  if (c.tile_rows > 0) {
    if (!ensure_dynamic_smem(reinterpret_cast<const void*>(merge_tiles_kernel), smem)) return KVQ_ERR_CUDA;
    const int tiles = c.RI > c.tile_rows ? 2 : 1;
    const int last = c.RI - (tiles - 1) * c.tile_rows;                 // rows of the last tile
    if (launch_pdl(merge_tiles_kernel,
                   dim3(static_cast<unsigned>(grid), 4 * (tiles - 1) + (last + 31) / 32, c.D / 32), dim3(256), smem, s,
                   p) != cudaSuccess)
      return KVQ_ERR_CUDA;
    count_launch();
    return KVQ_OK;
  }
  if (!ensure_dynamic_smem(reinterpret_cast<const void*>(merge_rows_kernel), smem)) return KVQ_ERR_CUDA;
  if (launch_pdl(merge_rows_kernel, dim3(static_cast<unsigned>(grid)), dim3(kMergeThreads), smem, s, p) !=
      cudaSuccess)
    return KVQ_ERR_CUDA;
  count_launch();
  return KVQ_OK;
}

}  // namespace paged
}  // namespace kvq
