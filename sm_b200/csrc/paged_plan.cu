// Paged attention: the item list of a ragged batch, and the merge of the
// states that several workers computed for one (item, KV head).
//
// The merge is the block rule of "Block KV decoding: less workspace, more
// time" (huhohoo.com/en/docs/llm/kv-block-decode-cost, section "Do not average
// independently normalized blocks"): M = max m_c, w_c = 2^(m_c - M),
// O = sum w_c u_c / sum w_c z_c over the parts c that hold a key.  It is
// bound by latency: the m and z of up to 32 parts come in one round (lane =
// part), the u rows in a second whose loads do not depend on one another.  (9 us
// with cold caches, of which the launch and the plan run beside the attention.)
#include "paged.cuh"

namespace kvq {
namespace paged {
namespace {

constexpr int kPlanThreads = 1024;

// Sum of two counts of items, held below 2^30: a cu that is not as stated can
// give the sequences more rows than there are, and the prefix must stay ordered.
__device__ __forceinline__ int add(int a, int b) { return min(a + b, 0x3fffffff); }
// Of blocks: at most 2^30 items of 2^26 each.
__device__ __forceinline__ long long add(long long a, long long b) { return a + b; }

// Inclusive scan of one count per thread over the CTA.
template <typename T>
__device__ __forceinline__ T block_scan(T v, T* s_warp) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T n = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v = add(v, n);
  }
  if (lane == 31) s_warp[w] = v;
  __syncthreads();
  if (w == 0) {
    T x = s_warp[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const T n = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x = add(x, n);
    }
    s_warp[lane] = x;
  }
  __syncthreads();
  const T before = w > 0 ? s_warp[w - 1] : T(0);
  __syncthreads();
  return add(v, before);
}

// One CTA.  Item counts of the sequences are summed into s_first (shared memory,
// sequences 1024 at a time), then the items' block counts into the plan.
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(Batch t, PlanMem m, int RI, int BT, int max_items,
                                                            unsigned int* err) {
  griddep_wait();
  extern __shared__ int s_first[];              // [S + 1] first item of each sequence
  __shared__ int s_warp[32];
  __shared__ long long s_warp_blocks[32];
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
    if (b < t.S) s_first[b + 1] = add(carry, inc);
    __syncthreads();
    carry = s_first[min(base + kPlanThreads, t.S)];
  }
  if (threadIdx.x == 0) s_first[0] = 0;
  __syncthreads();
  const int items = min(s_first[t.S], max_items);
  long long blocks = 0;
  for (int base = 0; base < items; base += kPlanThreads) {
    const int i = base + static_cast<int>(threadIdx.x);
    long long v = 0;
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
    const long long inc = block_scan(v, s_warp_blocks);
    if (i < items) m.pre[i + 1] = add(blocks, inc);
    if (threadIdx.x == kPlanThreads - 1) s_warp_blocks[0] = inc;
    __syncthreads();
    blocks = add(blocks, s_warp_blocks[0]);
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
  int by_item;           // a unit is an (item, head); else a boundary between two workers
  int units;             // units of the launch; CTAs past them write the rows of items without a key
};

struct Parts {
  int i, h;
  Item it;
  SeqView s;
  int rows;              // rows of the item
  long long c_first;     // first worker
  int n;                 // workers (0: no key, zero rows)
  bool first_is_start;   // the first worker's range begins at this head's first block
  bool mine;             // this unit merges it
};

// The (item, head) of a unit and the workers whose ranges meet its blocks.
// Where there are more (item, head)s than workers, the units are the
// boundaries between workers: the first boundary inside an (item, head)
// merges it, and the many that one worker covers cost nothing.
// (By a whole warp.)
__device__ __forceinline__ Parts find_parts(const MergeParams& p, const PlanView& v, int unit) {
  const MergeCall& c = p.c;
  const int H = c.t.H;
  Parts q{};
  const Range r = worker_range(v, H, c.workers, 0, c.spread);
  long long start;
  int nb;
  if (p.by_item) {
    q.i = unit / H;
    q.h = unit % H;
    if (q.i >= v.items) return q;
    nb = v.blocks(q.i);
    start = static_cast<long long>(H) * v.pre[q.i] + static_cast<long long>(q.h) * nb;
    q.mine = true;
  } else {
    const long long x = (unit + 1) * r.per;
    if (x >= r.total) return q;
    q.i = find_item(v, H, x);
    nb = v.blocks(q.i);
    q.h = static_cast<int>((x - static_cast<long long>(H) * v.pre[q.i]) / nb);
    start = static_cast<long long>(H) * v.pre[q.i] + static_cast<long long>(q.h) * nb;
    q.mine = x > start && x - r.per <= start;
    if (!q.mine) return q;
  }
  q.it = plan_item(v, q.i);
  q.s = seq_view(c.t, q.it.b);
  q.rows = min(c.RI, q.s.n * c.t.G - q.it.r0);
  if (nb > 0) {
    q.c_first = start / r.per;
    q.n = static_cast<int>((start + nb - 1) / r.per - q.c_first + 1);
    q.first_is_start = q.c_first * r.per == start;
  }
  if (q.n == 1) q.mine = false;                // that worker wrote the rows
  return q;
}

// Slot of part k: every worker after the first begins inside this head's
// blocks; the first does only if its range starts exactly at them.
__device__ __forceinline__ long long part_slot(const Parts& p, int k) {
  return 2 * (p.c_first + k) + ((k > 0 || p.first_is_start) ? 0 : 1);
}

// Row r of item row space within O's [T, H_q] rows.
__device__ __forceinline__ long long out_row(const MergeCall& c, const Parts& q, int r) {
  const int rr = q.it.r0 + r;
  return static_cast<long long>(q.s.q0 + rr / c.t.G) * (c.t.H * c.t.G) + q.h * c.t.G + rr % c.t.G;
}

__device__ __forceinline__ float exp2_w(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The plan, the unit's parts (computed by one warp: their 64-bit divisions run
// once per CTA) and the wait for the attention kernel.  The inline plan reads
// only the call's inputs (through the L2), so it runs while that kernel
// drains; the workspace's plan is read after the wait.
__device__ __forceinline__ PlanView merge_prologue(const MergeParams& p, int unit, long long* s_pre,
                                                   Parts* s_parts) {
  const bool global = p.c.plan.count != nullptr;
  if (global) griddep_wait();
  if (threadIdx.x < 32) {
    if (!global) warp_prefix(p.c.t, p.c.RI, p.c.BT, s_pre);
    __syncwarp();
    Parts q{};
    if (unit < p.units) q = find_parts(p, plan_view(p.c.plan, s_pre, p.c.t.S), unit);
    if (threadIdx.x == 0) *s_parts = q;
  }
  __syncthreads();
  if (!global) griddep_wait();
  return plan_view(p.c.plan, s_pre, p.c.t.S);
}

// CTA `z` of `nz` that look after what no unit does: zero rows for the items
// without a key (units by boundary), and the report of bad sequences (inline
// plan; plan_kernel reports its own).
__device__ __forceinline__ void odd_jobs(const MergeParams& p, const PlanView& v, int z, int nz) {
  const MergeCall& c = p.c;
  if (!c.plan.count)
    for (int b = z * static_cast<int>(blockDim.x) + static_cast<int>(threadIdx.x); b < c.t.S; b += nz * blockDim.x)
      if (seq_view(c.t, b).bad) record_error(p.err, KVQ_ERR_LENGTH);
  if (p.by_item) return;
  for (int i = z; i < v.items; i += nz) {
    if (v.blocks(i) != 0) continue;
    Parts q{};
    q.it = plan_item(v, i);
    q.s = seq_view(c.t, q.it.b);
    const int rows = min(c.RI, q.s.n * c.t.G - q.it.r0);
    for (int h = 0; h < c.t.H; ++h) {
      q.h = h;
      for (int x = threadIdx.x; x < rows * c.D; x += blockDim.x)
        store_from_f32(c.O, out_row(c, q, x / c.D) * c.D + x % c.D, 0.f, c.o_dtype);
    }
  }
}

// Row-major partials: one CTA per unit and row.  Its four warps divide the
// parts; a warp loads the (m, z) of 32 parts at once (lane = part), then the u
// rows of its own parts with independent 16-byte loads, eight in flight, and
// the warps' sums meet in shared memory.  kVec: D a multiple of 4.
constexpr int kMergeWarps = 4;
template <bool kVec>
__global__ void __launch_bounds__(32 * kMergeWarps) merge_rows_kernel(MergeParams p) {
  extern __shared__ long long s_pre[];
  __shared__ Parts s_parts;
  __shared__ float s_u[kMergeWarps][256];
  const MergeCall& c = p.c;
  const int unit = blockIdx.x, r = blockIdx.y;
  const PlanView v = merge_prologue(p, unit, s_pre, &s_parts);
  if (unit >= p.units) {
    if (r == 0) odd_jobs(p, v, unit - p.units, gridDim.x - p.units);
    return;
  }
  const Parts q = s_parts;
  if (!q.mine || r >= q.rows) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int D = c.D;
  const long long stride = static_cast<long long>(c.RI) * (D + 2);
  const float* mz0 = c.partials + static_cast<long long>(c.RI) * D + 2 * r;
  constexpr int F = 8;                         // features of a lane: 4 lane + 128 j .. + 3, or lane + 32 j
  float M = -INFINITY, Z = 0.f, U[F];
  bool nan = false;                            // a part whose sum is not a number: neither is the row
#pragma unroll
  for (int j = 0; j < F; ++j) U[j] = 0.f;
  for (int k0 = 0; k0 < q.n; k0 += 32) {
    const int k = k0 + lane;
    float m = -INFINITY, z = 0.f;
    if (k < q.n) {
      const float2 mz = *reinterpret_cast<const float2*>(mz0 + part_slot(q, k) * stride);
      z = mz.y;
      m = z > 0.f ? mz.x : -INFINITY;
    }
    nan |= __any_sync(0xffffffffu, z != z);
    float top = m;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
    top = fmaxf(top, M);
    if (top == -INFINITY) continue;
    const float keep = exp2_w(M - top), w = exp2_w(m - top);
    float zs = w * z;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) zs += __shfl_xor_sync(0xffffffffu, zs, x);
    M = top;
    Z = Z * keep + zs;
#pragma unroll
    for (int j = 0; j < F; ++j) U[j] *= keep;
    const int n = min(32, q.n - k0);
#pragma unroll
    for (int jj = 0; jj < 32 / kMergeWarps; ++jj) {
      const int j = jj * kMergeWarps + warp;
      const float wj = __shfl_sync(0xffffffffu, w, j);
      if (j < n && wj > 0.f) {                 // a part without a key holds nothing
        const float* u = c.partials + part_slot(q, k0 + j) * stride + static_cast<long long>(r) * D;
        if (kVec) {
#pragma unroll
          for (int e = 0; e < F; e += 4)
            if (4 * lane + 32 * e < D) {
              const float4 x = *reinterpret_cast<const float4*>(u + 4 * lane + 32 * e);
              U[e] = fmaf(wj, x.x, U[e]);
              U[e + 1] = fmaf(wj, x.y, U[e + 1]);
              U[e + 2] = fmaf(wj, x.z, U[e + 2]);
              U[e + 3] = fmaf(wj, x.w, U[e + 3]);
            }
        } else {
#pragma unroll
          for (int e = 0; e < F; ++e)
            if (lane + 32 * e < D) U[e] = fmaf(wj, u[lane + 32 * e], U[e]);
        }
      }
    }
  }
#pragma unroll
  for (int e = 0; e < F; ++e) {
    const int f = kVec ? 4 * lane + 128 * (e >> 2) + (e & 3) : lane + 32 * e;
    if (f < D) s_u[warp][f] = U[e];
  }
  __syncthreads();
  const float inv = nan ? NAN : (Z > 0.f ? 1.f / Z : 0.f);
  const long long o = out_row(c, q, r) * D;
  for (int f = threadIdx.x; f < D; f += 32 * kMergeWarps) {
    float x = 0.f;
#pragma unroll
    for (int k = 0; k < kMergeWarps; ++k) x += s_u[k][f];
    store_from_f32(c.O, o + f, x * inv, c.o_dtype);
  }
}

// Feature-major partials: one CTA per unit and 32-row chunk (blockIdx.y); lane =
// row, a warp takes D / 8 features, four at a time, two parts' loads in flight.
// (With a CTA for 32 features each, the unit's parts were looked for four times
// as often: five prompts took 397 instead of 385 us.)
template <int D>
__global__ void __launch_bounds__(256) merge_tiles_kernel(MergeParams p) {
  extern __shared__ long long s_pre[];
  __shared__ Parts s_parts;
  const MergeCall& c = p.c;
  const PlanView v = merge_prologue(p, blockIdx.x, s_pre, &s_parts);
  if (static_cast<int>(blockIdx.x) >= p.units) {
    if (blockIdx.y == 0) odd_jobs(p, v, blockIdx.x - p.units, gridDim.x - p.units);
    return;
  }
  const Parts q = s_parts;
  if (!q.mine) return;
  constexpr int F = D / 8, PB = 2;
  const int lane = threadIdx.x & 31, f = F * (threadIdx.x >> 5);
  const int pr = 32 * blockIdx.y + lane, tile = pr >> 7;               // padded row of the slot
  const int r = tile * c.tile_rows + (pr & 127);
  const bool real = (pr & 127) < c.tile_rows && r < q.rows;
  if (!__any_sync(0xffffffffu, real)) return;
  const long long stride = 256LL * (D + 2);
  const float* base = c.partials + static_cast<long long>(blockIdx.y) * (D + 2) * 32 + lane;
  float M = -INFINITY, Z = 0.f, U[F];
#pragma unroll
  for (int e = 0; e < F; ++e) U[e] = 0.f;
  bool nan = false;
  for (int k0 = 0; k0 < q.n; k0 += PB) {
    float m[PB], z[PB], u[PB][F];
#pragma unroll
    for (int k = 0; k < PB; ++k) {
      m[k] = -INFINITY;
      z[k] = 0.f;
      if (k0 + k < q.n && real) {
        const float* part = base + part_slot(q, k0 + k) * stride;
        m[k] = part[0];
        z[k] = part[32];
#pragma unroll
        for (int e = 0; e < F; ++e) u[k][e] = part[(2 + f + e) * 32];
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
    for (int e = 0; e < F; ++e) U[e] *= keep;
#pragma unroll
    for (int k = 0; k < PB; ++k)
      if (z[k] > 0.f) {
        const float w = exp2_w(m[k] - top);
        Z = fmaf(w, z[k], Z);
#pragma unroll
        for (int e = 0; e < F; ++e) U[e] = fmaf(w, u[k][e], U[e]);
      }
  }
  if (real) {
    const long long o = out_row(c, q, r) * D + f;
    const float inv = nan ? NAN : (Z > 0.f ? 1.f / Z : 0.f);
    uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(c.O) + o);
#pragma unroll
    for (int e = 0; e < F; e += 8) {
      unsigned x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(U[e + 2 * i] * inv, U[e + 2 * i + 1] * inv);
        x[i] = *reinterpret_cast<const unsigned*>(&b);
      }
      dst[e / 8] = make_uint4(x[0], x[1], x[2], x[3]);
    }
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
  MergeParams p{};
  p.c = c;
  p.err = error_word();
  if (!p.err) return KVQ_ERR_CUDA;
  const long long heads = c.items * c.t.H;
  // (By item throughout, 1000 sequences of 8 rows take 1709 instead of 494 us: the
  // CTAs of items that one worker covered look up their parts for nothing.)
  p.by_item = heads <= c.workers;
  p.units = p.by_item ? static_cast<int>(heads) : c.workers - 1;
  // one more CTA reports bad sequences; with units by boundary a few look for
  // items without a key
  const unsigned gx = static_cast<unsigned>(p.units) + (p.by_item ? 1 : 16);
  const size_t smem = c.plan.count ? 0 : (static_cast<size_t>(c.t.S) + 1) * sizeof(long long);
  cudaError_t e;
  if (c.tile_rows > 0) {
    auto kernel = c.D == 64 ? merge_tiles_kernel<64> : merge_tiles_kernel<128>;
    if (!ensure_dynamic_smem(reinterpret_cast<const void*>(kernel), smem)) return KVQ_ERR_CUDA;
    const int tiles = c.RI > c.tile_rows ? 2 : 1;
    const int last = c.RI - (tiles - 1) * c.tile_rows;                 // rows of the last tile
    e = launch_pdl(kernel, dim3(gx, 4 * (tiles - 1) + (last + 31) / 32), dim3(256), smem, s, p);
  } else {
    auto kernel = c.D % 4 == 0 ? merge_rows_kernel<true> : merge_rows_kernel<false>;
    if (!ensure_dynamic_smem(reinterpret_cast<const void*>(kernel), smem)) return KVQ_ERR_CUDA;
    const long long most = static_cast<long long>(c.t.max_q) * c.t.G;  // rows an item can have
    e = launch_pdl(kernel, dim3(gx, static_cast<unsigned>(most < c.RI ? most : c.RI)), dim3(32 * kMergeWarps), smem, s,
                   p);
  }
  if (e != cudaSuccess) return KVQ_ERR_CUDA;
  count_launch();
  return KVQ_OK;
}

}  // namespace paged
}  // namespace kvq
