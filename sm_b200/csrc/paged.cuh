// Shared by the paged-cache kernels: a sequence's rows and keys in a ragged
// batch, page lookup, the work plan of the attention kernels and their host
// arguments.
#pragma once
#include "kvq_internal.cuh"

namespace kvq {
namespace paged {

// ---------------------------------------------------------------------------
// ragged batch
// ---------------------------------------------------------------------------
// Rows [r0, r0 + n) of the call's row tensors belong to the sequence.  A cu
// that decreases, passes T or holds more than max_rows rows is clamped
// (`bad` is set), so no index a kernel forms leaves its buffer.
struct RowRange {
  int r0, n;
  bool bad;
};
__device__ __forceinline__ RowRange row_range(int c0, int c1, int T, int max_rows) {
  RowRange r;
  r.r0 = min(max(c0, 0), T);
  const int r1 = min(max(c1, r.r0), T);
  r.n = min(r1 - r.r0, max_rows);
  r.bad = c0 != r.r0 || c1 != r1 || r.n != r1 - r.r0;
  return r;
}

__device__ __forceinline__ RowRange row_range(const int32_t* cu, int b, int T, int max_rows) {
  return row_range(__ldcg(cu + b), __ldcg(cu + b + 1), T, max_rows);
}

// Page number of a block-table entry for reading: one outside the pool is
// recorded and read as page 0.
__device__ __forceinline__ int read_page(int page, int pages, unsigned int* err) {
  if (static_cast<unsigned>(page) < static_cast<unsigned>(pages)) return page;
  record_error(err, KVQ_ERR_INDEX);
  return 0;
}

// ---------------------------------------------------------------------------
// host arguments of append and gather
// ---------------------------------------------------------------------------
struct AppendCall {
  const kvq_paged_cache* cache;
  Geometry g;
  const void* K;
  const void* V;
  long long k_stride, v_stride;
  int in_dtype;
  const int32_t* table;
  int max_pages;
  const int32_t* lengths;
  const int32_t* cu;
  const int32_t* slots;
  int S, T, max_new;
  kvq_rope rope;
};
kvq_status launch_append(const AppendCall& a, cudaStream_t s);

struct GatherCall {
  const kvq_paged_cache* cache;
  Geometry g;
  const int32_t* table;
  int max_pages;
  const int32_t* starts;
  const int32_t* cu;
  int S, T, max_rows;
  void* K;
  void* V;
  int out_dtype;
};
kvq_status launch_gather(const GatherCall& a, cudaStream_t s);

// ---------------------------------------------------------------------------
// attention work plan
// ---------------------------------------------------------------------------
// The query rows of (sequence, KV head) -- token-major: row r is token r / G,
// head r % G of the group -- are cut into items of at most RI rows.  An item's
// keys are the tokens its last row sees, in blocks of BT.  The blocks of all
// items are listed item-major, then KV head, then block, and W workers take
// equal contiguous ranges of the list.  A worker that covers part of an (item,
// head) leaves a partial state (m, z, u); only the first and the last segment
// of a worker's range can be partial, so slot 2 w holds the segment its range
// begins in and 2 w + 1 the one it ends in.
struct Item {
  int b;        // sequence
  int r0;       // first row within the sequence's n * G rows
};

// (64 bits: f32 rows have an item a few rows, and 2^17 of these over 2^19 keys are
// 2^31 blocks, a matter of seconds.)
struct PlanView {
  const long long* pre; // [items + 1] prefix of block counts (one head)
  const Item* item;     // nullptr: item i is sequence i, row 0
  int items;
  // blocks of item i (below 2^26: the low words' difference)
  __device__ __forceinline__ int blocks(int i) const {
    return static_cast<int>(static_cast<unsigned>(pre[i + 1]) - static_cast<unsigned>(pre[i]));
  }
};

struct AttendArgs {
  const void* Q;
  int q_dtype;
  Geometry g;                    // g.B pages of g.N_cap tokens
  const uint8_t* k_codes;
  const float* k_scales;
  const uint8_t* v_codes;
  const float* v_scales;
  const int32_t* table;
  int max_pages;
  const int32_t* lengths;
  const int32_t* cu;
  int S, T, max_q, H_q, G;
  float scale;
  int causal;
  void* O;
  void* workspace;
  int splits;
};

// What the device side of the plan, the kernels and the merge read.
struct Batch {
  const int32_t* lengths;
  const int32_t* cu;
  const int32_t* table;
  int max_pages, S, T, max_q, G, H, P, pages, cap;   // cap = max_pages * P
  int causal;
};
inline Batch make_batch(const AttendArgs& a) {
  return Batch{a.lengths, a.cu, a.table, a.max_pages, a.S, a.T, a.max_q, a.G, a.g.H_kv, a.g.N_cap, a.g.B,
               a.max_pages * a.g.N_cap, a.causal};
}

struct SeqView {
  int q0, n, len;       // first row, rows, keys (clamped)
  bool bad;
};
__device__ __forceinline__ SeqView seq_view(const Batch& t, int b) {
  const RowRange r = row_range(t.cu, b, t.T, t.max_q);
  const int raw = __ldcg(t.lengths + b);
  SeqView s;
  s.q0 = r.r0;
  s.n = r.n;
  s.len = min(max(raw, 0), t.cap);
  s.bad = r.bad || (r.n > 0 && (raw < 1 || raw > t.cap || (t.causal && raw < r.n)));
  return s;
}
// Keys that row r (of the sequence's n * G) sees: tokens [0, limit).
__device__ __forceinline__ int row_limit(const Batch& t, const SeqView& s, int r) {
  return t.causal ? max(0, min(s.len, s.len - s.n + r / t.G + 1)) : s.len;
}
// Blocks of an item of at most RI rows from row r0 (its last row sees most).
__device__ __forceinline__ int item_blocks(const Batch& t, const SeqView& s, int r0, int RI, int BT) {
  const int rows = s.n * t.G;
  if (r0 >= rows) return 0;
  const int last = min(rows, r0 + RI) - 1;
  return (row_limit(t, s, last) + BT - 1) / BT;
}

// Largest item i with H * pre[i] <= g; by a whole warp, 32 probes a round.
__device__ __forceinline__ int find_item(const PlanView& v, int H, long long g) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = v.items;
  while (n > 1) {
    const int step = (n + 31) / 32, at = lane * step;
    const bool le = at < n && static_cast<long long>(H) * v.pre[lo + at] <= g;
    const int k = __popc(__ballot_sync(0xffffffffu, le));
    if (k == 0) break;
    lo += (k - 1) * step;
    n = min(step, n - (k - 1) * step);
  }
  return lo;
}

struct Range {
  long long g0, g1, per, total;
};
// spread > 0: a worker takes at least sqrt(spread * blocks of an average (item,
// head)) blocks, fewer workers with fewer parts to join than there could be: with
// t a block's time and u that of joining a part, n blocks over w workers take n /
// w t + w u, least at n / w = sqrt(n u / t).
__device__ __forceinline__ Range worker_range(const PlanView& v, int H, int workers, long long w, float spread = 0.f) {
  Range r;
  r.total = static_cast<long long>(H) * v.pre[v.items];
  r.per = (r.total + workers - 1) / workers;
  if (spread > 0.f && v.items > 0) {
    const float n = static_cast<float>(v.pre[v.items]) / static_cast<float>(v.items);
    r.per = max(r.per, static_cast<long long>(sqrtf(spread * n) + 0.5f));
  }
  r.g0 = min(r.total, w * r.per);
  r.g1 = min(r.total, r.g0 + r.per);
  return r;
}

// Host: an upper bound of the items of a call, and how its plan is made.  A
// call whose sequences have one item each (max_q * G <= RI) needs no item
// list: every CTA sums the block prefix over the sequences itself (S <=
// kMaxInline of them).  Otherwise plan_kernel writes the list to the workspace:
// one row a sequence over 1024 keys takes (inline / plan, us) 22 / 27 for 32
// sequences, 57 / 58 for 96, 73 / 70 for 128, 147 / 122 for 256.
constexpr int kMaxInline = 96;
inline bool plan_inline(const AttendArgs& a, int RI) {
  return static_cast<long long>(a.max_q) * a.G <= RI && a.S <= kMaxInline;
}
inline long long plan_items(const AttendArgs& a, int RI) {
  if (plan_inline(a, RI)) return a.S;
  // sum over b of ceil(n_b G / RI) <= T G / RI + S, and <= S ceil(max_q G / RI)
  const long long by_rows = static_cast<long long>(a.T) * a.G / RI + a.S;
  const long long by_seq = static_cast<long long>(a.S) * ((static_cast<long long>(a.max_q) * a.G + RI - 1) / RI);
  return by_rows < by_seq ? by_rows : by_seq;
}
inline size_t align16(size_t n) { return (n + 15) / 16 * 16; }
// Workspace bytes of the plan: count, pre[items + 1], item[items].
inline size_t plan_bytes(const AttendArgs& a, int RI) {
  if (plan_inline(a, RI)) return 0;
  const size_t n = static_cast<size_t>(plan_items(a, RI));
  return align16(16 + (n + 1) * sizeof(long long)) + align16(n * sizeof(Item));
}
struct PlanMem {
  int* count;           // nullptr: in-kernel prefix
  long long* pre;
  Item* item;
};
inline PlanMem plan_mem(const AttendArgs& a, int RI, void* ws) {
  if (plan_inline(a, RI)) return PlanMem{nullptr, nullptr, nullptr};
  char* p = static_cast<char*>(ws);
  const size_t n = static_cast<size_t>(plan_items(a, RI));
  return PlanMem{reinterpret_cast<int*>(p), reinterpret_cast<long long*>(p + 16),
                 reinterpret_cast<Item*>(p + align16(16 + (n + 1) * sizeof(long long)))};
}
kvq_status launch_plan(const AttendArgs& a, const PlanMem& m, int RI, int BT, cudaStream_t s);

// One warp: the block prefix over the sequences, into pre[0..S] (shared
// memory; the caller synchronises).
__device__ __forceinline__ void warp_prefix(const Batch& t, int RI, int BT, long long* pre) {
  const int lane = threadIdx.x & 31;
  long long carry = 0;
  for (int base = 0; base < t.S; base += 32) {
    const int b = base + lane;
    long long v = 0;
    if (b < t.S) v = item_blocks(t, seq_view(t, b), 0, RI, BT);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long n = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += n;
    }
    if (b < t.S) pre[b + 1] = carry + v;
    carry += __shfl_sync(0xffffffffu, v, 31);
  }
  if (lane == 0) pre[0] = 0;
}

// The view a kernel uses: the workspace's plan, or the CTA's own prefix.
__device__ __forceinline__ PlanView plan_view(const PlanMem& m, const long long* s_pre, int S) {
  if (m.count) return PlanView{m.pre, m.item, *m.count};
  return PlanView{s_pre, nullptr, S};
}
__device__ __forceinline__ Item plan_item(const PlanView& v, int i) {
  return v.item ? v.item[i] : Item{i, 0};
}

// ---------------------------------------------------------------------------
// merge of partial states
// ---------------------------------------------------------------------------
// partials: [2 * workers slots][RI * D + RI * 2] (u rows, then (m, z) per row;
// m in log2 units), or feature-major [slots][8][D + 2][32]: fields m, z, u of
// 32 rows each, tile t's rows from 128 t on.
struct MergeCall {
  Batch t;
  PlanMem plan;
  long long items;               // launch bound
  int RI, BT, workers, D;
  float spread;                  // of worker_range
  const float* partials;
  void* O;
  int o_dtype;
  int tile_rows;                 // feature-major: rows of a tile (0: row-major)
};
kvq_status launch_merge(const MergeCall& c, cudaStream_t s);

struct AttendImpl {
  const char* name;
  bool (*applies)(const AttendArgs&);
  size_t (*workspace)(const AttendArgs&);
  kvq_status (*launch)(const AttendArgs&, cudaStream_t);
};
const AttendImpl& generic_impl();
const AttendImpl& rows_impl();       // few rows a KV head
const AttendImpl& chunk_impl();      // many rows a KV head

}  // namespace paged
}  // namespace kvq
