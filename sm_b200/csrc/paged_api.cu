// C ABI of the paged cache: argument rules and dispatch.
#include "paged.cuh"

namespace kvq {
namespace paged {
namespace {

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// The pool's geometry; false for an invalid one.
bool pool_geometry(const kvq_paged_cache* c, Geometry* g) {
  if (!c || !make_geometry(&c->pages, g)) return false;
  return c->pages.N_cap % c->pages.group == 0;      // a K group lies in one page
}

// Rules that every call on a paged cache shares.
kvq_status check_pool(const kvq_paged_cache* c, const int32_t* table, int32_t max_pages, const int32_t* lengths,
                      const int32_t* cu, int32_t S, int32_t T, int32_t max_rows, Geometry* g) {
  if (!pool_geometry(c, g)) return KVQ_ERR_ARG;
  if (!c->pages.k_codes || !c->pages.k_scales || !c->pages.v_codes || !c->pages.v_scales) return KVQ_ERR_ARG;
  if (!table || !lengths || !cu) return KVQ_ERR_ARG;
  if (S < 1 || T < 1 || max_rows < 1 || max_pages < 1) return KVQ_ERR_ARG;
  if (static_cast<int64_t>(max_pages) * c->pages.N_cap > 0x7fffff00LL) return KVQ_ERR_ARG;
  if (S > 8192 || c->pages.D > 256 || c->pages.H_kv > 65535) return KVQ_ERR_UNSUPPORTED;
  if (!aligned(c->pages.k_codes, 16) || !aligned(c->pages.k_scales, 16) || !aligned(c->pages.v_codes, 16) ||
      !aligned(c->pages.v_scales, 16))
    return KVQ_ERR_ALIGN;
  if (!aligned(table, 4) || !aligned(lengths, 4) || !aligned(cu, 4)) return KVQ_ERR_ALIGN;
  return KVQ_OK;
}

const AttendImpl& choose(const AttendArgs& a) {
  if (chunk_impl().applies(a)) return chunk_impl();
  return rows_impl().applies(a) ? rows_impl() : generic_impl();
}

bool fill_sizes(const kvq_paged_cache* c, kvq_dtype q_dtype, int32_t S, int32_t T, int32_t max_q, int32_t H_q,
                int32_t splits, AttendArgs* a) {
  if (!pool_geometry(c, &a->g)) return false;
  if (q_dtype != KVQ_F32 && q_dtype != KVQ_BF16) return false;
  if (S < 1 || T < 1 || max_q < 1 || splits < 0 || H_q < 1 || H_q % c->pages.H_kv) return false;
  a->q_dtype = q_dtype;
  a->S = S;
  a->T = T;
  a->max_q = max_q < T ? max_q : T;
  a->H_q = H_q;
  a->G = H_q / c->pages.H_kv;
  a->splits = splits;
  return true;
}

}  // namespace
}  // namespace paged
}  // namespace kvq

using namespace kvq;
using namespace kvq::paged;

extern "C" {

kvq_status kvq_paged_append(const kvq_paged_cache* cache, const void* K, int64_t k_stride, const void* V,
                            int64_t v_stride, kvq_dtype in_dtype, const int32_t* block_table, int32_t max_pages,
                            const int32_t* lengths, const int32_t* cu_new, const int32_t* slots, int32_t S, int32_t T,
                            int32_t max_new, const kvq_rope* rope, void* stream) {
  AppendCall a{};
  const kvq_status st = check_pool(cache, block_table, max_pages, lengths, cu_new, S, T, max_new, &a.g);
  if (st != KVQ_OK) return st;
  if (!K || !V || !cache->k_tail || cache->tail_slots < 1) return KVQ_ERR_ARG;
  if (in_dtype != KVQ_F32 && in_dtype != KVQ_BF16) return KVQ_ERR_ARG;
  const int64_t width = static_cast<int64_t>(cache->pages.H_kv) * cache->pages.D;
  if (k_stride < width || v_stride < width) return KVQ_ERR_ARG;
  if (rope && rope->table &&
      (rope->rot_dim < 2 || (rope->rot_dim & 1) || rope->rot_dim > cache->pages.D || rope->n_pos < 1))
    return KVQ_ERR_ARG;
  if (static_cast<int64_t>(cache->pages.group) * cache->pages.D > 32768) return KVQ_ERR_UNSUPPORTED;
  const size_t esz = in_dtype == KVQ_F32 ? 4 : 2;
  if (!aligned(K, esz) || !aligned(V, esz) || !aligned(cache->k_tail, 16) || !aligned(slots, 4) ||
      (rope && !aligned(rope->table, 4)))
    return KVQ_ERR_ALIGN;
  a.cache = cache;
  a.K = K;
  a.V = V;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.in_dtype = in_dtype;
  a.table = block_table;
  a.max_pages = max_pages;
  a.lengths = lengths;
  a.cu = cu_new;
  a.slots = slots;
  a.S = S;
  a.T = T;
  a.max_new = max_new;
  if (rope) a.rope = *rope;
  return launch_append(a, static_cast<cudaStream_t>(stream));
}

kvq_status kvq_paged_gather(const kvq_paged_cache* cache, const int32_t* block_table, int32_t max_pages,
                            const int32_t* starts, const int32_t* cu_rows, int32_t S, int32_t T, int32_t max_rows,
                            void* K, void* V, kvq_dtype out_dtype, void* stream) {
  GatherCall a{};
  const kvq_status st = check_pool(cache, block_table, max_pages, starts, cu_rows, S, T, max_rows, &a.g);
  if (st != KVQ_OK) return st;
  if (!K && !V) return KVQ_ERR_ARG;
  if (out_dtype != KVQ_F32 && out_dtype != KVQ_BF16) return KVQ_ERR_ARG;
  if (!aligned(K, 16) || !aligned(V, 16)) return KVQ_ERR_ALIGN;
  a.cache = cache;
  a.table = block_table;
  a.max_pages = max_pages;
  a.starts = starts;
  a.cu = cu_rows;
  a.S = S;
  a.T = T;
  a.max_rows = max_rows;
  a.K = K;
  a.V = V;
  a.out_dtype = out_dtype;
  return launch_gather(a, static_cast<cudaStream_t>(stream));
}

size_t kvq_paged_workspace_size(const kvq_paged_cache* cache, kvq_dtype q_dtype, int32_t S, int32_t T, int32_t max_q,
                                int32_t H_q, int32_t splits) {
  paged::AttendArgs a{};
  if (!fill_sizes(cache, q_dtype, S, T, max_q, H_q, splits, &a)) return 0;
  return choose(a).workspace(a);
}

kvq_status kvq_paged_attend(const void* Q, kvq_dtype q_dtype, const kvq_paged_cache* cache, const int32_t* block_table,
                            int32_t max_pages, const int32_t* lengths, const int32_t* cu_q, int32_t S, int32_t T,
                            int32_t max_q, int32_t H_q, float scale, int32_t causal, void* O, void* workspace,
                            size_t ws_bytes, int32_t splits, void* stream) {
  paged::AttendArgs a{};
  if (!fill_sizes(cache, q_dtype, S, T, max_q, H_q, splits, &a)) return KVQ_ERR_ARG;
  const kvq_status st = check_pool(cache, block_table, max_pages, lengths, cu_q, S, T, max_q, &a.g);
  if (st != KVQ_OK) return st;
  if (!Q || !O) return KVQ_ERR_ARG;
  if (static_cast<int64_t>(T) * H_q > 0x3fffffffLL) return KVQ_ERR_UNSUPPORTED;
  if (!aligned(Q, 16) || !aligned(O, 16)) return KVQ_ERR_ALIGN;
  const paged::AttendImpl& impl = choose(a);
  const size_t need = impl.workspace(a);
  if (!workspace || ws_bytes < need) return KVQ_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return KVQ_ERR_ALIGN;
  a.Q = Q;
  a.k_codes = cache->pages.k_codes;
  a.k_scales = cache->pages.k_scales;
  a.v_codes = cache->pages.v_codes;
  a.v_scales = cache->pages.v_scales;
  a.table = block_table;
  a.max_pages = max_pages;
  a.lengths = lengths;
  a.cu = cu_q;
  a.scale = scale;
  a.causal = causal != 0;
  a.O = O;
  a.workspace = workspace;
  return impl.launch(a, static_cast<cudaStream_t>(stream));
}

const char* kvq_paged_kernel_name(const kvq_paged_cache* cache, kvq_dtype q_dtype, int32_t max_q, int32_t H_q) {
  paged::AttendArgs a{};
  if (!fill_sizes(cache, q_dtype, 1, max_q, max_q, H_q, 0, &a)) return "invalid";
  return choose(a).name;
}

}  // extern "C"
