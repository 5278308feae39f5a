// api.cu -- the C ABI of libpagedattn (declared in include/pagedattn.h).
// Host code only: argument checks and the calls into dispatch.cu.
#include <cuda_runtime.h>

#include <cstdint>

#include "common.cuh"
#include "dispatch.h"
#include "kernels.h"
#include "pagedattn.h"

using namespace pa;

namespace {
bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Checks shared by decode and its traced variant; on success *plan is the
// call's plan on the current device.
int prepare_decode(const pa_dims* dims, const void* q, const void* k_cache, const void* v_cache,
                   const int32_t* block_table, const int32_t* context_lens, int32_t n_query,
                   int32_t causal, int32_t window, float scale, int32_t kv_dtype, const void* out,
                   Plan* plan) {
  int rc = check_dims(dims, n_query);
  if (rc != PA_OK) return rc;
  rc = check_decode_args(q, k_cache, v_cache, block_table, context_lens, causal, window, scale,
                         kv_dtype, out);
  if (rc != PA_OK) return rc;
  if (dims->workspace == nullptr || !aligned(dims->workspace, 256)) return PA_ERR_WORKSPACE;
  const int sms = device_sm_count();
  if (sms <= 0) return PA_ERR_CUDA;
  *plan = make_plan(dims, n_query, kv_dtype, sms);
  if (dims->workspace_bytes < ws_layout(dims, n_query, *plan).total) return PA_ERR_WORKSPACE;
  return PA_OK;
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// Workspace of a shared-prefix call: the decode layout (any device, so that
// the offsets behind it are the same everywhere), the groups' CTAs, which CTAs
// gave up, the partials.
struct SharedWs {
  size_t meta, gave_up, part_lse, part_out, total;
};
SharedPlan shared_plan(const pa_dims* d, int n_query, int kv_dtype, int sms) {
  return make_shared_plan(d->num_seqs, n_query * (d->num_q_heads / d->num_kv_heads), d->num_kv_heads,
                          kv_dtype, sms);
}
SharedWs shared_ws(const pa_dims* d, int n_query, const SharedPlan& pl) {
  SharedWs w;
  w.meta = align256(ws_size_any_device(d, n_query));
  w.gave_up = w.meta + align256((size_t)(1 + pl.groups) * 2 * sizeof(int));
  w.part_lse = w.gave_up + align256(kMaxPrefixCtas * sizeof(int));
  w.part_out = w.part_lse + align256((size_t)pl.part_rows * sizeof(float));
  w.total = w.part_out + (size_t)pl.part_rows * kHeadDim * sizeof(float);
  return w;
}
int check_shared(const pa_dims* d, int n_query, int prefix_blocks) {
  const int rc = check_dims(d, n_query);
  if (rc != PA_OK) return rc;
  if (prefix_blocks < 1) return PA_ERR_INVALID_ARG;
  // Keys are numbered in ints, up to a tile's end behind the last one.
  if ((long long)prefix_blocks * d->block_size > INT32_MAX - 256 ||
      (long long)d->max_blocks_per_seq * d->block_size > INT32_MAX - 256)
    return PA_ERR_UNSUPPORTED;
  return PA_OK;
}

// Workspace of the page operations: status header, per-request and per-page
// scratch.
struct PagesWs {
  size_t rows, pages, small, total;
};
PagesWs pages_ws(const pa_dims* d) {
  PagesWs w;
  w.rows = kWsHeader;
  w.pages = w.rows + align256((size_t)d->num_seqs * 3 * sizeof(int));
  w.small = w.pages + align256((size_t)d->num_blocks * 3 * sizeof(int));
  w.total = w.small + 256;
  return w;
}
// The checks and parameters that the page operations have in common.
int prepare_pages(const pa_dims* d, PageParams* p) {
  const int rc = check_dims(d, 1);
  if (rc != PA_OK) return rc;
  const PagesWs w = pages_ws(d);
  if (d->workspace == nullptr || !aligned(d->workspace, 256) || d->workspace_bytes < w.total)
    return PA_ERR_WORKSPACE;
  char* ws = static_cast<char*>(d->workspace);
  *p = PageParams{};
  p->num_seqs = d->num_seqs;
  p->max_blocks_per_seq = d->max_blocks_per_seq;
  p->block_size = d->block_size;
  p->num_blocks = d->num_blocks;
  p->flags = reinterpret_cast<unsigned*>(ws);
  p->row_scratch = reinterpret_cast<int*>(ws + w.rows);
  p->page_scratch = reinterpret_cast<int*>(ws + w.pages);
  p->small_scratch = reinterpret_cast<int*>(ws + w.small);
  return PA_OK;
}
// The same with the books.
int prepare_books(const pa_dims* d, int32_t* block_table, int32_t* context_lens,
                  int32_t* ref_counts, PageParams* p) {
  const int rc = prepare_pages(d, p);
  if (rc != PA_OK) return rc;
  if (!block_table || !context_lens || !ref_counts || !aligned(block_table, 4) ||
      !aligned(context_lens, 4) || !aligned(ref_counts, 4))
    return PA_ERR_INVALID_ARG;
  p->block_table = block_table;
  p->context_lens = context_lens;
  p->ref_counts = ref_counts;
  return PA_OK;
}
}  // namespace

extern "C" {

size_t paged_attn_workspace_size(const pa_dims* dims, int32_t n_query) {
  if (check_dims(dims, n_query) != PA_OK) return 0;
  return ws_size_any_device(dims, n_query);
}

int32_t paged_attn_num_splits(const pa_dims* dims, int32_t n_query, int32_t kv_dtype) {
  const int rc = check_dims(dims, n_query);
  if (rc != PA_OK) return rc;
  if (kv_dtype != PA_KV_FP16 && kv_dtype != PA_KV_Q8_0 && kv_dtype != PA_KV_INT8_ROW)
    return PA_ERR_INVALID_ARG;
  const int sms = device_sm_count();
  if (sms <= 0) return PA_ERR_CUDA;
  const Plan pl = make_plan(dims, n_query, kv_dtype, sms);
  if (pl.mode == 1) return pl.slots_per_group;
  if (pl.split_ctas > 0) {  // the per-head split kernel: CTAs per (sequence, KV head)
    const int groups = dims->num_seqs * dims->num_kv_heads;
    return (pl.split_ctas + groups - 1) / groups;
  }
  // A KV head's chunks span ceil(Ce / Hkv) ranges, plus one where they start
  // inside a range.
  return (pl.ctas_per_set + dims->num_kv_heads - 1) / dims->num_kv_heads + 1;
}

int32_t paged_attn_launches_per_call(const pa_dims* dims, int32_t n_query, int32_t kv_dtype) {
  const int rc = check_dims(dims, n_query);
  if (rc != PA_OK) return rc;
  if (kv_dtype != PA_KV_FP16 && kv_dtype != PA_KV_Q8_0 && kv_dtype != PA_KV_INT8_ROW)
    return PA_ERR_INVALID_ARG;
  const int sms = device_sm_count();
  if (sms <= 0) return PA_ERR_CUDA;
  return make_plan(dims, n_query, kv_dtype, sms).launches;
}

int paged_attn_workspace_init(const pa_dims* dims, void* stream) {
  if (dims == nullptr || dims->workspace == nullptr) return PA_ERR_WORKSPACE;
  if (check_dims(dims, 1) == PA_ERR_INVALID_ARG) return PA_ERR_INVALID_ARG;
  const size_t n = ws_zero_prefix(dims);
  if (dims->workspace_bytes < n) return PA_ERR_WORKSPACE;
  if (cudaMemsetAsync(dims->workspace, 0, n, static_cast<cudaStream_t>(stream)) != cudaSuccess)
    return PA_ERR_CUDA;
  return PA_OK;
}

int paged_attn_decode(const pa_dims* dims, const void* q, const void* k_cache,
                      const void* v_cache, const int32_t* block_table,
                      const int32_t* context_lens, int32_t n_query, int32_t causal,
                      int32_t window, float scale, int32_t kv_dtype, void* out,
                      void* stream) {
  Plan plan;
  const int rc = prepare_decode(dims, q, k_cache, v_cache, block_table, context_lens, n_query,
                                causal, window, scale, kv_dtype, out, &plan);
  if (rc != PA_OK) return rc;
  return enqueue_decode(dims, plan, q, k_cache, v_cache, block_table, context_lens, n_query,
                        causal, window, scale, kv_dtype, out, dims->workspace, nullptr,
                        static_cast<cudaStream_t>(stream));
}

int paged_attn_decode_partial(const pa_dims* dims, const void* q, const void* k_cache,
                              const void* v_cache, const int32_t* block_table,
                              const int32_t* context_lens, const int32_t* key_begin,
                              const int32_t* key_count, int32_t n_query, int32_t causal,
                              int32_t window, float scale, int32_t kv_dtype, float* out,
                              float* out_lse, void* stream) {
  if (!key_begin || !key_count || !out_lse || !aligned(key_begin, 4) || !aligned(key_count, 4) ||
      !aligned(out_lse, 4))
    return PA_ERR_INVALID_ARG;
  Plan plan;
  const int rc = prepare_decode(dims, q, k_cache, v_cache, block_table, context_lens, n_query,
                                causal, window, scale, kv_dtype, out, &plan);
  if (rc != PA_OK) return rc;
  PartialArgs pa_args;
  pa_args.key_begin = key_begin;
  pa_args.key_count = key_count;
  pa_args.out = out;
  pa_args.out_lse = out_lse;
  return enqueue_decode(dims, plan, q, k_cache, v_cache, block_table, context_lens, n_query,
                        causal, window, scale, kv_dtype, nullptr, dims->workspace, nullptr,
                        static_cast<cudaStream_t>(stream), pa_args);
}

size_t paged_attn_shared_workspace_size(const pa_dims* dims, int32_t n_query,
                                        int32_t prefix_blocks) {
  if (check_shared(dims, n_query, prefix_blocks) != PA_OK) return 0;
  size_t need = 0;
  for (int kv : {PA_KV_FP16, PA_KV_Q8_0})
    need = std::max(need, shared_ws(dims, n_query, shared_plan(dims, n_query, kv, kMaxPrefixCtas)).total);
  return need;
}

int paged_attn_decode_shared(const pa_dims* dims, const void* q, const void* k_cache,
                             const void* v_cache, const int32_t* block_table,
                             const int32_t* context_lens, const int32_t* prefix_table,
                             const int32_t* prefix_len, int32_t prefix_blocks, int32_t n_query,
                             int32_t causal, int32_t window, float scale, int32_t kv_dtype,
                             void* out, void* stream) {
  int rc = check_shared(dims, n_query, prefix_blocks);
  if (rc != PA_OK) return rc;
  if (!prefix_table || !prefix_len || !aligned(prefix_table, 4) || !aligned(prefix_len, 4))
    return PA_ERR_INVALID_ARG;
  Plan plan;
  rc = prepare_decode(dims, q, k_cache, v_cache, block_table, context_lens, n_query, causal, window,
                      scale, kv_dtype, out, &plan);
  if (rc != PA_OK) return rc;
  const int sms = device_sm_count();
  if (sms <= 0) return PA_ERR_CUDA;
  const SharedPlan spl = shared_plan(dims, n_query, kv_dtype, sms);
  const SharedWs w = shared_ws(dims, n_query, spl);
  if (dims->workspace_bytes < w.total) return PA_ERR_WORKSPACE;
  char* ws = static_cast<char*>(dims->workspace);
  SharedParams p{};
  p.q = static_cast<const __half*>(q);
  p.k = k_cache;
  p.v = v_cache;
  p.prefix_table = prefix_table;
  p.prefix_len = prefix_len;
  p.block_table = block_table;
  p.context_lens = context_lens;
  p.num_seqs = dims->num_seqs;
  p.num_q_heads = dims->num_q_heads;
  p.num_kv_heads = dims->num_kv_heads;
  p.block_size = dims->block_size;
  p.max_blocks_per_seq = dims->max_blocks_per_seq;
  p.num_blocks = dims->num_blocks;
  p.n_query = n_query;
  p.causal = causal;
  p.window = window;
  p.kv_dtype = kv_dtype;
  p.group = dims->num_q_heads / dims->num_kv_heads;
  p.prefix_blocks = prefix_blocks;
  p.scale_log2 = scale == 0.f ? 1e-30f : scale * 1.4426950408889634f;  // as in enqueue_decode
  p.rows_head = spl.rows_head;
  p.row_tile = spl.row_tile;
  p.rows_seq = spl.rows_seq;
  p.parts = spl.parts;
  p.rows_part = spl.rows_part;
  p.own_row0 = spl.own_row0;
  p.ctas = spl.ctas;
  p.wait_limit_ns = wait_limit_ns();
  p.part_out = reinterpret_cast<float*>(ws + w.part_out);
  p.part_lse = reinterpret_cast<float*>(ws + w.part_lse);
  p.meta = reinterpret_cast<int*>(ws + w.meta);
  p.gave_up = reinterpret_cast<int*>(ws + w.gave_up);
  p.flags = reinterpret_cast<unsigned*>(ws);
  p.out = static_cast<__half*>(out);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (launch_shared_tc(p, st) != cudaSuccess) return PA_ERR_CUDA;
  return launch_shared_join(p, st) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

int paged_attn_trace(const pa_dims* dims, const void* q, const void* k_cache,
                     const void* v_cache, const int32_t* block_table,
                     const int32_t* context_lens, int32_t n_query, int32_t causal,
                     int32_t window, float scale, int32_t kv_dtype, void* out,
                     int32_t* trace, void* stream) {
  Plan plan;
  const int rc = prepare_decode(dims, q, k_cache, v_cache, block_table, context_lens, n_query,
                                causal, window, scale, kv_dtype, out, &plan);
  if (rc != PA_OK) return rc;
  if (trace == nullptr || !aligned(trace, 4)) return PA_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const long long rows = (long long)dims->num_seqs * n_query * dims->num_q_heads;
  if (launch_trace_init(trace, rows, st) != cudaSuccess) return PA_ERR_CUDA;
  const int r = enqueue_decode(dims, plan, q, k_cache, v_cache, block_table, context_lens, n_query,
                               causal, window, scale, kv_dtype, out, dims->workspace, trace, st);
  if (r != PA_OK) return r;
  return launch_trace_finish(trace, rows, st) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

int paged_attn_merge(const float* partial_out, const float* partial_lse, int32_t num_splits,
                     int32_t rows, int32_t head_dim, void* out, float* out_lse, void* stream) {
  if (!partial_out || !partial_lse || !out) return PA_ERR_INVALID_ARG;
  if (num_splits < 1 || rows < 0) return PA_ERR_INVALID_ARG;
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) return PA_ERR_UNSUPPORTED;
  if (!aligned(partial_out, 16) || !aligned(partial_lse, 4) || !aligned(out, 8) ||
      (out_lse && !aligned(out_lse, 4)))
    return PA_ERR_INVALID_ARG;
  MergeParams m{};
  m.part_out = partial_out;
  m.part_lse = partial_lse;
  m.num_seqs = 1;
  m.num_splits = num_splits;
  m.rows_per_seq = rows;
  m.head_dim = head_dim;
  m.out = static_cast<__half*>(out);
  m.out_lse = out_lse;
  if (launch_merge(m, static_cast<cudaStream_t>(stream)) != cudaSuccess) return PA_ERR_CUDA;
  return PA_OK;
}

int paged_attn_get_error(const pa_dims* dims, void* stream) {
  if (dims == nullptr || dims->workspace == nullptr || dims->workspace_bytes < kWsHeader)
    return PA_ERR_WORKSPACE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (cudaStreamSynchronize(st) != cudaSuccess) return PA_ERR_CUDA;
  unsigned flags = 0;
  if (cudaMemcpyAsync(&flags, dims->workspace, sizeof(flags), cudaMemcpyDeviceToHost, st) !=
      cudaSuccess)
    return PA_ERR_CUDA;
  if (cudaStreamSynchronize(st) != cudaSuccess) return PA_ERR_CUDA;
  // Clear the flag; after a timeout clear the counters too (a safety net:
  // the kernels keep them consistent on that path as well).
  size_t n = sizeof(flags);
  if ((flags & kFlagTimeout) && check_dims(dims, 1) != PA_ERR_INVALID_ARG &&
      dims->workspace_bytes >= ws_zero_prefix(dims))
    n = ws_zero_prefix(dims);
  if (cudaMemsetAsync(dims->workspace, 0, n, st) != cudaSuccess) return PA_ERR_CUDA;
  if (cudaStreamSynchronize(st) != cudaSuccess) return PA_ERR_CUDA;
  if (flags & kFlagTimeout) return PA_ERR_TIMEOUT;
  if (flags & kFlagBadBlock) return PA_ERR_BAD_BLOCK_INDEX;
  if (flags & kFlagBadLen) return PA_ERR_BAD_CONTEXT_LEN;
  if (flags & kFlagBadRequest) return PA_ERR_BAD_REQUEST;
  if (flags & kFlagNoPages) return PA_ERR_NO_PAGES;
  return PA_OK;
}

uint64_t paged_attn_set_wait_limit(uint64_t nanoseconds) {
  return set_wait_limit_ns(nanoseconds);
}

int paged_attn_cache_write(const pa_dims* dims, const void* k_new, const void* v_new,
                           const int32_t* block_table, const int32_t* context_lens,
                           int32_t n_new, int32_t kv_dtype, void* k_cache, void* v_cache,
                           void* stream) {
  const int rc = check_dims(dims, n_new);
  if (rc != PA_OK && rc != PA_ERR_UNSUPPORTED) return rc;
  if (dims->head_dim != kHeadDim) return PA_ERR_UNSUPPORTED;
  if (!k_new || !v_new || !block_table || !context_lens || !k_cache || !v_cache)
    return PA_ERR_INVALID_ARG;
  if (!aligned(k_new, 8) || !aligned(v_new, 8) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
      !aligned(block_table, 4) || !aligned(context_lens, 4))
    return PA_ERR_INVALID_ARG;
  if (kv_dtype != PA_KV_FP16 && kv_dtype != PA_KV_Q8_0 && kv_dtype != PA_KV_INT8_ROW)
    return PA_ERR_INVALID_ARG;
  if (dims->workspace == nullptr || dims->workspace_bytes < kWsHeader) return PA_ERR_WORKSPACE;
  CacheWriteParams p{};
  p.k_new = static_cast<const __half*>(k_new);
  p.v_new = static_cast<const __half*>(v_new);
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.block_table = block_table;
  p.context_lens = context_lens;
  p.num_seqs = dims->num_seqs;
  p.num_kv_heads = dims->num_kv_heads;
  p.block_size = dims->block_size;
  p.max_blocks_per_seq = dims->max_blocks_per_seq;
  p.num_blocks = dims->num_blocks;
  p.n_new = n_new;
  p.kv_dtype = kv_dtype;
  p.flags = static_cast<unsigned*>(dims->workspace);
  return launch_cache_write(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? PA_OK
                                                                                 : PA_ERR_CUDA;
}

size_t paged_attn_pages_workspace_size(const pa_dims* dims) {
  if (check_dims(dims, 1) != PA_OK) return 0;
  return pages_ws(dims).total;
}

int paged_attn_pages_workspace_init(const pa_dims* dims, void* stream) {
  const int rc = check_dims(dims, 1);
  if (rc != PA_OK) return rc;
  if (dims->workspace == nullptr || !aligned(dims->workspace, 256) ||
      dims->workspace_bytes < pages_ws(dims).total)
    return PA_ERR_WORKSPACE;
  return cudaMemsetAsync(dims->workspace, 0, kWsHeader, static_cast<cudaStream_t>(stream)) ==
                 cudaSuccess
             ? PA_OK
             : PA_ERR_CUDA;
}

int paged_attn_fork(const pa_dims* dims, int32_t* block_table, int32_t* context_lens,
                    int32_t* ref_counts, const int32_t* parents, const int32_t* children,
                    int32_t n, void* stream) {
  PageParams p;
  const int rc = prepare_books(dims, block_table, context_lens, ref_counts, &p);
  if (rc != PA_OK) return rc;
  if (n < 0 || n > dims->num_seqs) return PA_ERR_INVALID_ARG;
  if (n == 0) return PA_OK;
  if (!parents || !children || !aligned(parents, 4) || !aligned(children, 4))
    return PA_ERR_INVALID_ARG;
  p.parents = parents;
  p.rows = children;
  p.n = n;
  return launch_fork(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

int paged_attn_resize(const pa_dims* dims, int32_t* block_table, int32_t* context_lens,
                      int32_t* ref_counts, const int32_t* rows, const int32_t* new_lens, int32_t n,
                      int32_t* copy_src, int32_t* copy_dst, void* stream) {
  PageParams p;
  const int rc = prepare_books(dims, block_table, context_lens, ref_counts, &p);
  if (rc != PA_OK) return rc;
  if (n < 0 || n > dims->num_seqs) return PA_ERR_INVALID_ARG;
  if (n == 0) return PA_OK;
  if (!rows || !copy_src || !copy_dst || !aligned(rows, 4) || !aligned(copy_src, 4) ||
      !aligned(copy_dst, 4) || (new_lens && !aligned(new_lens, 4)))
    return PA_ERR_INVALID_ARG;
  p.rows = rows;
  p.new_lens = new_lens;
  p.copy_src = copy_src;
  p.copy_dst = copy_dst;
  p.n = n;
  return launch_resize(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

int paged_attn_compact(const pa_dims* dims, int32_t* block_table, int32_t* context_lens,
                       int32_t* ref_counts, int32_t* copy_src, int32_t* copy_dst, int32_t* count,
                       int32_t* remap, void* stream) {
  PageParams p;
  const int rc = prepare_books(dims, block_table, context_lens, ref_counts, &p);
  if (rc != PA_OK) return rc;
  if (!copy_src || !copy_dst || !count || !remap || !aligned(copy_src, 4) ||
      !aligned(copy_dst, 4) || !aligned(count, 4) || !aligned(remap, 4))
    return PA_ERR_INVALID_ARG;
  p.copy_src = copy_src;
  p.copy_dst = copy_dst;
  p.count = count;
  p.remap = remap;
  p.n = dims->num_blocks > 1 ? dims->num_blocks / 2 : 1;
  return launch_compact(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

int paged_attn_copy_blocks(const pa_dims* dims, const int32_t* copy_src, const int32_t* copy_dst,
                           int32_t n, const int32_t* count, int32_t kv_dtype, void* k_cache,
                           void* v_cache, void* stream) {
  PageParams p;
  const int rc = prepare_pages(dims, &p);
  if (rc != PA_OK) return rc;
  if (n < 0 || n > dims->num_blocks) return PA_ERR_INVALID_ARG;
  if (kv_dtype != PA_KV_FP16 && kv_dtype != PA_KV_Q8_0 && kv_dtype != PA_KV_INT8_ROW)
    return PA_ERR_INVALID_ARG;
  if (!k_cache || !v_cache || !aligned(k_cache, 16) || !aligned(v_cache, 16))
    return PA_ERR_INVALID_ARG;
  if (n == 0) return PA_OK;
  if (!copy_src || !copy_dst || !aligned(copy_src, 4) || !aligned(copy_dst, 4) ||
      (count && !aligned(count, 4)))
    return PA_ERR_INVALID_ARG;
  const int sms = device_sm_count();
  if (sms <= 0) return PA_ERR_CUDA;
  p.copy_src = const_cast<int32_t*>(copy_src);
  p.copy_dst = const_cast<int32_t*>(copy_dst);
  p.count = const_cast<int32_t*>(count);
  p.n = n;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.page_bytes = (long long)dims->num_kv_heads *
                 (kv_dtype == PA_KV_FP16 ? (long long)dims->block_size * kHeadDim * 2
                                         : quant_tile_bytes(kv_dtype, dims->block_size));
  return launch_copy_blocks(p, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? PA_OK
                                                                                      : PA_ERR_CUDA;
}

const char* paged_attn_status_string(int32_t status) {
  switch (status) {
    case PA_OK: return "ok";
    case PA_ERR_INVALID_ARG: return "invalid argument";
    case PA_ERR_UNSUPPORTED: return "unsupported shape or type";
    case PA_ERR_WORKSPACE: return "workspace missing, misaligned or too small";
    case PA_ERR_CUDA: return "CUDA runtime error";
    case PA_ERR_BAD_BLOCK_INDEX: return "block_table entry out of range";
    case PA_ERR_BAD_CONTEXT_LEN: return "context length out of range";
    case PA_ERR_TIMEOUT: return "a device-side wait timed out; output invalid";
    case PA_ERR_BAD_REQUEST: return "page request refused (repeated, occupied or out of range)";
    case PA_ERR_NO_PAGES: return "too few free pages";
    default: return "unknown status";
  }
}

}  // extern "C"
