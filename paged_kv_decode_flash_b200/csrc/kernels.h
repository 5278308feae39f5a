// kernels.h -- launchers of the libpagedattn kernels (internal to the library).
#pragma once

#include <cuda_runtime.h>

#include "common.cuh"

namespace pa {

// Split-KV paged decode on the tensor cores (tcgen05/TMEM, TMA / bulk-copy
// staged KV tiles), merge included: one launch per call (per kMaxQueueSeqs
// sequences in work-queue mode).  Records the key-resolution trace when
// p.trace is set.
cudaError_t launch_decode_tc(const DecodeParams& p, cudaStream_t stream);
// Most query rows one CTA handles per KV head for a cache type.
int max_rows_per_part(int kv_dtype);

// The per-head split kernel (decode_split.cu): fp16 cache, few (sequence,
// KV head) groups, up to 8 query tokens and 32 rows per KV head, every key
// of the context.  Each group's 128-key tiles are cut into contiguous runs
// over its share of `ctas` CTAs; partial slots are CTA-indexed (rows
// [cta * rows, cta * rows + rows)); merge included; records the trace when
// p.trace is set.  Only p's fields of a mode-0 plan are read.
bool split_decode_supported(int kv_dtype, int n_query, int rows, int num_blocks,
                            int num_kv_heads, int block_size);
cudaError_t launch_split_decode(const DecodeParams& p, int ctas, cudaStream_t stream);

// Log-sum-exp merge of split partials into fp16 rows.
cudaError_t launch_merge(const MergeParams& p, cudaStream_t stream);

// Key-resolution record: set every row to {0, INT32_MAX, -1, 0, 0} before
// a traced decode, and rows no key reached to {0, -1, -1, 0, 0} after it.
cudaError_t launch_trace_init(int32_t* trace, long long rows, cudaStream_t stream);
cudaError_t launch_trace_finish(int32_t* trace, long long rows, cudaStream_t stream);

// Quantise new keys/values and write them into the paged cache.
struct CacheWriteParams {
  const __half* k_new;         // [B][n_new][Hkv][D]
  const __half* v_new;
  void* k_cache;
  void* v_cache;
  const int32_t* block_table;  // [B][mbps]
  const int32_t* context_lens; // [B]: the new tokens are the last n_new positions
  int num_seqs, num_kv_heads, block_size, max_blocks_per_seq, num_blocks, n_new, kv_dtype;
  unsigned* flags;             // data-error flags (a workspace status word)
};
cudaError_t launch_cache_write(const CacheWriteParams& p, cudaStream_t stream);

// Shared-prefix decode: partials of the prefix's and of the sequences' own keys
// (shared_tc.cu) and their join (shared_prefix.cu).
constexpr int kMaxPrefixCtas = 160;  // bound of the grid, whatever the device
struct SharedPlan {
  int rows_head;        // query rows of a KV head: sequences x tokens x group
  int row_tile;         // prefix: rows of a group, 128 or 256
  int rows_seq;         // rows of a sequence on a KV head: tokens x group
  int parts, rows_part; // own keys: these in `parts` groups of at most 128
  int ctas;
  long long own_row0;   // first row of the own-keys partials
  long long part_rows;  // rows of part_out
  long long groups;     // prefix and own groups
};
struct SharedParams {
  const __half* q;              // [B][nq][Hq][D]
  const void* k;                // cache, see pagedattn.h
  const void* v;
  const int32_t* prefix_table;  // [prefix_blocks]
  const int32_t* prefix_len;    // [1]
  const int32_t* block_table;   // [B][mbps]
  const int32_t* context_lens;  // [B]
  int num_seqs, num_q_heads, num_kv_heads, block_size, max_blocks_per_seq;
  int num_blocks, n_query, causal, window, kv_dtype, group, prefix_blocks;
  float scale_log2;             // scale * log2(e)
  int rows_head, row_tile, rows_seq, parts, rows_part, ctas;  // SharedPlan
  long long own_row0;
  unsigned long long wait_limit_ns;
  float* part_out;              // partials [slots][row_tile][D], [own slots][rows_part][D]
  float* part_lse;              // natural log
  int* meta;                    // key tiles of the prefix, -; first and last CTA of every group
  int* gave_up;                 // [ctas] a CTA's waits ran out: its partials are not used
  unsigned* flags;              // workspace status word
  __half* out;                  // [B][nq][Hq][D]
};
// The shared prefix is whole blocks inside the caller's table.
__host__ __device__ __forceinline__ bool shared_prefix_ok(const SharedParams& p, int P) {
  return P >= 0 && P % p.block_size == 0 && P / p.block_size <= p.prefix_blocks;
}
__host__ __device__ __forceinline__ bool shared_seq_ok(const SharedParams& p, int L, int P) {
  return context_len_ok(L, p.n_query, p.max_blocks_per_seq, p.block_size) && P <= L;
}
SharedPlan make_shared_plan(int num_seqs, int rows_seq, int num_kv_heads, int kv_dtype, int sms);
cudaError_t launch_shared_tc(const SharedParams& p, cudaStream_t stream);
cudaError_t launch_shared_join(const SharedParams& p, cudaStream_t stream);

// Page operations (pages.cu).
struct PageParams {
  int32_t* block_table;   // [num_seqs][max_blocks_per_seq]
  int32_t* context_lens;  // [num_seqs]
  int32_t* ref_counts;    // [num_blocks]: table rows that hold a page (0: free)
  const int32_t* rows;    // requests: the row (fork: the child)
  const int32_t* parents; // fork
  const int32_t* new_lens;// resize; null: 0
  int32_t* copy_src;      // copies asked for (copy: to make), -1: none
  int32_t* copy_dst;
  int32_t* count;         // compact: moves made; copy: pairs of the list, or null
  int32_t* remap;         // compact: where every page went
  void* k_cache;
  void* v_cache;
  long long page_bytes;   // of one cache
  int num_seqs, max_blocks_per_seq, block_size, num_blocks, n;
  int tables_too;         // compact: the planning kernel rewrites the tables
  unsigned* flags;        // workspace status word
  int* row_scratch;       // [3][num_seqs]
  int* page_scratch;      // [3][num_blocks]
  int* small_scratch;     // [64]
};
cudaError_t launch_fork(const PageParams& p, cudaStream_t stream);
cudaError_t launch_resize(const PageParams& p, cudaStream_t stream);
cudaError_t launch_compact(const PageParams& p, cudaStream_t stream);
cudaError_t launch_copy_blocks(const PageParams& p, int sms, cudaStream_t stream);

}  // namespace pa
