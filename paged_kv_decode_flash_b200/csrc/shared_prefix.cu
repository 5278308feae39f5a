// shared_prefix.cu -- decode attention for a batch whose sequences share a
// long prefix: the prefix's keys are scored once for the query rows of all
// sequences, and joined with each sequence's own keys.
//
// For a query row with the visible prefix keys A and own keys B, with
// z_j = scale q.k_j, m_X = max_X z and l_X = sum_X e^(z_j - m_X):
//   out = (e^(m_A - m) l_A O_A + e^(m_B - m) l_B O_B) /
//         (e^(m_A - m) l_A + e^(m_B - m) l_B),   m = max(m_A, m_B),
// where O_X = sum_X e^(z_j - m_X) v_j / l_X.  The prefix part comes in pieces,
// one per CTA that had some of its keys (prefix_tc.cu), the own-keys part
// (O_B, lse_B) from the segment kernel (decode_tc.cu, own-keys mode); this
// file has the work plan and the join.
#include "common.cuh"
#include "kernels.h"
#include "sm100.cuh"

namespace pa {
namespace {

using namespace sm100;

// The join: one warp per output row over the row's prefix partials and its
// own-keys partial, weights e^(lse - max).  A NaN log-sum-exp (an
// out-of-range block, a timeout) and a bad length give a row of zeros.
__global__ void __launch_bounds__(128) shared_join_kernel(const SharedParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x % 32;
  const long long rows = (long long)p.num_seqs * p.n_query * p.num_q_heads;
  const long long row = (long long)blockIdx.x * 4 + threadIdx.x / 32;
  if (row >= rows) return;
  const int s = (int)(row / ((long long)p.num_q_heads * p.n_query));
  const int P = __ldg(p.prefix_len), L = __ldg(p.context_lens + s);
  bool ok = shared_prefix_ok(p, P);
  if (!ok && row == 0 && lane == 0) atomicOr(p.flags, kFlagBadLen);
  ok = ok && shared_seq_ok(p, L, P);
  // The row's partials: slots c + g of the CTAs c that cut its group's tiles.
  const int nt = __ldcg(p.meta), Ce = __ldcg(p.meta + 1);
  const int hq = (int)(row % p.num_q_heads), kvh = hq / p.group;
  const long long rh = row / p.num_q_heads * p.group + hq % p.group;
  const int NT = (p.rows_head + p.row_tile - 1) / p.row_tile;
  const int g = kvh * NT + (int)(rh / p.row_tile);
  int c0 = 0, n = 0;
  if (nt > 0) {
    const long long W = (long long)p.num_kv_heads * NT * nt, x0 = (long long)g * nt;
    c0 = (int)(((x0 + 1) * Ce - 1) / W);
    n = (int)(((x0 + nt) * Ce - 1) / W) - c0 + 1;
  }
  const long long at = (long long)(c0 + g) * p.row_tile + rh % p.row_tile;  // + k * row_tile
  float M = -INFINITY;
  bool bad = false;
  for (int k = lane; k <= n; k += 32) {
    const float e = k < n ? __ldcg(p.part_lse + at + (long long)k * p.row_tile) : __ldcg(p.own_lse + row);
    bad |= isnan(e);
    M = fmaxf(M, e);
  }
#pragma unroll
  for (int w = 16; w > 0; w >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, w));
  bad = __any_sync(0xffffffffu, bad);
  float o[4] = {0.f, 0.f, 0.f, 0.f}, l = 0.f;
  if (ok && !bad && M != -INFINITY) {
#pragma unroll 4
    for (int k = 0; k <= n; ++k) {
      const bool own = k == n;
      const long long slot = at + (long long)k * p.row_tile;
      const float e = own ? __ldcg(p.own_lse + row) : __ldcg(p.part_lse + slot);
      const float4 v = __ldcg(reinterpret_cast<const float4*>(own ? p.own_out + row * kHeadDim
                                                                  : p.part_out + slot * kHeadDim) +
                              lane);
      if (e == -INFINITY) continue;
      const float w = expf(e - M);
      l += w;
      o[0] = fmaf(w, v.x, o[0]);
      o[1] = fmaf(w, v.y, o[1]);
      o[2] = fmaf(w, v.z, o[2]);
      o[3] = fmaf(w, v.w, o[3]);
    }
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  const __half2 a = __floats2half2_rn(o[0] * inv, o[1] * inv);
  const __half2 b = __floats2half2_rn(o[2] * inv, o[3] * inv);
  uint2 u;
  u.x = *reinterpret_cast<const uint32_t*>(&a);
  u.y = *reinterpret_cast<const uint32_t*>(&b);
  reinterpret_cast<uint2*>(p.out + row * kHeadDim)[lane] = u;
}

cudaError_t launch_pdl(void (*kern)(const SharedParams), dim3 grid, const SharedParams& p,
                       cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(128);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace

SharedPlan make_shared_plan(long long rows_head, int num_kv_heads, long long prefix_keys, int kv_dtype,
                            int sms) {
  SharedPlan pl;
  pl.rows_head = (int)rows_head;
  pl.row_tile = kv_dtype == kKvFp16 && rows_head > 128 ? 256 : 128;
  const long long groups = num_kv_heads * ((rows_head + pl.row_tile - 1) / pl.row_tile);
  const long long tiles = groups * (prefix_keys / kTileKeys + 2);
  const long long most = sms < kMaxPrefixCtas ? sms : kMaxPrefixCtas;
  pl.ctas = (int)(tiles < most ? tiles : most);
  pl.part_rows = (pl.ctas + groups) * pl.row_tile;
  return pl;
}

cudaError_t launch_shared_join(const SharedParams& p, cudaStream_t stream) {
  const long long rows = (long long)p.num_seqs * p.n_query * p.num_q_heads;
  return launch_pdl(shared_join_kernel, dim3((unsigned)((rows + 3) / 4)), p, stream);
}

}  // namespace pa
