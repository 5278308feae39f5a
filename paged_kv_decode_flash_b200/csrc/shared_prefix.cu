// shared_prefix.cu -- decode attention for a batch whose sequences share a
// long prefix: the prefix's keys are scored once for the query rows of all
// sequences, and joined with each sequence's own keys.
//
// For a query row with the visible prefix keys A and own keys B, with
// z_j = scale q.k_j, m_X = max_X z and l_X = sum_X e^(z_j - m_X):
//   out = (e^(m_A - m) l_A O_A + e^(m_B - m) l_B O_B) /
//         (e^(m_A - m) l_A + e^(m_B - m) l_B),   m = max(m_A, m_B),
// where O_X = sum_X e^(z_j - m_X) v_j / l_X.  The own-keys part (O_B, lse_B)
// comes from the segment kernel (decode_tc.cu, own-keys mode); this file has
// the prefix part and the join.
//
// Prefix part: one warp per (query row, split of the prefix's keys); a lane
// holds four head_dim elements; one pass with a running maximum and sum.
#include "common.cuh"
#include "kernels.h"
#include "sm100.cuh"

namespace pa {
namespace {

using namespace sm100;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.69314718055994531f;
constexpr unsigned kInvalidLse = 0x7fc00000u;  // NaN: a partial that must not be used

// The shared prefix is whole blocks inside the caller's table.
__device__ __forceinline__ bool prefix_ok(const SharedParams& p, int P) {
  return P >= 0 && P % p.block_size == 0 && P / p.block_size <= p.prefix_blocks;
}
__device__ __forceinline__ bool seq_ok(const SharedParams& p, int L, int P) {
  return context_len_ok(L, p.n_query, p.max_blocks_per_seq, p.block_size) && P <= L;
}

// Four elements (4 lane .. 4 lane + 3) of one cache row.
__device__ __forceinline__ void load_row4(const SharedParams& p, const void* cache, long long phys,
                                          int kvh, int slot, int lane, float (&x)[4]) {
  if (p.kv_dtype == kKvFp16) {
    const long long row = (phys * p.num_kv_heads + kvh) * p.block_size + slot;
    const uint2 u = __ldg(
        reinterpret_cast<const uint2*>(static_cast<const __half*>(cache) + row * kHeadDim) + lane);
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&u.x));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&u.y));
    x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
    return;
  }
  const uint8_t* tile = static_cast<const uint8_t*>(cache) +
                        (phys * p.num_kv_heads + kvh) * quant_tile_bytes(p.kv_dtype, p.block_size);
  const uint8_t* sc = tile + (long long)p.block_size * kHeadDim;
  const char4 c = __ldg(reinterpret_cast<const char4*>(tile + (long long)slot * kHeadDim) + lane);
  const float d = p.kv_dtype == kKvQ8_0
                      ? __half2float(__ldg(reinterpret_cast<const __half*>(sc + slot * 8) + lane / 8))
                      : __ldg(reinterpret_cast<const float*>(sc) + slot);
  x[0] = c.x * d; x[1] = c.y * d; x[2] = c.z * d; x[3] = c.w * d;
}

// grid (rows / 4, splits), 4 warps; row = output row (s, i, query head).
__global__ void __launch_bounds__(128) prefix_rows_kernel(const SharedParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x % 32;
  const long long rows = (long long)p.num_seqs * p.n_query * p.num_q_heads;
  const long long row = (long long)blockIdx.x * 4 + threadIdx.x / 32;
  if (row >= rows) return;
  const int hq = (int)(row % p.num_q_heads), kvh = hq / p.group;
  const int i = (int)(row / p.num_q_heads % p.n_query);
  const int s = (int)(row / ((long long)p.num_q_heads * p.n_query));
  const int P = __ldg(p.prefix_len), L = __ldg(p.context_lens + s);
  float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  bool bad = false;
  if (prefix_ok(p, P) && seq_ok(p, L, P)) {
    int lo, hi;
    key_range(L, p.n_query, i, p.causal, p.window, lo, hi);
    const int per = (P + p.splits - 1) / p.splits;
    lo = max(lo, (int)blockIdx.y * per);
    hi = min(min(hi, P - 1), (int)(blockIdx.y + 1) * per - 1);
    float q[4];
    const uint2 u = __ldg(reinterpret_cast<const uint2*>(p.q + row * kHeadDim) + lane);
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&u.x));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&u.y));
    q[0] = a.x; q[1] = a.y; q[2] = b.x; q[3] = b.y;
    for (int j = lo; j <= hi; ++j) {
      const int phys = __ldg(p.prefix_table + j / p.block_size);
      if (phys < 0 || phys >= p.num_blocks) {
        bad = true;
        continue;
      }
      float k[4], v[4];
      load_row4(p, p.k, phys, kvh, j % p.block_size, lane, k);
      load_row4(p, p.v, phys, kvh, j % p.block_size, lane, v);
      float z = q[0] * k[0] + q[1] * k[1] + q[2] * k[2] + q[3] * k[3];
#pragma unroll
      for (int w = 16; w > 0; w >>= 1) z += __shfl_xor_sync(0xffffffffu, z, w);
      z *= p.scale_log2;
      const float mn = fmaxf(m, z);
      const float f = m == -INFINITY ? 0.f : exp2f(m - mn), e = exp2f(z - mn);
      m = mn;
      l = l * f + e;
#pragma unroll
      for (int x = 0; x < 4; ++x) o[x] = o[x] * f + e * v[x];
    }
  }
  if (bad && lane == 0) atomicOr(p.flags, kFlagBadBlock);
  const long long at = (long long)blockIdx.y * rows + row;
  const float inv = l > 0.f ? 1.f / l : 0.f;
  reinterpret_cast<float4*>(p.part_out + at * kHeadDim)[lane] =
      make_float4(o[0] * inv, o[1] * inv, o[2] * inv, o[3] * inv);
  if (lane == 0)
    p.part_lse[at] = bad       ? __uint_as_float(kInvalidLse)
                     : l > 0.f ? m * kLn2 + logf(l)
                               : -INFINITY;
}

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
  bool ok = prefix_ok(p, P);
  if (!ok && row == 0 && lane == 0) atomicOr(p.flags, kFlagBadLen);
  ok = ok && seq_ok(p, L, P);
  float M = -INFINITY;
  bool bad = false;
  for (int k = lane; k <= p.splits; k += 32) {
    const float e = k < p.splits ? __ldcg(p.part_lse + k * rows + row) : __ldcg(p.own_lse + row);
    bad |= isnan(e);
    M = fmaxf(M, e);
  }
#pragma unroll
  for (int w = 16; w > 0; w >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, w));
  bad = __any_sync(0xffffffffu, bad);
  float o[4] = {0.f, 0.f, 0.f, 0.f}, l = 0.f;
  if (ok && !bad && M != -INFINITY) {
    for (int k = 0; k <= p.splits; ++k) {
      const bool own = k == p.splits;
      const float e = own ? __ldcg(p.own_lse + row) : __ldcg(p.part_lse + k * rows + row);
      if (e == -INFINITY) continue;
      const float w = expf(e - M);
      const float4 v = __ldcg(reinterpret_cast<const float4*>(
                                  own ? p.own_out + row * kHeadDim
                                      : p.part_out + (k * rows + row) * kHeadDim) +
                              lane);
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

SharedPlan make_shared_plan(long long rows, long long prefix_keys) {
  SharedPlan pl;
  pl.splits = (int)(prefix_keys < 64 * 16 ? (prefix_keys + 63) / 64 : 16);
  pl.part_rows = rows * pl.splits;
  return pl;
}

cudaError_t launch_prefix(const SharedParams& p, cudaStream_t stream) {
  const long long rows = (long long)p.num_seqs * p.n_query * p.num_q_heads;
  return launch_pdl(prefix_rows_kernel, dim3((unsigned)((rows + 3) / 4), p.splits), p, stream);
}

cudaError_t launch_shared_join(const SharedParams& p, cudaStream_t stream) {
  const long long rows = (long long)p.num_seqs * p.n_query * p.num_q_heads;
  return launch_pdl(shared_join_kernel, dim3((unsigned)((rows + 3) / 4)), p, stream);
}

}  // namespace pa
