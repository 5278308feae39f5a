// shared_prefix.cu -- decode attention for a batch whose sequences share a
// long prefix: the prefix's keys are scored once for the query rows of all
// sequences, and joined with each sequence's own keys.
//
// For a query row with the visible prefix keys A and own keys B, with
// z_j = scale q.k_j, m_X = max_X z and l_X = sum_X e^(z_j - m_X):
//   out = (e^(m_A - m) l_A O_A + e^(m_B - m) l_B O_B) /
//         (e^(m_A - m) l_A + e^(m_B - m) l_B),   m = max(m_A, m_B),
// where O_X = sum_X e^(z_j - m_X) v_j / l_X.  Both come in pieces, one per CTA
// that had some of the keys (shared_tc.cu); this file has the work plan and
// the join.
#include "common.cuh"
#include "kernels.h"
#include "sm100.cuh"

namespace pa {
namespace {

using namespace sm100;

constexpr int kJoin = 16;  // partials loaded at a time: 18 a row (32 x 4 rows behind 16384 keys), 2.5 us less than by 8

// The join: one warp per output row over the row's partials, weights
// e^(lse - max).  A NaN log-sum-exp (an out-of-range block), a partial of a CTA
// that gave up and a bad length give a row of zeros, a log-sum-exp of +inf (a
// score that is not finite) a row of NaN.
__global__ void __launch_bounds__(128) shared_join_kernel(const SharedParams p) {
  const int lane = threadIdx.x % 32;
  const long long rows = (long long)p.num_seqs * p.n_query * p.num_q_heads;
  const long long row = (long long)blockIdx.x * 4 + threadIdx.x / 32;
  const int hq = (int)(row % p.num_q_heads), kvh = hq / p.group;
  const int tok = (int)(row / p.num_q_heads), s = tok / p.n_query;
  const int rh = tok * p.group + hq % p.group;  // row of the KV head
  const int NT = (p.rows_head + p.row_tile - 1) / p.row_tile;
  const int rs = rh - s * p.rows_seq, part = rs / p.rows_part;
  const int gp = kvh * NT + rh / p.row_tile, go = s * p.num_kv_heads * p.parts + kvh * p.parts + part;
  if (row >= rows) return;
  // (complete since before the other kernel began: that waited for them, too)
  const int P = __ldg(p.prefix_len), L = __ldg(p.context_lens + s);
  griddep_wait();
  griddep_launch_dependents();
  const int nt = __ldcg(p.meta);
  const int2 cp = __ldcg(reinterpret_cast<const int2*>(p.meta) + 1 + gp);
  const int2 co = __ldcg(reinterpret_cast<const int2*>(p.meta) + 1 + p.num_kv_heads * NT + go);
  bool ok = shared_prefix_ok(p, P);
  if (!ok && row == 0 && lane == 0) atomicOr(p.flags, kFlagBadLen);
  if (ok && !shared_seq_ok(p, L, P)) {
    ok = false;
    if (lane == 0) atomicOr(p.flags, kFlagBadLen);
  }
  // The row's partials: np of the prefix, then no of its own keys.
  int np = 0, no = 0;
  bool bad = false, odd = false;
  auto count = [&](int2 c) {
    if (c.x >= 0 && c.x <= c.y && c.y < p.ctas) return c.y - c.x + 1;
    bad = true;
    return 0;
  };
  if (ok) {
    if (nt > 0) np = count(cp);
    int lo, hi;
    union_range(L, p.n_query, p.causal, p.window, lo, hi);
    if (hi >= max(lo, P)) no = count(co);
  }
  const long long at_p = (long long)(cp.x + gp) * p.row_tile + rh % p.row_tile;
  const long long at_o = p.own_row0 + (long long)(co.x + go) * p.rows_part + rs % p.rows_part;
  auto slot = [&](int k) {
    return k < np ? at_p + (long long)k * p.row_tile : at_o + (long long)(k - np) * p.rows_part;
  };
  float o[4] = {0.f, 0.f, 0.f, 0.f}, l = 0.f, M = -INFINITY;
  for (int k0 = 0; k0 < np + no; k0 += 32) {  // 32 partials at a time, lane k their lse
    const int n = min(32, np + no - k0);
    float e = -INFINITY;
    if (lane < n) {
      const int k = k0 + lane, late = __ldcg(p.gave_up + (k < np ? cp.x + k : co.x + k - np));
      e = __ldcg(p.part_lse + slot(k));
      if (late != 0) e = __uint_as_float(0x7fc00000u);  // what lies there may be another call's
    }
    float mx = 0.f, we = 0.f;
    for (int k = 0; k < n; k += kJoin) {  // the first ones are loaded beside the lse
      float4 v[kJoin];
#pragma unroll
      for (int x = 0; x < kJoin; ++x)
        v[x] = k + x < n ? __ldcg(reinterpret_cast<const float4*>(p.part_out + slot(k0 + k + x) * kHeadDim) + lane)
                         : make_float4(0.f, 0.f, 0.f, 0.f);
      if (k == 0) {
        bad |= __any_sync(0xffffffffu, isnan(e));
        odd |= __any_sync(0xffffffffu, e == INFINITY);
        mx = fmaxf(e, M);
#pragma unroll
        for (int w = 16; w > 0; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
        if (mx == -INFINITY) break;
        const float f = expf(M - mx);
        we = expf(e - mx);
        M = mx;
        l *= f;
#pragma unroll
        for (int x = 0; x < 4; ++x) o[x] *= f;
      }
#pragma unroll
      for (int x = 0; x < kJoin; ++x) {
        const float w = __shfl_sync(0xffffffffu, we, (k + x) & 31);
        if (k + x >= n || w == 0.f) continue;  // (0: a partial without keys)
        l += w;
        o[0] = fmaf(w, v[x].x, o[0]);
        o[1] = fmaf(w, v[x].y, o[1]);
        o[2] = fmaf(w, v[x].z, o[2]);
        o[3] = fmaf(w, v[x].w, o[3]);
      }
    }
  }
  const float inv = bad ? 0.f : odd ? __uint_as_float(0x7fc00000u) : l > 0.f ? 1.f / l : 0.f;
  auto end = [&](float x) { return inv != 0.f ? x * inv : 0.f; };
  const __half2 a = __floats2half2_rn(end(o[0]), end(o[1]));
  const __half2 b = __floats2half2_rn(end(o[2]), end(o[3]));
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

SharedPlan make_shared_plan(int num_seqs, int rows_seq, int num_kv_heads, int kv_dtype, int sms) {
  SharedPlan pl;
  pl.rows_head = num_seqs * rows_seq;
  // 256 rows on a K and a V tile halve the traffic to shared memory and the
  // conversions; q8_0's operands, two tiles each, leave room for 128.
  pl.row_tile = kv_dtype != kKvQ8_0 && pl.rows_head > 128 ? 256 : 128;
  pl.rows_seq = rows_seq;
  pl.parts = (rows_seq + 127) / 128;
  pl.rows_part = (rows_seq + pl.parts - 1) / pl.parts;
  pl.ctas = sms < kMaxPrefixCtas ? sms : kMaxPrefixCtas;
  const long long gp = (long long)num_kv_heads * ((pl.rows_head + pl.row_tile - 1) / pl.row_tile);
  const long long go = (long long)num_seqs * num_kv_heads * pl.parts;
  pl.own_row0 = (pl.ctas + gp) * pl.row_tile;
  pl.part_rows = pl.own_row0 + (pl.ctas + go) * pl.rows_part;
  pl.groups = gp + go;
  return pl;
}

cudaError_t launch_shared_join(const SharedParams& p, cudaStream_t stream) {
  const long long rows = (long long)p.num_seqs * p.n_query * p.num_q_heads;
  return launch_pdl(shared_join_kernel, dim3((unsigned)((rows + 3) / 4)), p, stream);
}

}  // namespace pa
