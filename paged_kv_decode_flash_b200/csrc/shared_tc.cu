// shared_tc.cu -- the shared-prefix decode on the sm_100a tensor cores: every
// query row of the batch against the keys that all sequences share, and every
// sequence's rows against its own keys, in one launch.
//
// Mathematics: for a row with scores z_j (log2 units), weights
// 2^(z_j - m + 2) with a reference m that follows the running maximum
// lazily; l = sum of the weights, O = sum of weight * v, one pass over the
// keys; the partial is O / l with lse = (m - 2 + log2 l) ln 2.
//
// Work.  Prefix: the rows of a KV head (sequences x new tokens x the head's
// query heads) are cut into row tiles, 256 rows (fp16) or 128; a (KV head,
// row tile) is a group.  Own keys: a (sequence, KV head, part of at most 128
// of the sequence's rows) is a group.  A group's visible keys are numbered in
// tiles of 128.  The tiles of all groups, prefix first, are laid end to end
// (WorkCut below) and cut into equal ranges over the CTAs (one per SM); a
// CTA's run of tiles of one group is a segment and makes one partial per row.
//
// A CTA has two streams, each a softmax warpgroup (thread = query row), an
// S / P buffer and an O accumulator of 128 x 128 in TMEM, so that the tensor
// cores work for one stream while the other's softmax runs:
//   dual segment (more than 128 rows): stream w has rows 128 w .. and every
//           key tile (a K and a V tile in shared memory serve 256 rows);
//   single: both streams have the same rows, stream w every other key tile;
//           their sums are joined at the segment's end.
// S = Q K^T (M = 128 rows, N = 128 keys), P overwrites S in TMEM as fp16
// high parts and residuals (the weights to 2^-22, as in the other decode
// kernels), and O += [P_hi | P_lo] V takes P from TMEM and V as it lies in
// the cache.
//
// The int8 caches are converted on the way in, to operands that lose nothing
// that matters:
//   q8_0: a value qs * d has at most 19 significant bits and enters as fp16
//         high part and residual, K and V alike: S = Q K_hi + Q K_lo,
//         O += P_hi V_hi + P_lo V_hi + P_hi V_lo (2^-22);
//   int8 rows: qs enters as it is.  K's row scale multiplies the scores, V's
//         the weights before their split, so that both cost no MMA; the
//         row's reference covers the largest |V scale| of a tile, too.
// They run single segments only: 128 rows leave shared memory for the
// converted tiles.
//
// Roles: warps 0-3 and 4-7 the softmax warpgroups, which also stage Q and
// write the partials.  fp16: warp 8 K producer, warp 9 V producer (TMA boxes
// of 16 keys through the block table), warp 10 MMA issuer.  int8: warps 8-11
// converters (raw bytes through registers, one tile ahead), warp 12 MMA
// issuer.  The next warp cuts the CTA's range into segments.
//
// Every wait is bounded (SharedParams::wait_limit_ns): on a timeout the
// kernel raises kFlagTimeout, drains its copies and MMAs with a fixed bound,
// frees TMEM and marks its partials (NaN lse; the join writes zeros).
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <atomic>

#include "common.cuh"
#include "kernels.h"
#include "sm100.cuh"

namespace pa {
namespace {

using namespace sm100;

// A K, V or Q tile in shared memory: [row / 8][half][row % 8][64 fp16] with
// the 128-byte swizzle (1 KB atoms); a 16-key chunk is one TMA box.
constexpr uint32_t kAtomBytes = 1024;
constexpr uint32_t kGroupBytes = 2 * kAtomBytes;
constexpr uint32_t kTileBytes = kTileKeys / 8 * kGroupBytes;  // 32 KB
constexpr uint32_t kChunkBytes = kChunk * 256;
// Weights are scaled by 2^kShift and stay below 2^(kShift + kLazy) < 65504.
// A large kLazy makes rescaling rare; what it costs are weights 2^-25 below
// the reference's, which fp16's range cuts off.
constexpr float kShift = 2.f;
constexpr float kLazy = 13.f;
constexpr float kLn2 = 0.69314718055994531f;
constexpr unsigned kInvalidLse = 0x7fc00000u;  // NaN: a partial that must not be used
constexpr int kInfoSlots = 16;
constexpr int kOwnStart = 1;    // what the start of an own-keys segment costs, in units
constexpr int kScaleSlots = 8;  // tiles whose row scales are kept: more than are in flight

constexpr int kSegSlots = 4;

enum : int {
  BAR_KFULL = 0,   // [3]
  BAR_KEMPTY = 3,  // [3]
  BAR_VFULL = 6,   // [3]
  BAR_VEMPTY = 9,  // [3]
  BAR_SFULL = 12,  // [2] S of a stream's unit in TMEM
  BAR_PFULL = 14,  // [2] P of a stream's unit in TMEM
  BAR_QFULL = 16,  // a segment's Q staged, the previous one's O read
  BAR_SEG = 17,    // every MMA of a segment finished
  BAR_DONE = 18,
  BAR_GFULL = 19,  // [kSegSlots] a segment's description published
  BAR_GEMPTY = 23, // [kSegSlots] ... read by every role
  BAR_COUNT = 27
};

template <int KV>
struct Cfg {
  static constexpr bool kQuant = KV != kKvFp16;
  static constexpr bool kQ8 = KV == kKvQ8_0, kRow = KV == kKvInt8Row;
  static constexpr int kProdWarp = 8;                      // fp16: K, V producer; int8: converters
  static constexpr int kMmaWarp = kQuant ? 12 : 10;
  static constexpr int kReaders = kMmaWarp + 1;            // warps that follow the segments
  static constexpr int kThreads = kQuant ? 448 : 384;
  static constexpr uint32_t kSlot = (kQ8 ? 2 : 1) * kTileBytes;  // q8_0: the high tile, the residual
  static constexpr int KS = kQ8 ? 1 : kRow ? 2 : 3;
  static constexpr int VS = kRow ? 3 : 2;
  static constexpr uint32_t kQ = 0;
  static constexpr uint32_t kK = kQ + (kQuant ? 1 : 2) * kTileBytes;
  static constexpr uint32_t kV = kK + KS * kSlot;
  static constexpr uint32_t kBars = kV + VS * kSlot;
  static constexpr uint32_t kInfo = kBars + BAR_COUNT * 8 + 8;      // uint32 [kInfoSlots]
  static constexpr uint32_t kMisc = kInfo + kInfoSlots * 4;         // int [16], see below
  static constexpr uint32_t kSegs = kMisc + 64;             // Segment [kSegSlots]
  static constexpr uint32_t kScales = kSegs + kSegSlots * 64;  // int8 rows: float K [8][128], V [8][128], max [8][4]
  static constexpr uint32_t kTotal = kScales + (kRow ? kScaleSlots * (2 * 128 + 4) * 4 : 0);
  static_assert(kBars % 16 == 0 && kSegs % 16 == 0 && kScales % 16 == 0, "alignment");
  static_assert(kTotal + 1024 <= 232448, "shared memory per CTA");
};

__device__ __forceinline__ uint32_t h2_bits(__half2 h) { return *reinterpret_cast<const uint32_t*>(&h); }
__device__ __forceinline__ void sts_v4(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}

// Four signed bytes -> four exact fp16 values: byte b becomes the low mantissa
// byte of the fp16 1024 + (b + 128), minus 1152.
__device__ __forceinline__ void q8_to_half4(uint32_t q, __half2& lo, __half2& hi) {
  const uint32_t w = q ^ 0x80808080u;
  const uint32_t a = __byte_perm(w, 0x64646464u, 0x5140), b = __byte_perm(w, 0x64646464u, 0x7362);
  const __half2 off = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));  // 1152
  lo = __hsub2(*reinterpret_cast<const __half2*>(&a), off);
  hi = __hsub2(*reinterpret_cast<const __half2*>(&b), off);
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z, w;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
      "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, w;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "add.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, w;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mul.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// Tiles of a set of keys [lo, hi]: from `base` (lo rounded down to a chunk).
__device__ __forceinline__ int key_tiles(int lo, int hi) {
  return hi >= lo ? (hi - lo / kChunk * kChunk) / kTileKeys + 1 : 0;
}

// A run of key tiles of one group.
struct Segment {
  const int32_t* table;   // blocks of the keys
  long long out_row;      // of part_out / part_lse
  int kvh, row0, nrows;   // rows [row0, row0 + nrows) of the KV head's rows_head
  int lo, hi, base;       // keys that some row sees; key of the group's first tile
  int t0, n;              // tiles (n = 0: the end)
  int clo, chi;           // bounds of the keys: prefix or own
  int group, flags;       // kDual, kFirst, kLast
};
static_assert(sizeof(Segment) == 64, "Segment layout");
enum : int { kDual = 1, kFirst = 2, kLast = 4 };  // more than 128 rows; of the group's segments

template <int KV>
__global__ void __launch_bounds__(Cfg<KV>::kThreads, 1)
    shared_tc_kernel(const __grid_constant__ CUtensorMap tmap_k,
                     const __grid_constant__ CUtensorMap tmap_v, const SharedParams p) {
  using C = Cfg<KV>;
  constexpr bool kQuant = C::kQuant, kQ8 = C::kQ8, kRow = C::kRow;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  const uint32_t sQ = sbase + C::kQ, sK = sbase + C::kK, sV = sbase + C::kV;
  uint32_t* info = reinterpret_cast<uint32_t*>(smem + C::kInfo);
  // [0] TMEM base, [1] abort, [2] shortest sequence, [3] start sequence,
  // [4, 5] its start, [6, 7] own units of the batch, [8] segments given up
  int* misc = reinterpret_cast<int*>(smem + C::kMisc);
  volatile int* abort = misc + 1;
  const unsigned long long wl = p.wait_limit_ns;
  auto bar = [&](int i) { return sbase + C::kBars + 8u * i; };
  auto wait = [&](int b, int parity) { return mbar_wait(bar(b), (uint32_t)parity & 1u, abort, wl); };
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const float cs = fabsf(p.scale_log2);

  if (threadIdx.x == 0) {
    for (int i = 0; i < BAR_COUNT; ++i)
      mbar_init(bar(i), i == BAR_QFULL                                                   ? 8
                        : (i == BAR_PFULL || i == BAR_PFULL + 1)                         ? 4
                        : (kQuant && (i < BAR_KEMPTY || (i >= BAR_VFULL && i < BAR_VEMPTY))) ? 4
                        : i >= BAR_GEMPTY                                                ? C::kReaders
                                                                                         : 1);
    misc[1] = 0;
    misc[2] = INT32_MAX;
    misc[8] = 0;
    misc[3] = p.num_seqs;
    *reinterpret_cast<unsigned long long*>(misc + 6) = 0;
    fence_mbar_init();
  }
  if (warp == C::kMmaWarp) tmem_alloc(smem_u32(misc), 512);
  if constexpr (!kQuant) {
    if (threadIdx.x == 256) {
      prefetch_tmap(&tmap_k);
      prefetch_tmap(&tmap_v);
    }
  }
  griddep_wait();
  griddep_launch_dependents();
  const int P = __ldg(p.prefix_len);
  const bool prefix_ok = shared_prefix_ok(p, P);
  __syncthreads();

  // ---- the work cut ---------------------------------------------------------
  // A unit is the product of 128 rows and 128 keys.  Prefix groups: tiles of
  // one or two (dual) units; own groups: kOwnStart units for the start of a
  // segment, then tiles of one.  CTA c has the tiles that begin in units
  // [c W / Ce, (c + 1) W / Ce).
  auto own_keys = [&](int L, int& lo, int& hi) {  // of all of a sequence's rows
    lo = 0;
    hi = -1;
    if (prefix_ok && shared_seq_ok(p, L, P)) {
      union_range(L, p.n_query, p.causal, p.window, lo, hi);
      lo = max(lo, P);
    }
  };
  const int hp = p.num_kv_heads * p.parts;  // own groups of a sequence
  auto own_units = [&](int L) -> long long {
    int lo, hi;
    own_keys(L, lo, hi);
    const int t = key_tiles(lo, hi);
    return t > 0 ? (long long)hp * (t + kOwnStart) : 0;
  };
  {
    int m = INT32_MAX;
    long long u = 0;
    for (int s = threadIdx.x; s < p.num_seqs; s += C::kThreads) {
      const int L = __ldg(p.context_lens + s);
      if (prefix_ok && shared_seq_ok(p, L, P)) m = min(m, L);
      u += own_units(L);
    }
    m = __reduce_min_sync(0xffffffffu, m);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) u += __shfl_xor_sync(0xffffffffu, u, o);
    if (lane == 0 && m != INT32_MAX) {
      atomicMin(misc + 2, m);
      atomicAdd(reinterpret_cast<unsigned long long*>(misc + 6), (unsigned long long)u);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc[0];
  int vlo = 0, vhi = -1;  // the prefix's visible keys: from the shortest sequence's first on
  if (misc[2] != INT32_MAX) {
    int hi;
    key_range(misc[2], p.n_query, 0, p.causal, p.window, vlo, hi);
    vhi = P - 1;
  }
  const int nt = key_tiles(vlo, vhi), R = p.rows_head;
  const int u1 = p.row_tile / 128;                          // units of a full row tile's key tile
  const int uh = (R + 127) / 128;                           // ... of all row tiles of a head
  const int NT = (R + p.row_tile - 1) / p.row_tile;
  const long long Wp = (long long)p.num_kv_heads * uh * nt;
  const long long W = Wp + *reinterpret_cast<long long*>(misc + 6);
  // a range holds the beginning of a tile at least: no CTA between two
  // segments of a group is without one
  const int Ce = (int)min(W / u1 > 1 ? W / u1 : 1, (long long)p.ctas);
  const int cta = blockIdx.x;
  long long a = 0, b = 0;
  if (cta < Ce) {
    a = cta * W / Ce;
    b = (cta + 1) * W / Ce;
  }
  if (cta == 0 && threadIdx.x == 0) p.meta[0] = nt;  // for the join
  if (a > Wp) {  // the sequence in which this CTA's range begins (as b > a, the whole CTA is here)
    long long run = Wp;
    long long* sums = reinterpret_cast<long long*>(smem + C::kK);  // [warps], no copy is in flight yet
    for (int s0 = 0; s0 < p.num_seqs && run <= a; s0 += C::kThreads) {
      const int s = s0 + threadIdx.x;
      const long long u = s < p.num_seqs ? own_units(__ldg(p.context_lens + s)) : 0;
      long long x = u;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (lane == 31) sums[warp] = x;
      __syncthreads();
      long long before = run, total = 0;
      for (int w = 0; w < C::kThreads / 32; ++w) {
        if (w < warp) before += sums[w];
        total += sums[w];
      }
      const long long at = before + x - u;
      if (at <= a && a < at + u) {
        misc[3] = s;
        *reinterpret_cast<long long*>(misc + 4) = at;
      }
      run += total;
      __syncthreads();
    }
    fence_proxy_async_smem();
  } else if (threadIdx.x == 0) {
    misc[3] = 0;
    *reinterpret_cast<long long*>(misc + 4) = Wp;
  }
  __syncthreads();

  Segment* segs = reinterpret_cast<Segment*>(smem + C::kSegs);
  // These waits do not end with *abort: after a timeout the roles still pass
  // every segment, so that each partial is marked.
  auto seg_wait = [&](int b, int parity) { return mbar_wait(bar(b), (uint32_t)parity & 1u, misc + 8); };
  // Calls f(segment) for every segment of this CTA.
  auto segments = [&](auto&& f) {
    for (int i = 0;; ++i) {
      if (!__all_sync(0xffffffffu, seg_wait(BAR_GFULL + i % kSegSlots, i / kSegSlots))) break;
      const Segment& g = segs[i % kSegSlots];
      if (g.n == 0) break;
      f(g);
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(BAR_GEMPTY + i % kSegSlots));
    }
  };

  if constexpr (kQuant) {
    if (warp >= C::kProdWarp && warp < C::kMmaWarp) {
      // ===================== int8 converters ================================
      // A warp takes 32 keys of every tile, eight lanes a key: coalesced loads
      // into registers one tile ahead, then the operand layout.
      const int cw = warp % 4, kq = lane / 8, cl = lane % 8;
      const long long tile_bytes = quant_tile_bytes(KV, p.block_size);
      struct Raw {  // 32 keys of K or V
        uint4 q[8];
        uint16_t d8[kQ8 ? 8 : 1];  // q8_0: the scale of this lane's 16 values
        float d1;                  // int8 rows: the scale of key `lane`
      };
      int T = 0;
      bool ok = true;
      segments([&](const Segment& g) {
        const int base = g.base, t0 = g.t0, te = g.t0 + g.n, vlo = g.lo, vhi = g.hi;
        const int32_t* table = g.table;
        // The block of this warp's two chunks of tile t (lanes 0, 1).
        auto lookup = [&](int t) -> int {
          const int key0 = base + t * kTileKeys + (2 * cw + lane) * kChunk;
          return lane < 2 && t < te && key0 <= vhi ? __ldg(table + key0 / p.block_size) : 0;
        };
        auto fetch = [&](const void* cache, int t, int phys, Raw& x) {
          x.d1 = 0.f;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int key0 = base + t * kTileKeys + (2 * cw + h) * kChunk;
            const long long ph = __shfl_sync(0xffffffffu, phys, h);
            const bool on = t < te && key0 <= vhi;
            const uint8_t* tile =
                static_cast<const uint8_t*>(cache) + (ph * p.num_kv_heads + g.kvh) * tile_bytes;
            const int slot = key0 % p.block_size;
#pragma unroll
            for (int i = 4 * h; i < 4 * h + 4; ++i) {
              const int k = slot + (4 * i) % kChunk + kq;
              x.q[i] = make_uint4(0, 0, 0, 0);
              if constexpr (kQ8) x.d8[i] = 0;
              if (on) {
                x.q[i] = __ldg(reinterpret_cast<const uint4*>(tile + k * kHeadDim) + cl);
                if constexpr (kQ8)
                  x.d8[i] = __ldg(reinterpret_cast<const unsigned short*>(
                                      tile + p.block_size * kHeadDim + k * 8) + cl / 2);
              }
            }
            if constexpr (kRow) {
              if (on && lane / kChunk == h)
                x.d1 = __ldg(reinterpret_cast<const float*>(tile + p.block_size * kHeadDim) + slot +
                             lane % kChunk);
            }
          }
        };
        // Writes the operand tile at `slot`; keys outside [klo, vhi] get scale 0.
        auto convert = [&](const Raw& x, uint32_t slot, int kw, int klo) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int r = 32 * cw + 4 * i + kq;
            const uint32_t dst = slot + (r / 8) * kGroupBytes + (r % 8) * 128 + (cl / 4) * kAtomBytes;
            __half2 y[8];
            const uint32_t wd[4] = {x.q[i].x, x.q[i].y, x.q[i].z, x.q[i].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) q8_to_half4(wd[e], y[2 * e], y[2 * e + 1]);
            // Lanes 4-7 of a key write their second half first: the eight
            // lanes of a store then cover all banks.
            const int sw = cl >= 4;
            const uint32_t a0 = dst + (((2 * cl + sw) % 8) ^ (r % 8)) * 16;
            const uint32_t a1 = dst + (((2 * cl + 1 - sw) % 8) ^ (r % 8)) * 16;
            auto put = [&](const __half2 (&h)[8], uint32_t off) {
              const uint4 u0 = make_uint4(h2_bits(h[0]), h2_bits(h[1]), h2_bits(h[2]), h2_bits(h[3]));
              const uint4 u1 = make_uint4(h2_bits(h[4]), h2_bits(h[5]), h2_bits(h[6]), h2_bits(h[7]));
              sts_v4(a0 + off, sw ? u1 : u0);
              sts_v4(a1 + off, sw ? u0 : u1);
            };
            if constexpr (kQ8) {
              __half d = __ushort_as_half(x.d8[i]);
              const int key = kw + 4 * i + kq;
              if (key < klo || key > vhi) d = __ushort_as_half(0);
              const __half2 d2 = __halves2half2(d, d);
              __half2 hi8[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                hi8[e] = __hmul2(y[e], d2);
                y[e] = __hfma2(y[e], d2, __hneg2(hi8[e]));  // the residual, exact above 2^-24
              }
              put(hi8, 0);
              put(y, kTileBytes);
            } else {
              put(y, 0);
            }
          }
        };
        float* scales = reinterpret_cast<float*>(smem + C::kScales);  // K [8][128], V, max [8][4]
        Raw k, v;
        int phys = 0;
        uint32_t bad = 0, bad_next = 0;  // out-of-range blocks of this warp's chunks
        auto next = [&](int t) {         // tile t's blocks
          phys = lookup(t);
          const bool b = phys < 0 || phys >= p.num_blocks;
          bad_next = __ballot_sync(0xffffffffu, b);
          if (b) phys = 0;  // a stand-in: the rows that see it are marked
        };
        next(t0);
        bad = bad_next;
        fetch(p.k, t0, phys, k);
        fetch(p.v, t0, phys, v);
        next(t0 + 1);
        for (int t = t0; t < te; ++t, ++T) {
          const int kw = base + t * kTileKeys + 32 * cw;
          const int sk = T % C::KS, sv = T % C::VS, ss = T % kScaleSlots;
          ok = ok && __all_sync(0xffffffffu, wait(BAR_KEMPTY + sk, (T / C::KS) ^ 1));
          if (!ok) break;
          if (lane == 0) {
            reinterpret_cast<uint8_t*>(info + T % kInfoSlots)[cw] = (uint8_t)bad;
            if (bad) atomicOr(p.flags, kFlagBadBlock);
          }
          if constexpr (kRow) scales[ss * 128 + 32 * cw + lane] = k.d1 * cs;
          convert(k, sK + sk * C::kSlot, kw, 0);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(BAR_KFULL + sk));
          fetch(p.k, t + 1, phys, k);
          ok = __all_sync(0xffffffffu, wait(BAR_VEMPTY + sv, (T / C::VS) ^ 1));
          if (!ok) break;
          if constexpr (kRow) {  // scales of hidden keys may be anything
            const float d = kw + lane >= vlo && kw + lane <= vhi ? v.d1 : 0.f;
            float mx = fabsf(d);
            scales[(kScaleSlots + ss) * 128 + 32 * cw + lane] = d;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            if (lane == 0) scales[2 * kScaleSlots * 128 + ss * 4 + cw] = mx;
          }
          convert(v, sV + sv * C::kSlot, kw, vlo);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(BAR_VFULL + sv));
          fetch(p.v, t + 1, phys, v);
          bad = bad_next;
          next(t + 2);
        }
      });
    }
  } else if (warp == C::kProdWarp || warp == C::kProdWarp + 1) {
    // ===================== K and V producers ================================
    const bool isk = warp == C::kProdWarp;
    const int NS = isk ? C::KS : C::VS;
    const uint32_t ring = isk ? sK : sV;
    const int full = isk ? BAR_KFULL : BAR_VFULL, empty = isk ? BAR_KEMPTY : BAR_VEMPTY;
    const CUtensorMap* tmap = isk ? &tmap_k : &tmap_v;
    int T = 0;  // tiles issued
    bool ok = true;
    constexpr int kNone = INT32_MIN;
    segments([&](const Segment& g) {
      const int kvh = g.kvh, base = g.base, t0 = g.t0, n = g.n, vhi = g.hi;
      const int32_t* table = g.table;
      auto lookup = [&](int t) -> int {
        const int key0 = base + t * kTileKeys + lane * kChunk;
        if (lane >= kChunksPerTile || t >= t0 + n || key0 > vhi) return kNone;
        return __ldg(table + key0 / p.block_size);
      };
      int raw = lookup(t0);
      for (int t = t0; t < t0 + n && ok; ++t, ++T) {
        const int next = lookup(t + 1);
        bool bad = false;
        int row8 = -1;
        const int key0 = base + t * kTileKeys + lane * kChunk;
        if (raw != kNone || (lane < kChunksPerTile && key0 <= vhi)) {
          int phys = raw;
          bad = phys < 0 || phys >= p.num_blocks;
          if (bad) phys = 0;  // a stand-in: the rows that see it are marked
          row8 = (int)((((long long)phys * p.num_kv_heads + kvh) * p.block_size + key0 % p.block_size) / 8);
        }
        const uint32_t mask = __ballot_sync(0xffffffffu, row8 >= 0);
        const uint32_t badmask = __ballot_sync(0xffffffffu, bad);
        const int st = T % NS;
        int w = 1;
        if (lane == 0) w = wait(empty + st, (T / NS) ^ 1);
        ok = __shfl_sync(0xffffffffu, w, 0) != 0;
        if (!ok) break;
        if (lane == 0) {
          if (isk) {
            info[T % kInfoSlots] = badmask;
            if (badmask) atomicOr(p.flags, kFlagBadBlock);
          }
          mbar_arrive_expect_tx(bar(full + st), __popc(mask) * kChunkBytes);
        }
        __syncwarp();
        if (row8 >= 0)
          tma_load_4d(ring + st * C::kSlot + lane * kChunkBytes, tmap, 0, 0, 0, row8, bar(full + st));
        __syncwarp();
        raw = next;
      }
    });
    // No copy outlives the CTA: the last of every slot (landed already unless
    // a wait gave up).
    if (lane == 0) {
      volatile int no_abort = 0;
      for (int u = max(0, T - NS); u < T; ++u) mbar_wait(bar(full + u % NS), (u / NS) & 1, &no_abort);
    }
  }
  if (warp == C::kMmaWarp) {
    // ===================== MMA issuer =======================================
    const uint32_t id_qk = idesc_f16_f32(128, 128, false, false);
    const uint32_t id_pv = idesc_f16_f32(128, 128, false, true);
    const uint64_t dQ = smem_desc(sQ, 16, kGroupBytes, kSwizzle128B);
    const uint64_t dK = smem_desc(sK, 16, kGroupBytes, kSwizzle128B);
    const uint64_t dV = smem_desc(sV, kAtomBytes, kGroupBytes, kSwizzle128B);
    int T0 = 0, seg = 0, np0 = 0, np1 = 0;  // np: P of each stream
    bool ok = true;
    segments([&](const Segment& g) {
      if (!ok || lane != 0) return;
      const bool dual = !kQuant && (g.flags & kDual);
      const int n = g.n, X = dual ? 2 * n : n;
      ok = wait(BAR_QFULL, seg);
      if (!ok) return;
      tc_fence_after();
      auto qk = [&](int x) -> bool {
        const int w = x & 1, T = T0 + (dual ? x >> 1 : x), st = T % C::KS;
        if ((!dual || w == 0) && !wait(BAR_KFULL + st, T / C::KS)) return false;
        tc_fence_after();
        const uint64_t qo = dual ? (uint64_t)(w * kTileBytes) >> 4 : 0;
        const uint64_t ko = (uint64_t)(st * C::kSlot) >> 4;
#pragma unroll
        for (int part = 0; part < (kQ8 ? 2 : 1); ++part)  // high parts, residuals of K
#pragma unroll
          for (int k = 0; k < kHeadDim / 16; ++k) {
            const uint64_t o = ((k / 4) * kAtomBytes + (k % 4) * 32) >> 4;
            tc_mma_f16_ss(tmem + w * 128, dQ + qo + o, dK + ko + ((part * kTileBytes) >> 4) + o,
                          id_qk, part > 0 || k > 0);
          }
        tc_commit(bar(BAR_SFULL + w));
        if (!dual || w == 1) tc_commit(bar(BAR_KEMPTY + st));
        return true;
      };
      for (int x = 0; x < 2 && x < X && ok; ++x) ok = qk(x);
      for (int x = 0; x < X && ok; ++x) {
        const int w = x & 1, T = T0 + (dual ? x >> 1 : x), st = T % C::VS;
        ok = wait(BAR_PFULL + w, w ? np1 : np0) &&
             ((dual && w == 1) || wait(BAR_VFULL + st, T / C::VS));
        if (!ok) break;
        w ? ++np1 : ++np0;
        tc_fence_after();
        const uint64_t vo = (uint64_t)(st * C::kSlot) >> 4;
        const uint32_t d = tmem + 256 + w * 128;
        // P_hi V, P_lo V and, q8_0, P_hi V_lo
#pragma unroll
        for (int part = 0; part < (kQ8 ? 3 : 2); ++part)
#pragma unroll
          for (int k = 0; k < kTileKeys / 16; ++k)
            tc_mma_f16_ts(d, tmem + w * 128 + (k / 2) * 32 + (part == 1) * 16 + (k % 2) * 8,
                          dV + vo + ((k * 2 * kGroupBytes + (part == 2) * kTileBytes) >> 4), id_pv,
                          x > 1 || part > 0 || k > 0);
        if (!dual || w == 1) tc_commit(bar(BAR_VEMPTY + st));
        if (x + 2 < X) ok = qk(x + 2);
      }
      if (ok) tc_commit(bar(BAR_SEG));
      T0 += n;
      ++seg;
    });
    if (lane == 0) {
      tc_commit(bar(BAR_DONE));
      volatile int no_abort = 0;
      mbar_wait(bar(BAR_DONE), 0, &no_abort);
    }
    __syncwarp();
  } else if (warp == C::kMmaWarp + 1) {
    // ===================== segments =========================================
    if (lane == 0) {
      int count = 0;
      auto publish = [&](const Segment& g) {
        const int st = count % kSegSlots;
        if (!seg_wait(BAR_GEMPTY + st, (count / kSegSlots) ^ 1)) return;
        segs[st] = g;
        mbar_arrive(bar(BAR_GFULL + st));
        ++count;
      };
      long long x = a;
      while (x < b && x < Wp) {
        Segment g;
        const long long head = (long long)uh * nt, tile = (long long)u1 * nt;
        g.kvh = (int)(x / head);
        const int i = (int)((x - g.kvh * head) / tile);
        const long long at = g.kvh * head + i * tile;
        g.row0 = i * p.row_tile;
        g.nrows = min(R - g.row0, p.row_tile);
        const int u = g.nrows > 128 ? 2 : 1;
        g.t0 = (int)((x - at + u - 1) / u);
        const int te = (int)min((long long)nt, (b - at + u - 1) / u);
        g.n = te - g.t0;
        g.table = p.prefix_table;
        g.lo = vlo;
        g.hi = vhi;
        g.base = vlo / kChunk * kChunk;
        g.clo = 0;
        g.chi = P - 1;
        g.group = g.kvh * NT + i;
        g.out_row = (long long)(cta + g.group) * p.row_tile;
        g.flags = (u == 2 ? kDual : 0) | (g.t0 == 0 ? kFirst : 0) | (te == nt ? kLast : 0);
        if (g.n > 0) publish(g);
        x = at + (long long)u * nt;
      }
      long long at = *reinterpret_cast<volatile long long*>(misc + 4);  // where sequence s begins
      for (int s = misc[3]; x < b && s < p.num_seqs; ++s) {
        Segment g;
        own_keys(__ldg(p.context_lens + s), g.lo, g.hi);
        const int tiles = key_tiles(g.lo, g.hi), len = tiles + kOwnStart;
        if (tiles == 0) continue;
        g.table = p.block_table + (long long)s * p.max_blocks_per_seq;
        g.base = g.lo / kChunk * kChunk;
        g.clo = P;
        g.chi = INT32_MAX;
        for (int j = (int)((x - at) / len); j < hp && x < b; ++j) {
          const long long st = at + (long long)j * len + kOwnStart;  // unit of the first tile
          const int part = j % p.parts;
          g.kvh = j / p.parts;
          g.row0 = s * p.rows_seq + part * p.rows_part;
          g.nrows = min(p.rows_part, p.rows_seq - part * p.rows_part);
          g.t0 = (int)max(0LL, x - st);
          const int te = (int)min((long long)tiles, b - st);
          g.n = te - g.t0;
          g.group = p.num_kv_heads * NT + s * hp + j;
          g.out_row = p.own_row0 + ((long long)cta + s * hp + j) * p.rows_part;
          g.flags = (g.t0 == 0 ? kFirst : 0) | (te == tiles ? kLast : 0);
          if (g.n > 0) publish(g);
          x = st + tiles;
        }
        at += (long long)hp * len;
      }
      Segment end{};
      publish(end);
    }
    __syncwarp();
  } else if (warp < 8) {
    // ===================== softmax warpgroups ===============================
    const int w = warp / 4, r = threadIdx.x % 128;
    const uint32_t lane_off = (uint32_t)(warp % 4 * 32) << 16;
    const uint32_t tS = tmem + lane_off + w * 128, tO = tmem + lane_off + 256;
    const uint32_t flip = p.scale_log2 < 0.f ? 0x80008000u : 0u;  // a negative scale negates Q
    int T0 = 0, seg = 0, ns = 0;  // ns: units of this stream
    bool ok = true;
    segments([&](const Segment& g) {
      const bool dual = !kQuant && (g.flags & kDual);
      const int local = (dual ? w * 128 : 0) + r, row = g.row0 + local;
      const bool mine = local < g.nrows;
      const int tok = row / p.group;  // of all sequences' new tokens
      // ---- Q: this warpgroup's rows (single: half of every row) -------------
      {
        const __half* src = p.q + ((long long)(mine ? tok : 0) * p.num_q_heads + g.kvh * p.group +
                                   (mine ? row % p.group : 0)) * kHeadDim;
        const uint32_t dst = sQ + (dual ? w * kTileBytes : 0) + (r / 8) * kGroupBytes + (r % 8) * 128;
        const int c_lo = dual ? 0 : w * 8, c_hi = dual ? 16 : w * 8 + 8;
#pragma unroll 8
        for (int c = c_lo; c < c_hi; ++c) {
          uint4 v = make_uint4(0, 0, 0, 0);
          if (mine) {
            v = __ldg(reinterpret_cast<const uint4*>(src) + c);
            v.x ^= flip; v.y ^= flip; v.z ^= flip; v.w ^= flip;
          }
          sts_v4(dst + (c / 8) * kAtomBytes + (((c % 8) ^ (r % 8)) * 16), v);
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(BAR_QFULL));
      }
      // ---- this row's keys ----------------------------------------------------
      int lo = 0, hi = -1;
      if (mine) {
        const int L = __ldg(p.context_lens + tok / p.n_query);
        if (shared_seq_ok(p, L, P)) {
          key_range(L, p.n_query, tok % p.n_query, p.causal, p.window, lo, hi);
          lo = max(lo, g.clo);
          hi = min(hi, g.chi);
        }
      }
      const bool warp_rows = __any_sync(0xffffffffu, mine);
      float m = -INFINITY, l = 0.f;  // reference (log2 units) and scaled sum
      bool row_bad = false;
      const int x0 = dual ? 0 : w, step = dual ? 1 : 2;
      for (int t = x0; t < g.n && ok; t += step, ++ns) {
        const int T = T0 + t, kb = g.base + (g.t0 + t) * kTileKeys;
        ok = __all_sync(0xffffffffu, wait(BAR_SFULL + w, ns));
        if (!ok) break;
        tc_fence_after();
        // Keys that no row sees must not reach PV: their V rows become 0 (the
        // converters see to that themselves).
        if (!kQuant && (kb < g.lo || kb + kTileKeys - 1 > g.hi) && (!dual || w == 0)) {
          const int st = T % C::VS;
          ok = __all_sync(0xffffffffu, wait(BAR_VFULL + st, T / C::VS));
          if (ok && (kb + r < g.lo || kb + r > g.hi)) {
            const uint32_t v = sV + st * C::kSlot + (r / 8) * kGroupBytes + (r % 8) * 128;
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              sts_v4(v + c * 16, make_uint4(0, 0, 0, 0));
              sts_v4(v + kAtomBytes + c * 16, make_uint4(0, 0, 0, 0));
            }
          }
          fence_proxy_async_smem();
        }
        if (warp_rows) {
          const uint32_t badmask = info[T % kInfoSlots];
          if (badmask != 0) {  // rows that see a chunk of an out-of-range block
            for (int c = 0; c < kChunksPerTile; ++c)
              if ((badmask >> (kQuant ? c / 2 * 8 + c % 2 : c) & 1) && kb + c * kChunk <= hi &&
                  kb + c * kChunk + kChunk - 1 >= lo)
                row_bad = true;
          }
          const bool whole = __all_sync(0xffffffffu, !mine || (lo <= kb && hi >= kb + kTileKeys - 1));
          // int8 rows: the tile's scales of K (times the softmax scale) and V.
          const float4* ks = reinterpret_cast<const float4*>(smem + C::kScales) + T % kScaleSlots * 32;
          const float4* vs = ks + kScaleSlots * 32;
          // Hidden keys among the 32 from kb + 32 c: -inf in their place.
          auto mask = [&](float (&v)[32], int c) {
            if (whole) return;
            const int k0 = kb + c * 32;
            const int f = max(lo - k0, 0), e = min(hi - k0, 31);  // visible: f .. e
            const uint32_t see = f > e ? 0u : (0xffffffffu >> (31 - (e - f))) << f;
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (!(see >> i & 1)) v[i] = -INFINITY;
          };
          auto top_of = [&](float (&v)[32], int c) -> float {
            if constexpr (kRow) {
#pragma unroll
              for (int e = 0; e < 32; e += 4) {
                const float4 k = ks[c * 8 + e / 4];
                v[e] *= k.x; v[e + 1] *= k.y; v[e + 2] *= k.z; v[e + 3] *= k.w;
              }
            }
            mask(v, c);
            float t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              t0 = fmaxf(t0, fmaxf(v[e], v[e + 1]));
              t1 = fmaxf(t1, fmaxf(v[e + 2], v[e + 3]));
            }
            return fmaxf(t0, t1);
          };
          // Two passes over S in TMEM (a second read costs less than the 128
          // registers of a tile's scores), one chunk of 32 keys ahead.
          float va[32], vb[32];
          tmem_ld32(tS, va);
          tmem_ld_wait(va);
          tmem_ld32(tS + 32, vb);
          float mx = top_of(va, 0);
          tmem_ld_wait(vb);
          tmem_ld32(tS + 64, va);
          mx = fmaxf(mx, top_of(vb, 1));
          tmem_ld_wait(va);
          tmem_ld32(tS + 96, vb);
          mx = fmaxf(mx, top_of(va, 2));
          tmem_ld_wait(vb);
          tmem_ld32(tS, va);
          mx = fmaxf(mx, top_of(vb, 3));
          // The reference m: log2 of the largest weight so far and, int8 rows,
          // of the power of two above the tile's largest |V scale|.
          float top = kRow ? mx : mx * cs;
          if constexpr (kRow) {
            const int st = T % C::VS;
            ok = __all_sync(0xffffffffu, wait(BAR_VFULL + st, T / C::VS));
            if (!ok) {
              tmem_ld_wait();
              break;
            }
            const float4 q4 = *(reinterpret_cast<const float4*>(smem + C::kScales) +
                                2 * kScaleSlots * 32 + T % kScaleSlots);
            const float vm = fmaxf(fmaxf(q4.x, q4.y), fmaxf(q4.z, q4.w));
            const int ex = (int)(__float_as_uint(vm) >> 23) - 126;  // vm < 2^ex
            top += (float)min(max(ex, -64), 64);
          }
          tmem_ld_wait(va);
          const bool raise = top > m + kLazy;
          if (__any_sync(0xffffffffu, raise)) {
            const float mn = raise ? top : m;
            const float f = mn == -INFINITY ? 1.f : fast_exp2(m - mn);
            m = mn;
            l *= f;
            if (t != x0) {  // rescale what this stream has accumulated (PV of its last unit is done)
#pragma unroll 1
              for (int c = 0; c < 4; ++c) {
                float o[32];
                tmem_ld32(tO + w * 128 + c * 32, o);
                tmem_ld_wait(o);
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] *= f;
                tmem_st<16>(tO + w * 128 + c * 32, o);
                tmem_st<16, 16>(tO + w * 128 + c * 32 + 16, o);
              }
              tmem_st_wait();
            }
          }
          const float bias = m == -INFINITY ? 0.f : kShift - m;
          float2 sum = make_float2(0.f, 0.f);
          // Weights of 32 keys over their scores: 16 columns of high parts,
          // 16 of residuals.
          auto weights = [&](float (&v)[32], int c) {
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              float4 k = make_float4(cs, cs, cs, cs);
              if constexpr (kRow) k = ks[c * 8 + e / 4];
              const float2 z0 = fma2(make_float2(v[e], v[e + 1]), make_float2(k.x, k.y),
                                     make_float2(bias, bias));
              const float2 z1 = fma2(make_float2(v[e + 2], v[e + 3]), make_float2(k.z, k.w),
                                     make_float2(bias, bias));
              v[e] = z0.x; v[e + 1] = z0.y; v[e + 2] = z1.x; v[e + 3] = z1.y;
            }
            mask(v, c);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t ph[8], pl[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const int e = 16 * h + 2 * i;
                float2 x = make_float2(fast_exp2(v[e]), fast_exp2(v[e + 1]));
                sum = add2(sum, x);
                if constexpr (kRow) x = mul2(x, reinterpret_cast<const float2*>(vs)[c * 16 + e / 2]);
                // the high part by truncation, so that the residual is exact
                const float2 hi2 = make_float2(__uint_as_float(__float_as_uint(x.x) & 0xffffe000u),
                                               __uint_as_float(__float_as_uint(x.y) & 0xffffe000u));
                const float2 res = add2(x, make_float2(-hi2.x, -hi2.y));
                ph[i] = h2_bits(__floats2half2_rn(hi2.x, hi2.y));
                pl[i] = h2_bits(__floats2half2_rn(res.x, res.y));
              }
              tmem_st8(tS + c * 32 + h * 8, ph);
              tmem_st8(tS + c * 32 + 16 + h * 8, pl);
            }
          };
          tmem_ld32(tS + 32, vb);
          weights(va, 0);
          tmem_ld_wait(vb);
          tmem_ld32(tS + 64, va);
          weights(vb, 1);
          tmem_ld_wait(va);
          tmem_ld32(tS + 96, vb);
          weights(va, 2);
          tmem_ld_wait(vb);
          weights(vb, 3);
          l += sum.x + sum.y;
          tmem_st_wait();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(BAR_PFULL + w));
      }
      // ---- the segment's partial ------------------------------------------------
      ok = __all_sync(0xffffffffu, ok && wait(BAR_SEG, seg));
      if (threadIdx.x == 0) {
        if (g.flags & kFirst) p.meta[2 + 2 * g.group] = cta;
        if (g.flags & kLast) p.meta[3 + 2 * g.group] = cta;
      }
      const long long at = g.out_row + local;
      float* out = p.part_out + at * kHeadDim;
      if (dual) {
        if (mine)
          p.part_lse[at] = (!ok || row_bad || l != l) ? __uint_as_float(kInvalidLse)
                           : l > 0.f                  ? (m - kShift + log2f(l)) * kLn2
                                                      : -INFINITY;
        if (ok && warp_rows) {
          tc_fence_after();
          const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            float o[32];
            tmem_ld32(tO + w * 128 + c * 32, o);
            tmem_ld_wait(o);
            if (mine) {
#pragma unroll
              for (int e = 0; e < 8; ++e)
                reinterpret_cast<float4*>(out + c * 32)[e] =
                    make_float4(o[4 * e] * inv, o[4 * e + 1] * inv, o[4 * e + 2] * inv, o[4 * e + 3] * inv);
            }
          }
        }
      } else {
        // Both streams' sums for this row; each warpgroup writes 64 columns.
        float2* stat = reinterpret_cast<float2*>(smem + C::kQ);  // Q has been read
        stat[w * 128 + r] = make_float2(row_bad ? __uint_as_float(kInvalidLse) : m, l);
        ok = named_bar_and(1, 256, ok);
        const float2 s0 = stat[r], s1 = stat[128 + r];
        const bool bad = !ok || isnan(s0.x + s0.y) || isnan(s1.x + s1.y);
        const float mm = fmaxf(s0.x, s1.x);
        const float w0 = s0.y > 0.f ? fast_exp2(s0.x - mm) : 0.f;
        const float w1 = s1.y > 0.f ? fast_exp2(s1.x - mm) : 0.f;
        const float ll = s0.y * w0 + s1.y * w1;
        if (w == 0 && mine)
          p.part_lse[at] = bad        ? __uint_as_float(kInvalidLse)
                           : ll > 0.f ? (mm - kShift + log2f(ll)) * kLn2
                                      : -INFINITY;
        if (ok && warp_rows) {
          tc_fence_after();
          const float inv = ll > 0.f ? 1.f / ll : 0.f;
          const float f0 = w0 * inv, f1 = w1 * inv;
#pragma unroll 1
          for (int c = 0; c < 2; ++c) {
            float o0[32], o1[32];
            tmem_ld32(tO + w * 64 + c * 32, o0);
            tmem_ld32(tO + 128 + w * 64 + c * 32, o1);
            tmem_ld_wait(o0);
            tmem_ld_wait(o1);
            if (mine) {
#pragma unroll
              for (int e = 0; e < 32; ++e)  // a stream without keys holds no sums
                o0[e] = (f0 > 0.f ? o0[e] * f0 : 0.f) + (f1 > 0.f ? o1[e] * f1 : 0.f);
#pragma unroll
              for (int e = 0; e < 8; ++e)
                reinterpret_cast<float4*>(out + w * 64 + c * 32)[e] =
                    make_float4(o0[4 * e], o0[4 * e + 1], o0[4 * e + 2], o0[4 * e + 3]);
            }
          }
        }
        named_bar_sync(2, 256);  // the sums have been read: Q may be staged again
      }
      T0 += g.n;
      ++seg;
    });
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == C::kMmaWarp) {
    tmem_relinquish();
    tmem_dealloc(tmem, 512);
  }
  if (threadIdx.x == 0 && *abort) atomicOr(p.flags, kFlagTimeout);
}

// ---- host side --------------------------------------------------------------
PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> fn{nullptr};
  PFN_cuTensorMapEncodeTiled_v12000 f = fn.load(std::memory_order_acquire);
  if (f == nullptr) {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess) {
      f = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
      fn.store(f, std::memory_order_release);
    }
  }
  return f;
}

// The fp16 cache as {64 columns, 8 rows, 2 halves, rows / 8}: one box of 16
// rows lands as [row / 8][half][8 rows][64 columns].
bool encode_cache_map(CUtensorMap* m, const void* cache, long long rows) {
  auto fn = encode_fn();
  if (fn == nullptr || rows % 8 != 0) return false;
  cuuint64_t dims[4] = {64, 8, 2, (cuuint64_t)(rows / 8)};
  cuuint64_t strides[3] = {(cuuint64_t)kHeadDim * 2, 128, 8 * (cuuint64_t)kHeadDim * 2};
  cuuint32_t box[4] = {64, 8, 2, 2};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, const_cast<void*>(cache), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int KV>
cudaError_t launch_tc(const SharedParams& p, cudaStream_t stream) {
  auto kern = shared_tc_kernel<KV>;
  const size_t smem = Cfg<KV>::kTotal + 1024;
  static std::atomic<unsigned long long> ready{0};  // devices whose attribute is set
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!(ready.load(std::memory_order_acquire) >> dev & 1)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    ready.fetch_or(1ull << dev, std::memory_order_release);
  }
  CUtensorMap mk{}, mv{};
  const long long rows = (long long)p.num_blocks * p.num_kv_heads * p.block_size;
  if (KV == kKvFp16 && (!encode_cache_map(&mk, p.k, rows) || !encode_cache_map(&mv, p.v, rows)))
    return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.ctas);
  cfg.blockDim = dim3(Cfg<KV>::kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, mk, mv, p);
}

}  // namespace

cudaError_t launch_shared_tc(const SharedParams& p, cudaStream_t stream) {
  switch (p.kv_dtype) {
    case kKvQ8_0: return launch_tc<kKvQ8_0>(p, stream);
    case kKvInt8Row: return launch_tc<kKvInt8Row>(p, stream);
    default: return launch_tc<kKvFp16>(p, stream);
  }
}

}  // namespace pa
