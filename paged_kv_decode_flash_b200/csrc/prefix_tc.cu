// prefix_tc.cu -- the prefix part of the shared-prefix decode on the sm_100a
// tensor cores: every query row of the batch against the keys that all
// sequences share.
//
// Mathematics: for a row with scores z_j (log2 units), weights
// 2^(z_j - m + 8) with a reference m that follows the running maximum
// lazily; l = sum of the weights, O = sum of weight * v, one pass over the
// keys; the partial is O / l with lse = (m - 8 + log2 l) ln 2.
//
// Work.  The rows of a KV head (sequences x new tokens x the head's query
// heads) are cut into row tiles of 128, or 256 where there are more than
// 128; a (KV head, row tile) is a group.  The prefix's visible keys are
// numbered in tiles of 128.  The tiles of all groups, laid end to end, are
// cut into equal ranges over the CTAs (one per SM); a CTA's run of tiles of
// one group is a segment and makes one partial per row.
//
// A CTA has two streams, each a softmax warpgroup (thread = query row), an
// S / P buffer and an O accumulator of 128 x 128 in TMEM, so that the tensor
// cores work for one stream while the other's softmax runs:
//   pair:   stream w has row tile half w and every key tile (a K and a V
//           tile in shared memory serve 256 rows);
//   single: both streams have the same 128 rows, stream w every other key
//           tile; their sums are joined at the segment's end.
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
// They always run the single form: its 128 rows leave shared memory for the
// converted tiles.
//
// Roles: warps 0-3 and 4-7 the softmax warpgroups, which also stage Q and
// write the partials.  fp16: warp 8 K producer, warp 9 V producer (TMA boxes
// of 16 keys through the block table), warp 10 MMA issuer.  int8: warps 8-11
// K converters, 12-15 V converters (raw bytes through registers, one tile
// ahead), warp 16 MMA issuer.
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
constexpr float kShift = 8.f;   // weights are scaled by 2^kShift
constexpr float kLazy = 7.f;    // ... and stay below 2^(kShift + kLazy) < 65504
constexpr float kLn2 = 0.69314718055994531f;
constexpr unsigned kInvalidLse = 0x7fc00000u;  // NaN: a partial that must not be used
constexpr int kInfoSlots = 16;
constexpr int kScaleSlots = 8;  // tiles whose row scales are kept: more than are in flight

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
  BAR_COUNT = 19
};

template <bool kPair, int KV>
struct Cfg {
  static constexpr bool kQuant = KV != kKvFp16;
  static constexpr bool kQ8 = KV == kKvQ8_0, kRow = KV == kKvInt8Row;
  static constexpr int kProdWarp = 8;                      // fp16: K, V producer; int8: converters
  static constexpr int kMmaWarp = kQuant ? 16 : 10;
  static constexpr int kThreads = 32 * (kMmaWarp + 1);
  static constexpr int kRowTile = kPair ? 256 : 128;
  static constexpr uint32_t kSlot = (kQ8 ? 2 : 1) * kTileBytes;  // q8_0: the high tile, the residual
  static constexpr int KS = kQ8 ? 1 : kRow ? 2 : 3;
  static constexpr int VS = kPair || kQ8 ? 2 : 3;
  static constexpr uint32_t kQ = 0;
  static constexpr uint32_t kK = kQ + (kPair ? 2 : 1) * kTileBytes;
  static constexpr uint32_t kV = kK + KS * kSlot;
  static constexpr uint32_t kBars = kV + VS * kSlot;
  static constexpr uint32_t kInfo = kBars + BAR_COUNT * 8 + 8;      // uint32 [kInfoSlots]
  static constexpr uint32_t kMisc = kInfo + kInfoSlots * 4;         // int [8]
  static constexpr uint32_t kScales = kMisc + 32;  // int8 rows: float K [8][128], V [8][128], max [8][4]
  static constexpr uint32_t kTotal = kScales + (kRow ? kScaleSlots * (2 * 128 + 4) * 4 : 0);
  static_assert(kBars % 16 == 0 && kScales % 16 == 0, "alignment");
  static_assert(kTotal + 1024 <= 232448, "shared memory per CTA");
  static_assert(!(kPair && kQuant), "int8: single form");
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

template <bool kPair, int KV>
__global__ void __launch_bounds__(Cfg<kPair, KV>::kThreads, 1)
    prefix_tc_kernel(const __grid_constant__ CUtensorMap tmap_k,
                     const __grid_constant__ CUtensorMap tmap_v, const SharedParams p) {
  using C = Cfg<kPair, KV>;
  constexpr bool kQuant = C::kQuant, kQ8 = C::kQ8, kRow = C::kRow;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  const uint32_t sQ = sbase + C::kQ, sK = sbase + C::kK, sV = sbase + C::kV;
  uint32_t* info = reinterpret_cast<uint32_t*>(smem + C::kInfo);
  int* misc = reinterpret_cast<int*>(smem + C::kMisc);  // [0] TMEM base, [1] abort, [2] min L
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
                                                                                         : 1);
    misc[1] = 0;
    misc[2] = INT32_MAX;
    fence_mbar_init();
  }
  if (warp == C::kMmaWarp) tmem_alloc(smem_u32(misc), 512);
  griddep_wait();
  griddep_launch_dependents();
  // The visible prefix keys [vlo, vhi] of the batch (shared_range), with the
  // shortest valid sequence where a window hides early keys.
  const int P = __ldg(p.prefix_len);
  int vlo = 0, vhi = -1;
  if (shared_prefix_ok(p, P)) {
    vhi = P - 1;
    if (p.window > 0) {
      __syncthreads();
      int m = INT32_MAX;
      for (int s = threadIdx.x; s < p.num_seqs; s += C::kThreads) {
        const int L = __ldg(p.context_lens + s);
        if (shared_seq_ok(p, L, P)) m = min(m, L);
      }
      if (m != INT32_MAX) atomicMin(misc + 2, m);
      __syncthreads();
      m = misc[2];
      if (m == INT32_MAX) {
        vhi = -1;
      } else {
        int hi;
        key_range(m, p.n_query, 0, p.causal, p.window, vlo, hi);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc[0];

  const int base = vlo / kChunk * kChunk;
  const int nt = vhi >= vlo ? (vhi + 1 - base + kTileKeys - 1) / kTileKeys : 0;
  const int NT = (p.rows_head + C::kRowTile - 1) / C::kRowTile;
  const int groups = p.num_kv_heads * NT;
  const long long W = (long long)groups * nt;
  const int Ce = (int)min(W, (long long)p.ctas);
  const int cta = blockIdx.x;
  if (cta == 0 && threadIdx.x == 0) {  // for the join
    p.meta[0] = nt;
    p.meta[1] = Ce;
  }
  long long a = 0, b = 0;
  if (cta < Ce) {
    a = cta * W / Ce;
    b = (cta + 1) * W / Ce;
  }
  // Calls f(group, first tile, tiles) for every segment of this CTA.
  auto segments = [&](auto&& f) {
    for (long long x = a; x < b;) {
      const int g = (int)(x / nt), t0 = (int)(x - (long long)g * nt);
      const int n = (int)min((long long)(nt - t0), b - x);
      f(g, t0, n);
      x += n;
    }
  };

  if constexpr (kQuant) {
    if (warp >= C::kProdWarp && warp < C::kMmaWarp) {
      // ===================== int8 converters ================================
      // A warp takes 32 keys of every tile, eight lanes a key: coalesced loads
      // into registers one tile ahead, then the operand layout.
      const bool isk = warp < C::kProdWarp + 4;
      const int cw = warp % 4, kq = lane / 8, cl = lane % 8;
      const int NS = isk ? C::KS : C::VS;
      const uint32_t ring = isk ? sK : sV;
      const int full = isk ? BAR_KFULL : BAR_VFULL, empty = isk ? BAR_KEMPTY : BAR_VEMPTY;
      const uint8_t* cache = static_cast<const uint8_t*>(isk ? p.k : p.v);
      const long long tile_bytes = quant_tile_bytes(KV, p.block_size);
      float* scales = reinterpret_cast<float*>(smem + C::kScales) + (isk ? 0 : kScaleSlots * 128);
      float* vmax = reinterpret_cast<float*>(smem + C::kScales) + 2 * kScaleSlots * 128;
      int T = 0;
      bool ok = true;
      segments([&](int g, int t0, int n) {
        const int kvh = g / NT, te = t0 + n;
        // The block of this warp's two chunks of tile t (lanes 0, 1).
        auto lookup = [&](int t) -> int {
          const int key0 = base + t * kTileKeys + (2 * cw + lane) * kChunk;
          return lane < 2 && t < te && key0 <= vhi ? __ldg(p.prefix_table + key0 / p.block_size) : 0;
        };
        uint4 raw[8];
        uint16_t sc8[kQ8 ? 8 : 1];
        float sc1 = 0.f;
        uint32_t bad = 0;  // out-of-range blocks of the tile in registers
        auto fetch = [&](int t, int phys) {
          const bool b = phys < 0 || phys >= p.num_blocks;
          bad = __ballot_sync(0xffffffffu, b);
          if (b) phys = 0;  // a stand-in: the rows that see it are marked
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int key0 = base + t * kTileKeys + (2 * cw + h) * kChunk;
            const long long ph = __shfl_sync(0xffffffffu, phys, h);
            const bool on = t < te && key0 <= vhi;
            const uint8_t* tile = cache + (ph * p.num_kv_heads + kvh) * tile_bytes;
            const int slot = key0 % p.block_size;
#pragma unroll
            for (int i = 4 * h; i < 4 * h + 4; ++i) {
              const int k = slot + (4 * i) % kChunk + kq;
              raw[i] = make_uint4(0, 0, 0, 0);
              if constexpr (kQ8) sc8[i] = 0;
              if (on) {
                raw[i] = __ldg(reinterpret_cast<const uint4*>(tile + k * kHeadDim) + cl);
                if constexpr (kQ8)
                  sc8[i] = __ldg(reinterpret_cast<const unsigned short*>(
                                     tile + p.block_size * kHeadDim + k * 8) + cl / 2);
              }
            }
            if constexpr (kRow) {
              if (lane / kChunk == h) {
                sc1 = 0.f;
                if (on)
                  sc1 = __ldg(reinterpret_cast<const float*>(tile + p.block_size * kHeadDim) + slot +
                              lane % kChunk);
              }
            }
          }
        };
        fetch(t0, lookup(t0));
        int phys = lookup(t0 + 1);
        for (int t = t0; t < te && ok; ++t, ++T) {
          const int st = T % NS, kw = base + t * kTileKeys + 32 * cw;
          ok = __all_sync(0xffffffffu, wait(empty + st, (T / NS) ^ 1));
          if (!ok) break;
          if (isk && lane == 0) {
            reinterpret_cast<uint8_t*>(info + T % kInfoSlots)[cw] = (uint8_t)bad;
            if (bad) atomicOr(p.flags, kFlagBadBlock);
          }
          if constexpr (kRow) {  // scales of hidden keys may be anything
            const bool seen = kw + lane >= vlo && kw + lane <= vhi;
            const float d = isk ? sc1 * cs : seen ? sc1 : 0.f;
            scales[T % kScaleSlots * 128 + 32 * cw + lane] = d;
            if (!isk) {
              float mx = fabsf(d);
#pragma unroll
              for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
              if (lane == 0) vmax[T % kScaleSlots * 4 + cw] = mx;
            }
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int r = 32 * cw + 4 * i + kq;
            const uint32_t dst = ring + st * C::kSlot + (r / 8) * kGroupBytes + (r % 8) * 128 +
                                 (cl / 4) * kAtomBytes;
            __half2 x[8];
            const uint32_t wd[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
            for (int y = 0; y < 4; ++y) q8_to_half4(wd[y], x[2 * y], x[2 * y + 1]);
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
              __half d = __ushort_as_half(sc8[i]);
              const int key = kw + 4 * i + kq;
              if (!isk && (key < vlo || key > vhi)) d = __ushort_as_half(0);
              const __half2 d2 = __halves2half2(d, d);
              __half2 hi8[8];
#pragma unroll
              for (int y = 0; y < 8; ++y) {
                hi8[y] = __hmul2(x[y], d2);
                x[y] = __hfma2(x[y], d2, __hneg2(hi8[y]));  // the residual, exact above 2^-24
              }
              put(hi8, 0);
              put(x, kTileBytes);
            } else {
              put(x, 0);
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(full + st));
          fetch(t + 1, phys);
          phys = lookup(t + 2);
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
    segments([&](int g, int t0, int n) {
      const int kvh = g / NT;
      auto lookup = [&](int t) -> int {
        const int key0 = base + t * kTileKeys + lane * kChunk;
        if (lane >= kChunksPerTile || t >= t0 + n || key0 > vhi) return kNone;
        return __ldg(p.prefix_table + key0 / p.block_size);
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
    if (lane == 0) {
      const uint32_t id_qk = idesc_f16_f32(128, 128, false, false);
      const uint32_t id_pv = idesc_f16_f32(128, 128, false, true);
      const uint64_t dQ = smem_desc(sQ, 16, kGroupBytes, kSwizzle128B);
      const uint64_t dK = smem_desc(sK, 16, kGroupBytes, kSwizzle128B);
      const uint64_t dV = smem_desc(sV, kAtomBytes, kGroupBytes, kSwizzle128B);
      int T0 = 0, seg = 0, np[2] = {0, 0};
      bool ok = true;
      segments([&](int, int, int n) {
        if (!ok) return;
        const int X = kPair ? 2 * n : n;
        ok = wait(BAR_QFULL, seg);
        if (!ok) return;
        tc_fence_after();
        auto qk = [&](int x) -> bool {
          const int w = x & 1, T = T0 + (kPair ? x >> 1 : x), st = T % C::KS;
          if ((!kPair || w == 0) && !wait(BAR_KFULL + st, T / C::KS)) return false;
          tc_fence_after();
          const uint64_t qo = kPair ? (uint64_t)(w * kTileBytes) >> 4 : 0;
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
          if (!kPair || w == 1) tc_commit(bar(BAR_KEMPTY + st));
          return true;
        };
        for (int x = 0; x < 2 && x < X && ok; ++x) ok = qk(x);
        for (int x = 0; x < X && ok; ++x) {
          const int w = x & 1, T = T0 + (kPair ? x >> 1 : x), st = T % C::VS;
          ok = wait(BAR_PFULL + w, np[w]) &&
               ((kPair && w == 1) || wait(BAR_VFULL + st, T / C::VS));
          if (!ok) break;
          ++np[w];
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
          if (!kPair || w == 1) tc_commit(bar(BAR_VEMPTY + st));
          if (x + 2 < X) ok = qk(x + 2);
        }
        if (ok) tc_commit(bar(BAR_SEG));
        T0 += n;
        ++seg;
      });
      tc_commit(bar(BAR_DONE));
      volatile int no_abort = 0;
      mbar_wait(bar(BAR_DONE), 0, &no_abort);
    }
    __syncwarp();
  } else if (warp < 8) {
    // ===================== softmax warpgroups ===============================
    const int w = warp / 4, r = threadIdx.x % 128;
    const uint32_t lane_off = (uint32_t)(warp % 4 * 32) << 16;
    const uint32_t tS = tmem + lane_off + w * 128, tO = tmem + lane_off + 256;
    const uint32_t flip = p.scale_log2 < 0.f ? 0x80008000u : 0u;  // a negative scale negates Q
    const int R = p.rows_head;
    int T0 = 0, seg = 0, ns = 0;  // ns: units of this stream
    bool ok = true;
    segments([&](int g, int t0, int n) {
      const int kvh = g / NT, row0 = (g % NT) * C::kRowTile;
      const int row = row0 + (kPair ? w * 128 : 0) + r;
      // ---- Q: this warpgroup's rows (single: half of every row) -------------
      {
        const int rr = row;
        const bool in = rr < R;
        const __half* src = p.q + ((long long)(in ? rr / p.group : 0) * p.num_q_heads + kvh * p.group +
                                   (in ? rr % p.group : 0)) * kHeadDim;
        const uint32_t dst = sQ + (kPair ? w * kTileBytes : 0) + (r / 8) * kGroupBytes + (r % 8) * 128;
        const int c_lo = kPair ? 0 : w * 8, c_hi = kPair ? 16 : w * 8 + 8;
#pragma unroll 8
        for (int c = c_lo; c < c_hi; ++c) {
          uint4 v = make_uint4(0, 0, 0, 0);
          if (in) {
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
      if (row < R) {
        const int tok = row / p.group, s = tok / p.n_query;
        const int L = __ldg(p.context_lens + s);
        if (shared_seq_ok(p, L, P)) {
          key_range(L, p.n_query, tok % p.n_query, p.causal, p.window, lo, hi);
          hi = min(hi, P - 1);
        }
      }
      const bool warp_rows = __any_sync(0xffffffffu, row < R);
      float m = -INFINITY, l = 0.f;  // reference (log2 units) and scaled sum
      bool row_bad = false;
      const int x0 = kPair ? 0 : w, step = kPair ? 1 : 2;
      for (int t = x0; t < n && ok; t += step, ++ns) {
        const int T = T0 + t, kb = base + (t0 + t) * kTileKeys;
        ok = __all_sync(0xffffffffu, wait(BAR_SFULL + w, ns));
        if (!ok) break;
        tc_fence_after();
        // Keys that no row sees must not reach PV: their V rows become 0 (the
        // converters see to that themselves).
        if (!kQuant && (kb < vlo || kb + kTileKeys - 1 > vhi) && (!kPair || w == 0)) {
          const int st = T % C::VS;
          ok = __all_sync(0xffffffffu, wait(BAR_VFULL + st, T / C::VS));
          if (ok && (kb + r < vlo || kb + r > vhi)) {
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
              if ((badmask >> (kQuant ? c / 2 * 8 + c % 2 : c) & 1) && kb + c * kChunk <= hi && kb + c * kChunk + kChunk - 1 >= lo)
                row_bad = true;
          }
          const bool whole = __all_sync(0xffffffffu, row >= R || (lo <= kb && hi >= kb + kTileKeys - 1));
          // Scores of 32 keys: z = v * (scale and, int8 rows, K's row scale).
          const float4* ks = reinterpret_cast<const float4*>(smem + C::kScales) + T % kScaleSlots * 32;
          const float4* vs = ks + kScaleSlots * 32;
          auto hidden = [&](int key) { return key < lo || key > hi; };
          auto top_of = [&](const float (&v)[32], int c) -> float {
            float t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              float z[4] = {v[e], v[e + 1], v[e + 2], v[e + 3]};
              if constexpr (kRow) {
                const float4 k = ks[c * 8 + e / 4];
                z[0] *= k.x; z[1] *= k.y; z[2] *= k.z; z[3] *= k.w;
              }
              if (!whole) {
#pragma unroll
                for (int x = 0; x < 4; ++x)
                  if (hidden(kb + c * 32 + e + x)) z[x] = -INFINITY;
              }
              t0 = fmaxf(t0, fmaxf(z[0], z[1]));
              t1 = fmaxf(t1, fmaxf(z[2], z[3]));
            }
            return fmaxf(t0, t1);
          };
          // fp16 keeps the tile's 128 scores in registers; the int8 forms,
          // whose converters need registers too, read them a second time.
          constexpr int kHold = kQuant ? 1 : 4;
          float v[kHold][32];
          float mx = -INFINITY;
          if constexpr (kHold == 4) {
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld32(tS + c * 32, v[c % kHold]);
            tmem_ld_wait();
#pragma unroll
            for (int c = 0; c < 4; ++c) mx = fmaxf(mx, top_of(v[c % kHold], c));
          } else {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              tmem_ld32(tS + c * 32, v[0]);
              tmem_ld_wait();
              mx = fmaxf(mx, top_of(v[0], c));
            }
          }
          // The reference m: log2 of the largest weight so far and, int8 rows,
          // of the power of two above the tile's largest |V scale|.
          float top = kRow ? mx : mx * cs;
          if constexpr (kRow) {
            const int st = T % C::VS;
            ok = __all_sync(0xffffffffu, wait(BAR_VFULL + st, T / C::VS));
            if (!ok) break;
            const float4 q4 = *(reinterpret_cast<const float4*>(smem + C::kScales) +
                                2 * kScaleSlots * 32 + T % kScaleSlots);
            const float vm = fmaxf(fmaxf(q4.x, q4.y), fmaxf(q4.z, q4.w));
            const int ex = (int)(__float_as_uint(vm) >> 23) - 126;  // vm < 2^ex
            top += (float)min(max(ex, -64), 64);
          }
          const bool raise = top > m + kLazy;
          if (__any_sync(0xffffffffu, raise)) {
            const float mn = raise ? top : m;
            const float f = mn == -INFINITY ? 1.f : fast_exp2(m - mn);
            m = mn;
            l *= f;
            if (t != x0) {  // rescale what this stream has accumulated (PV of its last unit is done)
#pragma unroll
              for (int c = 0; c < 8; ++c) {
                float o[16];
                tmem_ld<16>(tO + w * 128 + c * 16, o);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] *= f;
                tmem_st<16>(tO + w * 128 + c * 16, o);
              }
              tmem_st_wait();
            }
          }
          const float bias = m == -INFINITY ? 0.f : kShift - m;
          float sum = 0.f;
          // Weights of 32 keys over their scores: 16 columns of high parts,
          // 16 of residuals.
          auto weights = [&](const float (&v)[32], int c) {
            uint32_t ph[16], pl[16];
            float s0 = 0.f, s1 = 0.f;
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              float k4[4] = {cs, cs, cs, cs}, x[4];
              if constexpr (kRow) {
                const float4 k = ks[c * 8 + e / 4];
                k4[0] = k.x; k4[1] = k.y; k4[2] = k.z; k4[3] = k.w;
              }
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                float z = fmaf(v[e + y], k4[y], bias);
                if (!whole && hidden(kb + c * 32 + e + y)) z = -INFINITY;
                x[y] = fast_exp2(z);
              }
              s0 += x[0] + x[2];
              s1 += x[1] + x[3];
              if constexpr (kRow) {
                const float4 d = vs[c * 8 + e / 4];
                x[0] *= d.x; x[1] *= d.y; x[2] *= d.z; x[3] *= d.w;
              }
#pragma unroll
              for (int y = 0; y < 4; y += 2) {
                // the high part by truncation, so that the residual is exact
                const float xh = __uint_as_float(__float_as_uint(x[y]) & 0xffffe000u);
                const float yh = __uint_as_float(__float_as_uint(x[y + 1]) & 0xffffe000u);
                ph[(e + y) / 2] = h2_bits(__floats2half2_rn(xh, yh));
                pl[(e + y) / 2] = h2_bits(__floats2half2_rn(x[y] - xh, x[y + 1] - yh));
              }
            }
            sum += s0 + s1;
            tmem_st16(tS + c * 32, ph);
            tmem_st16(tS + c * 32 + 16, pl);
          };
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            if constexpr (kHold == 1) {
              tmem_ld32(tS + c * 32, v[0]);
              tmem_ld_wait();
            }
            weights(v[c % kHold], c);
          }
          l += sum;
          tmem_st_wait();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(BAR_PFULL + w));
      }
      // ---- the segment's partial ------------------------------------------------
      ok = __all_sync(0xffffffffu, ok && wait(BAR_SEG, seg));
      const long long slot = (long long)cta + g;
      const int pr = (kPair ? w * 128 : 0) + r;  // row of the slot
      float* out = p.part_out + (slot * C::kRowTile + pr) * kHeadDim;
      if constexpr (kPair) {
        if (row < R)
          p.part_lse[slot * C::kRowTile + pr] = (!ok || row_bad || l != l) ? __uint_as_float(kInvalidLse)
                                                : l > 0.f ? (m - kShift + log2f(l)) * kLn2
                                                          : -INFINITY;
        if (ok && warp_rows) {
          tc_fence_after();
          const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            float o[32];
            tmem_ld32(tO + w * 128 + c * 32, o);
            tmem_ld_wait();
            if (row < R) {
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
        if (w == 0 && row < R)
          p.part_lse[slot * C::kRowTile + pr] = bad        ? __uint_as_float(kInvalidLse)
                                                : ll > 0.f ? (mm - kShift + log2f(ll)) * kLn2
                                                           : -INFINITY;
        if (ok && warp_rows) {
          tc_fence_after();
          const float inv = ll > 0.f ? 1.f / ll : 0.f;
          const float f0 = w0 * inv, f1 = w1 * inv;
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float o0[32], o1[32];
            tmem_ld32(tO + w * 64 + c * 32, o0);
            tmem_ld32(tO + 128 + w * 64 + c * 32, o1);
            tmem_ld_wait();
            if (row < R) {
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
      T0 += n;
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

template <bool kPair, int KV>
cudaError_t launch_tc(const SharedParams& p, cudaStream_t stream) {
  auto kern = prefix_tc_kernel<kPair, KV>;
  const size_t smem = Cfg<kPair, KV>::kTotal + 1024;
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
  cfg.blockDim = dim3(Cfg<kPair, KV>::kThreads);
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

cudaError_t launch_prefix_tc(const SharedParams& p, cudaStream_t stream) {
  switch (p.kv_dtype) {
    case kKvQ8_0: return launch_tc<false, kKvQ8_0>(p, stream);
    case kKvInt8Row: return launch_tc<false, kKvInt8Row>(p, stream);
    default: break;
  }
  return p.row_tile == 256 ? launch_tc<true, kKvFp16>(p, stream)
                           : launch_tc<false, kKvFp16>(p, stream);
}

}  // namespace pa
