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
// query heads) are cut into row tiles of 256 rows (128 where there are no
// more, and for q8_0); a (KV head, row tile) is a group.  Own keys: a
// (sequence, KV head, part of at most 128 of the sequence's rows) is a group.
// A group's visible keys are numbered in tiles of 128.  The tiles of all
// groups, prefix first, are laid end to end and cut into equal ranges over the
// CTAs (one per SM; a group's start counts as a few tiles); a CTA's run of
// tiles of one group is a segment and makes one partial per row.
//
// A CTA has two streams, each a softmax warpgroup (thread = query row) and an
// O accumulator of 128 x 128 in TMEM:
//   dual segment (more than 128 rows): stream w has rows 128 w .. and every
//           key (a K and a V tile in shared memory serve 256 rows);
//   single: both streams have the same rows, stream w keys 64 w .. of every
//           tile; their sums are joined at the segment's end.
// A stream works in steps of 64 keys with two S / P buffers of 64 columns, so
// that its next scores are there when a step's softmax ends: S = Q K^T
// (M = 128 rows, N = 64 keys), P overwrites S in TMEM as fp16 high parts and
// residuals (the weights to 2^-22, as in the other decode kernels), and
// O += [P_hi | P_lo] V takes P from TMEM and V as it lies in the cache.
//
// The int8 caches are converted on the way in, to operands that lose nothing
// that matters:
//   q8_0: a value qs * d has at most 19 significant bits and enters as fp16
//         high part and residual, K and V alike: S = Q K_hi + Q K_lo,
//         O += P_hi V_hi + P_lo V_hi + P_hi V_lo (2^-22);
//   int8 rows: qs enters as it is.  K's row scale multiplies the scores, V's
//         the weights before their split, so that both cost no MMA.  What has
//         to fit fp16 is then weight x V scale: the reference of a row is the
//         largest z_j + log2 |V scale j| (within 2^+-kScaleLog), key by key.
// q8_0 runs single segments only: 128 rows leave shared memory for operands of
// two tiles.
//
// Precision.  The tensor cores add to O in 32 bits but cut off what does not
// fit, toward zero, twice for every 16 keys (P_hi V, P_lo V).  Over a CTA's run
// of keys that is a bias: 2e-5 of the output's size after 14,000 keys, 8.5e-5
// after 113,000 (fp16's half step: 4.9e-4).  The sums of weights, the join and
// all references are rounded to nearest.
//
// Roles: warps 0-7 the softmax, which also stages Q and writes the partials.
// Then, fp16: a producer (TMA boxes of 16 keys through the block table);
// int8: eight converters (raw bytes through registers, one tile ahead).  Then
// an MMA issuer for each stream (one for both was the bottleneck: with the
// waits, a step's sixteen products take a warp 1750 cycles to issue and the
// tensor cores 780), and a warp that cuts the CTA's range into segments.
//
// Bounds.  Many rows: the tensor cores.  A step's products take 8 x 49 cycles
// (Q K^T with N = 64: Q and K come from shared memory, 6 KB a product) and
// 8 x 64 (P V), 1808 for both streams; a pair of steps was measured at 2210
// (512 rows a KV head, 8 of them, 131072 keys: 392 us at full clocks, 463 to 475
// in a row of such calls under the power cap), 2366 with the commits
// between the products and V awaited behind P, 4800 with one issuer that is one
// lane.  The exponentials (2 x 64 a lane, 1024 cycles) and the conversions
// to fp16 share what is left.  q8_0: 4400 a pair, int8 rows 3440, set by the
// converters and the softmax together (48% of the issue slots).  Few rows: a
// chain of latencies, 4.1 us to the first scores, 8 to the end of a segment
// of one tile.  Tried without gain: the streams' exponentials in turn, half a
// step's keys a warp (four softmax warps a scheduler), the scores of both
// streams of a single segment in one product of N = 128, q8_0 slots of 64 keys.
//
// Every wait is bounded (SharedParams::wait_limit_ns; the wait for a segment's
// slot by that much a tile of the segment in it): a role that gives up sets the
// CTA's abort word, at which every other wait ends, too.  The kernel then
// raises kFlagTimeout, drains its copies and MMAs with a fixed bound and frees
// TMEM.  Every CTA writes, in every call, whether it gave up and which groups
// begin and end with it, so that the join never takes an earlier call's
// partials (it writes zeros).  An lse of NaN marks a row that sees a block out
// of range (zeros), one of +inf a row with a score of NaN or +inf (NaN).
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
// Weights are scaled by 2^kShift.  A row keeps its reference while the sum of
// a step's weights stays below kSumLimit, so that each is inside fp16's range;
// what the large limit costs are weights 2^-27 below the reference's, which
// fp16's range cuts off.
constexpr float kShift = 2.f;
constexpr float kSumLimit = 32768.f;
constexpr float kLn2 = 0.69314718055994531f;
constexpr unsigned kInvalidLse = 0x7fc00000u;  // NaN: a partial that must not be used
constexpr int kStep = 64;       // keys of a step of a stream
// What the start of a segment costs (5 us), in units: 1.4 us each where two of
// them are a dual segment's tile, else 2 to 2.5 us.  (Not weighed for the
// prefix, 32 sequences behind 16 keys took 47 us: one CTA had five of the eight
// heads' segments.)
constexpr int kStart = 4;
constexpr int kScaleSlots = 8;  // tiles whose row scales are kept: more than are in flight
// int8 rows: a V scale counts as one between 2^-kScaleLog and 2^kScaleLog in a
// row's reference.  Below, its products are nothing beside an fp16 output's
// smallest step; above, an output is beyond fp16.  Two references whose weights
// are within 2^30 of each other then differ by at most 2^126, and with the
// weights up to kMaxWeight all sums stay inside fp32.
constexpr int kScaleLog = 48;
constexpr float kMaxWeight = 1.2676506e30f;  // 2^100

constexpr int kSegSlots = 4;

enum : int {
  BAR_KFULL = 0,   // [3]
  BAR_KEMPTY = 3,  // [3]
  BAR_VFULL = 6,   // [3]
  BAR_VEMPTY = 9,  // [3]
  BAR_SFULL = 12,  // [stream][buffer] S of a step in TMEM
  BAR_PFULL = 16,  // [stream][buffer] P of a step in TMEM
  BAR_OFULL = 20,  // [stream] PV of all of a segment's steps but the last accumulated
  BAR_QFULL = 22,  // a segment's Q staged, the previous one's O read
  BAR_SEG = 23,    // every MMA of a segment finished
  BAR_DONE = 24,
  BAR_GFULL = 25,  // [kSegSlots] a segment's description published
  BAR_GEMPTY = 29, // [kSegSlots] ... read by every role
  BAR_OEMPTY = 33, // a segment's O accumulators read
  BAR_COUNT = 34
};

template <int KV>
struct Cfg {
  static constexpr bool kQuant = KV != kKvFp16;
  static constexpr bool kQ8 = KV == kKvQ8_0, kRow = KV == kKvInt8Row;
  static constexpr bool kDualOk = !kQ8;  // q8_0 operands are two tiles each
  static constexpr int kProdWarp = 8;                      // fp16: producer; int8: converters
  static constexpr int kMmaWarp = kProdWarp + (kQuant ? 8 : 1);  // [2], then the segments' warp
  static constexpr int kReaders = kMmaWarp + 2;            // warps that follow the segments
  static constexpr int kThreads = kQuant ? 640 : 384;
  static constexpr uint32_t kSlot = (kQ8 ? 2 : 1) * kTileBytes;  // q8_0: the high tile, the residual
  static constexpr int KS = kQ8 ? 1 : kRow ? 2 : 3;
  static constexpr int VS = 2;
  static constexpr uint32_t kQ = 0;
  static constexpr uint32_t kK = kQ + (kDualOk ? 2 : 1) * kTileBytes;
  static constexpr uint32_t kV = kK + KS * kSlot;
  static constexpr uint32_t kBars = kV + VS * kSlot;
  static constexpr uint32_t kMisc = kBars + (BAR_COUNT * 8 + 15) / 16 * 16;         // int [16], see below
  static constexpr uint32_t kSegs = kMisc + 64;             // Segment [kSegSlots]
  static constexpr uint32_t kScales = kSegs + kSegSlots * 64;  // int8 rows: float K [8][128], V, log2 |V|
  static constexpr uint32_t kTotal = kScales + (kRow ? kScaleSlots * 3 * 128 * 4 : 0);
  static_assert(kBars % 16 == 0 && kSegs % 16 == 0 && kScales % 16 == 0, "alignment");
  static_assert(kTotal + 1024 <= 232448, "shared memory per CTA");
};

__device__ __forceinline__ uint32_t h2_bits(__half2 h) { return *reinterpret_cast<const uint32_t*>(&h); }
__device__ __forceinline__ void sts_v4(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}

__device__ __forceinline__ uint4 lds_v4(uint32_t addr) {
  uint4 r;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "r"(addr)
               : "memory");
  return r;
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

// x - h for two fp16 values (exact).
__device__ __forceinline__ float2 residual(float2 x, uint32_t h) {
  float2 d;
  asm("{\n\t.reg .b16 a, b, m;\n\tmov.b32 {a, b}, %2;\n\tmov.b16 m, 0xBC00;\n\t"  // -1
      "fma.rn.f32.f16 %0, a, m, %3;\n\tfma.rn.f32.f16 %1, b, m, %4;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "r"(h), "f"(x.x), "f"(x.y));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
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

// a / b for a >= 0, b > 0, mostly in 32 bits.
__device__ __forceinline__ long long div_pos(long long a, long long b) {
  return (a | b) >> 32 == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
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
// kDual: more than 128 rows; kFirst, kLast: of the group's segments; kBuf: Q in the second buffer
enum : int { kDual = 1, kFirst = 2, kLast = 4, kBuf = 8 };

template <int KV>
__global__ void __launch_bounds__(Cfg<KV>::kThreads, 1)
    shared_tc_kernel(const __grid_constant__ CUtensorMap tmap_k,
                     const __grid_constant__ CUtensorMap tmap_v, const SharedParams p) {
  using C = Cfg<KV>;
  constexpr bool kQuant = C::kQuant, kQ8 = C::kQ8, kRow = C::kRow, kDualOk = C::kDualOk;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  const uint32_t sQ = sbase + C::kQ, sK = sbase + C::kK, sV = sbase + C::kV;
  // [0] TMEM base, [1] abort, [2] shortest sequence, [3] start sequence,
  // [4, 5] its start, [6, 7] own tiles and sequences behind the first round, [9] a block was out of
  // range
  int* misc = reinterpret_cast<int*>(smem + C::kMisc);
  volatile int* abort = misc + 1;
  const unsigned long long wl = p.wait_limit_ns;
  auto bar = [&](int i) { return sbase + C::kBars + 8u * i; };
  auto wait = [&](int b, int parity) { return mbar_wait(bar(b), (uint32_t)parity & 1u, abort, wl); };
  // For the segments' descriptions the limit is kept to the nanosecond, so that a
  // short one is sure to be met whatever the cache type (for every wait it cost
  // 1 to 4%: int8 rows 91.5 us against 88.5).
  auto seg_wait = [&](int b, int parity) { return mbar_wait_strict(bar(b), (uint32_t)parity & 1u, abort, wl); };
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const float cs = fabsf(p.scale_log2);

  if (threadIdx.x == 0) {
    for (int i = 0; i < BAR_COUNT; ++i)
      mbar_init(bar(i), i == BAR_QFULL || i == BAR_OEMPTY                                ? 8
                        : (i >= BAR_PFULL && i < BAR_OFULL)                              ? 4
                        : (i < BAR_SFULL && (i % 6 >= 3 || kQuant)) ? (i % 6 >= 3 ? 2 : 4)  // empty, full
                        : i == BAR_SEG || i == BAR_DONE                                  ? 2
                        : i >= BAR_GEMPTY                                                ? C::kReaders
                                                                                         : 1);
    misc[1] = 0;
    misc[2] = INT32_MAX;
    misc[9] = 0;
    misc[3] = p.num_seqs;
    *reinterpret_cast<unsigned long long*>(misc + 6) = 0;
    fence_mbar_init();
  }
  if (warp == C::kMmaWarp) tmem_alloc(smem_u32(misc), 512);
  if constexpr (!kQuant) {
    if (threadIdx.x == 32 * C::kProdWarp) {
      prefetch_tmap(&tmap_k);
      prefetch_tmap(&tmap_v);
    }
  }
  griddep_wait();
  griddep_launch_dependents();
  const int P = __ldg(p.prefix_len);
  const int own_s = threadIdx.x;  // this thread's sequence of the first round
  const int own_L = own_s < p.num_seqs ? __ldg(p.context_lens + own_s) : 0;
  const bool prefix_ok = shared_prefix_ok(p, P);
  __syncthreads();

  // ---- the work cut ---------------------------------------------------------
  // A unit is the product of 128 rows and 128 keys.  A group: `start` units for
  // the start of a segment, then its tiles, of two units in a dual group of the
  // prefix, else of one.  CTA c has the tiles that begin in units
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
  auto own_tiles = [&](int L) -> int {
    int lo, hi;
    own_keys(L, lo, hi);
    return key_tiles(lo, hi);
  };
  // Of the batch: the shortest sequence, the sequences with keys of their own,
  // their tiles; tiles before this thread's sequence among the first round's.
  long long* sums = reinterpret_cast<long long*>(smem + C::kK);  // [2][warps], no copy is in flight yet
  const int own_t = own_tiles(own_L);
  long long ahead = ((long long)own_t << 22) + (own_t > 0);  // tiles, sequences
  {
    int m = prefix_ok && shared_seq_ok(p, own_L, P) && own_s < p.num_seqs ? own_L : INT32_MAX;
    const long long mine = ahead;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, ahead, o);
      if (lane >= o) ahead += y;
    }
    if (lane == 31) sums[warp] = ahead;
    ahead -= mine;
    long long more = 0;
    for (int s = own_s + C::kThreads; s < p.num_seqs; s += C::kThreads) {
      const int L = __ldg(p.context_lens + s);
      if (prefix_ok && shared_seq_ok(p, L, P)) m = min(m, L);
      const int t = own_tiles(L);
      more += ((long long)t << 22) + (t > 0);
    }
    m = __reduce_min_sync(0xffffffffu, m);
    if (lane == 0 && m != INT32_MAX) atomicMin(misc + 2, m);
    if (p.num_seqs > C::kThreads && more != 0)
      atomicAdd(reinterpret_cast<unsigned long long*>(misc + 6), (unsigned long long)more);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc[0];
  long long both = *reinterpret_cast<long long*>(misc + 6);
#pragma unroll
  for (int x = 0; x < C::kThreads / 32; ++x) {
    const long long y = sums[x];
    if (x < warp) ahead += y;
    both += y;
  }
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
  const long long tiles_p = (long long)p.num_kv_heads * uh * nt;
  // A call with a tile for every CTA at most: none gets two.
  const int start = tiles_p + (both >> 22) * hp <= p.ctas ? 0 : u1 == 2 && !kQuant ? kStart : kStart / 2;
  const long long Wp = nt > 0 ? tiles_p + (long long)p.num_kv_heads * NT * start : 0;
  auto own_units = [&](long long tiles_and_seqs) {
    return hp * ((tiles_and_seqs >> 22) + start * (tiles_and_seqs & 0x3fffff));
  };
  const long long W = Wp + own_units(both);
  // a range holds the beginning of a tile at least: no CTA between two
  // segments of a group is without one
  const int Ce = (int)min(max(u1 == 2 ? W >> 1 : W, 1LL), (long long)p.ctas);
  const int cta = blockIdx.x;
  long long a = 0, b = 0;
  if (cta < Ce) {
    a = div_pos(cta * W, Ce);
    b = div_pos((cta + 1) * W, Ce);
  }
  if (cta == 0 && threadIdx.x == 0) p.meta[0] = nt;  // for the join
  // The sequence in which this CTA's range begins, where it begins behind the
  // prefix.
  if (threadIdx.x == 0 && a <= Wp) {
    misc[3] = 0;
    *reinterpret_cast<long long*>(misc + 4) = Wp;
  }
  if (a > Wp) {
    const long long at = Wp + own_units(ahead), u = own_units(((long long)own_t << 22) + (own_t > 0));
    if (at <= a && a < at + u) {
      misc[3] = own_s;
      *reinterpret_cast<long long*>(misc + 4) = at;
    }
    if (p.num_seqs > C::kThreads && warp == 0) {  // the further rounds, 32 sequences at a time
      long long run = 0;
      for (int x = 0; x < C::kThreads / 32; ++x) run += sums[x];
      for (int s0 = C::kThreads; s0 < p.num_seqs && Wp + own_units(run) <= a; s0 += 32) {
        const int s = s0 + lane, t = s < p.num_seqs ? own_tiles(__ldg(p.context_lens + s)) : 0;
        const long long mine = ((long long)t << 22) + (t > 0);
        long long x = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const long long y = __shfl_up_sync(0xffffffffu, x, o);
          if (lane >= o) x += y;
        }
        const long long first = Wp + own_units(run + x - mine);
        if (first <= a && a < first + own_units(mine)) {
          misc[3] = s;
          *reinterpret_cast<long long*>(misc + 4) = first;
        }
        run += __shfl_sync(0xffffffffu, x, 31);
      }
    }
  }
  fence_proxy_async_smem();  // the sums lie where copies will land
  __syncthreads();

  Segment* segs = reinterpret_cast<Segment*>(smem + C::kSegs);
  // Calls f(segment) for every segment of this CTA.
  auto segments = [&](auto&& f) {
    for (int i = 0;; ++i) {
      if (!__all_sync(0xffffffffu, seg_wait(BAR_GFULL + i % kSegSlots, i / kSegSlots))) break;
      const Segment& g = segs[i % kSegSlots];
      if (__reduce_max_sync(0xffffffffu, g.n) == 0) break;
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
      const bool isk = warp < C::kProdWarp + 4;  // four warps for K, four for V
      const int cw = warp % 4, kq = lane / 8, cl = lane % 8;
      const int NS = isk ? C::KS : C::VS;
      const uint32_t ring = isk ? sK : sV;
      const int full = isk ? BAR_KFULL : BAR_VFULL, empty = isk ? BAR_KEMPTY : BAR_VEMPTY;
      const uint8_t* cache = static_cast<const uint8_t*>(isk ? p.k : p.v);
      const long long tile_bytes = quant_tile_bytes(KV, p.block_size);
      float* scales = reinterpret_cast<float*>(smem + C::kScales);  // K [8][128], V, log2 |V|
      int T = 0, st = 0, ph = 0;
      bool ok = true;
      segments([&](const Segment& g) {
        const int base = g.base, t0 = g.t0, te = g.t0 + g.n, vlo = g.lo, vhi = g.hi;
        const int32_t* table = g.table;
        uint4 q[8];                    // 32 keys' values
        uint16_t d8[kQ8 ? 8 : 1];      // q8_0: the scales of this lane's 16 values
        float d1 = 0.f;                // int8 rows: the scale of key `lane`
        // The block of this warp's two chunks of tile t (lanes 0, 1).
        auto lookup = [&](int t) -> int {
          const int key0 = base + t * kTileKeys + (2 * cw + lane) * kChunk;
          int phys = lane < 2 && t < te && key0 <= vhi ? __ldg(table + key0 / p.block_size) : 0;
          if (phys < 0 || phys >= p.num_blocks) {
            misc[9] = 1;
            atomicOr(p.flags, kFlagBadBlock);
            phys = -1;  // zeros are read: the rows that see it are marked, the others unharmed
          }
          return phys;
        };
        auto fetch = [&](int t, int phys) {
          d1 = 0.f;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int key0 = base + t * kTileKeys + (2 * cw + h) * kChunk;
            const long long b = __shfl_sync(0xffffffffu, phys, h);
            const bool on = t < te && key0 <= vhi && b >= 0;
            const uint8_t* tile = cache + (b * p.num_kv_heads + g.kvh) * tile_bytes;
            const int slot = key0 % p.block_size;
            const uint8_t* at = tile + (slot + kq) * kHeadDim + cl * 16;
            const uint8_t* sc = tile + p.block_size * kHeadDim + (slot + kq) * 8 + cl / 2 * 2;
#pragma unroll
            for (int i = 4 * h; i < 4 * h + 4; ++i) {
              q[i] = make_uint4(0, 0, 0, 0);
              if constexpr (kQ8) d8[i] = 0;
              if (on) {
                q[i] = __ldg(reinterpret_cast<const uint4*>(at + i % 4 * 4 * kHeadDim));
                if constexpr (kQ8) d8[i] = __ldg(reinterpret_cast<const unsigned short*>(sc + i % 4 * 32));
              }
            }
            if constexpr (kRow) {
              if (on && lane / kChunk == h)
                d1 = __ldg(reinterpret_cast<const float*>(tile + p.block_size * kHeadDim) + slot +
                           lane % kChunk);
            }
          }
        };
        fetch(t0, lookup(t0));
        int phys = lookup(t0 + 1);
        const bool sw = cl >= 4;
        const uint32_t row0 = 4 * cw * kGroupBytes + kq * 128 + (cl / 4) * kAtomBytes;
        for (int t = t0; t < te && ok; ++t, ++T) {
          const int kw = base + t * kTileKeys + 32 * cw, ss = T % kScaleSlots;
          ok = __all_sync(0xffffffffu, wait(empty + st, ph ^ 1));
          if (!ok) break;
          if constexpr (kRow) {
            if (isk) {
              scales[ss * 128 + 32 * cw + lane] = d1 * cs;
            } else {  // scales of hidden keys may be anything
              const float d = kw + lane >= vlo && kw + lane <= vhi ? d1 : 0.f;
              const int ex = (int)(__float_as_uint(fabsf(d)) >> 23) - 126;  // |d| < 2^ex
              scales[(kScaleSlots + ss) * 128 + 32 * cw + lane] = d;
              scales[(2 * kScaleSlots + ss) * 128 + 32 * cw + lane] =
                  (float)min(max(ex, -kScaleLog), kScaleLog);
            }
          }
          const bool inside = isk || (kw >= vlo && kw + 31 <= vhi);
          const uint32_t dst = ring + st * C::kSlot + row0;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            // Row 32 cw + 4 i + kq.  Lanes 4-7 of a key write their second half
            // first: the eight lanes of a store then cover all banks.
            const int r8 = 4 * (i & 1) + kq;
            const uint32_t at = dst + (i / 2) * kGroupBytes + (i & 1) * 512;
            const uint32_t a0 = at + (((2 * cl + sw) % 8) ^ r8) * 16, a1 = at + (((2 * cl + 1 - sw) % 8) ^ r8) * 16;
            const uint32_t wd[4] = {sw ? q[i].z : q[i].x, sw ? q[i].w : q[i].y, sw ? q[i].x : q[i].z,
                                    sw ? q[i].y : q[i].w};
            __half2 y[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) q8_to_half4(wd[e], y[2 * e], y[2 * e + 1]);
            auto put = [&](const __half2 (&h)[8], uint32_t off) {
              sts_v4(a0 + off, make_uint4(h2_bits(h[0]), h2_bits(h[1]), h2_bits(h[2]), h2_bits(h[3])));
              sts_v4(a1 + off, make_uint4(h2_bits(h[4]), h2_bits(h[5]), h2_bits(h[6]), h2_bits(h[7])));
            };
            if constexpr (kQ8) {
              __half d = __ushort_as_half(d8[i]);
              if (!inside) {  // hidden keys' scales may be anything
                const int key = kw + 4 * i + kq;
                if (key < vlo || key > vhi) d = __ushort_as_half(0);
              }
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
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(full + st));
          fetch(t + 1, phys);
          phys = lookup(t + 2);
          if (++st == NS) {
            st = 0;
            ph ^= 1;
          }
        }
      });
    }
  } else if (warp == C::kProdWarp) {
    // ===================== K and V producer =================================
    int TK = 0, TV = 0;  // tiles issued
    bool ok = true;
    segments([&](const Segment& g) {
      const int base = g.base, t0 = g.t0, n = g.n, vhi = g.hi;
      // Lane's chunk of tile t: its TMA row coordinate (-1: none).
      auto row8_of = [&](int t, bool& bad) -> int {
        const int key0 = base + t * kTileKeys + lane * kChunk;
        if (lane >= kChunksPerTile || key0 > vhi) return -1;
        const int phys = __ldg(g.table + key0 / p.block_size);
        bad = phys < 0 || phys >= p.num_blocks;
        // Rows behind the cache, which are read as zeros: the rows that see the
        // block are marked, the others unharmed by what some other block holds.
        if (bad) return (int)((long long)p.num_blocks * p.num_kv_heads * p.block_size / 8);
        return (int)((((long long)phys * p.num_kv_heads + g.kvh) * p.block_size + key0 % p.block_size) / 8);
      };
      auto issue = [&](bool isk, int T, int row8) {
        const int st = isk ? T % C::KS : T % C::VS, full = (isk ? BAR_KFULL : BAR_VFULL) + st;
        const uint32_t mask = __ballot_sync(0xffffffffu, row8 >= 0);
        if (lane == 0) mbar_arrive_expect_tx(bar(full), __popc(mask) * kChunkBytes);
        __syncwarp();
        if (row8 >= 0)
          tma_load_4d((isk ? sK : sV) + st * C::kSlot + lane * kChunkBytes, isk ? &tmap_k : &tmap_v, 0, 0,
                      0, row8, bar(full));
        __syncwarp();
      };
      int jk = 0, jv = 0;  // tiles of the segment issued
      bool badk = false, badv = false;
      int rk = row8_of(t0, badk), rv = rk;  // of tiles jk, jv
      while (ok && jv < n) {
        // Whichever slot is free; K leads.
        bool k = false, v = false;
        unsigned long long since = 0;
        for (;;) {
          k = jk < n && mbar_test_wait(bar(BAR_KEMPTY + TK % C::KS), ((TK / C::KS) & 1) ^ 1);
          v = jv < jk && mbar_test_wait(bar(BAR_VEMPTY + TV % C::VS), ((TV / C::VS) & 1) ^ 1);
          k = __any_sync(0xffffffffu, k);
          v = __any_sync(0xffffffffu, v);
          if (k || v) break;
          const unsigned long long now = globaltimer();
          if (since == 0) since = now;
          if (now - since > wl) *abort = 1;
          if (__any_sync(0xffffffffu, *abort != 0)) break;
          __nanosleep(64);
        }
        ok = k || v;
        if (k) {
          if (badk) {
            misc[9] = 1;
            atomicOr(p.flags, kFlagBadBlock);
          }
          issue(true, TK++, rk);
          badk = false;
          if (++jk < n) rk = row8_of(t0 + jk, badk);
        }
        if (v) {
          issue(false, TV++, rv);
          if (++jv < n) rv = row8_of(t0 + jv, badv);
        }
      }
    });
    // No copy outlives the CTA: the last of every slot (landed already unless
    // a wait gave up).
    if (lane == 0) {
      volatile int no_abort = 0;
      for (int u = max(0, TK - C::KS); u < TK; ++u)
        mbar_wait(bar(BAR_KFULL + u % C::KS), (u / C::KS) & 1, &no_abort);
      for (int u = max(0, TV - C::VS); u < TV; ++u)
        mbar_wait(bar(BAR_VFULL + u % C::VS), (u / C::VS) & 1, &no_abort);
    }
  }
  if (warp == C::kMmaWarp || warp == C::kMmaWarp + 1) {
    // ===================== MMA issuers ======================================
    const int w = warp - C::kMmaWarp;  // the stream
    const uint32_t id_qk = idesc_f16_f32(128, kStep, false, false);
    const uint32_t id_pv = idesc_f16_f32(128, 128, false, true);
    const uint64_t dQ = smem_desc(sQ, 16, kGroupBytes, kSwizzle128B);
    const uint64_t dK = smem_desc(sK, 16, kGroupBytes, kSwizzle128B);
    const uint64_t dV = smem_desc(sV, kAtomBytes, kGroupBytes, kSwizzle128B);
    constexpr uint32_t kHalfTile = kTileBytes / 2;   // 64 keys
    // The whole warp runs this code and one elected lane issues: what the
    // products take stays in uniform registers (a lane on its own spends 126
    // cycles a product on moving operands there).
    const uint32_t lead = elect_one();
    const uint32_t tm = __reduce_max_sync(0xffffffffu, tmem), ob = tm + 256 + w * 128;
    auto wait1 = [&](int b, int parity) { return __all_sync(0xffffffffu, wait(b, parity)) != 0; };
    int ks = 0, kp = 0, vs = 0, vp = 0;  // ring slots and their phases
    int c = 0, seg = 0;                  // steps and segments before
    bool ok = true;
    segments([&](const Segment& g) {
      if (!ok) return;
      const int gn = __reduce_max_sync(0xffffffffu, g.n);
      const int flags = __reduce_max_sync(0xffffffffu, g.flags);
      const bool dual = kDualOk && (flags & kDual);
      const int Y = dual ? 2 * gn : gn;  // steps of the stream
      const uint64_t q = dQ + ((dual ? w : (flags & kBuf) ? 1 : 0) * kTileBytes >> 4);
      ok = wait1(BAR_QFULL, seg);
      if (!ok) return;
      // S of step y (its buffer (c + y) & 1), products of K's high parts, then
      // q8_0's residuals.
      auto scores = [&](int y) {
        const int half = dual ? y & 1 : w;
        if (!dual || half == 0) {
          ok = wait1(BAR_KFULL + ks, kp);
          if (!ok) return;
          tc_fence_after();
        }
        const uint32_t sb = tm + w * 128 + ((c + y) & 1) * kStep;
        const uint64_t kd = dK + ((uint64_t)(ks * C::kSlot + half * kHalfTile) >> 4);
#pragma unroll
        for (int i = 0; i < (kQ8 ? 16 : 8); ++i) {
          const uint64_t o = ((i % 8 / 4) * kAtomBytes + (i % 4) * 32) >> 4;
          tc_mma_f16_ss(lead, sb, q + o, kd + ((i / 8 * kTileBytes) >> 4) + o, id_qk, i > 0);
        }
        tc_commit(lead, bar(BAR_SFULL + w * 2 + ((c + y) & 1)));
        if (!dual || half == 1) {
          tc_commit(lead, bar(BAR_KEMPTY + ks));
          if (++ks == C::KS) {
            ks = 0;
            kp ^= 1;
          }
        }
      };
      scores(0);
      if (ok && Y > 1) scores(1);
      for (int y = 0; y < Y && ok; ++y) {
        const int half = dual ? y & 1 : w, buf = (c + y) & 1;
        ok = ((dual && half == 1) || wait1(BAR_VFULL + vs, vp)) &&  // (there before P as a rule)
             (y > 0 || seg == 0 || wait1(BAR_OEMPTY, seg - 1)) &&
             wait1(BAR_PFULL + w * 2 + buf, (c + y) >> 1);
        if (!ok) break;
        tc_fence_after();
        const uint32_t pb = tm + w * 128 + buf * kStep;
        const uint64_t vd = dV + ((uint64_t)(vs * C::kSlot + half * kHalfTile) >> 4);
        // P_hi V, P_lo V and, q8_0, P_hi V_lo
#pragma unroll
        for (int i = 0; i < (kQ8 ? 12 : 8); ++i) {
          const int part = i / 4, k = i % 4;
          tc_mma_f16_ts(lead, ob, pb + (k / 2) * 32 + (part == 1) * 16 + (k % 2) * 8,
                        vd + ((k * 2 * kGroupBytes + (part == 2) * kTileBytes) >> 4), id_pv,
                        y > 0 || i > 0);
        }
        const int slot = vs;
        if (!dual || half == 1) {
          if (kQuant) tc_commit(lead, bar(BAR_VEMPTY + slot));  // (K may have to be waited for)
          if (++vs == C::VS) {
            vs = 0;
            vp ^= 1;
          }
        }
        if (y + 2 < Y) scores(y + 2);
        if (!kQuant && (!dual || half == 1)) tc_commit(lead, bar(BAR_VEMPTY + slot));
        if (y == Y - 2) tc_commit(lead, bar(BAR_OFULL + w));
      }
      if (ok) {
        if (Y == 1) tc_commit(lead, bar(BAR_OFULL + w));
        tc_commit(lead, bar(BAR_SEG));
      }
      c += Y;
      ++seg;
    });
    if (lead) {
      tc_commit(bar(BAR_DONE));
      volatile int no_abort = 0;
      mbar_wait(bar(BAR_DONE), 0, &no_abort);
    }
    __syncwarp();
  } else if (warp == C::kMmaWarp + 2) {
    // ===================== segments =========================================
    if (lane == 0) {
      int count = 0, buf = kBuf;
      bool ok = true;
      auto publish = [&](const Segment& g) {
        const int st = count % kSegSlots;
        if (ok) {  // (the slot's segment may last as long as its tiles may wait)
          const unsigned long long n = count < kSegSlots ? 0 : segs[st].n;
          ok = mbar_wait_strict(bar(BAR_GEMPTY + st), (count / kSegSlots & 1) ^ 1, abort,
                                wl >> 40 ? wl : wl * (1 + n));
        }
        if (ok) {
          segs[st] = g;
          // Q of a single segment: the two buffers in turn (q8_0 has one).
          buf = !kDualOk || (g.flags & kDual) ? 0 : buf ^ kBuf;
          segs[st].flags |= buf;
          mbar_arrive(bar(BAR_GFULL + st));
          ++count;
        }
        // For the join, whether or not this CTA comes to it.
        if (g.flags & kFirst) p.meta[2 + 2 * g.group] = cta;
        if (g.flags & kLast) p.meta[3 + 2 * g.group] = cta;
      };
      long long x = a;
      while (x < b && x < Wp) {
        Segment g;
        const long long head = (long long)uh * nt + NT * start, tile = (long long)u1 * nt + start;
        g.kvh = (int)div_pos(x, head);
        const int i = (int)div_pos(x - g.kvh * head, tile);
        const long long st = g.kvh * head + i * tile + start;  // unit of the first tile
        g.row0 = i * p.row_tile;
        g.nrows = min(R - g.row0, p.row_tile);
        const int u = g.nrows > 128 ? 2 : 1, u_log = u - 1;
        g.t0 = (int)max(0LL, (x - st + u - 1) >> u_log);
        const int te = (int)min((long long)nt, (b - st + u - 1) >> u_log);
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
        x = st + (long long)u * nt;
      }
      long long at = *reinterpret_cast<volatile long long*>(misc + 4);  // where sequence s begins
      for (int s = misc[3]; x < b && s < p.num_seqs; ++s) {
        Segment g;
        own_keys(__ldg(p.context_lens + s), g.lo, g.hi);
        const int tiles = key_tiles(g.lo, g.hi), len = tiles + start;
        if (tiles == 0) continue;
        g.table = p.block_table + (long long)s * p.max_blocks_per_seq;
        g.base = g.lo / kChunk * kChunk;
        g.clo = P;
        g.chi = INT32_MAX;
        for (int j = (int)div_pos(x - at, len); j < hp && x < b; ++j) {
          const long long st = at + (long long)j * len + start;  // unit of the first tile
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
  } else if (warp < C::kProdWarp) {
    // ===================== softmax warpgroups ===============================
    const int w = warp / 4, r = threadIdx.x % 128;
    constexpr int kSoftThreads = 256;
    constexpr bool kHold = !kQuant;  // a step's scores stay in registers
    const uint32_t lane_off = (uint32_t)(warp % 4 * 32) << 16;
    const uint32_t tO = tmem + lane_off + 256;
    const uint32_t flip = p.scale_log2 < 0.f ? 0x80008000u : 0u;  // a negative scale negates Q
    int T0 = 0, c0 = 0, seg = 0;  // tiles, steps and segments before
    bool ok = true;
    // Stages this warpgroup's share of a segment's Q rows.
    auto stage_q = [&](const Segment& g) {
      const bool dual = kDualOk && (g.flags & kDual);
      const int local = (dual ? w * 128 : 0) + r, row = g.row0 + local;
      const bool in = local < g.nrows;
      const __half* src = p.q + ((long long)(in ? row / p.group : 0) * p.num_q_heads + g.kvh * p.group +
                                 (in ? row % p.group : 0)) * kHeadDim;
      const uint32_t dst = sQ + ((dual ? w : (g.flags & kBuf) ? 1 : 0) * kTileBytes) +
                           (r / 8) * kGroupBytes + (r % 8) * 128;
      const int c_lo = dual ? 0 : w * 8, c_hi = dual ? 16 : w * 8 + 8;
#pragma unroll 1
      for (int c0 = c_lo; c0 < c_hi; c0 += 8) {
        uint4 v[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          v[c] = make_uint4(0, 0, 0, 0);
          if (in) v[c] = __ldg(reinterpret_cast<const uint4*>(src) + c0 + c);
        }
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          v[c].x ^= flip; v[c].y ^= flip; v[c].z ^= flip; v[c].w ^= flip;
          sts_v4(dst + (c0 / 8) * kAtomBytes + ((c ^ (r % 8)) * 16), in ? v[c] : make_uint4(0, 0, 0, 0));
        }
      }
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(BAR_QFULL));
    };
    // Whether there is a segment is voted on, so that all softmax warps come to
    // the named barriers below or none does.
    bool got = named_bar_and(2, kSoftThreads, seg_wait(BAR_GFULL, 0));
    got = got && segs[0].n != 0;
    if (got) stage_q(segs[0]);
    while (got) {
      const Segment& g = segs[seg % kSegSlots];
      const bool dual = kDualOk && (g.flags & kDual);
      const int local = (dual ? w * 128 : 0) + r, row = g.row0 + local;
      const bool mine = local < g.nrows;
      const int tok = row / p.group;  // of all sequences' new tokens
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
      float bias = 0.f;              // kShift - m, 0 before the first key
      bool fresh = true;             // int8: some row of the warp is before its first key
      const int Y = dual ? 2 * g.n : g.n;
      // Steps from key wlo to whi need no mask in this warp.
      const int wlo = __reduce_max_sync(0xffffffffu, mine ? max(lo, g.lo) : g.lo);
      const int whi = __reduce_min_sync(0xffffffffu, mine ? min(hi, g.hi) : g.hi);
      const int glo = g.lo, ghi = g.hi, key0 = g.base + g.t0 * kTileKeys;
      // S of step y: awaited and (its first or second 32 columns) loaded.
      float va[32], vb[kHold ? 32 : 1];
      auto s_wait = [&](int y) -> bool {
        const int c = c0 + y;
        const bool got = __all_sync(0xffffffffu, wait(BAR_SFULL + w * 2 + (c & 1), c >> 1));
        tc_fence_after();
        return got;
      };
      auto s_load = [&](int y, int x, float (&v)[32]) {
        if (warp_rows) tmem_ld32(tmem + lane_off + w * 128 + ((c0 + y) & 1) * kStep + x * 32, v);
      };
      for (int y = 0; y < Y && ok; ++y) {
        const int T = T0 + (dual ? y >> 1 : y), half = dual ? y & 1 : w, c = c0 + y;
        const int kb = key0 + (T - T0) * kTileKeys + half * kStep;  // the step's first key
        const uint32_t tS = tmem + lane_off + w * 128 + (c & 1) * kStep;
        ok = s_wait(y);
        if (!ok) break;
        s_load(y, 0, va);
        if constexpr (kHold) s_load(y, 1, vb);
        // Keys that no row sees must not reach PV: their V rows become 0 (in a
        // dual segment by both streams, each before its own PV; the converters
        // see to that themselves).
        const bool whole = kb >= wlo && kb + kStep - 1 <= whi;  // no row of the warp needs a mask
        if (!kQuant && !whole && (kb < glo || kb + kStep - 1 > ghi)) {
          const int st = T % C::VS, key = r % kStep;
          ok = __all_sync(0xffffffffu, wait(BAR_VFULL + st, T / C::VS));
          if (ok && (kb + key < glo || kb + key > ghi)) {
            const int vr = half * kStep + key;
            const uint32_t v = sV + st * C::kSlot + (vr / 8) * kGroupBytes + (r / kStep) * kAtomBytes +
                               (vr % 8) * 128;
#pragma unroll
            for (int x = 0; x < 8; ++x) sts_v4(v + x * 16, make_uint4(0, 0, 0, 0));
          }
          fence_proxy_async_smem();
        }
        if (warp_rows) {
          // int8 rows: the tile's scales of K (times the softmax scale), V, log2 |V|.
          const float4* ks = reinterpret_cast<const float4*>(smem + C::kScales) + T % kScaleSlots * 32 +
                             half * (kStep / 4);
          const float4* vs = ks + kScaleSlots * 32;
          const float4* vlog = vs + kScaleSlots * 32;
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
          if constexpr (kRow) {  // the V scales are there
            const int st = T % C::VS;
            ok = __all_sync(0xffffffffu, wait(BAR_VFULL + st, T / C::VS));
            if (!ok) break;
          }
          auto scaled = [&](float (&v)[32], int c) {
            if constexpr (kRow) {
#pragma unroll
              for (int e = 0; e < 32; e += 4) {
                const float4 k = ks[c * 8 + e / 4];
                const float2 a = mul2(make_float2(v[e], v[e + 1]), make_float2(k.x, k.y));
                const float2 b = mul2(make_float2(v[e + 2], v[e + 3]), make_float2(k.z, k.w));
                v[e] = a.x; v[e + 1] = a.y; v[e + 2] = b.x; v[e + 3] = b.y;
              }
            }
            mask(v, c);
          };
          // Scores to weights, in place; their sum.
          float2 sum, sum2;
          auto weights = [&](float (&v)[32]) {
            const float k = cs;
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              const float2 z = fma2(make_float2(v[e], v[e + 1]), make_float2(k, k), make_float2(bias, bias));
              v[e] = fast_exp2(z.x);
              v[e + 1] = fast_exp2(z.y);
              float2& to = e & 2 ? sum2 : sum;
              to = add2(to, make_float2(v[e], v[e + 1]));
            }
          };
          // Moves the reference of the rows that `need` it up to `top`, and what
          // the stream has accumulated for them.
          auto move = [&](bool need, float top) -> bool {
            const float mn = need ? fmaxf(m, top) : m;
            const bool moved = mn != m;
            const float f = moved ? fast_exp2(m - mn) : 1.f;
            m = mn;
            bias = m == -INFINITY ? 0.f : kShift - m;
            l *= f;
            if (y > 0 && __any_sync(0xffffffffu, moved)) {
              // rescale what this stream has accumulated, once the last step's
              // PV is done (S of the next step is committed behind it)
              ok = y + 1 < Y ? s_wait(y + 1) : __all_sync(0xffffffffu, wait(BAR_OFULL + w, seg)) != 0;
              if (!ok) return false;
              tc_fence_after();
#pragma unroll 1
              for (int x = 0; x < 8; ++x) {
                float o[16];
                tmem_ld<16>(tO + w * 128 + x * 16, o);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] *= f;
                tmem_st<16>(tO + w * 128 + x * 16, o);
              }
              tmem_st_wait();
            }
            return true;
          };
          // Weights of 32 keys over their scores: 16 columns of high parts, 16
          // of residuals (exact: w - fp16(w) fits fp32).
          constexpr int kPack = kHold ? 16 : 8;  // words of each at a time
          uint32_t ph[kPack], pl[kPack];
          auto pack = [&](const float (&v)[32], int c, int z) {  // from key 2 z of the chunk on
#pragma unroll
            for (int i = 0; i < kPack; ++i) {
              const float2 x = make_float2(v[2 * (z + i)], v[2 * (z + i) + 1]);
              ph[i] = h2_bits(__floats2half2_rn(x.x, x.y));
              const float2 lo2 = residual(x, ph[i]);
              pl[i] = h2_bits(__floats2half2_rn(lo2.x, lo2.y));
            }
          };
          auto put = [&](int c, int z) {
            tmem_st(tS + c * 32 + z, ph);
            tmem_st(tS + c * 32 + 16 + z, pl);
          };
          if constexpr (!kHold) {
            // 32 columns at a time: the converters leave no registers for a
            // step's 64 scores.  As below, a row keeps its reference while its
            // sums stay below the limit: of the weights, or, int8 rows, of the
            // squares of what is rounded to fp16, so that the V scale of a key
            // with little weight costs the others nothing.
            auto top_of = [&](int x) -> float {  // the chunk's largest, read again
              tmem_ld32(tS + x * 32, va);
              tmem_ld_wait(va);
              scaled(va, x);
              float mx = -INFINITY;  // (scores of NaN are passed over)
#pragma unroll
              for (int e = 0; e < 32; e += 4) {
                if constexpr (kRow) {
                  const float4 g = vlog[x * 8 + e / 4];
                  va[e] += g.x; va[e + 1] += g.y; va[e + 2] += g.z; va[e + 3] += g.w;
                }
                mx = max3(mx, va[e], va[e + 1]);
                mx = max3(mx, va[e + 2], va[e + 3]);
              }
              return kRow ? mx : mx * cs;
            };
            auto chunk_weights = [&](int x, bool& fits) -> float {
              tmem_ld32(tS + x * 32, va);
              tmem_ld_wait(va);
#pragma unroll
              for (int e = 0; e < 32; e += 4) {
                float4 k = make_float4(cs, cs, cs, cs);
                if constexpr (kRow) k = ks[x * 8 + e / 4];
                const float2 a = fma2(make_float2(va[e], va[e + 1]), make_float2(k.x, k.y), make_float2(bias, bias));
                const float2 b = fma2(make_float2(va[e + 2], va[e + 3]), make_float2(k.z, k.w), make_float2(bias, bias));
                va[e] = a.x; va[e + 1] = a.y; va[e + 2] = b.x; va[e + 3] = b.y;
              }
              mask(va, x);
              float2 a = make_float2(0.f, 0.f), b = a, sq = a;
#pragma unroll
              for (int e = 0; e < 32; e += 4) {
#pragma unroll
                for (int i = 0; i < 4; ++i) va[e + i] = fast_exp2(va[e + i]);
                float2 u = make_float2(va[e], va[e + 1]), w = make_float2(va[e + 2], va[e + 3]);
                a = add2(a, u);
                b = add2(b, w);
                if constexpr (kRow) {
                  const float4 g = vs[x * 8 + e / 4];
                  u = mul2(u, make_float2(g.x, g.y));
                  w = mul2(w, make_float2(g.z, g.w));
                  sq = fma2(u, u, sq);
                  sq = fma2(w, w, sq);
                  va[e] = u.x; va[e + 1] = u.y; va[e + 2] = w.x; va[e + 3] = w.y;
                }
              }
              const float total = (a.x + a.y) + (b.x + b.y);
              fits = kRow ? sq.x + sq.y <= kSumLimit * kSumLimit && total <= kMaxWeight
                          : total <= kSumLimit;
              return total;
            };
            if (fresh) {  // rows at their first keys
              const float t0 = top_of(0), top = fmaxf(t0, top_of(1));
              if (!move(mine && m == -INFINITY, top)) break;
              fresh = __any_sync(0xffffffffu, mine && m == -INFINITY);
            }
            bool up = true;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              bool fits;
              float total = chunk_weights(x, fits);
              const bool need = mine && m != -INFINITY && !fits;
              if (__any_sync(0xffffffffu, need)) {
                const float before = m;
                up = move(need, top_of(x));
                if (x == 1 && up) {  // the first chunk's weights, stored already
                  tmem_st_wait();    // (the stores may still be under way)
                  tmem_ld32(tS, va);
                  tmem_ld_wait(va);
                  const float f = fast_exp2(before - m);
#pragma unroll
                  for (int i = 0; i < 16; ++i) {
                    const uint32_t h = __float_as_uint(va[i]), r = __float_as_uint(va[16 + i]);
                    const float2 hf = __half22float2(*reinterpret_cast<const __half2*>(&h));
                    const float2 rf = __half22float2(*reinterpret_cast<const __half2*>(&r));
                    const float2 w2 = mul2(add2(hf, rf), make_float2(f, f));
                    const uint32_t nh = h2_bits(__floats2half2_rn(w2.x, w2.y));
                    const float2 lo2 = residual(w2, nh);
                    const uint32_t nr = h2_bits(__floats2half2_rn(lo2.x, lo2.y));
                    va[i] = __uint_as_float(before == m ? h : nh);
                    va[16 + i] = __uint_as_float(before == m ? r : nr);
                  }
                  tmem_st<16>(tS, va);
                  tmem_st<16, 16>(tS + 16, va);
                }
                total = chunk_weights(x, fits);
              }
              l += total;
#pragma unroll
              for (int z = 0; z < 16; z += kPack) {
                pack(va, x, z);
                put(x, z);
              }
            }
            if (!up) break;
          } else {
            auto all_weights = [&]() -> float {
              scaled(va, 0);
              scaled(vb, 1);
              sum = sum2 = make_float2(0.f, 0.f);
              weights(va);
              weights(vb);
              return (sum.x + sum.y) + (sum2.x + sum2.y);
            };
            tmem_ld_wait(va);
            tmem_ld_wait(vb);
            // The weights against the reference so far; a row whose sum stays
            // below the limit keeps it, without its maximum ever being taken.
            float total = 0.f;
            bool need = mine;
            if (y > 0) {
              total = all_weights();
              need = mine && (m == -INFINITY || !(total <= kSumLimit));
              pack(va, 0, 0);  // (in the shadow of the vote)
            }
            if (__any_sync(0xffffffffu, need)) {
              // Rows over the limit and rows at their first keys: the reference
              // becomes the step's maximum; the scores are read again.
              if (y > 0) {
                tmem_ld32(tS, va);
                tmem_ld32(tS + 32, vb);
                tmem_ld_wait(va);
                tmem_ld_wait(vb);
              }
              scaled(va, 0);
              scaled(vb, 1);
              float mx = -INFINITY;
#pragma unroll
              for (int e = 0; e < 32; ++e) mx = max3(mx, va[e], vb[e]);
              if (!move(need, mx * cs)) break;
              sum = sum2 = make_float2(0.f, 0.f);
              weights(va);
              weights(vb);
              total = (sum.x + sum.y) + (sum2.x + sum2.y);
              pack(va, 0, 0);
            }
            l += total;
            put(0, 0);
            pack(vb, 1, 0);
            put(1, 0);
          }
          tmem_st_wait();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(BAR_PFULL + w * 2 + (c & 1)));
      }
      if (!ok) {
        tmem_ld_wait();
        tmem_st_wait();
      }
      // ---- the segment's partial ------------------------------------------------
      // The next segment's Q goes into the other buffer, where there is one.
      const Segment& gn = segs[(seg + 1) % kSegSlots];
      bool more = __all_sync(0xffffffffu, seg_wait(BAR_GFULL + (seg + 1) % kSegSlots, (seg + 1) / kSegSlots));
      const bool q_ahead = kDualOk && more && gn.n != 0 && !dual && !(gn.flags & kDual);
      if (q_ahead) stage_q(gn);
      ok = __all_sync(0xffffffffu, ok && wait(BAR_SEG, seg));
      bool row_bad = false;
      if (*reinterpret_cast<volatile int*>(misc + 9) != 0) {  // rows that see an out-of-range block
        const int k0 = max(lo, key0), k1 = min(min(hi, ghi), key0 + g.n * kTileKeys - 1);
        for (int k = k0 / kChunk * kChunk; k <= k1; k += kChunk) {
          const int phys = __ldg(g.table + k / p.block_size);
          row_bad |= phys < 0 || phys >= p.num_blocks;
        }
      }
      // Every warpgroup's m and l of its rows, through Q's buffer (it has been read).
      const uint32_t q_off = !dual && (g.flags & kBuf) ? kTileBytes : 0;
      float2* stat = reinterpret_cast<float2*>(smem + C::kQ + q_off);  // [2][128]
      stat[w * 128 + r] = make_float2(row_bad ? __uint_as_float(kInvalidLse) : m, l);
      ok = named_bar_and(1, kSoftThreads, ok);
      const float2 s0 = stat[(dual ? w : 0) * 128 + r];
      const float2 s1 = dual ? make_float2(-INFINITY, 0.f) : stat[128 + r];
      more = named_bar_and(2, kSoftThreads, more);  // (the same for all)
      if (!ok) break;  // (in all softmax warps: the CTA gave up)
      // single: the two streams' sums; f0, f1: the accumulators' factors
      const bool bad = isnan(s0.x) || isnan(s1.x);
      const float mm = fmaxf(s0.x, s1.x);
      const float w0 = s0.y > 0.f ? fast_exp2(s0.x - mm) : 0.f;
      const float w1 = s1.y > 0.f ? fast_exp2(s1.x - mm) : 0.f;
      const float ll = s0.y * w0 + s1.y * w1;
      if ((dual || w == 0) && mine)
        p.part_lse[g.out_row + local] = bad         ? __uint_as_float(kInvalidLse)
                                        : ll > 0.f  ? (mm - kShift + log2f(ll)) * kLn2
                                        : ll == 0.f ? -INFINITY
                                                    : INFINITY;  // a score was not finite
      if (warp_rows) {
        tc_fence_after();
        const float inv = ll > 0.f ? 1.f / ll : 0.f;
        const float f0 = w0 * inv, f1 = w1 * inv;
        const int nx = dual ? 4 : 2, x0 = dual ? 0 : w * 2;  // this warpgroup's chunks of 32 columns
        const uint32_t stage = sQ + q_off + warp * 4096;
        float* out = p.part_out + (g.out_row + local - lane) * kHeadDim;     // the warp's first row
#pragma unroll 1
        for (int c = x0; c < x0 + nx; ++c) {
          float o[32];
          tmem_ld32(tO + (dual ? w * 128 : 0) + c * 32, o);
          tmem_ld_wait(o);
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = f0 > 0.f ? o[e] * f0 : 0.f;  // a stream without keys holds no sums
          if (!dual) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              float o1[16];
              tmem_ld<16>(tO + 128 + c * 32 + x * 16, o1);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 16; ++e) o[x * 16 + e] += f1 > 0.f ? o1[e] * f1 : 0.f;
            }
          }
          // rows to coalesced lines through this warp's 4 KB of the buffer
#pragma unroll
          for (int e = 0; e < 8; ++e)
            sts_v4(stage + lane * 128 + ((e ^ (lane % 8)) * 16),
                   make_uint4(__float_as_uint(o[4 * e]), __float_as_uint(o[4 * e + 1]),
                              __float_as_uint(o[4 * e + 2]), __float_as_uint(o[4 * e + 3])));
          __syncwarp();
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int y = e * 4 + lane / 8;  // row of the warp
            const uint4 u = lds_v4(stage + y * 128 + (((lane % 8) ^ (y % 8)) * 16));
            if (local - lane + y < g.nrows)
              *(reinterpret_cast<uint4*>(out + (long long)y * kHeadDim + c * 32) + lane % 8) = u;
          }
          __syncwarp();
        }
      }
      T0 += g.n;
      c0 += Y;
      tc_fence_before();
      __syncwarp();  // no lane reads g any more: its slot is given back
      if (lane == 0) {
        mbar_arrive(bar(BAR_OEMPTY));
        mbar_arrive(bar(BAR_GEMPTY + seg % kSegSlots));
      }
      ++seg;
      named_bar_sync(3, kSoftThreads);  // this segment's buffer may be staged again
      got = more && gn.n != 0;
      if (got && !q_ahead) stage_q(gn);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == C::kMmaWarp) {
    tmem_relinquish();
    tmem_dealloc(tmem, 512);
  }
  if (threadIdx.x == 0) {
    const int late = *abort;
    p.gave_up[cta] = late;
    if (late) atomicOr(p.flags, kFlagTimeout);
  }
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
