// pages.cu -- the page operations of a paged KV cache: sequences that share
// pages (fork), grow, shrink and end (resize), a pool that is closed up
// (compact), and the copies of whole pages that these ask for.
//
// The books are three device arrays: block_table, context_lens and
// ref_counts[num_blocks], the number of table rows that hold a page (0: the
// page is free).  There is no free list: the fresh pages of a call are the
// lowest-numbered free ones, handed out in the order of the requests, so
// every result follows from the books and the requests alone, whatever order
// the threads run in (integer sums and minima commute; nothing else is
// atomic).
//
// Bound: the bookkeeping calls move a few hundred kilobytes and are latency
// (dependent trips to L2 between barriers); the copies are HBM bandwidth.
// The planning kernels are one thread-block cluster, whose hardware barrier
// joins the phases without a second launch.
#include <atomic>
#include <climits>

#include "common.cuh"
#include "kernels.h"
#include "sm100.cuh"

namespace pa {
namespace {

using namespace sm100;

constexpr int kPlanCtas = 8;        // CTAs of a planning kernel (one cluster)
constexpr int kPlanThreads = 1024;
constexpr int kPlanAll = kPlanCtas * kPlanThreads;

__device__ __forceinline__ unsigned cluster_rank() {
  unsigned r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// Every thread of the cluster; what was written before is visible after (to
// the cluster's threads: the barrier releases and acquires).
__device__ __forceinline__ void cluster_sync() {
  asm volatile(
      "barrier.cluster.arrive.release;\n\t"
      "barrier.cluster.wait.acquire;" ::
          : "memory");
}

__device__ __forceinline__ bool page_ok(const PageParams& p, int page) {
  return page >= 0 && page < p.num_blocks;
}
__device__ __forceinline__ bool row_ok(const PageParams& p, int row) {
  return row >= 0 && row < p.num_seqs;
}
__device__ __forceinline__ bool len_ok(const PageParams& p, int len) {
  return len >= 0 && (long long)len <= (long long)p.max_blocks_per_seq * p.block_size;
}
__device__ __forceinline__ int pages_of(const PageParams& p, int len) {
  return (int)(((long long)len + p.block_size - 1) / p.block_size);
}
__device__ __forceinline__ int32_t* table_row(const PageParams& p, int row) {
  return p.block_table + (long long)row * p.max_blocks_per_seq;
}

// Exclusive prefix sum over the CTA's threads, and the CTA's total.
template <typename T>
__device__ __forceinline__ T block_scan(T v, T* warp_sums, T& total) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  T x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();  // an earlier scan's sums have been read
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    T s = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const T y = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += y;
    }
    warp_sums[lane] = s;
  }
  __syncthreads();
  total = warp_sums[31];
  return x - v + (warp > 0 ? warp_sums[warp - 1] : 0);
}

// The pages of one CTA's share of the pool.
__device__ __forceinline__ void pool_share(int num_blocks, int rank, int& b0, int& b1) {
  b0 = (int)((long long)rank * num_blocks / kPlanCtas);
  b1 = (int)((long long)(rank + 1) * num_blocks / kPlanCtas);
}

// ------------------------------------------------------------------- fork
// One CTA per request.  A request stands unless a row is out of range, the
// child has tokens, an earlier request has the same child, or the parent is
// a child of the call itself (its row is being written).  Each CTA reads all
// children for that: n^2 of them, 5 us for 64 requests of 63 pages, 17 for
// 1024, 38 for 4096, 174 for 16384 and 1.5 ms for 65536.
constexpr int kForkThreads = 256;

__global__ void __launch_bounds__(kForkThreads) fork_kernel(const PageParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int i = blockIdx.x, tid = threadIdx.x;
  const int par = __ldg(p.parents + i), child = __ldg(p.rows + i);
  bool bad = !row_ok(p, par) || !row_ok(p, child);
  for (int j = tid; j < p.n; j += kForkThreads) {
    const int c = __ldg(p.rows + j);
    bad |= c == par || (c == child && j < i);
  }
  int L = 0;
  bool bad_len = false;
  if (!bad) {
    bad = __ldcg(p.context_lens + child) != 0;
    L = __ldcg(p.context_lens + par);
    bad_len = !len_ok(p, L);
  }
  if (__syncthreads_or(bad)) {
    if (tid == 0) atomicOr(p.flags, kFlagBadRequest);
    return;
  }
  if (__syncthreads_or(bad_len)) {
    if (tid == 0) atomicOr(p.flags, kFlagBadLen);
    return;
  }
  const int held = pages_of(p, L);
  const int32_t* from = table_row(p, par);
  int32_t* to = table_row(p, child);
  // The first pages stay in registers between the check and the copy.
  constexpr int kKeep = 4;
  int kept[kKeep];
  bool bad_page = false;
#pragma unroll
  for (int e = 0; e < kKeep; ++e) {
    const int b = tid + e * kForkThreads;
    kept[e] = b < held ? __ldcg(from + b) : 0;
  }
#pragma unroll
  for (int e = 0; e < kKeep; ++e) bad_page |= !page_ok(p, kept[e]);
  for (int b = tid + kKeep * kForkThreads; b < held; b += kForkThreads) bad_page |= !page_ok(p, __ldcg(from + b));
  if (__syncthreads_or(bad_page)) {
    if (tid == 0) atomicOr(p.flags, kFlagBadBlock);
    return;
  }
#pragma unroll
  for (int e = 0; e < kKeep; ++e) {
    const int b = tid + e * kForkThreads;
    if (b < held) {
      to[b] = kept[e];
      atomicAdd(p.ref_counts + kept[e], 1);
    }
  }
  for (int b = tid + kKeep * kForkThreads; b < held; b += kForkThreads) {
    const int page = __ldcg(from + b);
    to[b] = page;
    atomicAdd(p.ref_counts + page, 1);
  }
  if (tid == 0) p.context_lens[child] = L;
}

// ----------------------------------------------------------------- resize
// Requests (row, new length).  Scratch: row_mark[row] the lowest request on
// a row; holders[page] and keeper[page] how many requests grow out of the
// ragged page and the last of them; need[i] / end[i] fresh pages of request
// i and their running total; fresh[k] the k-th lowest free page.
enum : int { kStands = 1, kGrows = 2 };

__global__ void __launch_bounds__(kPlanThreads, 1) resize_kernel(const PageParams p) {
  __shared__ int sums[32];
  __shared__ long long long_sums[32];
  griddep_wait();
  griddep_launch_dependents();
  const int rank = (int)cluster_rank(), tid = threadIdx.x;
  const int gt = rank * kPlanThreads + tid;
  int* row_mark = p.row_scratch;
  int* need = p.row_scratch + p.num_seqs;
  int* end = p.row_scratch + 2LL * p.num_seqs;
  int* holders = p.page_scratch;
  int* keeper = p.page_scratch + p.num_blocks;
  int* fresh = p.page_scratch + 2LL * p.num_blocks;
  int* share = p.small_scratch;  // [kPlanCtas] free pages of every CTA's share

  // What request i asks for: its row, both lengths and, where it grows out
  // of a ragged page, that page (-1: none).  0: it cannot stand on its own.
  auto request = [&](int i, int& row, int& L, int& want, int& page) -> int {
    row = __ldg(p.rows + i);
    want = p.new_lens != nullptr ? __ldg(p.new_lens + i) : 0;
    page = -1;
    if (!row_ok(p, row)) {
      atomicOr(p.flags, kFlagBadRequest);
      return 0;
    }
    L = __ldcg(p.context_lens + row);
    if (!len_ok(p, want) || !len_ok(p, L)) {
      atomicOr(p.flags, kFlagBadLen);
      return 0;
    }
    if (want > L && L % p.block_size != 0) {
      page = __ldcg(table_row(p, row) + L / p.block_size);
      if (!page_ok(p, page)) {
        atomicOr(p.flags, kFlagBadBlock);
        return 0;
      }
    }
    return kStands | (want > L ? kGrows : 0);
  };

  for (int i = gt; i < p.n; i += kPlanAll) {
    int row, L, want, page;
    if (request(i, row, L, want, page) == 0) continue;
    row_mark[row] = INT_MAX;
    if (page >= 0) {
      holders[page] = 0;
      keeper[page] = -1;
    }
  }
  cluster_sync();
  for (int i = gt; i < p.n; i += kPlanAll) {
    int row, L, want, page;
    if (request(i, row, L, want, page) != 0) atomicMin(row_mark + row, i);
  }
  cluster_sync();
  for (int i = gt; i < p.n; i += kPlanAll) {
    int row, L, want, page;
    if (request(i, row, L, want, page) == 0) continue;
    if (__ldcg(row_mark + row) != i) {
      atomicOr(p.flags, kFlagBadRequest);
      continue;
    }
    if (page >= 0) {
      atomicAdd(holders + page, 1);
      atomicMax(keeper + page, i);
    }
  }
  cluster_sync();
  for (int i = gt; i < p.n; i += kPlanAll) {
    int row, L, want, page, nd = 0;
    const int st = request(i, row, L, want, page);
    if ((st & kGrows) && __ldcg(row_mark + row) == i) {
      nd = pages_of(p, want) - pages_of(p, L);
      if (page >= 0) {
        const int refs = __ldcg(p.ref_counts + page);
        const bool keeps = __ldcg(holders + page) == refs && __ldcg(keeper + page) == i;
        if (refs > 1 && !keeps) ++nd;
      }
    }
    need[i] = nd;
  }
  int b0, b1, total;
  pool_share(p.num_blocks, rank, b0, b1);
  int mine = 0;
  for (int b = b0 + tid; b < b1; b += kPlanThreads) mine += __ldcg(p.ref_counts + b) == 0;
  block_scan(mine, sums, total);
  if (tid == 0) share[rank] = total;
  cluster_sync();
  if (rank == 0) {
    // 64 bits: many large requests may add up past the 32-bit range
    long long run = 0, sum = 0;
    for (int i0 = 0; i0 < p.n; i0 += kPlanThreads) {
      const int i = i0 + tid;
      const long long nd = i < p.n ? __ldcg(need + i) : 0;
      const long long e = run + block_scan(nd, long_sums, sum) + nd;
      if (i < p.n) end[i] = (int)min(e, (long long)INT_MAX);
      run += sum;
    }
    if (tid == 0) share[kPlanCtas] = (int)min(run, (long long)INT_MAX);
  }
  cluster_sync();
  int base = 0, nfree = 0;
  for (int r = 0; r < kPlanCtas; ++r) {
    const int c = __ldcg(share + r);
    if (r < rank) base += c;
    nfree += c;
  }
  const int wanted = min(__ldcg(share + kPlanCtas), nfree);
  for (int t0 = b0; t0 < b1 && base < wanted; t0 += kPlanThreads) {
    const int b = t0 + tid;
    const bool is_free = b < b1 && __ldcg(p.ref_counts + b) == 0;
    const int k = base + block_scan((int)is_free, sums, total);
    if (is_free && k < wanted) fresh[k] = b;
    base += total;
  }
  cluster_sync();
  // Carry out: one warp per request.
  const int lane = tid % 32;
  for (int i = gt / 32; i < p.n; i += kPlanAll / 32) {
    // Lane 0 reads the request (it also writes the row's new length, last).
    int row = 0, L = 0, want = 0, page = -1, st = 0;
    if (lane == 0) {
      row = __ldg(p.rows + i);
      if (row_ok(p, row) && __ldcg(row_mark + row) == i) st = request(i, row, L, want, page);
    }
    st = __shfl_sync(0xffffffffu, st, 0);
    row = __shfl_sync(0xffffffffu, row, 0);
    L = __shfl_sync(0xffffffffu, L, 0);
    want = __shfl_sync(0xffffffffu, want, 0);
    page = __shfl_sync(0xffffffffu, page, 0);
    const bool stands = st != 0;
    int src = -1, dst = -1;
    if (stands && (st & kGrows)) {
      const int nd = __ldcg(need + i), e = __ldcg(end + i);
      if (e > nfree) {
        if (lane == 0) atomicOr(p.flags, kFlagNoPages);
      } else {
        const int have = pages_of(p, L), add = pages_of(p, want) - have;
        const int32_t* f = fresh + (e - nd);
        int32_t* t = table_row(p, row);
        if (nd > add) {  // the ragged page is shared: its copy comes first
          src = page;
          dst = __ldcg(f);
          ++f;
          if (lane == 0) {
            t[L / p.block_size] = dst;
            atomicAdd(p.ref_counts + dst, 1);
            atomicSub(p.ref_counts + page, 1);
          }
        }
        for (int b = lane; b < add; b += 32) {
          const int pg = __ldcg(f + b);
          t[have + b] = pg;
          atomicAdd(p.ref_counts + pg, 1);
        }
        if (lane == 0) p.context_lens[row] = want;
      }
    } else if (stands) {
      // (whatever the entries hold: a row with damaged ones can be ended)
      const int32_t* t = table_row(p, row);
      for (int b = pages_of(p, want) + lane; b < pages_of(p, L); b += 32) {
        const int pg = __ldcg(t + b);
        if (!page_ok(p, pg)) {
          atomicOr(p.flags, kFlagBadBlock);
        } else if (atomicSub(p.ref_counts + pg, 1) <= 0) {  // was not held: the books are wrong
          atomicAdd(p.ref_counts + pg, 1);
          atomicOr(p.flags, kFlagBadRequest);
        }
      }
      __syncwarp();
      if (lane == 0) p.context_lens[row] = want;
    }
    if (lane == 0) {
      p.copy_src[i] = src;
      p.copy_dst[i] = dst;
    }
  }
}

// The same for at most kOneRequests requests on at most kOnePages pages, with
// one cluster barrier: every CTA makes the whole plan by itself (a request and
// 32 pages a thread; the requests are compared in shared memory), and after
// the barrier, when all have read the books, each changes its share of the
// table entries and counts.  Bound: the chain of dependent trips to L2
// (request, length, page, count; entry, count); the other form's phases cost a
// fence, a cluster barrier and a trip each, and are shared by all CTAs.
// Us a call on the GPU, one page grown or given up a row, pool of 32768 pages,
// this form | the other: 8 rows 8.6 | 9.8, 64 rows 9.8 | 12, 256 rows 11.7 | 12,
// 384 rows 14.6 | 13.8, 1024 rows 40 | 18.6 (the requests are compared pair by
// pair).  A hundred pages a row, all given up or taken: 64 rows 10.4 | 14.5, 256
// rows 22.9 | 15.5.
constexpr int kOneRequests = 256, kOnePages = 32 * kPlanThreads;
constexpr int kPiece = 256;      // table entries a warp changes at a time
constexpr int kOneFresh = 8192;  // fresh pages listed in shared memory

__global__ void __launch_bounds__(kPlanThreads, 1) resize_one_kernel(const PageParams p) {
  __shared__ int sums[32];
  __shared__ long long long_sums[32];
  __shared__ uint16_t near_list[kOneFresh];
  // (an entry a thread: those behind the requests are written, too)
  __shared__ int last_piece[kPlanThreads];
  __shared__ __align__(16) int at_row[kPlanThreads], at_page[kPlanThreads];
  __shared__ int at_fresh[kPlanThreads], at_count[kPlanThreads];
  extern __shared__ int given_up[];  // [num_blocks]
  griddep_wait();
  griddep_launch_dependents();
  const int rank = (int)cluster_rank(), i = threadIdx.x, lane = i % 32, warp = i / 32;
  const bool mine = i < p.n;
  const int row = mine ? __ldg(p.rows + i) : -1;
  const int want = mine && p.new_lens != nullptr ? __ldg(p.new_lens + i) : 0;
  int L = mine && row_ok(p, row) ? __ldcg(p.context_lens + row) : 0;
  // Pages 32 i .. 32 i + 31: bit set = free.
  uint32_t free_mask = 0;
  {
    int c[32];
#pragma unroll
    for (int k = 0; k < 32; ++k) {
      const int b = (warp * 32 + k) * 32 + lane;
      c[k] = b < p.num_blocks ? __ldcg(p.ref_counts + b) : 1;
    }
#pragma unroll
    for (int k = 0; k < 32; ++k) {
      const uint32_t m = __ballot_sync(0xffffffffu, c[k] == 0);
      if (lane == k) free_mask = m;
    }
  }
  // ---- the request on its own
  unsigned flags = 0;
  bool stands = false, grows = false;
  int page = -1;
  if (mine) {
    stands = row_ok(p, row);
    if (!stands) {
      flags = kFlagBadRequest;
      L = 0;
    } else if (!len_ok(p, want) || !len_ok(p, L)) {
      flags = kFlagBadLen;
      stands = false;
    } else if (want > L) {
      grows = true;
      if (L % p.block_size != 0) {
        page = __ldcg(table_row(p, row) + L / p.block_size);
        if (!page_ok(p, page)) {
          flags = kFlagBadBlock;
          stands = false;
        }
      }
    }
  }
  // ---- among the others: the first of its row; who grows out of a page
  at_row[i] = stands ? row : -1;
  __syncthreads();
  const int n4 = (p.n + 3) / 4;
  if (stands) {
    int lowest = i;
#pragma unroll 8
    for (int j = n4 - 1; j >= 0; --j) {
      const int4 r = reinterpret_cast<const int4*>(at_row)[j];
      if (r.w == row) lowest = min(lowest, 4 * j + 3);
      if (r.z == row) lowest = min(lowest, 4 * j + 2);
      if (r.y == row) lowest = min(lowest, 4 * j + 1);
      if (r.x == row) lowest = min(lowest, 4 * j);
    }
    if (lowest != i) {
      flags = kFlagBadRequest;
      stands = false;
    }
  }
  const bool ragged = stands && grows && page >= 0;
  const int refs = ragged ? __ldcg(p.ref_counts + page) : 0;
  at_page[i] = ragged ? page : -1;
  __syncthreads();
  bool split = refs > 1;
  if (split) {
    int holders = 0, keeper = 0;
#pragma unroll 8
    for (int j = 0; j < n4; ++j) {
      const int4 q = reinterpret_cast<const int4*>(at_page)[j];
      holders += (q.x == page) + (q.y == page) + (q.z == page) + (q.w == page);
      if (q.x == page) keeper = max(keeper, 4 * j);
      if (q.y == page) keeper = max(keeper, 4 * j + 1);
      if (q.z == page) keeper = max(keeper, 4 * j + 2);
      if (q.w == page) keeper = max(keeper, 4 * j + 3);
    }
    split = !(holders == refs && keeper == i);
  }
  // ---- fresh pages: the lowest free ones in the order of the requests
  const int have = pages_of(p, L), wanted = pages_of(p, want);
  const long long need = stands && grows ? (long long)wanted - have + split : 0;
  // Both running totals in one: the needs, which may add up past 32 bits, and
  // in the low 20 bits the free pages.
  const long long both = need << 20 | __popc(free_mask);
  long long all;
  const long long before = block_scan(both, long_sums, all);
  const long long all_need = all >> 20, end = (before >> 20) + need;
  const int nfree = (int)(all & 0xfffff);
  int k = (int)(before & 0xfffff);
  const int listed = (int)min(all_need, (long long)nfree);
  const bool near = listed <= kOneFresh;
  int* far_list = p.page_scratch + 2LL * p.num_blocks;
  for (uint32_t m = free_mask; m != 0 && k < listed; m &= m - 1, ++k) {
    const int b = 32 * i + __ffs(m) - 1;
    if (near) near_list[k] = (uint16_t)b;
    else if (rank == 0) far_list[k] = b;
  }
  if (stands && grows && end > nfree) {
    flags = kFlagNoPages;
    stands = false;
  }
  const int change = stands ? wanted - have : 0;  // entries taken, or (negative) given up
  // Pieces of kPiece entries; last_piece: their running total.
  int pieces;
  last_piece[i] = block_scan((abs(change) + kPiece - 1) / kPiece, sums, pieces) +
                  (abs(change) + kPiece - 1) / kPiece;
  at_count[i] = change;
  at_row[i] = row;
  at_page[i] = grows ? have : wanted;
  at_fresh[i] = (int)(end - change);
  cluster_sync();  // the books have been read
  auto fresh = [&](int x) { return near ? (int)near_list[x] : __ldcg(far_list + x); };
  if (mine && rank == 0) {
    int src = -1, dst = -1;
    if (stands) {
      if (split) {
        src = page;
        dst = fresh((int)(end - need));
        table_row(p, row)[L / p.block_size] = dst;
        p.ref_counts[dst] = 1;
        atomicSub(p.ref_counts + page, 1);
      }
      p.context_lens[row] = want;
    }
    p.copy_src[i] = src;
    p.copy_dst[i] = dst;
  }
  if (rank != 0) flags = 0;
  const bool drops = __syncthreads_or(change < 0);
  if (drops) {
    for (int b = i; b < p.num_blocks; b += kPlanThreads) given_up[b] = 0;
    __syncthreads();
  }
  // This CTA's run of the pieces, a warp each.
  const int q1 = (int)((long long)pieces * (rank + 1) / kPlanCtas);
  for (int q = (int)((long long)pieces * rank / kPlanCtas) + warp; q < q1; q += kPlanThreads / 32) {
    int lo = 0, hi = p.n - 1;  // the first request with last_piece > q
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      if (last_piece[mid] > q) hi = mid;
      else lo = mid + 1;
    }
    const int o0 = (q - (lo > 0 ? last_piece[lo - 1] : 0)) * kPiece, count = at_count[lo];
    int32_t* entry = table_row(p, at_row[lo]) + at_page[lo] + o0 + lane;
    const int left = abs(count) - o0 - lane;  // this lane's entries: 0, 32, .. below it
    if (count > 0) {
#pragma unroll
      for (int e = 0; e < kPiece; e += 32) {
        if (e >= left) continue;
        const int pg = fresh(at_fresh[lo] + o0 + lane + e);
        entry[e] = pg;
        p.ref_counts[pg] = 1;
      }
    } else {
      int pg[kPiece / 32];
#pragma unroll
      for (int e = 0; e < kPiece; e += 32) pg[e / 32] = e < left ? __ldcg(entry + e) : 0;
#pragma unroll
      for (int e = 0; e < kPiece; e += 32) {
        if (e >= left) continue;
        if (page_ok(p, pg[e / 32])) atomicAdd(given_up + pg[e / 32], 1);
        else flags |= kFlagBadBlock;
      }
    }
  }
  if (drops) {  // (the same in every CTA)
    // Given-up pages are counted in shared memory first: they lie anywhere, and
    // a GPC's atomics on single words of L2 are slow (63,000 of them: 40 us).
    __syncthreads();
#pragma unroll 8
    for (int b = i; b < p.num_blocks; b += kPlanThreads)
      if (given_up[b] != 0) atomicSub(p.ref_counts + b, given_up[b]);
    cluster_sync();
    bool wrong = false;
#pragma unroll 8
    for (int b = i; b < p.num_blocks; b += kPlanThreads) {
      const int c = __ldcg(p.ref_counts + b);
      wrong |= c < 0 && given_up[b] != 0;
    }
    if (wrong) {  // pages that were not held: the books were wrong
      flags |= kFlagBadRequest;
      for (int b = i; b < p.num_blocks; b += kPlanThreads)
        if (given_up[b] != 0) atomicMax(p.ref_counts + b, 0);
    }
  }
  if (flags != 0) atomicOr(p.flags, flags);
}

// ---------------------------------------------------------------- compact
// A row's entries after a compaction, by `step` threads of which this is `at`.
__device__ __forceinline__ void remap_row(const PageParams& p, int row, int at, int step) {
  const int L = __ldcg(p.context_lens + row);
  if (!len_ok(p, L)) {
    if (at == 0) atomicOr(p.flags, kFlagBadLen);
    return;
  }
  const int held = pages_of(p, L);
  int32_t* t = table_row(p, row);
#pragma unroll 4
  for (int b = at; b < held; b += step) {
    const int page = __ldcg(t + b);
    if (!page_ok(p, page)) {
      atomicOr(p.flags, kFlagBadBlock);
      continue;
    }
    const int to = __ldcg(p.remap + page);
    if (to < 0) atomicOr(p.flags, kFlagBadRequest);  // the row holds a free page
    else if (to != page) t[b] = to;
  }
}

// n_live live pages; the k-th lowest live page at or above n_live moves to
// the k-th lowest free page below it.
__global__ void __launch_bounds__(kPlanThreads, 1) compact_kernel(const PageParams p) {
  __shared__ int sums[32];
  griddep_wait();
  griddep_launch_dependents();
  const int rank = (int)cluster_rank(), tid = threadIdx.x;
  int* share = p.small_scratch;
  int b0, b1, total, mine = 0;
  pool_share(p.num_blocks, rank, b0, b1);
  for (int b = b0 + tid; b < b1; b += kPlanThreads) mine += __ldcg(p.ref_counts + b) > 0;
  block_scan(mine, sums, total);
  if (tid == 0) share[rank] = total;
  cluster_sync();
  int before = 0, n_live = 0;
  for (int r = 0; r < kPlanCtas; ++r) {
    const int c = __ldcg(share + r);
    if (r < rank) before += c;
    n_live += c;
  }
  // Every page's rank among the live ones; gaps go into copy_dst by theirs.
  // remap holds a high page's rank until its target is known.
  if (n_live == p.num_blocks && rank == 0 && tid == 0) share[kPlanCtas] = 0;
  for (int t0 = b0; t0 < b1; t0 += kPlanThreads) {
    const int b = t0 + tid;
    const bool live = b < b1 && __ldcg(p.ref_counts + b) > 0;
    const int below = before + block_scan((int)live, sums, total);  // live pages below b
    if (b < b1) {
      p.remap[b] = !live ? -1 : b < n_live ? b : below;
      if (!live && b < n_live) p.copy_dst[b - below] = b;
      if (b == n_live) share[kPlanCtas] = n_live - below;  // live pages at or above n_live
    }
    before += total;
  }
  cluster_sync();
  const int moves = __ldcg(share + kPlanCtas);
  for (int b = max(b0, n_live) + tid; b < b1; b += kPlanThreads) {
    const int below = p.remap[b];
    if (below < 0) continue;
    const int k = below - (n_live - moves);
    const int to = __ldcg(p.copy_dst + k);
    p.copy_src[k] = b;
    p.remap[b] = to;
    p.ref_counts[to] = p.ref_counts[b];
    p.ref_counts[b] = 0;
  }
  for (int k = moves + rank * kPlanThreads + tid; k < p.n; k += kPlanAll) {
    p.copy_src[k] = -1;
    p.copy_dst[k] = -1;
  }
  if (rank == 0 && tid == 0) *p.count = moves;
  if (!p.tables_too) return;
  cluster_sync();  // every page's new place is known
  for (int row = rank * (kPlanThreads / 32) + tid / 32; row < p.num_seqs; row += kPlanAll / 32)
    remap_row(p, row, tid % 32, 32);
}

// The tables after a compaction: one CTA per row.
__global__ void __launch_bounds__(256) remap_kernel(const PageParams p) {
  griddep_wait();
  griddep_launch_dependents();
  remap_row(p, blockIdx.x, threadIdx.x, 256);
}

// ------------------------------------------------------------------- copy
// Pairs (src, dst); a negative src is skipped.  A pair stands unless a page
// is out of range, an earlier standing-range pair has the same target, or
// its source is a target: then no page is written twice and none that is
// read is written, whatever the order of the copies.  The list that stands
// (-1 elsewhere) goes to scratch for copy_kernel.
__global__ void __launch_bounds__(kPlanThreads, 1) copy_check_kernel(const PageParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int gt = (int)cluster_rank() * kPlanThreads + threadIdx.x;
  int* owner = p.page_scratch;
  int* src_ok = p.page_scratch + p.num_blocks;
  const int n = p.count != nullptr ? max(0, min(p.n, __ldcg(p.count))) : p.n;
  auto pair = [&](int i, int& s, int& d) -> bool {
    s = __ldcg(p.copy_src + i);
    d = __ldcg(p.copy_dst + i);
    return s >= 0 && page_ok(p, s) && page_ok(p, d);
  };
  for (int i = gt; i < n; i += kPlanAll) {
    int s, d;
    if (pair(i, s, d)) {
      owner[s] = INT_MAX;
      owner[d] = INT_MAX;
    } else if (s >= 0) {
      atomicOr(p.flags, kFlagBadBlock);
    }
  }
  cluster_sync();
  for (int i = gt; i < n; i += kPlanAll) {
    int s, d;
    if (pair(i, s, d)) atomicMin(owner + d, i);
  }
  cluster_sync();
  for (int i = gt; i < n; i += kPlanAll) {
    int s, d;
    bool ok = pair(i, s, d);
    if (ok && (__ldcg(owner + d) != i || __ldcg(owner + s) != INT_MAX)) {
      ok = false;
      atomicOr(p.flags, kFlagBadRequest);
    }
    src_ok[i] = ok ? s : -1;
  }
}

// A page is copied in equal pieces, each a multiple of 128 bytes, one CTA a
// piece.  Up to 40 KB a piece, so that common pages are one: 5001 pages of
// 34 KB, K and V, 120 us against 130 in pieces of 20 KB and 132 in 16 KB and a
// rest.
constexpr int kCopyThreads = 512;
constexpr int kCopyVecs = 5;  // 16-byte vectors per thread, at most
__host__ __device__ inline int copy_pieces(long long page_bytes) {
  const long long most = kCopyThreads * kCopyVecs * 16;
  return (int)((page_bytes + most - 1) / most);
}
// Up to this many pairs every CTA looks its own ones over against the list
// (four entries a thread): no launch and no cluster barriers before the
// copies, 5.1 us instead of 6.1 for 7 pairs, and one launch less on the host.
constexpr int kCopySelfCheck = 2048;

// Units (pair, K or V, piece of a page) over the grid.
template <bool kCheck>
__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const PageParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int* src_ok = p.page_scratch + p.num_blocks;
  const int n = p.count != nullptr ? max(0, min(p.n, __ldcg(p.count))) : p.n;
  const int pieces = copy_pieces(p.page_bytes);
  const long long piece = ((p.page_bytes + pieces - 1) / pieces + 127) / 128 * 128;
  const long long units = (long long)n * 2 * pieces;
  int seen = -1, s = -1, d = -1;  // the pair that was looked over last
  for (long long u = blockIdx.x; u < units; u += gridDim.x) {
    const int i = (int)(u / (2 * pieces)), r = (int)(u % (2 * pieces));
    if (!kCheck) {
      s = __ldcg(src_ok + i);
      d = __ldcg(p.copy_dst + i);
    } else if (i != seen) {
      seen = i;
      s = __ldcg(p.copy_src + i);
      d = __ldcg(p.copy_dst + i);
      if (s >= 0) {
        unsigned bad = page_ok(p, s) && page_ok(p, d) ? 0u : kFlagBadBlock;
        if (bad == 0) {
          bool clash = false;
          for (int j = threadIdx.x; j < n; j += kCopyThreads) {
            const int sj = __ldcg(p.copy_src + j), dj = __ldcg(p.copy_dst + j);
            if (sj >= 0 && page_ok(p, sj) && page_ok(p, dj)) clash |= dj == s || (dj == d && j < i);
          }
          if (__syncthreads_or(clash)) bad = kFlagBadRequest;
        }
        if (bad != 0) {
          if (threadIdx.x == 0) atomicOr(p.flags, bad);
          s = -1;
        }
      }
    }
    if (s < 0) continue;
    uint8_t* base = static_cast<uint8_t*>(r < pieces ? p.k_cache : p.v_cache);
    const long long off = r % pieces * piece + threadIdx.x * 16;
    const long long end = min(p.page_bytes, (r % pieces + 1) * piece);
    const uint4* from = reinterpret_cast<const uint4*>(base + s * p.page_bytes + off);
    uint4* to = reinterpret_cast<uint4*>(base + d * p.page_bytes + off);
    uint4 x[kCopyVecs];
#pragma unroll
    for (int e = 0; e < kCopyVecs; ++e)
      if (off + e * kCopyThreads * 16 < end) x[e] = __ldcs(from + e * kCopyThreads);
#pragma unroll
    for (int e = 0; e < kCopyVecs; ++e)
      if (off + e * kCopyThreads * 16 < end) __stcs(to + e * kCopyThreads, x[e]);
  }
}

cudaError_t launch(void (*kern)(const PageParams), unsigned grid, unsigned threads, int cluster,
                   const PageParams& p, cudaStream_t stream, size_t smem = 0) {
  cudaLaunchConfig_t cfg = {};
  cfg.dynamicSmemBytes = smem;
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace

cudaError_t launch_fork(const PageParams& p, cudaStream_t stream) {
  return launch(fork_kernel, p.n, kForkThreads, 1, p, stream);
}
cudaError_t launch_resize(const PageParams& p, cudaStream_t stream) {
  if (p.n <= kOneRequests && p.num_blocks <= kOnePages) {
    static std::atomic<unsigned long long> ready{0};  // devices whose attribute is set
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!(ready.load(std::memory_order_acquire) >> dev & 1)) {
      e = cudaFuncSetAttribute(resize_one_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               kOnePages * (int)sizeof(int));
      if (e != cudaSuccess) return e;
      ready.fetch_or(1ull << dev, std::memory_order_release);
    }
    return launch(resize_one_kernel, kPlanCtas, kPlanThreads, kPlanCtas, p, stream,
                  p.num_blocks * sizeof(int));
  }
  return launch(resize_kernel, kPlanCtas, kPlanThreads, kPlanCtas, p, stream);
}
// Tables of up to this many entries are rewritten by the planning cluster
// itself; larger ones by a launch over all SMs (184,000 entries: 4 us).
constexpr long long kTablesInside = 32768;

cudaError_t launch_compact(const PageParams& params, cudaStream_t stream) {
  PageParams p = params;
  p.tables_too = (long long)p.num_seqs * p.max_blocks_per_seq <= kTablesInside;
  const cudaError_t e = launch(compact_kernel, kPlanCtas, kPlanThreads, kPlanCtas, p, stream);
  if (e != cudaSuccess || p.tables_too) return e;
  return launch(remap_kernel, p.num_seqs, 256, 1, p, stream);
}
cudaError_t launch_copy_blocks(const PageParams& p, int sms, cudaStream_t stream) {
  const long long units = (long long)p.n * 2 * copy_pieces(p.page_bytes);
  // More CTAs than fit at a time (4 an SM do), so that they do not load and
  // store in step: 117 us against 120 with 8 an SM, 128 with 4.  One for every
  // piece (116) is slow for a list whose count is far below n: 124 us against
  // 95 for 8192 entries of which about 3300 stand.
  const long long most = (long long)sms * 32;
  const unsigned grid = (unsigned)(units < most ? units : most);
  if (p.n <= kCopySelfCheck) return launch(copy_kernel<true>, grid, kCopyThreads, 1, p, stream);
  const cudaError_t e = launch(copy_check_kernel, kPlanCtas, kPlanThreads, kPlanCtas, p, stream);
  if (e != cudaSuccess) return e;
  return launch(copy_kernel<false>, grid, kCopyThreads, 1, p, stream);
}

}  // namespace pa
