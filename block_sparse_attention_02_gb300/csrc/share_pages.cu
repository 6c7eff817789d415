// share_pages.cu -- pages that several requests hold, requests that start from another's cache, pages gathered at the
// pool's front, and the copies that these need.
//
// A request that continues another one's text (parallel samples, beams) needs its cached tokens.  Its full pages are
// not written again (as long as lengths only grow), so both may hold them; only the page that is partly filled is copied.  page_shares counts a page's
// holders beyond the first, so that pages given out by msa_plan_step (0) need nothing, and a page goes back on the stack
// when the count would fall below 0.
//
// Each of the three index kernels is one thread-block cluster, or one CTA for small pools and tables: it forms the sums over
// the requests for itself, goes through the table entries and the pages side by side, and meets at a barrier where one step
// needs all of the step before (counts before the search for freed pages, marks before ranks, ranks before the table).  So a
// call is one launch without scratch, lengths and counts may be updated in place, and whatever is counted by atomics is a sum,
// the same in any order; freed pages and moves are ordered by page number.
//
// Bound: latency (the barriers, of which a cluster's takes half a microsecond; dependent loads of lengths, tables and counts): release
// and fork of 64 requests in a pool of 3,463 pages 6.1 and 5.0 us, compaction of 2,048 pages 8.8.  The copies are bound by HBM: 512 pages of
// 640 KB 107 us, 93 % of a copy's rate.
#include <cooperative_groups.h>

#include <climits>

#include "launch_early.cuh"
#include "msa_internal.h"
#include "msa_ptx.cuh"

namespace cg = cooperative_groups;

namespace msa {
namespace {

constexpr int kAlone = 1024, kThreads = 512;              // threads of a CTA alone, and of a cluster's
constexpr int kCluster = 8;                                // CTAs (the portable maximum)
constexpr int kPer = kMaxDecodeBatch / kThreads;           // requests (or forks) of a thread in the sums, at most
// Entries or pages up to which one CTA releases or compacts (compaction of 512 / 1,024 / 1,536 / 4,096 pages 6.1 / 7.1 / 8.7 / 14.4 us
// for a cluster's 7.4 / 8.4 / 8.7 / 9.0, release of 1,024 / 8,192 5.4 / 12.7 for 5.3 / 6.2).  Forks, with one barrier, are a
// cluster's at every size (128 pages 4.8 for 6.1).
constexpr int kAloneItems = 1024;
constexpr int kOwn = 4;                                    // pages of a thread that it looks at together
constexpr int kCopyThreads = 256;
constexpr int kCopyUnroll = 4;
constexpr int kCopyChunk = kCopyThreads * kCopyUnroll * 16;   // bytes of a page that a CTA copies at a time

// Exclusive prefix sum over the CTA's threads; the total in *total.
__device__ __forceinline__ int block_exclusive(int v, int* total) {
  __shared__ int s_warp[kAlone / 32 + 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  int inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += x;
  }
  __syncthreads();                          // an earlier call's sums are read
  if (lane == 31) s_warp[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    const int own = lane < warps ? s_warp[lane] : 0;
    int w = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += x;
    }
    if (lane < warps) s_warp[lane] = w - own;
    if (lane == 31) s_warp[kAlone / 32] = w;
  }
  __syncthreads();
  *total = s_warp[kAlone / 32];
  return s_warp[warp] + inc - v;
}

// Last index i in [0, n) with first[i] <= x (first ascending, first[0] <= x).
__device__ __forceinline__ int last_at_most(const int* first, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

// The CTA, or the cluster's CTAs.
struct Team {
  int rank, ctas;
  __device__ Team() : rank(blockIdx.x), ctas(gridDim.x) {}
  __device__ __forceinline__ void sync() const {
    if (ctas > 1) cg::this_cluster().sync();
    else __syncthreads();
  }
  // `value` into place i of every CTA's array.  (Read by its own CTA after sync(): none leaves while another reads its memory.)
  __device__ __forceinline__ void tell(int* array, int i, int value) const {
    if (ctas == 1) array[i] = value;
    else
      for (int c = 0; c < ctas; ++c) *cg::this_cluster().map_shared_rank(array + i, c) = value;
  }
  __device__ __forceinline__ int first() const { return rank * blockDim.x + threadIdx.x; }
  __device__ __forceinline__ int stride() const { return ctas * blockDim.x; }
};

__device__ __forceinline__ void copy_counts(const int32_t* from, int32_t* to, int64_t n, const Team& team) {
  if (from == to) return;
#pragma unroll 4
  for (int64_t i = team.first(); i < n; i += team.stride()) to[i] = from[i];
}

// The table entries of the requests: entry x is of request b = last_at_most(first, B, x), page x - first[b].  For this thread's
// share, four side by side: page = load(b, j), then use(b, j, page).
template <class L, class U>
__device__ __forceinline__ void for_entries(const int* first, int B, int total, const Team& team, L load, U use) {
  constexpr int kDeep = 4;
  for (int x0 = team.first(); x0 < total; x0 += kDeep * team.stride()) {
    int b[kDeep], j[kDeep], page[kDeep];
#pragma unroll
    for (int i = 0; i < kDeep; ++i) {
      const int x = x0 + i * team.stride();
      b[i] = j[i] = page[i] = -1;
      if (x < total) {
        b[i] = last_at_most(first, B, x);
        j[i] = x - first[b[i]];
        page[i] = load(b[i], j[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < kDeep; ++i)
      if (b[i] >= 0) use(b[i], j[i], page[i]);
  }
}

__global__ void __launch_bounds__(kThreads) fork_kernel(const msa_fork_args p) {
  wait_for_stream();
  extern __shared__ int s_mem[];
  int* s_first = s_mem;                     // [F + 1] shared table entries of the forks before
  int* s_src = s_first + p.F + 1;           // [F] -1: not served
  int* s_dst = s_src + p.F;                 // [F]
  int* s_owner = s_dst + p.F;               // [B] the first fork that names a request
  const Team team;
  const int tid = threadIdx.x, F = p.F, threads = blockDim.x;
  const int64_t cap = p.max_pages * kBk;
  const int raw = *p.free_count;
  const int count = static_cast<int>(min(max(static_cast<int64_t>(raw), int64_t(0)), p.free_cap));
  int32_t err = raw == count ? 0 : MSA_DEVERR_NO_PAGES;
  for (int b = tid; b < p.B; b += threads) s_owner[b] = INT_MAX;
  __syncthreads();
  const int per = (F + threads - 1) / threads;
  int src[kPer], dst[kPer], L[kPer];
  int need = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int x = tid * per + i;
    src[i] = dst[i] = -1;
    if (i < per && x < F) {
      src[i] = p.src[x];
      dst[i] = p.dst[x];
    }
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    L[i] = 0;
    if (src[i] < 0) continue;
    if (src[i] >= p.B || dst[i] < 0 || dst[i] >= p.B || p.seq_len[dst[i]] != 0) {
      err |= MSA_DEVERR_BAD_ROW;
      src[i] = -1;
      continue;
    }
    L[i] = p.seq_len[src[i]];
    if (L[i] < 0 || L[i] > cap) {
      err |= MSA_DEVERR_BAD_LEN;
      src[i] = -1;
      continue;
    }
    atomicMin(&s_owner[dst[i]], tid * per + i);
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (src[i] < 0) continue;
    if (s_owner[dst[i]] != tid * per + i) {
      err |= MSA_DEVERR_BAD_ROW;
      src[i] = -1;
      continue;
    }
    need += L[i] % kBk != 0;
  }
  int pages_needed;
  int off = block_exclusive(need, &pages_needed);
  int share = 0;
  int page_at[kPer];                        // place on the stack of a fork's own page, -1: needs none
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    page_at[i] = -1;
    if (src[i] < 0) continue;
    if (L[i] % kBk != 0) {
      if (off >= count) {
        err |= MSA_DEVERR_NO_PAGES;
        src[i] = -1;
      } else {
        page_at[i] = count - 1 - off;
      }
      ++off;
    }
    if (src[i] >= 0) share += L[i] / kBk;
  }
  int total;
  int first = block_exclusive(share, &total);
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int x = tid * per + i;
    if (i < per && x < F) {
      s_first[x] = first;
      s_src[x] = src[i];
      s_dst[x] = dst[i];
      if (src[i] >= 0) first += L[i] / kBk;
    }
  }
  if (tid == 0) s_first[F] = total;
  copy_counts(p.page_shares, p.page_shares_out, p.num_pages, team);
  if (team.rank == 0 && err != 0) report(p.dev_err, err);
  // the last CTA, which has the fewest table entries, writes lengths, copies and the stack's height; lengths of all first
  int len[kPer];
  const int per_b = (p.B + threads - 1) / threads;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int b = tid + i * threads;
    len[i] = i < per_b && b < p.B ? p.seq_len[b] : 0;
  }
  bool bad = false;
  team.sync();                              // lengths, counts and the stack's height are read, counts copied
  if (team.rank == team.ctas - 1) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int b = tid + i * threads;
      if (i < per_b && b < p.B && (s_owner[b] == INT_MAX || s_src[s_owner[b]] < 0)) p.seq_len_out[b] = len[i];
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int x = tid * per + i;
      if (i >= per || x >= F) continue;
      int from = -1, to = -1;
      if (src[i] >= 0) {
        p.seq_len_out[dst[i]] = L[i];
        if (page_at[i] >= 0) {
          from = p.seq_pt[src[i] * p.max_pages + L[i] / kBk];
          to = p.free_pages[page_at[i]];
          p.seq_pt_out[dst[i] * p.max_pages + L[i] / kBk] = to;
          // a copy that msa_copy_pages cannot make, or takes for a row without one (a stack's height outside it is named already)
          bad |= from < 0 || from >= p.num_pages || (raw == count && (to < 0 || to >= p.num_pages));
        }
      }
      p.copy_src[x] = from;
      p.copy_dst[x] = to;
    }
    if (tid == 0) *p.free_count_out = count - min(pages_needed, count);
  }
  for_entries(
      s_first, F, total, team, [&](int x, int j) { return p.seq_pt[s_src[x] * p.max_pages + j]; },
      [&](int x, int j, int page) {
        p.seq_pt_out[s_dst[x] * p.max_pages + j] = page;
        if (page >= 0 && page < p.num_pages) atomicAdd(p.page_shares_out + page, 1);
        else bad = true;
      });
  if (bad) report(p.dev_err, MSA_DEVERR_BAD_PAGE);
}

// The pages of one thread, when all threads share the pool's: [lo, hi), in order.
__device__ __forceinline__ void own_pages(int64_t num_pages, const Team& team, int* lo, int* hi) {
  const int64_t per = (num_pages + team.stride() - 1) / team.stride();
  const int64_t at = static_cast<int64_t>(team.first()) * per;
  *lo = static_cast<int>(min(at, num_pages));
  *hi = static_cast<int>(min(at + per, num_pages));
}
// f(x, value) for these pages, in order, kOwn values loaded together.
template <class F>
__device__ __forceinline__ void for_pages(const int32_t* values, int lo, int hi, F f) {
  for (int x0 = lo; x0 < hi; x0 += kOwn) {
    int v[kOwn];
#pragma unroll
    for (int i = 0; i < kOwn; ++i) v[i] = x0 + i < hi ? __ldcg(values + x0 + i) : 0;
#pragma unroll
    for (int i = 0; i < kOwn; ++i)
      if (x0 + i < hi) f(x0 + i, v[i]);
  }
}

__global__ void __launch_bounds__(kAlone) release_shared_kernel(const msa_release_shared_args p) {
  wait_for_stream();
  extern __shared__ int s_first[];          // [B + 1] table entries of the ended requests before
  __shared__ int s_back[kCluster];          // pages that come back, of each CTA
  const Team team;
  const int tid = threadIdx.x, B = p.B, threads = blockDim.x;
  const int64_t cap = p.max_pages * kBk;
  const int raw = *p.free_count;
  const int64_t count = min(max(static_cast<int64_t>(raw), int64_t(0)), p.free_cap);
  int32_t err = raw == count ? 0 : MSA_DEVERR_NO_PAGES;
  const int per = (B + threads - 1) / threads;
  int len[kPer], gone[kPer], sum = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int b = tid * per + i;
    len[i] = gone[i] = 0;
    if (i < per && b < B) {
      len[i] = p.seq_len[b];
      if (p.done[b] != 0) {
        if (len[i] < 0 || len[i] > cap) {
          err |= MSA_DEVERR_BAD_LEN;
        } else {
          gone[i] = (len[i] + kBk - 1) / kBk;
          len[i] = 0;
        }
      }
      sum += gone[i];
    }
  }
  copy_counts(p.page_shares, p.page_shares_out, p.num_pages, team);
  int total;
  int first = block_exclusive(sum, &total);
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int b = tid * per + i;
    if (i < per && b < B) s_first[b] = first;
    first += gone[i];
  }
  if (tid == 0) s_first[B] = total;
  team.sync();                              // counts copied, lengths and the stack's height read
  if (team.rank == team.ctas - 1) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int b = tid * per + i;
      if (i < per && b < B) p.seq_len_out[b] = len[i];
    }
  }
  bool bad = false;
  for_entries(
      s_first, B, total, team, [&](int b, int j) { return p.seq_pt[b * p.max_pages + j]; },
      [&](int, int, int page) {
        if (page >= 0 && page < p.num_pages) atomicSub(p.page_shares_out + page, 1);
        else bad = true;
      });
  team.sync();                              // every holder that ended is taken off
  int lo, hi, back = 0;
  own_pages(p.num_pages, team, &lo, &hi);
  for_pages(p.page_shares_out, lo, hi, [&](int, int left) { back += left < 0 ? 1 : 0; });
  int in_cta;
  int before = block_exclusive(back, &in_cta);
  if (tid == 0) team.tell(s_back, team.rank, in_cta);
  team.sync();
  int all = 0;
  for (int c = 0; c < team.ctas; ++c) {
    if (c < team.rank) before += s_back[c];
    all += s_back[c];
  }
  int64_t to = count + before;
  if (back > 0)
    for_pages(p.page_shares_out, lo, hi, [&](int x, int left) {
      if (left >= 0) return;
      bad |= left < -1;                     // given up more often than it was held
      p.page_shares_out[x] = 0;
      if (to < p.free_cap) p.free_pages[to] = x;
      ++to;
    });
  if (count + all > p.free_cap) err |= MSA_DEVERR_NO_PAGES;
  if (team.rank == 0 && tid == 0) *p.free_count_out = static_cast<int>(min(count + all, p.free_cap));
  if (bad) err |= MSA_DEVERR_BAD_PAGE;
  if ((bad || team.rank == 0) && err != 0) report(p.dev_err, err);
}

__global__ void __launch_bounds__(kAlone) compact_kernel(const msa_compact_args p) {
  wait_for_stream();
  extern __shared__ int s_first[];          // [B + 1] table entries of the requests before
  __shared__ int s_used[kCluster], s_low[1];   // pages in use: of each CTA's share, and among the first n
  const Team team;
  const int tid = threadIdx.x, B = p.B, threads = blockDim.x;
  const int64_t cap = p.max_pages * kBk, P = p.num_pages;
  int32_t err = 0;
  int32_t* const place = p.free_pages;      // until the end: whether a page is in use, then where it goes
  const int per = (B + threads - 1) / threads;
  int pages[kPer], sum = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int b = tid * per + i;
    pages[i] = 0;
    if (i < per && b < B) {
      const int L = p.seq_len[b];
      if (L < 0 || L > cap) err |= MSA_DEVERR_BAD_LEN;
      else pages[i] = (L + kBk - 1) / kBk;
    }
    sum += pages[i];
  }
  for (int64_t x = team.first(); x < P; x += team.stride()) {
    place[x] = 0;
    p.move_src[x] = -1;
    p.move_dst[x] = -1;
  }
  int total;
  int first = block_exclusive(sum, &total);
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int b = tid * per + i;
    if (i < per && b < B) s_first[b] = first;
    first += pages[i];
  }
  if (tid == 0) {
    s_first[B] = total;
    s_low[0] = 0;
  }
  team.sync();
  for_entries(
      s_first, B, total, team, [&](int b, int j) { return p.seq_pt[b * p.max_pages + j]; },
      [&](int, int, int page) {
        if (page >= 0 && page < P) place[page] = 1;
        else err |= MSA_DEVERR_BAD_PAGE;
      });
  team.sync();                              // every page in use is marked
  int lo, hi, used = 0;
  own_pages(P, team, &lo, &hi);
  for_pages(place, lo, hi, [&](int, int live) { used += live; });
  int in_cta;
  int before = block_exclusive(used, &in_cta);
  if (tid == 0) team.tell(s_used, team.rank, in_cta);
  team.sync();
  int n = 0;                                // pages in use: they end up as 0 .. n - 1
  for (int c = 0; c < team.ctas; ++c) {
    if (c < team.rank) before += s_used[c];
    n += s_used[c];
  }
  // The k-th page in use behind the first n goes to the k-th free one among them.  Where the first n end, the pages in use
  // before give the first rank behind.
  int rank = before;
  for_pages(place, lo, hi, [&](int x, int live) {
    if (x == n) team.tell(s_low, 0, rank);
    if (live == 0 && x < n) p.move_dst[x - rank] = x;
    rank += live;
  });
  team.sync();                              // the free places are known
  const int low = s_low[0];
  rank = before;
  for_pages(place, lo, hi, [&](int x, int live) {
    const int shares = live != 0 ? p.page_shares[x] : 0;
    if (x >= n) p.page_shares_out[x] = 0;
    if (live == 0) return;
    int to = x;
    if (x >= n) {
      to = __ldcg(p.move_dst + (rank - low));
      p.move_src[rank - low] = x;
    }
    place[x] = to;
    p.page_shares_out[to] = shares;
    ++rank;
  });
  team.sync();                              // where each page goes is known
  for_entries(
      s_first, B, total, team, [&](int b, int j) { return p.seq_pt[b * p.max_pages + j]; },
      [&](int b, int j, int page) { p.seq_pt_out[b * p.max_pages + j] = page >= 0 && page < P ? __ldcg(place + page) : page; });
  team.sync();                              // the places are read: the stack takes their room
  for (int64_t x = team.first(); x < p.free_cap; x += team.stride()) p.free_pages[x] = x < P - n ? static_cast<int32_t>(P - 1 - x) : -1;
  if (team.rank == 0 && tid == 0) *p.free_count = static_cast<int32_t>(P - n);
  if (err != 0) report(p.dev_err, err);
}

// smem: of this call, at most `most` (of any call).  The kernel's limit is the same in every call: it belongs to the kernel, and
// another thread's call of fewer requests must not lower it before this launch.
template <class Args>
msa_status launch_team(void (*kernel)(const Args), const Args& a, bool alone, size_t smem, size_t most, cudaStream_t stream, const char* what) {
  if (smem > (40u << 10)) {                 // with the sums' own shared memory past the 48 KiB default
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(most));
    if (e != cudaSuccess) return cuda_fail(e, what);
  }
  const int ctas = alone ? 1 : kCluster;
  const cudaError_t e = launch_early(kernel, ctas, alone ? kAlone : kThreads, smem, stream, ctas, a);
  if (e != cudaSuccess) return cuda_fail(e, what);
  return MSA_OK;
}

struct CopyParams {
  int64_t n, num_pages;
  const int32_t *src, *dst;
  int pools;
  int first[MSA_MAX_POOLS + 1];             // chunks of the pools before
  uint8_t* base[MSA_MAX_POOLS];
  int64_t stride[MSA_MAX_POOLS], bytes[MSA_MAX_POOLS];
  int32_t* dev_err;
};

template <class T>
__device__ __forceinline__ void copy_units(const uint8_t* from, uint8_t* to, int64_t units) {
  const T* a = reinterpret_cast<const T*>(from) + threadIdx.x;
  T* b = reinterpret_cast<T*>(to) + threadIdx.x;
  for (int64_t u = threadIdx.x; u < units; u += kCopyThreads * kCopyUnroll, a += kCopyThreads * kCopyUnroll, b += kCopyThreads * kCopyUnroll) {
    T v[kCopyUnroll];
#pragma unroll
    for (int i = 0; i < kCopyUnroll; ++i)
      if (u + i * kCopyThreads < units) v[i] = a[i * kCopyThreads];
#pragma unroll
    for (int i = 0; i < kCopyUnroll; ++i)
      if (u + i * kCopyThreads < units) b[i * kCopyThreads] = v[i];
  }
}

// A CTA copies one chunk of a page (its place in x: pool and bytes are settled once) for its share of the pairs (y),
// of which it looks at 32 at a time, so that rows without a pair cost little.
__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(const __grid_constant__ CopyParams p) {
  wait_for_stream();
  int pool = 0;
  while (pool + 1 < p.pools && static_cast<int>(blockIdx.x) >= p.first[pool + 1]) ++pool;
  const int64_t at = static_cast<int64_t>(blockIdx.x - p.first[pool]) * kCopyChunk, bytes = min(p.bytes[pool] - at, static_cast<int64_t>(kCopyChunk));
  uint8_t* base = p.base[pool] + at;
  const int64_t stride = p.stride[pool];
  const bool wide = ((reinterpret_cast<uintptr_t>(base) | stride | bytes) & 15) == 0;
  const int lane = threadIdx.x & 31;
  for (int64_t i0 = blockIdx.y; i0 < p.n; i0 += 32 * gridDim.y) {
    const int64_t i = i0 + lane * gridDim.y;
    int from = -1, to = -1;
    if (i < p.n) {
      from = p.src[i];
      to = p.dst[i];
    }
    const bool some = from >= 0 && to >= 0, good = some && from < p.num_pages && to < p.num_pages;
    if (some && !good && blockIdx.x == 0 && threadIdx.x < 32) report(p.dev_err, MSA_DEVERR_BAD_PAGE);
    for (uint32_t todo = __ballot_sync(0xffffffffu, good); todo != 0; todo &= todo - 1) {
      const int k = __ffs(todo) - 1;
      const int a = __shfl_sync(0xffffffffu, from, k), b = __shfl_sync(0xffffffffu, to, k);
      if (wide) copy_units<uint4>(base + a * stride, base + b * stride, bytes / 16);
      else copy_units<uint8_t>(base + a * stride, base + b * stride, bytes);
    }
  }
}

}  // namespace

msa_status launch_fork(const msa_fork_args& a, cudaStream_t stream) {
  const size_t smem = (3 * static_cast<size_t>(a.F) + a.B + 1) * sizeof(int);
  return launch_team(fork_kernel, a, false, smem, (4 * kMaxDecodeBatch + 1) * sizeof(int), stream, "fork_kernel launch");
}

constexpr size_t kTableSmem = (kMaxDecodeBatch + 1) * sizeof(int);

msa_status launch_release_shared(const msa_release_shared_args& a, cudaStream_t stream) {
  const size_t smem = (static_cast<size_t>(a.B) + 1) * sizeof(int);
  const bool alone = std::max<int64_t>(static_cast<int64_t>(a.B) * a.max_pages / 8, a.num_pages) <= kAloneItems;
  return launch_team(release_shared_kernel, a, alone, smem, kTableSmem, stream, "release_shared_kernel launch");
}

msa_status launch_compact(const msa_compact_args& a, cudaStream_t stream) {
  const size_t smem = (static_cast<size_t>(a.B) + 1) * sizeof(int);
  return launch_team(compact_kernel, a, a.num_pages <= kAloneItems, smem, kTableSmem, stream, "compact_kernel launch");
}

msa_status launch_copy_pages(const msa_copy_pages_args& a, cudaStream_t stream) {
  DeviceInfo dev;
  if (msa_status st = current_device(&dev); st != MSA_OK) return st;
  CopyParams p = {};
  p.n = a.n; p.num_pages = a.num_pages;
  p.src = a.src; p.dst = a.dst;
  p.pools = a.pools;
  for (int i = 0; i < a.pools; ++i) {
    p.base[i] = static_cast<uint8_t*>(a.pool[i]);
    p.stride[i] = a.page_stride[i];
    p.bytes[i] = a.page_bytes[i];
    p.first[i + 1] = p.first[i] + static_cast<int>((a.page_bytes[i] + kCopyChunk - 1) / kCopyChunk);
  }
  p.dev_err = a.dev_err;
  const int chunks = p.first[a.pools];
  const int64_t share = std::max<int64_t>(1, 8 * dev.num_sms / chunks);
  const dim3 grid(static_cast<unsigned>(chunks), static_cast<unsigned>(std::min<int64_t>(std::min(a.n, share), 65535)));
  const cudaError_t e = launch_early(copy_pages_kernel, grid, kCopyThreads, 0, stream, 1, p);
  if (e != cudaSuccess) return cuda_fail(e, "copy_pages_kernel launch");
  return MSA_OK;
}

}  // namespace msa
