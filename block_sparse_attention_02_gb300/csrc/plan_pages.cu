// plan_pages.cu -- page tables and token slots from request lengths, and the
// return of ended requests' pages.
//
// Fixed-size pages ("MiniMax M3 preparado para inferencia en produccion",
// paragraph "MSA con paged attention") leave a serving loop an index problem
// before every step: with have = ceil(L / Bk) and need = ceil((L + n) / Bk) - have
// per request, prefix sums of n give each request its token rows and prefix
// sums of need its pages on the free stack.  The sums run over at most 4096
// requests, so every CTA forms them for itself in shared memory and then fills its
// share of the token rows and table entries by binary search in the sums: no
// second launch and no scratch.  Lengths and the stack's height may be updated
// in place; the CTAs then form one thread-block cluster, whose barrier tells that all
// of them have read the old values.  With outputs of their own there is nothing to
// wait for and the grid is as large as the rows ask for.
//
// Bound: latency (the lengths, the sums, one page id per row, the stores); the
// 16 bytes written per token row are far below it.  8 requests 2.9 us, one kernel after
// another; with the release of ended requests, two launches, 64 requests (0.5 MB of rows and
// table entries) 6.2 us, 1,024 requests (1.1 MB) 7.9 us.
#include <cooperative_groups.h>

#include <climits>

#include "launch_early.cuh"
#include "msa_internal.h"
#include "msa_ptx.cuh"

namespace cg = cooperative_groups;

namespace msa {
namespace {

constexpr int kPlanThreads = 512;
constexpr int kPerThread = kMaxDecodeBatch / kPlanThreads;   // requests per thread in the prefix sums, at most
constexpr int kPlanCluster = 8;                              // CTAs of an update in place (portable maximum)

// Exclusive prefix sums of (a, b) over the CTA's threads; returns the totals.
struct Sum2 {
  int64_t a, b;
};
__device__ __forceinline__ Sum2 block_exclusive(Sum2 v, Sum2* total) {
  __shared__ Sum2 s_warp[kPlanThreads / 32 + 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  Sum2 inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t a = __shfl_up_sync(0xffffffffu, inc.a, o), b = __shfl_up_sync(0xffffffffu, inc.b, o);
    if (lane >= o) { inc.a += a; inc.b += b; }
  }
  if (lane == 31) s_warp[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    Sum2 w = lane < warps ? s_warp[lane] : Sum2{0, 0};
    const Sum2 own = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t a = __shfl_up_sync(0xffffffffu, w.a, o), b = __shfl_up_sync(0xffffffffu, w.b, o);
      if (lane >= o) { w.a += a; w.b += b; }
    }
    if (lane < warps) s_warp[lane] = Sum2{w.a - own.a, w.b - own.b};
    if (lane == 31) s_warp[kPlanThreads / 32] = w;
  }
  __syncthreads();
  *total = s_warp[kPlanThreads / 32];
  return Sum2{s_warp[warp].a + inc.a - v.a, s_warp[warp].b + inc.b - v.b};
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

__global__ void __launch_bounds__(kPlanThreads) plan_step_kernel(const msa_plan_args p, const bool in_place) {
  wait_for_stream();
  extern __shared__ int s_plan[];
  int* s_cu = s_plan;                       // [B + 1] first token row, at most N
  int* s_off = s_cu + p.B + 1;              // [B + 1] pages given to the requests before b
  int* s_len = s_off + p.B + 1;             // [B] cached tokens; -1: not served
  const int tid = threadIdx.x, B = p.B, rank = blockIdx.x, ctas = gridDim.x;
  const int per = (B + blockDim.x - 1) / blockDim.x;   // <= kPerThread
  const int64_t cap = p.max_pages * kBk;
  const int raw = *p.free_count;
  const int count = static_cast<int>(min(max(static_cast<int64_t>(raw), int64_t(0)), p.free_cap));
  int32_t err = raw == count ? 0 : MSA_DEVERR_NO_PAGES;

  int L[kPerThread], n[kPerThread], need[kPerThread];
  Sum2 own{0, 0};
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    const int b = tid * per + i;
    L[i] = n[i] = need[i] = 0;
    if (i < per && b < B) {
      L[i] = p.seq_len[b];
      n[i] = p.new_len[b];
    }
  }
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    const int64_t end = static_cast<int64_t>(L[i]) + n[i];
    if (L[i] >= 0 && n[i] >= 0 && end <= cap)
      need[i] = static_cast<int>((end + kBk - 1) / kBk) - static_cast<int>((static_cast<int64_t>(L[i]) + kBk - 1) / kBk);
    own.a += max(n[i], 0);
    own.b += need[i];
  }
  Sum2 total;
  Sum2 before = block_exclusive(own, &total);
  if (total.a > p.N) {                      // rare: a request whose rows pass N needs no pages, so the sums change
    int64_t row = before.a;
    own.b = 0;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
      row += max(n[i], 0);
      if (row > p.N) need[i] = 0;
      own.b += need[i];
    }
    __syncthreads();                        // the first sums are read
    before = block_exclusive(own, &total);
  }
  {
    int64_t row = before.a, off = before.b;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
      const int b = tid * per + i;
      if (i < per && b < B) {
        const int64_t end = static_cast<int64_t>(L[i]) + n[i];
        const bool fits = L[i] >= 0 && n[i] >= 0 && end <= cap && row + n[i] <= p.N;
        const bool served = fits && (need[i] == 0 || off + need[i] <= count);
        if (!fits) err |= MSA_DEVERR_BAD_LEN;
        else if (!served) err |= MSA_DEVERR_NO_PAGES;
        s_cu[b] = static_cast<int>(min(row, p.N));
        // past the first refusal nothing that needs a page is served, so the sums
        // clamped to the stack's height stay exact for every served request
        s_off[b] = static_cast<int>(min(off, static_cast<int64_t>(count) + 1));
        s_len[b] = served ? L[i] : -1;
        row += max(n[i], 0);
        off += need[i];
      }
    }
  }
  const int64_t all_rows = total.a;
  if (tid == 0) {
    s_cu[B] = static_cast<int>(min(all_rows, p.N));
    s_off[B] = static_cast<int>(min(total.b, static_cast<int64_t>(count) + 1));
  }
  if (rank == 0 && err != 0) report(p.dev_err, err);
  __syncthreads();
  if (in_place && ctas > 1) cg::this_cluster().sync();   // every CTA has read the lengths and the stack's height

  const int stride = ctas * blockDim.x, first = rank * blockDim.x + tid;
  // lengths and offsets out, by the last CTA, which has the fewest rows
  if (rank == ctas - 1) {
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
      const int b = tid * per + i;
      if (i < per && b < B) p.seq_len_out[b] = L[i] + (s_len[b] >= 0 ? n[i] : 0);
    }
    for (int b = tid; b <= B; b += blockDim.x) p.cu[b] = s_cu[b];
  }
  // new table entries: item x of the pages given is entry have + (x - off_b) of request b.
  // A refused request ends the pages given; the ones before it are all served.
  const int entries = s_off[B];
  int given = 0;
  for (int x = first; x < min(entries, count); x += stride) {
    const int b = last_at_most(s_off, B, x);
    if (s_len[b] < 0) continue;             // the request that did not fit
    const int have = (s_len[b] + kBk - 1) / kBk;
    p.seq_pt[b * p.max_pages + have + (x - s_off[b])] = p.free_pages[count - 1 - x];
  }
  if (rank == ctas - 1 && tid == 0) {
    given = min(entries, count);
    if (entries > count) given = s_off[last_at_most(s_off, B, count)];   // pages before the first refusal
    *p.free_count_out = count - given;
  }
  // token rows
  const int used = s_cu[B];
  bool bad = false;
  for (int64_t r = first; r < p.N; r += stride) {
    int64_t slot = -1;
    int pos = -1, seq = -1;
    if (r < used) {
      const int b = last_at_most(s_cu, B, static_cast<int>(r));
      if (s_len[b] >= 0) {
        seq = b;
        pos = s_len[b] + static_cast<int>(r) - s_cu[b];
        const int have = (s_len[b] + kBk - 1) / kBk, j = pos / kBk;
        const int page = j >= have ? p.free_pages[count - 1 - (s_off[b] + j - have)] : p.seq_pt[b * p.max_pages + j];
        if (page >= 0 && page < p.num_pages) slot = static_cast<int64_t>(page) * kBk + pos % kBk;
        else bad = true;
      }
    }
    p.tok_slot[r] = slot;
    p.tok_pos[r] = pos;
    if (p.tok_seq != nullptr) p.tok_seq[r] = seq;
  }
  if (bad) report(p.dev_err, MSA_DEVERR_BAD_PAGE);
}

__global__ void __launch_bounds__(kPlanThreads) release_kernel(const msa_release_args p, const bool in_place) {
  wait_for_stream();
  extern __shared__ int s_off[];            // [B + 1] pages returned by the requests before b
  const int tid = threadIdx.x, B = p.B, rank = blockIdx.x, ctas = gridDim.x;
  const int per = (B + blockDim.x - 1) / blockDim.x;
  const int64_t cap = p.max_pages * kBk;
  const int raw = *p.free_count;
  const int64_t count = min(max(static_cast<int64_t>(raw), int64_t(0)), p.free_cap);
  int32_t err = raw == count ? 0 : MSA_DEVERR_NO_PAGES;
  int out_len[kPerThread], gone[kPerThread];
  Sum2 own{0, 0}, total;
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    const int b = tid * per + i;
    out_len[i] = gone[i] = 0;
    if (i < per && b < B) {
      out_len[i] = p.seq_len[b];
      if (p.done[b] != 0) {
        if (out_len[i] < 0 || out_len[i] > cap) {
          err |= MSA_DEVERR_BAD_LEN;
        } else {
          gone[i] = static_cast<int>((static_cast<int64_t>(out_len[i]) + kBk - 1) / kBk);
          out_len[i] = 0;
        }
      }
      own.a += gone[i];
    }
  }
  int64_t off = block_exclusive(own, &total).a;
  const int64_t room = p.free_cap - count;
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    const int b = tid * per + i;
    if (i < per && b < B) {
      s_off[b] = static_cast<int>(min(off, room));
      off += gone[i];
    }
  }
  const int64_t back = min(total.a, room);
  if (total.a > room) err |= MSA_DEVERR_NO_PAGES;
  if (rank == 0 && err != 0) report(p.dev_err, err);
  __syncthreads();
  if (in_place && ctas > 1) cg::this_cluster().sync();
  if (rank == 0) {
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
      const int b = tid * per + i;
      if (i < per && b < B) p.seq_len_out[b] = out_len[i];
    }
    if (tid == 0) *p.free_count_out = static_cast<int>(count + back);
  }
  bool bad = false;
  for (int64_t x = rank * blockDim.x + tid; x < back; x += ctas * blockDim.x) {
    const int b = last_at_most(s_off, B, static_cast<int>(x));
    const int page = p.seq_pt[b * p.max_pages + (x - s_off[b])];
    bad |= page < 0 || (p.num_pages != 0 && page >= p.num_pages);
    p.free_pages[count + x] = page;
  }
  if (bad) report(p.dev_err, MSA_DEVERR_BAD_PAGE);
}

// One CTA, a plain grid, or (an update in place with more than one CTA's rows) one cluster.
template <class Args>
msa_status launch_rows(void (*kernel)(const Args, const bool), const Args& a, int64_t items, bool in_place, size_t smem,
                       cudaStream_t stream, const char* what) {
  DeviceInfo dev;
  if (msa_status st = current_device(&dev); st != MSA_OK) return st;
  // enough threads for the sums (8 requests each at most), few for the small steps that come once a token
  const int threads = a.B > 512 ? kPlanThreads : a.B > 128 ? 256 : 128;
  const int64_t want = std::max<int64_t>((items + threads - 1) / threads, 1);
  const int ctas = static_cast<int>(std::min<int64_t>(want, in_place ? kPlanCluster : 2 * dev.num_sms));
  if (smem > (40u << 10)) {   // with the prefix sums' own shared memory past the 48 KiB default
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return cuda_fail(e, what);
  }
  const cudaError_t e = launch_early(kernel, ctas, threads, smem, stream, in_place ? ctas : 1, a, in_place);
  if (e != cudaSuccess) return cuda_fail(e, what);
  return MSA_OK;
}

}  // namespace

msa_status launch_plan_step(const msa_plan_args& a, cudaStream_t stream) {
  const bool in_place = a.seq_len_out == a.seq_len || a.free_count_out == a.free_count;
  const size_t smem = (3 * static_cast<size_t>(a.B) + 2) * sizeof(int);
  return launch_rows(plan_step_kernel, a, a.N, in_place, smem, stream, "plan_step_kernel launch");
}

msa_status launch_release_pages(const msa_release_args& a, cudaStream_t stream) {
  const bool in_place = a.seq_len_out == a.seq_len || a.free_count_out == a.free_count;
  const size_t smem = (static_cast<size_t>(a.B) + 1) * sizeof(int);
  // at most B * max_pages pages come back, a few of the requests' as a rule
  return launch_rows(release_kernel, a, static_cast<int64_t>(a.B) * a.max_pages / 8, in_place, smem, stream,
                     "release_kernel launch");
}

}  // namespace msa
