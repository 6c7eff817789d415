// window_prefill.cu -- attention of many queries through a sliding window with sinks, over contiguous tensors (a
// prompt) or pages (a chunk after a cached prefix, draft tokens).
//
//     O[i, h] = sum_t softmax_t(scale * Q[i, h] . K[t]) V[t],  LSE[i, h] = ln sum_t e^(..),
//     t <= i with t > i - window or t < sinks.
//
// A tile is 128 rows of one KV head: nq = 128 / G queries with all their G heads (126 rows for G = 6), row = query * G +
// head.  So a tile's queries are few and their windows nearly one: it needs window / 128 + 1.2 blocks of 128 keys where 128
// queries of one head need window / 128 + 2 (blocks start at multiples of 128, as pages do), and a handful of queries
// (draft tokens) is one tile.  Two neighbouring tiles ("slots") share a stream of K/V blocks: the sinks' blocks, then those
// from the window's first key on.
//   S  = Q K_j^T   M = 128 rows, N = 128 keys, K = D   (tensor memory, 128 columns)
//   softmax (thread = row): block max, P = 2^(S * scale * log2 e - m) written back over S as bf16 pairs
//   O += P V_j     M = 128, N = D, K = 128 keys, P read from tensor memory (128 columns)
// The running max m is updated lazily: O and the running sum are rescaled only when a block's max exceeds m by more than
// 2^8, so P <= 256 and the result is exact whichever m is used.  Blocks that some row does not see whole are masked.
//
// Roles: warp 0 TMA of K and V (a ring of 32 KiB units, K and V apart), warp 1 tcgen05 issuer, warps 2-5 and 6-9 the two
// slots' softmax and epilogue; a slot's softmax also sends for its next Q tile, once its last S is done.  Each slot goes
// through its items on its own: S(j + 1) is issued right behind O(j), which reads P from the same columns (one thread's
// MMAs run in order), and the other slot's products run meanwhile.
#include <algorithm>
#include <climits>
#include <type_traits>

#include "msa_internal.h"
#include "msa_ptx.cuh"

namespace msa {
namespace {

constexpr int kHalf = 128 * 64 * 2;          // 16 KiB: 128 rows x 64 bf16
constexpr int kUnit = 2 * kHalf;             // 32 KiB: a tile of Q, K or V
constexpr int kUnits = 5;                    // of K and V in shared memory
constexpr int kNotes = 8;                    // blocks whose page's state is kept (more than are in flight)
constexpr int kThreads = 320;                // w0 TMA, w1 MMA, w2-5 slot 0, w6-9 slot 1
constexpr int kTmemCols = 512;               // per slot: S / P (128 columns) and O (128 columns)
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescale = 8.0f;             // log2 of the largest P before the running max moves
constexpr float kFusedMost = 16777216.f;     // scores up to which scale and max go into one rounding

struct Params {
  int B, S, Hq, Hkv, G, nq, pairs;           // nq: queries of a tile; pairs: pairs of tiles of a sequence
  int window, sinks;
  int n_items;
  float scale_log2;
  int paged;
  int64_t num_pages, max_pages;
  const int32_t *seq_pt, *q_pos;
  __nv_bfloat16* O;                          // [B, S, Hq, D] dense
  float* LSE;                                // [B, S, Hq] dense, or null
  int32_t* dev_err;
};

// A pair of tiles: queries q0 .. of sequence b, head g, at positions pos ..; blocks: sink_blocks ones from 0 on, then from
// `first` on.
struct Item {
  int b, g, q0, pos, tiles, sink_blocks, first, blocks;
  __device__ __forceinline__ int block(int j) const { return j < sink_blocks ? j : j - sink_blocks + first; }
};
// The pairs with the most blocks first: from the last to the first of a sequence.
__device__ __forceinline__ Item item_of(const Params& p, int it) {
  Item x;
  const int heads = p.B * p.Hkv;
  const int pair = p.pairs - 1 - it / heads;
  const int rest = it % heads;
  x.g = rest % p.Hkv;
  x.b = rest / p.Hkv;
  x.q0 = pair * 2 * p.nq;
  x.tiles = x.q0 + p.nq < p.S ? 2 : 1;
  const int start = p.paged ? p.q_pos[x.b] : 0;
  x.pos = start + x.q0;
  if (p.paged && (start < 0 || start + static_cast<int64_t>(p.S) > p.max_pages * kBk)) {
    x.sink_blocks = x.first = x.blocks = 0;
    return x;
  }
  const int last = start + min(x.q0 + 2 * p.nq, p.S) - 1;
  x.first = max(x.pos - p.window + 1, 0) / kBk;
  x.sink_blocks = min((min(p.sinks, last + 1) + kBk - 1) / kBk, x.first);
  x.blocks = x.sink_blocks + last / kBk - x.first + 1;
  return x;
}

__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  __nv_bfloat162 h2 = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h2);
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
                 "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
               : "r"(taddr));
}
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float* lo, float* hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(*lo), "=f"(*hi) : "l"(v)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

__global__ void __launch_bounds__(kThreads, 1)
window_prefill_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                      const __grid_constant__ CUtensorMap vmap, const Params p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* s_q = smem;                       // [2] Q tiles
  uint8_t* s_kv = smem + 2 * kUnit;          // [kUnits] of K and V: unit 2 n is K of the CTA's n-th block, 2 n + 1 its V

  __shared__ __align__(8) uint64_t bar_qfull[2], bar_full[kUnits], bar_empty[kUnits];
  __shared__ __align__(8) uint64_t bar_sfull[2], bar_pready[2], bar_ofull[2], bar_drain;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ volatile int s_gone[kNotes];    // of block n % kNotes: no such page

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < kUnits; ++i) { mbar_init(&bar_full[i], 1); mbar_init(&bar_empty[i], 1); }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar_qfull[i], 1);
      mbar_init(&bar_sfull[i], 1); mbar_init(&bar_pready[i], 4); mbar_init(&bar_ofull[i], 1);
    }
    mbar_init(&bar_drain, 1);
    s_abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(&s_tmem, kTmemCols);
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  volatile int* abort_flag = &s_abort;

  if (warp == 0) {
    // ===================== TMA producer of K and V (warp-uniform loop, lane 0 issues) =====================
    int n = 0;                               // blocks sent for
    bool ok = true;
    for (int it = blockIdx.x; it < p.n_items && ok; it += gridDim.x) {
      const Item x = item_of(p, it);
      for (int j0 = 0; j0 < x.blocks && ok; j0 += 32) {
        // lane l looks up the page of block j0 + l
        int pg = 0;
        if (p.paged && j0 + lane < x.blocks) pg = p.seq_pt[x.b * p.max_pages + x.block(j0 + lane)];
        for (int i = 0; i < 32 && j0 + i < x.blocks; ++i, ++n) {
          const int page = __shfl_sync(0xffffffffu, pg, i);
          int go = 1;
          if (lane == 0) {
            const bool gone = p.paged && (page < 0 || page >= p.num_pages);
            // a page that there is not is read as zeros: from past the end of the pool
            const int c1 = p.paged ? 0 : x.g, c2 = p.paged ? x.g : x.block(j0 + i) * kBk;
            const int c3 = p.paged ? (gone ? static_cast<int>(p.num_pages) : page) : x.b;
            for (int kv = 0; kv < 2 && go; ++kv) {
              const int u = 2 * n + kv, st = u % kUnits;
              go = mbar_wait(&bar_empty[st], ((u / kUnits) & 1) ^ 1, abort_flag, p.dev_err);
              if (!go) break;
              if (kv == 0) s_gone[n % kNotes] = gone;
              uint8_t* to = s_kv + st * kUnit;
              mbar_arrive_expect_tx(&bar_full[st], kUnit);
              tma_load_4d(to, kv ? &vmap : &kmap, &bar_full[st], 0, c1, c2, c3);
              tma_load_4d(to + kHalf, kv ? &vmap : &kmap, &bar_full[st], 64, c1, c2, c3);
            }
            if (gone) report(p.dev_err, MSA_DEVERR_BAD_PAGE);
          }
          if (!__shfl_sync(0xffffffffu, go, 0)) {
            ok = false;
            break;
          }
        }
      }
    }
    if (lane == 0 && *abort_flag) {          // let loads in flight land before the CTA exits
      const uint64_t t0 = global_timer_ns();
      for (int u = max(0, 2 * n - kUnits); u < 2 * n; ++u)
        while (!mbar_try_wait(&bar_full[u % kUnits], (u / kUnits) & 1) && global_timer_ns() - t0 < MSA_WAIT_LIMIT_NS) {
        }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ===================== tcgen05 issuer =====================
    // Per slot: S(j) of its item needs K(j), the item's Q tile (j = 0) and O(j - 1) issued before it; O(j) needs P(j) and
    // V(j).  Whatever is ready is issued.
    if (lane == 0) {
      constexpr uint32_t idesc_s = idesc_bf16(128, 128, false, false);
      constexpr uint32_t idesc_o = idesc_bf16(128, 128, false, true);
      int it[2];
      int j[2] = {0, 0}, blocks[2] = {0, 0};  // the slot's next block of its item, and the item's blocks
      int ns[2] = {0, 0}, no[2] = {0, 0};     // blocks of the CTA whose S / O is issued, or that the slot sits out
      int waits[2] = {0, 0}, items[2] = {0, 0};   // S issued; items begun (phases of pready and qfull)
      bool pending[2] = {false, false};       // S issued, O not yet
      int free_k = 0, free_v = 0;             // blocks whose unit is given back
      constexpr int kEnd = INT_MAX / 2;       // ns and no of a slot that has no item left
      // the slot's next item, from item `i` on; the blocks of one that has no tile for it pass at once
      auto take_item = [&](int s, int i) {
        j[s] = 0;
        for (; i < p.n_items; i += gridDim.x) {
          const Item x = item_of(p, i);
          blocks[s] = x.blocks;
          if (x.blocks > 0 && s < x.tiles) break;
          ns[s] += x.blocks;
          no[s] += x.blocks;
        }
        it[s] = i;
        if (i >= p.n_items) ns[s] = no[s] = kEnd;
      };
      // units that both slots have read (or will not) are free when the products issued so far are done
      auto give_back = [&] {
        for (const int n = min(ns[0], ns[1]); free_k < n && n < kEnd; ++free_k) umma_commit(&bar_empty[2 * free_k % kUnits]);
        for (const int n = min(no[0], no[1]); free_v < n && n < kEnd; ++free_v) umma_commit(&bar_empty[(2 * free_v + 1) % kUnits]);
      };
      take_item(0, blockIdx.x);
      take_item(1, blockIdx.x);
      uint32_t spins = 0;
      uint64_t idle_since = 0;
      while (it[0] < p.n_items || it[1] < p.n_items) {
        bool progress = false;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          if (it[s] >= p.n_items) continue;
          if (pending[s] && mbar_test_wait(&bar_pready[s], (waits[s] - 1) & 1)) {
            const int u = 2 * no[s] + 1, st = u % kUnits;
            if (mbar_test_wait(&bar_full[st], (u / kUnits) & 1)) {
              tc_fence_after();
              const uint32_t vb = smem_u32(s_kv + st * kUnit);
#pragma unroll
              for (int kk = 0; kk < 8; ++kk)
                umma_bf16_ts(tmem + s * 256 + 128, tmem + s * 256 + kk * 8, sdesc_sw128(vb + kk * 2048, kHalf, 1024), idesc_o,
                             (j[s] > 0 || kk > 0) ? 1u : 0u);
              ++no[s];
              pending[s] = false;
              if (++j[s] == blocks[s]) {
                umma_commit(&bar_ofull[s]);
                take_item(s, it[s] + gridDim.x);
              }
              give_back();
              progress = true;
              if (it[s] >= p.n_items) continue;
            }
          }
          // (a slot is a block ahead of the other at most: further on, a unit's phase could be taken for the one before last)
          if (!pending[s] && ns[s] <= ns[1 - s] + 1) {
            const int u = 2 * ns[s], st = u % kUnits;
            if ((j[s] > 0 || mbar_test_wait(&bar_qfull[s], items[s] & 1)) && mbar_test_wait(&bar_full[st], (u / kUnits) & 1)) {
              tc_fence_after();
              if (j[s] == 0) ++items[s];
              const uint32_t qb = smem_u32(s_q + s * kUnit), kb = smem_u32(s_kv + st * kUnit);
#pragma unroll
              for (int kk = 0; kk < 8; ++kk)
                umma_bf16(tmem + s * 256, sdesc_sw128(qb + (kk >> 2) * kHalf + 32 * (kk & 3), 16, 1024),
                          sdesc_sw128(kb + (kk >> 2) * kHalf + 32 * (kk & 3), 16, 1024), idesc_s, kk > 0);
              umma_commit(&bar_sfull[s]);
              ++ns[s];
              ++waits[s];
              pending[s] = true;
              give_back();
              progress = true;
            }
          }
        }
        if (progress) {
          spins = 0;
        } else if ((++spins & 63u) == 0) {
          const uint64_t now = global_timer_ns();
          if (spins == 64) idle_since = now;
          if (*abort_flag) break;
          if (now - idle_since > MSA_WAIT_LIMIT_NS) {
            *abort_flag = 1;
            report(p.dev_err, MSA_DEVERR_TIMEOUT);
            break;
          }
        }
      }
      umma_commit(&bar_drain);
      const uint64_t t0 = global_timer_ns();
      while (!mbar_try_wait(&bar_drain, 0) && global_timer_ns() - t0 < MSA_WAIT_LIMIT_NS) {
      }
    }
    __syncwarp();
  } else {
    // ===================== softmax + epilogue of slot s (thread = row) =====================
    const int s = (warp - 2) >> 2;
    const int q = warp & 3;
    const int r = q * 32 + lane;
    const int query = r / p.G, head = r - query * p.G;
    const bool leader = q == ((2 + 4 * s) & 3) && lane == 0;
    const uint32_t lane_addr = static_cast<uint32_t>(q * 32) << 16;
    const uint32_t sbase = tmem + lane_addr + s * 256;     // S, then P (bf16 pairs) in its first 64 columns
    const uint32_t obase = sbase + 128;
    const float sc = p.scale_log2;
    int sent = 0;                                          // Q tiles sent for
    auto send_q = [&](const Item& x) {
      const uint32_t bytes = static_cast<uint32_t>(p.nq * p.G) * 128;
      mbar_arrive_expect_tx(&bar_qfull[s], 2 * bytes);
      tma_load_4d(s_q + s * kUnit, &qmap, &bar_qfull[s], 0, x.g * p.G, x.q0 + s * p.nq, x.b);
      tma_load_4d(s_q + s * kUnit + kHalf, &qmap, &bar_qfull[s], 64, x.g * p.G, x.q0 + s * p.nq, x.b);
      ++sent;
    };
    // this slot's next item from `it` on (one without blocks is a refused sequence: its rows are 0)
    auto next_of = [&](int it, Item* x) {
      for (; it < p.n_items; it += gridDim.x) {
        *x = item_of(p, it);
        if (s < x->tiles) break;
      }
      return it;
    };
    Item x;
    int it = next_of(blockIdx.x, &x);
    int nS = 0, nO = 0, n = 0;                             // waits done on sfull, ofull; blocks of the CTA so far
    int seen = blockIdx.x;                                 // items whose blocks n counts
    auto send_next = [&](int from) {                       // the Q tile of the next item with blocks
      Item y;
      for (int k = next_of(from, &y); k < p.n_items; k = next_of(k + gridDim.x, &y))
        if (y.blocks > 0) {
          send_q(y);
          return;
        }
    };
    if (leader) send_next(blockIdx.x);
    bool alive = true;
    while (it < p.n_items && alive) {
      for (; seen < it; seen += gridDim.x) n += item_of(p, seen).blocks;
      const int row = x.q0 + s * p.nq + query;             // of the sequence's S queries
      const bool real = query < p.nq && row < p.S;
      const int i = x.pos + s * p.nq + query;              // its position
      const int low = x.pos + s * p.nq, high = low + p.nq - 1;
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < x.blocks; ++j) {
        const bool ok_s = mbar_wait(&bar_sfull[s], nS & 1, abort_flag, p.dev_err);
        ++nS;
        if (!__all_sync(0xffffffffu, ok_s)) { alive = false; break; }
        tc_fence_after();
        if (j == x.blocks - 1 && leader) send_next(it + gridDim.x);   // this item's Q tile is read
        const int t0 = x.block(j) * kBk;
        uint32_t v[4][32];
#pragma unroll
        for (int cc = 0; cc < 4; ++cc) tmem_ld32(sbase + cc * 32, v[cc]);
        tmem_ld_wait();
        const bool gone = p.paged && s_gone[(n + j) % kNotes] != 0;
        if (gone || t0 + kBk - 1 > low || (t0 <= high - p.window && t0 + kBk > p.sinks)) {
          // some row does not see all of it: columns c <= last, and c >= from or c < sinks
          const int last = gone ? -1 : i - t0, from = i - p.window + 1 - t0, sinks = p.sinks - t0;
#pragma unroll
          for (int cc = 0; cc < 4; ++cc)
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const int c = cc * 32 + e;
              if (c > last || (c < from && c >= sinks)) v[cc][e] = 0xff800000u;   // -inf
            }
        }
        float mx[4];
#pragma unroll
        for (int cc = 0; cc < 4; ++cc) {
          mx[cc] = __uint_as_float(v[cc][0]);
#pragma unroll
          for (int e = 1; e < 32; ++e) mx[cc] = fmaxf(mx[cc], __uint_as_float(v[cc][e]));
        }
        const float bm = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sc;   // scale > 0: max of the scaled scores
        const bool up = bm > m + kRescale;
        if (__any_sync(0xffffffffu, up)) {                 // O and the sum to the new max (O(j - 1) is done: S(j) came after it)
          const float alpha = up ? fast_exp2(m - bm) : 1.f;
          if (up) m = bm;
          l *= alpha;
          if (j > 0) {
#pragma unroll
            for (int cc = 0; cc < 8; ++cc) {
              uint32_t o[16];
              tmem_ld16(obase + cc * 16, o);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
              tmem_st16(obase + cc * 16, o);
            }
          }
        }
        const float off = m == -INFINITY ? 0.f : -m;       // a row that has seen nothing yet
        const uint64_t sc2 = pair(sc, sc), off2 = pair(off, off);
        uint64_t sum2[2] = {0, 0};
        auto form = [&](auto fused) {
#pragma unroll
          for (int cc = 0; cc < 4; ++cc) {
            uint32_t pw[16];
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              const float y = __uint_as_float(v[cc][e]), z = __uint_as_float(v[cc][e + 1]);
              float a, b;
              if (decltype(fused)::value) {
                unpair(fma2(pair(y, z), sc2, off2), &a, &b);
              } else {
                a = __fadd_rn(__fmul_rn(y, sc), off);
                b = __fadd_rn(__fmul_rn(z, sc), off);
              }
              a = fast_exp2(a);
              b = fast_exp2(b);
              sum2[(e >> 1) & 1] = add2(sum2[(e >> 1) & 1], pair(a, b));
              pw[e >> 1] = pack_bf16x2(a, b);
            }
            tmem_st16(sbase + cc * 16, pw);                // P columns 16 cc .. hold keys 32 cc ..
          }
        };
        // scale and max in one rounding, unless scores are so large that the max's own rounding would count as a score
        if (__any_sync(0xffffffffu, fabsf(off) > kFusedMost)) form(std::false_type{});
        else form(std::true_type{});
        float a, b;
        unpair(add2(sum2[0], sum2[1]), &a, &b);
        l += a + b;
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar_pready[s]);
      }
      if (!alive) break;
      // ---- epilogue: O complete -> O / l in bf16, LSE
      if (x.blocks > 0) {
        const bool ok_o = mbar_wait(&bar_ofull[s], nO & 1, abort_flag, p.dev_err);
        ++nO;
        if (!__all_sync(0xffffffffu, ok_o)) break;
        tc_fence_after();
      } else if (leader) {
        report(p.dev_err, MSA_DEVERR_BAD_LEN);
      }
      const float inv = l == 0.f ? 0.f : 1.0f / l;
      const int64_t at = (static_cast<int64_t>(x.b) * p.S + row) * p.Hq + x.g * p.G + head;
#pragma unroll
      for (int cc = 0; cc < 4; ++cc) {
        uint32_t o[32];
        tmem_ld32(obase + cc * 32, o);
        tmem_ld_wait();
        if (real) {
          uint4* to = reinterpret_cast<uint4*>(p.O + at * kD + cc * 32);
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            uint4 w;
            w.x = pack_bf16x2(__uint_as_float(o[e + 0]) * inv, __uint_as_float(o[e + 1]) * inv);
            w.y = pack_bf16x2(__uint_as_float(o[e + 2]) * inv, __uint_as_float(o[e + 3]) * inv);
            w.z = pack_bf16x2(__uint_as_float(o[e + 4]) * inv, __uint_as_float(o[e + 5]) * inv);
            w.w = pack_bf16x2(__uint_as_float(o[e + 6]) * inv, __uint_as_float(o[e + 7]) * inv);
            to[e / 8] = l == 0.f ? make_uint4(0, 0, 0, 0) : w;   // (tensor memory may hold anything where nothing was added)
          }
        }
      }
      if (real && p.LSE != nullptr) p.LSE[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
      // the O loads above are complete (wait::ld) before this slot's next pready arrive, which gates the next item's first O
      tc_fence_before();
      it = next_of(it + gridDim.x, &x);
    }
    if (leader && sent > 0 && *abort_flag) {               // let a load in flight land before the CTA exits
      const uint64_t since = global_timer_ns();
      while (!mbar_try_wait(&bar_qfull[s], (sent - 1) & 1) && global_timer_ns() - since < MSA_WAIT_LIMIT_NS) {
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

}  // namespace

msa_status launch_window_prefill(const msa_window_prefill_args& a, cudaStream_t stream) {
  DeviceInfo dev;
  if (msa_status st = current_device(&dev); st != MSA_OK) return st;
  const int G = a.Hq / a.Hkv;
  const bool paged = a.mode == MSA_MODE_CHUNK;
  Params p = {};
  p.B = a.B; p.S = a.S; p.Hq = a.Hq; p.Hkv = a.Hkv; p.G = G;
  p.nq = 128 / G;
  p.pairs = (a.S + 2 * p.nq - 1) / (2 * p.nq);
  p.window = std::min(a.window, 1 << 30); p.sinks = std::min(a.sinks, 1 << 30);   // positions lie below 2^30
  p.n_items = static_cast<int>(static_cast<int64_t>(p.pairs) * a.B * a.Hkv);   // (below 2^31: checked before)
  CUtensorMap qmap, kmap, vmap;
  auto u64 = [](int64_t v) { return static_cast<uint64_t>(v); };
  {
    // Q as 4-D (d, h, s, b); box = 64 columns of all heads of a group, for a tile's queries
    const uint64_t dims[4] = {u64(a.D), u64(a.Hq), u64(a.S), u64(a.B)};
    const uint64_t strides[3] = {u64(a.Q_stride[2] * 2), u64(a.Q_stride[1] * 2), u64(a.Q_stride[0] * 2)};
    const uint32_t box[4] = {64, static_cast<uint32_t>(G), static_cast<uint32_t>(p.nq), 1};
    if (msa_status st = encode_tiled_map(&qmap, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, a.Q, dims, strides, box,
                                         CU_TENSOR_MAP_SWIZZLE_128B, "Q");
        st != MSA_OK)
      return st;
  }
  for (int kv = 0; kv < 2; ++kv) {
    // K, V as (d, g, s, b) or pages (d, t, g, page); box = 64 columns of 128 tokens of one head
    const int64_t* st3 = kv ? a.V_stride : a.K_stride;
    const uint64_t dims[4] = {u64(a.D), u64(paged ? kBk : a.Hkv), u64(paged ? a.Hkv : a.S), u64(paged ? a.num_pages : a.B)};
    const uint64_t strides[3] = {u64(st3[2] * 2), u64(st3[1] * 2), u64(st3[0] * 2)};
    const uint32_t box[4] = {64, paged ? 128u : 1u, paged ? 1u : 128u, 1};
    if (msa_status st = encode_tiled_map(kv ? &vmap : &kmap, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, kv ? a.V : a.K, dims, strides, box,
                                         CU_TENSOR_MAP_SWIZZLE_128B, kv ? "V" : "K");
        st != MSA_OK)
      return st;
  }
  const float scale = a.softmax_scale > 0.f ? a.softmax_scale : 1.0f / sqrtf(static_cast<float>(a.D));
  p.scale_log2 = scale * kLog2e;
  p.paged = paged;
  p.num_pages = a.num_pages; p.max_pages = a.max_pages;
  p.seq_pt = a.seq_pt; p.q_pos = a.q_pos;
  p.O = static_cast<__nv_bfloat16*>(a.O);
  p.LSE = a.LSE;
  p.dev_err = a.dev_err;
  const size_t smem = 1024 + static_cast<size_t>(2 + kUnits) * kUnit;
  if (smem > dev.max_smem_optin) return fail(MSA_ERR_UNSUPPORTED, "window prefill: not enough shared memory");
  cudaError_t e = cudaFuncSetAttribute(window_prefill_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(window_prefill)");
  const int grid = std::min(dev.num_sms, p.n_items);
  window_prefill_kernel<<<grid, kThreads, smem, stream>>>(qmap, kmap, vmap, p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "window_prefill_kernel launch");
  return MSA_OK;
}

}  // namespace msa
