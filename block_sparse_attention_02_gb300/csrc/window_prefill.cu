// window_prefill.cu -- attention of many queries through a sliding window with sinks, over contiguous tensors (a
// prompt) or pages (a chunk after a cached prefix, draft tokens).
//
//     O[i, h] = sum_t softmax_t(scale * Q[i, h] . K[t]) V[t],  LSE[i, h] = ln sum_t e^(..),
//     t <= i with t > i - window or t < sinks.
//
// A tile is 128 rows of one KV head: nq = 128 / G queries with all their G heads (126 rows for G = 6), row = query * G +
// head.  So a tile's queries are few and their windows nearly one: it needs window / 64 + 1.3 blocks of 64 keys where 128
// queries of one head need window / 64 + 3, and a handful of queries (draft tokens) is one tile.  Two neighbouring tiles
// ("slots") share a stream of K/V blocks: the sinks' blocks, then those from the window's first key on.
//   S  = Q K_j^T   M = 128 rows, N = 64 keys, K = D    (tensor memory, two buffers of 64 columns a slot)
//   softmax (thread = row): block max, P = 2^(S * scale * log2 e - m) written back over S as bf16 pairs
//   O += P V_j     M = 128, N = D, K = 64 keys, P read from tensor memory (128 columns a slot)
// The running max m is updated lazily: O and the running sum are rescaled only when a block's max exceeds m by more than
// 2^8, so P <= 256 and the result is exact whichever m is used.  Blocks that some row does not see whole are masked.
//
// Roles: warp 0 TMA of K and V (a ring of eight 16 KiB units, K and V apart; ten are no faster), warps 1 and 2 the slots' tcgen05
// issuers, warps 4-7 and 8-11 their softmax, warps 12-15 the outputs of both.  Each slot goes through its items on its own.  Its issuer keeps S two blocks ahead:
// O(j - 2), then S(j) into the buffer whose P that product reads (a warp's products run in order).  An issuer's whole warp runs the
// loop, and one lane's products and commits are under a predicate: branches on a lane would take the descriptors out of uniform
// registers and 58 cycles a product, 170 to 190 a commit, which is more than the products themselves.
//
// The softmax warps hold an item's first P back until the outputs of the item before are read.  What is rare in their
// loop (rescaling) is not unrolled, so that it fits in the 128 registers of 512 threads.
//
// Few tiles (SPLIT: at most one an SM): the two slots, and the CTAs of a cluster, share out the blocks of one tile and join
// their outputs in shared memory; the softmax warps write them.
//
// Bound: the tensor cores' operands, and tile ends.  S reads 6 KiB of shared memory a step of 16 channels, 48 cycles for 32 of products
// (tensor memory has no room for Q: 2 x (64 + 64 + 128) columns), so a block takes 640 cycles of 512.  32,768 tokens of 8 x 6 heads, window
// 512 / 2,048 / 8,192: 0.51 / 1.26 / 3.92 ms, which is 0.78 us a block of both slots (1,630 TFLOP/s) and 5 us a pair of tiles: masked
// blocks (three of a tile; 0.5 us), the wait for the next Q (1 us), and what the slots' chains take to empty and fill.
// Over pages 2 to 8 % more for the same tiles (0.47, 1.29 and 4.25 ms for 0.46, 1.21 and 4.05 in one run).
// With the outputs written by the softmax warps 0.55 / 1.31 / 3.94 ms, masks by comparisons instead of bits 0.52 / 1.27 / 3.92.
// 128-key blocks without a second buffer: 131,072 tokens in 11.5 ms for 5.5; pairs of blocks (S with N = 128, no block ahead): 1.67 / 5.2 ms
// where this form took 1.34 / 3.95.
#include <cooperative_groups.h>

#include <algorithm>

#include "launch_early.cuh"
#include "msa_internal.h"
#include "msa_ptx.cuh"

namespace cg = cooperative_groups;

namespace msa {
namespace {

constexpr int kKeys = 64;                    // of a block
constexpr int kQHalf = 128 * 64 * 2;         // 16 KiB: 128 rows x 64 bf16
constexpr int kQTile = 2 * kQHalf;
constexpr int kHalf = kKeys * 64 * 2;        // 8 KiB: a block's rows x 64 bf16
constexpr int kUnit = 2 * kHalf;             // 16 KiB: K or V of a block
// Units of K and V in shared memory.  Few tiles wait for HBM and gain by more (8 x 4 queries 19.9 us for 21.8 with eight), many do not
// (131,072 tokens 5.47 ms with either).
constexpr int units_of(bool split) { return split ? 10 : 8; }
constexpr int kMaxSplit = 8;                 // CTAs of an item
static_assert(units_of(true) * kUnit >= 2 * 128 * kD * 4, "room for two slots' outputs");
constexpr int kNotes = 16;                   // blocks whose page's state is kept (more than are in flight)

// w0 TMA of K and V, w1-2 the slots' issuers, w4-7 slot 0, w8-11 slot 1, w12-15 outputs
constexpr int kWorkers = 384, kAll = 512;
constexpr int kTmemCols = 512;               // per slot: two of S / P (64 columns each) and O (128 columns)
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescale = 8.0f;             // log2 of the largest P before the running max moves
constexpr float kFusedMost = 16777216.f;     // scores up to which scale and max go into one rounding

struct Params {
  int B, S, Hq, Hkv, G, nq;                  // nq: queries of a tile
  int of_sequence;                           // items of a sequence: pairs of tiles, or (SPLIT) tiles
  int split;                                 // SPLIT: CTAs of an item
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

// A pair of tiles (SPLIT: one tile): queries q0 .. of sequence b, head g, at positions pos ..  Its blocks are sink_blocks ones
// from 0 on, then those from `first` on; a CTA's are `blocks` ones of this list from `from` on.
struct Item {
  int b, g, q0, pos, end, tiles, sink_blocks, first, from, blocks;   // (end: of the sequence's tokens)
  __device__ __forceinline__ int block(int j) const {
    j += from;
    return j < sink_blocks ? j : j - sink_blocks + first;
  }
};
// The items with the most blocks first: from the last to the first of a sequence.
template <bool SPLIT>
__device__ __forceinline__ Item item_of(const Params& p, int it) {
  Item x;
  const int heads = p.B * p.Hkv, queries = SPLIT ? p.nq : 2 * p.nq;
  const int i = p.of_sequence - 1 - it / heads;
  const int rest = it % heads;
  x.g = rest % p.Hkv;
  x.b = rest / p.Hkv;
  x.q0 = i * queries;
  x.tiles = SPLIT || x.q0 + p.nq < p.S ? 2 : 1;
  x.from = 0;
  const int start = p.paged ? p.q_pos[x.b] : 0;
  x.pos = start + x.q0;
  x.end = start + p.S;
  if (p.paged && (start < 0 || start + static_cast<int64_t>(p.S) > p.max_pages * kBk)) {
    x.sink_blocks = x.first = x.blocks = 0;
    return x;
  }
  const int last = start + min(x.q0 + queries, p.S) - 1;
  x.first = max(x.pos - p.window + 1, 0) / kKeys;
  x.sink_blocks = min((min(p.sinks, last + 1) + kKeys - 1) / kKeys, x.first);
  x.blocks = x.sink_blocks + last / kKeys - x.first + 1;
  if (SPLIT) {
    const int per = (x.blocks + p.split - 1) / p.split;
    x.from = min(static_cast<int>(blockIdx.x % p.split) * per, x.blocks);
    x.blocks = min(per, x.blocks - x.from);
  }
  return x;
}

__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  __nv_bfloat162 h2 = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h2);
}
// Products and commits by an elected lane of a converged warp (the same lane every time), under a predicate: control flow stays
// that of the whole warp, so that descriptors are kept in uniform registers.
__device__ __forceinline__ void umma_elect(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void umma_ts_elect(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void commit_elect(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar))
      : "memory");
}
// A bounded wait as mbar_wait, which reads the clock only after some tries: a read takes about as long as a block's products,
// and most waits here are shorter.
__device__ __forceinline__ bool wait_here(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int32_t* dev_err) {
  uint64_t since = 0;
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 31u) != 0) continue;
    if (*abort_flag) return false;
    const uint64_t now = global_timer_ns();
    if (i == 32) since = now;
    if (now - since > MSA_WAIT_LIMIT_NS) {
      *abort_flag = 1;
      report(dev_err, MSA_DEVERR_TIMEOUT);
      return false;
    }
  }
}
__device__ __noinline__ bool wait_long(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int32_t* dev_err) {
  return wait_here(bar, parity, abort_flag, dev_err);
}
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int32_t* dev_err) {
  return mbar_try_wait(bar, parity) || wait_long(bar, parity, abort_flag, dev_err);
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

template <bool SPLIT>
__global__ void __launch_bounds__(SPLIT ? kWorkers : kAll, 1)
window_prefill_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                      const __grid_constant__ CUtensorMap vmap, const Params p) {
  constexpr int kThreads = SPLIT ? kWorkers : kAll, kUnits = units_of(SPLIT), kRings = SPLIT ? 2 : 1, kRing = kUnits / kRings;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* s_q = smem;                       // [2] Q tiles
  // [kRings][kRing] units of K and V: of a ring's n-th block unit 2 n % kRing is K, the next one V.  With SPLIT, where the slots
  // take the blocks in turn, each has a ring of its own: in a common one of ten a unit would go from slot to slot, and a slot
  // that waits for its phase would take the phase before, still under way for the other slot, for the one before that.
  uint8_t* s_kv = smem + 2 * kQTile;

  __shared__ __align__(8) uint64_t bar_qfull[2], bar_qempty[2], bar_full[kUnits], bar_empty[kUnits], bar_end;
  // per slot; of S and P one for each of the two buffers: an S or P may be complete before the one before it is looked at
  __shared__ __align__(8) uint64_t bar_sfull[2][2], bar_pready[2][2], bar_odone[2][2], bar_drain[2], bar_stat[2], bar_ofree[2];   // (odone: of an item's last two O)
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ volatile int s_gone[kNotes];    // of block n % kNotes: no such page
  __shared__ float s_inv[2][128];            // of a slot's finished tile: 1 / the rows' sums (0 of an empty row)
  // SPLIT, at the end: the slots' outputs take the units' place, each row's max and sum that of Q
  float(*s_ml)[2][128] = reinterpret_cast<float(*)[2][128]>(s_q);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < kUnits; ++i) { mbar_init(&bar_full[i], 1); mbar_init(&bar_empty[i], SPLIT ? 1 : 2); }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar_qfull[i], 1);
      mbar_init(&bar_qempty[i], 1);
      for (int k = 0; k < 2; ++k) { mbar_init(&bar_sfull[i][k], 1); mbar_init(&bar_pready[i][k], 4); }
      for (int k = 0; k < 2; ++k) mbar_init(&bar_odone[i][k], 1);
      mbar_init(&bar_drain[i], 1);
      mbar_init(&bar_stat[i], 4);
      mbar_init(&bar_ofree[i], 4);
    }
    mbar_init(&bar_end, 1);
    s_abort = 0;
    fence_mbar_init();
  }
  // rows past a tile's queries, which no load writes: zeros, so that their scores are numbers
  for (int i = tid; i < 4 * (128 - p.nq * p.G) * 8; i += kThreads)
    reinterpret_cast<uint4*>(s_q + (i & 3) * kQHalf + p.nq * p.G * 128)[i >> 2] = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  if (warp == 1) tmem_alloc(&s_tmem, kTmemCols);
  wait_for_stream();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  volatile int* abort_flag = &s_abort;
  const int it0 = SPLIT ? blockIdx.x / p.split : blockIdx.x, stride = SPLIT ? p.n_items : gridDim.x;

  // blocks of an item that slot s works on
  auto own = [](const Item& x, int s) { return SPLIT ? (x.blocks + 1 - s) >> 1 : x.blocks; };

  if (warp == 0) {
    // ===================== TMA producer of K and V (warp-uniform loop, lane 0 issues) =====================
    int n = 0, sent = 0;                     // blocks and units sent for
    uint32_t end_phase = 0;
    bool ok = true;
    for (int it = it0; it < p.n_items && ok; it += stride) {
      const Item x = item_of<SPLIT>(p, it);
      for (int j0 = 0; j0 < x.blocks && ok; j0 += 32) {
        // lane l looks up the page of block j0 + l
        int pg = 0;
        if (p.paged && j0 + lane < x.blocks) pg = p.seq_pt[x.b * p.max_pages + x.block(j0 + lane) * kKeys / kBk];
        for (int i = 0; i < 32 && j0 + i < x.blocks; ++i, ++n) {
          const int page = __shfl_sync(0xffffffffu, pg, i);
          // Slots of a page behind the sequence's last token may hold anything, and 0 * NaN is NaN: V's rows there become zeros
          // before the unit is handed on.  (Only a sequence's last block waits for this.)
          const bool ends = p.paged && j0 + i + 1 == x.blocks && x.end - x.block(j0 + i) * kKeys < kKeys;
          int go = 1, st = 0;
          if (lane == 0) {
            const bool gone = p.paged && (page < 0 || page >= p.num_pages);
            // a page that there is not is read as zeros: from past the end of the pool
            const int t = x.block(j0 + i) * kKeys, c1 = p.paged ? t % kBk : t;
            const int c4 = p.paged ? (gone ? static_cast<int>(p.num_pages) : page) : x.b;
            for (int kv = 0; kv < 2 && go; ++kv) {
              const int u = n / kRings * 2 + kv;               // of the block's ring
              st = n % kRings * kRing + u % kRing;
              go = wait(&bar_empty[st], (u / kRing & 1) ^ 1, abort_flag, p.dev_err);
              if (!go) break;
              if (kv == 0) s_gone[n % kNotes] = gone;
              uint64_t* bar = kv && ends ? &bar_end : &bar_full[st];
              mbar_arrive_expect_tx(bar, kUnit);
              tma_load_5d(s_kv + st * kUnit, kv ? &vmap : &kmap, bar, 0, c1, 0, x.g, c4);
              ++sent;
            }
            if (gone) report(p.dev_err, MSA_DEVERR_BAD_PAGE);
          }
          if (ends) {
            if (lane == 0 && go) go = wait(&bar_end, end_phase, abort_flag, p.dev_err);
            end_phase ^= 1;
            const int unit = __shfl_sync(0xffffffffu, st, 0), all = __shfl_sync(0xffffffffu, go, 0);
            __syncwarp();
            for (int e = (x.end - x.block(j0 + i) * kKeys) * 8 + lane; all && e < kKeys * 8; e += 32)   // 16 bytes of each half
              for (int half = 0; half < 2; ++half) reinterpret_cast<uint4*>(s_kv + unit * kUnit + half * kHalf)[e] = make_uint4(0, 0, 0, 0);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0 && go) mbar_arrive(&bar_full[unit]);
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
      for (int k = 0; k < kRings; ++k)
        for (int all = (sent / 2 + kRings - 1 - k) / kRings * 2 + (sent / 2 % kRings == k ? sent & 1 : 0), u = max(0, all - kRing); u < all; ++u)
          while (!mbar_try_wait(&bar_full[k * kRing + u % kRing], (u / kRing) & 1) && global_timer_ns() - t0 < MSA_WAIT_LIMIT_NS) {
          }
    }
    __syncwarp();
  } else if (warp < 3) {
    // ===================== tcgen05 issuer of slot s (warp-uniform loop, an elected lane issues) =====================
    // Step j of an item: O(j - 2), then S(j) into the buffer whose P that O reads.  So S is two blocks ahead and the
    // softmax always has one to work on.
    const int s = warp - 1;
    constexpr uint32_t idesc_s = idesc_bf16(128, kKeys, false, false);
    constexpr uint32_t idesc_o = idesc_bf16(128, 128, false, true);
    const uint32_t sp = tmem + s * 256, out = sp + 128;
    const uint64_t q_desc = sdesc_sw128(smem_u32(s_q + s * kQTile), 16, 1024), k_desc = sdesc_sw128(smem_u32(s_kv), 16, 1024),
                   v_desc = sdesc_sw128(smem_u32(s_kv), kHalf, 1024);
    // units of the next K and V, and their phases
    const int ring_end = (SPLIT ? s + 1 : 1) * kRing;
    int sk = ring_end - kRing, sv = sk + 1;
    uint32_t pk = 0, pv = 0;
    int n = 0, items = 0, sent = 0;          // blocks and items done, Q tiles sent for
    bool ok = true;
    auto next_k = [&] {
      sk += 2;
      if (sk >= ring_end) { sk -= kRing; pk ^= 1; }
    };
    auto next_v = [&] {
      sv += 2;
      if (sv >= ring_end) { sv -= kRing; pv ^= 1; }
    };
    // the Q tile of this slot's first item from `it` on that has blocks, once the last S of the one before is done
    auto send_q = [&](int it) {
      for (; it < p.n_items; it += stride) {
        const Item x = item_of<SPLIT>(p, it);
        if (s >= x.tiles || own(x, s) == 0) continue;
        if (lane == 0 && wait(&bar_qempty[s], (sent & 1) ^ 1, abort_flag, p.dev_err)) {
          mbar_arrive_expect_tx(&bar_qfull[s], static_cast<uint32_t>(p.nq * p.G) * 256);
          for (int half = 0; half < 2; ++half)
            tma_load_5d(s_q + s * kQTile + half * kQHalf, &qmap, &bar_qfull[s], 0, x.g * p.G, x.q0 + (SPLIT ? 0 : s * p.nq), half, x.b);
        }
        ++sent;
        break;
      }
    };
    send_q(it0);
    for (int it = it0; it < p.n_items && ok; it += stride) {
      const Item x = item_of<SPLIT>(p, it);
      const int blocks = __shfl_sync(0xffffffffu, own(x, s), 0);   // (from lane 0: the compiler then knows that the warp goes one way)
      if (s >= __shfl_sync(0xffffffffu, x.tiles, 0)) {
        // an item without a tile for this slot: its units pass
        for (int j = 0; j < blocks && ok; ++j) {
          ok = wait(&bar_full[sk], pk, abort_flag, p.dev_err) && wait(&bar_full[sv], pv, abort_flag, p.dev_err);
          ok = __all_sync(0xffffffffu, ok);
          if (ok && lane == 0) {
            mbar_arrive(&bar_empty[sk]);
            mbar_arrive(&bar_empty[sv]);
          }
          next_k();
          next_v();
        }
        continue;
      }
      if (blocks == 0) continue;
      for (int j = 0; j < blocks + 2; ++j) {
        const uint32_t buf = (n + j) & 1;    // of O(j - 2) and S(j)
        if (j >= 2) {
          ok = wait(&bar_full[sv], pv, abort_flag, p.dev_err) && wait(&bar_pready[s][buf], ((n + j - 2) >> 1) & 1, abort_flag, p.dev_err);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < kKeys / 16; ++kk)
            umma_ts_elect(out, sp + buf * kKeys + kk * 8, v_desc + sv * (kUnit / 16) + kk * (2048 / 16), idesc_o,
                       (j > 2 || kk > 0) ? 1u : 0u);
          commit_elect(&bar_empty[sv]);
          next_v();
        }
        if (j >= blocks) commit_elect(&bar_odone[s][j - blocks]);   // O(j - 2), one of the last two
        if (j < blocks) {
          ok = wait(&bar_full[sk], pk, abort_flag, p.dev_err) && (j > 0 || wait(&bar_qfull[s], items & 1, abort_flag, p.dev_err));
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            umma_elect(sp + buf * kKeys, q_desc + (kk >> 2) * (kQHalf / 16) + 2 * (kk & 3),
                    k_desc + sk * (kUnit / 16) + (kk >> 2) * (kHalf / 16) + 2 * (kk & 3), idesc_s, kk > 0);
          commit_elect(&bar_sfull[s][buf]);
          commit_elect(&bar_empty[sk]);
          if (j == blocks - 1) commit_elect(&bar_qempty[s]);
          next_k();
        } else if (j == blocks) {
          send_q(it + stride);
        }
      }
      n += blocks;
      ++items;
    }
    __syncwarp();
    commit_elect(&bar_drain[s]);
    if (lane == 0) {
      const uint64_t t0 = global_timer_ns();
      while (!mbar_try_wait(&bar_drain[s], 0) && global_timer_ns() - t0 < MSA_WAIT_LIMIT_NS) {
      }
      while (sent > 0 && *abort_flag && !mbar_try_wait(&bar_qfull[s], (sent - 1) & 1) && global_timer_ns() - t0 < MSA_WAIT_LIMIT_NS) {
      }                                      // (a load in flight lands before the CTA exits)
    }
    __syncwarp();
  } else if (warp >= 4 && warp < 12) {
    // ===================== softmax of slot s (thread = row) =====================
    const int s = (warp >> 2) - 1;
    const int q = warp & 3;
    const int r = q * 32 + lane;
    const int query = r / p.G;
    const uint32_t lane_addr = static_cast<uint32_t>(q * 32) << 16;
    const uint32_t sbase = tmem + lane_addr + s * 256;     // two buffers: S, then P (bf16 pairs) in its first 32 columns
    const uint32_t obase = sbase + 128;
    const float sc = p.scale_log2;
    int nS = 0, nI = 0, n = 0;                             // blocks done; items done; blocks of the CTA so far
    bool alive = true;
    for (int it = it0; it < p.n_items && alive; it += stride) {
      const Item x = item_of<SPLIT>(p, it);
      const int n0 = n;
      n += x.blocks;
      if (s >= x.tiles) continue;
      const int row0 = x.q0 + (SPLIT ? 0 : s * p.nq);      // the tile's first query, of the sequence's S
      const int low = x.pos + row0 - x.q0, high = low + p.nq - 1, i = low + query;   // positions: of the tile, and this row's
      const int blocks = own(x, s);
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < blocks; ++j, ++nS) {
        const bool ok_s = wait(&bar_sfull[s][nS & 1], (nS >> 1) & 1, abort_flag, p.dev_err);
        if (!__all_sync(0xffffffffu, ok_s)) { alive = false; break; }
        tc_fence_after();
        const uint32_t sb = sbase + (nS & 1) * kKeys;
        const int listed = SPLIT ? 2 * j + s : j, t0 = x.block(listed) * kKeys;
        uint32_t v[2][32];
        tmem_ld32(sb, v[0]);
        tmem_ld32(sb + 32, v[1]);
        tmem_ld_wait();
        const bool gone = p.paged && s_gone[(n0 + listed) % kNotes] != 0;
        if (gone || t0 + kKeys - 1 > low || (t0 <= high - p.window && t0 + kKeys > p.sinks)) {
          // some row does not see all of it: columns c <= last, and c >= from or c < sinks; a bit each
          const int last = gone ? -1 : i - t0, from = i - p.window + 1 - t0, sinks = p.sinks - t0;
          auto below = [](int n) { return n >= kKeys ? ~0ull : n <= 0 ? 0ull : (1ull << n) - 1; };
          const uint64_t seen = below(last + 1) & (~below(from) | below(sinks));
#pragma unroll
          for (int cc = 0; cc < 2; ++cc) {
            const uint32_t bits = static_cast<uint32_t>(seen >> (32 * cc));
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if ((bits >> e & 1) == 0) v[cc][e] = 0xff800000u;   // -inf
          }
        }
        float mx[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t* y = v[k >> 1] + (k & 1) * 16;
          mx[k] = max3(__uint_as_float(y[0]), __uint_as_float(y[1]), __uint_as_float(y[2]));
#pragma unroll
          for (int e = 3; e < 15; e += 2) mx[k] = max3(mx[k], __uint_as_float(y[e]), __uint_as_float(y[e + 1]));
          mx[k] = fmaxf(mx[k], __uint_as_float(y[15]));
        }
        const float bm = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]) * sc;   // scale > 0: max of the scaled scores
        const bool up = bm > m + kRescale;
        if (__any_sync(0xffffffffu, up)) {                 // O and the sum to the new max
          const float alpha = up ? fast_exp2(m - bm) : 1.f;
          if (up) m = bm;
          l *= alpha;
          if (j > 0) {
            // O(j - 1) is done when S(j + 1), issued right behind it, is; behind the last S there is a commit for it
            // (not a call: all of the scores are in registers)
            const bool next = j + 1 < blocks;
            const bool ok_o = wait_here(next ? &bar_sfull[s][(nS + 1) & 1] : &bar_odone[s][0], (next ? (nS + 1) >> 1 : nI) & 1, abort_flag, p.dev_err);
            if (!__all_sync(0xffffffffu, ok_o)) { alive = false; break; }
            tc_fence_after();
#pragma unroll 1                                           // (rare; the scores are in registers)
            for (int cc = 0; cc < 4; ++cc) {
              uint32_t o[32];
              tmem_ld32(obase + cc * 32, o);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
              tmem_st32(obase + cc * 32, o);
            }
          }
        }
        const float off = m == -INFINITY ? 0.f : -m;       // a row that has seen nothing yet
        float by = sc;
        if (__any_sync(0xffffffffu, fabsf(off) > kFusedMost)) {
          // scores so large that the max's own rounding would count as one: scale and max in two roundings
          by = 1.f;
#pragma unroll
          for (int cc = 0; cc < 2; ++cc)
#pragma unroll
            for (int e = 0; e < 32; ++e) v[cc][e] = __float_as_uint(__fmul_rn(__uint_as_float(v[cc][e]), sc));
        }
        const uint64_t sc2 = pair(by, by), off2 = pair(off, off);
        uint64_t sum2[2] = {0, 0};
        uint32_t pw[32];
#pragma unroll
        for (int cc = 0; cc < 2; ++cc) {
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            float a, b;
            unpair(fma2(pair(__uint_as_float(v[cc][e]), __uint_as_float(v[cc][e + 1])), sc2, off2), &a, &b);
            a = fast_exp2(a);
            b = fast_exp2(b);
            sum2[(e >> 1) & 1] = add2(sum2[(e >> 1) & 1], pair(a, b));
            pw[cc * 16 + (e >> 1)] = pack_bf16x2(a, b);
          }
        }
        tmem_st32(sb, pw);                                 // P column c holds keys 2 c, 2 c + 1
        float a, b;
        unpair(add2(sum2[0], sum2[1]), &a, &b);
        l += a + b;
        tmem_st_wait();
        if (!SPLIT && j == 0 && nI > 0) {                  // the tile before is read
          const bool ok_o = wait(&bar_ofree[s], (nI & 1) ^ 1, abort_flag, p.dev_err);
          if (!__all_sync(0xffffffffu, ok_o)) { alive = false; break; }
          tc_fence_after();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar_pready[s][nS & 1]);
      }
      if (!alive) break;
      // ---- epilogue: O complete -> O / l in bf16, LSE
      if (SPLIT) {
        // both slots' products done: K's and V's units give way to the outputs, unscaled
        const bool ok_o = (own(x, 0) == 0 || wait(&bar_odone[0][1], 0, abort_flag, p.dev_err)) &&
                          (own(x, 1) == 0 || wait(&bar_odone[1][1], 0, abort_flag, p.dev_err));
        if (!__all_sync(0xffffffffu, ok_o)) break;
        tc_fence_after();
        if (x.blocks == 0 && x.from == 0 && r == 0 && s == 0 && blockIdx.x % p.split == 0) report(p.dev_err, MSA_DEVERR_BAD_LEN);
        s_ml[s][0][r] = m;
        s_ml[s][1][r] = l;
        float4* to = reinterpret_cast<float4*>(s_kv) + (s * 128 + r) * 32;
#pragma unroll
        for (int cc = 0; cc < 4; ++cc) {
          uint32_t o[32];
          tmem_ld32(obase + cc * 32, o);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 8; ++e) {                    // (chunks in another order in every row: no two lanes meet a bank)
            float4 w = make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]), __uint_as_float(o[4 * e + 2]), __uint_as_float(o[4 * e + 3]));
            if (l == 0.f) w = make_float4(0.f, 0.f, 0.f, 0.f);
            to[(cc * 8 + e) ^ (r & 31)] = w;
          }
        }
        tc_fence_before();
        break;
      }
      if (blocks > 0) {
        ++nI;
        s_inv[s][r] = l == 0.f ? 0.f : 1.0f / l;
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar_stat[s]);
      }
      if (p.LSE != nullptr && query < p.nq && row0 + query < p.S)
        p.LSE[(static_cast<int64_t>(x.b) * p.S + row0 + query) * p.Hq + x.g * p.G + r - query * p.G] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
    }
  } else if (!SPLIT && warp >= 12) {
    // ===================== outputs: O / l in bf16, LSE (thread = row) =====================
    const int q = warp & 3;
    const int r = q * 32 + lane;
    const int per_query = 65536 / p.G + 1;                 // (row * per_query) >> 16 is row / G
    int nI[2] = {0, 0};
    bool alive = true;
    for (int it = it0; it < p.n_items && alive; it += stride) {
      const Item x = item_of<SPLIT>(p, it);
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        if (s >= x.tiles) break;
        const int row0 = x.q0 + s * p.nq;                  // the tile's first query, of the sequence's S
        const uint32_t obase = tmem + (static_cast<uint32_t>(q * 32) << 16) + s * 256 + 128;
        float inv = 0.f;
        if (x.blocks > 0) {
          const bool ok_o = wait(&bar_stat[s], nI[s] & 1, abort_flag, p.dev_err) && wait(&bar_odone[s][1], nI[s] & 1, abort_flag, p.dev_err);
          if (!__all_sync(0xffffffffu, ok_o)) { alive = false; break; }
          ++nI[s];
          inv = s_inv[s][r];
          tc_fence_after();
        } else if (r == 0) {
          report(p.dev_err, MSA_DEVERR_BAD_LEN);
        }
        uint32_t w[2][8][4];
#pragma unroll
        for (int cc = 0; cc < 4; ++cc) {
          uint32_t o[32];
          tmem_ld32(obase + cc * 32, o);
          tmem_ld_wait();
#pragma unroll
          for (int k = 0; k < 32; k += 2) {
            uint32_t& to = w[cc >> 1][(cc & 1) * 4 + (k >> 3)][(k >> 1) & 3];
            to = pack_bf16x2(__uint_as_float(o[k]) * inv, __uint_as_float(o[k + 1]) * inv);
            if (inv == 0.f) to = 0;                        // (tensor memory may hold anything where nothing was added)
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0 && x.blocks > 0) mbar_arrive(&bar_ofree[s]);
        // A row's 256 bytes are one thread's; written so, each store would touch 32 lines.  Eight lanes exchange their rows'
        // 16-byte chunks (an 8 x 8 transposition), so that they write 128 bytes of one row together.
        const int queries = min(p.nq, p.S - row0);
        __nv_bfloat16* tile = p.O + ((static_cast<int64_t>(x.b) * p.S + row0) * p.Hq + x.g * p.G) * kD + (lane & 7) * 8;
#pragma unroll
        for (int cc = 0; cc < 2; ++cc) {
#pragma unroll
          for (int bit = 1; bit < 8; bit <<= 1) {
            const bool high = (lane & bit) != 0;
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              if (c & bit) continue;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const uint32_t got = __shfl_xor_sync(0xffffffffu, high ? w[cc][c][e] : w[cc][c | bit][e], bit);
                if (high) w[cc][c][e] = got;
                else w[cc][c | bit][e] = got;
              }
            }
          }
#pragma unroll
          for (int c = 0; c < 8; ++c) {                    // chunk lane % 8 of row r - lane % 8 + c
            const int rr = (r & ~7) + c, qq = (rr * per_query) >> 16;
            if (qq < queries)
              *reinterpret_cast<uint4*>(tile + (static_cast<int64_t>(qq) * p.Hq + rr - qq * p.G) * kD + cc * 64) =
                  make_uint4(w[cc][c][0], w[cc][c][1], w[cc][c][2], w[cc][c][3]);
          }
        }
      }
    }
    tc_fence_before();
  }

  if (SPLIT) {
    // the item's parts, two of each CTA, joined: four channels of a row by a thread
    cg::cluster_group cluster = cg::this_cluster();
    if (p.split > 1) cluster.sync(); else __syncthreads();
    const Item x = item_of<SPLIT>(p, it0);
    const int rows = min(p.nq, p.S - x.q0) * p.G, parts = 2 * p.split, ctas = p.split, mine = blockIdx.x % p.split;
    if (*abort_flag == 0) {
      for (int e = mine * kThreads + tid; e < rows * 32; e += ctas * kThreads) {
        const int r = e >> 5, c = e & 31;
        float m[2 * kMaxSplit], top = -INFINITY;
#pragma unroll
        for (int k = 0; k < 2 * kMaxSplit; ++k) {
          m[k] = -INFINITY;
          if (k < parts) m[k] = p.split > 1 ? *cluster.map_shared_rank(&s_ml[k & 1][0][r], k >> 1) : s_ml[k & 1][0][r];
          top = fmaxf(top, m[k]);
        }
        float l = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < 2 * kMaxSplit; ++k) {
          if (k >= parts || m[k] == -INFINITY) continue;
          const float f = fast_exp2(m[k] - top);
          const float* sum = &s_ml[k & 1][1][r];
          const float4* from = reinterpret_cast<const float4*>(s_kv) + ((k & 1) * 128 + r) * 32 + (c ^ (r & 31));
          const float lk = p.split > 1 ? *cluster.map_shared_rank(sum, k >> 1) : *sum;
          const float4 v = p.split > 1 ? *cluster.map_shared_rank(from, k >> 1) : *from;
          l = fmaf(f, lk, l);
          o.x = fmaf(f, v.x, o.x); o.y = fmaf(f, v.y, o.y); o.z = fmaf(f, v.z, o.z); o.w = fmaf(f, v.w, o.w);
        }
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const int query = r / p.G;
        const int64_t at = (static_cast<int64_t>(x.b) * p.S + x.q0 + query) * p.Hq + x.g * p.G + r - query * p.G;
        *reinterpret_cast<uint2*>(p.O + at * kD + 4 * c) = make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
        if (c == 0 && p.LSE != nullptr) p.LSE[at] = l == 0.f ? -INFINITY : (top + log2f(l)) * kLn2;
      }
    }
    if (p.split > 1) cluster.sync();         // no CTA leaves while another reads its memory
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
  p.window = std::min(a.window, 1 << 30); p.sinks = std::min(a.sinks, 1 << 30);   // positions lie below 2^30
  // Few tiles: each is a CTA's or a cluster's, whose slots share out its blocks and join their outputs in shared memory.
  // (Clusters of more than two that nearly fill the GPU would not all fit at once.  A slot has two blocks at least.)
  const int64_t tiles = static_cast<int64_t>((a.S + p.nq - 1) / p.nq) * a.B * a.Hkv;
  const bool split = tiles <= dev.num_sms;
  if (split) {
    const int64_t reach = paged ? a.max_pages * kBk : a.S;
    const int64_t most = std::min(reach / kKeys + 1, (int64_t(p.window) + p.nq) / kKeys + 2 + (int64_t(p.sinks) + kKeys - 1) / kKeys);
    p.split = 1;
    while (p.split < kMaxSplit && (p.split == 1 ? 2 * tiles <= dev.num_sms : 8 * p.split * tiles <= 3 * dev.num_sms) && 8 * p.split <= most) p.split *= 2;
  }
  p.of_sequence = split ? (a.S + p.nq - 1) / p.nq : (a.S + 2 * p.nq - 1) / (2 * p.nq);
  p.n_items = static_cast<int>(static_cast<int64_t>(p.of_sequence) * a.B * a.Hkv);   // (below 2^31: checked before)
  CUtensorMap qmap, kmap, vmap;
  auto u64 = [](int64_t v) { return static_cast<uint64_t>(v); };
  // rows of 128 values are two halves of 64, each a tile of 128-byte rows: of a block both come in one box
  {
    // Q as (d, h, s, half, b); all heads of a group, a tile's queries (whose halves do not end where a swizzle's rows do)
    const uint64_t dims[5] = {64, u64(a.Hq), u64(a.S), 2, u64(a.B)};
    const uint64_t strides[4] = {u64(a.Q_stride[2] * 2), u64(a.Q_stride[1] * 2), 128, u64(a.Q_stride[0] * 2)};
    const uint32_t box[5] = {64, static_cast<uint32_t>(G), static_cast<uint32_t>(p.nq), 1, 1};
    if (msa_status st = encode_tiled_map(&qmap, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, a.Q, dims, strides, box,
                                         CU_TENSOR_MAP_SWIZZLE_128B, "Q");
        st != MSA_OK)
      return st;
  }
  for (int kv = 0; kv < 2; ++kv) {
    // K, V as (d, s, half, g, b) or pages (d, t, half, g, page); a block's tokens of one head
    const int64_t* str = kv ? a.V_stride : a.K_stride;     // (b, s, g) or (page, g, t)
    const uint64_t dims[5] = {64, u64(paged ? kBk : a.S), 2, u64(a.Hkv), u64(paged ? a.num_pages : a.B)};
    const uint64_t strides[4] = {u64(str[paged ? 2 : 1] * 2), 128, u64(str[paged ? 1 : 2] * 2), u64(str[0] * 2)};
    const uint32_t box[5] = {64, kKeys, 2, 1, 1};
    if (msa_status st = encode_tiled_map(kv ? &vmap : &kmap, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, kv ? a.V : a.K, dims, strides, box,
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
  const size_t smem = 1024 + 2 * static_cast<size_t>(kQTile) + static_cast<size_t>(units_of(split)) * kUnit;
  if (smem > dev.max_smem_optin) return fail(MSA_ERR_UNSUPPORTED, "window prefill: not enough shared memory");
  auto* kernel = split ? window_prefill_kernel<true> : window_prefill_kernel<false>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(window_prefill)");
  const int grid = split ? p.n_items * p.split : std::min(dev.num_sms, p.n_items);
  e = launch_early(kernel, grid, split ? kWorkers : kAll, smem, stream, std::max(p.split, 1), qmap, kmap, vmap, p);
  if (e != cudaSuccess) return cuda_fail(e, "window_prefill_kernel launch");
  return MSA_OK;
}

}  // namespace msa
