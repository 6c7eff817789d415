// attn_decode_q4.cu -- decode attention over the paged cache in 4 bits, over the
// selected pages (sparse) or every cached token (dense).
//
//     z[h][t] = scale * Q[h] . K[t],  O[h] = sum_t softmax_t(z[h]) V[t],  LSE[h] = ln sum_t e^z
// for the G query heads that share a KV head.  A token costs 144 bytes (two rows
// of 64 code and 8 scale bytes), so HBM is the floor and the work beside the
// loads is turning codes into matrix operands.
//
// Products.  mma.m16n8k16 in fp16 with fp32 sums, straight from registers:
//   S^T[t][h]: A = 16 tokens x 16 channels of K, B = Q (8 heads: G padded)
//   O^T[d][h]: A = 16 channels x 16 tokens of V, B = P
// The eight columns fit the heads exactly, where a 128-row tensor-memory tile would
// need the dequantised block written to shared memory first (64 KiB a page) and read
// back.  The order of the channels in S's sum and of the rows in O is free, so
// each lane takes 16 bytes (32 channels) of a token's K row and 8 bytes (one
// scale group) of a V row as they lie in the page.
//
// Exactness.  code * sf has 6 bits and lies in [2^-10, 2688]: exact in fp16, so
// the cached values enter the products unrounded; the pools' powers of two and the
// softmax scale multiply the fp32 sums.  Q is brought to [1, 2) per head by a power
// of two; P = 2^(z - m + 8) with m the running maximum or up to 7 below it, at most
// 2^15, is rounded to fp16 (2^-11 of the value down to 2^-22 of the largest).
//
// Work.  Dense: the (row, page) units of all rows form one list; each CTA takes an equal
// run of it, or, where there are few pages, one part of one row.  Sparse: a CTA has a row, or
// one of its equal parts where there are few rows.  Four warps share a page; a warp takes 32
// tokens of it through two stages in shared memory of its own (more bytes in flight serve
// HBM worse, see kStages) with a softmax of its own; the warps' softmaxes are joined in
// shared memory at the end of a row's part.  Parts of a row are joined through the workspace by
// the CTA that arrives last, or, if they are a few equal ones, through a cluster's shared memory.
//
// Bound: 261 instructions a warp for 16 tokens, 164 of them conversions, scalings and
// products, leave the SMs issuing in 60 % of their cycles at 94 % of the copy
// rate (1,048,576 tokens 189 us, floor 178); 8 x 60,001 tokens 94 us (floor 82)
// pay 6 us of starting, joining and ending besides.
#include <cooperative_groups.h>
#include <cuda_fp16.h>

#include <cfloat>

#include "launch_early.cuh"
#include "msa_internal.h"
#include "msa_ptx.cuh"
#include "q4.cuh"

namespace cg = cooperative_groups;

namespace msa {
namespace {

// Warps of a CTA: four, and for few long rows eight.  With four, twice as many CTAs leave an SM less idle while one
// of them ends a row and waits for the next one's first pages (64 sequences of 1 to 2,000 tokens 23.6 -> 15.8
// us); with eight a row that many CTAs share has half as many parts (1,048,576 tokens 6 % faster).
constexpr int kFew = 4, kMany = 8;
constexpr int kSmWarps = 16;                            // that the registers of an SM hold
constexpr int kStages = 2;                              // tiles of 32 tokens per warp in shared memory (three: 3 % slower)
constexpr int kBins = 256;                              // that the dense form's units are counted by
constexpr int kRowCost = 3;                             // pages' time that a row's end and the next one's start take
constexpr int kMaxParts = 4;                            // CTAs of a row up to which they form a cluster
constexpr int kGroup = 16, kMostFlat = 32;              // parts joined at a time where a row has more than kMostFlat
constexpr int kMostParts = 80;                          // of a row, up to which a kernel without groups is used (1-2 % faster)
constexpr int kMaxGrid = 1024;                          // CTAs per launch at most (sizes the workspace)
constexpr int kPart = kMaxG * kD + 2 * kMaxG;           // floats of a partial: O, m, l of eight heads
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kPShift = 8.f;                          // P is held as 2^(z - m + 8)
constexpr float kNoMax = -FLT_MAX;                      // m before a first score: finite, so that no difference is NaN
constexpr float kPMost = 32768.f;                       // most of a lane's sum of P (fp16 ends at 65504)

struct Params {
  int B, Hq, Hkv, G, k;
  // Units of a row.  Sparse: row_units for every one (k or a few more, the last ones without a page).  Dense: each
  // row's own pages and row_cost more, counted by bins of bin_size sequences.
  int row_units, bin_size, row_cost;
  bool whole_parts;                     // dense: the units may become parts of rows, one per CTA
  int parts;                            // sparse: CTAs of a row that form a cluster (0 or 1: none)
  float scale_log2, v_scale;
  const uint8_t* Q;
  int64_t q0, q1;                       // byte strides (b, h)
  const uint8_t *K_codes, *K_scales, *V_codes, *V_scales;
  int64_t c0, c1, s0, s1;               // byte strides (page, g)
  int64_t num_pages;
  const int32_t *pt, *n, *last_len;     // sparse
  const int32_t *seq_pt, *seq_len;      // dense
  int64_t max_pages;
  int32_t* counter;                     // [B * Hkv] parts (or groups of parts) of a row that have arrived, zero on entry
  int32_t* group_counter;               // [kMaxGrid][2] parts of a group that have arrived, zero on entry
  float* part;                          // [grid][2][kPart]
  __nv_bfloat16* O;
  float* LSE;
  int32_t* dev_err;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t h2u(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The low half of each byte of a and the high half of b's, in one instruction (written out, it takes two).
__device__ __forceinline__ uint32_t low_halves(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xE4;" : "=r"(r) : "r"(a), "r"(b), "r"(0x0f0f0f0fu));
  return r;
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// 16 bytes from the cache to shared memory, asynchronously and past L1: the cache is read once per step.
__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A warp's tile of 32 tokens in shared memory: K codes, V codes, K scales, V
// scales, rows as in the page but for V's 16-byte chunks, of which rows with bit 2 set hold
// them in the order 2, 3, 0, 1.  It is worked on as two halves of 16 rows.
// Row m of a half of S^T is token m ^ (m >> 1 & 1), so that the rows whose
// probabilities lane t holds after the transposition are tokens 2t and 2t + 1 (swapped
// for odd t) and these + 8.  With both, eight lanes that read 16 bytes of K, or
// sixteen that read 8 of V, meet every bank once.
constexpr int kTile = 32;
static_assert(kStages == 2, "the stages alternate");
constexpr int kVAt = kTile * 64, kKsAt = 2 * kVAt, kVsAt = kKsAt + kTile * 8, kTileBytes = kVsAt + kTile * 8;

__device__ __forceinline__ int token_of_row(int m) { return m ^ ((m >> 1) & 1); }

// Where a warp's tile of page 0 starts in the four pools, plus a lane's 16 bytes.
struct Bases {
  const uint8_t *kc, *vc, *scales;   // scales: K's in lanes 0-15, V's in lanes 16-31
};

// base + page * stride in one instruction (page strides lie below 2^32 bytes).
__device__ __forceinline__ const uint8_t* page_at(const uint8_t* base, uint32_t page, uint32_t stride) {
  uint64_t r;
  asm("mad.wide.u32 %0, %1, %2, %3;" : "=l"(r) : "r"(page), "r"(stride), "l"(reinterpret_cast<uint64_t>(base)));
  return reinterpret_cast<const uint8_t*>(r);
}

__device__ __forceinline__ void fetch_tile(const Bases& at, uint32_t page, uint32_t code_stride, uint32_t scale_stride,
                                           uint32_t dst, int lane) {
  const uint32_t dk = dst + lane * 16;                                  // row lane / 4, chunk lane % 4
  const uint32_t dv = dst + kVAt + (lane ^ ((lane >> 4) << 1)) * 16;    // chunk ^ 2 in rows 4-7 of 8
  const uint8_t* kc = page_at(at.kc, page, code_stride);
  const uint8_t* vc = page_at(at.vc, page, code_stride);
#pragma unroll
  for (int i = 0; i < kTile / 8; ++i) {
    copy16(dk + i * 512, kc + i * 512);
    copy16(dv + i * 512, vc + i * 512);
  }
  copy16(dk + kKsAt, page_at(at.scales, page, scale_stride));
}

// The softmax state of a warp: lane (g, t) holds heads 2t and 2t + 1, of which
// acc[i] are channels 16g + 2i (elements 0, 1) and 16g + 2i + 1 (elements 2, 3).
struct State {
  float acc[8][4];
  float m[2], l[2];      // m the same in every g; l this lane's share
};

// WHOLE: every token of the tile is live; else the first `valid` of them.
template <bool WHOLE>
__device__ __forceinline__ void attend_tile(const uint32_t (&q)[16], const float (&coef)[2], const uint8_t* tile, int valid,
                                            int g, int t, State* st) {
  float s[2][4];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const uint8_t* row = tile + (u * 16 + token_of_row(g)) * 64 + t * 16;
    const uint8_t* sf = tile + kKsAt + (u * 16 + token_of_row(g)) * 8 + t * 2;
    const uint4 ka = *reinterpret_cast<const uint4*>(row), kb = *reinterpret_cast<const uint4*>(row + 8 * 64);
    const __half2 sa = e4m3x2_to_half2(*reinterpret_cast<const uint16_t*>(sf));
    const __half2 sb = e4m3x2_to_half2(*reinterpret_cast<const uint16_t*>(sf + 8 * 8));
    const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) s[u][i] = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 fa = i < 2 ? __low2half2(sa) : __high2half2(sa), fb = i < 2 ? __low2half2(sb) : __high2half2(sb);
      __half2 a[4], b[4];
      e2m1x8_to_half2(wa[i], a);
      e2m1x8_to_half2(wb[i], b);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        a[e] = __hmul2(a[e], fa);
        b[e] = __hmul2(b[e], fb);
      }
      mma16816(s[u], h2u(a[0]), h2u(b[0]), h2u(a[1]), h2u(b[1]), q[4 * i], q[4 * i + 1]);
      mma16816(s[u], h2u(a[2]), h2u(b[2]), h2u(a[3]), h2u(b[3]), q[4 * i + 2], q[4 * i + 3]);
    }
  }
  if (!WHOLE) {          // slots past the last token may hold anything, a NaN scale too
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (u * 16 + token_of_row(g) + (i < 2 ? 0 : 8) >= valid) s[u][i] = -INFINITY;
  }
  // P as 2^(z - m + 8): infinite against kNoMax, and 0 where z is -inf.  A sum above 2^15
  // means that some score passed m by more than 5: m follows and P is formed again.
  // z is rounded before m goes off it, as m was: fused, scores of 2^24 and more left their product's rounding error, 2^x of
  // which is anything.  8 - m is rounded down, so that P ends at 2^8 where that sum is not exact (m of 2^27 and more).
  float e[2][4], sum[2];
  auto form = [&] {
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i) e[u][i] = ex2(__fadd_rn(__fmul_rn(s[u][i], coef[i & 1]), __fsub_rd(kPShift, st->m[i & 1])));
#pragma unroll
    for (int c = 0; c < 2; ++c) sum[c] = (e[0][c] + e[0][c + 2]) + (e[1][c] + e[1][c + 2]);
  };
  form();
  if (__any_sync(0xffffffffu, fmaxf(sum[0], sum[1]) > kPMost)) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float z = fmaxf(fmaxf(s[0][c], s[0][c + 2]), fmaxf(s[1][c], s[1][c + 2])) * coef[c];
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) z = fmaxf(z, __shfl_xor_sync(0xffffffffu, z, o));
      const float m = fmaxf(st->m[c], z);
      const float f = ex2(st->m[c] - m);
      st->m[c] = m;
      st->l[c] *= f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        st->acc[i][c] *= f;
        st->acc[i][c + 2] *= f;
      }
    }
    form();
  }
  st->l[0] += sum[0];
  st->l[1] += sum[1];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    // P^T: from (row g, heads 2t, 2t + 1) to (head g, rows 2t, 2t + 1)
    const uint32_t b0 = transpose8x8(h2u(__floats2half2_rn(e[u][0], e[u][1])));
    const uint32_t b1 = transpose8x8(h2u(__floats2half2_rn(e[u][2], e[u][3])));
    uint2 v[4];          // the tokens of rows 2t, 2t + 1 and these + 8, channels 16g .. 16g + 15
    uint32_t sf[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int tok = u * 16 + token_of_row(2 * t + (i & 1)) + 8 * (i >> 1);
      v[i] = *reinterpret_cast<const uint2*>(tile + kVAt + tok * 64 + ((g * 8) ^ ((tok & 4) << 3)));
      sf[i] = tile[kVsAt + tok * 8 + g];
    }
    if (!WHOLE) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (u * 16 + token_of_row(2 * t + (i & 1)) + 8 * (i >> 1) >= valid) sf[i] = 0;
    }
    const __half2 s01 = e4m3x2_to_half2(sf[0] | sf[1] << 8), s23 = e4m3x2_to_half2(sf[2] | sf[3] << 8);
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      // the codes of two tokens side by side: even and odd channels' bytes (token, next token)
      const uint32_t a = w ? v[0].y : v[0].x, b = w ? v[1].y : v[1].x;
      const uint32_t c = w ? v[2].y : v[2].x, d = w ? v[3].y : v[3].x;
      __half2 even01[4], odd01[4], even23[4], odd23[4];
      e2m1x8_to_half2(low_halves(a, b << 4), even01);
      e2m1x8_to_half2(low_halves(a >> 4, b), odd01);
      e2m1x8_to_half2(low_halves(c, d << 4), even23);
      e2m1x8_to_half2(low_halves(c >> 4, d), odd23);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        mma16816(st->acc[w * 4 + i], h2u(__hmul2(even01[i], s01)), h2u(__hmul2(odd01[i], s01)),
                 h2u(__hmul2(even23[i], s23)), h2u(__hmul2(odd23[i], s23)), b0, b1);
    }
  }
}

template <bool DENSE, int kWarps, bool TREE>
__global__ void __launch_bounds__(32 * kWarps, kSmWarps / kWarps) attn_q4_kernel(const Params p) {
  constexpr int kThreads = 32 * kWarps;
  constexpr int kTeams = kWarps / 4;        // four warps share a page, 32 tokens each; the teams alternate pages
  constexpr int kRep = 8 / kWarps;          // of the joined outputs' eight parts, those of a warp
  constexpr int kDeep = 8;                  // parts of a row that a lane loads at a time
  extern __shared__ __align__(128) uint8_t s_ring[];
  float4(*s_o)[8][32] = reinterpret_cast<float4(*)[8][32]>(s_ring);   // after a row's part: [warp][i][lane]
  __shared__ __align__(8) float s_m[kWarps][kMaxG], s_l[kWarps][kMaxG];
  __shared__ int s_pre[kBins + 1];          // dense: units before a bin of sequences (of one head)
  __shared__ int s_wsum[kWarps];
  __shared__ int s_last;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int rows = p.B * p.Hkv;
  wait_for_stream();

  // pages of one head of sequence x (dense) or of row x (sparse), and its units (dense)
  auto pages_of = [&](int x) {
    if (!DENSE) return min(max(p.n[x], 0), p.k);
    const int L = p.seq_len[x];
    return L < 0 || L > p.max_pages * kBk ? 0 : (L + kBk - 1) / kBk;
  };
  bool settled = !p.whole_parts;            // what a unit is
  int chunk = 1, row_cost = settled ? p.row_cost : 0;   // pages of a unit, units that a row has more
  auto units_of = [&](int x) {
    const int pages = pages_of(x);
    return pages > 0 ? (chunk > 1 ? (pages + chunk - 1) / chunk : pages) + row_cost : 0;
  };
  const int bins = DENSE ? (p.B + p.bin_size - 1) / p.bin_size : 0;
  if (DENSE) {
    constexpr int kPer = (kBins + kThreads - 1) / kThreads;
    int mine[kPer], sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int b = tid * kPer + i;
      mine[i] = 0;
      if (b < bins) {
        for (int x = b * p.bin_size; x < min(p.B, (b + 1) * p.bin_size); ++x) {
          mine[i] += units_of(x);
          if (blockIdx.x == 0 && (p.seq_len[x] < 0 || p.seq_len[x] > p.max_pages * kBk))
            report(p.dev_err, MSA_DEVERR_BAD_LEN);
        }
      }
      sum += mine[i];
    }
    while (true) {
      int inc = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
      }
      if (lane == 31) s_wsum[warp] = inc;
      __syncthreads();
      int before = inc - sum;
      for (int w = 0; w < warp; ++w) before += s_wsum[w];
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int b = tid * kPer + i;
        if (b <= bins) s_pre[b] = before;
        before += mine[i];
      }
      if (tid == kThreads - 1 && bins == kBins) s_pre[bins] = before;
      __syncthreads();
      if (settled) break;
      settled = true;
      // Few pages: a unit becomes a part of a row that is all a CTA has, if that makes the longest one at most
      // kRowCost pages longer (a row's end costs that much; 40 sequences of 437 to 1,825 tokens of one head 10.5 us
      // for 14.5).  ceil(x / c) <= x / c + 1, so as many fit.
      const int total = s_pre[bins] * p.Hkv, ctas = gridDim.x;
      const int pages = (total + ctas - rows - 1) / (ctas - rows);
      if (pages <= (total + ctas - 1) / ctas + kRowCost) chunk = max(pages, 1);
      else row_cost = p.row_cost;
      if (chunk == 1 && row_cost == 0) break;
      sum = 0;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        mine[i] = chunk > 1 ? (mine[i] + chunk - 1) / chunk : mine[i] > 0 ? mine[i] + row_cost : 0;
        sum += mine[i];
      }
      __syncthreads();                      // the pages' sums are read
    }
  }
  const int64_t units = DENSE ? static_cast<int64_t>(s_pre[bins]) * p.Hkv : static_cast<int64_t>(rows) * p.row_units;
  const uint32_t pool_pages = static_cast<uint32_t>(p.num_pages);
  const uint32_t code_stride = static_cast<uint32_t>(p.c0), scale_stride = static_cast<uint32_t>(p.s0);
  const int64_t per = (units + gridDim.x - 1) / gridDim.x;
  const int64_t lo = min(units, static_cast<int64_t>(blockIdx.x) * per), hi = min(units, lo + per);

  for (int64_t u = lo; u < hi;) {
    // the part of a row that starts at unit u: pages p0 .. p1 of its list
    int b, head, p0, row_pages, tokens;
    const int32_t* list;
    int item, rem;                          // sequence (dense) or row (sparse), and the unit within it
    if (DENSE) {
      int x = 0, y = bins;                  // the last bin whose units start at or before u
      while (y - x > 1) {
        const int mid = (x + y) >> 1;
        if (static_cast<int64_t>(s_pre[mid]) * p.Hkv <= u) x = mid; else y = mid;
      }
      item = x * p.bin_size;
      rem = static_cast<int>(u - static_cast<int64_t>(s_pre[x]) * p.Hkv);
      for (row_pages = units_of(item); rem >= row_pages * p.Hkv; row_pages = units_of(++item)) rem -= row_pages * p.Hkv;
    } else {
      item = static_cast<int>(u / p.row_units);
      rem = static_cast<int>(u - static_cast<int64_t>(item) * p.row_units);
      row_pages = p.row_units;
    }
    if (DENSE) {
      b = item;
      head = rem / row_pages;
      p0 = rem - head * row_pages;
      tokens = p.seq_len[b];
      list = p.seq_pt + b * p.max_pages;
    } else {
      b = item / p.Hkv;
      head = item - b * p.Hkv;
      p0 = rem;
      const int live = pages_of(item);
      tokens = live == 0 ? 0 : (live - 1) * kBk + min(max(p.last_len[item], 0), kBk);
      list = p.pt + static_cast<int64_t>(item) * p.k;
    }
    const int row = b * p.Hkv + head;
    const int64_t row_first = u - p0;
    int p1 = static_cast<int>(min(static_cast<int64_t>(row_pages), p0 + hi - u));
    u += p1 - p0;
    if (DENSE) {
      p0 *= chunk;
      p1 *= chunk;
    }

    // this warp's 32 tokens of its team's pages, the next one's in flight
    const int tok0 = (warp & 3) * kTile, j0 = p0 + (warp >> 2);
    const int live = min(p1, (tokens - tok0 + kBk - 1) / kBk);   // pages before here have a token of this warp's
    // (from lane 0: the compiler then knows that the warp goes one way)
    const int count = __shfl_sync(0xffffffffu, (live - j0 + kTeams - 1) / kTeams, 0);
    const Bases at = {p.K_codes + head * p.c1 + tok0 * 64 + lane * 16, p.V_codes + head * p.c1 + tok0 * 64 + lane * 16,
                      (lane < 16 ? p.K_scales : p.V_scales) + head * p.s1 + tok0 * 8 + (lane & 15) * 16};
    uint8_t* ring = s_ring + warp * (kStages * kTileBytes);
    // lane i: page of the i-th of the present run of 32 (known before the row's length, so both loads go together)
    const int listed = min(p1, DENSE ? static_cast<int>(p.max_pages) : p.k);
    int32_t ids = j0 + kTeams * lane < listed ? list[j0 + kTeams * lane] : -1;
    uint4 raw[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      raw[i] = make_uint4(0, 0, 0, 0);
      if (g < p.G) raw[i] = *reinterpret_cast<const uint4*>(p.Q + b * p.q0 + (head * p.G + g) * p.q1 + t * 64 + i * 16);
    }
    uint32_t bad = 0;                       // bit n % 32: the n-th page has no valid id
    int into = 0, from = 0;                 // byte offsets of the ring's next stages
    auto fetch = [&](int n) {
      if (n < count) {
        if ((n & 31) == 0 && n > 0) ids = j0 + kTeams * (n + lane) < listed ? list[j0 + kTeams * (n + lane)] : -1;
        const uint32_t page = __shfl_sync(0xffffffffu, ids, n & 31);
        if (page < pool_pages) {
          if (bad != 0) bad &= ~(1u << (n & 31));
          fetch_tile(at, page, code_stride, scale_stride, smem_u32(ring + into), lane);
        } else {
          bad |= 1u << (n & 31);
          if (lane == 0) report(p.dev_err, MSA_DEVERR_BAD_PAGE);
        }
      }
      into = kTileBytes - into;
      copies_commit();
    };
#pragma unroll
    for (int n = 0; n < kStages - 1; ++n) fetch(n);
    // Q of head g as fp16, scaled by a power of two: channels 32t + 2i, 32t + 2i + 1 in q[i]
    uint32_t q[16];
    float coef[2];
    {
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          top = fmaxf(top, fmaxf(fabsf(__uint_as_float(w[e] << 16)), fabsf(__uint_as_float(w[e] & 0xffff0000u))));
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int ex = min(max(static_cast<int>(__float_as_uint(top) >> 23), 1), 253);
      const float down = __uint_as_float(static_cast<uint32_t>(254 - ex) << 23);   // 2^(127 - ex)
      const float up = __uint_as_float(static_cast<uint32_t>(ex) << 23);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          q[4 * i + e] = h2u(__floats2half2_rn(__uint_as_float(w[e] << 16) * down, __uint_as_float(w[e] & 0xffff0000u) * down));
      }
#pragma unroll
      for (int c = 0; c < 2; ++c)
        coef[c] = fmaxf(__shfl_sync(0xffffffffu, up, 8 * t + 4 * c) * p.scale_log2, FLT_MIN);   // > 0: -inf stays so
    }
    State st;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) st.acc[i][e] = 0.f;
    st.m[0] = st.m[1] = kNoMax;
    st.l[0] = st.l[1] = 0.f;

    // all tiles but a warp's last one of a row are whole
    const int valid = tokens - (j0 + kTeams * (count - 1)) * kBk - tok0;   // live tokens from the last one's start on
    const int whole = count - (count > 0 && valid < kTile ? 1 : 0);
    auto next_tile = [&](int n) {           // waits for tile n and sends for the one kStages - 1 ahead; false: a bad page
      copies_wait<kStages - 2>();
      __syncwarp();                         // every lane's share of tile n is there, and tile n - 1 is read
      fetch(n + kStages - 1);
      return bad == 0 || (bad >> (n & 31) & 1) == 0;
    };
    for (int n = 0; n < whole; ++n) {
      if (next_tile(n)) attend_tile<true>(q, coef, ring + from, kTile, g, t, &st);
      from = kTileBytes - from;
    }
    if (whole < count && next_tile(whole)) attend_tile<false>(q, coef, ring + from, valid, g, t, &st);
    copies_wait<0>();
    __syncthreads();                        // the rings give way to the joined outputs

    // the warps' softmaxes joined, in the order the products left them: element [i][lane] of
    // a warp's outputs is its lane's acc[i], and a warp joins elements i = warp (and + 4) of all
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) st.l[c] += __shfl_xor_sync(0xffffffffu, st.l[c], o);
    if (g == 0) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        s_m[warp][2 * t + c] = st.m[c];
        s_l[warp][2 * t + c] = st.l[c];
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) s_o[warp][i][lane] = make_float4(st.acc[i][0], st.acc[i][1], st.acc[i][2], st.acc[i][3]);
    __syncthreads();
    float M[2] = {kNoMax, kNoMax}, l[2] = {0.f, 0.f};    // of heads 2t, 2t + 1
    float4 o[kRep];                                      // their channel 16g + 2i (x, y) and the next (z, w)
#pragma unroll
    for (int i = 0; i < kRep; ++i) o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](float4& x, float f0, float f1, float4 v) {
      x.x = fmaf(f0, v.x, x.x); x.y = fmaf(f1, v.y, x.y); x.z = fmaf(f0, v.z, x.z); x.w = fmaf(f1, v.w, x.w);
    };
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
#pragma unroll
      for (int c = 0; c < 2; ++c) M[c] = fmaxf(M[c], s_m[w][2 * t + c]);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      float f[2];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        f[c] = ex2(s_m[w][2 * t + c] - M[c]);
        l[c] = fmaf(f[c], s_l[w][2 * t + c], l[c]);
      }
#pragma unroll
      for (int i = 0; i < kRep; ++i) add(o[i], f[0], f[1], s_o[w][warp + i * kWarps][lane]);
    }
    // element [i][lane] of the row's outputs, of heads 2t, 2t + 1 for lane (g, t)
    auto put = [&](int i, int ln, float4 v, const float* sum, const float* top) {
      const float out[2][2] = {{v.x, v.z}, {v.y, v.w}};
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int h = 2 * (ln & 3) + c;
        if (h >= p.G) break;
        const int64_t at = static_cast<int64_t>(b) * p.Hq + head * p.G + h;
        const float r = sum[c] == 0.f ? 0.f : p.v_scale / sum[c];
        *reinterpret_cast<__nv_bfloat162*>(p.O + at * kD + 16 * (ln >> 2) + 2 * i) = __floats2bfloat162_rn(out[c][0] * r, out[c][1] * r);
        if (p.LSE != nullptr && i == 0 && ln < 4)
          p.LSE[at] = sum[c] == 0.f ? -INFINITY : (top[c] - kPShift + log2f(sum[c])) * kLn2;
      }
    };
    if (!DENSE && p.parts > 1) {
      // the row's parts are the CTAs of this cluster: joined through their shared memory, an equal share by each
      cg::cluster_group cluster = cg::this_cluster();
      const int parts = p.parts, rank = static_cast<int>(cluster.block_rank());
      float4* mine = reinterpret_cast<float4*>(s_ring);
      __syncthreads();                                   // the warps' outputs are read
#pragma unroll
      for (int i = 0; i < kRep; ++i) mine[tid + i * kThreads] = o[i];
      if (warp == 0 && g == 0) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          s_m[0][2 * t + c] = M[c];
          s_l[0][2 * t + c] = l[c];
        }
      }
      cluster.sync();
      const int item = tid * parts + rank;
      if (item < 256) {
        const int h0 = 2 * (item & 3);
        float m[kMaxParts][2], top[2] = {kNoMax, kNoMax}, sum[2] = {0.f, 0.f};
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int c = 0; c < kMaxParts; ++c) {
          if (c >= parts) break;
          const float2 x = *reinterpret_cast<const float2*>(cluster.map_shared_rank(&s_m[0][h0], c));
          m[c][0] = x.x;
          m[c][1] = x.y;
          top[0] = fmaxf(top[0], x.x);
          top[1] = fmaxf(top[1], x.y);
        }
#pragma unroll
        for (int c = 0; c < kMaxParts; ++c) {
          if (c >= parts) break;
          const float f0 = ex2(m[c][0] - top[0]), f1 = ex2(m[c][1] - top[1]);
          const float2 x = *reinterpret_cast<const float2*>(cluster.map_shared_rank(&s_l[0][h0], c));
          sum[0] = fmaf(f0, x.x, sum[0]);
          sum[1] = fmaf(f1, x.y, sum[1]);
          add(v, f0, f1, *cluster.map_shared_rank(mine + item, c));
        }
        put(item >> 5, item & 31, v, sum, top);
      }
      cluster.sync();                                    // no CTA leaves while another reads its memory
      return;
    }
    const int first = static_cast<int>(row_first / per), last = static_cast<int>((row_first + row_pages - 1) / per);
    bool write = first == last;
    if (!write) {
      // a part in the workspace: O as [8][32] float4, m [8], l [8]; slot 0: the one at the start
      // of a CTA's run, slot 1: the one at its end
      auto part_of = [&](int c) { return p.part + (static_cast<int64_t>(c) * 2 + (c * per >= row_first ? 0 : 1)) * kPart; };
      // The parts joined: CTAs base, base + step, .., `count` of them, by the last to arrive.  Many parts are joined
      // in groups first, whose results take the place of their first part (a CTA that reads 300 parts waits
      // for 38 rounds of loads: 1,000,000 tokens of one head 54 us for 36).
      const int members = last - first + 1;
      const bool tree = TREE && members > kMostFlat;
      const int group = tree ? (static_cast<int>(blockIdx.x) - first) / kGroup : 0;
      int own = blockIdx.x, base = first + group * kGroup, step = 1, count = tree ? min(kGroup, members - group * kGroup) : members;
      // (a CTA is the first of at most one group that starts a row and of one that does not)
      int32_t* counter = tree ? p.group_counter + 2 * base + (group == 0) : p.counter + row;
      while (true) {
        float* mine = part_of(own);
#pragma unroll
        for (int i = 0; i < kRep; ++i) reinterpret_cast<float4*>(mine)[tid + i * kThreads] = o[i];
        if (warp == 0 && g == 0) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            mine[kMaxG * kD + 2 * t + c] = M[c];
            mine[kMaxG * kD + kMaxG + 2 * t + c] = l[c];
          }
        }
        __threadfence();
        __syncthreads();
        if (tid == 0) s_last = atomicAdd(counter, 1) == count - 1;
        __syncthreads();
        if (s_last == 0) break;
        __threadfence();
        // 64 parts at a time: lane (g, t) takes m and l of parts g, g + 8, .. in one batch of
        // loads, and each lane its share of O kDeep parts deep
        M[0] = M[1] = kNoMax;
        l[0] = l[1] = 0.f;
#pragma unroll
        for (int i = 0; i < kRep; ++i) o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int c0 = 0; c0 < count; c0 += 64) {
          float2 m[8], sum[8];
          float top[2] = {M[0], M[1]};
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int c = c0 + g + 8 * k;
            m[k] = make_float2(kNoMax, kNoMax);
            sum[k] = make_float2(0.f, 0.f);
            if (c < count) {
              const float2* x = reinterpret_cast<const float2*>(part_of(base + c * step) + kMaxG * kD);
              m[k] = __ldcg(x + t);
              sum[k] = __ldcg(x + kMaxG / 2 + t);
            }
          }
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            top[0] = fmaxf(top[0], m[k].x);
            top[1] = fmaxf(top[1], m[k].y);
          }
#pragma unroll
          for (int c = 0; c < 2; ++c) {
#pragma unroll
            for (int i = 4; i < 32; i <<= 1) top[c] = fmaxf(top[c], __shfl_xor_sync(0xffffffffu, top[c], i));
          }
          const float s0 = ex2(M[0] - top[0]), s1 = ex2(M[1] - top[1]);
          M[0] = top[0];
          M[1] = top[1];
          float part_l[2] = {0.f, 0.f};
#pragma unroll
          for (int k = 0; k < 8; ++k) {      // m becomes the part's factor
            m[k].x = ex2(m[k].x - top[0]);
            m[k].y = ex2(m[k].y - top[1]);
            part_l[0] = fmaf(m[k].x, sum[k].x, part_l[0]);
            part_l[1] = fmaf(m[k].y, sum[k].y, part_l[1]);
          }
#pragma unroll
          for (int c = 0; c < 2; ++c) {
#pragma unroll
            for (int i = 4; i < 32; i <<= 1) part_l[c] += __shfl_xor_sync(0xffffffffu, part_l[c], i);
          }
          l[0] = fmaf(l[0], s0, part_l[0]);
          l[1] = fmaf(l[1], s1, part_l[1]);
#pragma unroll
          for (int i = 0; i < kRep; ++i) o[i] = make_float4(o[i].x * s0, o[i].y * s1, o[i].z * s0, o[i].w * s1);
#pragma unroll
          for (int k = 0; k < 8; k += kDeep / 8) {
            if (c0 + 8 * k >= count) break;
            float4 v[kDeep][kRep];
#pragma unroll
            for (int x = 0; x < kDeep; ++x)
#pragma unroll
              for (int i = 0; i < kRep; ++i) {
                v[x][i] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (c0 + 8 * k + x < count)
                  v[x][i] = __ldcg(reinterpret_cast<const float4*>(part_of(base + (c0 + 8 * k + x) * step)) + tid + i * kThreads);
              }
#pragma unroll
            for (int x = 0; x < kDeep; ++x) {
              const int from = x % 8 * 4 + t;
              const float f0 = __shfl_sync(0xffffffffu, m[k + x / 8].x, from), f1 = __shfl_sync(0xffffffffu, m[k + x / 8].y, from);
#pragma unroll
              for (int i = 0; i < kRep; ++i) add(o[i], f0, f1, v[x][i]);
            }
          }
        }
        if (tid == 0) *counter = 0;
        write = !tree || step > 1;
        if (write) break;
        own = base;
        base = first;
        step = kGroup;
        count = (members + kGroup - 1) / kGroup;
        counter = p.counter + row;
        __syncthreads();                    // the group's first part is read, and s_last
      }
    }
    if (write) {
#pragma unroll
      for (int i = 0; i < kRep; ++i) put(warp + i * kWarps, lane, o[i], l, M);
    }
    __syncthreads();
  }

  if (DENSE) {             // rows without a page have no units
    for (int r = blockIdx.x; r < rows; r += gridDim.x) {
      const int b = r / p.Hkv, head = r - b * p.Hkv;
      if (pages_of(b) != 0) continue;
      for (int h = warp; h < p.G; h += kWarps) {
        const int64_t at = static_cast<int64_t>(b) * p.Hq + head * p.G + h;
        *reinterpret_cast<uint2*>(p.O + at * kD + lane * 4) = make_uint2(0, 0);
        if (p.LSE != nullptr && lane == 0) p.LSE[at] = -INFINITY;
      }
    }
  }
}

// The workspace: the parts, then the counters of groups and rows.  They start at the same bytes for every B and Hkv,
// so that a call of one shape leaves those of another zero.
constexpr size_t kPartBytes = static_cast<size_t>(kMaxGrid) * 2 * kPart * sizeof(float);
constexpr size_t kGroupBytes = kMaxGrid * 2 * sizeof(int32_t);

template <class Args>
Params common_params(const Args& a, void* ws) {
  Params p = {};
  p.B = a.B; p.Hq = a.Hq; p.Hkv = a.Hkv; p.G = a.Hq / a.Hkv;
  const float scale = a.softmax_scale > 0.f ? a.softmax_scale : 1.0f / sqrtf(static_cast<float>(a.D));
  p.scale_log2 = scale * kLog2e * a.cache.k_scale;
  p.v_scale = a.cache.v_scale;
  p.Q = static_cast<const uint8_t*>(a.Q);
  p.q0 = a.Q_stride[0] * 2; p.q1 = a.Q_stride[1] * 2;
  p.K_codes = static_cast<const uint8_t*>(a.cache.K_codes);
  p.K_scales = static_cast<const uint8_t*>(a.cache.K_scales);
  p.V_codes = static_cast<const uint8_t*>(a.cache.V_codes);
  p.V_scales = static_cast<const uint8_t*>(a.cache.V_scales);
  p.c0 = a.cache.code_stride[0]; p.c1 = a.cache.code_stride[1];
  p.s0 = a.cache.scale_stride[0]; p.s1 = a.cache.scale_stride[1];
  p.num_pages = a.cache.num_pages;
  p.part = static_cast<float*>(ws);
  p.group_counter = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(ws) + kPartBytes);
  p.counter = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(ws) + kPartBytes + kGroupBytes);
  p.O = static_cast<__nv_bfloat16*>(a.O);
  p.LSE = a.LSE;
  p.dev_err = a.dev_err;
  return p;
}

template <bool DENSE, int kWarps, bool TREE>
msa_status launch(const Params& p, int grid, int scratch_zeroed, cudaStream_t stream) {
  if (!scratch_zeroed) {   // otherwise zero by contract (every error-free call leaves them zero)
    const cudaError_t e = cudaMemsetAsync(p.group_counter, 0, kGroupBytes + static_cast<size_t>(p.B) * p.Hkv * sizeof(int32_t), stream);
    if (e != cudaSuccess) return cuda_fail(e, "cudaMemsetAsync(4-bit decode counters)");
  }
  constexpr int smem = kWarps * std::max<int>(kStages * kTileBytes, kMaxG * kD * sizeof(float));
  cudaError_t e = cudaFuncSetAttribute(attn_q4_kernel<DENSE, kWarps, TREE>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(attn_q4)");
  e = launch_early(attn_q4_kernel<DENSE, kWarps, TREE>, grid, 32 * kWarps, smem, stream, std::max(p.parts, 1), p);
  if (e != cudaSuccess) return cuda_fail(e, "attn_q4_kernel launch");
  return MSA_OK;
}

// CTAs of this many warps that run at once.
msa_status room_for(int warps, int* room) {
  DeviceInfo dev;
  if (msa_status st = current_device(&dev); st != MSA_OK) return st;
  *room = std::min(dev.num_sms * (kSmWarps / warps), kMaxGrid);
  return MSA_OK;
}

}  // namespace

size_t attn_decode_q4_workspace_size(int B, int Hkv) {
  return kPartBytes + kGroupBytes + (static_cast<size_t>(B) * Hkv * sizeof(int32_t) + 255) / 256 * 256;
}

msa_status launch_sparse_decode_q4(const msa_decode_q4_args& a, void* ws, cudaStream_t stream) {
  int room;
  if (msa_status st = room_for(kFew, &room); st != MSA_OK) return st;
  Params p = common_params(a, ws);
  p.k = a.k;
  p.pt = a.pt; p.n = a.n; p.last_len = a.last_len;
  const int rows = a.B * a.Hkv;
  int grid = rows;
  if (rows <= room) {
    // Few rows: each is cut into equal parts, so that no CTA has pages of two rows (32 pages of 64 rows in runs of
    // 7 units, most of them across two rows, took a quarter longer).  Up to four parts are a cluster, which joins its
    // row without the workspace.  That costs so much less that four parts of up to eight pages, or two, are better
    // than parts for every CTA (64 rows of 16 pages 8.9 us for 10.3 in eight parts, 200 rows 16.5 for 18.1 in three);
    // longer rows take those, but few rows no more than half of them (8 rows of 64 pages 10.8 us for 13.4).
    // Clusters of three and four that nearly fill the GPU do not all fit at once (200 rows in three: 22.4 us for
    // 17.7 through the workspace); those of two do.
    const int cluster = 16 * rows <= 3 * room ? 4 : 2 * rows <= room ? 2 : 1;
    const int most = a.k <= 8 * cluster ? cluster : std::max((16 * rows <= room ? room / 2 : room) / rows, cluster);
    const int per = (a.k + most - 1) / most;
    const int parts = (a.k + per - 1) / per;
    p.row_units = parts * per;
    grid = rows * parts;
    p.parts = parts == 2 || (parts <= kMaxParts && 4 * grid <= 3 * room) ? parts : 1;
  } else {
    // Many rows: a CTA each, a new one where one ends.  (Equal runs of pages over the CTAs that run at once cut rows
    // and join them: 192 sequences of 16 pages 87 us for 80, 116 of 4 pages 27.4 for 20.7.)
    p.row_units = a.k;
  }
  return launch<false, kFew, false>(p, grid, a.scratch_zeroed, stream);
}

msa_status launch_dense_decode_q4(const msa_dense_decode_q4_args& a, void* ws, cudaStream_t stream) {
  int few, many;
  if (msa_status st = room_for(kFew, &few); st != MSA_OK) return st;
  if (msa_status st = room_for(kMany, &many); st != MSA_OK) return st;
  Params p = common_params(a, ws);
  p.seq_pt = a.seq_pt; p.seq_len = a.seq_len; p.max_pages = a.max_pages;
  p.bin_size = (a.B + kBins - 1) / kBins;
  const int64_t rows = static_cast<int64_t>(a.B) * a.Hkv;
  // Many rows, whose ends count (their lengths are on the device).  Four warps from half as many rows as there are
  // CTAs of eight on: 256 rows of 500 to 4,000 tokens 22 us for 29, of 30,000 tokens 173 for 171.
  if (2 * rows > many) {
    p.row_cost = kRowCost;
    p.whole_parts = p.bin_size == 1 && 2 * rows <= few;
    if (few > kMostParts * a.Hkv) return launch<true, kFew, true>(p, few, a.scratch_zeroed, stream);
    return launch<true, kFew, false>(p, few, a.scratch_zeroed, stream);
  }
  const int grid = static_cast<int>(std::min<int64_t>(many, rows * a.max_pages));
  p.whole_parts = p.bin_size == 1 && 2 * rows <= grid;
  // (a sequence may be all that there is to do, and its Hkv heads are equally long)
  if (grid > kMostParts * a.Hkv) return launch<true, kMany, true>(p, grid, a.scratch_zeroed, stream);
  return launch<true, kMany, false>(p, grid, a.scratch_zeroed, stream);
}

}  // namespace msa
