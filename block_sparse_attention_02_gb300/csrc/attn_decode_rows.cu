// attn_decode_rows.cu -- decode attention over a paged cache, one query a sequence: over 8-bit pages the selected
// ones (sparse), every cached token (dense) or a window with sinks; over bf16 pages a window with sinks.
//
//     z[h][t] = scale * Q[h] . K[t],  O[h] = sum_t softmax_t(z[h]) V[t],  LSE[h] = ln sum_t e^z
// for the G query heads that share a KV head, t over the tokens that the query sees.  A token costs 256 bytes (8 bits) or
// 512 (bf16), so HBM is the floor.
//
// Products.  mma.m16n8k16 with fp32 sums, straight from registers: S^T[t][h] with A = 16 tokens x 16 channels of K and
// B = Q (8 heads: G padded), O^T[d][h] with A = 16 channels x 16 tokens of V and B = P.  A 128-row tensor-memory tile
// would need the converted block written to shared memory and read back for eight columns.  The order of the channels in
// S's sum and of O's rows is free, so each lane takes whole 16-byte chunks of a row as they lie in the page.
//
// 8 bits.  A code is exact in fp16, its block's power of two multiplies the fp32 scores (K) or goes into P's
// exponent (V), so cached values enter unrounded.  Q is brought to [1, 2) per head by a power of two (exact, but for
// values below 2^-17 of a head's largest: multiples of 2^-24 of it); P is rounded once to fp16 (2^-11).
//   P is held as 2^(z - m + 8 + e - E), e the exponent of the V block and (m, E) a pair kept for each head: m the score
// and E the block exponent of some token so far.  What counts is the size of p * 2^e, the contribution to O: kept as
// two numbers the pair stays exact where m is large, and a block of large values after small ones (2^80 apart at most) does
// not overflow.  A tile whose sum passes 2^15 moves the pair; the sum of p itself, without 2^e, is taken beside it in fp32.
//   A block of small values after large ones would end in fp16's subnormals (from 2^-14 of P on, for equal scores 2^22 apart), and
// its channels may be ones that the large block leaves at 0.  So a tile whose e is more than kApart below E forms P against
// its own largest score, and its products are added to O in fp32 times what is left, 2^(z_max - m + e - E).  A token's weight is
// therefore off by 2^-11 of it, or by 2^-25 of the largest token's weight, whatever the blocks' scales.  (8 x 60,001 tokens with blocks
// of like scales 151 us, with every block but the first 2^28 below it 168.)
//   bf16 values need no e: P is rounded to bf16 (2^-8), as everywhere over bf16 pages.
//
// Work.  As in the 4-bit kernel: dense rows' pages form one list that CTAs share equally (or in whole parts of rows where
// there are few), sparse rows go to a CTA or a few; a warp takes tiles of 16 tokens through a ring of its own in
// shared memory; parts of a row are joined in shared memory, a cluster's shared memory, or through the workspace by the
// last CTA to arrive.  A window's pages are a list of their own: the sinks' pages, then those from the window's first
// token on; tiles of them without a visible token are not fetched.
//
// Bound.  HBM for long rows: 8 x 60,001 tokens of eight heads 150 us (6.5 TB/s, 97 % of a copy), 1,048,576 tokens 317 us (100 %); the
// conversions take a third of the issue slots (4 bits: two thirds).  A window of 4,096 over 64 sequences 69 us (84 %): rows'
// starts and ends.  Selected pages of many sequences: 64 / 192 of 16 pages 45 / 130 us (87 / 91 %).  Few rows are a launch, lengths, page ids, three to four tiles and a join, one after another: 8 x 16
// selected pages 10.6 us (floor 4.9), a window of 2,048 over 8 sequences of bf16 16.2 (10.0).
#include <cooperative_groups.h>
#include <cuda_fp16.h>

#include <cfloat>

#include "launch_early.cuh"
#include "msa_internal.h"
#include "msa_ptx.cuh"
#include "q8.cuh"

namespace cg = cooperative_groups;

namespace msa {
namespace {

constexpr int kFew = 4, kMany = 8;                      // warps of a CTA: four, and for few long rows eight
constexpr int kTile = 16;                               // tokens that a warp works on at a time
constexpr int kBins = 256;                              // that the dense form's units are counted by
constexpr int kRowCost = 2;                             // pages' time that a row's end and the next one's start take
constexpr int kMaxParts = 4;                            // CTAs of a row up to which they form a cluster
constexpr int kGroup = 16, kMostFlat = 32;              // parts joined at a time where a row has more than kMostFlat
constexpr int kMostParts = 80;                          // of a row, up to which a kernel without groups is used
constexpr int kMaxGrid = 1024;                          // CTAs per launch at most (sizes the workspace)
constexpr int kPart = kMaxG * kD + 2 * kMaxG;           // floats of a partial: O, m, l of eight heads
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kPShift = 8.f;                          // P is held as 2^(z - m + 8)
constexpr float kNoMax = -FLT_MAX;                      // m before a first score: finite, so that no difference is NaN
constexpr float kPMost = 32768.f;                       // most of a lane's sum of P (fp16 ends at 65504)
constexpr float kApart = 8.f;                           // a block's exponent may lie so far below E before its products are apart

// Dense rows and windows are shared out by the pages that each has; rows of at most k pages (selected ones, short windows) by k.
enum Mode { kSparse, kShortWindow, kDense, kWindow };
constexpr bool window_mode(Mode m) { return m == kWindow || m == kShortWindow; }

struct Params {
  int B, Hq, Hkv, G, k;
  // Units of a row.  Sparse: row_units for every one (k or a few more, the last ones without a page).  Dense: each
  // row's own pages and row_cost more, counted by bins of bin_size sequences.
  int row_units, bin_size, row_cost;
  bool whole_parts;                     // dense: the units may become parts of rows, one per CTA
  int parts;                            // sparse: CTAs of a row that form a cluster (0 or 1: none)
  int window, sinks;                    // kWindow
  float scale_log2;
  const uint8_t* Q;
  int64_t q0, q1;                       // byte strides (b, h)
  const uint8_t *K, *V, *K_scales, *V_scales;
  int64_t c0, c1, c2, s0, s1;           // byte strides (page, g, token) of K and V, (page, g) of the scales
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
__device__ __forceinline__ uint32_t b2u(__nv_bfloat162 h) { return *reinterpret_cast<uint32_t*>(&h); }
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
// 2^n of a whole number n in [-126, 127].
__device__ __forceinline__ float power_of_two(float n) { return __uint_as_float(static_cast<uint32_t>(127 + static_cast<int>(n)) << 23); }

// A tile in shared memory: 16 rows of K, then of V, their 16-byte chunks where eight lanes that read together meet every
// bank once.  K: lanes (g, t) read chunk 4 i + t of row g, so odd rows hold the chunks with bit 2 flipped.  V: lanes read the
// chunks of channels 16 g .. of rows 2 t (+ 1, + 8, + 9).
struct Q8 {
  static constexpr bool kScaled = true;
  static constexpr int kSmWarps = 16;                   // on an SM: registers, and 8 KiB of ring each
  static constexpr int kRow = kD, kSteps = 4;           // bytes of a row; copies of a lane for K (as many for V)
  static constexpr int kTileBytes = 2 * kTile * kRow;
  static __device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  }
  static __device__ __forceinline__ uint32_t pack(float a, float b) { return h2u(__floats2half2_rn(a, b)); }
  // the row and chunk of a lane's first copy; step i is 4 i rows on
  static __device__ __forceinline__ int row(int lane) { return lane >> 3; }
  static __device__ __forceinline__ int chunk(int lane) { return lane & 7; }
  static __device__ __forceinline__ uint32_t k_at(int lane) { return row(lane) * kRow + (chunk(lane) ^ ((row(lane) & 1) << 2)) * 16; }
  static __device__ __forceinline__ uint32_t v_at(int lane) { return row(lane) * kRow + (chunk(lane) ^ ((row(lane) >> 1) << 1)) * 16; }
  static __device__ __forceinline__ uint32_t v_step(int i) { return (i & 1) * 64; }
  // S += K Q: chunks t and t + 4 of rows g and g + 8
  static __device__ __forceinline__ void scores(const uint8_t* tile, const uint32_t (&q)[16], int g, int t, float (&s)[4]) {
    const uint8_t* at = tile + g * kRow;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int x = ((t + 4 * c) ^ ((g & 1) << 2)) * 16;
      const uint4 a = *reinterpret_cast<const uint4*>(at + x), b = *reinterpret_cast<const uint4*>(at + 8 * kRow + x);
      const uint32_t wa[4] = {a.x, a.y, a.z, a.w}, wb[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        uint32_t a0, a1, a2, a3;
        e4m3x4_to_f16(wa[w], &a0, &a2);
        e4m3x4_to_f16(wb[w], &a1, &a3);
        mma(s, a0, a1, a2, a3, q[(c * 4 + w) * 2], q[(c * 4 + w) * 2 + 1]);
      }
    }
  }
  // the two 16-byte loads of Q's head g that belong to chunk pair c: channels 16 (t + 4 c) ..
  static __device__ __forceinline__ int q_at(int t, int i) { return (t + 4 * (i >> 1)) * 32 + (i & 1) * 16; }
  struct Values {
    uint4 v[4];
  };
  // the tokens of rows 2t, 2t + 1 and these + 8, channels 16g .. 16g + 15
  static __device__ __forceinline__ void load(const uint8_t* tile, int g, int t, Values* x) {
    const uint8_t* at = tile + kTile * kRow + 2 * t * kRow + ((g ^ (t << 1)) & 7) * 16;
#pragma unroll
    for (int i = 0; i < 4; ++i) x->v[i] = *reinterpret_cast<const uint4*>(at + ((i & 1) + 8 * (i >> 1)) * kRow);
  }
  static __device__ __forceinline__ void drop(Values* x, int i) { x->v[i] = make_uint4(0, 0, 0, 0); }
  static __device__ __forceinline__ void outputs(const Values& x, uint32_t b0, uint32_t b1, float (&acc)[8][4]) {
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      auto word = [&](int i) { return w == 0 ? x.v[i].x : w == 1 ? x.v[i].y : w == 2 ? x.v[i].z : x.v[i].w; };
      uint32_t a0, a1, a2, a3;
      // (token, next token) of a channel side by side
      e4m3x4_to_f16(__byte_perm(word(0), word(1), 0x5140), &a0, &a1);
      e4m3x4_to_f16(__byte_perm(word(2), word(3), 0x5140), &a2, &a3);
      mma(acc[2 * w], a0, a1, a2, a3, b0, b1);
      e4m3x4_to_f16(__byte_perm(word(0), word(1), 0x7362), &a0, &a1);
      e4m3x4_to_f16(__byte_perm(word(2), word(3), 0x7362), &a2, &a3);
      mma(acc[2 * w + 1], a0, a1, a2, a3, b0, b1);
    }
  }
  // acc += by[head] * (V^T P), the products in fp32 of their own first; rows i with keep[i] only.  (Rare: a word of V at a time, so
  // that the registers are those of the common form.)
  static __device__ __forceinline__ void outputs_apart(const uint8_t* tile, int g, int t, const bool (&keep)[4], uint32_t b0,
                                                       uint32_t b1, const float (&by)[2], float (&acc)[8][4]) {
    const uint8_t* at = tile + kTile * kRow + 2 * t * kRow + ((g ^ (t << 1)) & 7) * 16;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      uint32_t v[4], a[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = keep[i] ? *reinterpret_cast<const volatile uint32_t*>(at + ((i & 1) + 8 * (i >> 1)) * kRow + (w >> 1) * 4) : 0;
      e4m3x4_to_f16(__byte_perm(v[0], v[1], w & 1 ? 0x7362 : 0x5140), &a[0], &a[1]);
      e4m3x4_to_f16(__byte_perm(v[2], v[3], w & 1 ? 0x7362 : 0x5140), &a[2], &a[3]);
      float own[4] = {0.f, 0.f, 0.f, 0.f};
      mma(own, a[0], a[1], a[2], a[3], b0, b1);
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[w][i] = fmaf(own[i], by[i & 1], acc[w][i]);
    }
  }
};

struct Bf16 {
  static constexpr bool kScaled = false;
  static constexpr int kSmWarps = 12;                   // on an SM: 16 KiB of ring each
  static constexpr int kRow = 2 * kD, kSteps = 8;
  static constexpr int kTileBytes = 2 * kTile * kRow;
  static __device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  }
  static __device__ __forceinline__ uint32_t pack(float a, float b) { return b2u(__floats2bfloat162_rn(a, b)); }
  static __device__ __forceinline__ int row(int lane) { return lane >> 4; }
  static __device__ __forceinline__ int chunk(int lane) { return lane & 15; }
  static __device__ __forceinline__ uint32_t k_at(int lane) { return row(lane) * kRow + (chunk(lane) ^ (row(lane) << 2)) * 16; }
  static __device__ __forceinline__ uint32_t v_at(int lane) { return row(lane) * kRow + chunk(lane) * 16; }
  static __device__ __forceinline__ uint32_t v_step(int i) { return ((i & 1) | ((i >> 1 & 1) << 2)) * 16; }
  // S += K Q: chunks t, t + 4, t + 8, t + 12 of rows g and g + 8
  static __device__ __forceinline__ void scores(const uint8_t* tile, const uint32_t (&q)[16], int g, int t, float (&s)[4]) {
    const uint8_t* at = tile + g * kRow;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int x = ((4 * i + t) ^ ((g & 1) << 2)) * 16;
      const uint4 a = *reinterpret_cast<const uint4*>(at + x), b = *reinterpret_cast<const uint4*>(at + 8 * kRow + x);
      mma(s, a.x, b.x, a.y, b.y, q[4 * i], q[4 * i + 1]);
      mma(s, a.z, b.z, a.w, b.w, q[4 * i + 2], q[4 * i + 3]);
    }
  }
  static __device__ __forceinline__ int q_at(int t, int i) { return (4 * i + t) * 16; }
  struct Values {
    uint4 v[4][2];
  };
  static __device__ __forceinline__ void load(const uint8_t* tile, int g, int t, Values* x) {
    const uint8_t* at = tile + kTile * kRow + 2 * t * kRow;
    const int flip = (t & 1) | ((t >> 1) << 2);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int c = 0; c < 2; ++c)
        x->v[i][c] = *reinterpret_cast<const uint4*>(at + ((i & 1) + 8 * (i >> 1)) * kRow + ((2 * g + c) ^ flip) * 16);
  }
  static __device__ __forceinline__ void drop(Values* x, int i) { x->v[i][0] = x->v[i][1] = make_uint4(0, 0, 0, 0); }
  static __device__ __forceinline__ void outputs(const Values& x, uint32_t b0, uint32_t b1, float (&acc)[8][4]) {
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      auto word = [&](int i) {
        const uint4& v = x.v[i][w >> 2];
        return (w & 3) == 0 ? v.x : (w & 3) == 1 ? v.y : (w & 3) == 2 ? v.z : v.w;
      };
      mma(acc[w], __byte_perm(word(0), word(1), 0x5410), __byte_perm(word(0), word(1), 0x7632),
          __byte_perm(word(2), word(3), 0x5410), __byte_perm(word(2), word(3), 0x7632), b0, b1);
    }
  }
};

// The softmax state of a warp: lane (g, t) holds heads 2t and 2t + 1, of which
// acc[i] are channels 16g + 2i (elements 0, 1) and 16g + 2i + 1 (elements 2, 3).
struct State {
  float acc[8][4];
  float m[2], E[2], l[2];      // m and E the same in every g; l this lane's share
};

// The tokens that a query sees, as places in the sequence: [first, end) and [0, sinks).
struct Seen {
  int first, end, sinks;
  __device__ __forceinline__ bool has(int pos) const { return pos < end && (pos >= first || pos < sinks); }
};

// WHOLE: every token of the tile is seen; else those of `seen`, the tile's first one being token a.  coef: the softmax scale
// in base 2 times the scales of Q's heads and of K's block; ev: exponent of V's block.
template <class F, bool WHOLE>
__device__ __forceinline__ void attend_tile(const uint32_t (&q)[16], const float (&coef)[2], float ev, const uint8_t* tile,
                                            const Seen& seen, int a, int g, int t, State* st) {
  float s[4] = {0.f, 0.f, 0.f, 0.f};
  F::scores(tile, q, g, t, s);
  if (!WHOLE) {          // other slots may hold anything, a NaN too
    if (!seen.has(a + g)) s[0] = s[1] = -INFINITY;
    if (!seen.has(a + g + 8)) s[2] = s[3] = -INFINITY;
  }
  // P as 2^(z - m + 8 + ev - E): infinite against kNoMax, and 0 where z is -inf.  A sum above 2^15 means that some token
  // passed the pair (m, E) by more than 4: the pair follows and P is formed again.  z is rounded before m goes off it, as m was:
  // fused, scores of 2^24 and more left their product's rounding error, 2^x of which is anything.
  float e[4], sum[2];
  auto form = [&] {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const float up = F::kScaled ? kPShift + (ev - st->E[c]) : kPShift;
#pragma unroll
      for (int i = c; i < 4; i += 2) e[i] = ex2(__fadd_rn(__fadd_rn(__fmul_rn(s[i], coef[c]), -st->m[c]), up));
      sum[c] = e[c] + e[c + 2];
    }
  };
  form();
  auto largest = [&](int c) {     // score of the tile, of head c (the same in every g)
    float z = __fmul_rn(fmaxf(s[c], s[c + 2]), coef[c]);
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) z = fmaxf(z, __shfl_xor_sync(0xffffffffu, z, o));
    return z;
  };
  auto far_below = [&] { return F::kScaled && ev < fmaxf(st->E[0], st->E[1]) - kApart; };
  bool apart = false;
  if (__any_sync(0xffffffffu, fmaxf(sum[0], sum[1]) > kPMost || far_below())) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const float z = largest(c);
      const float ahead = (z - st->m[c]) + (F::kScaled ? ev - st->E[c] : 0.f);
      if (ahead > 0.f) {
        const float f = ex2(-ahead);
        st->m[c] = z;
        if (F::kScaled) st->E[c] = ev;
        st->l[c] *= f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          st->acc[i][c] *= f;
          st->acc[i][c + 2] *= f;
        }
      }
    }
    form();
    apart = __any_sync(0xffffffffu, far_below());
  }
  const float down = F::kScaled ? power_of_two(-ev) : 1.f;
  st->l[0] = F::kScaled ? fmaf(sum[0], down, st->l[0]) : st->l[0] + sum[0];
  st->l[1] = F::kScaled ? fmaf(sum[1], down, st->l[1]) : st->l[1] + sum[1];
  // P^T: from (row g, heads 2t, 2t + 1) to (head g, rows 2t, 2t + 1)
  auto sees = [&](int i) { return WHOLE || seen.has(a + 2 * t + (i & 1) + 8 * (i >> 1)); };
  if constexpr (F::kScaled) {
    if (apart) {
      float by[2];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float z = largest(c), own = z == -INFINITY ? 0.f : z;
#pragma unroll
        for (int i = c; i < 4; i += 2) e[i] = ex2(__fadd_rn(__fadd_rn(__fmul_rn(s[i], coef[c]), -own), kPShift));
        // (-inf: no token of the tile is seen, every P is 0, and m may be none yet)
        by[c] = z == -INFINITY ? 0.f : ex2(__fadd_rn(__fadd_rn(own, -st->m[c]), ev - st->E[c]));
      }
      const bool keep[4] = {sees(0), sees(1), sees(2), sees(3)};
      F::outputs_apart(tile, g, t, keep, transpose8x8(F::pack(e[0], e[1])), transpose8x8(F::pack(e[2], e[3])), by, st->acc);
      return;
    }
  }
  const uint32_t b0 = transpose8x8(F::pack(e[0], e[1])), b1 = transpose8x8(F::pack(e[2], e[3]));
  typename F::Values v;
  F::load(tile, g, t, &v);
  if (!WHOLE) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (!sees(i)) F::drop(&v, i);
  }
  F::outputs(v, b0, b1, st->acc);
}

// STAGES: tiles of a warp in shared memory: two, three where there are few warps with bf16 pages.
template <class F, Mode MODE, int kWarps, bool TREE, int STAGES>
__global__ void __launch_bounds__(32 * kWarps, F::kSmWarps / kWarps) attn_rows_kernel(const Params p) {
  constexpr bool DENSE = MODE == kDense || MODE == kWindow, WINDOW = window_mode(MODE);
  constexpr int kThreads = 32 * kWarps;
  constexpr int kRep = 8 / kWarps;          // tiles of a page, and of the joined outputs' eight parts, those of a warp
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

  // what a sequence of L tokens (dense) shows its query: the first page of the window, and the sinks' pages before it
  auto first_of = [&](int L) { return WINDOW ? max(L - p.window, 0) : 0; };
  auto sink_pages = [&](int first) { return WINDOW ? min(static_cast<int>((min(p.sinks, first) + kBk - 1u) / kBk), first / kBk) : 0; };
  // pages of one head of sequence x (dense) or of row x (sparse), and its units (dense)
  auto pages_of = [&](int x) {
    if (MODE == kSparse) return min(max(p.n[x], 0), p.k);
    const int L = p.seq_len[x];
    if (L <= 0 || L > p.max_pages * kBk) return 0;
    const int first = first_of(L);
    return (L + kBk - 1) / kBk - first / kBk + sink_pages(first);
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
  const int64_t per = (units + gridDim.x - 1) / gridDim.x;
  const int64_t lo = min(units, static_cast<int64_t>(blockIdx.x) * per), hi = min(units, lo + per);

  for (int64_t u = lo; u < hi;) {
    // the part of a row that starts at unit u: pages p0 .. p1 of its list
    int b, head, p0, row_pages, live;       // live: the pages that the row has
    Seen seen;
    const int32_t* list;
    int item, rem;                          // sequence (dense) or row (sparse), and the unit within it
    int skip = 0, sink_end = 0;             // window: place n of the list is page n, from sink_end on page n + skip
    if (DENSE) {
      int x = 0, y = bins;                  // the last bin whose units start at or before u
      while (y - x > 1) {
        const int mid = (x + y) >> 1;
        if (static_cast<int64_t>(s_pre[mid]) * p.Hkv <= u) x = mid; else y = mid;
      }
      item = x * p.bin_size;
      rem = static_cast<int>(u - static_cast<int64_t>(s_pre[x]) * p.Hkv);
      for (row_pages = units_of(item); rem >= row_pages * p.Hkv; row_pages = units_of(++item)) rem -= row_pages * p.Hkv;
      b = item;
      head = rem / row_pages;
      p0 = rem - head * row_pages;
    } else {
      item = static_cast<int>(u / p.row_units);
      rem = static_cast<int>(u - static_cast<int64_t>(item) * p.row_units);
      row_pages = p.row_units;
      b = item / p.Hkv;
      head = item - b * p.Hkv;
      p0 = rem;
    }
    if (MODE == kSparse) {
      live = pages_of(item);
      seen.end = live == 0 ? 0 : (live - 1) * kBk + min(max(p.last_len[item], 0), kBk);
      seen.first = seen.sinks = 0;
      list = p.pt + static_cast<int64_t>(item) * p.k;
    } else {
      seen.end = p.seq_len[b];
      if (!DENSE && (seen.end < 0 || seen.end > p.max_pages * kBk)) {
        seen.end = 0;
        if (head == 0 && p0 == 0 && tid == 0) report(p.dev_err, MSA_DEVERR_BAD_LEN);
      }
      seen.first = first_of(seen.end);
      seen.sinks = WINDOW ? p.sinks : 0;
      sink_end = sink_pages(seen.first);
      skip = seen.first / kBk - sink_end;
      live = (seen.end + kBk - 1) / kBk - skip;
      list = p.seq_pt + b * p.max_pages;
    }
    const int row = b * p.Hkv + head;
    const int64_t row_first = u - p0;
    int p1 = static_cast<int>(min(static_cast<int64_t>(row_pages), p0 + hi - u));
    u += p1 - p0;
    if (DENSE) {
      p0 *= chunk;
      p1 *= chunk;
    }
    p1 = min(p1, live);

    // this warp's kRep tiles of each page, the next one in flight: tile n is of the list's page p0 + n / kRep, tokens
    // (warp * kRep + n % kRep) * kTile on.  The last page of the row may end before them.
    const int tail = seen.end - (live - 1 + skip) * kBk;         // tokens of the last page
    const int past = p1 < live || live == 0 ? 0 : kRep - min(max((tail + kTile - 1) / kTile - warp * kRep, 0), kRep);
    // (from lane 0: the compiler then knows that the warp goes one way)
    const int count = __shfl_sync(0xffffffffu, max(p1 - p0, 0) * kRep - (p1 > p0 ? past : 0), 0);
    const int tok0 = warp * kRep * kTile;
    const int64_t in_block = head * p.c1 + (tok0 + F::row(lane)) * p.c2 + F::chunk(lane) * 16;
    const uint8_t *k_base = p.K + in_block, *v_base = p.V + in_block;
    uint8_t* ring = s_ring + warp * (STAGES * F::kTileBytes);
    const uint32_t dk = smem_u32(ring) + F::k_at(lane), dv = smem_u32(ring) + kTile * F::kRow + F::v_at(lane);
    // Page ids (lane i: of the i-th of a run of 32 pages) and their blocks' scales (K's in the low byte) a run ahead
    auto page_id = [&](int n) {             // of the list's page p0 + n
      n += p0;
      return n < p1 ? list[n + (WINDOW && n >= sink_end ? skip : 0)] : -1;
    };
    auto scales_of = [&](int32_t id) {
      uint32_t x = 0;
      if (F::kScaled && id >= 0 && id < p.num_pages) {
        const int64_t at = id * p.s0 + head * p.s1;
        x = q8_byte(p.K_scales[at]) | q8_byte(p.V_scales[at]) << 8;
      }
      return x;
    };
    int32_t ids = page_id(lane), next_ids = -1;
    uint32_t scales = 0, old_scales = 0, next_scales = 0;
    uint4 raw[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      raw[i] = make_uint4(0, 0, 0, 0);
      if (g < p.G) raw[i] = *reinterpret_cast<const uint4*>(p.Q + b * p.q0 + (head * p.G + g) * p.q1 + F::q_at(t, i));
    }
    // where tile n starts in its sequence
    auto token_of = [&](int n) {
      const int j = p0 + n / kRep;
      return (j + (WINDOW && j >= sink_end ? skip : 0)) * kBk + tok0 + n % kRep * kTile;
    };
    // a tile that the query sees nothing of (window)
    auto unseen = [&](int a) { return WINDOW && a + kTile <= seen.first && a >= seen.sinks; };
    int into = 0, from = 0;                 // byte offsets of the ring's next stages
    uint32_t there = 0;                     // bit n % 32: tile n was fetched
    auto fetch = [&](int n) {               // (n falls into the next run of 32 pages before its tiles do)
      there &= ~(1u << (n & 31));
      if (n < count) {
        const int page_n = n / kRep;
        if ((n & (32 * kRep - 1)) == 0 && n > 0) {
          ids = next_ids;
          old_scales = scales;
          scales = next_scales;
        }
        if ((n & (32 * kRep - 1)) == 0) next_ids = page_id(page_n + 32 + lane);
        if (F::kScaled && (n & (32 * kRep - 1)) == 16 * kRep) next_scales = scales_of(next_ids);
        const int32_t page = __shfl_sync(0xffffffffu, ids, page_n & 31);
        if (static_cast<uint32_t>(page) < pool_pages) {
          if (!unseen(token_of(n))) {
            there |= 1u << (n & 31);
            const int64_t off = page * p.c0 + n % kRep * kTile * p.c2;
            const uint8_t *k = k_base + off, *v = v_base + off;
#pragma unroll
            for (int i = 0; i < F::kSteps; ++i) {
              copy16(dk + into + i * 512, k + i * (kTile / F::kSteps) * p.c2);
              copy16((dv + into + i * 512) ^ F::v_step(i), v + i * (kTile / F::kSteps) * p.c2);
            }
          }
        } else if (lane == 0) {
          report(p.dev_err, MSA_DEVERR_BAD_PAGE);
        }
      }
      into = into == (STAGES - 1) * F::kTileBytes ? 0 : into + F::kTileBytes;
      copies_commit();
    };
#pragma unroll
    for (int n = 0; n < STAGES - 1; ++n) fetch(n);
    if (F::kScaled) scales = scales_of(ids);
    // Q of head g as the products take it, in 8 bits' case as fp16 scaled by a power of two: pair e of its load i in q[4 i + e]
    uint32_t q[16];
    float coef[2];
    if (F::kScaled) {
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
      for (int c = 0; c < 2; ++c) coef[c] = __shfl_sync(0xffffffffu, up, 8 * t + 4 * c) * p.scale_log2;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        q[4 * i] = raw[i].x; q[4 * i + 1] = raw[i].y; q[4 * i + 2] = raw[i].z; q[4 * i + 3] = raw[i].w;
      }
      coef[0] = coef[1] = fmaxf(p.scale_log2, FLT_MIN);
    }
    State st;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) st.acc[i][e] = 0.f;
    st.m[0] = st.m[1] = kNoMax;
    st.E[0] = st.E[1] = 0.f;
    st.l[0] = st.l[1] = 0.f;

    for (int n = 0; n < count; ++n) {
      copies_wait<STAGES - 2>();
      __syncwarp();                         // every lane's share of tile n is there, and tile n - 1 is read
      fetch(n + STAGES - 1);
      if ((there >> (n & 31) & 1) != 0) {
        const int a = token_of(n);
        float tile_coef[2] = {coef[0], coef[1]}, ev = 0.f;
        if (F::kScaled) {
          // the fetches ahead may have moved on to the next run of pages
          const bool moved = (min(n + STAGES - 1, count - 1) ^ n) >= 32 * kRep;
          const uint32_t x = __shfl_sync(0xffffffffu, moved ? old_scales : scales, n / kRep & 31);
          ev = static_cast<float>(static_cast<int>(x >> 8) - 127);
#pragma unroll
          for (int c = 0; c < 2; ++c) tile_coef[c] = fmaxf(coef[c] * q8_scale(x & 0xffu), FLT_MIN);   // > 0: -inf stays so
        }
        if (a + kTile <= seen.end && (!WINDOW || a >= seen.first || a + kTile <= seen.sinks))
          attend_tile<F, true>(q, tile_coef, ev, ring + from, seen, a, g, t, &st);
        else
          attend_tile<F, false>(q, tile_coef, ev, ring + from, seen, a, g, t, &st);
      }
      from = from == (STAGES - 1) * F::kTileBytes ? 0 : from + F::kTileBytes;
    }
    copies_wait<0>();
    if (F::kScaled) {                       // outputs and sum of p alone, without 2^-E: below 2^(15 + 80 + 20)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float up = power_of_two(st.E[c]);
        st.l[c] *= up;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          st.acc[i][c] *= up;
          st.acc[i][c + 2] *= up;
        }
      }
    }
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
        const float r = sum[c] == 0.f ? 0.f : 1.f / sum[c];
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
  p.scale_log2 = scale * kLog2e;
  p.Q = static_cast<const uint8_t*>(a.Q);
  p.q0 = a.Q_stride[0] * 2; p.q1 = a.Q_stride[1] * 2;
  p.part = static_cast<float*>(ws);
  p.group_counter = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(ws) + kPartBytes);
  p.counter = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(ws) + kPartBytes + kGroupBytes);
  p.O = static_cast<__nv_bfloat16*>(a.O);
  p.LSE = a.LSE;
  p.dev_err = a.dev_err;
  return p;
}
void take_cache(const msa_q8_cache& c, Params* p) {
  p->K = static_cast<const uint8_t*>(c.K_codes);
  p->K_scales = static_cast<const uint8_t*>(c.K_scales);
  p->V = static_cast<const uint8_t*>(c.V_codes);
  p->V_scales = static_cast<const uint8_t*>(c.V_scales);
  p->c0 = c.code_stride[0]; p->c1 = c.code_stride[1]; p->c2 = kD;
  p->s0 = c.scale_stride[0]; p->s1 = c.scale_stride[1];
  p->num_pages = c.num_pages;
}

template <class F, Mode MODE, int kWarps, bool TREE, int STAGES = 2>
msa_status launch(const Params& p, int grid, int scratch_zeroed, cudaStream_t stream) {
  if (!scratch_zeroed) {   // otherwise zero by contract (every error-free call leaves them zero)
    const cudaError_t e = cudaMemsetAsync(p.group_counter, 0, kGroupBytes + static_cast<size_t>(p.B) * p.Hkv * sizeof(int32_t), stream);
    if (e != cudaSuccess) return cuda_fail(e, "cudaMemsetAsync(decode counters)");
  }
  constexpr int smem = kWarps * std::max<int>(STAGES * F::kTileBytes, kMaxG * kD * sizeof(float));
  cudaError_t e = cudaFuncSetAttribute(attn_rows_kernel<F, MODE, kWarps, TREE, STAGES>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(attn_rows)");
  e = launch_early(attn_rows_kernel<F, MODE, kWarps, TREE, STAGES>, grid, 32 * kWarps, smem, stream, std::max(p.parts, 1), p);
  if (e != cudaSuccess) return cuda_fail(e, "attn_rows_kernel launch");
  return MSA_OK;
}

// CTAs of this many warps that run at once.
template <class F>
msa_status room_for(int warps, int* room) {
  DeviceInfo dev;
  if (msa_status st = current_device(&dev); st != MSA_OK) return st;
  *room = std::min(dev.num_sms * (F::kSmWarps / warps), kMaxGrid);
  return MSA_OK;
}

// Rows of `most` pages each at most (known on the host; their lengths are on the device).
template <class F, Mode MODE>
msa_status launch_lists(Params p, int64_t most, int scratch_zeroed, cudaStream_t stream) {
  int few, many;
  if (msa_status st = room_for<F>(kFew, &few); st != MSA_OK) return st;
  if (msa_status st = room_for<F>(kMany, &many); st != MSA_OK) return st;
  p.bin_size = (p.B + kBins - 1) / kBins;
  const int64_t rows = static_cast<int64_t>(p.B) * p.Hkv;
  if (!F::kScaled || 2 * rows > many) {     // many rows, whose ends count
    const int grid = static_cast<int>(std::min<int64_t>(few, rows * most));
    p.row_cost = kRowCost;
    p.whole_parts = p.bin_size == 1 && 2 * rows <= grid;
    if (grid > kMostParts * p.Hkv) return launch<F, MODE, kFew, true>(p, grid, scratch_zeroed, stream);
    return launch<F, MODE, kFew, false>(p, grid, scratch_zeroed, stream);
  }
  if constexpr (F::kScaled) {
    const int grid = static_cast<int>(std::min<int64_t>(many, rows * most));
    p.whole_parts = p.bin_size == 1 && 2 * rows <= grid;
    // (a sequence may be all that there is to do, and its Hkv heads are equally long)
    if (grid > kMostParts * p.Hkv) return launch<F, MODE, kMany, true>(p, grid, scratch_zeroed, stream);
    return launch<F, MODE, kMany, false>(p, grid, scratch_zeroed, stream);
  }
  return MSA_OK;
}

// Rows of up to k pages each.
template <class F, Mode MODE>
msa_status launch_rows(Params p, int scratch_zeroed, cudaStream_t stream) {
  DeviceInfo dev;
  if (msa_status st = current_device(&dev); st != MSA_OK) return st;
  int room;
  if (msa_status st = room_for<F>(kFew, &room); st != MSA_OK) return st;
  const int rows = p.B * p.Hkv;
  int grid = rows;
  if (rows <= room) {
    // Few rows: each is cut into equal parts, so that no CTA has pages of two rows.  Up to four parts are a cluster, which
    // joins its row without the workspace; clusters of three and four that nearly fill the GPU do not all fit at once.
    const int cluster = 16 * rows <= 3 * room ? 4 : 2 * rows <= room ? 2 : 1;
    const int most = p.k <= 8 * cluster ? cluster : std::max((16 * rows <= room ? room / 2 : room) / rows, cluster);
    const int per = (p.k + most - 1) / most;
    const int parts = (p.k + per - 1) / per;
    p.row_units = parts * per;
    grid = rows * parts;
    p.parts = parts == 2 || (parts <= kMaxParts && 4 * grid <= 3 * room) ? parts : 1;
  } else {
    p.row_units = p.k;                      // many rows: a CTA each, a new one where one ends
  }
  // Few CTAs: those over 8-bit pages get eight warps (8 rows of 16 pages 8.3 us for 9.6, 64 rows 12.1 for 13.1), those over
  // bf16 pages, whose ring is twice as large, a third stage (64 rows of 17 pages 16.1 for 17.3).
  if (grid <= 2 * dev.num_sms) return launch<F, MODE, F::kScaled ? kMany : kFew, false, F::kScaled ? 2 : 3>(p, grid, scratch_zeroed, stream);
  return launch<F, MODE, kFew, false>(p, grid, scratch_zeroed, stream);
}

// A window's rows have at most the window's pages (its first token anywhere in a page) and the sinks'.
template <class F>
msa_status launch_window(Params p, int scratch_zeroed, cudaStream_t stream) {
  const int64_t most = std::min<int64_t>(p.max_pages, (static_cast<int64_t>(p.window) + kBk - 2) / kBk + 1 + (static_cast<int64_t>(p.sinks) + kBk - 1) / kBk);
  int room;
  if (msa_status st = room_for<F>(kFew, &room); st != MSA_OK) return st;
  if (most > kMaxK || 2 * p.B * p.Hkv > room) return launch_lists<F, kWindow>(p, most, scratch_zeroed, stream);
  p.k = static_cast<int>(most);
  return launch_rows<F, kShortWindow>(p, scratch_zeroed, stream);
}

}  // namespace

size_t attn_rows_workspace_size(int B, int Hkv) {
  return kPartBytes + kGroupBytes + (static_cast<size_t>(B) * Hkv * sizeof(int32_t) + 255) / 256 * 256;
}

msa_status launch_sparse_decode_q8(const msa_decode_q8_args& a, void* ws, cudaStream_t stream) {
  Params p = common_params(a, ws);
  take_cache(a.cache, &p);
  p.k = a.k;
  p.pt = a.pt; p.n = a.n; p.last_len = a.last_len;
  return launch_rows<Q8, kSparse>(p, a.scratch_zeroed, stream);
}

msa_status launch_dense_decode_q8(const msa_dense_decode_q8_args& a, void* ws, cudaStream_t stream) {
  Params p = common_params(a, ws);
  take_cache(a.cache, &p);
  p.seq_pt = a.seq_pt; p.seq_len = a.seq_len; p.max_pages = a.max_pages;
  p.window = a.window; p.sinks = a.sinks;
  if (a.window == 0) return launch_lists<Q8, kDense>(p, a.max_pages, a.scratch_zeroed, stream);
  return launch_window<Q8>(p, a.scratch_zeroed, stream);
}

msa_status launch_window_decode(const msa_window_decode_args& a, void* ws, cudaStream_t stream) {
  Params p = common_params(a, ws);
  p.K = static_cast<const uint8_t*>(a.K_pool);
  p.V = static_cast<const uint8_t*>(a.V_pool);
  p.c0 = a.kv_stride[0] * 2; p.c1 = a.kv_stride[1] * 2; p.c2 = a.kv_stride[2] * 2;
  p.num_pages = a.num_pages;
  p.seq_pt = a.seq_pt; p.seq_len = a.seq_len; p.max_pages = a.max_pages;
  p.window = a.window; p.sinks = a.sinks;
  return launch_window<Bf16>(p, a.scratch_zeroed, stream);
}

}  // namespace msa
