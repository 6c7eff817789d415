// qk_norm_rope.cu -- RMS norm of every query and key head and the position
// rotation in one pass, the keys and values written straight into their pages.
//
// Per token and head of D values:  y = x * rsqrt(mean(x^2) + eps) * w, then the
// first rot values turned in pairs (a, b) -> (a cos t - b sin t, b cos t + a sin t)
// with t = pos * inv_freq[i].  All of it in fp32 with one rounding at the end.
//
// The angle.  A position of a million times a frequency near 1 needs more than
// fp32's 24 bits.  Only the fraction of a turn matters, so each lane keeps its
// frequencies as turns per token in 64-bit fixed point (2^64 = one turn) and
// pos * that, modulo 2^64, is the angle: one integer product, off by at most 2^-43
// turns at 2^20 tokens (two units of 2^-64 turns a token), for frequencies of any size.
//
// Layout: D / 16 lanes hold a head, 16 values each as two 16-byte chunks that
// contain both members of every pair (chunks i and i + rot / 16 for split pairs,
// any chunk for adjacent ones), so the rotation needs no exchange and the norm
// log2(D / 16) shuffles.  The chunks past the rotated ones are taken so that neighbouring lanes'
// lie side by side (in twos per lane, each request had half of a 32-byte sector: 16,384 tokens
// with half of each head rotated 106 us for 87).  A warp takes one token and walks its heads, which
// share the token's sines; with few tokens the heads are split over warps.
//
// Bound: HBM, every value read and written once: 65,536 tokens of 48 + 8 + 8 heads of
// 128 in 318 us, the copy rate.  Each lane copies its chunks into shared memory
// three steps (of four or eight heads) ahead, across tokens (370 us with plain loads).  16
// warps on an SM are enough, and more in flight serves HBM worse: 323 us with four steps ahead, 325 with 18 or
// 20 warps and two, 338 with 24 and two, 351 with 24 and three.  4,097 tokens of 40 heads of 64,
// which fit L2: 11.5 us (floor 6.2), bound by latency (issue 45 %): two rounds of tokens on 2,432 warps, each a
// position, its sines and five steps; 8 tokens: 3.3 us, a launch's latency.
#include "launch_early.cuh"
#include "msa_internal.h"
#include "msa_ptx.cuh"

namespace msa {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kCtasPerSm = 4;
constexpr int kAhead = 4;                     // steps of 1 KiB per warp in shared memory, one of them worked on

struct NormRopeParams {
  int64_t N, num_pages;
  int Hq, Hkv, rot, weight_fp32, parts;
  float eps;
  const uint8_t *Q, *K, *V;
  int64_t q0, q1, k0, k1, v0, v1;             // byte strides (n, h)
  const int32_t* pos;
  const float* inv_freq;
  const void *q_weight, *k_weight;
  uint8_t *Q_out, *K_out, *V_out;
  int64_t qo0, qo1;                           // byte strides (n, h)
  int64_t ko0, ko1, ko2, vo0, vo1, vo2;       // (n, h, -), or (page, g, t) with slots
  const int64_t* slots;
  int32_t* dev_err;
};

__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void unpack8(const uint4 u, float* x) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float* x) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// 1 / (2 pi), 2^-1 in the top bit of the first word: enough words for the 96 bits at any power of two of a float.
__constant__ uint32_t kTurnWords[7] = {0x28be60db, 0x9391054a, 0x7f09d5f4, 0x7d4d3770, 0x36d8a566, 0x4f10e410, 0x7f9458ea};
// f / (2 pi) modulo 1 in units of 2^-64, off by two of them at most, for any finite f (Payne and Hanek, "Radian
// reduction for trigonometric functions", 1983: of 1 / (2 pi) only the bits that reach the fraction are multiplied): f's
// 24 bits times 96 of 1 / (2 pi), shifted.  (In doubles, which this GPU has few units for: 500 tokens 7 % slower.)
__device__ __forceinline__ uint64_t turns_of(float f) {
  const uint32_t bits = __float_as_uint(f), ex = bits >> 23 & 0xff;
  const uint64_t m = (bits & 0x7fffffu) | (ex != 0 ? 0x800000u : 0u);       // f = m * 2^(max(ex, 1) - 150)
  uint32_t w0 = 0x28be60db, w1 = 0x9391054a, w2 = 0x7f09d5f4;
  if (ex > 150) {          // 2^24 or more: the bits before the window give whole turns
    const uint32_t up = ex - 150, i = min(up >> 5, 3u);                     // (3: infinite and NaN)
    w0 = __funnelshift_l(kTurnWords[i + 1], kTurnWords[i], up);
    w1 = __funnelshift_l(kTurnWords[i + 2], kTurnWords[i + 1], up);
    w2 = __funnelshift_l(kTurnWords[i + 3], kTurnWords[i + 2], up);
  }
  const uint64_t low = m * w2, mid = m * w1 + (low >> 32), top = m * w0 + (mid >> 32);   // of the product's 2^-96 turns
  const uint32_t down = ex < 150 ? 150 - max(ex, 1u) : 0;                   // of top and mid's 32 bits, from 2^-64 turns
  uint64_t t = down < 32 ? top << (32 - down) | static_cast<uint32_t>(mid) >> down : down < 96 ? top >> (down - 32) : 0;
  return bits >> 31 ? 0 - t : t;
}

template <int D, bool PAIRS>   // PAIRS: the rotated pairs are neighbours (2i, 2i + 1)
__global__ void __launch_bounds__(kThreads, kCtasPerSm) norm_rope_kernel(const NormRopeParams p) {
  constexpr int kLanes = D / 16;              // lanes per head
  constexpr int kHeads = 32 / kLanes;         // heads per warp and step
  __shared__ __align__(16) float s_weight[2][D];
  __shared__ float2 s_turn[kWarps][D / 2];    // cosine and sine of every pair of a warp's token
  __shared__ __align__(16) uint8_t s_ring[kWarps][kAhead * 1024];
  wait_for_stream();
  // (from lane 0: the compiler then knows that a warp goes one way; 4,097 tokens 4 % faster)
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int sub = lane % kLanes, hl = lane / kLanes;
  const int half = p.rot >> 4;                // chunks of 8 values in each half of the rotated ones
  int c0, c1;                                 // this lane's chunks
  bool turn0, turn1;
  if (PAIRS) {
    c0 = sub;
    c1 = sub + kLanes;
    turn0 = c0 < 2 * half;
    turn1 = c1 < 2 * half;
  } else {
    c0 = sub < half ? sub : sub + half;
    c1 = sub < half ? sub + half : sub + kLanes;
    turn0 = turn1 = sub < half;
  }
  const int q_steps = (p.Hq + kHeads - 1) / kHeads, k_steps = (p.Hkv + kHeads - 1) / kHeads;
  const int steps = q_steps + k_steps + (p.V != nullptr ? k_steps : 0);
  const int64_t items = p.N * p.parts, stride = static_cast<int64_t>(gridDim.x) * kWarps;
  const int64_t item0 = static_cast<int64_t>(blockIdx.x) * kWarps + warp;

  // The loads run kAhead - 1 steps before the work, across tokens (they need no position): each lane
  // copies its two chunks into shared memory places that it alone reads.
  const uint32_t ring = smem_u32(s_ring[warp]) + lane * 16;
  int64_t load_item = item0, load_n = 0;
  int load_step = 0;
  uint32_t load_at = 0, read_at = 0;
  auto load_token = [&] {
    load_n = p.parts == 1 ? load_item : load_item / p.parts;
    load_step = p.parts == 1 ? 0 : static_cast<int>(load_item - load_n * p.parts);
  };
  auto fetch = [&] {
    if (load_item < items) {
      const bool is_q = load_step < q_steps, is_v = load_step >= q_steps + k_steps;
      const int head = (load_step - (is_q ? 0 : is_v ? q_steps + k_steps : q_steps)) * kHeads + hl;
      if (head < (is_q ? p.Hq : p.Hkv)) {
        const uint8_t* src = is_q   ? p.Q + load_n * p.q0 + head * p.q1
                             : is_v ? p.V + load_n * p.v0 + head * p.v1
                                    : p.K + load_n * p.k0 + head * p.k1;
        copy16(ring + load_at, src + c0 * 16);
        copy16(ring + load_at + 512, src + c1 * 16);
      }
      load_at = load_at + 1024 == kAhead * 1024 ? 0 : load_at + 1024;
      load_step += p.parts;
      if (load_step >= steps) {
        load_item += stride;
        if (load_item < items) load_token();
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  if (load_item < items) load_token();
#pragma unroll
  for (int i = 0; i < kAhead - 1; ++i) fetch();
  for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
    const void* w = i < D ? p.q_weight : p.k_weight;
    float x = 1.f;
    if (w != nullptr)
      x = p.weight_fp32 ? static_cast<const float*>(w)[i % D] : __bfloat162float(static_cast<const __nv_bfloat16*>(w)[i % D]);
    s_weight[i / D][i % D] = x;
  }
  // turns per token, in units of 2^-64 turns, of pairs lane and lane + 32
  uint64_t turns[D / 64];
  float half_turns[D / 64];                   // in a unit of an angle's top 32 bits: 2^-31, or NaN where the frequency is not finite
#pragma unroll
  for (int e = 0; e < D / 64; ++e) {
    turns[e] = 0;
    half_turns[e] = 4.656612873077393e-10f;
    if (lane + 32 * e < p.rot / 2) {
      const float f = p.inv_freq[lane + 32 * e];
      turns[e] = turns_of(f);
      if (!isfinite(f)) half_turns[e] = NAN;
    }
  }
  __syncthreads();

  bool bad = false;
  for (int64_t item = item0; item < items; item += stride) {
    const int64_t n = p.parts == 1 ? item : item / p.parts;
    const int first = p.parts == 1 ? 0 : static_cast<int>(item - n * p.parts);
    const int pos = p.pos[n];
    const bool store_q = pos >= 0;
    // where this token's key and value rows go
    int64_t k_row = n * p.ko0, v_row = 0;
    bool store_kv = store_q;
    if (p.slots != nullptr) {
      const int64_t slot = p.slots[n], page = slot / kBk;
      const int t = static_cast<int>(slot & (kBk - 1));
      store_kv = store_q && slot >= 0 && page < p.num_pages;
      bad |= store_q && slot >= 0 && page >= p.num_pages;
      k_row = page * p.ko0 + t * p.ko2;
      v_row = page * p.vo0 + t * p.vo2;
    }
    __syncwarp();                             // the last token's turns are read
#pragma unroll
    for (int e = 0; e < D / 64; ++e) {
      if (lane + 32 * e < p.rot / 2) {
        const int32_t a = static_cast<int32_t>((turns[e] * static_cast<uint64_t>(max(pos, 0))) >> 32);
        float2 cs;
        sincospif(static_cast<float>(a) * half_turns[e], &cs.y, &cs.x);
        s_turn[warp][lane + 32 * e] = cs;
      }
    }
    __syncwarp();
    float cs[8], sn[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int i = PAIRS ? 4 * (e < 4 ? c0 : c1) + (e & 3) : 8 * sub + e;
      const float2 v = (e < 4 ? turn0 : turn1) ? s_turn[warp][i] : make_float2(1.f, 0.f);
      cs[e] = v.x;
      sn[e] = v.y;
    }
    for (int step = first; step < steps; step += p.parts) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 2) : "memory");
      const uint4 u0 = *reinterpret_cast<const uint4*>(s_ring[warp] + read_at + lane * 16);
      const uint4 u1 = *reinterpret_cast<const uint4*>(s_ring[warp] + read_at + 512 + lane * 16);
      read_at = read_at + 1024 == kAhead * 1024 ? 0 : read_at + 1024;
      fetch();
      const bool is_q = step < q_steps, is_v = step >= q_steps + k_steps;
      const int head = (step - (is_q ? 0 : is_v ? q_steps + k_steps : q_steps)) * kHeads + hl;
      const bool live = head < (is_q ? p.Hq : p.Hkv) && (is_q ? store_q : store_kv);
      if (is_v) {                             // values go as they are
        if (live) {
          uint8_t* dst = p.V_out + v_row + head * p.vo1;
          *reinterpret_cast<uint4*>(dst + c0 * 16) = u0;
          *reinterpret_cast<uint4*>(dst + c1 * 16) = u1;
        }
        continue;
      }
      float x[16];
      unpack8(u0, x);
      unpack8(u1, x + 8);
      if ((is_q ? p.q_weight : p.k_weight) != nullptr) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
        for (int o = 1; o < kLanes; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float r = rsqrtf(ss * (1.0f / D) + p.eps);
        const float* w = s_weight[is_q ? 0 : 1];
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
          const float4 f = *reinterpret_cast<const float4*>(w + (i < 8 ? c0 * 8 + i : c1 * 8 + i - 8));
          x[i] *= r * f.x;
          x[i + 1] *= r * f.y;
          x[i + 2] *= r * f.z;
          x[i + 3] *= r * f.w;
        }
      }
      if (PAIRS) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (e < 4 ? turn0 : turn1) {
            const float a = x[2 * e], b = x[2 * e + 1];
            x[2 * e] = a * cs[e] - b * sn[e];
            x[2 * e + 1] = b * cs[e] + a * sn[e];
          }
        }
      } else if (turn0) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float a = x[e], b = x[8 + e];
          x[e] = a * cs[e] - b * sn[e];
          x[8 + e] = b * cs[e] + a * sn[e];
        }
      }
      if (live) {
        uint8_t* dst = is_q ? p.Q_out + n * p.qo0 + head * p.qo1 : p.K_out + k_row + head * p.ko1;
        *reinterpret_cast<uint4*>(dst + c0 * 16) = pack8(x);
        *reinterpret_cast<uint4*>(dst + c1 * 16) = pack8(x + 8);
      }
    }
  }
  if (bad && lane == 0) report(p.dev_err, MSA_DEVERR_BAD_PAGE);
}

}  // namespace

msa_status launch_qk_norm_rope(const msa_norm_rope_args& a, cudaStream_t stream) {
  DeviceInfo dev;
  if (msa_status st = current_device(&dev); st != MSA_OK) return st;
  NormRopeParams p;
  p.N = a.N; p.num_pages = a.num_pages; p.Hq = a.Hq; p.Hkv = a.Hkv; p.rot = a.rot;
  p.weight_fp32 = a.weight_fp32; p.eps = a.eps;
  p.Q = static_cast<const uint8_t*>(a.Q);
  p.K = static_cast<const uint8_t*>(a.K);
  p.V = static_cast<const uint8_t*>(a.V);
  p.q0 = a.Q_stride[0] * 2; p.q1 = a.Q_stride[1] * 2;
  p.k0 = a.K_stride[0] * 2; p.k1 = a.K_stride[1] * 2;
  p.v0 = a.V_stride[0] * 2; p.v1 = a.V_stride[1] * 2;
  p.pos = a.pos; p.inv_freq = a.inv_freq; p.q_weight = a.q_weight; p.k_weight = a.k_weight;
  p.Q_out = static_cast<uint8_t*>(a.Q_out);
  p.K_out = static_cast<uint8_t*>(a.K_out);
  p.V_out = static_cast<uint8_t*>(a.V_out);
  p.qo0 = a.Q_out_stride[0] * 2; p.qo1 = a.Q_out_stride[1] * 2;
  p.ko0 = a.K_out_stride[0] * 2; p.ko1 = a.K_out_stride[1] * 2; p.ko2 = a.K_out_stride[2] * 2;
  p.vo0 = a.V_out_stride[0] * 2; p.vo1 = a.V_out_stride[1] * 2; p.vo2 = a.V_out_stride[2] * 2;
  p.slots = a.slots; p.dev_err = a.dev_err;
  const int heads = a.D == 128 ? 4 : 8;       // per warp and step
  const int steps = (a.Hq + heads - 1) / heads + (a.V != nullptr ? 2 : 1) * ((a.Hkv + heads - 1) / heads);
  // few tokens: their heads spread over the warps that run at once, in equal parts, but not over more (2,000
  // tokens of 64 heads in two parts, some warps having a second one, took 7 % longer)
  const int64_t warps = static_cast<int64_t>(dev.num_sms) * kCtasPerSm * kWarps;
  const int most = static_cast<int>(std::min<int64_t>(std::max<int64_t>(warps / a.N, 1), steps));
  const int part_steps = (steps + most - 1) / most;
  p.parts = (steps + part_steps - 1) / part_steps;
  const int64_t items = a.N * p.parts;
  const unsigned grid =
      static_cast<unsigned>(std::min<int64_t>((items + kWarps - 1) / kWarps, static_cast<int64_t>(dev.num_sms) * kCtasPerSm));
  cudaError_t e;
  if (a.D == 128) {
    if (a.interleaved) e = launch_early(norm_rope_kernel<128, true>, grid, kThreads, 0, stream, 1, p);
    else e = launch_early(norm_rope_kernel<128, false>, grid, kThreads, 0, stream, 1, p);
  } else {
    if (a.interleaved) e = launch_early(norm_rope_kernel<64, true>, grid, kThreads, 0, stream, 1, p);
    else e = launch_early(norm_rope_kernel<64, false>, grid, kThreads, 0, stream, 1, p);
  }
  if (e != cudaSuccess) return cuda_fail(e, "norm_rope_kernel launch");
  return MSA_OK;
}

}  // namespace msa
