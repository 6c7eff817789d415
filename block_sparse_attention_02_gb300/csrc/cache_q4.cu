// cache_q4.cu -- the paged cache in 4 bits: tokens stored, pages expanded.
//
// A group of 16 channels holds codes of a 4-bit float (E2M1: 0, 0.5, 1, 1.5, 2,
// 3, 4, 6 and a sign) times an 8-bit scale (E4M3) times the pool's power of two:
//     sf = e4m3(amax / (6 gs)),  code = e2m1(x / (sf gs)),  value = code * sf * gs.
// 72 bytes per token and head instead of 256.
//
// Rounding.  x is bf16 (8 bits), sf has at most 4 bits and gs is a power of two.  A
// quotient x / (sf gs) that lies halfway between two codes is a multiple of 1/4 up
// to 5; one that does not is at least 2^-10 away from every halfway point.  With r =
// 1 / (sf gs) rounded to fp32, x r + 1536 in one rounding is a multiple of 2^-13: the first kind comes
// out exact, the second stays on its side, so the code is that of the real
// quotient, at two instructions a value where a division takes ten.  (In the
// same way amax / 6 against the scale's halfway points: a product with 1 / 6 that has
// at most 7 bits rounds to itself.)  Values past the range end at the largest code.
//
// Bound: latency of the loads, then HBM.  A block takes one head, so that the tokens of a
// prompt, whose slots follow one another, write whole runs of a page.  Store: a thread takes a
// group (32 bytes in, 8 code bytes and a scale byte out) of two tokens, whose loads are issued
// before the slots are known; six blocks on an SM keep more in flight than longer
// threads do (four tokens: 9.8 us for 8.7 at 8,192 tokens).  Expand: a thread takes half groups, 16
// bytes out, so that a warp's store is one run of 512 bytes, eight of them loaded ahead.
// 8,192 tokens of 8 heads stored and expanded again take 18.0 us in two launches (87 MB; floor
// 12.8); of 8 sequences' last tokens and pages 5.1 us, two launches' latency.
#include <cuda_fp16.h>

#include "launch_early.cuh"
#include "msa_internal.h"
#include "msa_ptx.cuh"
#include "q4.cuh"

namespace msa {
namespace {

constexpr int kThreads = 256;
constexpr int kStoreUnroll = 2;                             // tokens per thread
constexpr int kStoreCtas = 6;                               // per SM
constexpr int kStoreTokens = kThreads / 16 * kStoreUnroll;  // and per block
constexpr int kExpandUnroll = 8;                            // half groups per thread and run
constexpr unsigned kMaxGridY = 65535;

struct StoreParams {
  int64_t N, num_pages;
  int Hkv;
  const uint8_t *K, *V;
  int64_t k0, k1, v0, v1;       // byte strides (n, h)
  const int64_t* slots;
  uint8_t *K_codes, *K_scales, *V_codes, *V_scales;
  int64_t c0, c1, s0, s1;       // byte strides (page, g)
  float k_inv, v_inv;           // 1 / scale, exact
  int32_t* dev_err;
};

__device__ __forceinline__ uint32_t abs_max2(uint32_t a, uint32_t b) { return __vmaxu2(a & 0x7fff7fffu, b & 0x7fff7fffu); }

// Codes and scale byte of the 16 bf16 values in u[0..7] (two per word); inv = 1 / gs.
__device__ __forceinline__ void quantise16(const uint32_t (&u)[8], float inv, uint2* codes, uint32_t* scale) {
  uint32_t m = abs_max2(u[0], u[1]);
#pragma unroll
  for (int i = 2; i < 8; ++i) m = abs_max2(m, u[i]);
  const uint32_t top = max(m & 0xffffu, m >> 16);      // bf16 bits order as magnitudes, NaN above infinity
  const float amax = __uint_as_float(top << 16) * inv;
  const uint32_t sf = top > 0x7f80u ? 0x7fu : e4m3_from_float(fminf(amax, 2688.f) * (1.0f / 6.0f));
  const float s = e4m3_to_float(sf);
  const bool some = s > 0.f;                            // not a group of zeros, nor of NaN scale: their codes are 0
  const float r = some ? __frcp_rn(s) * inv : 0.f;
  uint32_t out[2];
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t v = u[w * 4 + (i >> 1)];
      q[i] = __fadd_rn(__fmaf_rn(__uint_as_float(i & 1 ? v & 0xffff0000u : v << 16), r, 1536.f), -1536.f);
    }
    out[w] = some ? e2m1x8_from_floats(q) : 0u;
  }
  *codes = make_uint2(out[0], out[1]);
  *scale = sf;
}

__global__ void __launch_bounds__(kThreads, kStoreCtas) append_q4_kernel(const StoreParams p) {
  wait_for_stream();
  const int group = threadIdx.x & 7;
  const bool is_v = threadIdx.x >> 3 & 1;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kStoreTokens + (threadIdx.x >> 4);
  const int64_t n_stride = is_v ? p.v0 : p.k0;
  const float inv = is_v ? p.v_inv : p.k_inv;
  int64_t slot[kStoreUnroll];
#pragma unroll
  for (int i = 0; i < kStoreUnroll; ++i) {
    const int64_t n = first + i * (kThreads / 16);
    slot[i] = n < p.N ? p.slots[n] : -1;
  }
  bool bad = false;
  for (int h = blockIdx.y; h < p.Hkv; h += gridDim.y) {
    const uint8_t* src = (is_v ? p.V + h * p.v1 : p.K + h * p.k1) + first * n_stride + group * 32;
    uint8_t* codes = (is_v ? p.V_codes : p.K_codes) + h * p.c1 + group * 8;
    uint8_t* scales = (is_v ? p.V_scales : p.K_scales) + h * p.s1 + group;
    uint4 a[kStoreUnroll], b[kStoreUnroll];
#pragma unroll
    for (int i = 0; i < kStoreUnroll; ++i) {   // rows without a slot too: nothing waits for the slots
      a[i] = b[i] = make_uint4(0, 0, 0, 0);
      if (first + i * (kThreads / 16) >= p.N) continue;
      const uint4* x = reinterpret_cast<const uint4*>(src + i * (kThreads / 16) * n_stride);
      a[i] = x[0];
      b[i] = x[1];
    }
#pragma unroll
    for (int i = 0; i < kStoreUnroll; ++i) {
      if (slot[i] < 0) continue;
      const int64_t page = slot[i] / kBk;
      const int t = static_cast<int>(slot[i] & (kBk - 1));
      if (page >= p.num_pages) {
        bad = true;
        continue;
      }
      const uint32_t u[8] = {a[i].x, a[i].y, a[i].z, a[i].w, b[i].x, b[i].y, b[i].z, b[i].w};
      uint2 c;
      uint32_t sf;
      quantise16(u, inv, &c, &sf);
      *reinterpret_cast<uint2*>(codes + page * p.c0 + t * 64) = c;
      scales[page * p.s0 + t * 8] = static_cast<uint8_t>(sf);
    }
  }
  if (bad && group == 0 && !is_v) report(p.dev_err, MSA_DEVERR_BAD_PAGE);
}

struct ExpandParams {
  int64_t n, num_pages;
  int Hkv;
  const int32_t* pages;
  const uint8_t *K_codes, *K_scales, *V_codes, *V_scales;
  int64_t c0, c1, s0, s1;
  uint8_t *K_out, *V_out;
  float k_scale, v_scale;
  int32_t* dev_err;
};

__global__ void __launch_bounds__(kThreads) expand_q4_kernel(const ExpandParams p) {
  wait_for_stream();
  const int64_t page = p.pages[blockIdx.x];
  if (page < 0 || page >= p.num_pages) {
    if (blockIdx.y == 0 && threadIdx.x == 0) report(p.dev_err, MSA_DEVERR_BAD_PAGE);
    return;
  }
  constexpr int kHalves = kBk * kD / 8;                 // half groups of a block of K, as many of V
  static_assert(kHalves % (kThreads * kExpandUnroll) == 0, "whole runs");
  for (int h = blockIdx.y; h < p.Hkv; h += gridDim.y) {
#pragma unroll 1
    for (int part = 0; part < 2 * kHalves / (kThreads * kExpandUnroll); ++part) {
      const bool is_v = part >= kHalves / (kThreads * kExpandUnroll);
      const int first = part * kThreads * kExpandUnroll - (is_v ? kHalves : 0) + threadIdx.x;
      const uint8_t* codes = (is_v ? p.V_codes : p.K_codes) + page * p.c0 + h * p.c1;
      const uint8_t* scales = (is_v ? p.V_scales : p.K_scales) + page * p.s0 + h * p.s1;
      uint4* out = reinterpret_cast<uint4*>(is_v ? p.V_out : p.K_out) +
                   (static_cast<int64_t>(blockIdx.x) * p.Hkv + h) * kHalves;
      const float gs = is_v ? p.v_scale : p.k_scale;
      uint32_t c[kExpandUnroll], sf[kExpandUnroll];
#pragma unroll
      for (int i = 0; i < kExpandUnroll; ++i) {
        const int x = first + i * kThreads;
        c[i] = reinterpret_cast<const uint32_t*>(codes)[x];
        sf[i] = scales[x >> 1];
      }
#pragma unroll
      for (int i = 0; i < kExpandUnroll; ++i) {
        const __half2 s = e4m3_to_half2(sf[i]);
        __half2 v[4];
        e2m1x8_to_half2(c[i], v);
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 f = __half22float2(__hmul2(v[e], s));   // exact: 2 bits times 4 bits, at least 2^-10
          const __nv_bfloat162 b = __floats2bfloat162_rn(f.x * gs, f.y * gs);
          w[e] = *reinterpret_cast<const uint32_t*>(&b);
        }
        out[first + i * kThreads] = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  }
}

}  // namespace

msa_status launch_append_q4(const msa_append_q4_args& a, cudaStream_t stream) {
  StoreParams p;
  p.N = a.N; p.num_pages = a.cache.num_pages; p.Hkv = a.Hkv;
  p.K = static_cast<const uint8_t*>(a.K);
  p.V = static_cast<const uint8_t*>(a.V);
  p.k0 = a.K_stride[0] * 2; p.k1 = a.K_stride[1] * 2;
  p.v0 = a.V_stride[0] * 2; p.v1 = a.V_stride[1] * 2;
  p.slots = a.slots;
  p.K_codes = static_cast<uint8_t*>(a.cache.K_codes);
  p.K_scales = static_cast<uint8_t*>(a.cache.K_scales);
  p.V_codes = static_cast<uint8_t*>(a.cache.V_codes);
  p.V_scales = static_cast<uint8_t*>(a.cache.V_scales);
  p.c0 = a.cache.code_stride[0]; p.c1 = a.cache.code_stride[1];
  p.s0 = a.cache.scale_stride[0]; p.s1 = a.cache.scale_stride[1];
  p.k_inv = 1.0f / a.cache.k_scale; p.v_inv = 1.0f / a.cache.v_scale;
  p.dev_err = a.dev_err;
  const dim3 grid(static_cast<unsigned>((a.N + kStoreTokens - 1) / kStoreTokens),
                  std::min<unsigned>(static_cast<unsigned>(a.Hkv), kMaxGridY));
  const cudaError_t e = launch_early(append_q4_kernel, grid, kThreads, 0, stream, 1, p);
  if (e != cudaSuccess) return cuda_fail(e, "append_q4_kernel launch");
  return MSA_OK;
}

msa_status launch_expand_q4(const msa_expand_q4_args& a, cudaStream_t stream) {
  ExpandParams p;
  p.n = a.n; p.num_pages = a.cache.num_pages; p.Hkv = a.Hkv;
  p.pages = a.pages;
  p.K_codes = static_cast<const uint8_t*>(a.cache.K_codes);
  p.K_scales = static_cast<const uint8_t*>(a.cache.K_scales);
  p.V_codes = static_cast<const uint8_t*>(a.cache.V_codes);
  p.V_scales = static_cast<const uint8_t*>(a.cache.V_scales);
  p.c0 = a.cache.code_stride[0]; p.c1 = a.cache.code_stride[1];
  p.s0 = a.cache.scale_stride[0]; p.s1 = a.cache.scale_stride[1];
  p.K_out = static_cast<uint8_t*>(a.K_out);
  p.V_out = static_cast<uint8_t*>(a.V_out);
  p.k_scale = a.cache.k_scale; p.v_scale = a.cache.v_scale;
  p.dev_err = a.dev_err;
  const dim3 grid(static_cast<unsigned>(a.n), std::min<unsigned>(static_cast<unsigned>(a.Hkv), kMaxGridY));
  const cudaError_t e = launch_early(expand_q4_kernel, grid, kThreads, 0, stream, 1, p);
  if (e != cudaSuccess) return cuda_fail(e, "expand_q4_kernel launch");
  return MSA_OK;
}

}  // namespace msa
