// cache_q4.cu -- the paged cache in 4 bits: tokens stored, pages expanded.
//
// A group of 16 channels holds codes of a 4-bit float (E2M1: 0, 0.5, 1, 1.5, 2,
// 3, 4, 6 and a sign) times an 8-bit scale (E4M3) times the pool's power of two:
//     sf = e4m3(amax / (6 gs)),  code = e2m1(x / (sf gs)),  value = code * sf * gs.
// 72 bytes per token and head instead of 256.
//
// Rounding.  x is bf16 (8 bits), sf has 4 bits and gs is a power of two, so an
// exact quotient x / (sf gs) that lies halfway between two codes has at most 8 bits,
// and one that does not differs from a halfway point by more than 2^-13 of
// itself.  q = x r + (x - (x r) sf) r with r = 1 / sf in fp32 returns the first kind exactly
// and the second within 2^-22, so the code is that of the real quotient.  The
// same holds for amax / 6 against the scale's halfway points.
//
// One thread per group: 32 bytes in, 8 codes bytes and a scale byte out; eight
// neighbouring threads share a row, so every access fills its sectors.
// Bound: HBM.
#include <cuda_fp16.h>

#include "msa_internal.h"
#include "msa_ptx.cuh"
#include "q4.cuh"

namespace msa {
namespace {

constexpr int kThreads = 256;

struct StoreParams {
  int64_t N, num_pages;
  int Hkv, Bk;
  const uint8_t *K, *V;
  int64_t k0, k1, v0, v1;       // byte strides (n, h)
  const int64_t* slots;
  uint8_t *K_codes, *K_scales, *V_codes, *V_scales;
  int64_t c0, c1, s0, s1;       // byte strides (page, g)
  float k_inv, v_inv;           // 1 / scale, exact
  int32_t* dev_err;
};

__device__ __forceinline__ uint32_t abs_max2(uint32_t a, uint32_t b) { return __vmaxu2(a & 0x7fff7fffu, b & 0x7fff7fffu); }

// Codes and scale byte of the 16 bf16 values in u[0..7] (two per word).
__device__ __forceinline__ void quantise16(const uint32_t (&u)[8], float inv, uint2* codes, uint32_t* scale) {
  uint32_t m = abs_max2(u[0], u[1]);
#pragma unroll
  for (int i = 2; i < 8; ++i) m = abs_max2(m, u[i]);
  const uint32_t top = max(m & 0xffffu, m >> 16);      // bf16 bits order as magnitudes, NaN above infinity
  const float amax = __uint_as_float(top << 16);
  const uint32_t sf = top > 0x7f80u ? 0x7fu : e4m3_from_float(fminf(amax * inv, 2688.f) * (1.0f / 6.0f));
  const float s = e4m3_to_float(sf);
  const float r = s > 0.f ? __fdiv_rn(1.0f, s) : 0.f;   // a group of zeros, or of NaN scale: codes 0
  uint32_t out[2];
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    uint32_t c = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t v = u[w * 4 + i];
      float q[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float raw = __uint_as_float(e ? v & 0xffff0000u : v << 16) * inv;
        const float x = fminf(fmaxf(raw, -2688.f), 2688.f);
        const float q0 = x * r;
        q[e] = fmaf(fmaf(-q0, s, x), r, q0);
      }
      c |= e2m1x2_from_floats(q[0], q[1]) << (8 * i);
    }
    out[w] = s > 0.f ? c : 0u;
  }
  *codes = make_uint2(out[0], out[1]);
  *scale = sf;
}

__global__ void __launch_bounds__(kThreads) append_q4_kernel(const StoreParams p) {
  const int64_t total = p.N * p.Hkv * 16;               // (token, head, K or V, group)
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * kThreads) {
    const int group = static_cast<int>(i & 7);
    const bool is_v = (i >> 3) & 1;
    const int64_t nh = i >> 4;
    const int64_t n = nh / p.Hkv;
    const int h = static_cast<int>(nh - n * p.Hkv);
    const int64_t slot = p.slots[n];
    if (slot < 0) continue;
    const int64_t page = slot / p.Bk;
    const int t = static_cast<int>(slot - page * p.Bk);
    if (page >= p.num_pages) {
      if (group == 0 && h == 0 && !is_v) report(p.dev_err, MSA_DEVERR_BAD_PAGE);
      continue;
    }
    const uint4* src = reinterpret_cast<const uint4*>((is_v ? p.V + n * p.v0 + h * p.v1 : p.K + n * p.k0 + h * p.k1) +
                                                      group * 32);
    const uint4 a = src[0], b = src[1];
    const uint32_t u[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    uint2 codes;
    uint32_t scale;
    quantise16(u, is_v ? p.v_inv : p.k_inv, &codes, &scale);
    *reinterpret_cast<uint2*>((is_v ? p.V_codes : p.K_codes) + page * p.c0 + h * p.c1 + t * 64 + group * 8) = codes;
    (is_v ? p.V_scales : p.K_scales)[page * p.s0 + h * p.s1 + t * 8 + group] = static_cast<uint8_t>(scale);
  }
}

struct ExpandParams {
  int64_t n, num_pages;
  int Hkv, Bk;
  const int32_t* pages;
  const uint8_t *K_codes, *K_scales, *V_codes, *V_scales;
  int64_t c0, c1, s0, s1;
  uint8_t *K_out, *V_out;
  float k_scale, v_scale;
  int32_t* dev_err;
};

__global__ void __launch_bounds__(kThreads) expand_q4_kernel(const ExpandParams p) {
  const int64_t rows = p.n * p.Hkv * p.Bk;              // output rows of K, as many of V
  const int64_t total = rows * 16;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * kThreads) {
    const bool is_v = i >= rows * 8;
    const int64_t at = is_v ? i - rows * 8 : i;
    const int group = static_cast<int>(at & 7);
    const int64_t row = at >> 3;
    const int t = static_cast<int>(row % p.Bk);
    const int64_t xh = row / p.Bk;
    const int h = static_cast<int>(xh % p.Hkv);
    const int64_t x = xh / p.Hkv;
    const int64_t page = p.pages[x];
    if (page < 0 || page >= p.num_pages) {
      if (group == 0 && t == 0 && h == 0 && !is_v) report(p.dev_err, MSA_DEVERR_BAD_PAGE);
      continue;
    }
    const uint2 c = *reinterpret_cast<const uint2*>((is_v ? p.V_codes : p.K_codes) + page * p.c0 + h * p.c1 + t * 64 +
                                                    group * 8);
    const uint32_t sf = (is_v ? p.V_scales : p.K_scales)[page * p.s0 + h * p.s1 + t * 8 + group];
    const __half2 s = e4m3_to_half2(sf);
    const float gs = is_v ? p.v_scale : p.k_scale;
    uint32_t out[8];
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      __half2 v[4];
      e2m1x8_to_half2(w ? c.y : c.x, v);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 f = __half22float2(__hmul2(v[e], s));   // exact: 2 bits times 4 bits, at least 2^-10
        const __nv_bfloat162 b = __floats2bfloat162_rn(f.x * gs, f.y * gs);
        out[w * 4 + e] = *reinterpret_cast<const uint32_t*>(&b);
      }
    }
    uint4* dst = reinterpret_cast<uint4*>((is_v ? p.V_out : p.K_out) + row * 256 + group * 32);
    dst[0] = make_uint4(out[0], out[1], out[2], out[3]);
    dst[1] = make_uint4(out[4], out[5], out[6], out[7]);
  }
}

unsigned grid_for(int64_t threads, int sms) {
  return static_cast<unsigned>(std::min<int64_t>((threads + kThreads - 1) / kThreads, static_cast<int64_t>(sms) * 32));
}

}  // namespace

msa_status launch_append_q4(const msa_append_q4_args& a, cudaStream_t stream) {
  DeviceInfo dev;
  if (msa_status st = current_device(&dev); st != MSA_OK) return st;
  StoreParams p;
  p.N = a.N; p.num_pages = a.cache.num_pages; p.Hkv = a.Hkv; p.Bk = a.Bk;
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
  append_q4_kernel<<<grid_for(a.N * a.Hkv * 16, dev.num_sms), kThreads, 0, stream>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "append_q4_kernel launch");
  return MSA_OK;
}

msa_status launch_expand_q4(const msa_expand_q4_args& a, cudaStream_t stream) {
  DeviceInfo dev;
  if (msa_status st = current_device(&dev); st != MSA_OK) return st;
  ExpandParams p;
  p.n = a.n; p.num_pages = a.cache.num_pages; p.Hkv = a.Hkv; p.Bk = a.Bk;
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
  expand_q4_kernel<<<grid_for(a.n * a.Hkv * a.Bk * 16, dev.num_sms), kThreads, 0, stream>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "expand_q4_kernel launch");
  return MSA_OK;
}

}  // namespace msa
