// cache_q8.cu -- the paged cache in 8 bits: tokens stored, pages expanded.
//
// A block (the 128 tokens of a page and head) holds E4M3 codes times one power of two:
//     scale = the smallest 2^e, e in [-40, 40], with amax <= 448 * 2^e,  code = e4m3(x / scale).
// A power of two costs an E4M3 code nothing (its relative step is the same at every exponent), and makes x / scale and
// the rescaling below exact before their one rounding.
//
// Tokens come to a block a few at a time.  A call's tokens of one page are a run: consecutive token rows in consecutive
// slots (msa_plan_step's rows are).  A run that starts at row 0 starts the block anew, whatever an earlier owner of the
// page left; one that starts later keeps the rows before it, and where it needs a larger scale these are rounded again
// (the exponent moves, so only codes that become subnormal change).  So a block's scale is that of its own tokens alone.
//
// Work.  A CTA takes a window of token rows for one head of K or V: it reads their slots, and those behind them as far as a run
// may reach, and stores the runs that start in the window.  Runs of up to 8 tokens go to a warp each, longer ones to the
// CTA, which holds the run (at most 128 rows of 256 bytes) in registers between the maximum and the rounding: every token
// is read once.  A window is as long as half a page, so that a prompt's CTAs have a run each or none; for few tokens it is one
// row for each warp.
#include "launch_early.cuh"
#include "msa_internal.h"
#include "msa_ptx.cuh"
#include "q8.cuh"

namespace msa {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kShort = 8;                      // rows of a run that a warp stores: 16 lanes a row, four rows a lane
constexpr int kFewTokens = 1024;               // up to here a CTA's window is kWarps token rows, a run for every warp
constexpr int kManyWindow = 64;
constexpr int kStoreCtas = 4;                  // per SM
static_assert(kManyWindow + kBk + 1 <= kThreads, "a slot for every thread");
constexpr unsigned kMaxGridY = 65535;

struct StoreParams {
  int64_t N, num_pages;
  int Hkv, window;
  const uint8_t *K, *V;
  int64_t k0, k1, v0, v1;       // byte strides (n, h)
  const int64_t* slots;
  uint8_t *K_codes, *K_scales, *V_codes, *V_scales;
  int64_t c0, c1, s0, s1;       // byte strides (page, g)
  int32_t* dev_err;
};

// The larger finite magnitudes of bf16 pairs a and b (an infinity or NaN sets no scale).
__device__ __forceinline__ uint32_t finite_max2(uint32_t a, uint32_t b) {
  b &= 0x7fff7fffu;
  return __vmaxu2(a, b & __vcmpltu2(b, 0x7f807f80u));
}
__device__ __forceinline__ uint32_t finite_max(uint32_t m, uint4 v) {
  return finite_max2(finite_max2(finite_max2(finite_max2(m, v.x), v.y), v.z), v.w);
}
__device__ __forceinline__ uint32_t warp_top(uint32_t m) { return redux_max_u32(max(m & 0xffffu, m >> 16)); }

// Eight bf16 values to codes; inv = 1 / scale.
__device__ __forceinline__ uint2 encode8(uint4 v, float inv) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
  float f[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(u[i] << 16) * inv;
    f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u) * inv;
  }
  return make_uint2(e4m3x4_from_floats(f[0], f[1], f[2], f[3]), e4m3x4_from_floats(f[4], f[5], f[6], f[7]));
}

// Rows [0, rows) of a block rounded again under a scale 1 / f as large, by `threads` threads.
__device__ __forceinline__ void rescale_rows(uint8_t* codes, int rows, float f, int tid, int threads) {
  uint4* at = reinterpret_cast<uint4*>(codes);
  const int n = rows * 8;
  for (int i = tid; i < n; i += 4 * threads) {
    uint4 v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (i + k * threads < n) v[k] = at[i + k * threads];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (i + k * threads < n)
        at[i + k * threads] = make_uint4(e4m3x4_rescaled(v[k].x, f), e4m3x4_rescaled(v[k].y, f), e4m3x4_rescaled(v[k].z, f),
                                         e4m3x4_rescaled(v[k].w, f));
  }
}

__global__ void __launch_bounds__(kThreads, kStoreCtas) append_q8_kernel(const StoreParams p) {
  wait_for_stream();
  __shared__ uint32_t s_top[kWarps];
  __shared__ int64_t s_slot[kThreads];           // of token rows begin - 1 ..
  __shared__ int s_first[kManyWindow], s_rows[kManyWindow], s_long;   // long runs of the window
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const bool is_v = blockIdx.z != 0;
  const int64_t begin = static_cast<int64_t>(blockIdx.x) * p.window;
  const int64_t n_stride = is_v ? p.v0 : p.k0;
  const int part = lane & 15;                   // 16 bytes of a row
  const uint8_t* src = (is_v ? p.V + blockIdx.y * p.v1 : p.K + blockIdx.y * p.k1) + begin * n_stride + part * 16;
  const int here = static_cast<int>(min(static_cast<int64_t>(p.window), p.N - begin));
  // the first row of this warp does not wait for the slots
  uint4 early = make_uint4(0, 0, 0, 0);
  if (lane < 16 && warp < here) early = *reinterpret_cast<const uint4*>(src + warp * n_stride);
  {
    const int64_t r = begin + tid - 1;
    s_slot[tid] = r >= 0 && r < p.N && tid < p.window + kBk + 1 ? p.slots[r] : -2;
    if (tid == 0) s_long = 0;
  }
  __syncthreads();
  // rows of the run that starts at row r of the window; 0: none does, or it is not stored
  auto run_at = [&](int r) {
    const int64_t at = s_slot[r + 1];
    if (at < 0 || at >= p.num_pages * kBk) {
      if (at >= 0 && blockIdx.y == 0 && !is_v && lane == 0) report(p.dev_err, MSA_DEVERR_BAD_PAGE);
      return 0;
    }
    const int t0 = static_cast<int>(at & (kBk - 1));
    if (t0 != 0 && s_slot[r] == at - 1) return 0;
    int n = 0;
    for (int k = 0; k < kBk; k += 32) {
      const uint32_t stops = ~__ballot_sync(0xffffffffu, t0 + k + lane < kBk && s_slot[r + 1 + k + lane] == at + k + lane);
      if (stops != 0) return n + __ffs(stops) - 1;
      n += 32;
    }
    return n;
  };
  uint8_t* all_codes = is_v ? p.V_codes : p.K_codes;
  uint8_t* all_scales = is_v ? p.V_scales : p.K_scales;
  for (int h = blockIdx.y; h < p.Hkv; h += gridDim.y) {
    const uint8_t* rows = src + (h - blockIdx.y) * (is_v ? p.v1 : p.k1);
    for (int r = warp; r < here; r += kWarps) {
      const int n = run_at(r);
      if (n == 0) continue;
      if (n > kShort) {
        if (lane == 0 && h == blockIdx.y) {
          const int x = atomicAdd(&s_long, 1);
          s_first[x] = r;
          s_rows[x] = n;
        }
        continue;
      }
      const int64_t at = s_slot[r + 1], page = at / kBk;
      const int t0 = static_cast<int>(at & (kBk - 1));
      uint8_t* scale = all_scales + page * p.s0 + h * p.s1;
      uint8_t* block = all_codes + page * p.c0 + h * p.c1;
      const uint32_t stored = t0 > 0 ? *scale : 0;
      const uint8_t* row = rows + r * n_stride;
      uint4 v[kShort / 2];
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < kShort / 2; ++i) {
        const int k = 2 * i + (lane >> 4);
        v[i] = i == 0 && r == warp && h == blockIdx.y && lane < 16 ? early
               : k < n ? *reinterpret_cast<const uint4*>(row + k * n_stride) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < kShort / 2; ++i) m = finite_max(m, v[i]);
      uint32_t byte = q8_byte_for(warp_top(m));
      if (t0 > 0) {
        const uint32_t old = q8_byte(stored);
        if (byte > old) rescale_rows(block, t0, q8_inverse(byte - old + 127), lane, 32);
        byte = max(byte, old);
      }
      const float inv = q8_inverse(byte);
#pragma unroll
      for (int i = 0; i < kShort / 2; ++i) {
        const int k = 2 * i + (lane >> 4);
        if (k < n) *reinterpret_cast<uint2*>(block + (t0 + k) * kD + part * 8) = encode8(v[i], inv);
      }
      if (lane == 0) *scale = static_cast<uint8_t>(byte);
    }
    if (h == blockIdx.y) __syncthreads();
    // the long runs, one after another (in whatever order: they are of different pages)
    for (int x = 0; x < s_long; ++x) {
      const int r = s_first[x], n = s_rows[x], first = tid >> 4;
      const int64_t at = s_slot[r + 1], page = at / kBk;
      const int t0 = static_cast<int>(at & (kBk - 1));
      uint8_t* scale = all_scales + page * p.s0 + h * p.s1;
      uint8_t* block = all_codes + page * p.c0 + h * p.c1;
      const uint32_t stored = t0 > 0 ? *scale : 0;
      const uint8_t* row = rows + (r + first) * n_stride;
      constexpr int kEach = kBk * 16 / kThreads;      // rows of a thread: first, first + 16, ..
      uint4 v[kEach];
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < kEach; ++i)
        v[i] = first + i * (kThreads / 16) < n ? *reinterpret_cast<const uint4*>(row + i * (kThreads / 16) * n_stride) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int i = 0; i < kEach; ++i) m = finite_max(m, v[i]);
      const uint32_t mine = warp_top(m);
      if (lane == 0) s_top[warp] = mine;
      __syncthreads();
      uint32_t top = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = max(top, s_top[w]);
      __syncthreads();                                // the maxima are read, and the stored scale by every thread
      uint32_t byte = q8_byte_for(top);
      if (t0 > 0) {
        const uint32_t old = q8_byte(stored);
        if (byte > old) rescale_rows(block, t0, q8_inverse(byte - old + 127), tid, kThreads);
        byte = max(byte, old);
      }
      const float inv = q8_inverse(byte);
#pragma unroll
      for (int i = 0; i < kEach; ++i)
        if (first + i * (kThreads / 16) < n)
          *reinterpret_cast<uint2*>(block + (t0 + first + i * (kThreads / 16)) * kD + part * 8) = encode8(v[i], inv);
      if (tid == 0) *scale = static_cast<uint8_t>(byte);
    }
  }
}

struct ExpandParams {
  int64_t num_pages;
  int Hkv;
  const int32_t* pages;
  const uint8_t *K_codes, *K_scales, *V_codes, *V_scales;
  int64_t c0, c1, s0, s1;
  uint8_t *K_out, *V_out;
  int32_t* dev_err;
};

// A thread takes 8 codes to 16 bytes, so that a warp's store is one run of 512 bytes, eight of them loaded ahead.
__global__ void __launch_bounds__(kThreads) expand_q8_kernel(const ExpandParams p) {
  wait_for_stream();
  const int64_t page = p.pages[blockIdx.x];
  if (page < 0 || page >= p.num_pages) {
    if (blockIdx.y == 0 && blockIdx.z == 0 && threadIdx.x == 0) report(p.dev_err, MSA_DEVERR_BAD_PAGE);
    return;
  }
  constexpr int kEach = kBk * kD / 8 / kThreads;        // of a block, for a thread
  const bool is_v = blockIdx.z != 0;
  for (int h = blockIdx.y; h < p.Hkv; h += gridDim.y) {
    const uint2* codes = reinterpret_cast<const uint2*>((is_v ? p.V_codes : p.K_codes) + page * p.c0 + h * p.c1) + threadIdx.x;
    const float scale = q8_scale(q8_byte((is_v ? p.V_scales : p.K_scales)[page * p.s0 + h * p.s1]));
    uint4* out = reinterpret_cast<uint4*>(is_v ? p.V_out : p.K_out) +
                 (static_cast<int64_t>(blockIdx.x) * p.Hkv + h) * (kBk * kD / 8) + threadIdx.x;
    uint2 c[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) c[i] = codes[i * kThreads];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      uint32_t f[4], w[4];
      e4m3x4_to_f16(c[i].x, &f[0], &f[1]);
      e4m3x4_to_f16(c[i].y, &f[2], &f[3]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 x = __half22float2(*reinterpret_cast<__half2*>(&f[e]));
        const __nv_bfloat162 b = __floats2bfloat162_rn(x.x * scale, x.y * scale);   // 4 bits: exact
        w[e] = *reinterpret_cast<const uint32_t*>(&b);
      }
      out[i * kThreads] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

}  // namespace

msa_status launch_append_q8(const msa_append_q8_args& a, cudaStream_t stream) {
  StoreParams p;
  p.N = a.N; p.num_pages = a.cache.num_pages; p.Hkv = a.Hkv;
  p.window = a.N <= kFewTokens ? kWarps : kManyWindow;
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
  p.dev_err = a.dev_err;
  const dim3 grid(static_cast<unsigned>((a.N + p.window - 1) / p.window), std::min<unsigned>(static_cast<unsigned>(a.Hkv), kMaxGridY), 2);
  const cudaError_t e = launch_early(append_q8_kernel, grid, kThreads, 0, stream, 1, p);
  if (e != cudaSuccess) return cuda_fail(e, "append_q8_kernel launch");
  return MSA_OK;
}

msa_status launch_expand_q8(const msa_expand_q8_args& a, cudaStream_t stream) {
  ExpandParams p;
  p.num_pages = a.cache.num_pages; p.Hkv = a.Hkv;
  p.pages = a.pages;
  p.K_codes = static_cast<const uint8_t*>(a.cache.K_codes);
  p.K_scales = static_cast<const uint8_t*>(a.cache.K_scales);
  p.V_codes = static_cast<const uint8_t*>(a.cache.V_codes);
  p.V_scales = static_cast<const uint8_t*>(a.cache.V_scales);
  p.c0 = a.cache.code_stride[0]; p.c1 = a.cache.code_stride[1];
  p.s0 = a.cache.scale_stride[0]; p.s1 = a.cache.scale_stride[1];
  p.K_out = static_cast<uint8_t*>(a.K_out);
  p.V_out = static_cast<uint8_t*>(a.V_out);
  p.dev_err = a.dev_err;
  const dim3 grid(static_cast<unsigned>(a.n), std::min<unsigned>(static_cast<unsigned>(a.Hkv), kMaxGridY), 2);
  const cudaError_t e = launch_early(expand_q8_kernel, grid, kThreads, 0, stream, 1, p);
  if (e != cudaSuccess) return cuda_fail(e, "expand_q8_kernel launch");
  return MSA_OK;
}

}  // namespace msa
