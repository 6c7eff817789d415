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
// (the exponent moves, so only codes that become subnormal change).  So a block's scale is the largest that the tokens stored in it
// since row 0 was last written needed: that of its own tokens, and of any that the program dropped again.
//
// Work.  A CTA takes a window of token rows for one or a few heads of K or V: it reads their slots, and those behind them as
// far as a run may reach, and stores the runs that start in the window, while the window's rows are on their way to L2.
// Longer runs go to the CTA, which holds the run (at most 128 rows of 256 bytes) in registers between the maximum and the
// rounding: every token is read once.  Runs of up to 8 tokens (decoded ones) go to half a warp each, for one head.  The window is a
// page long, so that a prompt's CTAs have about one run; for few tokens it is short, and heads share a CTA where there would
// be more CTAs than run at once.  Blocks that have to be rounded again wait until the end and are done by all warps (one warp alone
// would need 5 us for a full one).
//
// Bound: for few tokens a launch and three dependent loads (slots, scales, rows): 8 tokens of eight heads 3.6 us, 64 4.1, 1,024 decoded
// ones 10.0 (half of them rescaled blocks' reads); for a prompt issue and latency: 8,192 tokens 13.9 us (3.6 TB/s; outputs
// stay in L2), 32,768 41.5 (4.9 TB/s).  Windows of 8 or 64 rows, and a warp for several heads, were slower.
// The expansion runs at the copy rate.
#include "launch_early.cuh"
#include "msa_internal.h"
#include "msa_ptx.cuh"
#include "q8.cuh"

namespace msa {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kShort = 8;                      // rows of a run that half a warp stores
constexpr int kHalves = 2 * kWarps, kDeep = 2; // half warps, and runs that each has in flight
constexpr int kFewTokens = 1024;               // up to here a CTA's window is short
constexpr int kFewWindow = 16, kManyWindow = kBk;
constexpr int kFewHeads = 8;                   // heads of a CTA with a short window, at most
constexpr int kStoreCtas = 4;                  // per SM
constexpr unsigned kMaxGridY = 65535;

struct StoreParams {
  int64_t N, num_pages;
  int Hkv, window, heads;       // token rows and heads of a CTA
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
  constexpr int kDeep = 4;
  for (int i = tid; i < n; i += kDeep * threads) {
    uint4 v[kDeep];
#pragma unroll
    for (int k = 0; k < kDeep; ++k)
      if (i + k * threads < n) v[k] = at[i + k * threads];
#pragma unroll
    for (int k = 0; k < kDeep; ++k)
      if (i + k * threads < n)
        at[i + k * threads] = make_uint4(e4m3x4_rescaled(v[k].x, f), e4m3x4_rescaled(v[k].y, f), e4m3x4_rescaled(v[k].z, f),
                                         e4m3x4_rescaled(v[k].w, f));
  }
}
// A block whose scale grows: its page, its head, the rows before the new ones, and how far the exponent moves.
struct Growth {
  int page, head, rows, by;
};

__global__ void __launch_bounds__(kThreads, kStoreCtas) append_q8_kernel(const StoreParams p) {
  wait_for_stream();
  __shared__ uint32_t s_top[kWarps];
  __shared__ int64_t s_slot[kManyWindow + kBk + 1];   // of token rows begin - 1 ..
  __shared__ uint32_t s_break[(kManyWindow + kBk) / 32];   // bit i % 32 of word i / 32: row i does not go on where row i - 1 ended
  __shared__ int s_run[kManyWindow], s_runs;   // short runs: first row, and rows << 16
  __shared__ Growth s_growth[kManyWindow > kFewWindow * kFewHeads ? kManyWindow : kFewWindow * kFewHeads];
  __shared__ int s_grown;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const bool is_v = blockIdx.z != 0;
  const int64_t begin = static_cast<int64_t>(blockIdx.x) * p.window;
  const int64_t n_stride = is_v ? p.v0 : p.k0, h_stride = is_v ? p.v1 : p.k1;
  const int part = lane & 15;                   // 16 bytes of a row
  const uint8_t* src = (is_v ? p.V : p.K) + begin * n_stride + part * 16;
  const int h_lo = blockIdx.y * p.heads, h_hi = min(h_lo + p.heads, p.Hkv);
  const int here = static_cast<int>(min(static_cast<int64_t>(p.window), p.N - begin));
  for (int i = tid; i < p.window + kBk + 1; i += kThreads) {
    const int64_t r = begin + i - 1;
    s_slot[i] = r >= 0 && r < p.N ? p.slots[r] : -2;
  }
  for (int i = tid; i < here * (h_hi - h_lo) * 2; i += kThreads) {   // 128 bytes each
    const int row = (i >> 1) % here, h = h_lo + (i >> 1) / here;
    asm volatile("prefetch.global.L2 [%0];" ::"l"(src - part * 16 + row * n_stride + h * h_stride + (i & 1) * 128));
  }
  if (tid == 0) s_grown = s_runs = 0;
  __syncthreads();
  bool bad = false;
  for (int i = tid; i < kManyWindow + kBk; i += kThreads) {
    bool is = true;
    if (i < p.window + kBk) {
      const int64_t at = s_slot[i + 1];
      is = at < 0 || (at & (kBk - 1)) == 0 || s_slot[i] != at - 1;
      bad |= i < p.window && at >= p.num_pages * kBk;
    }
    const uint32_t word = __ballot_sync(0xffffffffu, is);
    if (lane == 0) s_break[i >> 5] = word;
  }
  if (bad && blockIdx.y == 0 && !is_v) report(p.dev_err, MSA_DEVERR_BAD_PAGE);
  __syncthreads();
  // the first row at or behind row r of the window where a run may start; of a run that starts at r, its end
  auto next_break = [&](int r) {
    for (int w = r >> 5; w < (kManyWindow + kBk) / 32; ++w) {
      const uint32_t word = s_break[w] & (w == r >> 5 ? ~0u << (r & 31) : ~0u);
      if (word != 0) return w * 32 + __ffs(word) - 1;
    }
    return kManyWindow + kBk;
  };
  auto stored_at = [&](int r) { return s_slot[r + 1] >= 0 && s_slot[r + 1] < p.num_pages * kBk; };
  uint8_t* all_codes = is_v ? p.V_codes : p.K_codes;
  uint8_t* all_scales = is_v ? p.V_scales : p.K_scales;
  if (tid < here && (s_break[tid >> 5] >> (tid & 31) & 1) != 0 && stored_at(tid)) {
    const int n = next_break(tid + 1) - tid;
    if (n <= kShort) s_run[atomicAdd(&s_runs, 1)] = tid | n << 16;   // (in whatever order: they are of different pages)
  }
  __syncthreads();
  const int heads = h_hi - h_lo, units = s_runs * heads;
  for (int u0 = 0; u0 < units; u0 += kHalves * kDeep) {
    int n[kDeep], t0[kDeep], head[kDeep];
    int64_t page[kDeep];
    const uint8_t* row[kDeep];
    uint4 v[kDeep];
    uint32_t old[kDeep];
#pragma unroll
    for (int d = 0; d < kDeep; ++d) {
      const int u = u0 + d * kHalves + warp * 2 + (lane >> 4);
      const int run = u < units ? s_run[u / heads] : 0, r = run & 0xffff;
      const int64_t at = s_slot[r + 1];
      n[d] = run >> 16;
      head[d] = h_lo + u % heads;
      page[d] = at / kBk;
      t0[d] = static_cast<int>(at & (kBk - 1));
      row[d] = src + r * n_stride + head[d] * h_stride;
      v[d] = make_uint4(0, 0, 0, 0);
      old[d] = 0;
      if (n[d] > 0) {
        v[d] = *reinterpret_cast<const uint4*>(row[d]);
        if (t0[d] > 0) old[d] = q8_byte(all_scales[page[d] * p.s0 + head[d] * p.s1]);
      }
    }
#pragma unroll
    for (int d = 0; d < kDeep; ++d) {
      uint32_t m = finite_max(0, v[d]);
      for (int k = 1; __any_sync(0xffffffffu, k < n[d]); ++k)
        if (k < n[d]) m = finite_max(m, *reinterpret_cast<const uint4*>(row[d] + k * n_stride));
      uint32_t top = max(m & 0xffffu, m >> 16);
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
      if (n[d] == 0) continue;
      const uint32_t byte = max(q8_byte_for(top), old[d]);
      if (part == 0) {
        if (old[d] != 0 && byte > old[d])
          s_growth[atomicAdd(&s_grown, 1)] = Growth{static_cast<int>(page[d]), head[d], t0[d], static_cast<int>(byte - old[d])};
        all_scales[page[d] * p.s0 + head[d] * p.s1] = static_cast<uint8_t>(byte);
      }
      const float inv = q8_inverse(byte);
      uint8_t* to = all_codes + page[d] * p.c0 + head[d] * p.c1 + t0[d] * kD + part * 8;
      *reinterpret_cast<uint2*>(to) = encode8(v[d], inv);
      for (int k = 1; k < n[d]; ++k)
        *reinterpret_cast<uint2*>(to + k * kD) = encode8(*reinterpret_cast<const uint4*>(row[d] + k * n_stride), inv);
    }
    __syncwarp();
  }
  for (int h = h_lo; h < h_hi; ++h) {
    const uint8_t* rows = src + h * h_stride;
    // the long runs, one after another
    for (int r = next_break(0), end; r < here; r = end) {
      end = next_break(r + 1);
      if (end - r <= kShort || !stored_at(r)) continue;
      const int n = end - r, first = tid >> 4;
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
  __syncthreads();
  // the blocks that grew: a few by all warps, or many by one each
  const int grown = s_grown, team = grown == 1 ? kWarps : grown == 2 ? kWarps / 2 : grown <= 4 ? kWarps / 4 : 1;
  for (int x = warp / team; x < grown; x += kWarps / team) {
    const Growth y = s_growth[x];
    rescale_rows(all_codes + y.page * p.c0 + y.head * p.c1, y.rows, q8_inverse(y.by + 127), warp % team * 32 + lane, team * 32);
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
  DeviceInfo dev;
  if (msa_status st = current_device(&dev); st != MSA_OK) return st;
  p.window = a.N <= kFewTokens ? kFewWindow : kManyWindow;
  p.heads = 1;
  if (a.N <= kFewTokens) {
    const int64_t windows = (a.N + kFewWindow - 1) / kFewWindow;
    while (p.heads < kFewHeads && 2 * windows * ((a.Hkv + p.heads - 1) / p.heads) > kStoreCtas * dev.num_sms) p.heads *= 2;
  }
  if (a.Hkv / p.heads >= static_cast<int>(kMaxGridY)) return fail(MSA_ERR_UNSUPPORTED, "8-bit store: too many heads");
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
  const dim3 grid(static_cast<unsigned>((a.N + p.window - 1) / p.window), static_cast<unsigned>((a.Hkv + p.heads - 1) / p.heads), 2);
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
