// AdamW over many tensors in one launch: the table of tensors travels in the
// kernel's parameters. A warp takes one state block of 256 elements of one
// tensor, 8 neighbours a lane, so that the largest magnitude of an 8-bit block
// is a warp reduction.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <math.h>

#include "post_training.h"
#include "ptx.cuh"

namespace flce {
namespace {

constexpr int kBlock = 256;          // elements of a state block
constexpr int kThreads = 256;
constexpr unsigned kC1 = 0x9E3779B1u, kC2 = 0x85A308D3u;

#ifdef FLCE_DEBUG
__device__ int g_adamw_status;
#endif

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
template <typename T> __device__ __forceinline__ T from_f32(float x);
template <> __device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}
template <> __device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }

__device__ __forceinline__ float e4m3_to_f32(unsigned char b) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(b, __NV_E4M3)));
}

// Larger of two magnitudes, NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ unsigned pair_hash(unsigned pair, unsigned key) {
  unsigned x = (pair ^ key) * kC1;
  x ^= x >> 15;
  x *= kC2;
  x ^= x >> 13;
  x *= kC1;
  return x ^ (x >> 16);
}

// r x 448 / (largest) in [0, 448], or NaN -> e4m3 byte with the 16 random
// bits. x 2^-120 has e4m3's exponent field where fp32 has its own (bias 7
// against 127, subnormals included), so the code is its bits without the last
// 20, and adding random bits below them rounds up with the right probability.
__device__ __forceinline__ unsigned char e4m3_stochastic(float x, unsigned random16) {
  if (isnan(x)) return 0x7F;
  unsigned code = (__float_as_uint(x * 0x1p-120f) + (random16 << 4) + 8u) >> 20;
  code = code > 0x7Eu ? 0x7Eu : code;
  return static_cast<unsigned char>(x > 0.f && code == 0u ? 1u : code);
}

template <typename P, typename G, int kBits>
__global__ void __launch_bounds__(kThreads) adamw_kernel(const __grid_constant__ AdamWArgs a) {
  const int lane = threadIdx.x & 31;
  const unsigned gb = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);   // of this launch
  if (gb >= a.block0[a.count]) return;
  int lo = 0, hi = a.count;   // the last tensor that starts at or before gb
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.block0[mid] <= gb) lo = mid; else hi = mid;
  }
  const flce_adamw_tensor& t = a.t[lo];
  const unsigned sb = gb - a.block0[lo];
  const long long e0 = static_cast<long long>(sb) * kBlock + lane * 8;
  const float gs = a.grad_scale != nullptr ? *a.grad_scale : 1.f;
  P* p = static_cast<P*>(t.param);
  const G* g = static_cast<const G*>(t.grad);
  float ms = 0.f, vs = 0.f, m[8], r[8];
  if (kBits == 8) {
    ms = t.exp_avg_scale[sb];
    vs = t.exp_avg_sq_scale[sb];
  }
  float top_m = 0.f, top_r = 0.f;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    m[k] = 0.f;
    r[k] = 0.f;
    const long long i = e0 + k;
    if (i >= t.numel) continue;
    float mm, v;
    if (kBits == 8) {
      mm = e4m3_to_f32(static_cast<const unsigned char*>(t.exp_avg)[i]) * ms;
      v = e4m3_to_f32(static_cast<const unsigned char*>(t.exp_avg_sq)[i]) * vs;
      v *= v;
    } else {
      mm = static_cast<const float*>(t.exp_avg)[i];
      v = static_cast<const float*>(t.exp_avg_sq)[i];
    }
    const float gr = to_f32(g[i]) * gs;
    // rounded product by product, not fused: an 8-bit state is then the same on every
    // implementation of the formula, where one last bit could pick another code
    mm = __fadd_rn(__fmul_rn(a.beta1, mm), __fmul_rn(a.one_beta1, gr));
    v = __fadd_rn(__fmul_rn(a.beta2, v), __fmul_rn(a.one_beta2, __fmul_rn(gr, gr)));
    const float root = sqrtf(v);
    float x = t.master != nullptr ? t.master[i] : to_f32(p[i]);
    x = x * a.decay - a.step_size * mm / (root * a.inv_root_bc2 + a.eps);
    if (t.master != nullptr) t.master[i] = x;
    if (store_allowed(p + i, sizeof(P), DevRegion{p, t.numel * sizeof(P)}, a.status)) p[i] = from_f32<P>(x);
    if (kBits == 32) {
      static_cast<float*>(t.exp_avg)[i] = mm;
      static_cast<float*>(t.exp_avg_sq)[i] = v;
    } else {
      m[k] = mm;
      r[k] = root;
      top_m = max_nan(top_m, fabsf(mm));
      top_r = max_nan(top_r, root);
    }
  }
  if (kBits == 32) return;
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) {
    top_m = max_nan(top_m, __shfl_xor_sync(0xffffffffu, top_m, o));
    top_r = max_nan(top_r, __shfl_xor_sync(0xffffffffu, top_r, o));
  }
  // !(x < y): a NaN takes the first branch and makes the block NaN
  const float im = !(top_m < 0x1p-100f) ? 448.f / top_m : 0.f;
  const float ir = !(top_r < 0x1p-100f) ? 448.f / top_r : 0.f;
  if (lane == 0) {
    t.exp_avg_scale[sb] = !(top_m < 0x1p-100f) ? top_m / 448.f : 0.f;
    t.exp_avg_sq_scale[sb] = !(top_r < 0x1p-100f) ? top_r / 448.f : 0.f;
  }
  const unsigned pair0 = (a.first_block + gb) * (kBlock / 2) + lane * 4;   // mod 2^32
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const long long i = e0 + k;
    if (i >= t.numel) continue;
    const unsigned x = pair_hash(pair0 + k / 2, a.key);
    static_cast<unsigned char*>(t.exp_avg)[i] = __nv_cvt_float_to_fp8(m[k] * im, __NV_SATFINITE, __NV_E4M3);
    static_cast<unsigned char*>(t.exp_avg_sq)[i] = e4m3_stochastic(r[k] * ir, k & 1 ? x >> 16 : x & 0xffffu);
  }
}

template <typename P, typename G>
cudaError_t launch_bits(const AdamWArgs& a, int bits, unsigned grid, cudaStream_t s) {
  if (bits == 8)
    adamw_kernel<P, G, 8><<<grid, kThreads, 0, s>>>(a);
  else
    adamw_kernel<P, G, 32><<<grid, kThreads, 0, s>>>(a);
  note_launch();
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_adamw(const AdamWArgs& a, int dtype, int grad_dtype, int bits, cudaStream_t s) {
  const unsigned grid = (a.block0[a.count] + kThreads / 32 - 1) / (kThreads / 32);
  if (dtype == FLCE_F32) return launch_bits<float, float>(a, bits, grid, s);
  if (dtype == FLCE_BF16)
    return grad_dtype == FLCE_F32 ? launch_bits<__nv_bfloat16, float>(a, bits, grid, s)
                                  : launch_bits<__nv_bfloat16, __nv_bfloat16>(a, bits, grid, s);
  return grad_dtype == FLCE_F32 ? launch_bits<__half, float>(a, bits, grid, s)
                                : launch_bits<__half, __half>(a, bits, grid, s);
}

cudaError_t adamw_status(int** status) {
  *status = nullptr;
#ifdef FLCE_DEBUG
  void* p = nullptr;
  const cudaError_t e = cudaGetSymbolAddress(&p, g_adamw_status);
  if (e != cudaSuccess) return e;
  *status = static_cast<int*>(p);
#endif
  return cudaSuccess;
}

}  // namespace flce
