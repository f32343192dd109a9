// Policy and preference losses on per-token log probabilities, with their
// gradients. One block takes one sequence.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include "post_training.h"
#include "ptx.cuh"

namespace flce {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }

// Block sum in a fixed order; every thread gets it.
template <typename V>
__device__ __forceinline__ V block_total(V v) {
  __shared__ V sh[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();   // an earlier use of sh is over
  if (lane == 0) sh[warp] = v;
  __syncthreads();
  V r = 0;
  for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) r += sh[w];
  return r;
}

// Tokens of sequence s: `first` is the packed index of its first token (0 in
// padded batches, whose rows the callers address by s). Packed bounds are
// clamped to the tensor, so wrong ones cannot lead outside it.
__device__ __forceinline__ void sequence_range(const TokenView& t, long long s, long long* first,
                                               long long* len) {
  *first = 0;
  *len = s < t.S ? t.cols : 0;   // a batch without sequences has one idle block
  if (t.cu == nullptr || s >= t.S) return;
  long long a = t.cu[s], b = t.cu[s + 1];
  a = a < 0 ? 0 : (a > t.N ? t.N : a);
  b = b < a ? a : (b > t.N ? t.N : b);
  *first = a;
  *len = b - a;
}

// Offset of token c of sequence s in a tensor of row stride ld.
__device__ __forceinline__ long long token_at(const TokenView& t, long long s, long long first,
                                              long long c, long long ld) {
  return t.cu == nullptr ? s * ld + c : first + c;
}

__device__ __forceinline__ bool counts(const TokenView& t, long long s, long long first, long long c) {
  if (t.mask_kind == FLCE_MASK_NONE) return true;
  const long long i = token_at(t, s, first, c, t.ld_mask);
  if (t.mask_kind == FLCE_MASK_BYTES) return static_cast<const unsigned char*>(t.mask)[i] != 0;
  return static_cast<const long long*>(t.mask)[i] != t.ignore_index;
}

// True in every thread of the last block of the grid to get here (each block
// makes its stores visible before it counts itself).
__device__ __forceinline__ bool last_block(int* done) {
  __shared__ int s_last;
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) s_last = atomicAdd(done, 1) == static_cast<int>(gridDim.x) - 1;
  __syncthreads();
  if (s_last) __threadfence();
  return s_last != 0;
}

__global__ void __launch_bounds__(kThreads) token_count_kernel(const PolicyArgs a) {
  const long long s = blockIdx.x;
  long long first, len, n = 0;
  sequence_range(a.t, s, &first, &len);
  for (long long c = threadIdx.x; c < len; c += kThreads) n += counts(a.t, s, first, c) ? 1 : 0;
  n = block_total(n);
  if (threadIdx.x == 0 && store_allowed(a.counts + s, 8, a.r_ws, a.status)) a.counts[s] = n;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) policy_kernel(const PolicyArgs a) {
  const long long s = blockIdx.x;
  const T* lp = static_cast<const T*>(a.lp);
  const T* old = static_cast<const T*>(a.old);
  const T* ref = static_cast<const T*>(a.ref);
  long long tokens = 0;
  for (long long i = threadIdx.x; i < a.t.S; i += kThreads) tokens += a.counts[i];
  tokens = block_total(tokens);
  double w = 1.0;
  if (a.reduction == FLCE_TOKEN_MEAN) {
    w = 1.0 / static_cast<double>(tokens);
  } else if (a.reduction == FLCE_SEQUENCE_MEAN) {
    const long long n = a.counts[s];
    w = 1.0 / (static_cast<double>(a.t.S) * static_cast<double>(n > 0 ? n : 1));
  }
  const float wf = static_cast<float>(w);
  long long first, len;
  sequence_range(a.t, s, &first, &len);
  double sum = 0.0, kls = 0.0;
  long long clipped = 0;
  for (long long c = threadIdx.x; c < len; c += kThreads) {
    float grad = 0.f;
    if (counts(a.t, s, first, c)) {
      const float x = a.sign * to_f32(lp[token_at(a.t, s, first, c, a.ld_lp)]);
      const float adv = a.adv_per_token ? a.adv[token_at(a.t, s, first, c, a.ld_adv)] : a.adv[s];
      const float d = old != nullptr ? x - to_f32(old[token_at(a.t, s, first, c, a.ld_old)]) : 0.f;
      const float r = expf(d);
      float pg = 0.f;
      if (adv != 0.f) pg = fmaxf(-adv * r, -adv * expf(fminf(fmaxf(d, a.lo), a.hi)));
      bool clip = (adv > 0.f && d > a.hi) || (adv < 0.f && d < a.lo);
      if (a.dual > 0.f && adv < 0.f && d > a.log_dual) {
        pg = -a.dual * adv;
        clip = true;
      }
      if (!clip && adv != 0.f) grad = -adv * r;
      if (isnan(d)) pg = d;
      clipped += clip ? 1 : 0;
      if (a.kl_coef != 0.f) {
        const float e = x - to_f32(ref[token_at(a.t, s, first, c, a.ld_ref)]);
        float kl = e, dkl = 1.f;
        if (a.kl == FLCE_KL_K2) {
          kl = 0.5f * e * e;
          dkl = e;
        } else if (a.kl == FLCE_KL_K3) {
          const float q = expm1f(-e);
          kl = q + e;
          dkl = -q;
        }
        pg += a.kl_coef * kl;
        grad += a.kl_coef * dkl;
        kls += kl;
      }
      sum += static_cast<double>(pg) * w;
      grad *= wf * a.sign;
    }
    if (a.grad != nullptr) {
      float* const g = a.grad + token_at(a.t, s, first, c, a.ld_grad);
      if (store_allowed(g, 4, a.r_grad, a.status)) *g = grad;
    }
  }
  sum = block_total(sum);
  kls = block_total(kls);
  clipped = block_total(clipped);
  if (threadIdx.x == 0) {
    a.part_loss[s] = sum;
    a.part_kl[s] = kls;
    a.part_clipped[s] = clipped;
  }
  // tokens before the first sequence and after the last one
  if (a.t.cu != nullptr && a.grad != nullptr) {
    if (s == 0)
      for (long long i = threadIdx.x; i < first; i += kThreads) a.grad[i] = 0.f;
    if (s + 1 >= a.t.S)
      for (long long i = first + len + threadIdx.x; i < a.t.N; i += kThreads) a.grad[i] = 0.f;
  }
  if (!last_block(a.done)) return;
  sum = 0.0;
  kls = 0.0;
  clipped = 0;
  for (long long i = threadIdx.x; i < a.t.S; i += kThreads) {
    sum += __ldcg(a.part_loss + i);
    kls += __ldcg(a.part_kl + i);
    clipped += __ldcg(a.part_clipped + i);
  }
  sum = block_total(sum);
  kls = block_total(kls);
  clipped = block_total(clipped);
  if (threadIdx.x == 0) {
    const bool none = (a.reduction == FLCE_TOKEN_MEAN && tokens == 0) ||
                      (a.reduction == FLCE_SEQUENCE_MEAN && a.t.S == 0);
    *a.loss = none ? NAN : static_cast<float>(sum);
    if (a.num_tokens != nullptr) *a.num_tokens = tokens;
    if (a.num_clipped != nullptr) *a.num_clipped = clipped;
    if (a.kl_sum != nullptr) *a.kl_sum = static_cast<float>(kls);
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) sequence_sum_kernel(const PreferenceArgs a) {
  const long long s = blockIdx.x;
  const T* lp = static_cast<const T*>(a.lp);
  const T* ref = static_cast<const T*>(a.ref);
  long long first, len, n = 0;
  sequence_range(a.t, s, &first, &len);
  double sum = 0.0;
  for (long long c = threadIdx.x; c < len; c += kThreads) {
    if (!counts(a.t, s, first, c)) continue;
    float x = a.sign * to_f32(lp[token_at(a.t, s, first, c, a.ld_lp)]);
    if (ref != nullptr) x -= to_f32(ref[token_at(a.t, s, first, c, a.ld_ref)]);
    sum += x;
    ++n;
  }
  sum = block_total(sum);
  n = block_total(n);
  if (threadIdx.x == 0) {
    a.sums[s] = sum;
    a.counts[s] = n;
  }
}

__global__ void __launch_bounds__(kThreads) preference_kernel(const PreferenceArgs a) {
  const long long s = blockIdx.x, pairs = a.t.S / 2, b = s < pairs ? s : s - pairs;
  double inv_c = 1.0, inv_r = 1.0;
  if (a.average) {
    inv_c = 1.0 / static_cast<double>(a.counts[b] > 0 ? a.counts[b] : 1);
    inv_r = 1.0 / static_cast<double>(a.counts[pairs + b] > 0 ? a.counts[pairs + b] : 1);
  }
  const double sc = a.sums[b] * inv_c, sr = a.sums[pairs + b] * inv_r;
  const double beta = a.beta, e = a.smoothing;
  const double z = beta * (sc - sr) - a.margin;
  double loss, dz;
  if (a.type == FLCE_PREF_SIGMOID) {
    const double soft = log1p(exp(-fabs(z)));
    loss = (1.0 - e) * (soft + fmax(-z, 0.0)) + e * (soft + fmax(z, 0.0));
    dz = e - 1.0 / (1.0 + exp(z));
  } else if (a.type == FLCE_PREF_HINGE) {
    loss = fmax(0.0, 1.0 - z);
    dz = z < 1.0 ? -1.0 : 0.0;
  } else {
    const double u = (z - 0.5) / beta;
    loss = u * u;
    dz = 2.0 * u / beta;
  }
  if (threadIdx.x == 0 && s < pairs) {
    a.pair_loss[b] = loss;
    if (a.chosen != nullptr) a.chosen[b] = static_cast<float>(beta * sc);
    if (a.rejected != nullptr) a.rejected[b] = static_cast<float>(beta * sr);
  }
  if (a.grad != nullptr) {
    const float g = static_cast<float>(a.sign * beta * dz / static_cast<double>(pairs) *
                                       (s < pairs ? inv_c : -inv_r));
    long long first, len;
    sequence_range(a.t, s, &first, &len);
    for (long long c = threadIdx.x; c < len; c += kThreads) {
      float* const p = a.grad + token_at(a.t, s, first, c, a.ld_grad);
      if (store_allowed(p, 4, a.r_grad, a.status)) *p = counts(a.t, s, first, c) ? g : 0.f;
    }
    if (a.t.cu != nullptr) {
      if (s == 0)
        for (long long i = threadIdx.x; i < first; i += kThreads) a.grad[i] = 0.f;
      if (s + 1 >= a.t.S)
        for (long long i = first + len + threadIdx.x; i < a.t.N; i += kThreads) a.grad[i] = 0.f;
    }
  }
  if (!last_block(a.done)) return;
  double sum = 0.0;
  for (long long i = threadIdx.x; i < pairs; i += kThreads) sum += __ldcg(a.pair_loss + i);
  sum = block_total(sum);
  if (threadIdx.x == 0) *a.loss = static_cast<float>(sum / static_cast<double>(pairs));
}

unsigned blocks(const TokenView& t) { return t.S > 0 ? static_cast<unsigned>(t.S) : 1u; }

}  // namespace

cudaError_t launch_token_count(const PolicyArgs& a, cudaStream_t s) {
  token_count_kernel<<<blocks(a.t), kThreads, 0, s>>>(a);
  note_launch();
  return cudaGetLastError();
}

cudaError_t launch_policy(const PolicyArgs& a, int dtype, cudaStream_t s) {
  const unsigned grid = blocks(a.t);
  if (dtype == FLCE_BF16)
    policy_kernel<__nv_bfloat16><<<grid, kThreads, 0, s>>>(a);
  else if (dtype == FLCE_F16)
    policy_kernel<__half><<<grid, kThreads, 0, s>>>(a);
  else
    policy_kernel<float><<<grid, kThreads, 0, s>>>(a);
  note_launch();
  return cudaGetLastError();
}

cudaError_t launch_sequence_sum(const PreferenceArgs& a, int dtype, cudaStream_t s) {
  const unsigned grid = blocks(a.t);
  if (dtype == FLCE_BF16)
    sequence_sum_kernel<__nv_bfloat16><<<grid, kThreads, 0, s>>>(a);
  else if (dtype == FLCE_F16)
    sequence_sum_kernel<__half><<<grid, kThreads, 0, s>>>(a);
  else
    sequence_sum_kernel<float><<<grid, kThreads, 0, s>>>(a);
  note_launch();
  return cudaGetLastError();
}

cudaError_t launch_preference(const PreferenceArgs& a, int, cudaStream_t s) {
  preference_kernel<<<blocks(a.t), kThreads, 0, s>>>(a);
  note_launch();
  return cudaGetLastError();
}

}  // namespace flce
