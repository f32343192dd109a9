// Policy and preference losses on per-token log probabilities, with their
// gradients. Both are bound by memory traffic, or by latency for the batches
// of a few thousand tokens, so they read each token once, four neighbours a
// thread, and read nothing but the mask where no token of the four counts.
//
// Policy loss. A gradient needs its weight, 1 / (tokens that count) of the
// batch or of the sequence, before it can be written. A small batch is one
// cluster of eight blocks that keeps its tokens in registers while it counts
// them (policy_small_kernel, one launch). A large one counts the mask first
// (count kernels, 1 byte of the 17 to 21 a token), then streams the tokens
// (policy_kernel). The streaming kernel cuts the tokens into contiguous
// ranges, one a block, so that walking from sequence to sequence is cheap
// whatever their lengths.
//
// Preference loss. A pair's gradient is one number a sequence, known once
// both sums are: a cluster of 1 to 8 blocks takes a pair, adds it up, and
// writes its gradient (preference_kernel); a small batch is again one cluster,
// each block of which takes pairs by itself.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include "post_training.h"
#include "ptx.cuh"

namespace flce {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 256;          // streaming and counting kernels
constexpr int kSmallThreads = 1024;    // policy_small_kernel
constexpr int kPairThreads = 512;      // preference kernels
constexpr int kCluster = 8;

// ------------------------------------------------------------- reductions
// A sum in fp32 together with the rounding errors of its additions, which is
// about as exact as fp64. A GB300 SM adds two fp64 numbers a cycle: one fp64
// reduction over a block of 512 takes more than a microsecond.
struct Sum {
  float s, c;
  __device__ __forceinline__ void add(float x) {
    const float t = __fadd_rn(s, x), u = __fsub_rn(t, s);
    c = __fadd_rn(c, __fadd_rn(__fsub_rn(s, __fsub_rn(t, u)), __fsub_rn(x, u)));
    s = t;
  }
  // An infinity or NaN stays itself: what it leaves in c does not count.
  __device__ __forceinline__ float total() const { return isfinite(s) ? __fadd_rn(s, c) : s; }
};
__device__ __forceinline__ Sum operator+(Sum a, const Sum& b) {
  a.add(b.s);
  a.c = __fadd_rn(a.c, b.c);
  return a;
}
__device__ __forceinline__ Sum shuffle_xor(const Sum& v, int o) {
  return Sum{__shfl_xor_sync(0xffffffffu, v.s, o), __shfl_xor_sync(0xffffffffu, v.c, o)};
}
template <typename V>
__device__ __forceinline__ V shuffle_xor(V v, int o) { return __shfl_xor_sync(0xffffffffu, v, o); }

// Total over the block in a fixed order; every thread gets it.
template <typename V>
__device__ __forceinline__ V block_total(V v) {
  __shared__ V sh[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v = v + shuffle_xor(v, o);
  __syncthreads();   // an earlier use of sh is over
  if (lane == 0) sh[warp] = v;
  __syncthreads();
  V r = lane < static_cast<int>(blockDim.x >> 5) ? sh[lane] : V{};
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) r = r + shuffle_xor(r, o);
  return r;
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

// Programmatic dependent launch: the next kernel of the stream may start; this
// kernel's reads of what the one before it wrote may begin.
__device__ __forceinline__ void allow_next() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void wait_for_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// ------------------------------------------------------- groups of 4 tokens
__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }

__device__ __forceinline__ void load4_vec(const float* p, float (&x)[4]) {
  const float4 v = __ldg(reinterpret_cast<const float4*>(p));
  x[0] = v.x;
  x[1] = v.y;
  x[2] = v.z;
  x[3] = v.w;
}
template <typename T>
__device__ __forceinline__ void load4_vec(const T* p, float (&x)[4]) {
  const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
  x[0] = Elem<T>::lo(v.x);
  x[1] = Elem<T>::hi(v.x);
  x[2] = Elem<T>::lo(v.y);
  x[3] = Elem<T>::hi(v.y);
}
// The tokens of `bits`; the others read as 0. `vec`: p is aligned to four
// elements and all four are in the tensor.
template <typename T>
__device__ __forceinline__ void load4(const T* p, unsigned bits, bool vec, float (&x)[4]) {
  if (vec) {
    load4_vec(p, x);
    return;
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) x[k] = bits >> k & 1u ? to_f32(p[k]) : 0.f;
}
// The tokens of `range` (a subset of the four). `r`: the tensor the store must
// stay in (checked in FLCE_DEBUG builds).
__device__ __forceinline__ void store4(float* p, unsigned range, bool vec, const float (&x)[4],
                                       const DevRegion& r, int* status) {
  if (vec) {
    if (store_allowed(p, 16, r, status))
      *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
    return;
  }
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if ((range >> k & 1u) && store_allowed(p + k, 4, r, status)) p[k] = x[k];
}

// Which of the tokens i .. i + 3 of the mask (of those in `range`) count.
__device__ __forceinline__ unsigned mask4(const TokenView& t, long long i, unsigned range, bool vec) {
  if (t.mask_kind == FLCE_MASK_NONE) return range;
  unsigned bits = 0;
  if (t.mask_kind == FLCE_MASK_BYTES) {
    const unsigned char* m = static_cast<const unsigned char*>(t.mask) + i;
    if (vec) {
      const unsigned w = __vsetgtu4(__ldg(reinterpret_cast<const unsigned*>(m)), 0u);   // 1 a byte
      return (w * 0x01020408u) >> 24;   // byte k to bit 24 + k, without carries
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (range >> k & 1u) bits |= (m[k] != 0 ? 1u : 0u) << k;
    return bits;
  }
  const long long* m = static_cast<const long long*>(t.mask) + i;
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (range >> k & 1u) bits |= (__ldg(m + k) != t.ignore_index ? 1u : 0u) << k;
  return bits;
}

// ------------------------------------------------------------- sequences
// Packed bounds are clamped to the tensor, so wrong ones cannot lead outside it.
__device__ __forceinline__ long long clamp_to(long long x, long long n) {
  return x < 0 ? 0 : (x > n ? n : x);
}
__device__ __forceinline__ long long sequence_first(const TokenView& t, long long s) {
  return t.cu != nullptr ? clamp_to(__ldg(t.cu + s), t.N) : s * t.cols;
}
__device__ __forceinline__ long long sequence_end(const TokenView& t, long long s, long long first) {
  if (t.cu == nullptr) return first + t.cols;
  const long long e = clamp_to(__ldg(t.cu + s + 1), t.N);
  return e < first ? first : e;
}

// The sequence that flat token i lies in, and its end, walking on from an
// earlier one.
struct Walker {
  long long s = 0, end = -1;
  __device__ __forceinline__ void to(const TokenView& t, long long i) {
    if (i < end) return;
    if (t.cu == nullptr) {
      s = t.N <= 0x7fffffffll ? static_cast<unsigned>(i) / static_cast<unsigned>(t.cols) : i / t.cols;
      end = (s + 1) * t.cols;
      return;
    }
    // the last sequence that begins at or before i: doubling steps, then halving ones
    long long step = 1;
    while (s + step < t.S && __ldg(t.cu + s + step) <= i) {
      s += step;
      step *= 2;
    }
    for (; step >= 1; step /= 2)
      if (s + step < t.S && __ldg(t.cu + s + step) <= i) s += step;
    end = sequence_end(t, s, 0);
  }
};

// Group q of the batch. Flat (every token tensor is contiguous): tokens 4q ..
// 4q + 3, which may belong to several sequences. Strided: four neighbours in a
// row, tokens 4 (q mod groups a row) .. of row q / groups a row.
template <bool kFlat>
struct Group {
  long long row, at;      // strided: row, column; flat: -, first token
  unsigned range, bits;   // the tokens that exist, and those that count
  bool whole;             // all four exist
  __device__ __forceinline__ long long index(long long ld) const { return kFlat ? at : row * ld + at; }
  __device__ __forceinline__ void find(const PolicyArgs& a, long long q) {
    const TokenView& t = a.t;
    long long rest;
    if (kFlat) {
      row = 0;
      at = q * 4;
      rest = t.N - at;
    } else {
      row = a.groups <= 0x7fffffffll ? static_cast<unsigned>(q) / static_cast<unsigned>(a.row_groups)
                                     : q / a.row_groups;
      at = (q - row * a.row_groups) * 4;
      rest = t.cols - at;
    }
    whole = rest >= 4;
    range = whole ? 15u : (1u << rest) - 1u;
    unsigned in = range;
    if (kFlat && t.cu != nullptr) {
      // tokens outside every sequence do not count
      const long long first = __ldg(t.cu), end = t.S > 0 ? __ldg(t.cu + t.S) : 0;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (at + k < first || at + k >= end) in &= ~(1u << k);
    }
    bits = mask4(t, index(t.ld_mask), range, a.vec_mask && whole) & in;
  }
};

// --------------------------------------------------------------- policy
// The terms of one token, not yet weighted.
struct Term {
  float loss, grad, kl;
  bool clipped;
};

__device__ __forceinline__ Term policy_term(const PolicyArgs& a, float x, float old, float ref,
                                            float adv) {
  Term o{0.f, 0.f, 0.f, false};
  const float d = a.old != nullptr ? __fsub_rn(x, old) : 0.f;
  const float r = expf(d);
  const bool over = d > a.hi, under = d < a.lo;
  // max(-A r, -A clipped r): the clip takes the term where it lowers the gain
  o.clipped = (adv > 0.f && over) || (adv < 0.f && under);
  o.loss = -adv * (o.clipped ? (over ? a.ratio_hi : a.ratio_lo) : r);
  o.grad = o.clipped ? 0.f : -adv * r;
  if (a.dual > 0.f && adv < 0.f && d > a.log_dual) {
    o.loss = -a.dual * adv;
    o.grad = 0.f;
    o.clipped = true;
  }
  if (adv == 0.f && !isnan(d)) o.loss = o.grad = 0.f;   // not 0 x infinity
  if (a.kl_coef != 0.f) {
    const float e = __fsub_rn(x, ref);
    float dkl = 1.f;
    o.kl = e;
    if (a.kl == FLCE_KL_K2) {
      o.kl = 0.5f * e * e;
      dkl = e;
    } else if (a.kl == FLCE_KL_K3) {
      const float q = expm1f(-e);
      o.kl = q + e;
      dkl = -q;
    }
    o.loss = fmaf(a.kl_coef, o.kl, o.loss);
    o.grad = fmaf(a.kl_coef, dkl, o.grad);
  }
  return o;
}

template <typename T, bool kFlat>
__device__ __forceinline__ void policy_load(const PolicyArgs& a, const Group<kFlat>& g, float (&x)[4],
                                            float (&old)[4], float (&ref)[4], float (&adv)[4]) {
  const bool vec = a.vec && g.whole;
  load4(static_cast<const T*>(a.lp) + g.index(a.ld_lp), g.bits, vec, x);
  if (a.old != nullptr) load4(static_cast<const T*>(a.old) + g.index(a.ld_old), g.bits, vec, old);
  if (a.kl_coef != 0.f) load4(static_cast<const T*>(a.ref) + g.index(a.ld_ref), g.bits, vec, ref);
  if (a.adv_per_token) load4(a.adv + g.index(a.ld_adv), g.bits, vec, adv);
}

// What the reduced outputs are made of.
struct Totals {
  Sum loss, kl;
  long long clipped, tokens;
};

__device__ __forceinline__ void policy_outputs(const PolicyArgs& a, const Totals& v) {
  const bool none = (a.reduction == FLCE_TOKEN_MEAN && v.tokens == 0) ||
                    (a.reduction == FLCE_SEQUENCE_MEAN && a.t.S == 0);
  *a.loss = none ? NAN : v.loss.total();
  if (a.num_tokens != nullptr) *a.num_tokens = v.tokens;
  if (a.num_clipped != nullptr) *a.num_clipped = v.clipped;
  if (a.kl_sum != nullptr) *a.kl_sum = v.kl.total();
}

__device__ __forceinline__ float sequence_weight(const PolicyArgs& a, long long n) {
  return 1.f / (static_cast<float>(a.t.S) * static_cast<float>(n > 0 ? n : 1));
}

// One cluster, one group a thread. For "sequence_mean" with a mask each block
// counts its tokens of each sequence in shared memory (at most
// kPolicySmallSequences of them), and a thread adds the eight counts of its
// sequences.
template <typename T, bool kFlat>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kSmallThreads)
    policy_small_kernel(const PolicyArgs a) {
  __shared__ int s_count[kPolicySmallSequences];
  __shared__ Totals s_totals;
  cg::cluster_group cluster = cg::this_cluster();
  const bool by_sequence = a.reduction == FLCE_SEQUENCE_MEAN;
  const bool count_rows = by_sequence && a.t.mask_kind != FLCE_MASK_NONE;
  if (count_rows) {
    for (int i = threadIdx.x; i < a.t.S; i += kSmallThreads) s_count[i] = 0;
    __syncthreads();
  }
  const long long q = static_cast<long long>(blockIdx.x) * kSmallThreads + threadIdx.x;
  Group<kFlat> g{};
  float x[4], old[4], ref[4], adv[4];
  if (q < a.groups) g.find(a, q);
  if (g.bits != 0) policy_load<T>(a, g, x, old, ref, adv);
  int row[4];
  Term term[4];
  Walker w;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    row[k] = 0;
    term[k] = Term{0.f, 0.f, 0.f, false};
    if (!(g.bits >> k & 1u)) continue;
    if (by_sequence || !a.adv_per_token) {
      if (kFlat) w.to(a.t, g.at + k); else w.s = g.row;
      row[k] = static_cast<int>(w.s);
    }
    if (count_rows) atomicAdd(s_count + row[k], 1);
    term[k] = policy_term(a, a.sign * x[k], old[k], ref[k], a.adv_per_token ? adv[k] : a.adv[row[k]]);
  }
  const int n = block_total(__popc(g.bits));
  if (threadIdx.x == 0) s_totals.tokens = n;
  cluster.sync();
  long long tokens = 0;
  for (int b = 0; b < kCluster; ++b) tokens += cluster.map_shared_rank(&s_totals, b)->tokens;
  float weight = a.reduction == FLCE_TOKEN_MEAN ? 1.f / static_cast<float>(tokens) : 1.f;
  Sum loss{}, kl{};
  int clipped = 0;
  float out[4];
  int have = -1;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    out[k] = 0.f;
    if (!(g.bits >> k & 1u)) continue;
    if (by_sequence && row[k] != have) {
      have = row[k];
      long long c = 0;
      if (count_rows)
        for (int b = 0; b < kCluster; ++b) c += *cluster.map_shared_rank(s_count + have, b);
      else
        c = sequence_end(a.t, have, sequence_first(a.t, have)) - sequence_first(a.t, have);
      weight = sequence_weight(a, c);
    }
    out[k] = term[k].grad * weight * a.sign;
    loss.add(term[k].loss * weight);
    kl.add(term[k].kl);
    clipped += term[k].clipped ? 1 : 0;
  }
  if (a.grad != nullptr && q < a.groups)
    store4(a.grad + g.index(a.ld_grad), g.range, a.vec_grad && g.whole, out, a.r_grad, a.status);
  loss = block_total(loss);
  kl = block_total(kl);
  clipped = block_total(clipped);
  if (threadIdx.x == 0) {
    s_totals.loss = loss;
    s_totals.kl = kl;
    s_totals.clipped = clipped;
  }
  cluster.sync();
  if (cluster.block_rank() == 0 && threadIdx.x == 0) {
    Totals v{};
    for (int b = 0; b < kCluster; ++b) {
      const Totals* o = cluster.map_shared_rank(&s_totals, b);
      v.loss = v.loss + o->loss;
      v.kl = v.kl + o->kl;
      v.clipped += o->clipped;
    }
    v.tokens = tokens;
    policy_outputs(a, v);
  }
  cluster.sync();   // the other blocks' shared memory stays until it has been read
}

// Tokens that count, one number a block ("mean").
template <bool kFlat>
__global__ void __launch_bounds__(kThreads) count_tokens_kernel(const PolicyArgs a) {
  allow_next();
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.done = 0;
  int n = 0;
  const long long step = static_cast<long long>(gridDim.x) * kThreads;
  for (long long q = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x; q < a.groups; q += step) {
    Group<kFlat> g;
    g.find(a, q);
    n += __popc(g.bits);
  }
  const long long total = block_total(static_cast<long long>(n));
  if (threadIdx.x == 0 && store_allowed(a.counts + blockIdx.x, 8, a.r_ws, a.status))
    a.counts[blockIdx.x] = total;
}

// Tokens that count, one number a sequence ("sequence_mean"): kLanes threads a
// sequence, a warp for short ones and a block for long ones.
template <int kLanes>
__global__ void __launch_bounds__(kThreads) count_sequences_kernel(const PolicyArgs a) {
  allow_next();
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.done = 0;
  const int lane = threadIdx.x % kLanes;
  const long long teams = static_cast<long long>(gridDim.x) * (kThreads / kLanes);
  for (long long s = static_cast<long long>(blockIdx.x) * (kThreads / kLanes) + threadIdx.x / kLanes;
       s < a.t.S; s += teams) {
    const long long first = sequence_first(a.t, s), len = sequence_end(a.t, s, first) - first;
    const long long base = a.t.cu != nullptr ? first : s * a.t.ld_mask;
    // groups begin where the mask is aligned: up to three tokens before the sequence
    const long long shift = a.vec_mask ? base & 3 : 0;
    long long n = 0;
    for (long long c = 4ll * lane - shift; c < len; c += 4 * kLanes) {
      unsigned range = 15u;
      if (c < 0) range = 15u << -c & 15u;
      if (len - c < 4) range &= (1u << (len - c)) - 1u;
      n += __popc(mask4(a.t, base + c, range, a.vec_mask && range == 15u));
    }
    if (kLanes == 32) {
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
    } else {
      n = block_total(n);
    }
    if (lane == 0 && store_allowed(a.counts + s, 8, a.r_ws, a.status)) a.counts[s] = n;
  }
}

// a.per groups a block, kThreads at a time; the mask of the next ones is on
// its way while these are computed.
template <typename T, bool kFlat>
__global__ void __launch_bounds__(kThreads, kPolicyBlocksPerSm) policy_kernel(const PolicyArgs a) {
  const bool by_sequence = a.reduction == FLCE_SEQUENCE_MEAN;
  const bool need_row = by_sequence || !a.adv_per_token;
  long long q = blockIdx.x * a.per + threadIdx.x;
  const long long end = min(a.groups, (blockIdx.x + 1) * a.per);
  Group<kFlat> g{}, next{};
  if (q < end) next.find(a, q);
  wait_for_previous();
  long long tokens = 0;
  float weight = 1.f;
  if (a.reduction == FLCE_TOKEN_MEAN) {
    if (a.num_counts > 0) {
      for (int i = threadIdx.x; i < a.num_counts; i += kThreads) tokens += a.counts[i];
      tokens = block_total(tokens);
    } else {   // without a mask: what lies in sequences
      tokens = a.t.cu == nullptr ? a.t.N
               : a.t.S > 0 ? max(0ll, clamp_to(a.t.cu[a.t.S], a.t.N) - clamp_to(a.t.cu[0], a.t.N)) : 0;
    }
    weight = 1.f / static_cast<float>(tokens);
  }
  Sum loss{}, kl{};
  int clipped = 0, seen = 0;
  Walker w;
  long long have = -1;
  float adv_row = 0.f;
  for (; q < end; q += kThreads) {
    g = next;
    if (q + kThreads < end) next.find(a, q + kThreads);
    float out[4] = {0.f, 0.f, 0.f, 0.f};
    if (g.bits != 0) {
      float x[4], old[4], ref[4], adv[4];
      policy_load<T>(a, g, x, old, ref, adv);
      float l = 0.f, kk = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (!(g.bits >> k & 1u)) continue;
        if (need_row) {
          if (kFlat) w.to(a.t, g.at + k); else w.s = g.row;
          if (w.s != have) {
            have = w.s;
            if (!a.adv_per_token) adv_row = __ldg(a.adv + have);
            if (by_sequence) {
              const long long first = sequence_first(a.t, have);
              weight = sequence_weight(a, a.num_counts > 0 ? a.counts[have]
                                                           : sequence_end(a.t, have, first) - first);
            }
          }
        }
        const Term o = policy_term(a, a.sign * x[k], old[k], ref[k], a.adv_per_token ? adv[k] : adv_row);
        out[k] = o.grad * weight * a.sign;
        l += o.loss * weight;
        kk += o.kl;
        clipped += o.clipped ? 1 : 0;
      }
      loss.add(l);
      kl.add(kk);
      seen += __popc(g.bits);
    }
    if (a.grad != nullptr)
      store4(a.grad + g.index(a.ld_grad), g.range, a.vec_grad && g.whole, out, a.r_grad, a.status);
  }
  loss = block_total(loss);
  kl = block_total(kl);
  const long long both = block_total(static_cast<long long>(clipped) << 32 | static_cast<long long>(seen));
  if (threadIdx.x == 0 && store_allowed(a.partials + blockIdx.x, sizeof(PolicyPartial), a.r_ws, a.status))
    a.partials[blockIdx.x] = PolicyPartial{loss.s, loss.c, kl.s, kl.c, both};
  if (!last_block(a.done)) return;
  Totals v{};
  for (unsigned i = threadIdx.x; i < gridDim.x; i += kThreads) {
    const PolicyPartial* o = a.partials + i;
    const float4 f = __ldcg(reinterpret_cast<const float4*>(o));
    const long long n = __ldcg(&o->both);
    v.loss = v.loss + Sum{f.x, f.y};
    v.kl = v.kl + Sum{f.z, f.w};
    v.clipped += n >> 32;
    v.tokens += n & 0xffffffffll;
  }
  v.loss = block_total(v.loss);
  v.kl = block_total(v.kl);
  v.clipped = block_total(v.clipped);
  v.tokens = block_total(v.tokens);
  if (threadIdx.x == 0) policy_outputs(a, v);
}

// ------------------------------------------------------------ preference
// The tokens of one sequence, as the groups of four that a team of threads
// goes through: group j of the sequence is tokens 4j - shift .. + 3, so that
// the groups of a contiguous batch are aligned wherever the sequence begins.
struct Row {
  long long first, len;   // flat token of the start; tokens
  long long shift;
  __device__ __forceinline__ void find(const PreferenceArgs& a, long long s) {
    first = sequence_first(a.t, s);
    len = sequence_end(a.t, s, first) - first;
    shift = a.flat ? first & 3 : 0;
  }
  __device__ __forceinline__ long long groups() const { return (len + shift + 3) / 4; }
  __device__ __forceinline__ unsigned range(long long c) const {
    unsigned r = 15u;
    if (c < 0) r = 15u << -c & 15u;
    if (len - c < 4) r &= (1u << (len - c)) - 1u;
    return r;
  }
};

constexpr int kKept = 16;   // groups of a thread whose mask stays in a register

// Both sequences of pair b by `team` threads, of which this is number
// `member`. `total` adds a value over the team. Returns the pair's loss.
template <typename T, class Total>
__device__ __forceinline__ float preference_pair(const PreferenceArgs& a, long long b, int member,
                                                  int team, Total total) {
  const long long pairs = a.t.S / 2;
  unsigned long long kept = 0;
  int j = 0, n[2] = {0, 0};
  Sum sum[2] = {};
  Row row;
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    const long long s = side == 0 ? b : pairs + b;
    row.find(a, s);
    const long long at_lp = a.flat ? row.first : s * a.ld_lp, at_ref = a.flat ? row.first : s * a.ld_ref;
    const long long at_mask = a.flat ? row.first : s * a.t.ld_mask;
    const long long groups = row.groups();
    for (long long q = member; q < groups; q += team, ++j) {
      const long long c = 4 * q - row.shift;
      const unsigned range = row.range(c);
      const unsigned bits = mask4(a.t, at_mask + c, range, a.vec_mask && range == 15u);
      if (j < kKept) kept |= static_cast<unsigned long long>(bits) << (4 * j);
      if (bits == 0) continue;
      float x[4], r[4];
      load4(static_cast<const T*>(a.lp) + at_lp + c, bits, a.vec && range == 15u, x);
      if (a.ref != nullptr)
        load4(static_cast<const T*>(a.ref) + at_ref + c, bits, a.vec && range == 15u, r);
      float d = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (bits >> k & 1u) d += a.ref != nullptr ? a.sign * x[k] - r[k] : a.sign * x[k];
      sum[side].add(d);
      n[side] += __popc(bits);
    }
  }
  long long count = static_cast<long long>(n[0]) << 32 | static_cast<long long>(n[1]);
  total(sum[0], sum[1], count);
  float inv_c = 1.f, inv_r = 1.f;
  if (a.average) {
    inv_c = 1.f / static_cast<float>(max(1ll, count >> 32));
    inv_r = 1.f / static_cast<float>(max(1ll, count & 0xffffffffll));
  }
  const float s_c = sum[0].total() * inv_c, s_r = sum[1].total() * inv_r;
  const float e = a.smoothing, z = a.beta * (s_c - s_r) - a.margin;
  float loss, dz;
  if (a.type == FLCE_PREF_SIGMOID) {
    const float soft = log1pf(expf(-fabsf(z)));
    loss = isnan(z) ? z : (1.f - e) * (soft + fmaxf(-z, 0.f)) + e * (soft + fmaxf(z, 0.f));
    dz = e - 1.f / (1.f + expf(z));
  } else if (a.type == FLCE_PREF_HINGE) {
    loss = isnan(z) ? z : fmaxf(0.f, 1.f - z);
    dz = z < 1.f ? -1.f : 0.f;
  } else {
    const float u = (z - 0.5f) / a.beta;
    loss = u * u;
    dz = 2.f * u / a.beta;
  }
  if (member == 0) {
    if (a.chosen != nullptr) a.chosen[b] = a.beta * s_c;
    if (a.rejected != nullptr) a.rejected[b] = a.beta * s_r;
  }
  if (a.grad == nullptr) return loss;
  const float g = a.sign * a.beta * dz / static_cast<float>(pairs);
  j = 0;
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    const long long s = side == 0 ? b : pairs + b;
    row.find(a, s);
    const float w = side == 0 ? g * inv_c : -g * inv_r;
    const long long at_mask = a.flat ? row.first : s * a.t.ld_mask;
    float* const out = a.grad + (a.flat ? row.first : s * a.ld_grad);
    const long long groups = row.groups();
    for (long long q = member; q < groups; q += team, ++j) {
      const long long c = 4 * q - row.shift;
      const unsigned range = row.range(c);
      const unsigned bits = j < kKept ? static_cast<unsigned>(kept >> (4 * j)) & 15u
                                      : mask4(a.t, at_mask + c, range, a.vec_mask && range == 15u);
      float v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = bits >> k & 1u ? w : 0.f;
      store4(out + c, range, a.vec_grad && range == 15u, v, a.r_grad, a.status);
    }
  }
  if (b == 0 && a.t.cu != nullptr) {   // tokens outside every sequence
    const long long first = sequence_first(a.t, 0), last = sequence_first(a.t, a.t.S);
    for (long long i = member; i < first; i += team) a.grad[i] = 0.f;
    for (long long i = last + member; i < a.t.N; i += team) a.grad[i] = 0.f;
  }
  return loss;
}

// A cluster takes a pair; the last block to finish averages the pairs' losses.
template <typename T>
__global__ void __launch_bounds__(kPairThreads) preference_kernel(const PreferenceArgs a) {
  struct Part {
    Sum c, r;
    long long n;
  };
  __shared__ Part s_part;
  cg::cluster_group cluster = cg::this_cluster();
  const int blocks = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  const long long b = blockIdx.x / blocks;
  const float loss = preference_pair<T>(
      a, b, rank * kPairThreads + threadIdx.x, blocks * kPairThreads,
      [&](Sum& c, Sum& r, long long& n) {
        c = block_total(c);
        r = block_total(r);
        n = block_total(n);
        if (blocks == 1) return;
        if (threadIdx.x == 0) s_part = Part{c, r, n};
        cluster.sync();
        c = r = Sum{};
        n = 0;
        for (int i = 0; i < blocks; ++i) {
          const Part* o = cluster.map_shared_rank(&s_part, i);
          c = c + o->c;
          r = r + o->r;
          n += o->n;
        }
      });
  if (blocks > 1) cluster.sync();   // s_part stays until it has been read
  if (rank == 0 && threadIdx.x == 0 && store_allowed(a.pair_loss + b, 4, a.r_ws, a.status))
    a.pair_loss[b] = loss;
  if (!last_block(a.done)) return;
  Sum sum{};
  for (long long i = threadIdx.x; i < a.t.S / 2; i += kPairThreads) sum.add(__ldcg(a.pair_loss + i));
  sum = block_total(sum);
  if (threadIdx.x == 0) *a.loss = sum.total() / static_cast<float>(a.t.S / 2);
}

// One cluster; its blocks take the pairs in turn.
template <typename T>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kPairThreads)
    preference_small_kernel(const PreferenceArgs a) {
  __shared__ Sum s_loss;
  cg::cluster_group cluster = cg::this_cluster();
  const long long pairs = a.t.S / 2;
  Sum loss{};
  for (long long b = blockIdx.x; b < pairs; b += kCluster)
    loss.add(preference_pair<T>(a, b, threadIdx.x, kPairThreads, [](Sum& c, Sum& r, long long& n) {
      c = block_total(c);
      r = block_total(r);
      n = block_total(n);
    }));
  if (threadIdx.x == 0) s_loss = loss;
  cluster.sync();
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    Sum sum{};
    for (int i = 0; i < kCluster; ++i) sum = sum + *cluster.map_shared_rank(&s_loss, i);
    *a.loss = sum.total() / static_cast<float>(pairs);
  }
  cluster.sync();   // s_loss stays until it has been read
}

template <class... K>
cudaError_t launch_with(cudaLaunchAttribute attr, unsigned grid, unsigned threads, cudaStream_t s,
                        void (*kernel)(K...), const K&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  if (e != cudaSuccess) return e;
  note_launch();
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_policy_small(const PolicyArgs& a, int dtype, cudaStream_t s) {
  const auto go = [&](auto* kernel) {
    kernel<<<kCluster, kSmallThreads, 0, s>>>(a);
    note_launch();
    return cudaGetLastError();
  };
  if (dtype == FLCE_BF16)
    return a.flat ? go(policy_small_kernel<__nv_bfloat16, true>) : go(policy_small_kernel<__nv_bfloat16, false>);
  if (dtype == FLCE_F16)
    return a.flat ? go(policy_small_kernel<__half, true>) : go(policy_small_kernel<__half, false>);
  return a.flat ? go(policy_small_kernel<float, true>) : go(policy_small_kernel<float, false>);
}

cudaError_t launch_count(const PolicyArgs& a, int blocks, cudaStream_t s) {
  if (a.reduction == FLCE_TOKEN_MEAN) {
    if (a.flat)
      count_tokens_kernel<true><<<blocks, kThreads, 0, s>>>(a);
    else
      count_tokens_kernel<false><<<blocks, kThreads, 0, s>>>(a);
  } else if (a.t.N / (a.t.S > 0 ? a.t.S : 1) < 1024) {
    count_sequences_kernel<32><<<blocks, kThreads, 0, s>>>(a);
  } else {
    count_sequences_kernel<kThreads><<<blocks, kThreads, 0, s>>>(a);
  }
  note_launch();
  return cudaGetLastError();
}

cudaError_t launch_policy(const PolicyArgs& a, int dtype, bool after_count, unsigned grid, cudaStream_t s) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = after_count ? 1 : 0;
  const auto go = [&](auto* kernel) { return launch_with(attr, grid, kThreads, s, kernel, a); };
  if (dtype == FLCE_BF16)
    return a.flat ? go(policy_kernel<__nv_bfloat16, true>) : go(policy_kernel<__nv_bfloat16, false>);
  if (dtype == FLCE_F16)
    return a.flat ? go(policy_kernel<__half, true>) : go(policy_kernel<__half, false>);
  return a.flat ? go(policy_kernel<float, true>) : go(policy_kernel<float, false>);
}

cudaError_t launch_preference_small(const PreferenceArgs& a, int dtype, cudaStream_t s) {
  if (dtype == FLCE_BF16)
    preference_small_kernel<__nv_bfloat16><<<kCluster, kPairThreads, 0, s>>>(a);
  else if (dtype == FLCE_F16)
    preference_small_kernel<__half><<<kCluster, kPairThreads, 0, s>>>(a);
  else
    preference_small_kernel<float><<<kCluster, kPairThreads, 0, s>>>(a);
  note_launch();
  return cudaGetLastError();
}

cudaError_t launch_preference(const PreferenceArgs& a, int dtype, int cluster, cudaStream_t s) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = static_cast<unsigned>(cluster);
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  const unsigned grid = static_cast<unsigned>(a.t.S / 2) * static_cast<unsigned>(cluster);
  if (dtype == FLCE_BF16)
    return launch_with(attr, grid, kPairThreads, s, preference_kernel<__nv_bfloat16>, a);
  if (dtype == FLCE_F16) return launch_with(attr, grid, kPairThreads, s, preference_kernel<__half>, a);
  return launch_with(attr, grid, kPairThreads, s, preference_kernel<float>, a);
}

}  // namespace flce
