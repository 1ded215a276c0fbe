// Losses over per-token log-probabilities of packed sequences, with their
// gradients: the clipped policy loss with a KL term, and the preference loss
// over pairs of sequences.
//
// Tokens lie in one array; sequence s is [cu[s], cu[s+1]). A thread block takes
// SEQ_CHUNK consecutive tokens, whatever sequences they belong to, so ragged
// lengths leave no block idle and a long sequence is spread over many blocks.
// Where a sum per sequence is needed, block b writes its part of sequence s
// to slot b + s: walking along the tokens either the block or the sequence
// advances, so no two pairs (b, s) share a slot and blocks + sequences slots
// hold them all. Sums are joined in a fixed order (no floating-point atomics):
// the results do not change from run to run.
//
// What bounds both on long batches: DRAM (21 bytes a token for the policy loss
// with per-token advantages, 13 for the preference loss, whose gradient pass
// reads the mask once more). On short ones: the launches.
#include <cuda_bf16.h>
#include <math.h>
#include <stdint.h>

#include "kdkl_internal.h"
#include "tc_primitives.cuh"

namespace kdkl {

namespace {

constexpr int SEQ_THREADS = 256;
constexpr int SEQ_TOK = 8;  // consecutive tokens per thread
constexpr int SEQ_CHUNK = SEQ_THREADS * SEQ_TOK;

// First sequence in [lo, lo + n) whose end is past token t (the last one if
// none is), found by the whole warp: 32 probes a step.
__device__ __forceinline__ int seq_find_warp(const int32_t* cu, int lo, int n, int t) {
  const int lane = threadIdx.x & 31;
  const int last = lo + n - 1;
  const int end = lo + n;
  while (n > 0) {
    const int step = (n + 31) / 32;
    const int i = lo + lane * step + step - 1;
    const bool before = i < end && i < lo + n && __ldg(cu + i + 1) <= t;
    lo += __popc(__ballot_sync(0xffffffffu, before)) * step;
    n = min(step - 1, end - lo);
  }
  return min(lo, last);
}

// The same by one thread.
__device__ __forceinline__ int seq_find(const int32_t* cu, int lo, int last, int t) {
  while (lo < last) {
    const int mid = (lo + last) >> 1;
    if (__ldg(cu + mid + 1) <= t) lo = mid + 1; else last = mid;
  }
  return lo;
}

// Sequences of the block's first and last token, to every thread.
__device__ __forceinline__ void block_range(const int32_t* cu, int S, int t0, int t1, int* range,
                                            int& s_lo, int& s_hi) {
  const int warp = threadIdx.x >> 5;
  if (warp < 2) {
    const int s = seq_find_warp(cu, 0, S, warp == 0 ? t0 : t1 - 1);
    if ((threadIdx.x & 31) == 0) range[warp] = s;
  }
  __syncthreads();
  s_lo = range[0];
  s_hi = max(range[0], range[1]);
}

// Eight consecutive values from token t on; those at or past T read as zero.
__device__ __forceinline__ void load_f8(const float* p, int t, int T, bool vec,
                                        float (&x)[SEQ_TOK]) {
  if (vec && t + SEQ_TOK <= T) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p + t));
    const float4 b = __ldg(reinterpret_cast<const float4*>(p + t) + 1);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  } else {
#pragma unroll
    for (int j = 0; j < SEQ_TOK; ++j) x[j] = t + j < T ? __ldg(p + t + j) : 0.f;
  }
}

__device__ __forceinline__ void store_f8(float* p, int t, int T, bool vec,
                                         const float (&x)[SEQ_TOK]) {
  if (vec && t + SEQ_TOK <= T) {
    *reinterpret_cast<float4*>(p + t) = make_float4(x[0], x[1], x[2], x[3]);
    *(reinterpret_cast<float4*>(p + t) + 1) = make_float4(x[4], x[5], x[6], x[7]);
  } else {
#pragma unroll
    for (int j = 0; j < SEQ_TOK; ++j)
      if (t + j < T) p[t + j] = x[j];
  }
}

// Bit j: token t + j exists and counts.
__device__ __forceinline__ uint32_t load_mask8(const uint8_t* mask, int t, int T, bool vec) {
  uint32_t on = 0;
  if (mask == nullptr) {
#pragma unroll
    for (int j = 0; j < SEQ_TOK; ++j) on |= (t + j < T ? 1u : 0u) << j;
  } else if (vec && t + SEQ_TOK <= T) {
    const uint2 w = __ldg(reinterpret_cast<const uint2*>(mask + t));
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      on |= ((w.x >> (8 * j)) & 0xffu ? 1u : 0u) << j;
      on |= ((w.y >> (8 * j)) & 0xffu ? 1u : 0u) << (4 + j);
    }
  } else {
#pragma unroll
    for (int j = 0; j < SEQ_TOK; ++j) on |= (t + j < T && __ldg(mask + t + j) != 0 ? 1u : 0u) << j;
  }
  return on;
}

template <typename T>
__device__ __forceinline__ T warp_sum(T v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sum over the block in a fixed order, valid in thread 0.
template <typename T>
__device__ __forceinline__ T block_sum(T v, T* part) {
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  T r = 0;
  if (threadIdx.x == 0)
    for (int i = 0; i < (int)blockDim.x / 32; ++i) r += part[i];
  __syncthreads();
  return r;
}

// True in every thread of the block that finishes last.
__device__ __forceinline__ bool last_block(int* ticket, int* flag) {
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) *flag = atomicAdd(ticket, 1) == (int)gridDim.x - 1;
  __syncthreads();
  if (*flag) __threadfence();
  return *flag != 0;
}

// cu must start at 0, end at T and never fall.
__device__ __forceinline__ void check_cu(const int32_t* cu, int S, int T, int* status) {
  const long long stride = (long long)gridDim.x * blockDim.x;
  for (long long s = (long long)blockIdx.x * blockDim.x + threadIdx.x; s < S; s += stride) {
    const int a = __ldg(cu + s), b = __ldg(cu + s + 1);
    if (a > b || (s == 0 && a != 0) || (s == S - 1 && b != T))
      record_error(status, DEV_ERR_INVALID_ARG);
  }
}

// --------------------------------------------------------------- policy loss

// Counted tokens: of all (n_seq == nullptr) into n_count[0], or of every
// sequence into n_seq[s], and then into n_count[1] how many have any. Whole
// numbers, so atomics give the same answer in any order.
__global__ void __launch_bounds__(SEQ_THREADS)
    policy_count_kernel(const uint8_t* __restrict__ mask, const int32_t* __restrict__ cu, int T,
                        int S, int vec, int* __restrict__ n_seq, int* __restrict__ n_count,
                        int* __restrict__ ticket) {
  __shared__ int range[2], part[SEQ_THREADS / 32], flag;
  const int t0 = blockIdx.x * SEQ_CHUNK;
  const int t1 = min(T, t0 + SEQ_CHUNK);
  const int t = t0 + threadIdx.x * SEQ_TOK;
  const uint32_t on = load_mask8(mask, t, T, vec != 0);
  const int all = block_sum(__popc(on), part);
  if (threadIdx.x == 0 && all) atomicAdd(n_count, all);
  if (n_seq == nullptr) return;
  int s_lo, s_hi;
  block_range(cu, S, t0, t1, range, s_lo, s_hi);
  if (s_lo == s_hi) {
    if (threadIdx.x == 0 && all) atomicAdd(n_seq + s_lo, all);
  } else if (t < t1) {
    int s = seq_find(cu, s_lo, s_hi, t);
    int run = 0;
#pragma unroll
    for (int j = 0; j < SEQ_TOK; ++j) {
      while (s < s_hi && t + j >= __ldg(cu + s + 1)) {
        if (run) atomicAdd(n_seq + s, run);
        run = 0;
        ++s;
      }
      run += (on >> j) & 1u;
    }
    if (run) atomicAdd(n_seq + s, run);
  }
  if (!last_block(ticket, &flag)) return;
  int any = 0;
  for (int s = threadIdx.x; s < S; s += SEQ_THREADS) any += __ldcg(n_seq + s) > 0 ? 1 : 0;
  any = block_sum(any, part);
  if (threadIdx.x == 0) n_count[1] = any;
}

// a - b against a border that takes 64 bits: the difference of two floats is
// the rounded one plus an error that is a float too, and the border is held
// the same way, as a float and a remainder.
__device__ __forceinline__ bool exceeds(float d, float e, float hi, float lo) {
  return d > hi || (d == hi && e > lo);
}

// e^x - 1 - x without its cancellation near 0: for |x| < 1 the power series
// x^2 (1/2! + x/3! + ... + x^10/12!), whose next term is below 2^-29 of the sum.
__device__ __forceinline__ float exp_rest(float x) {
  if (fabsf(x) < 1.f) {
    float p = 1.f / 479001600.f;
    p = fmaf(p, x, 1.f / 39916800.f);
    p = fmaf(p, x, 1.f / 3628800.f);
    p = fmaf(p, x, 1.f / 362880.f);
    p = fmaf(p, x, 1.f / 40320.f);
    p = fmaf(p, x, 1.f / 5040.f);
    p = fmaf(p, x, 1.f / 720.f);
    p = fmaf(p, x, 1.f / 120.f);
    p = fmaf(p, x, 1.f / 24.f);
    p = fmaf(p, x, 1.f / 6.f);
    p = fmaf(p, x, 0.5f);
    return p * x * x;
  }
  return (expf(x) - 1.f) - x;
}

// One pass over the tokens: ratio, clip, KL term, gradient, and per block the
// weighted sums of the two parts of the loss and the number of clipped tokens;
// the block that finishes last joins the blocks' sums.
//   NEED_SEQ: a token's sequence is looked up (advantages or weights per sequence).
template <bool NEED_SEQ>
__global__ void __launch_bounds__(SEQ_THREADS)
    policy_loss_kernel(const PolicyArgs a, int* status) {
  __shared__ int range[2], ipart[SEQ_THREADS / 32], flag;
  __shared__ double part[SEQ_THREADS / 32];
  const int t0 = blockIdx.x * SEQ_CHUNK;
  const int t1 = min(a.T, t0 + SEQ_CHUNK);
  const int t = t0 + threadIdx.x * SEQ_TOK;
  const bool vec = a.vec != 0;
  const uint32_t on = load_mask8(a.mask, t, a.T, vec);
  float lp[SEQ_TOK], lo[SEQ_TOK], lr[SEQ_TOK], adv[SEQ_TOK];
  load_f8(a.logp, t, a.T, vec, lp);
  if (a.old_logp) load_f8(a.old_logp, t, a.T, vec, lo);
  if (a.ref_logp) load_f8(a.ref_logp, t, a.T, vec, lr);
  if (!a.adv_per_seq) load_f8(a.advantages, t, a.T, vec, adv);

  int s = 0, s_hi = 0;
  if (NEED_SEQ) {
    check_cu(a.cu, a.S, a.T, status);
    int s_lo;
    block_range(a.cu, a.S, t0, t1, range, s_lo, s_hi);
    s = t < t1 ? seq_find(a.cu, s_lo, s_hi, t) : s_hi;
  }
  // Counted tokens: given (no mask), counted before, or counted here by every
  // block for itself (a short mask, which saves the launch that would count it).
  int n = a.T;
  if (a.mask) {
    if (a.count_here) {
      int c = 0;
      for (int i = threadIdx.x * SEQ_TOK; i < a.T; i += SEQ_CHUNK)
        c += __popc(load_mask8(a.mask, i, a.T, vec));
      c = block_sum(c, ipart);
      if (threadIdx.x == 0) range[0] = c;
      __syncthreads();
      n = range[0];
    } else {
      n = *a.n_count;
    }
  }
  const int n_any = a.reduction == 1 ? a.n_count[1] : 0;
  float w = a.reduction == 0 ? (n > 0 ? 1.f / (float)n : 0.f) : a.inv_norm;
  float w_adv = 0.f;  // the sequence's advantage
  auto enter = [&]() {  // the sequence's values
    if (a.adv_per_seq) w_adv = __ldg(a.advantages + s);
    if (a.reduction == 1) {
      const int ns = __ldg(a.n_seq + s);
      w = ns > 0 ? 1.f / ((float)ns * (float)n_any) : 0.f;
    }
  };
  if (NEED_SEQ) enter();

  float g[SEQ_TOK];
  float pg = 0.f, kl = 0.f;
  int clipped = 0;
#pragma unroll
  for (int j = 0; j < SEQ_TOK; ++j) {
    if (NEED_SEQ) {
      bool moved = false;
      while (s < s_hi && t + j >= __ldg(a.cu + s + 1)) {
        ++s;
        moved = true;
      }
      if (moved) enter();
    }
    g[j] = 0.f;
    if ((on >> j) & 1u) {  // what lies under the mask is never used
      const float A = a.adv_per_seq ? w_adv : adv[j];
      float d = 0.f, e = 0.f;
      if (a.old_logp) {
        d = lp[j] - lo[j];
        const float bb = d - lp[j];
        e = (lp[j] - (d - bb)) - (lo[j] + bb);
      }
      const bool pos = A >= 0.f;
      float bound = pos ? a.r_high : a.r_low;
      bool clip = pos ? exceeds(d, e, a.high_hi, a.high_lo)
                      : exceeds(-d, -e, -a.low_hi, -a.low_lo);
      if (a.dual && !pos && exceeds(d, e, a.dual_hi, a.dual_lo)) {
        clip = true;
        bound = a.r_dual;
      }
      const float r = clip ? bound : expf(d);
      pg = fmaf(-w * r, A, pg);
      float gj = clip ? 0.f : -r * A;
      if (a.ref_logp) {
        const float x = lr[j] - lp[j];
        const float k = exp_rest(x);
        kl = fmaf(w, k, kl);
        gj -= a.kl_coef * (x + k);
      }
      g[j] = w * gj * a.grad_loss;
      clipped += clip ? 1 : 0;
    }
  }
  if (a.grad && t < t1) store_f8(a.grad, t, a.T, vec, g);

  const double spg = block_sum((double)pg, part);
  const double skl = block_sum((double)kl, part);
  const int scl = block_sum(clipped, ipart);
  if (threadIdx.x == 0) {
    a.block_part[3 * (long long)blockIdx.x] = spg;
    a.block_part[3 * (long long)blockIdx.x + 1] = skl;
    a.block_part[3 * (long long)blockIdx.x + 2] = (double)scl;
  }
  if (!last_block(a.ticket, &flag)) return;
  double v[3] = {0.0, 0.0, 0.0};
  for (int b = threadIdx.x; b < (int)gridDim.x; b += SEQ_THREADS)
#pragma unroll
    for (int q = 0; q < 3; ++q) v[q] += __ldcg(a.block_part + 3 * (long long)b + q);
#pragma unroll
  for (int q = 0; q < 3; ++q) v[q] = block_sum(v[q], part);
  if (threadIdx.x == 0) {
    a.loss[0] = (float)(v[0] + (double)a.kl_coef * v[1]);
    if (a.stats) {
      a.stats[0] = (float)v[0];
      a.stats[1] = (float)v[1];
      a.stats[2] = n > 0 ? (float)(v[2] / (double)n) : 0.f;
    }
  }
}

// ----------------------------------------------------------- preference loss

// Block b's part of every sequence s that it meets, to slot b + s: the sum of
// the counted tokens' log ratios, and how many they are.
__global__ void __launch_bounds__(SEQ_THREADS)
    pref_sums_kernel(const float* __restrict__ logp, const float* __restrict__ ref,
                     const uint8_t* __restrict__ mask, const int32_t* __restrict__ cu, int T, int S,
                     int vec, double* __restrict__ slot_sum, int* __restrict__ slot_n,
                     int* __restrict__ status) {
  __shared__ int range[2], ipart[SEQ_THREADS / 32];
  __shared__ double part[SEQ_THREADS / 32];
  __shared__ float gap[SEQ_CHUNK];
  __shared__ uint8_t cnt[SEQ_CHUNK];
  const int t0 = blockIdx.x * SEQ_CHUNK;
  const int t1 = min(T, t0 + SEQ_CHUNK);
  const int t = t0 + threadIdx.x * SEQ_TOK;
  const uint32_t on = load_mask8(mask, t, T, vec != 0);
  float x[SEQ_TOK], y[SEQ_TOK];
  load_f8(logp, t, T, vec != 0, x);
  if (ref) load_f8(ref, t, T, vec != 0, y);
  check_cu(cu, S, T, status);
  int s_lo, s_hi;
  block_range(cu, S, t0, t1, range, s_lo, s_hi);
#pragma unroll
  for (int j = 0; j < SEQ_TOK; ++j)
    x[j] = (on >> j) & 1u ? (ref ? x[j] - y[j] : x[j]) : 0.f;
  if (s_lo == s_hi) {
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < SEQ_TOK; ++j) sum += x[j];
    const double all = block_sum((double)sum, part);
    const int n = block_sum(__popc(on), ipart);
    if (threadIdx.x == 0) {
      slot_sum[(long long)blockIdx.x + s_lo] = all;
      slot_n[(long long)blockIdx.x + s_lo] = n;
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < SEQ_TOK; ++j) {
    gap[threadIdx.x * SEQ_TOK + j] = x[j];
    cnt[threadIdx.x * SEQ_TOK + j] = (uint8_t)((on >> j) & 1u);
  }
  __syncthreads();
  // a warp per sequence, its lanes across the sequence's tokens
  const int lane = threadIdx.x & 31;
  for (int s = s_lo + (threadIdx.x >> 5); s <= s_hi; s += SEQ_THREADS / 32) {
    const int a = max(__ldg(cu + s), t0) - t0, b = min(__ldg(cu + s + 1), t1) - t0;
    float sum = 0.f;
    int n = 0;
    for (int i = a + lane; i < b; i += 32) {
      sum += gap[i];
      n += cnt[i];
    }
    const double all = warp_sum((double)sum);
    n = warp_sum(n);
    if (lane == 0) {
      slot_sum[(long long)blockIdx.x + s] = all;
      slot_n[(long long)blockIdx.x + s] = n;
    }
  }
}

// A warp per pair: both sequences' sums from their slots, the pair's loss, and
// the gradient that each counted token of either sequence gets.
__global__ void __launch_bounds__(SEQ_THREADS) pref_pairs_kernel(const PrefArgs a) {
  __shared__ int flag;
  __shared__ double part[SEQ_THREADS / 32];
  const int lane = threadIdx.x & 31;
  const int i = blockIdx.x * (SEQ_THREADS / 32) + (threadIdx.x >> 5);
  if (i < a.P) {
    int seq[2] = {a.halves ? i : 2 * i, a.halves ? a.P + i : 2 * i + 1};
    double ratio[2], share[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int s = seq[k];
      const int c0 = max(0, min(a.T, __ldg(a.cu + s))), c1 = max(0, min(a.T, __ldg(a.cu + s + 1)));
      double sum = 0.0;
      int n = 0;
      if (c1 > c0)
        for (int b = c0 / SEQ_CHUNK + lane; b <= (c1 - 1) / SEQ_CHUNK; b += 32) {
          sum += a.slot_sum[(long long)b + s];
          n += a.slot_n[(long long)b + s];
        }
      sum = warp_sum(sum);
      n = warp_sum(n);
      share[k] = a.average ? 1.0 / (double)max(n, 1) : 1.0;
      ratio[k] = sum * share[k];
    }
    if (lane == 0) {
      const double h = ratio[0] - ratio[1] - a.margin;
      const double b = a.beta * h, eps = a.label_smoothing;
      double each, slope;
      if (a.kind == 0) {
        // -log sigma(b) = log(1 + e^-|b|) + max(-b, 0); its mirror for -b
        const double soft = log1p(exp(-fabs(b)));
        each = (1.0 - eps) * (soft + fmax(-b, 0.0)) + eps * (soft + fmax(b, 0.0));
        slope = a.beta * (eps - 1.0 / (1.0 + exp(b)));
      } else if (a.kind == 1) {
        const double off = h - 0.5 / a.beta;
        each = off * off;
        slope = 2.0 * off;
      } else {
        each = fmax(1.0 - b, 0.0);
        slope = b < 1.0 ? -a.beta : 0.0;
      }
      if (b != b) each = slope = b;  // fmax drops a NaN
      a.pair_loss[i] = each;
      a.rewards[2 * i] = (float)(a.beta * ratio[0]);
      a.rewards[2 * i + 1] = (float)(a.beta * ratio[1]);
      slope *= a.grad_loss / (double)a.P;
      a.coef[seq[0]] = (float)(slope * share[0]);
      a.coef[seq[1]] = (float)(-slope * share[1]);
    }
  }
  if (!last_block(a.ticket, &flag)) return;
  double v = 0.0;
  for (int p = threadIdx.x; p < a.P; p += SEQ_THREADS) v += __ldcg(a.pair_loss + p);
  v = block_sum(v, part);
  if (threadIdx.x == 0) a.loss[0] = (float)(v / (double)a.P);
}

__global__ void __launch_bounds__(SEQ_THREADS)
    pref_grad_kernel(const uint8_t* __restrict__ mask, const int32_t* __restrict__ cu,
                     const float* __restrict__ coef, int T, int S, int vec,
                     float* __restrict__ grad) {
  __shared__ int range[2];
  const int t0 = blockIdx.x * SEQ_CHUNK;
  const int t1 = min(T, t0 + SEQ_CHUNK);
  const int t = t0 + threadIdx.x * SEQ_TOK;
  const uint32_t on = load_mask8(mask, t, T, vec != 0);
  int s_lo, s_hi;
  block_range(cu, S, t0, t1, range, s_lo, s_hi);
  if (t >= t1) return;
  int s = seq_find(cu, s_lo, s_hi, t);
  float c = __ldg(coef + s);
  float g[SEQ_TOK];
#pragma unroll
  for (int j = 0; j < SEQ_TOK; ++j) {
    bool moved = false;
    while (s < s_hi && t + j >= __ldg(cu + s + 1)) {
      ++s;
      moved = true;
    }
    if (moved) c = __ldg(coef + s);
    g[j] = (on >> j) & 1u ? c : 0.f;
  }
  store_f8(grad, t, T, vec != 0, g);
}

}  // namespace

int seq_blocks(int T) { return (T + SEQ_CHUNK - 1) / SEQ_CHUNK; }

cudaError_t launch_policy_loss(const PolicyArgs& a, int* status, cudaStream_t stream) {
  const bool per_seq = a.reduction == 1;
  const dim3 grid((unsigned)seq_blocks(a.T)), block(SEQ_THREADS);
  if (per_seq || (a.mask && !a.count_here)) {
    const cudaError_t e =
        launch_kernel("policy_count", policy_count_kernel, grid, block, 0, stream, a.mask, a.cu,
                      a.T, a.S, a.vec, per_seq ? a.n_seq : nullptr, a.n_count, a.ticket + 1);
    if (e != cudaSuccess) return e;
  }
  if (per_seq || a.adv_per_seq)
    return launch_kernel("policy_loss", policy_loss_kernel<true>, grid, block, 0, stream, a,
                         status);
  return launch_kernel("policy_loss", policy_loss_kernel<false>, grid, block, 0, stream, a, status);
}

cudaError_t launch_pref_loss(const PrefArgs& a, int* status, cudaStream_t stream) {
  const dim3 grid((unsigned)seq_blocks(a.T)), block(SEQ_THREADS);
  cudaError_t e;
  if (a.T > 0) {
    e = launch_kernel("pref_sums", pref_sums_kernel, grid, block, 0, stream, a.logp, a.ref_logp,
                      a.mask, a.cu, a.T, 2 * a.P, a.vec, a.slot_sum, a.slot_n, status);
    if (e != cudaSuccess) return e;
  }
  const int warps = SEQ_THREADS / 32;
  e = launch_kernel("pref_pairs", pref_pairs_kernel, dim3((unsigned)((a.P + warps - 1) / warps)),
                    block, 0, stream, a);
  if (e != cudaSuccess || !a.grad || a.T == 0) return e;
  return launch_kernel("pref_grad", pref_grad_kernel, grid, block, 0, stream, a.mask, a.cu, a.coef,
                       a.T, 2 * a.P, a.vec, a.grad);
}

}  // namespace kdkl
