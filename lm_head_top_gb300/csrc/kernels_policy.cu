// Losses over per-token log-probabilities of packed sequences, with their
// gradients: the clipped policy loss with a KL term, and the preference loss
// over pairs of sequences.
//
// Tokens lie in one array; sequence s is [cu[s], cu[s+1]). The unit of work is a
// warp and a run of consecutive tokens, whatever sequences they belong to:
// ragged lengths leave no warp idle and a long sequence is spread over many. A
// warp walks its run in pieces of 128 tokens, four per lane, and keeps its
// place among the sequences as it goes, so that finding a token's sequence costs
// one search per run. Nothing in the walk waits for the other warps of the block.
// Where a sum per sequence is needed, warp w writes its part of sequence s to
// slot w + s: along the tokens either the warp or the sequence advances, so no
// two pairs (w, s) share a slot, and warps + sequences slots hold them all. Sums
// are joined in a fixed order (no floating-point atomics): the results do not
// change from run to run.
//
// What bounds them. Their bytes are 17 a token for the policy loss with an
// advantage per sequence (21 with one per token) and 13 for the preference loss,
// whose gradient pass reads the mask once more. On short batches it is the
// launches: a batch that one block can hold takes one. In between it is chains of
// dependent lookups, joins and starts, about 10 us a launch. On 8.4M tokens the
// policy loss takes 38 us after a count of 9 (21 at the copy rate): about 95
// instructions a token. Not the lever there: 128 or 256 tokens a piece, 16 to 40
// warps an SM, runs by block instead of by warp, the next piece prefetched to L2
// or to registers, arithmetic without branches; each measured within 10 %.
#include <cuda_bf16.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "kdkl_internal.h"
#include "tc_primitives.cuh"

namespace kdkl {

namespace {

constexpr int SEQ_THREADS = 512;
constexpr int SEQ_WARPS = SEQ_THREADS / 32;
constexpr int SEQ_TOK = 4;              // consecutive tokens per lane: a 16-byte load
constexpr int SEQ_PIECE = 32 * SEQ_TOK;  // tokens of a warp's step
constexpr int SEQ_RESIDENT = 2;          // blocks of a walk on an SM
constexpr int RING_STAGES = 2;
constexpr int RING_BYTES = 4 * SEQ_PIECE * 4 + SEQ_PIECE;  // a piece of four arrays and the mask
constexpr int PREF_ONE_THREADS = 512;    // the one-block preference loss

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

// First sequence from s on whose end is past token t (the last one if none
// is), by one thread: steps that double, then bisection.
__device__ __noinline__ int seq_advance(const int32_t* cu, int S, int s, int t) {
  if (s >= S - 1 || __ldg(cu + s + 1) > t) return min(s, S - 1);
  int lo = s + 1, step = 1;
  while (lo + step < S && __ldg(cu + lo + step) <= t) {
    lo += step;
    step <<= 1;
  }
  int last = min(lo + step - 1, S - 1);
  while (lo < last) {
    const int mid = (lo + last) >> 1;
    if (__ldg(cu + mid + 1) <= t) lo = mid + 1; else last = mid;
  }
  return lo;
}

// A lane's consecutive values from token t on. whole: aligned, and all of them
// exist; else those at or past T read as zero.
__device__ __forceinline__ void load_tok(const float* p, int t, int T, bool whole,
                                         float (&x)[SEQ_TOK]) {
  if (whole) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p + t));
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  } else {
#pragma unroll
    for (int j = 0; j < SEQ_TOK; ++j) x[j] = t + j < T ? __ldg(p + t + j) : 0.f;
  }
}

__device__ __forceinline__ void store_tok(float* p, int t, int T, bool whole,
                                          const float (&x)[SEQ_TOK]) {
  if (whole) {
    *reinterpret_cast<float4*>(p + t) = make_float4(x[0], x[1], x[2], x[3]);
  } else {
#pragma unroll
    for (int j = 0; j < SEQ_TOK; ++j)
      if (t + j < T) p[t + j] = x[j];
  }
}

// Bit j: byte j of the word is not zero. Each byte's bits are folded onto its
// lowest (what a shift brings in from the byte above lands on bits not used
// again), and a product brings the four lowest bits together.
__device__ __forceinline__ uint32_t nonzero_bytes(uint32_t x) {
  x |= x >> 4;
  x |= x >> 2;
  x |= x >> 1;
  return ((x & 0x01010101u) * 0x10204080u) >> 28;
}

// Bit j: token t + j exists and counts, for a lane's tokens.
__device__ __forceinline__ uint32_t load_mask(const uint8_t* mask, int t, int T, bool vec) {
  if (mask == nullptr)
    return t + SEQ_TOK <= T ? (1u << SEQ_TOK) - 1u : t < T ? (1u << (T - t)) - 1u : 0u;
  if (vec && t + SEQ_TOK <= T)
    return nonzero_bytes(__ldg(reinterpret_cast<const uint32_t*>(mask + t)));
  uint32_t on = 0;
#pragma unroll 1
  for (int j = 0; j < SEQ_TOK && t + j < T; ++j) on |= (__ldg(mask + t + j) != 0 ? 1u : 0u) << j;
  return on;
}

// The same for 16 tokens.
__device__ __forceinline__ uint32_t load_mask16(const uint8_t* mask, int t, int T, bool vec) {
  if (mask && vec && t + 16 <= T) {
    const uint4 w = __ldg(reinterpret_cast<const uint4*>(mask + t));
    return nonzero_bytes(w.x) | nonzero_bytes(w.y) << 4 | nonzero_bytes(w.z) << 8 |
           nonzero_bytes(w.w) << 12;
  }
  uint32_t on = 0;
#pragma unroll
  for (int k = 0; k < 16; k += SEQ_TOK) on |= load_mask(mask, t + k, T, vec) << k;
  return on;
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

// A sum in two floats: each addition's rounding error is kept, 48 bits in all.
// The fp64 unit here takes 16 cycles for a warp's addition: joining the warps'
// sums in fp64 alone cost the policy loss 4 us whatever its length.
struct Sum2 {
  float hi = 0.f, lo = 0.f;
  __device__ __forceinline__ void add(float x, float x_lo = 0.f) {
    const float t = hi + x, b = t - hi;
    lo += ((hi - (t - b)) + (x - b)) + x_lo;
    hi = t;
  }
  // (an infinite sum has no error term)
  __device__ __forceinline__ float value() const { return lo == lo ? hi + lo : hi; }
};

// Lane 0 has the warp's sum, in a fixed order.
__device__ __forceinline__ Sum2 warp_sum(Sum2 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float hi = __shfl_down_sync(0xffffffffu, v.hi, o);
    const float lo = __shfl_down_sync(0xffffffffu, v.lo, o);
    v.add(hi, lo);
  }
  return v;
}

// Tokens of one warp's run when `warps` of them share T tokens.
__host__ __device__ __forceinline__ int run_length(int T, int warps) {
  return (int)(((long long)T + (long long)warps * SEQ_PIECE - 1) /
               ((long long)warps * SEQ_PIECE)) * SEQ_PIECE;
}

// Copies to shared memory that the thread waits for by groups.
__device__ __forceinline__ void copy_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int LEFT>
__device__ __forceinline__ void copy_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}
__device__ __forceinline__ uint32_t ld_shared_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// --------------------------------------------------------------- policy loss

// Counted tokens: of all into n_count[0]; with n_seq, of every sequence into
// n_seq[s], and how many sequences have any into n_count[1] (whoever finds a
// sequence's count at zero counts it). Whole numbers, so atomics give the same
// answer in any order.
__global__ void __launch_bounds__(SEQ_THREADS)
    policy_count_kernel(const uint8_t* __restrict__ mask, const int32_t* __restrict__ cu, int T,
                        int S, int vec, int* __restrict__ n_seq, int* __restrict__ n_count) {
  __shared__ int block_count;
  grid_dependents_go();
  if (threadIdx.x == 0) block_count = 0;
  __syncthreads();
  const int lane = threadIdx.x & 31;
  constexpr int TOK = 16, PIECE = 32 * TOK;  // per lane and step here
  const int R = (run_length(T, (int)gridDim.x * SEQ_WARPS) + PIECE - 1) / PIECE * PIECE;
  const long long first = (long long)(blockIdx.x * SEQ_WARPS + (threadIdx.x >> 5)) * R;
  const int run_end = (int)min((long long)T, first + R);
  // the whole run's mask is on its way while the first sequence is looked for
  if (mask)
    for (long long i = first + lane * 128; i < run_end; i += 32 * 128) prefetch_l2(mask + i);
  auto put = [&](int s, int c) {
    if (c && atomicAdd(n_seq + s, c) == 0) atomicAdd(n_count + 1, 1);
  };
  int total = 0;
  int s = 0, end = -1;
  int held = 0, count = 0;  // a sequence's count not put yet
  if (n_seq && first < T) s = seq_find_warp(cu, 0, S, (int)first);
  for (int p = (int)min((long long)T, first); p < run_end; p += PIECE) {
    const int t = p + lane * TOK;
    const uint32_t on = load_mask16(mask, t, T, vec != 0);
    const int c = __popc(on);
    total += c;
    if (n_seq == nullptr) continue;
    if (t < run_end && t >= end) {
      s = seq_advance(cu, S, s, t);
      end = s < S - 1 ? __ldg(cu + s + 1) : T;
    }
    const int s0 = __shfl_sync(0xffffffffu, s, 0);
    if (__all_sync(0xffffffffu, t >= run_end || (s == s0 && min(t + TOK, T) <= end))) {
      // the whole piece in one sequence: its count waits for the sequence's end
      // (4 sequences of 2M tokens: 14 us with an atomic a piece, 8 so)
      if (s0 != held) {
        if (lane == 0) put(held, count);
        held = s0;
        count = 0;
      }
      count += __reduce_add_sync(0xffffffffu, c);
    } else if (t < run_end) {
      int at = 0;  // the lane's tokens from here on are not put yet
      while (end < t + TOK && s < S - 1) {
        const int upto = max(at, end - t);
        put(s, __popc(on & ((1u << upto) - 1u) & ~((1u << at) - 1u)));
        at = upto;
        if (t + at >= T) break;
        s = seq_advance(cu, S, s, t + at);
        end = s < S - 1 ? __ldg(cu + s + 1) : T;
      }
      put(s, __popc(on & ~((1u << at) - 1u)));
    }
  }
  if (n_seq && lane == 0) put(held, count);
  total = __reduce_add_sync(0xffffffffu, total);
  if (lane == 0 && total) atomicAdd(&block_count, total);
  __syncthreads();
  if (threadIdx.x == 0 && block_count) atomicAdd(n_count, block_count);
}

// Whether p - q exceeds a border that takes 64 bits. d is the difference
// rounded to a float, the border a float and a remainder. Rounding is monotone,
// so d decides unless it is the border's own float (hardly ever): then the
// rounding error of d, which is a float too, is held against the remainder.
__device__ __forceinline__ bool exceeds(float d, float p, float q, float hi, float lo) {
  bool over = d > hi;
  if (d == hi) {
    const float b = d - p;
    over = (p - (d - b)) - (q + b) > lo;
  }
  return over;
}

// e^x by the hardware's base-2 exponential: 2 ulp and the rounding of x log2(e).
__device__ __forceinline__ float exp_fast(float x) { return ex2_approx(x * 1.4426950408889634f); }

// e^x - 1 - x without its cancellation near 0: for |x| < 0.35 the power series
// x^2 (1/2! + x/3! + ... + x^6/8!), whose next term is below 2^-27 of the sum.
__device__ __forceinline__ float exp_rest(float x) {
  float p = 1.f / 40320.f;
  p = fmaf(p, x, 1.f / 5040.f);
  p = fmaf(p, x, 1.f / 720.f);
  p = fmaf(p, x, 1.f / 120.f);
  p = fmaf(p, x, 1.f / 24.f);
  p = fmaf(p, x, 1.f / 6.f);
  p = fmaf(p, x, 0.5f);
  const float far = (exp_fast(x) - 1.f) - x;
  return fabsf(x) < 0.35f ? p * x * x : far;
}

// One pass over the tokens: ratio, clip, KL term, gradient, and per block the
// weighted sums of the two parts of the loss and the number of clipped tokens;
// the block that finishes last joins the blocks' sums.
//   NEED_SEQ: a token's sequence is looked up (advantages or weights per sequence).
//   RING: pieces come through shared memory, one ahead of the arithmetic, each
//   lane copying what it will read itself (no barrier). For runs of several
//   pieces and aligned arrays: loads waited for in registers were half of the
//   stalls, and registers for the next piece do not fit beside this one's (the
//   loss of 8.4M tokens 42 -> 38 us; two ahead the same).
template <bool NEED_SEQ, bool RING>
__global__ void __launch_bounds__(SEQ_THREADS, SEQ_RESIDENT)
    policy_loss_kernel(const PolicyArgs a, int* status) {
  __shared__ int count, any, clips;
  __shared__ float2 part[2][SEQ_WARPS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool alone = gridDim.x == 1;
  const bool vec = a.vec != 0;
  if (threadIdx.x == 0) {
    count = any = clips = 0;
    if (alone) *status = 0;  // with more blocks the call has cleared it
  }
  __syncthreads();
  const int R = run_length(a.T, (int)gridDim.x * SEQ_WARPS);
  const long long first = (long long)(blockIdx.x * SEQ_WARPS + warp) * R;
  const int begin = (int)min((long long)a.T, first);
  const int run_end = (int)min((long long)a.T, first + R);

  extern __shared__ __align__(16) unsigned char ring_mem[];
  const uint32_t ring = smem_u32(ring_mem) + warp * (RING_STAGES * RING_BYTES);
  auto copy_ahead = [&](int t, int stage) {
    if (t + SEQ_TOK <= run_end) {  // (a run ends at T or at a piece's end)
      const uint32_t d = ring + stage * RING_BYTES + lane * 16;
      copy_async16(d, a.logp + t);
      if (a.old_logp) copy_async16(d + 512, a.old_logp + t);
      if (a.ref_logp) copy_async16(d + 1024, a.ref_logp + t);
      if (!a.adv_per_seq) copy_async16(d + 1536, a.advantages + t);
      if (a.mask) copy_async4(ring + stage * RING_BYTES + 2048 + lane * 4, a.mask + t);
    }
    copy_async_commit();
  };
  auto read4 = [](uint32_t addr, float (&x)[SEQ_TOK]) {
    const uint4 v = ld_shared_v4(addr);
    x[0] = __uint_as_float(v.x);
    x[1] = __uint_as_float(v.y);
    x[2] = __uint_as_float(v.z);
    x[3] = __uint_as_float(v.w);
  };
  int stage = 0;
  // the first pieces are on their way during the lookups
  if (RING) {
    for (int k = 0; k < RING_STAGES - 1; ++k)
      copy_ahead(begin + lane * SEQ_TOK + k * SEQ_PIECE, k);
  } else if (lane < 8 && begin + lane * 32 < run_end) {
    prefetch_l2(a.logp + begin + lane * 32);
    if (a.old_logp) prefetch_l2(a.old_logp + begin + lane * 32);
    if (a.ref_logp) prefetch_l2(a.ref_logp + begin + lane * 32);
  }
  int s = 0, end = a.T;
  if (NEED_SEQ && begin < run_end) s = seq_find_warp(a.cu, 0, a.S, begin);
  grid_dependency_wait();  // the counts, and the cleared status
  if (NEED_SEQ) check_cu(a.cu, a.S, a.T, status);
  // Counted tokens: given (no mask), counted before, or counted here by every
  // block for itself (a short mask, which saves the launch that would count it).
  int n = a.T;
  if (a.mask && a.count_here) {
    int c = 0;
    for (int i = threadIdx.x * 16; i < a.T; i += SEQ_THREADS * 16)
      c += __popc(load_mask16(a.mask, i, a.T, vec));
    c = __reduce_add_sync(0xffffffffu, c);
    if (lane == 0 && c) atomicAdd(&count, c);
  }
  // One thread of a block reads the counts: every warp of the grid at the same
  // line of L2 is a queue of its own (3 us of a large batch's 50).
  if (threadIdx.x == 0) {
    if (a.mask && !a.count_here) count = __ldcg(a.n_count);
    if (a.reduction == 1) any = __ldcg(a.n_count + 1);
  }
  __syncthreads();
  if (a.mask) n = count;
  const int n_any = any;
  float w = a.reduction == 0 ? (n > 0 ? 1.f / (float)n : 0.f) : a.inv_norm;
  float w_adv = 0.f;  // the sequence's advantage
  auto enter = [&](int t) {  // the sequence of token t and its values
    s = seq_advance(a.cu, a.S, s, t);
    end = s < a.S - 1 ? __ldg(a.cu + s + 1) : a.T;
    if (a.adv_per_seq) w_adv = __ldg(a.advantages + s);
    if (a.reduction == 1) {
      const int ns = __ldcg(a.n_seq + s);
      w = ns > 0 ? 1.f / ((float)ns * (float)n_any) : 0.f;
    }
  };
  if (NEED_SEQ) end = -1;  // enter at the first token

  Sum2 pg, kl;  // of the lane's sums over eight pieces, 32 tokens
  float pg1 = 0.f, kl1 = 0.f;
  int left = 8, clipped = 0;
  for (int p = begin; p < run_end; p += SEQ_PIECE) {
    const int t = p + lane * SEQ_TOK;
    if (t >= run_end) break;  // nothing below is collective
    const bool whole = vec && t + SEQ_TOK <= a.T;
    uint32_t on;
    float lp[SEQ_TOK], lo[SEQ_TOK], lr[SEQ_TOK], adv[SEQ_TOK];
    if (RING) {
      const int last = stage == 0 ? RING_STAGES - 1 : stage - 1;
      copy_ahead(t + (RING_STAGES - 1) * SEQ_PIECE, last);
      copy_async_wait<RING_STAGES - 1>();
    }
    if (RING && whole) {
      const uint32_t d = ring + stage * RING_BYTES + lane * 16;
      read4(d, lp);
      if (a.old_logp) read4(d + 512, lo);
      if (a.ref_logp) read4(d + 1024, lr);
      if (!a.adv_per_seq) read4(d + 1536, adv);
      on = (1u << SEQ_TOK) - 1u;
      if (a.mask)
        on = nonzero_bytes(ld_shared_u32(ring + stage * RING_BYTES + 2048 + lane * 4));
      stage = stage == RING_STAGES - 1 ? 0 : stage + 1;
    } else {
      on = load_mask(a.mask, t, a.T, vec);
    }
    if (whole && !RING) {  // one test for all the loads
      load_tok(a.logp, t, a.T, true, lp);
      if (a.old_logp) load_tok(a.old_logp, t, a.T, true, lo);
      if (a.ref_logp) load_tok(a.ref_logp, t, a.T, true, lr);
      if (!a.adv_per_seq) load_tok(a.advantages, t, a.T, true, adv);
    } else if (!whole) {
      load_tok(a.logp, t, a.T, false, lp);
      if (a.old_logp) load_tok(a.old_logp, t, a.T, false, lo);
      if (a.ref_logp) load_tok(a.ref_logp, t, a.T, false, lr);
      if (!a.adv_per_seq) load_tok(a.advantages, t, a.T, false, adv);
    }
    float g[SEQ_TOK];
#pragma unroll
    for (int j = 0; j < SEQ_TOK; ++j) g[j] = 0.f;
    // The lane's tokens, a sequence at a time: once, but where one ends.
    int at = t;
    do {
      uint32_t mine = on;
      int upto = t + SEQ_TOK;
      if (NEED_SEQ) {
        if (at >= end) enter(at);
        // (an end that is not past `at` comes of bad offsets: the last sequence's then)
        if (at > t || end < upto) {
          if (end > at && end < upto) upto = end;
          mine &= ((1u << (upto - t)) - 1u) & ~((1u << (at - t)) - 1u);
        }
      }
      at = upto;
#pragma unroll
      for (int j = 0; j < SEQ_TOK; ++j) {
        // What lies under the mask is replaced before it is used: with d = x = A = 0
        // a token is inside every border and adds nothing.
        const bool counts = (mine >> j) & 1u;
        const float A = counts ? (a.adv_per_seq ? w_adv : adv[j]) : 0.f;
        const bool pos = A >= 0.f;
        float r = 1.f;
        bool clip = false;
        if (a.old_logp) {
          const float d = counts ? lp[j] - lo[j] : 0.f;
          const float side = pos ? d : -d, border = pos ? a.high_hi : -a.low_hi;
          clip = side > border;
          if (counts && side == border)  // hardly ever (what is not counted may not be looked at)
            clip = pos ? exceeds(d, lp[j], lo[j], a.high_hi, a.high_lo)
                       : exceeds(-d, lo[j], lp[j], -a.low_hi, -a.low_lo);
          r = clip ? (pos ? a.r_high : a.r_low) : exp_fast(d);
          if (a.dual && !pos && d >= a.dual_hi && exceeds(d, lp[j], lo[j], a.dual_hi, a.dual_lo)) {
            clip = true;
            r = a.r_dual;
          }
        }
        const float rA = r * A;
        pg1 = fmaf(-w, rA, pg1);
        float gj = clip ? 0.f : -rA;
        if (a.ref_logp) {
          const float x = counts ? lr[j] - lp[j] : 0.f;
          const float k = exp_rest(x);
          kl1 = fmaf(w, k, kl1);
          gj = fmaf(-a.kl_coef, x + k, gj);
        }
        clipped += clip ? 1 : 0;
        g[j] = fmaf(w * a.grad_loss, gj, g[j]);
      }
    } while (NEED_SEQ && at < min(t + SEQ_TOK, a.T));
    if (a.grad) {
      if (whole)
        store_tok(a.grad, t, a.T, true, g);
      else
        store_tok(a.grad, t, a.T, false, g);
    }
    if (--left == 0) {
      pg.add(pg1);
      kl.add(kl1);
      pg1 = kl1 = 0.f;
      left = 8;
    }
  }
  pg.add(pg1);
  kl.add(kl1);
  __syncwarp();
  pg = warp_sum(pg);
  kl = warp_sum(kl);
  clipped = __reduce_add_sync(0xffffffffu, clipped);
  if (lane == 0) {
    part[0][warp] = make_float2(pg.hi, pg.lo);
    part[1][warp] = make_float2(kl.hi, kl.lo);
    if (clipped) atomicAdd(&clips, clipped);
  }
  __syncthreads();
  if (warp != 0) return;
  // Warp 0: the block's sums (lanes 0 to 15 hold the warps'), then, in the block
  // that finishes last, all blocks'.
  auto load = [](const float2& v) {
    Sum2 r;
    r.hi = v.x;
    r.lo = v.y;
    return r;
  };
  pg = lane < SEQ_WARPS ? load(part[0][lane]) : Sum2();
  kl = lane < SEQ_WARPS ? load(part[1][lane]) : Sum2();
  pg = warp_sum(pg);
  kl = warp_sum(kl);
  clipped = clips;
  if (!alone) {
    int done = 0;
    if (lane == 0) {
      a.block_part[blockIdx.x] = make_float4(pg.hi, pg.lo, kl.hi, kl.lo);
      a.block_clips[blockIdx.x] = clipped;
      __threadfence();
      done = atomicAdd(a.ticket, 1) == (int)gridDim.x - 1;
    }
    if (!__shfl_sync(0xffffffffu, done, 0)) return;
    __threadfence();
    pg = kl = Sum2();
    clipped = 0;
#pragma unroll 8
    for (int b = lane; b < (int)gridDim.x; b += 32) {
      const float4 v = __ldcg(a.block_part + b);
      pg.add(v.x, v.y);
      kl.add(v.z, v.w);
      clipped += __ldcg(a.block_clips + b);
    }
    pg = warp_sum(pg);
    kl = warp_sum(kl);
    clipped = __reduce_add_sync(0xffffffffu, clipped);
  }
  if (lane == 0) {
    Sum2 loss = pg;
    loss.add(a.kl_coef * kl.hi, a.kl_coef * kl.lo);
    a.loss[0] = loss.value();
    if (a.stats) {
      a.stats[0] = pg.value();
      a.stats[1] = kl.value();
      a.stats[2] = n > 0 ? (float)clipped / (float)n : 0.f;
    }
  }
}

// ----------------------------------------------------------- preference loss

// Warp w's part of every sequence s that it meets, to slot w + s: the sum of
// the counted tokens' log ratios, and how many they are.
__device__ __forceinline__ void pref_sums(const PrefArgs& a, int w, int R) {
  const int lane = threadIdx.x & 31;
  const int S = 2 * a.P;
  const long long first = (long long)w * R;
  if (first >= a.T) return;
  const int run_end = (int)min((long long)a.T, first + R);
  int s = seq_find_warp(a.cu, 0, S, (int)first);
  int end = s < S - 1 ? __ldg(a.cu + s + 1) : a.T;  // uniform, as s
  Sum2 sum;
  int n = 0;
  auto flush = [&]() {
    sum = warp_sum(sum);
    const int c = __reduce_add_sync(0xffffffffu, n);
    if (lane == 0) {
      a.slot_sum[(long long)w + s] = make_float2(sum.hi, sum.lo);
      a.slot_n[(long long)w + s] = c;
    }
    sum = Sum2();
    n = 0;
  };
  for (int p = (int)first; p < run_end; p += SEQ_PIECE) {
    const int t = p + lane * SEQ_TOK;
    const uint32_t on = load_mask(a.mask, t, a.T, a.vec != 0);
    const bool whole = a.vec != 0 && t + SEQ_TOK <= a.T;
    float x[SEQ_TOK], y[SEQ_TOK];
    load_tok(a.logp, t, a.T, whole, x);
    if (a.ref_logp) load_tok(a.ref_logp, t, a.T, whole, y);
#pragma unroll
    for (int j = 0; j < SEQ_TOK; ++j)
      x[j] = (on >> j) & 1u ? (a.ref_logp ? x[j] - y[j] : x[j]) : 0.f;
    const int piece_end = min(run_end, p + SEQ_PIECE);
    int at = p;  // tokens of the piece before it have been added
    while (end < piece_end && s < S - 1) {
      // the sequence ends inside the piece
      float part = 0.f;
#pragma unroll
      for (int j = 0; j < SEQ_TOK; ++j) {
        const bool mine = t + j >= at && t + j < end;
        part += mine ? x[j] : 0.f;
        n += mine ? (int)((on >> j) & 1u) : 0;
      }
      sum.add(part);
      flush();
      at = max(at, end);
      s = seq_advance(a.cu, S, s, at);
      end = s < S - 1 ? __ldg(a.cu + s + 1) : a.T;
    }
    float part = 0.f;
#pragma unroll
    for (int j = 0; j < SEQ_TOK; ++j) {
      const bool mine = t + j >= at;
      part += mine ? x[j] : 0.f;
      n += mine ? (int)((on >> j) & 1u) : 0;
    }
    sum.add(part);
  }
  flush();
}

// One warp: both sequences' sums of pair i from their slots, the pair's loss,
// and the gradient that each counted token of either sequence gets.
__device__ __forceinline__ void pref_pair(const PrefArgs& a, int i, int R, int* status) {
  const int lane = threadIdx.x & 31;
  const int S = 2 * a.P;
  const int seq[2] = {a.halves ? i : 2 * i, a.halves ? a.P + i : 2 * i + 1};
  Sum2 q[2];
  float share[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int s = seq[k];
    const int b0 = __ldg(a.cu + s), b1 = __ldg(a.cu + s + 1);
    if (lane == 0 && (b0 > b1 || (s == 0 && b0 != 0) || (s == S - 1 && b1 != a.T)))
      record_error(status, DEV_ERR_INVALID_ARG);
    const int c0 = max(0, min(a.T, b0)), c1 = max(0, min(a.T, b1));
    int n = 0;
    if (c1 > c0)
      for (int w = c0 / R + lane; w <= (c1 - 1) / R; w += 32) {
        const float2 v = a.slot_sum[(long long)w + s];
        q[k].add(v.x, v.y);
        n += a.slot_n[(long long)w + s];
      }
    q[k] = warp_sum(q[k]);
    n = __reduce_add_sync(0xffffffffu, n);
    share[k] = 1.f;
    if (a.average) {  // the quotient in two floats too: h is a difference of these
      const float m = (float)max(n, 1);
      share[k] = 1.f / m;
      const float hi = q[k].hi / m;
      q[k].lo = (fmaf(-hi, m, q[k].hi) + q[k].lo) / m;
      q[k].hi = hi;
    }
  }
  if (lane == 0) {
    Sum2 gap = q[0];
    gap.add(-q[1].hi, -q[1].lo);
    gap.add(-a.margin);
    const float h = gap.value(), b = a.beta * h, eps = a.label_smoothing;
    float each, slope;
    if (a.kind == 0) {
      // -log sigma(b) = log(1 + e^-|b|) + max(-b, 0), its mirror for -b, and
      // sigma(-b), from one exponential of -|b|
      const float e = expf(-fabsf(b)), soft = log1pf(e);
      each = (1.f - eps) * (soft + fmaxf(-b, 0.f)) + eps * (soft + fmaxf(b, 0.f));
      slope = a.beta * (eps - (b > 0.f ? e : 1.f) / (1.f + e));
    } else if (a.kind == 1) {
      gap.add(-a.half_inv_beta);
      const float off = gap.value();
      each = off * off;
      slope = 2.f * off;
    } else {
      each = fmaxf(1.f - b, 0.f);
      slope = b < 1.f ? -a.beta : 0.f;
    }
    if (b != b) each = slope = b;  // fmaxf drops a NaN
    a.pair_loss[i] = each;
    a.rewards[2 * i] = a.beta * q[0].value();
    a.rewards[2 * i + 1] = a.beta * q[1].value();
    slope *= a.grad_over_P;
    a.coef[seq[0]] = slope * share[0];
    a.coef[seq[1]] = -slope * share[1];
  }
}

// Every counted token of warp w's run gets its sequence's gradient. coef was
// written by the launch, or by the part of the block, before.
__device__ __forceinline__ void pref_grads(const PrefArgs& a, int w, int R) {
  const int lane = threadIdx.x & 31;
  const int S = 2 * a.P;
  const long long first = (long long)w * R;
  if (first >= a.T) return;
  const int run_end = (int)min((long long)a.T, first + R);
  if (a.mask)
    for (long long i = first + lane * 128; i < run_end; i += 32 * 128) prefetch_l2(a.mask + i);
  int s = seq_find_warp(a.cu, 0, S, (int)first);
  grid_dependency_wait();  // coef
  int end = -1;
  float c = 0.f;
  for (int p = (int)first; p < run_end; p += SEQ_PIECE) {
    const int t = p + lane * SEQ_TOK;
    if (t >= run_end) break;  // nothing below is collective
    const uint32_t on = load_mask(a.mask, t, a.T, a.vec != 0);
    float g[SEQ_TOK];
#pragma unroll
    for (int j = 0; j < SEQ_TOK; ++j) {
      if (t + j >= end && t + j < a.T) {
        s = seq_advance(a.cu, S, s, t + j);
        end = s < S - 1 ? __ldg(a.cu + s + 1) : a.T;
        c = __ldcg(a.coef + s);
      }
      g[j] = (on >> j) & 1u ? c : 0.f;
    }
    store_tok(a.grad, t, a.T, a.vec != 0 && t + SEQ_TOK <= a.T, g);
  }
}

// The pairs' mean by one warp, in a fixed order.
__device__ __forceinline__ void pref_mean(const PrefArgs& a) {
  const int lane = threadIdx.x & 31;
  Sum2 v;
#pragma unroll 8
  for (int i = lane; i < a.P; i += 32) v.add(__ldcg(a.pair_loss + i));
  v = warp_sum(v);
  if (lane == 0) a.loss[0] = v.value() / (float)a.P;
}

__global__ void __launch_bounds__(SEQ_THREADS)
    pref_sums_kernel(const PrefArgs a, int warps, int* status) {
  grid_dependents_go();
  if (blockIdx.x == 0 && threadIdx.x == 0) *status = 0;  // the next launch records errors
  pref_sums(a, blockIdx.x * SEQ_WARPS + (threadIdx.x >> 5), run_length(a.T, warps));
}

__global__ void __launch_bounds__(SEQ_THREADS)
    pref_pairs_kernel(const PrefArgs a, int warps, int* status) {
  const int i = blockIdx.x * SEQ_WARPS + (threadIdx.x >> 5);
  grid_dependents_go();
  grid_dependency_wait();
  if (i < a.P) pref_pair(a, i, run_length(a.T, warps), status);
}

__global__ void __launch_bounds__(SEQ_THREADS) pref_grad_kernel(const PrefArgs a, int warps) {
  if (a.grad)
    pref_grads(a, blockIdx.x * SEQ_WARPS + (threadIdx.x >> 5), run_length(a.T, warps));
  if (blockIdx.x == 0 && threadIdx.x < 32) {
    grid_dependency_wait();
    pref_mean(a);
  }
}

// The three parts in one block, for batches that one block holds.
__global__ void __launch_bounds__(PREF_ONE_THREADS)
    pref_one_block_kernel(const PrefArgs a, int* status) {
  constexpr int WARPS = PREF_ONE_THREADS / 32;
  const int w = threadIdx.x >> 5;
  const int R = run_length(a.T, WARPS);
  if (threadIdx.x == 0) *status = 0;
  pref_sums(a, w, R);
  __syncthreads();
  for (int i = w; i < a.P; i += WARPS) pref_pair(a, i, R, status);
  __syncthreads();
  if (w == WARPS - 1) pref_mean(a);
  if (a.grad) pref_grads(a, w, R);
}

}  // namespace

// Blocks of the walks: as many as are resident at once, and none without a
// piece of tokens for each warp.
int seq_blocks(int T, int num_sms) {
  const long long pieces = ((long long)T + SEQ_PIECE - 1) / SEQ_PIECE;
  return (int)std::max<long long>(
      1, std::min<long long>((pieces + SEQ_WARPS - 1) / SEQ_WARPS, (long long)SEQ_RESIDENT * num_sms));
}
int seq_warps(int T, int num_sms) { return seq_blocks(T, num_sms) * SEQ_WARPS; }

cudaError_t launch_policy_loss(const PolicyArgs& a, int num_sms, int* status,
                               cudaStream_t stream) {
  const bool per_seq = a.reduction == 1;
  const dim3 block(SEQ_THREADS);
  const dim3 grid(policy_one_block(a.T, a.reduction) ? 1u : (unsigned)seq_blocks(a.T, num_sms));
  const bool seq = per_seq || a.adv_per_seq;
  const bool ring = a.vec && run_length(a.T, (int)grid.x * SEQ_WARPS) >= 4 * SEQ_PIECE;
  const auto kernel = seq ? (ring ? policy_loss_kernel<true, true> : policy_loss_kernel<true, false>)
                          : (ring ? policy_loss_kernel<false, true>
                                  : policy_loss_kernel<false, false>);
  const size_t smem = ring ? (size_t)SEQ_WARPS * RING_STAGES * RING_BYTES : 0;
  if (ring) {  // (the same value every time: concurrent first calls do no harm)
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  if (!per_seq && (!a.mask || a.count_here))
    return launch_kernel("policy_loss", kernel, grid, block, smem, stream, a, status);
  // What the loss kernel reads before its wait was complete before the count began.
  const cudaError_t e =
      launch_kernel("policy_count", policy_count_kernel, grid, block, 0, stream, a.mask, a.cu, a.T,
                    a.S, a.vec, per_seq ? a.n_seq : nullptr, a.n_count);
  if (e != cudaSuccess) return e;
  return launch_kernel_early("policy_loss", kernel, grid, block, smem, stream, a, status);
}

cudaError_t launch_pref_loss(const PrefArgs& a, int num_sms, int* status, cudaStream_t stream) {
  if (pref_one_block(a.T, a.P))
    return launch_kernel("pref_one_block", pref_one_block_kernel, dim3(1), dim3(PREF_ONE_THREADS),
                         0, stream, a, status);
  const int blocks = seq_blocks(a.T, num_sms), warps = blocks * SEQ_WARPS;
  const dim3 grid((unsigned)blocks), block(SEQ_THREADS);
  cudaError_t e =
      launch_kernel("pref_sums", pref_sums_kernel, grid, block, 0, stream, a, warps, status);
  if (e != cudaSuccess) return e;
  e = launch_kernel_early("pref_pairs", pref_pairs_kernel,
                          dim3((unsigned)((a.P + SEQ_WARPS - 1) / SEQ_WARPS)), block, 0, stream, a,
                          warps, status);
  if (e != cudaSuccess) return e;
  return launch_kernel_early("pref_grad", pref_grad_kernel, a.grad ? grid : dim3(1), block, 0, stream,
                             a, warps);
}

}  // namespace kdkl
