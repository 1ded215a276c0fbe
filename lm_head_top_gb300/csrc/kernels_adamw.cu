// AdamW over a list of tensors in one launch, states in 32 or in 8 bits.
//
//   g' = g * grad_scale            m' = b1 m + (1 - b1) g'
//   v' = b2 v + (1 - b2) g'^2      p' = p (1 - lr wd) - lr/(1-b1^t) * m' / (sqrt(v') / sqrt(1-b2^t) + eps)
//
// Every product and sum is rounded to fp32 by itself, in the order written (no
// contraction into fused multiply-adds), so m' and v' are those of the
// elementwise formula, bit for bit, whichever path computes them; with 32-bit
// states so are the root and the quotient, and p'.
//
// 8-bit states: m and the root r = sqrt(v) are held in e4m3, 256 consecutive
// elements sharing one fp32 power of two, the least with which the block's
// largest magnitude stays within 463.04 (which rounds to e4m3's largest, 448). The root, not v: e4m3 spans 2^17.8 from
// its smallest step to its largest value, which as a root spans 2^35 of v. A
// root that is not zero is never stored as zero (it would divide by eps
// alone). This step's update uses the 32-bit m' and sqrt(v'); only what is
// kept for the next step is rounded to 8 bits (m to a relative 2^-4, the root
// likewise: what the user chose when asking for 8-bit states). A power of two
// as the scale makes scaling exact, so e4m3 is the only rounding. With 16 to 22
// bytes an element the correctly rounded quotient and root are what the kernel
// would wait for (64 % of issue slots at 69 % of the DRAM rate). So the quotient
// is the hardware's approximation: 2 ulp of the step, which is a thousandth of p.
// The root is one step of Newton's iteration better than the hardware's: a root
// next to halfway between two codes falls on the formula's side, where an
// approximate one fell on the other for some one element in a million, a whole
// step of e4m3 (341M elements: 0.836 ms approximate, 0.844, correctly rounded 0.869).
//
// What bounds it: DRAM. Read g, p, m, v and write p, m, v (and the bf16 copy):
// 30 bytes per element with fp32 gradients, 32-bit states and a copy.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include <algorithm>

#include "kdkl_internal.h"
#include "tc_primitives.cuh"

namespace kdkl {

namespace {

constexpr int ADAM_THREADS = 256;
constexpr int ADAM_VEC = 8;      // consecutive elements per thread; a warp covers one scale block
constexpr int ADAM_BLOCK = 256;  // elements per scale
constexpr int ADAM_PASS = ADAM_THREADS * ADAM_VEC;  // elements of a thread block's pass

static_assert(ADAM_VEC * 32 == ADAM_BLOCK, "a warp's pass is one scale block");

// The tensors of one launch travel as a kernel parameter: no table in device
// memory to build, upload or keep in step with the tensors.
template <int CAP>
struct AdamTable {
  AdamTensor t[CAP];
  int n;
};

struct Vec8 {
  float x[ADAM_VEC];
};

__device__ __forceinline__ float bf16_to_f32(uint16_t v) {
  return __uint_as_float((uint32_t)v << 16);
}
__device__ __forceinline__ uint16_t f32_to_bf16(float v) {
  return __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

// Eight consecutive elements from index i; those at or past n read as zero.
__device__ __forceinline__ Vec8 load8(const float* p, long long i, long long n, bool vec) {
  Vec8 r;
  if (vec && i + ADAM_VEC <= n) {
    const float4 a = __ldcs(reinterpret_cast<const float4*>(p + i));
    const float4 b = __ldcs(reinterpret_cast<const float4*>(p + i) + 1);
    r.x[0] = a.x; r.x[1] = a.y; r.x[2] = a.z; r.x[3] = a.w;
    r.x[4] = b.x; r.x[5] = b.y; r.x[6] = b.z; r.x[7] = b.w;
  } else {
#pragma unroll
    for (int j = 0; j < ADAM_VEC; ++j) r.x[j] = i + j < n ? p[i + j] : 0.f;
  }
  return r;
}

__device__ __forceinline__ Vec8 load8(const uint16_t* p, long long i, long long n, bool vec) {
  Vec8 r;
  if (vec && i + ADAM_VEC <= n) {
    const uint4 a = __ldcs(reinterpret_cast<const uint4*>(p + i));
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      r.x[2 * j] = __uint_as_float(w[j] << 16);
      r.x[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int j = 0; j < ADAM_VEC; ++j) r.x[j] = i + j < n ? bf16_to_f32(p[i + j]) : 0.f;
  }
  return r;
}

__device__ __forceinline__ void store8(float* p, long long i, long long n, bool vec,
                                       const Vec8& r) {
  if (vec && i + ADAM_VEC <= n) {
    __stcs(reinterpret_cast<float4*>(p + i), make_float4(r.x[0], r.x[1], r.x[2], r.x[3]));
    __stcs(reinterpret_cast<float4*>(p + i) + 1, make_float4(r.x[4], r.x[5], r.x[6], r.x[7]));
  } else {
#pragma unroll
    for (int j = 0; j < ADAM_VEC; ++j)
      if (i + j < n) p[i + j] = r.x[j];
  }
}

__device__ __forceinline__ void store8(uint16_t* p, long long i, long long n, bool vec,
                                       const Vec8& r) {
  if (vec && i + ADAM_VEC <= n) {
    uint4 w;
    w.x = pack_bf16x2(r.x[0], r.x[1]);
    w.y = pack_bf16x2(r.x[2], r.x[3]);
    w.z = pack_bf16x2(r.x[4], r.x[5]);
    w.w = pack_bf16x2(r.x[6], r.x[7]);
    __stcs(reinterpret_cast<uint4*>(p + i), w);
  } else {
#pragma unroll
    for (int j = 0; j < ADAM_VEC; ++j)
      if (i + j < n) p[i + j] = f32_to_bf16(r.x[j]);
  }
}

// Eight e4m3 codes from index i as their values; codes past n read as zero.
__device__ __forceinline__ Vec8 load_e4m3(const uint8_t* p, long long i, long long n, bool vec) {
  uint32_t w[2] = {0u, 0u};
  if (vec && i + ADAM_VEC <= n) {
    const uint2 a = __ldcs(reinterpret_cast<const uint2*>(p + i));
    w[0] = a.x;
    w[1] = a.y;
  } else {
#pragma unroll
    for (int j = 0; j < ADAM_VEC; ++j)
      if (i + j < n) w[j >> 2] |= (uint32_t)p[i + j] << (8 * (j & 3));
  }
  Vec8 r;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const __nv_fp8x2_storage_t two = (__nv_fp8x2_storage_t)(w[j >> 1] >> (16 * (j & 1)));
    const float2 f = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(two, __NV_E4M3)));
    r.x[2 * j] = f.x;
    r.x[2 * j + 1] = f.y;
  }
  return r;
}

__device__ __forceinline__ void store_e4m3(uint8_t* p, long long i, long long n, bool vec,
                                           const Vec8& r) {
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const __nv_fp8x2_storage_t two = __nv_cvt_float2_to_fp8x2(
        make_float2(r.x[2 * j], r.x[2 * j + 1]), __NV_SATFINITE, __NV_E4M3);
    w[j >> 1] |= (uint32_t)two << (16 * (j & 1));
  }
  if (vec && i + ADAM_VEC <= n) {
    __stcs(reinterpret_cast<uint2*>(p + i), make_uint2(w[0], w[1]));
  } else {
#pragma unroll
    for (int j = 0; j < ADAM_VEC; ++j)
      if (i + j < n) p[i + j] = (uint8_t)(w[j >> 2] >> (8 * (j & 3)));
  }
}

// Least power of two (not below 2^-126) that keeps a block whose largest
// magnitude is `top` (finite, as bits) within 512 * 0.904383 = 463.04, which
// rounds to 448. (448 itself, or any border of few bits, is met exactly by sums
// of 8-bit states and bf16 gradients, and the last bit of such a sum would then
// set the scale.) An all-zero block gets 1.
__device__ __forceinline__ float scale_for(uint32_t top) {
  if (top == 0u) return 1.f;
  const float half = __uint_as_float((top & 0x7fffffu) | 0x3f000000u);  // in [0.5, 1)
  const int e = (int)(top >> 23) - 126 - 9 + (half > 0.904383f ? 1 : 0);
  return __uint_as_float((uint32_t)(max(e, -126) + 127) << 23);
}

__device__ __forceinline__ float pow2_inverse(float s) {  // s = 2^e, -126 <= e <= 120
  return __uint_as_float(0x7f000000u - __float_as_uint(s));
}

constexpr uint32_t kInfBits = 0x7f800000u;

// Bits of the warp's largest magnitude; NaN are passed over.
__device__ __forceinline__ uint32_t warp_top(const Vec8& r) {
  float a = 0.f;
#pragma unroll
  for (int j = 0; j < ADAM_VEC; ++j) a = fmaxf(a, fabsf(r.x[j]));
  return __reduce_max_sync(0xffffffffu, __float_as_uint(a));
}

// A block that holds infinities: they set no scale and are kept as NaN, which
// e4m3 has and infinities it has not.
__device__ __forceinline__ uint32_t drop_infinities(Vec8& r) {
#pragma unroll
  for (int j = 0; j < ADAM_VEC; ++j)
    if (fabsf(r.x[j]) == INFINITY) r.x[j] = __uint_as_float(0x7fffffffu);
  return warp_top(r);
}

// sqrt(v) from the hardware's approximate 1 / sqrt(v), y: r = v y, and one step of Newton's
// iteration, r + (v - r^2) / (2 r), with y / 2 for 1 / (2 r) and v - r^2 in one rounding. The
// correctly rounded root but for one in some 2^22 (8-bit states only).
__device__ __forceinline__ float sqrt_newton(float v) {
  float y;
  asm("rsqrt.approx.f32 %0, %1;" : "=f"(y) : "f"(v));
  const float r = v * y;
  const float better = fmaf(fmaf(-r, r, v), 0.5f * y, r);
  return v > 0.f && v < INFINITY ? better : v;
}

// The lines of a warp's pass from element i on, a lane each: p, g, m and v
// cover 256 elements in at most 8 + 8 + 2 + 2 lines of 128 bytes.
template <typename P, typename G>
__device__ __forceinline__ void prefetch_pass8(const AdamTensor& t, long long i) {
  constexpr int PL = 2 * sizeof(P), GL = 2 * sizeof(G);  // lines
  const int lane = threadIdx.x & 31;
  const char* a = nullptr;
  if (lane < PL)
    a = static_cast<const char*>(t.param) + i * sizeof(P) + lane * 128;
  else if (lane < PL + GL)
    a = static_cast<const char*>(t.grad) + i * sizeof(G) + (lane - PL) * 128;
  else if (lane < PL + GL + 2)
    a = static_cast<const char*>(t.exp_avg) + i + (lane - PL - GL) * 128;
  else if (lane < PL + GL + 4)
    a = static_cast<const char*>(t.exp_avg_sq) + i + (lane - PL - GL - 2) * 128;
  if (a) prefetch_l2(a);
}

template <typename P, typename G, bool STATE8, int CAP>
__global__ void __launch_bounds__(ADAM_THREADS)
    adamw_kernel(const __grid_constant__ AdamTable<CAP> table, const AdamScalars s) {
  // The tensor of this block: the last one whose first block is not past it.
  int lo = 0, hi = table.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (table.t[mid].block0 <= (int)blockIdx.x) lo = mid; else hi = mid - 1;
  }
  const AdamTensor& t = table.t[lo];
  const long long n = t.n;
  const bool vec = t.vec != 0;
  const float keep = t.decay ? s.keep : 1.f;
  const float gs = s.grad_scale_dev ? __fmul_rn(s.grad_scale, __ldg(s.grad_scale_dev))
                                    : s.grad_scale;
  const long long base = (long long)((int)blockIdx.x - t.block0) * s.passes * ADAM_PASS;
#pragma unroll 1
  for (int k = 0; k < s.passes; ++k) {
    const long long first = base + (long long)k * ADAM_PASS +
                            (threadIdx.x & ~31) * ADAM_VEC;  // the warp's first element
    if (first >= n) return;                                  // the whole warp
    const long long i = first + (threadIdx.x & 31) * ADAM_VEC;
    // The next pass's lines set out before this pass's arithmetic.
    if (STATE8 && k + 1 < s.passes && first + ADAM_PASS + ADAM_BLOCK <= n)
      prefetch_pass8<P, G>(t, first + ADAM_PASS);
    const Vec8 g = load8(static_cast<const G*>(t.grad), i, n, vec);
    Vec8 p = load8(static_cast<const P*>(t.param), i, n, vec);
    Vec8 m, v;
    if (STATE8) {
      m = load_e4m3(static_cast<const uint8_t*>(t.exp_avg), i, n, vec);
      v = load_e4m3(static_cast<const uint8_t*>(t.exp_avg_sq), i, n, vec);
      const float ms = t.m_scale[first / ADAM_BLOCK], vs = t.v_scale[first / ADAM_BLOCK];
#pragma unroll
      for (int j = 0; j < ADAM_VEC; ++j) {
        m.x[j] = __fmul_rn(m.x[j], ms);
        const float r = __fmul_rn(v.x[j], vs);
        v.x[j] = __fmul_rn(r, r);
      }
    } else {
      m = load8(static_cast<const float*>(t.exp_avg), i, n, vec);
      v = load8(static_cast<const float*>(t.exp_avg_sq), i, n, vec);
    }
    Vec8 root;
#pragma unroll
    for (int j = 0; j < ADAM_VEC; ++j) {
      const float gj = __fmul_rn(g.x[j], gs);
      m.x[j] = __fadd_rn(__fmul_rn(m.x[j], s.b1), __fmul_rn(gj, s.one_b1));
      v.x[j] = __fadd_rn(__fmul_rn(v.x[j], s.b2), __fmul_rn(__fmul_rn(gj, gj), s.one_b2));
      root.x[j] = STATE8 ? sqrt_newton(v.x[j]) : __fsqrt_rn(v.x[j]);
      const float den = __fadd_rn(__fmul_rn(root.x[j], s.inv_root_bc2), s.eps);
      const float q = STATE8 ? __fdividef(m.x[j], den) : __fdiv_rn(m.x[j], den);
      const float u = __fmul_rn(q, s.step);
      p.x[j] = __fsub_rn(__fmul_rn(p.x[j], keep), u);
    }
    store8(static_cast<P*>(t.param), i, n, vec, p);
    if (t.copy) store8(t.copy, i, n, vec, p);
    if (STATE8) {
      // Elements past n are zero here and set no scale. The root's scale comes
      // from the largest v by one correctly rounded root.
      uint32_t top_m = warp_top(m), top_v = warp_top(v);
      if (top_m == kInfBits) top_m = drop_infinities(m);
      if (top_v == kInfBits) {
        drop_infinities(root);
        top_v = drop_infinities(v);
      }
      const float ms = scale_for(top_m);
      const float vs = scale_for(__float_as_uint(__fsqrt_rn(__uint_as_float(top_v))));
      const float inv_m = pow2_inverse(ms), inv_v = pow2_inverse(vs);
#pragma unroll
      for (int j = 0; j < ADAM_VEC; ++j) {
        m.x[j] *= inv_m;
        const float y = root.x[j] * inv_v;
        root.x[j] = root.x[j] > 0.f ? fmaxf(y, 0.001953125f) : y;  // 2^-9, e4m3's least step
      }
      store_e4m3(static_cast<uint8_t*>(t.exp_avg), i, n, vec, m);
      store_e4m3(static_cast<uint8_t*>(t.exp_avg_sq), i, n, vec, root);
      if ((threadIdx.x & 31) == 0) {
        t.m_scale[first / ADAM_BLOCK] = ms;
        t.v_scale[first / ADAM_BLOCK] = vs;
      }
    } else {
      store8(static_cast<float*>(t.exp_avg), i, n, vec, m);
      store8(static_cast<float*>(t.exp_avg_sq), i, n, vec, v);
    }
  }
}

template <typename P, typename G, bool STATE8, int CAP>
cudaError_t launch_table(const AdamTensor* t, int n, int blocks, const AdamScalars& s,
                         cudaStream_t stream) {
  AdamTable<CAP> table;
  for (int i = 0; i < n; ++i) table.t[i] = t[i];
  table.n = n;
  return launch_kernel("adamw", adamw_kernel<P, G, STATE8, CAP>, dim3((unsigned)blocks),
                       dim3(ADAM_THREADS), 0, stream, table, s);
}

template <typename P, typename G, bool STATE8>
cudaError_t launch_typed(const AdamTensor* t, int n, int blocks, const AdamScalars& s,
                         cudaStream_t stream) {
  // A short list takes the short parameter.
  if (n <= ADAMW_SHORT_LIST)
    return launch_table<P, G, STATE8, ADAMW_SHORT_LIST>(t, n, blocks, s, stream);
  return launch_table<P, G, STATE8, ADAMW_LIST>(t, n, blocks, s, stream);
}

}  // namespace

// With 32-bit states a block makes one pass: they are all bytes, and as many
// blocks as fit keep the most of them on the way (341M elements: 1.45 ms, 4
// passes 1.51). With 8-bit states a pass is more arithmetic on fewer bytes, and
// a warp that waits for memory in each leaves DRAM idle: a block makes up to 8,
// its next lines on their way to L2 during each (0.84 ms; 4 passes 0.87, without
// the prefetch 1.00, one pass 0.95), as long as that leaves the SMs ten blocks each.
int adamw_passes(long long elements, bool state8, int num_sms) {
  if (!state8) return 1;
  return (int)std::max<long long>(1, std::min<long long>(8, elements / (10LL * num_sms * ADAM_PASS)));
}

int adamw_blocks(long long n, int passes) {
  const long long chunk = (long long)passes * ADAM_PASS;
  return (int)((n + chunk - 1) / chunk);
}

cudaError_t launch_adamw(const AdamTensor* t, int n, int blocks, bool param_bf16, bool grad_bf16,
                         bool state8, const AdamScalars& s, cudaStream_t stream) {
  const int kind = (param_bf16 ? 4 : 0) | (grad_bf16 ? 2 : 0) | (state8 ? 1 : 0);
  switch (kind) {
    case 0: return launch_typed<float, float, false>(t, n, blocks, s, stream);
    case 1: return launch_typed<float, float, true>(t, n, blocks, s, stream);
    case 2: return launch_typed<float, uint16_t, false>(t, n, blocks, s, stream);
    case 3: return launch_typed<float, uint16_t, true>(t, n, blocks, s, stream);
    case 4: return launch_typed<uint16_t, float, false>(t, n, blocks, s, stream);
    case 5: return launch_typed<uint16_t, float, true>(t, n, blocks, s, stream);
    case 6: return launch_typed<uint16_t, uint16_t, false>(t, n, blocks, s, stream);
    default: return launch_typed<uint16_t, uint16_t, true>(t, n, blocks, s, stream);
  }
}

}  // namespace kdkl
