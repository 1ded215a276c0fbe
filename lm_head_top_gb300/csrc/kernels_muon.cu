// A step of the Muon optimizer over matrices: the small ones in one launch, a block each
// (see there), the others all of them in every launch.
//
//   m = mu m + s g,   u = s g + mu m or m,   X = u / max(|u|, eps)      (r x k, r <= k)
//   5 times:  S = X X^T,  P = B S + C S^2,  X = A X + P X
//   p = p keep - step X
//
// Launches: momentum (m, and sums of squares of u by pieces of MUON_CHUNK elements),
// layout (u / |u|, transposed where the matrix is tall, as fp16 halves), and three
// products a step, the last of which updates the parameters in its epilogue: no
// product is written in 32 bits and read again.
//
// Numbers. The quintic multiplies what is left of small singular values by 3.4 a
// step, and errors with them: factors rounded to bf16 leave X some 1e-2 off, to
// tf32 or fp16 some 1e-3. So every matrix is held as two fp16 halves, x 2^e = hi +
// lo (22 bits), and a product is hi hi + hi lo + lo hi, three products on the tensor
// cores with fp32 sums. The powers of two keep fp16's range: |X| and |S| stay below
// 1.6 (singular values up to 1.21), 2^13 of which fp16 holds, and the low halves of
// all but the smallest elements above its subnormals; |P| stays below 13, 2^11.
// The tensor core's fp32 sum loses up to a unit in the last place with every
// instruction, always towards zero: 1e-5 over a few thousand terms of one sign, as
// on the diagonal of S. So the sum is taken out of TMEM every MUON_SUM_BLOCKS K
// blocks and added up in registers, rounded to nearest.
//
// S and S^2 are symmetric: tiles below the diagonal are neither computed nor stored. Where a
// product needs one, it copies the one across the diagonal and has the tensor core read it
// the other way (MN-major instead of K-major).
//
// |u| is that of u at any size: squares of fp32 vanish below 2^-75 and overflow above 2^64, so
// where a piece's largest magnitude is beyond 2^-40 or 2^40 its squares are taken again, of u by a
// power of two (SquareSum).
//
// What bounds it: the tensor cores, from r of about 1000 on. Work: 3 (r r k + r^3 +
// 2 r r k) flops a step, the 3 for the halves.
//
// Tile: 256 x 256 by a pair of CTAs (each 128 rows, its half of B's rows, its
// 128 x 256 accumulator), or, where those would be few, 128 x 128 by one; a K block of
// 64 of both halves of both factors: 64 KB a stage and CTA, which 12 instructions
// use; 3 stages. Two accumulators, so that
// one is emptied while the other is filled. Roles: warp 0 copies, warp 1 issues (2 and 3 are
// there for the registers that they give up), warps 4 to 11 empty the accumulators, 32 rows and
// half of the columns each.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <math.h>

#include <algorithm>
#include <atomic>

#include "kdkl_body.h"
#include "tc_halves.cuh"

namespace kdkl {

namespace {

constexpr float QUINTIC_A = 3.4445f, QUINTIC_B = -4.7750f, QUINTIC_C = 2.0315f;
constexpr float X_SCALE = 8192.f;  // 2^13; S the same, P 2^11

constexpr int EW_THREADS = 256;
constexpr int CTA_ROWS = 128;   // of A, and of B (or its columns), a CTA's share
// Rows and columns of a tile: a pair's, or a CTA's of its own.
__host__ __device__ constexpr int tile_of(bool pair) { return pair ? 2 * CTA_ROWS : CTA_ROWS; }
constexpr int KB = 64;
constexpr int BOX_BYTES = MUON_BOX * MUON_BOX * 2;
constexpr int HALF_BYTES = CTA_ROWS * KB * 2;  // one half of one factor: two boxes
constexpr int STAGE_BYTES = 4 * HALF_BYTES;
constexpr int STAGES = 3;
constexpr int EPI_WARPS = 8;
constexpr int EPI_WARP0 = 4;
constexpr int PRODUCT_THREADS = 32 * (EPI_WARP0 + EPI_WARPS);
// Registers of a thread: 168 at the launch, moved from the first four warps to the others,
// which hold 128 sums each.
constexpr int FEW_REGS = 40, MANY_REGS = 232;
static_assert(128 * FEW_REGS + 32 * EPI_WARPS * MANY_REGS <= PRODUCT_THREADS * 168,
              "what the block was launched with");
constexpr int EPI_BYTES = 32 * 128;  // its staging: 32 rows of 32 elements' two halves
constexpr int MUON_SUM_BLOCKS = 8;   // K blocks of one sum on the tensor core
constexpr uint32_t MN_BOX_BYTES = MUON_BOX * 128;  // from one box of columns to the next
constexpr int BARS = 2 * STAGES + 5;
constexpr int BAR_BYTES = 256;
constexpr int PRODUCT_SMEM = STAGES * STAGE_BYTES + EPI_WARPS * EPI_BYTES + BAR_BYTES + 1024;
static_assert(BARS * 8 + 8 <= BAR_BYTES, "barriers, TMEM address, abort flag");
static_assert(PRODUCT_SMEM <= 232448, "shared memory of a CTA");

// ------------------------------------------------------------- elementwise

template <typename G>
__device__ __forceinline__ float load_grad(const void* g, long long i) {
  if (sizeof(G) == 2) return __bfloat162float(static_cast<const __nv_bfloat16*>(g)[i]);
  return static_cast<const float*>(g)[i];
}

// Four consecutive gradients.
template <typename G>
__device__ __forceinline__ float4 load_grad4(const void* g, long long i) {
  if (sizeof(G) == 2) {
    const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(g) + i);
    return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u),
                       __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u));
  }
  return *reinterpret_cast<const float4*>(static_cast<const float*>(g) + i);
}

// mu m + s g, and by the same step what Nesterov's way adds to it: the product of s and g rounded,
// then one rounding, the same wherever a matrix is worked on.
__device__ __forceinline__ float new_momentum(float m, float mu, float sg) {
  return __fmaf_rn(mu, m, sg);
}

// Sum over the block, in every thread.
template <int THREADS>
__device__ __forceinline__ float block_sum(float v) {
  __shared__ float red[THREADS / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.f;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) s += red[w];
  return s;
}

// A sum of squares of u / unit. The unit is 1 where the largest magnitude is within 2^-40 and 2^40
// (squares of 2^32 elements stay below 2^112, and what is lost below 2^-63 of them is nothing beside
// it), else 2^84 or 2^-84, which bring all that lies beyond within 2^-65 and 2^44.
constexpr float U_LARGE = 0x1p40f, U_SMALL = 0x1p-40f, U_UNIT = 0x1p84f;

struct SquareSum {
  float sum = 0.f, most = 0.f;
  __device__ __forceinline__ void add(float u) {
    sum += u * u;
    most = fmaxf(most, fabsf(u));
  }
  // Of the block's: the sum, and the unit that it ought to have been taken in (a NaN is in the sum,
  // if not in the maximum).
  template <int THREADS>
  __device__ __forceinline__ float over_block() {
    __shared__ float2 red[THREADS / 32];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      sum += __shfl_xor_sync(0xffffffffu, sum, o);
      most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
    }
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = make_float2(sum, most);
    __syncthreads();
    sum = most = 0.f;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
      sum += red[w].x;
      most = fmaxf(most, red[w].y);
    }
    return most > U_LARGE ? U_UNIT : most > 0.f && most < U_SMALL ? 1.f / U_UNIT : 1.f;
  }
};

// The sum of a matrix's pieces where one of them is not in 1's, and the largest unit that there is,
// which it is in.
// (A call of its own: its registers would be a thread block less on an SM for the layout pass.)
__device__ __noinline__ float2 sum_of_units(const float2* piece, int pieces) {
  float ss = 0.f, large = 0.f, small = 0.f;
  for (int i = threadIdx.x; i < pieces; i += EW_THREADS) {
    const float2 p = piece[i];
    if (p.y == 1.f)
      ss += p.x;
    else if (p.y > 1.f)
      large += p.x;
    else
      small += p.x;
  }
  ss = block_sum<EW_THREADS>(ss);
  large = block_sum<EW_THREADS>(large);
  small = block_sum<EW_THREADS>(small);
  auto in_next = [](float sum) { return sum * (1.f / U_UNIT) * (1.f / U_UNIT); };
  if (!(large == 0.f)) return make_float2(large + in_next(ss + in_next(small)), U_UNIT);
  if (!(ss == 0.f)) return make_float2(ss + in_next(small), 1.f);
  return make_float2(small, 1.f / U_UNIT);
}

// What u is multiplied by to be X times 2^13: by max(|u|, eps), where u's squares over the unit's
// add up to ss (NaN stays NaN). Normal up to |u| = 2^139; at the most that a matrix can have, 2^144,
// it holds 18 bits.
__device__ __forceinline__ float to_x(float ss, float unit, float eps) {
  const float norm = sqrtf(ss), least = eps / unit;
  return X_SCALE / (norm < least ? least : norm) / unit;
}

// The group that number `x` of a launch falls in; `start` gives each group's first.
template <typename F>
__device__ __forceinline__ int group_of(const MuonRound& r, int x, F start) {
  int g = 0;
  while (g + 1 < r.n_groups && x >= start(r.g[g + 1])) ++g;
  return g;
}

template <typename G>
__global__ void __launch_bounds__(EW_THREADS)
    muon_momentum_kernel(const __grid_constant__ MuonRound r, const __grid_constant__ MuonList l) {
  grid_dependents_go();
  const int gi = group_of(r, blockIdx.x, [](const MuonGroup& g) { return g.blocks0; });
  const MuonGroup& g = r.g[gi];
  const int local = blockIdx.x - g.blocks0;
  const int which = local / g.parts, piece = local - which * g.parts;
  const MuonMatrix& m = l.m[g.first + which];
  const long long n = (long long)g.r * g.k;
  const long long begin = (long long)piece * MUON_CHUNK, end = min(n, begin + MUON_CHUNK);
  const float mu = r.momentum;
  grid_dependency_wait();
  const float s = r.grad_scale_dev ? r.grad_scale * *r.grad_scale_dev : r.grad_scale;
  SquareSum squares;
  auto one = [&](float grad, float& mom) {
    const float gs = __fmul_rn(grad, s);
    mom = new_momentum(mom, mu, gs);
    squares.add(r.nesterov ? new_momentum(mom, mu, gs) : mom);
  };
  long long i = begin;
  if (((uintptr_t)m.momentum & 15) == 0 && ((uintptr_t)m.grad & 15) == 0) {
    const long long whole = begin + ((end - begin) & ~3ll);
#pragma unroll 4
    for (i = begin + threadIdx.x * 4; i < whole; i += EW_THREADS * 4) {
      const float4 gr = load_grad4<G>(m.grad, i);
      float4 mo = *reinterpret_cast<const float4*>(m.momentum + i);
      one(gr.x, mo.x);
      one(gr.y, mo.y);
      one(gr.z, mo.z);
      one(gr.w, mo.w);
      *reinterpret_cast<float4*>(m.momentum + i) = mo;
    }
    i = whole;
  }
  for (i += threadIdx.x; i < end; i += EW_THREADS) one(load_grad<G>(m.grad, i), m.momentum[i]);
  const float unit = squares.over_block<EW_THREADS>();
  float ss = squares.sum;
  if (unit != 1.f) {  // all of the block: from what it has written
    ss = 0.f;
    for (i = begin + threadIdx.x; i < end; i += EW_THREADS) {
      const float mom = m.momentum[i];
      float u = r.nesterov ? new_momentum(mom, mu, __fmul_rn(load_grad<G>(m.grad, i), s)) : mom;
      u *= 1.f / unit;
      ss += u * u;
    }
    ss = block_sum<EW_THREADS>(ss);
  }
  if (threadIdx.x == 0) {
    r.part[g.part0 + local] = unit == 1.f ? ss : -INFINITY;
    r.piece[g.part0 + local] = make_float2(ss, unit);
  }
}

// x as two halves.
__device__ __forceinline__ void split(float x, __half& hi, __half& lo) {
  hi = __float2half_rn(x);
  lo = __float2half_rn(x - __half2float(hi));
}

// Two of them, a in the lower halves of the words.
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(a, b);
  const float2 f = __half22float2(h);
  const __half2 l = __floats2half2_rn(a - f.x, b - f.y);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  lo = *reinterpret_cast<const uint32_t*>(&l);
}

template <typename G>
__global__ void __launch_bounds__(EW_THREADS)
    muon_layout_kernel(const __grid_constant__ MuonRound r, const __grid_constant__ MuonList l) {
  __shared__ float tile[MUON_TILE][MUON_TILE + 1];
  grid_dependents_go();
  const int gi = group_of(r, blockIdx.x, [](const MuonGroup& g) { return g.tiles0; });
  const MuonGroup& g = r.g[gi];
  const int rows = g.tall ? g.k : g.r, cols = g.tall ? g.r : g.k;  // of the matrix itself
  const int tr = (rows + MUON_TILE - 1) / MUON_TILE, tc = (cols + MUON_TILE - 1) / MUON_TILE;
  int local = blockIdx.x - g.tiles0;
  const int which = local / (tr * tc);
  local -= which * tr * tc;
  const int row0 = local / tc * MUON_TILE, col0 = (local - local / tc * tc) * MUON_TILE;
  const MuonMatrix& m = l.m[g.first + which];
  grid_dependency_wait();
  const int part0 = g.part0 + which * g.parts;
  float2 sum = make_float2(0.f, 1.f);  // and its unit
  for (int i = threadIdx.x; i < g.parts; i += EW_THREADS) sum.x += r.part[part0 + i];
  sum.x = block_sum<EW_THREADS>(sum.x);
  if (!(sum.x >= 0.f)) sum = sum_of_units(r.piece + part0, g.parts);
  const float to = to_x(sum.x, sum.y, r.eps);
  const float s = r.grad_scale_dev ? r.grad_scale * *r.grad_scale_dev : r.grad_scale;
  __half* hi = g.X[0] + (long long)which * 2 * g.r * g.ldk;
  __half* lo = hi + (long long)g.r * g.ldk;
  // A thread has 4 consecutive elements of every 16th row, all of them read before one is used.
  constexpr int ROWS = EW_THREADS / 16, PASSES = MUON_TILE / ROWS;
  const int y0 = threadIdx.x >> 4, x4 = (threadIdx.x & 15) * 4;
  const bool vec = (cols & 3) == 0 && ((uintptr_t)m.momentum & 15) == 0 &&
                   ((uintptr_t)m.grad & 15) == 0;
  float v[PASSES][4], gr[PASSES][4];
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int row = row0 + y0 + i * ROWS, col = col0 + x4;
    const long long at = (long long)row * cols + col;
    if (vec && row < rows && col < cols) {
      const float4 mo = *reinterpret_cast<const float4*>(m.momentum + at);
      v[i][0] = mo.x, v[i][1] = mo.y, v[i][2] = mo.z, v[i][3] = mo.w;
      if (r.nesterov) {
        const float4 q = load_grad4<G>(m.grad, at);
        gr[i][0] = q.x, gr[i][1] = q.y, gr[i][2] = q.z, gr[i][3] = q.w;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bool in = row < rows && col + j < cols;
        v[i][j] = in ? m.momentum[at + j] : 0.f;
        gr[i][j] = in && r.nesterov ? load_grad<G>(m.grad, at + j) : 0.f;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < PASSES; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (r.nesterov) v[i][j] = new_momentum(v[i][j], r.momentum, __fmul_rn(gr[i][j], s));
      v[i][j] *= to;
    }
  if (g.tall) {
#pragma unroll
    for (int i = 0; i < PASSES; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) tile[y0 + i * ROWS][x4 + j] = v[i][j];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < PASSES; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) v[i][j] = tile[x4 + j][y0 + i * ROWS];
  }
  const int xr0 = g.tall ? col0 : row0, xc0 = g.tall ? row0 : col0;  // in X
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int xr = xr0 + y0 + i * ROWS;
    if (xr >= g.r) break;
    uint2 h, w;
    split2(v[i][0], v[i][1], h.x, w.x);
    split2(v[i][2], v[i][3], h.y, w.y);
    // rows are whole multiples of 64 elements long
    const long long at = (long long)xr * g.ldk + xc0 + x4;
    *reinterpret_cast<uint2*>(hi + at) = h;
    *reinterpret_cast<uint2*>(lo + at) = w;
  }
}

// ---------------------------------------------------------------- products

__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ float4 load4(const float* p) {
  return *reinterpret_cast<const float4*>(p);
}
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
  return load_grad4<__nv_bfloat16>(p, 0);
}
__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
}
__device__ __forceinline__ void st_shared_f32(uint32_t addr, float v) {
  asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ float ld_shared_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

struct ProductUnit {
  int g, which, m, n;  // group, matrix in it, tile
};

// A symmetric product's first tile of a row: the one on the diagonal, or (whole: a later product
// reads by pairs' tiles) of the pair's tile around it.
__host__ __device__ __forceinline__ int first_column(int m, bool whole) {
  return whole ? m & ~1 : m;
}

template <int WHAT, int TILE>
__device__ __forceinline__ ProductUnit product_unit(const MuonRound& r, int u) {
  constexpr int PHASE = WHAT < MUON_APPLY ? WHAT : MUON_APPLY;
  ProductUnit p;
  p.g = group_of(r, u, [](const MuonGroup& g) { return g.units0[PHASE]; });
  const MuonGroup& g = r.g[p.g];
  u -= g.units0[PHASE];
  const int per = g.units[PHASE];
  p.which = u / per;
  u -= p.which * per;
  const int t = (g.r + TILE - 1) / TILE;
  if (PHASE != MUON_APPLY) {
    const bool whole = TILE == CTA_ROWS && r.whole[PHASE];
    p.m = 0;
    while (u >= t - first_column(p.m, whole)) {
      u -= t - first_column(p.m, whole);
      ++p.m;
    }
    p.n = first_column(p.m, whole) + u;
  } else {
    p.n = u / t;
    p.m = u - p.n * t;
  }
  return p;
}

// 32 x 32 elements of a matrix from element `at` on, whose updates (times 2^13) a warp's staging
// area holds: four columns of a lane at a time where rows start on them, else one.
constexpr int ROWS_AHEAD = 16;

// (FOURS: all of a round's matrices are so, and the other way is not compiled in: it takes
// registers that the sums need.)
template <typename P, bool FOURS>
__device__ __forceinline__ void update_chunk(const MuonMatrix& m, long long at, int cols,
                                             int rows_left, int cols_left, uint32_t stage0) {
  const int lane = threadIdx.x & 31;
  const float step = m.step * 0x1p-13f, keep = m.keep;
  P* param = static_cast<P*>(m.param) + at;
  __nv_bfloat16* copy = m.copy ? reinterpret_cast<__nv_bfloat16*>(m.copy) + at : nullptr;
  if (FOURS || ((cols & 3) == 0 && ((uintptr_t)param & (4 * sizeof(P) - 1)) == 0 &&
                ((uintptr_t)copy & 7) == 0)) {
    const int row = lane >> 3, c = (lane & 7) * 4;
    if (c >= cols_left) return;
    param += (long long)row * cols + c;
    if (copy) copy += (long long)row * cols + c;
    float4 p[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (4 * i + row < rows_left) p[i] = load4(param + (long long)(4 * i) * cols);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (4 * i + row >= rows_left) break;
      const uint4 x = ld_shared_v4(stage0 + (4 * i + row) * 128 +
                                   (((lane & 7) ^ ((4 * i + row) & 7)) << 4));
      p[i].x = p[i].x * keep - step * __uint_as_float(x.x);
      p[i].y = p[i].y * keep - step * __uint_as_float(x.y);
      p[i].z = p[i].z * keep - step * __uint_as_float(x.z);
      p[i].w = p[i].w * keep - step * __uint_as_float(x.w);
      store4(param + (long long)(4 * i) * cols, p[i]);
      if (copy) store4(copy + (long long)(4 * i) * cols, p[i]);
    }
    return;
  }
  if (FOURS || lane >= cols_left) return;
  param += lane;
  if (copy) copy += lane;
  // a few rows read together, one address from the next: it is the registers that are few
  uint32_t x_row = stage0 + (lane & 3) * 4;
#pragma unroll 1
  for (int i0 = 0; i0 < 32; i0 += ROWS_AHEAD, x_row += ROWS_AHEAD * 128) {
    float p[ROWS_AHEAD];
    const P* from = param;
#pragma unroll
    for (int i = 0; i < ROWS_AHEAD; ++i, from += cols)
      if (i0 + i < rows_left) p[i] = load1(from);
#pragma unroll
    for (int i = 0; i < ROWS_AHEAD; ++i, param += cols) {
      if (i0 + i < rows_left) {
        const float x = ld_shared_f32(x_row + i * 128 + (((lane >> 2) ^ ((i0 + i) & 7)) << 4));
        p[i] = p[i] * keep - step * x;
        store1(param, p[i]);
        if (copy) store1(copy, p[i]);
      }
      if (copy) copy += cols;
    }
  }
}

template <int WHAT, typename P, bool PAIR, bool FOURS>
__global__ void __launch_bounds__(PRODUCT_THREADS, 1)
    muon_product_kernel(const __grid_constant__ MuonRound r, const __grid_constant__ MuonMaps ma,
                        const __grid_constant__ MuonMaps mb, const __grid_constant__ MuonList l,
                        const int from, const int units, int* status) {
  constexpr bool SYMMETRIC = WHAT == MUON_GRAM || WHAT == MUON_POLY;
  constexpr int TILE = tile_of(PAIR), CTAS = PAIR ? 2 : 1;
  constexpr int EPI_COLS = TILE / 2;  // of an epilogue warp
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint64_t* bars =
      reinterpret_cast<uint64_t*>(smem + STAGES * STAGE_BYTES + EPI_WARPS * EPI_BYTES);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + BARS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const uint32_t base = smem_u32(smem), bar0 = smem_u32(bars);
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (STAGES + s); };
  auto tfull_bar = [&](int b) { return bar0 + 8u * (2 * STAGES + b); };
  auto tempty_bar = [&](int b) { return bar0 + 8u * (2 * STAGES + 2 + b); };
  const uint32_t drain_bar = bar0 + 8u * (2 * STAGES + 4);

  grid_dependents_go();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = PAIR ? cluster_ctarank() : 0u;
  const bool leader = rank == 0;
  const int pair = blockIdx.x / CTAS, pairs = gridDim.x / CTAS;  // (or single CTAs)
  // Units come with the longest first, and pairs take them to and fro: who had the longest of
  // one turn has the shortest of the next. (A turn with no unit is a pair's last.)
  auto unit_of = [&](int turn) {
    return turn * pairs + ((turn & 1) ? pairs - 1 - pair : pair);
  };

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull_bar(b), 1);
      mbar_init(tempty_bar(b), CTAS * EPI_WARPS);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    __syncwarp();
    if constexpr (PAIR) {
      tmem_alloc_pair(smem_u32(tmem_slot), 512);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(smem_u32(tmem_slot), 512);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (PAIR) cluster_sync_all();  // the peer's barriers exist before any remote arrive
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  grid_dependency_wait();

  // Which way a K block of the factors lies: of a symmetric one, what is below the diagonal lies
  // across it; the second factor of P X lies along its columns.
  auto a_mn = [](const ProductUnit& u, int kb) {
    return WHAT != MUON_GRAM && kb * KB / TILE < u.m;
  };
  auto b_mn = [](const ProductUnit& u, int kb) {
    return WHAT == MUON_POLY ? kb * KB / TILE < u.n : WHAT != MUON_GRAM;
  };
  auto k_blocks = [&](const ProductUnit& u) {
    return ((WHAT == MUON_GRAM ? r.g[u.g].k : r.g[u.g].r) + KB - 1) / KB;
  };

  if (warp < EPI_WARP0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(FEW_REGS));
    if (warp == 0 && lane == 0) {
      // Both CTAs' copies count on the leader's barrier, which it arms for the two.
      int stage = 0;
      uint32_t phase = 0;
      long long fills = 0;
      bool ok = true;
      const uint32_t full_leader0 = PAIR ? mapa_shared(full_bar(0), 0) : full_bar(0);
      for (int turn = 0; ok && unit_of(turn) < units; ++turn) {
        const ProductUnit u = product_unit<WHAT, TILE>(r, unit_of(turn));
        const int blocks = k_blocks(u);
        const CUtensorMap *ta = &ma.m[u.g], *tb = &mb.m[u.g];
        const int a_row = u.m * TILE + (int)rank * CTA_ROWS;
        const int b_row = u.n * TILE + (int)rank * CTA_ROWS;  // rows of B, or columns (B_MN)
        for (int kb = 0; kb < blocks; ++kb) {
          if (!mbar_wait_bounded(empty_bar(stage), phase ^ 1u, abort_flag, status)) {
            ok = false;
            break;
          }
          if (leader) mbar_arrive_expect_tx(full_bar(stage), (uint32_t)(CTAS * STAGE_BYTES));
          const uint32_t fb = full_leader0 + 8u * stage;
          uint32_t dst = base + stage * STAGE_BYTES;
          const int k = kb * KB;
          auto load = [&](const CUtensorMap* tm, int row, bool mn) {
#pragma unroll
            for (int half = 0; half < 2; ++half)
#pragma unroll
              for (int b = 0; b < 2; ++b, dst += BOX_BYTES) {
                const int x = mn ? row + MUON_BOX * b : k, y = mn ? k : row + MUON_BOX * b;
                if constexpr (PAIR)
                  tma_load_3d_pair(dst, tm, fb, x, y, 2 * u.which + half);
                else
                  tma_load_3d(dst, tm, fb, x, y, 2 * u.which + half);
              }
          };
          load(ta, a_row, a_mn(u, kb));
          load(tb, b_row, b_mn(u, kb));
          ++fills;
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      // Every copy has landed before the CTA ends (the leader's barriers count both CTAs').
      if (leader)
        for (long long f = fills - 1; f >= 0 && f >= fills - STAGES; --f)
          mbar_drain_bounded(full_bar((int)(f % STAGES)), (uint32_t)((f / STAGES) & 1));
    }
    if (warp == 1 && lane == 0 && leader) {
      // (an arrival in every CTA of the tile)
      auto commit = [](uint32_t bar) {
        if constexpr (PAIR)
          tc_commit_pair_multicast(bar, 0x3);
        else
          tc_commit(bar);
      };
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      for (int turn = 0; ok && unit_of(turn) < units; ++turn) {
        const ProductUnit u = product_unit<WHAT, TILE>(r, unit_of(turn));
        const int blocks = k_blocks(u);
        for (int kb = 0; ok && kb < blocks; ++kb) {
          const bool first = kb % MUON_SUM_BLOCKS == 0;
          if (first) {
            const bool freed =
                PAIR ? mbar_wait_cluster_bounded(tempty_bar(acc), acc_phase ^ 1u, abort_flag,
                                                 status, kWaitLimitNs)
                     : mbar_wait_bounded(tempty_bar(acc), acc_phase ^ 1u, abort_flag, status);
            if (!freed) {
              ok = false;
              break;
            }
            tc_fence_after();
          }
          if (!mbar_wait_bounded(full_bar(stage), phase, abort_flag, status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d = tmem_base + (uint32_t)(acc * TILE);
          const uint32_t a0 = base + stage * STAGE_BYTES, b0 = a0 + 2 * HALF_BYTES;
          const bool am = a_mn(u, kb), bm = b_mn(u, kb);
          const uint32_t idesc = idesc_f16_f32(TILE, TILE, am, bm);
          // from one 16 of K to the next, and from one 64 of rows to the next
          const uint32_t a_step = am ? 2048 : 32, a_box = am ? MN_BOX_BYTES : 16;
          const uint32_t b_step = bm ? 2048 : 32, b_box = bm ? MN_BOX_BYTES : 16;
#pragma unroll
          for (int k = 0; k < KB / 16; ++k) {
            auto da = [&](int half) {
              return sdesc_sw128(a0 + half * HALF_BYTES + k * a_step, a_box, 1024);
            };
            auto db = [&](int half) {
              return sdesc_sw128(b0 + half * HALF_BYTES + k * b_step, b_box, 1024);
            };
            auto mma = [&](uint64_t x, uint64_t y, uint32_t more) {
              if constexpr (PAIR)
                tc_mma_bf16_pair(d, x, y, idesc, more);
              else
                tc_mma_bf16(d, x, y, idesc, more);
            };
            mma(da(0), db(0), !first || k != 0 ? 1u : 0u);
            mma(da(0), db(1), 1u);
            mma(da(1), db(0), 1u);
          }
          commit(empty_bar(stage));
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
          if (kb + 1 == blocks || (kb + 1) % MUON_SUM_BLOCKS == 0) {
            commit(tfull_bar(acc));
            acc ^= 1;
            if (acc == 0) acc_phase ^= 1u;
          }
        }
      }
      // All products are done before TMEM is given back.
      if constexpr (PAIR)
        tc_commit_pair_local(drain_bar);
      else
        tc_commit(drain_bar);
      mbar_drain_bounded(drain_bar, 0);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(MANY_REGS));
    const int q = warp & 3, side = (warp - EPI_WARP0) >> 2;
    const uint32_t tmem_mine = tmem_base + ((uint32_t)(q * 32) << 16) + side * EPI_COLS;
    const uint32_t tempty_leader0 = PAIR ? mapa_shared(tempty_bar(0), 0) : 0u;
    const uint32_t stage0 = base + STAGES * STAGE_BYTES + (warp - EPI_WARP0) * EPI_BYTES;
    // Staging: 16-byte piece c of row i lies at piece c ^ (i & 7). A lane's own row, and its
    // place in the passes of 8 rows x 4 pieces in which rows meet memory.
    auto own = [&](int c) { return stage0 + lane * 128 + ((c ^ (lane & 7)) << 4); };
    auto pass = [&](int i, int half) {
      const int row = i * 8 + (lane >> 2);
      return stage0 + row * 128 + (((half * 4 + (lane & 3)) ^ (row & 7)) << 4);
    };
    int acc = 0;
    uint32_t acc_phase = 0;
    bool ok = true;
    for (int turn = 0; ok && unit_of(turn) < units; ++turn) {
      const ProductUnit u = product_unit<WHAT, TILE>(r, unit_of(turn));
      const MuonGroup& g = r.g[u.g];
      const int row0 = u.m * TILE + (int)rank * CTA_ROWS + q * 32;
      const int col0 = u.n * TILE + side * EPI_COLS;
      const int width = SYMMETRIC ? g.r : g.k;
      const int ld = SYMMETRIC ? g.ldr : g.ldk;
      const long long half_at = (long long)g.r * ld;
      const long long matrix = (long long)u.which * 2 * half_at;
      const __half* src = WHAT == MUON_POLY ? g.S + matrix : g.X[from] + matrix;
      __half* dst = WHAT == MUON_GRAM   ? g.S + matrix
                    : WHAT == MUON_POLY ? g.P + matrix
                                        : g.X[1 - from] + matrix;
      // What stands where the product goes, 32 columns ahead of the arithmetic: 8 rows of 4
      // pieces a pass, the high halves' and then the low halves'.
      uint4 in[8];
      auto read_ahead = [&](int c0) {
        if (row0 >= g.r || c0 >= width) return;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int row = row0 + (i & 3) * 8 + (lane >> 2);
          in[i] = make_uint4(0, 0, 0, 0);
          if (row < g.r)
            in[i] = *reinterpret_cast<const uint4*>(src + (i >> 2) * half_at +
                                                    (long long)row * ld + c0 + (lane & 3) * 8);
        }
      };
      if constexpr (WHAT != MUON_GRAM) read_ahead(col0);
      const int sums = (k_blocks(u) + MUON_SUM_BLOCKS - 1) / MUON_SUM_BLOCKS;
      float sum[EPI_COLS];
#pragma unroll
      for (int j = 0; j < EPI_COLS; ++j) sum[j] = 0.f;
      for (int s = 0; ok && s < sums; ++s) {
        if (!mbar_wait_bounded(tfull_bar(acc), acc_phase, abort_flag, status)) {
          ok = false;
          break;
        }
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < EPI_COLS; c += 16) {
          float v[16];
          tmem_ld16(tmem_mine + acc * TILE + c, v);
#pragma unroll
          for (int j = 0; j < 16; ++j) sum[c + j] += v[j];
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if constexpr (PAIR)
            mbar_arrive_cluster_tmem(tempty_leader0 + 8u * acc);
          else
            mbar_arrive(tempty_bar(acc));
        }
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1u;
      }
      if (!ok) break;

#pragma unroll
      for (int cc = 0; cc < EPI_COLS; cc += 32) {
        const int c0 = col0 + cc;
        if (row0 >= g.r || c0 >= width) continue;  // uniform over the warp
        float v[32];
        if constexpr (WHAT == MUON_GRAM) {
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = sum[cc + j] * 0x1p-13f;
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) st_shared_v4(pass(i & 3, i >> 2), in[i]);
          __syncwarp();
          if (cc + 32 < EPI_COLS) read_ahead(c0 + 32);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const uint4 hi4 = ld_shared_v4(own(c)), lo4 = ld_shared_v4(own(4 + c));
            const uint32_t hw[4] = {hi4.x, hi4.y, hi4.z, hi4.w};
            const uint32_t lw[4] = {lo4.x, lo4.y, lo4.z, lo4.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&hw[j]));
              const float2 w = __half22float2(*reinterpret_cast<const __half2*>(&lw[j]));
              const float x[2] = {h.x + w.x, h.y + w.y};
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int at = 8 * c + 2 * j + e;
                v[at] = WHAT == MUON_POLY
                            ? fmaf(QUINTIC_B * 0x1p-2f, x[e], QUINTIC_C * 0x1p-15f * sum[cc + at])
                            : fmaf(QUINTIC_A, x[e], 0x1p-11f * sum[cc + at]);
              }
            }
          }
          __syncwarp();
        }
        if (WHAT != MUON_UPDATE) {
          uint32_t hw[16], lw[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) split2(v[2 * j], v[2 * j + 1], hw[j], lw[j]);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            st_shared_v4(own(c), make_uint4(hw[4 * c], hw[4 * c + 1], hw[4 * c + 2], hw[4 * c + 3]));
            st_shared_v4(own(4 + c),
                         make_uint4(lw[4 * c], lw[4 * c + 1], lw[4 * c + 2], lw[4 * c + 3]));
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int row = row0 + (i & 3) * 8 + (lane >> 2);
            const uint4 o = ld_shared_v4(pass(i & 3, i >> 2));
            if (row < g.r)
              *reinterpret_cast<uint4*>(dst + (i >> 2) * half_at + (long long)row * ld + c0 +
                                        (lane & 3) * 8) = o;
          }
          __syncwarp();
        } else {
          // The chunk as the parameters lie, rows of 32 columns, in the staging area.
          if (g.tall) {  // their rows are X's columns
#pragma unroll
            for (int j = 0; j < 32; ++j)
              st_shared_f32(stage0 + j * 128 + (((lane >> 2) ^ (j & 7)) << 4) + (lane & 3) * 4, v[j]);
          } else {
#pragma unroll
            for (int c = 0; c < 8; ++c)
              st_shared_v4(own(c), make_uint4(__float_as_uint(v[4 * c]), __float_as_uint(v[4 * c + 1]),
                                              __float_as_uint(v[4 * c + 2]),
                                              __float_as_uint(v[4 * c + 3])));
          }
          __syncwarp();
          const int rows_left = g.tall ? g.k - c0 : g.r - row0;
          const int cols_left = g.tall ? g.r - row0 : g.k - c0;
          const long long at = g.tall ? (long long)c0 * g.r + row0 : (long long)row0 * g.k + c0;
          update_chunk<P, FOURS>(l.m[g.first + u.which], at, g.tall ? g.r : g.k, rows_left, cols_left,
                          stage0);
          __syncwarp();
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (PAIR) cluster_sync_all();  // the leader's products into the peer's TMEM are done
  tc_fence_after();
  if (warp == 1) {
    __syncwarp();
    if constexpr (PAIR)
      tmem_dealloc_pair(tmem_base, 512);
    else
      tmem_dealloc(tmem_base, 512);
  }
}

// ------------------------------------------------------------ small matrices
//
// A matrix of at most 128 x 256 (or its transpose) fits an SM: a block takes one through
// the whole step in one launch, X and S as halves in shared memory, each product one
// accumulator. X's blocks of 64 columns are the first factors' layout (K-major) of S = X X^T and,
// read the other way, the second factor's (MN-major) of P X. 14 matrices of 96 x 96 and
// 96 x 250 take 61 us so and 226 by the launches above, each of which waits for its
// tiles' loads, products and stores one after the other.

constexpr int SMALL_THREADS = 512;
constexpr int SMALL_BATCH = 16;  // elements that a thread reads together
constexpr int SMALL_BLOCK = 128 * 128;      // bytes of a block of 64 columns
constexpr int SMALL_X_HALF = 4 * SMALL_BLOCK, SMALL_S_HALF = 2 * SMALL_BLOCK;
constexpr int SMALL_S = 2 * SMALL_X_HALF;
constexpr int SMALL_SMEM = SMALL_S + 2 * SMALL_S_HALF + 64 + 1024;

// 16-byte piece `p` of a row in a block of 64 columns.
__device__ __forceinline__ uint32_t small_piece(uint32_t block, int row, int p) {
  return block + row * 128 + ((p ^ (row & 7)) << 4);
}
__device__ __forceinline__ __half ld_shared_half(uint32_t addr) {
  unsigned short h;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(h) : "r"(addr) : "memory");
  return __ushort_as_half(h);
}
__device__ __forceinline__ void st_shared_half(uint32_t addr, __half h) {
  asm volatile("st.shared.u16 [%0], %1;" ::"r"(addr), "h"(__half_as_ushort(h)) : "memory");
}
template <typename G, typename P>
__global__ void __launch_bounds__(SMALL_THREADS, 1)
    muon_small_kernel(const __grid_constant__ MuonSmall a, int* status) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint64_t* bar_at = reinterpret_cast<uint64_t*>(smem + SMALL_S + 2 * SMALL_S_HALF);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar_at + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const uint32_t X = smem_u32(smem), S = X + SMALL_S, bar = smem_u32(bar_at);
  grid_dependents_go();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    mbar_init(bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    __syncwarp();
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_dependency_wait();

  const MuonMatrix& m = a.m[blockIdx.x];
  const int rows = a.rows[blockIdx.x], cols = a.cols[blockIdx.x];
  const bool tall = rows > cols;
  const int r = tall ? cols : rows, k = tall ? rows : cols;
  const int r16 = (r + 15) & ~15, k16 = (k + 15) & ~15;
  const float s = a.grad_scale_dev ? a.grad_scale * *a.grad_scale_dev : a.grad_scale;
  // X's zeros, up to whole 16s and more
  for (int i = threadIdx.x; i < 2 * SMALL_X_HALF / 16; i += SMALL_THREADS)
    st_shared_v4(X + 16 * i, make_uint4(0, 0, 0, 0));
  // A warp has every 16th row of the matrix, 32 columns of it at a time, SMALL_BATCH of those read
  // together: loops, for code that runs once is waited for.
  const int chunks = (cols + 31) / 32;
  const int places = (rows + SMALL_THREADS / 32 - 1) / (SMALL_THREADS / 32) * chunks;
  struct Place {
    int row, col;
  };
  auto next = [&](Place& p) {
    p.col += 32;
    if (p.col - lane >= cols) {
      p.col = lane;
      p.row += SMALL_THREADS / 32;
    }
  };
  auto in = [&](const Place& p) { return p.row < rows && p.col < cols; };
  auto index = [&](const Place& p) { return p.row * cols + p.col; };
  const Place start{warp, lane};
  // momentum, and the sum of squares
  SquareSum squares;
  Place at = start;
#pragma unroll 1
  for (int b = 0; b < places; b += SMALL_BATCH) {
    float gr[SMALL_BATCH], mom[SMALL_BATCH];
    Place read = at;
#pragma unroll
    for (int j = 0; j < SMALL_BATCH; ++j, next(read)) {
      gr[j] = in(read) ? load_grad<G>(m.grad, index(read)) : 0.f;
      mom[j] = in(read) ? m.momentum[index(read)] : 0.f;
    }
#pragma unroll
    for (int j = 0; j < SMALL_BATCH; ++j, next(at)) {
      const float gs = __fmul_rn(gr[j], s);
      mom[j] = new_momentum(mom[j], a.momentum, gs);
      if (in(at)) m.momentum[index(at)] = mom[j];
      squares.add(a.nesterov ? new_momentum(mom[j], a.momentum, gs) : mom[j]);
    }
  }
  const float unit = squares.over_block<SMALL_THREADS>();  // (X's zeros are there)
  float ss = squares.sum;
  if (unit != 1.f) {  // all of the block: from what it has written
    ss = 0.f;
    for (int i = threadIdx.x; i < rows * cols; i += SMALL_THREADS) {
      const float mom = m.momentum[i];
      float u = a.nesterov ? new_momentum(mom, a.momentum, __fmul_rn(load_grad<G>(m.grad, i), s)) : mom;
      u *= 1.f / unit;
      ss += u * u;
    }
    ss = block_sum<SMALL_THREADS>(ss);
  }
  const float to = to_x(ss, unit, a.eps);
  auto x_of = [&](const Place& p) {
    const int row = tall ? p.col : p.row, col = tall ? p.row : p.col;
    return small_piece(X + (col >> 6) * SMALL_BLOCK, row, (col & 63) >> 3) + (col & 7) * 2;
  };
  at = start;
#pragma unroll 1
  for (int b = 0; b < places; b += SMALL_BATCH) {
    float gr[SMALL_BATCH], mom[SMALL_BATCH];
    Place read = at;
#pragma unroll
    for (int j = 0; j < SMALL_BATCH; ++j, next(read)) {  // what this thread wrote
      gr[j] = in(read) && a.nesterov ? load_grad<G>(m.grad, index(read)) : 0.f;
      mom[j] = in(read) ? m.momentum[index(read)] : 0.f;
    }
#pragma unroll
    for (int j = 0; j < SMALL_BATCH; ++j, next(at)) {
      if (!in(at)) continue;
      const float u = a.nesterov ? new_momentum(mom[j], a.momentum, __fmul_rn(gr[j], s)) : mom[j];
      __half hi, lo;
      split(u * to, hi, lo);
      st_shared_half(x_of(at), hi);
      st_shared_half(x_of(at) + SMALL_X_HALF, lo);
    }
  }

  // rows of a warp's quarter of the accumulator, and a quarter of its columns
  const int row = (warp & 3) * 32 + lane, side = warp >> 2;
  const uint32_t tmem_row = tmem + ((uint32_t)((warp & 3) * 32) << 16);
  uint32_t phase = 0;
  bool ok = true;
  // D = first second^T (K-major) or first second (MN-major), three products of halves
  auto product = [&](uint32_t first, uint32_t first_half, uint32_t second, uint32_t second_half,
                     bool mn, int columns, int depth) {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0) {
      tc_fence_after();
      const uint32_t idesc = idesc_f16_f32(128, columns, false, mn);
      for (int t = 0; t < depth / 16; ++t) {
        const uint32_t fa = first + (t >> 2) * SMALL_BLOCK + (t & 3) * 32;
        const uint32_t fb = mn ? second + t * 2048 : second + (t >> 2) * SMALL_BLOCK + (t & 3) * 32;
        const uint32_t lbo = mn ? SMALL_BLOCK : 16;
        const uint64_t ah = sdesc_sw128(fa, 16, 1024), al = sdesc_sw128(fa + first_half, 16, 1024);
        const uint64_t bh = sdesc_sw128(fb, lbo, 1024), bl = sdesc_sw128(fb + second_half, lbo, 1024);
        tc_mma_bf16(tmem, ah, bh, idesc, t != 0 ? 1u : 0u);
        tc_mma_bf16(tmem, ah, bl, idesc, 1u);
        tc_mma_bf16(tmem, al, bh, idesc, 1u);
      }
      tc_commit(bar);
    }
    ok = __syncthreads_and(mbar_wait_bounded(bar, phase, abort_flag, status)) != 0;
    phase ^= 1u;
    tc_fence_after();
    return ok;
  };
  // This thread's row of the accumulator, 32 columns from c on, into a matrix of halves:
  // f(accumulator, what stood there), zero outside rows x columns.
  auto replace = [&](uint32_t block, uint32_t half, int c, int columns, bool old, auto f) {
    float v[32];
    tmem_ld32(tmem_row + c, v);
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const uint32_t at = small_piece(block, row, ((c & 63) >> 3) + p);
      float x[8] = {};
      if (old) {
        const uint4 h4 = ld_shared_v4(at), l4 = ld_shared_v4(at + half);
        const uint32_t hw[4] = {h4.x, h4.y, h4.z, h4.w}, lw[4] = {l4.x, l4.y, l4.z, l4.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&hw[j]));
          const float2 l = __half22float2(*reinterpret_cast<const __half2*>(&lw[j]));
          x[2 * j] = h.x + l.x;
          x[2 * j + 1] = h.y + l.y;
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = f(v[8 * p + j], x[j]);
      if (row >= r || c + 8 * p + 8 > columns) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (row >= r || c + 8 * p + j >= columns) x[j] = 0.f;
      }
      uint4 hi, lo;
      split2(x[0], x[1], hi.x, lo.x);
      split2(x[2], x[3], hi.y, lo.y);
      split2(x[4], x[5], hi.z, lo.z);
      split2(x[6], x[7], hi.w, lo.w);
      st_shared_v4(at, hi);
      st_shared_v4(at + half, lo);
    }
  };
  for (int step = 0; step < a.steps; ++step) {
    if (!product(X, SMALL_X_HALF, X, SMALL_X_HALF, false, r16, k16)) break;
    int c = side * 32;
    if (c < r16)
      replace(S + (c >> 6) * SMALL_BLOCK, SMALL_S_HALF, c, r, false,
              [](float d, float) { return d * 0x1p-13f; });
    if (!product(S, SMALL_S_HALF, S, SMALL_S_HALF, false, r16, r16)) break;
    if (c < r16)
      replace(S + (c >> 6) * SMALL_BLOCK, SMALL_S_HALF, c, r, true, [](float d, float x) {
        return fmaf(QUINTIC_B * 0x1p-2f, x, QUINTIC_C * 0x1p-15f * d);
      });
    if (!product(S, SMALL_S_HALF, X, SMALL_X_HALF, true, k16, r16)) break;
    for (c = side * 64; c < side * 64 + 64; c += 32)
      if (c < k16)
        replace(X + side * SMALL_BLOCK, SMALL_X_HALF, c, k, true,
                [](float d, float x) { return fmaf(QUINTIC_A, x, 0x1p-11f * d); });
  }
  tc_fence_before();
  __syncthreads();
  if (ok) {
    const float step = m.step * 0x1p-13f, keep = m.keep;
    P* param = static_cast<P*>(m.param);
    __nv_bfloat16* copy = reinterpret_cast<__nv_bfloat16*>(m.copy);
    at = start;
#pragma unroll 1
    for (int b = 0; b < places; b += SMALL_BATCH) {
      float p[SMALL_BATCH];
      Place read = at;
#pragma unroll
      for (int j = 0; j < SMALL_BATCH; ++j, next(read))
        p[j] = in(read) ? load1(param + index(read)) : 0.f;
#pragma unroll
      for (int j = 0; j < SMALL_BATCH; ++j, next(at)) {
        if (!in(at)) continue;
        const float x = __half2float(ld_shared_half(x_of(at))) +
                        __half2float(ld_shared_half(x_of(at) + SMALL_X_HALF));
        p[j] = p[j] * keep - step * x;
        store1(param + index(at), p[j]);
        if (copy) store1(copy + index(at), p[j]);
      }
    }
  }
  __syncthreads();
  tc_fence_after();
  if (warp == 0) {
    __syncwarp();
    tmem_dealloc(tmem, 512);
  }
}

constexpr int kMaxDevices = 64;

template <int WHAT, typename P, bool PAIR, bool FOURS>
cudaError_t launch_product(const char* name, const MuonRound& r, const MuonList& l, int from,
                           const MuonMaps& a, const MuonMaps& b, int units, int* status,
                           int num_sms, cudaStream_t stream) {
  auto kern = muon_product_kernel<WHAT, P, PAIR, FOURS>;
  constexpr unsigned ctas = PAIR ? 2 : 1;
  // Pairs (or CTAs) that fit on the device at once, and the shared-memory limit raised (per
  // device; concurrent first calls set the same).
  static std::atomic<int> known[kMaxDevices] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  int most = known[dev].load(std::memory_order_acquire);
  if (most == 0) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, PRODUCT_SMEM);
    if (e != cudaSuccess) return e;
    most = num_sms;
    if (PAIR) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(2);
      cfg.blockDim = dim3(PRODUCT_THREADS);
      cfg.dynamicSmemBytes = PRODUCT_SMEM;
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = 2;
      attr[0].val.clusterDim.y = 1;
      attr[0].val.clusterDim.z = 1;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      if ((e = cudaOccupancyMaxActiveClusters(&most, kern, &cfg)) != cudaSuccess) return e;
      if (most < 1) return cudaErrorInvalidConfiguration;
      most = std::min(most, num_sms / 2);
    }
    known[dev].store(most, std::memory_order_release);
  }
  return launch_kernel_cluster(name, kern, dim3(ctas * std::min(units, most)),
                               dim3(PRODUCT_THREADS), (size_t)PRODUCT_SMEM, stream, ctas, true, r,
                               a, b, l, from, units, status);
}

template <bool PAIR>
cudaError_t launch_product_of(MuonProduct what, const MuonRound& r, const MuonList& l, int from,
                              const MuonMaps& a, const MuonMaps& b, bool param_bf16, int units,
                              int* status, int num_sms, cudaStream_t stream) {
  switch (what) {
    case MUON_GRAM:
      return launch_product<MUON_GRAM, float, PAIR, true>("muon_gram", r, l, from, a, b, units, status,
                                                    num_sms, stream);
    case MUON_POLY:
      return launch_product<MUON_POLY, float, PAIR, true>("muon_poly", r, l, from, a, b, units, status,
                                                    num_sms, stream);
    case MUON_APPLY:
      return launch_product<MUON_APPLY, float, PAIR, true>("muon_apply", r, l, from, a, b, units, status,
                                                     num_sms, stream);
    case MUON_UPDATE: {
      auto go = [&](auto launch) {
        return launch("muon_update", r, l, from, a, b, units, status, num_sms, stream);
      };
      using bf16 = __nv_bfloat16;
      if (r.fours)
        return param_bf16 ? go(launch_product<MUON_UPDATE, bf16, PAIR, true>)
                          : go(launch_product<MUON_UPDATE, float, PAIR, true>);
      return param_bf16 ? go(launch_product<MUON_UPDATE, bf16, PAIR, false>)
                        : go(launch_product<MUON_UPDATE, float, PAIR, false>);
    }
  }
  return cudaErrorInvalidValue;
}

template <typename G, typename P>
cudaError_t launch_small(const MuonSmall& a, int count, int* status, cudaStream_t stream) {
  auto kern = muon_small_kernel<G, P>;
  static std::atomic<bool> done[kMaxDevices] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  if (!done[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMALL_SMEM);
    if (e != cudaSuccess) return e;
    done[dev].store(true, std::memory_order_release);
  }
  return launch_kernel_early("muon_small", kern, dim3(count), dim3(SMALL_THREADS),
                             (size_t)SMALL_SMEM, stream, a, status);
}

}  // namespace

cudaError_t launch_muon_small(const MuonSmall& a, int count, bool grad_bf16, bool param_bf16,
                              int* status, cudaStream_t stream) {
  using bf16 = __nv_bfloat16;
  if (grad_bf16)
    return param_bf16 ? launch_small<bf16, bf16>(a, count, status, stream)
                      : launch_small<bf16, float>(a, count, status, stream);
  return param_bf16 ? launch_small<float, bf16>(a, count, status, stream)
                    : launch_small<float, float>(a, count, status, stream);
}

int muon_units(int r, int k, MuonProduct what, bool pair, bool whole) {
  const int tile = tile_of(pair), t = (r + tile - 1) / tile;
  if (what >= MUON_APPLY) return t * ((k + tile - 1) / tile);
  int n = 0;
  for (int m = 0; m < t; ++m) n += t - first_column(m, whole && !pair);
  return n;
}

// Cycles of a product over groups of matrices, but for what either tile takes: turns of the
// tiles' K blocks. One takes a pair 1536 cycles (12 instructions of 128) and a single CTA 1157 for
// a quarter of the tile (its instructions wait for shared memory: 768 of their own); the last
// tile's way out is 5 us longer for a pair. Products of 4 matrices of 2000 x 2000: 129 us by
// pairs and 162; of 14 of 700 x 700: 36 and 28; of one of 512 x 512: 24 and 17.
double muon_cost(const MuonGroup* g, int n_groups, MuonProduct what, bool pair, bool whole,
                 int num_sms) {
  double units = 0, blocks = 0;
  for (int i = 0; i < n_groups; ++i) {
    const double n = (double)g[i].count * muon_units(g[i].r, g[i].k, what, pair, whole);
    units += n;
    blocks += n * (((what == MUON_GRAM ? g[i].k : g[i].r) + KB - 1) / KB);
  }
  const double turns = ceil(units / (pair ? num_sms / 2 : num_sms));
  return turns * (blocks / units) * (pair ? 1536 : 1157) + (pair ? 9000 : 0);
}

cudaError_t launch_muon_momentum(const MuonRound& r, const MuonList& l, bool grad_bf16, int blocks,
                                 cudaStream_t stream) {
  auto kern = grad_bf16 ? muon_momentum_kernel<__nv_bfloat16> : muon_momentum_kernel<float>;
  return launch_kernel_early("muon_momentum", kern, dim3(blocks), dim3(EW_THREADS), 0, stream, r, l);
}

cudaError_t launch_muon_layout(const MuonRound& r, const MuonList& l, bool grad_bf16, int blocks,
                               cudaStream_t stream) {
  auto kern = grad_bf16 ? muon_layout_kernel<__nv_bfloat16> : muon_layout_kernel<float>;
  return launch_kernel_early("muon_layout", kern, dim3(blocks), dim3(EW_THREADS), 0, stream, r, l);
}

cudaError_t launch_muon_product(MuonProduct what, const MuonRound& r, const MuonList& l, int from,
                                const MuonMaps& a, const MuonMaps& b, bool param_bf16, bool pair,
                                int units, int* status, int num_sms, cudaStream_t stream) {
  return pair ? launch_product_of<true>(what, r, l, from, a, b, param_bf16, units, status, num_sms,
                                        stream)
              : launch_product_of<false>(what, r, l, from, a, b, param_bf16, units, status, num_sms,
                                         stream);
}

}  // namespace kdkl
