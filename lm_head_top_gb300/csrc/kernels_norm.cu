// Layer and RMS norm of rows with the residual sum before it, and the way back.
//
//   h = x + r,  n = (h - mean) rstd   (RMS: mean = 0)
//   y = n w + b
//   g = dy w,  dx = rstd (g - n avg(g n) - avg(g)) + dh     (RMS: without avg(g))
//   dw = sum over rows of dy n,  db = sum over rows of dy  (RMS: no b)
//
// Rows are read and written 16 bytes at a time wherever the arrays start on 16
// bytes: a row that does not itself shares its first and last vector with its
// neighbours, and a block takes rows of one remainder alone (RowWalk).
//
// A row lies in the registers of its threads from its one read to its one write:
// of a warp where a lane holds at most 4 vectors (backward: one), else of a block. The
// variance is the mean square of h - mean, a second sum over registers (the
// difference of two large sums would lose what a row's mean has beyond its
// spread). Sums are fp32, over threads by shuffles in a fixed order.
//
// A block takes row after row and has the next ones under way meanwhile, in
// shared memory (RowRing). Products and sums are made two at a time (f32x2): the
// backward at d = 2880, bf16, was held up by its instructions (204 us with one at a
// time and rows read when they are needed, 123 now: 6.1 TB/s, 0.92 of a plain copy).
//
// Backward: a thread keeps its columns from row to row, so the sums over rows
// stay in its registers; every block leaves one row of them, and a second launch
// adds those up in their order: no atomics, the same bits every time. fp32 sums of
// the few hundred rows of a block and of the blocks' are off by some 1e-7.
//
// What bounds it: DRAM. 4 rows of d elements are read and written either way with
// a residual.
#include <algorithm>
#include <atomic>

#include "kdkl_body.h"
#include "rows.cuh"
#include "tc_primitives.cuh"

namespace kdkl {

namespace {

constexpr int NORM_WARPS = 8;       // rows of a block whose rows are warps'
constexpr int NORM_SUM_ROWS = 32;   // of the block that adds up partial sums
constexpr int KIND_LAYER = 0;       // KD_NORM_LAYER
// Rows of a block in shared memory. At d = 2880, bf16, three in the forward and two in the
// backward are 35 to 70 KB in flight on an SM.
constexpr int PLACES_FORWARD = 3, PLACES_BACKWARD = 2;
// Forward: rows of a block, at most, where a row is a block's. Blocks that come and go even
// out what SMs differ by: 32,768 rows of 2880 bf16 take 113 us so, and 120 to 150 (by their
// number) with blocks that stay.
constexpr int ROWS_FORWARD = 8;
// Backward: each block leaves a row of sums, so blocks stay. Threads on an SM: 123 us at 1160,
// 141 at 770. Fewer rows than this in a block only where there are not two blocks an SM.
constexpr int THREADS_BACKWARD = 1160, ROWS_BACKWARD = 8;
constexpr int NORM_MAX_PER_SM = 16;  // blocks
constexpr int NORM_RING_SMEM = 152 * 1024, NORM_BLOCK_SMEM = 216 * 1024;
constexpr int kMaxDevices = 64;

// Sums of N values over the row's threads, in every one of them. `red`: 2 buffers of 32 * N
// floats, zero where a block has no warp, taken in turn, so that one barrier a call is enough.
// Every thread adds up the warps' sums for itself, from broadcasts (shuffles once more would
// be a longer chain).
template <int N, bool WARP>
__device__ __forceinline__ void row_sum(float (&v)[N], float* red, int& turn) {
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  if (WARP) return;
  const int warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  float* buf = red + turn * 32 * N;
  turn ^= 1;
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) buf[i * 32 + warp] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = 0.f;
  for (int w = 0; w < warps; w += 4)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float4 q = *reinterpret_cast<const float4*>(buf + i * 32 + w);
      v[i] += (q.x + q.y) + (q.z + q.w);
    }
}

template <int N>
__device__ __forceinline__ void clear_row_sum(float* red) {
  for (int i = threadIdx.x; i < 2 * 32 * N; i += blockDim.x) red[i] = 0.f;
  __syncthreads();
}

// A row's weights (or bias, or `none` where there is none) as floats in shared memory, where its
// threads have the columns that they have of a row: 4 floats of every thread, then their next 4
// (one with VEC = 1). Where they do not fit they are read from memory again for every row.
template <int VEC, bool EDGES, int VPT>
struct RowWeights {
  static constexpr int UNIT = VEC < 4 ? 1 : 4;
  float* to;
  const void* from;
  int bf16, width, lane;
  float none;
  __device__ __forceinline__ float one(const RowSpan<VEC, EDGES>& sp, int j) const {
    if (!from || !sp.some() || !sp.in(j)) return none;
    return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(from)[sp.c + j])
                : static_cast<const float*>(from)[sp.c + j];
  }
  __device__ __forceinline__ void put(int i, const RowSpan<VEC, EDGES>& sp) const {
    if (!to) return;
#pragma unroll
    for (int j = 0; j < VEC; ++j)
      to[((i * VEC + j) / UNIT * width + lane) * UNIT + j % UNIT] = one(sp, j);
  }
  __device__ __forceinline__ void get(int i, const RowSpan<VEC, EDGES>& sp, float (&w)[VEC]) const {
    if (!to) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) w[j] = one(sp, j);
      return;
    }
#pragma unroll
    for (int j = 0; j < VEC; j += UNIT) {
      const float* at = to + ((i * VEC + j) / UNIT * width + lane) * UNIT;
      if constexpr (UNIT == 4) {
        const float4 q = *reinterpret_cast<const float4*>(at);
        w[j] = q.x, w[j + 1] = q.y, w[j + 2] = q.z, w[j + 3] = q.w;
      } else {
        w[j] = *at;
      }
    }
  }
};

// The rows of a thread: from `first` on, up to `end`. Where rows do not start on 16 bytes, every
// classes-th does so with the same remainder, and a block keeps to rows of one class: its
// vectors' columns stay the same. A block has rows that follow one another (in the
// backward 8 % faster than rows a grid apart).
struct RowWalk {
  long long first, end;
  int stride;
  int shift;  // elements of a row's first vector that lie before it
  template <typename T, bool WARP>
  static __device__ __forceinline__ RowWalk of(const NormArgs& a) {
    const int warps = WARP ? blockDim.x >> 5 : 1, me = WARP ? threadIdx.x >> 5 : 0;
    const int cls = blockIdx.x % a.classes, block = blockIdx.x / a.classes;
    const int blocks = gridDim.x / a.classes;
    // a class's rows, evenly over its blocks, in whole turns of a block's warps
    const long long rows = (a.T - cls + a.classes - 1) / a.classes;
    const long long per = ((rows + blocks - 1) / blocks + warps - 1) / warps * warps;
    RowWalk w;
    w.first = cls + a.classes * (block * per + me);
    w.end = min((long long)a.T, cls + a.classes * (block + 1) * per);
    w.stride = a.classes * warps;
    w.shift = (int)(((long long)cls * a.d * (int)sizeof(T)) & 15) / (int)sizeof(T);
    return w;
  }
};

template <typename T, bool LAYER, int VEC, bool EDGES, int VPT, bool WARP, int THREADS>
__global__ void __launch_bounds__(THREADS) norm_forward_kernel(const NormArgs a, const int places, const int w_smem) {
  __shared__ __align__(16) float red[2 * 32];
  extern __shared__ uint4 norm_smem[];
  const int per_row = WARP ? 32 : blockDim.x;
  const int lane = WARP ? threadIdx.x & 31 : threadIdx.x;
  const RowWalk walk = RowWalk::of<T, WARP>(a);
  const RowRing<T, VEC, EDGES, VPT, 2> ring(smem_u32(norm_smem), blockDim.x, places);
  auto span = [&](int i) {
    return RowSpan<VEC, EDGES>{(i * per_row + lane) * VEC - (EDGES ? walk.shift : 0), a.d};
  };
  float* floats = w_smem ? reinterpret_cast<float*>(norm_smem) +
                               places * ring.place_bytes(blockDim.x) / 4
                         : nullptr;
  const RowWeights<VEC, EDGES, VPT> weight{floats, a.weight, a.w_bf16, per_row, lane, 1.f};
  const RowWeights<VEC, EDGES, VPT> bias{floats ? floats + VPT * VEC * per_row : nullptr, a.bias,
                                         a.w_bf16, per_row, lane, 0.f};
  const T* x = static_cast<const T*>(a.x);
  const T* res = static_cast<const T*>(a.residual);
  T *y = static_cast<T*>(a.y), *h = static_cast<T*>(a.h);
  int turn = 0;
  auto fetch = [&](long long row, int place) {
    if (row < walk.end) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const RowSpan<VEC, EDGES> sp = span(i);
        if (sp.some()) {
          const long long at = row * a.d + sp.c;
          ring.copy(place, 0, i, x + at, sp.upto() * (int)sizeof(T));
          if (res) ring.copy(place, 1, i, res + at, sp.upto() * (int)sizeof(T));
        }
      }
    }
    ring.commit();
  };
  if (!WARP) clear_row_sum<1>(red);
  grid_dependents_go();
  grid_dependency_wait();
  for (int p = 0; p + 1 < places; ++p) fetch(walk.first + (long long)p * walk.stride, p);
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    if (a.weight) weight.put(i, span(i));
    if (LAYER && a.bias) bias.put(i, span(i));
  }
  if (WARP) __syncthreads();  // the warps' are the same
  int place = 0;
  for (long long row = walk.first; row < walk.end; row += walk.stride) {
    fetch(row + (long long)(places - 1) * walk.stride, place == 0 ? places - 1 : place - 1);
    ring.wait();
    const long long at = row * a.d;
    float v[VPT][VEC], part[VEC], s[1];
    row_fill(part, 0.f);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const RowSpan<VEC, EDGES> sp = span(i);
      row_fill(v[i], 0.f);
      if (sp.some()) {
        ring.get(place, 0, i, x + at + sp.c, sp, v[i]);
        if (res) {
          float t[VEC];
          ring.get(place, 1, i, res + at + sp.c, sp, t);
          row_add(v[i], v[i], t);
          sp.store(h + at, v[i]);
          RowVec<T, VEC> kept;  // what is normed is the sum as it is kept
          kept.set(v[i]);
          kept.get(v[i]);
        }
        if (LAYER)
          row_add(part, part, v[i]);
        else
          row_fma(part, v[i], v[i], part);
      }
    }
    s[0] = row_total(part);
    row_sum<1, WARP>(s, red, turn);
    float mean = 0.f;
    if (LAYER) {
      mean = s[0] / a.width;  // not times 1 / d: a constant row is its own mean
      float less[VEC];
      row_fill(less, -mean);
      row_fill(part, 0.f);
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const RowSpan<VEC, EDGES> sp = span(i);
        if (sp.some()) {
          row_add(v[i], v[i], less);
          sp.mask(v[i]);
          row_fma(part, v[i], v[i], part);
        }
      }
      s[0] = row_total(part);
      row_sum<1, WARP>(s, red, turn);
    }
    const float rstd = 1.f / sqrtf(s[0] / a.width + a.eps);
    if (lane == 0) {
      if (LAYER && a.mean_out) a.mean_out[row] = mean;
      if (a.rstd_out) a.rstd_out[row] = rstd;
    }
    float r[VEC];
    row_fill(r, rstd);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const RowSpan<VEC, EDGES> sp = span(i);
      if (sp.some()) {
        float w[VEC];
        row_mul(v[i], v[i], r);
        if (a.weight) {
          weight.get(i, sp, w);
          row_mul(v[i], v[i], w);
        }
        if (LAYER && a.bias) {
          bias.get(i, sp, w);
          row_add(v[i], v[i], w);
        }
        sp.store(y + at, v[i]);
      }
    }
    place = place + 1 == places ? 0 : place + 1;
  }
}

// Where the compiler, left alone, takes 127 registers for what 64 hold as well: layer norms of fp32
// rows off 16 bytes. Of more than 256 threads an SM then has one block: 32,768 x 2877 takes 376 us
// and not 315. (Fewer threads gain nothing: 32,768 x 1001 takes 103 us and, with 64 registers, 110.)
template <typename T, bool LAYER, bool EDGES>
constexpr bool two_blocks(int vpt, bool warp, int threads) {
  return sizeof(T) == 4 && LAYER && EDGES && vpt == 1 && !warp && threads > 256;
}

template <typename T, bool LAYER, int VEC, bool EDGES, int VPT, bool WARP, int THREADS>
__global__ void __launch_bounds__(THREADS, two_blocks<T, LAYER, EDGES>(VPT, WARP, THREADS) ? 2 : 0)
    norm_backward_kernel(const NormArgs a, const int places, const int w_smem) {
  constexpr int SUMS = LAYER ? 2 : 1;
  __shared__ __align__(16) float red[2 * 32 * SUMS];
  __shared__ float sums[WARP ? 2 * 32 * VEC : 1];
  extern __shared__ uint4 norm_smem[];
  constexpr bool KEEP = VPT * VEC <= 16;  // n and g stay in registers
  const int per_row = WARP ? 32 : blockDim.x;
  const int lane = WARP ? threadIdx.x & 31 : threadIdx.x;
  const RowWalk walk = RowWalk::of<T, WARP>(a);
  const RowRing<T, VEC, EDGES, VPT, 3> ring(smem_u32(norm_smem), blockDim.x, places);
  const RowWeights<VEC, EDGES, VPT> weights{
      w_smem ? reinterpret_cast<float*>(norm_smem) + places * ring.place_bytes(blockDim.x) / 4
             : nullptr,
      a.weight, a.w_bf16, per_row, lane, 1.f};
  auto span = [&](int i) {
    return RowSpan<VEC, EDGES>{(i * per_row + lane) * VEC - (EDGES ? walk.shift : 0), a.d};
  };
  const T *x = static_cast<const T*>(a.x), *dy = static_cast<const T*>(a.dy);
  const T* dh = static_cast<const T*>(a.dh);
  T* dx = static_cast<T*>(a.dx);
  int turn = 0;
  float dw[VPT][VEC], db[LAYER ? VPT : 1][VEC];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    row_fill(dw[i], 0.f);
    if (LAYER) row_fill(db[i], 0.f);
  }
  auto fetch = [&](long long row, int place) {
    if (row < walk.end) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const RowSpan<VEC, EDGES> sp = span(i);
        if (sp.some()) {
          const long long at = row * a.d + sp.c;
          const int bytes = sp.upto() * (int)sizeof(T);
          ring.copy(place, 0, i, x + at, bytes);
          ring.copy(place, 1, i, dy + at, bytes);
          if (dh) ring.copy(place, 2, i, dh + at, bytes);
        }
      }
    }
    ring.commit();
  };
  if (!WARP) clear_row_sum<SUMS>(red);
  grid_dependents_go();
  grid_dependency_wait();
  for (int p = 0; p + 1 < places; ++p) fetch(walk.first + (long long)p * walk.stride, p);
  if (a.weight)
#pragma unroll
    for (int i = 0; i < VPT; ++i) weights.put(i, span(i));
  if (WARP) __syncthreads();  // the warps' are the same
  const float inv_d = 1.f / a.width;
  int place = 0;
  float mean = 0.f, rstd = 0.f;
  if (walk.first < walk.end) {
    if (LAYER) mean = a.mean[walk.first];
    rstd = a.rstd[walk.first];
  }
  for (long long row = walk.first; row < walk.end; row += walk.stride) {
    fetch(row + (long long)(places - 1) * walk.stride, place == 0 ? places - 1 : place - 1);
    float next_mean = 0.f, next_rstd = 0.f;
    if (row + walk.stride < walk.end) {
      if (LAYER) next_mean = a.mean[row + walk.stride];
      next_rstd = a.rstd[row + walk.stride];
    }
    ring.wait();
    const long long at = row * a.d;
    float n[KEEP ? VPT : 1][VEC], g[KEEP ? VPT : 1][VEC];
    float r[VEC], less[VEC], part[VEC], part2[VEC], s[SUMS];
    row_fill(r, rstd);
    row_fill(less, -mean);
    row_fill(part, 0.f);
    row_fill(part2, 0.f);
    // n and g of vector i, in n[k] and g[k]
    auto terms = [&](int i, int k, const RowSpan<VEC, EDGES>& sp, bool first) {
      ring.get(place, 0, i, x + at + sp.c, sp, n[k]);
      ring.get(place, 1, i, dy + at + sp.c, sp, g[k]);
      if (LAYER) row_add(n[k], n[k], less);
      row_mul(n[k], n[k], r);
      if (first) {
        row_fma(dw[i], g[k], n[k], dw[i]);
        if (LAYER) row_add(db[LAYER ? i : 0], db[LAYER ? i : 0], g[k]);
      }
      if (a.weight) {
        float w[VEC];
        weights.get(i, sp, w);
        row_mul(g[k], g[k], w);
      }
      if (first) {
        row_fma(part, g[k], n[k], part);
        if (LAYER) row_add(part2, part2, g[k]);
      }
    };
#pragma unroll
    for (int i = 0; i < VPT; ++i)
      if (span(i).some()) terms(i, KEEP ? i : 0, span(i), true);
    s[0] = row_total(part);
    if (LAYER) s[SUMS - 1] = row_total(part2);
    row_sum<SUMS, WARP>(s, red, turn);
    // dx = g rstd - n (along rstd) - avg rstd + dh
    row_fill(part, -(s[0] * inv_d * rstd));
    if (LAYER) row_fill(part2, -(s[SUMS - 1] * inv_d * rstd));
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const RowSpan<VEC, EDGES> sp = span(i);
      const int k = KEEP ? i : 0;
      if (sp.some()) {
        if (!KEEP) terms(i, k, sp, false);  // once more: all of them would be too many registers
        row_mul(n[k], n[k], part);
        row_fma(g[k], g[k], r, n[k]);
        if (LAYER) row_add(g[k], g[k], part2);
        if (dh) {
          float t[VEC];
          ring.get(place, 2, i, dh + at + sp.c, sp, t);
          row_add(g[k], g[k], t);
        }
        sp.store(dx + at, g[k]);
      }
    }
    mean = next_mean;
    rstd = next_rstd;
    place = place + 1 == places ? 0 : place + 1;
  }
  if (!a.part) return;
  float* out = a.part + (long long)blockIdx.x * 2 * a.d;
  if constexpr (WARP) {  // the block's warps in their order
    for (int c = threadIdx.x; c < 2 * 32 * VEC; c += blockDim.x) sums[c] = 0.f;
    for (int w = 0; w < (int)blockDim.x >> 5; ++w) {
      __syncthreads();
      if ((threadIdx.x >> 5) != w) continue;
      const RowSpan<VEC, EDGES> sp = span(0);  // one vector a lane
#pragma unroll
      for (int j = 0; j < VEC; ++j)
        if (sp.some() && sp.in(j)) {
          sums[sp.c + j] += dw[0][j];
          if (LAYER) sums[a.d + sp.c + j] += db[0][j];
        }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < (LAYER ? 2 : 1) * a.d; c += blockDim.x) out[c] = sums[c];
  } else {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const RowSpan<VEC, EDGES> sp = span(i);
#pragma unroll
      for (int j = 0; j < VEC; ++j)
        if (sp.some() && sp.in(j)) {
          out[sp.c + j] = dw[i][j];
          if (LAYER) out[a.d + sp.c + j] = db[i][j];
        }
    }
  }
}

// dweight and dbias from the blocks' rows: 32 columns a block, its warps take every
// NORM_SUM_ROWS-th row, and then their sums are added in order. (It clears the status word too,
// which nothing here sets: in the rows' kernel that store took 52 registers to 58, a block less on
// an SM, and 32,768 x 2880 from 122 us to 133.)
__global__ void __launch_bounds__(32 * NORM_SUM_ROWS)
    norm_weight_sum_kernel(const float* __restrict__ part, int rows, int d, float* dweight,
                           float* dbias, int accumulate, int* status) {
  __shared__ float got[NORM_SUM_ROWS][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;  // of 2 d
  const bool here = c < 2 * d;
  grid_dependency_wait();
  if (c == 0) *status = DEV_OK;
  float s = 0.f;
  if (here)
#pragma unroll 8
    for (int r = warp; r < rows; r += NORM_SUM_ROWS) s += part[(long long)r * 2 * d + c];
  got[warp][lane] = s;
  __syncthreads();
  if (warp != 0 || !here) return;
#pragma unroll
  for (int w = 1; w < NORM_SUM_ROWS; ++w) s += got[w][lane];
  float* to = c < d ? dweight : dbias;
  if (!to) return;
  const int at = c < d ? c : c - d;
  to[at] = accumulate ? to[at] + s : s;
}

// How a row is laid over threads. Forward: a lane of a warp holds up to 4 vectors, a
// thread of a block as few as 1024 threads allow. Backward: one and two, for the sums over
// rows take registers too.
struct RowPlan {
  bool warp;
  int vpt, threads;
};

RowPlan plan_row(int d, int vec, int classes, bool backward) {
  const int vectors = vec == 1 ? d : (d + (classes > 1 ? 7 : 0) + 7) / 8;
  RowPlan p;
  p.warp = vectors <= (backward ? 32 : 128);
  if (p.warp) {
    p.vpt = vectors <= 32 ? 1 : vectors <= 64 ? 2 : 4;
    p.threads = 32 * NORM_WARPS;
    return p;
  }
  p.vpt = vec == 8 ? (vectors <= 512 ? 1 : vectors <= 1024 ? 2 : 4)
                   : vectors <= 1024 ? 2 : vectors <= 4096 ? 4 : 16;
  p.threads = ((vectors + p.vpt - 1) / p.vpt + 31) / 32 * 32;
  return p;
}

// Blocks that T rows are enough for, whole ones of every class, and at most `most` otherwise.
int row_blocks(const RowPlan& p, int T, int classes, int most) {
  const long long rows = (p.warp ? p.threads / 32 : 1) * classes;
  const long long n = std::min(((long long)T + rows - 1) / rows, (long long)(most / classes));
  return classes * (int)std::max(1ll, n);
}

// Rows that a block has in shared memory, `bytes` each.
int ring_places(int bytes, int most) {
  return bytes == 0 ? 1 : std::max(1, std::min(most, NORM_RING_SMEM / bytes));
}

int backward_most(const RowPlan& p, int T, int num_sms) {
  const int per_sm = std::max(1, std::min(NORM_MAX_PER_SM, THREADS_BACKWARD / p.threads));
  const int rows = ROWS_BACKWARD * (p.warp ? p.threads / 32 : 1);
  return std::min(per_sm * num_sms, std::max(2 * num_sms, T / rows));
}

// What is found once for a kernel and device (concurrent first calls find the same): that it may
// have more than 48 KB of shared memory, and, by a block's threads, on which the shared memory
// depends, how many blocks an SM holds at once.
struct KernelFacts {
  std::atomic<bool> allowed;
  std::atomic<int> blocks[33];
};

// Blocks that an SM holds, which a grid is a multiple of (a last block that waits for the others to
// end would be a round of its own).
template <typename K>
cudaError_t resident(K kern, KernelFacts* facts, int threads, int smem, int* blocks) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  KernelFacts& f = facts[dev];
  if (!f.allowed.load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, NORM_BLOCK_SMEM);
    if (e != cudaSuccess) return e;
    f.allowed.store(true, std::memory_order_release);
  }
  std::atomic<int>& k = f.blocks[threads / 32];
  *blocks = k.load(std::memory_order_acquire);
  if (*blocks > 0) return cudaSuccess;
  int n = 0;
  e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, threads, smem);
  if (e != cudaSuccess) return e;
  *blocks = std::max(1, std::min(n, NORM_MAX_PER_SM));
  k.store(*blocks, std::memory_order_release);
  return cudaSuccess;
}

template <typename T, bool LAYER, int VEC, bool EDGES, int VPT, bool WARP, int THREADS>
cudaError_t forward(const RowPlan& p, const NormArgs& a, int num_sms, cudaStream_t stream) {
  auto kern = norm_forward_kernel<T, LAYER, VEC, EDGES, VPT, WARP, THREADS>;
  static KernelFacts facts[kMaxDevices] = {};
  const int bytes = RowRing<T, VEC, EDGES, VPT, 2>::place_bytes(p.threads);
  const int places = ring_places(bytes, PLACES_FORWARD);
  const int w_bytes = (LAYER ? 2 : 1) * VPT * VEC * 4 * (WARP ? 32 : p.threads);
  const int w_smem = places * bytes + w_bytes <= NORM_BLOCK_SMEM;
  const int smem = places * bytes + (w_smem ? w_bytes : 0);
  int per_sm = 0;
  cudaError_t e = resident(kern, facts, p.threads, smem, &per_sm);
  if (e != cudaSuccess) return e;
  int most = per_sm * num_sms;
  if (!WARP) most = std::max(most, a.T / ROWS_FORWARD);
  const int grid = row_blocks(p, a.T, a.classes, most);
  return launch_kernel_early("norm_forward", kern, dim3(grid), dim3(p.threads),
                             (size_t)smem, stream, a, places, w_smem);
}

template <typename T, bool LAYER, int VEC, bool EDGES, int VPT, bool WARP, int THREADS>
cudaError_t backward(const RowPlan& p, const NormArgs& a, int num_sms, cudaStream_t stream) {
  auto kern = norm_backward_kernel<T, LAYER, VEC, EDGES, VPT, WARP, THREADS>;
  static KernelFacts facts[kMaxDevices] = {};
  const int bytes = RowRing<T, VEC, EDGES, VPT, 3>::place_bytes(p.threads);
  const int places = ring_places(bytes, PLACES_BACKWARD);
  const int w_bytes = VPT * VEC * 4 * (WARP ? 32 : p.threads);
  const int w_smem = places * bytes + w_bytes <= NORM_BLOCK_SMEM;
  const int smem = places * bytes + (w_smem ? w_bytes : 0);
  int per_sm = 0;
  cudaError_t e = resident(kern, facts, p.threads, smem, &per_sm);
  if (e != cudaSuccess) return e;
  const int most = std::min(backward_most(p, a.T, num_sms), per_sm * num_sms);
  const int grid = row_blocks(p, a.T, a.classes, most);
  e = launch_kernel_early("norm_backward", kern, dim3(grid), dim3(p.threads),
                          (size_t)smem, stream, a, places, w_smem);
  if (e != cudaSuccess || !a.part) return e;
  return launch_kernel_early("norm_weight_sum", norm_weight_sum_kernel,
                             dim3(((LAYER ? 2 : 1) * a.d + 31) / 32), dim3(32 * NORM_SUM_ROWS), 0,
                             stream, (const float*)a.part, grid, a.d, a.dweight, a.dbias,
                             a.accumulate, a.status);
}

template <typename T, bool LAYER>
cudaError_t pick_forward(const NormArgs& a, int num_sms, cudaStream_t stream) {
  const RowPlan p = plan_row(a.d, a.vec ? 8 : 1, a.classes, false);
  const bool edges = a.vec && a.d % 8 != 0;
#define KD_ROW(VEC, EDGES, VPT, WARP, THREADS)                                                    \
  if ((a.vec ? 8 : 1) == VEC && edges == EDGES && p.vpt == VPT && p.warp == WARP)                 \
    return forward<T, LAYER, VEC, EDGES, VPT, WARP, THREADS>(p, a, num_sms, stream);
  KD_ROW(8, false, 1, true, 256)
  KD_ROW(8, false, 2, true, 256)
  KD_ROW(8, false, 4, true, 256)
  KD_ROW(8, false, 1, false, 512)
  KD_ROW(8, false, 2, false, 512)
  KD_ROW(8, true, 1, true, 256)
  KD_ROW(8, true, 2, true, 256)
  KD_ROW(8, true, 4, true, 256)
  KD_ROW(8, true, 1, false, 512)
  KD_ROW(8, true, 2, false, 512)
  KD_ROW(8, false, 4, false, 576)
  KD_ROW(8, true, 4, false, 576)
  KD_ROW(1, false, 1, true, 256)
  KD_ROW(1, false, 2, true, 256)
  KD_ROW(1, false, 4, true, 256)
  KD_ROW(1, false, 2, false, 512)
  KD_ROW(1, false, 4, false, 1024)
  KD_ROW(1, false, 16, false, 1024)
#undef KD_ROW
  return cudaErrorInvalidValue;
}

template <typename T, bool LAYER>
cudaError_t pick_backward(const NormArgs& a, int num_sms, cudaStream_t stream) {
  const RowPlan p = plan_row(a.d, a.vec ? 8 : 1, a.classes, true);
  const bool edges = a.vec && a.d % 8 != 0;
#define KD_ROW(VEC, EDGES, VPT, WARP, THREADS)                                                    \
  if ((a.vec ? 8 : 1) == VEC && edges == EDGES && p.vpt == VPT && p.warp == WARP)                 \
    return backward<T, LAYER, VEC, EDGES, VPT, WARP, THREADS>(p, a, num_sms, stream);
  KD_ROW(8, false, 1, true, 256)
  KD_ROW(8, false, 1, false, 512)
  KD_ROW(8, false, 2, false, 512)
  KD_ROW(8, true, 1, true, 256)
  if constexpr (two_blocks<T, LAYER, true>(1, false, 512)) {
    if (p.threads <= 256) KD_ROW(8, true, 1, false, 256)
  }
  KD_ROW(8, true, 1, false, 512)
  KD_ROW(8, true, 2, false, 512)
  KD_ROW(8, false, 4, false, 576)
  KD_ROW(8, true, 4, false, 576)
  KD_ROW(1, false, 1, true, 256)
  KD_ROW(1, false, 2, false, 512)
  KD_ROW(1, false, 4, false, 1024)
  KD_ROW(1, false, 16, false, 1024)
#undef KD_ROW
  return cudaErrorInvalidValue;
}

}  // namespace

int norm_backward_blocks(int T, int d, int num_sms) {
  int most = 0;
  for (int vec : {1, 8})
    for (int classes : {1, 2, 4, 8}) {
      if (vec == 1 && classes > 1) continue;
      const RowPlan p = plan_row(d, vec, classes, true);
      most = std::max(most, row_blocks(p, T, classes, backward_most(p, T, num_sms)));
    }
  return most;
}

cudaError_t launch_norm_forward(const NormArgs& a, bool rows_bf16, int num_sms,
                                cudaStream_t stream) {
  if (a.kind == KIND_LAYER)
    return rows_bf16 ? pick_forward<__nv_bfloat16, true>(a, num_sms, stream)
                     : pick_forward<float, true>(a, num_sms, stream);
  return rows_bf16 ? pick_forward<__nv_bfloat16, false>(a, num_sms, stream)
                   : pick_forward<float, false>(a, num_sms, stream);
}

cudaError_t launch_norm_backward(const NormArgs& a, bool rows_bf16, int num_sms,
                                 cudaStream_t stream) {
  if (a.kind == KIND_LAYER)
    return rows_bf16 ? pick_backward<__nv_bfloat16, true>(a, num_sms, stream)
                     : pick_backward<float, true>(a, num_sms, stream);
  return rows_bf16 ? pick_backward<__nv_bfloat16, false>(a, num_sms, stream)
                   : pick_backward<float, false>(a, num_sms, stream);
}

}  // namespace kdkl
