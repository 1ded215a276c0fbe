// C ABI of what a head's body needs in training: embedding, norms, the Muon
// step. Argument checks, workspace plans and launches.
#include <math.h>
#include <string.h>

#include <algorithm>
#include <mutex>

#include "kdkl.h"
#include "kdkl_body.h"

namespace kdkl {
namespace {

constexpr size_t kHeader = 256;  // int status
// Bound on the SM count that sizes workspaces (the same with and without a device).
constexpr int kMaxSms = 256;
constexpr int64_t kMaxRows = (1ll << 31) - 4096;
constexpr int64_t kMaxMatrix = 65536;  // rows or columns
// Matrices of one round of launches: what fits in this (one at least), in rounds of like size.
// Above some ten tiles an SM pair a launch's start and end are a few per cent of it.
constexpr size_t kRoundBytes = 3ull << 30;

inline size_t pad256(size_t x) { return (x + 255) & ~(size_t)255; }
inline bool aligned_to(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
bool fits32(double x) { return isfinite((float)x); }

template <typename T>
T* place(void* ws, size_t off) {
  return reinterpret_cast<T*>(static_cast<char*>(ws) + off);
}

// -------------------------------------------------------------- embedding

struct EmbedLayout {
  size_t off_met, off_pairs[2], off_hist, off_part, total;
};
EmbedLayout embed_layout(const kd_embedding_problem& p, int which) {
  EmbedLayout L{};
  size_t o = kHeader;
  if (which == 1) {
    L.off_met = o;
    o += pad256((size_t)(p.V + 31) / 32 * 4);
    for (int i = 0; i < 2; ++i) {
      L.off_pairs[i] = o;
      o += pad256((size_t)p.T * 8);
    }
    L.off_hist = o;
    o += pad256(embed_sort_bytes((int)p.T));
    L.off_part = o;
    const size_t pieces = ((size_t)p.T + EMBED_PIECE - 1) / EMBED_PIECE;
    o += pad256(pieces * 2 * (size_t)p.d * 4);
  }
  L.total = o;
  return L;
}

kd_status embed_check(const kd_embedding_problem* p) {
  if (!p) return KD_ERR_INVALID_ARG;
  if (p->T < 0 || p->T >= kMaxRows || p->V < 1 || p->V >= kMaxRows || p->d < 1 ||
      p->d > (1ll << 20))
    return KD_ERR_SHAPE;
  // thread blocks of a launch in 31 bits: of 8 warps with 128 elements each, in the forward
  if (p->T * p->d >= (1ll << 40)) return KD_ERR_SHAPE;
  if (!isfinite(p->scale)) return KD_ERR_INVALID_ARG;
  return KD_OK;
}

// ------------------------------------------------------------------- norm

kd_status norm_check(const kd_norm_problem* p) {
  if (!p) return KD_ERR_INVALID_ARG;
  if (p->T < 0 || p->T >= kMaxRows || p->d < 1 || p->d > NORM_MAX_D) return KD_ERR_SHAPE;
  if (!(p->eps >= 0.0) || !fits32(p->eps)) return KD_ERR_INVALID_ARG;
  if (p->kind != KD_NORM_LAYER && p->kind != KD_NORM_RMS) return KD_ERR_INVALID_ARG;
  return KD_OK;
}

// Rows that start at different places within 16 bytes.
int row_classes(int d, int element) {
  int n = 1;
  while (n * d * element % 16 != 0) n *= 2;
  return n;
}

size_t norm_bytes(const kd_norm_problem& p) {
  return kHeader + pad256((size_t)norm_backward_blocks((int)p.T, (int)p.d, kMaxSms) * 2 *
                          (size_t)p.d * 4);
}

// ------------------------------------------------------------------- Muon

// A map of fp16 matrices [outer][rows][columns] for copies of 64 x 64 boxes, 128-byte swizzle;
// what lies outside reads as zero.
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn g_encode_boxes = nullptr;
std::once_flag g_encode_boxes_once;

bool encode_f16_boxes(CUtensorMap* tm, const void* base, uint64_t columns, uint64_t rows,
                      uint64_t outer, uint64_t ld) {
  std::call_once(g_encode_boxes_once, [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      g_encode_boxes = reinterpret_cast<EncodeTiledFn>(fn);
  });
  if (!g_encode_boxes) return false;
  cuuint64_t dims[3] = {columns, rows, outer};
  cuuint64_t strides[2] = {ld * 2, rows * ld * 2};
  cuuint32_t box[3] = {MUON_BOX, MUON_BOX, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return g_encode_boxes(tm, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(base), dims,
                        strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Which matrices, from `begin` on, are worked on together, and where what they need lies.
struct RoundPlan {
  int end, n_groups;
  int group_of[MUON_LIST];  // of matrix begin + i
  MuonGroup g[MUON_GROUPS];
  size_t off[MUON_GROUPS], x_bytes[MUON_GROUPS], s_bytes[MUON_GROUPS];  // of a matrix
  int64_t rows[MUON_GROUPS], cols[MUON_GROUPS];
  size_t off_piece, total;
};

int round64(int64_t x) { return (int)((x + 63) / 64 * 64); }

// Bytes that a matrix's X, twice, S and P take.
size_t matrix_bytes(const kd_muon_matrix& m) {
  const int64_t r = std::min(m.rows, m.cols), k = std::max(m.rows, m.cols);
  return (size_t)r * (size_t)(round64(k) + round64(r)) * 8;
}

// Bytes after which a round is full: the list's in as few rounds as kRoundBytes allows.
size_t round_bytes(const kd_muon_matrix* m, int n) {
  size_t all = 0;
  for (int i = 0; i < n; ++i) all += matrix_bytes(m[i]);
  return all / std::max<size_t>(1, (all + kRoundBytes - 1) / kRoundBytes);
}

void plan_round(const kd_muon_matrix* m, int n, int begin, size_t full, RoundPlan* plan) {
  RoundPlan& p = *plan;
  p.n_groups = 0;
  size_t bytes = 0;
  int i = begin;
  for (; i < n && i - begin < MUON_LIST; ++i) {
    int g = 0;
    while (g < p.n_groups && (p.rows[g] != m[i].rows || p.cols[g] != m[i].cols)) ++g;
    if (g == MUON_GROUPS) break;
    const int64_t r = std::min(m[i].rows, m[i].cols), k = std::max(m[i].rows, m[i].cols);
    const size_t x = (size_t)r * round64(k) * 4, s = (size_t)r * round64(r) * 4;
    if (i > begin && (bytes >= full || bytes + matrix_bytes(m[i]) > kRoundBytes)) break;
    bytes += matrix_bytes(m[i]);
    if (g == p.n_groups) {
      ++p.n_groups;
      p.rows[g] = m[i].rows;
      p.cols[g] = m[i].cols;
      p.x_bytes[g] = x;
      p.s_bytes[g] = s;
      MuonGroup& q = p.g[g];
      q = MuonGroup{};
      q.r = (int)r;
      q.k = (int)k;
      q.ldk = round64(k);
      q.ldr = round64(r);
      q.tall = m[i].rows > m[i].cols;
      q.parts = (int)((r * k + MUON_CHUNK - 1) / MUON_CHUNK);
    }
    ++p.g[g].count;
    p.group_of[i - begin] = g;
  }
  p.end = i;
  size_t o = kHeader, parts = 0;
  for (int g = 0; g < p.n_groups; ++g) parts += (size_t)p.g[g].parts * p.g[g].count;
  p.off_piece = o + pad256(parts * sizeof(float));
  o = p.off_piece + pad256(parts * sizeof(float2));
  for (int g = 0; g < p.n_groups; ++g) {
    p.off[g] = o;
    o += 2 * pad256(p.x_bytes[g] * p.g[g].count) + 2 * pad256(p.s_bytes[g] * p.g[g].count);
  }
  p.total = o;
}

kd_status muon_sizes(const kd_muon_matrix* m, int n) {
  if (n < 0 || (n > 0 && !m)) return KD_ERR_INVALID_ARG;
  for (int i = 0; i < n; ++i)
    if (m[i].rows < 1 || m[i].rows > kMaxMatrix || m[i].cols < 1 || m[i].cols > kMaxMatrix)
      return KD_ERR_SHAPE;
  return KD_OK;
}

// Whether all matrices are small: a block each, in one launch. Beside others they go with
// these, whose launches they fill (4 of 192 x 192 and 3 of 83 x 192: 190 us apart, 135 together).
bool all_small(const kd_muon_matrix* m, int n) {
  for (int i = 0; i < n; ++i)
    if (!muon_is_small(m[i].rows, m[i].cols)) return false;
  return true;
}

size_t muon_bytes(const kd_muon_matrix* m, int n) {
  size_t most = kHeader;
  if (all_small(m, n)) return most;
  RoundPlan p;
  const size_t full = round_bytes(m, n);
  for (int at = 0; at < n; at = p.end) {
    plan_round(m, n, at, full, &p);
    most = std::max(most, p.total);
  }
  return most;
}

// A matrix as the kernels take it.
MuonMatrix muon_matrix(const kd_muon_matrix& m, const kd_muon_options& o) {
  MuonMatrix x{};
  x.param = m.param;
  x.grad = m.grad;
  x.momentum = m.momentum;
  x.copy = m.copy;
  const double rows = (double)m.rows, cols = (double)m.cols;
  const double scale = o.scale == KD_MUON_SPECTRAL ? sqrt(std::max(1.0, rows / cols))
                                                   : 0.2 * sqrt(std::max(rows, cols));
  x.step = (float)(o.lr * scale);
  x.keep = m.decay ? (float)(1.0 - o.lr * o.weight_decay) : 1.f;
  return x;
}

kd_status muon_small(const kd_muon_matrix* m, int n, const kd_muon_options& o, int* status,
                     cudaStream_t stream) {
  MuonSmall a{};
  a.momentum = (float)o.momentum;
  a.eps = (float)o.eps;
  a.grad_scale = o.grad_scale;
  a.grad_scale_dev = o.grad_scale_dev;
  a.nesterov = o.nesterov != 0;
  a.steps = o.steps;
  int count = 0;
  for (int i = 0; i <= n; ++i) {
    if (count == MUON_LIST || (i == n && count > 0)) {
      if (launch_muon_small(a, count, o.grad_bf16 != 0, o.param_bf16 != 0, status, stream) !=
          cudaSuccess)
        return KD_ERR_CUDA;
      count = 0;
    }
    if (i == n) break;
    a.m[count] = muon_matrix(m[i], o);
    a.rows[count] = (unsigned short)m[i].rows;
    a.cols[count++] = (unsigned short)m[i].cols;
  }
  return KD_OK;
}

kd_status muon_round(const kd_muon_matrix* m, int begin, RoundPlan& p, const kd_muon_options& o, void* ws,
                     int num_sms, cudaStream_t stream) {
  MuonRound r{};
  MuonList l{};
  MuonMaps maps[4] = {};  // X[0], X[1], S, P
  r.n_groups = p.n_groups;
  r.momentum = (float)o.momentum;
  r.eps = (float)o.eps;
  r.grad_scale = o.grad_scale;
  r.grad_scale_dev = o.grad_scale_dev;
  r.nesterov = o.nesterov != 0;
  r.part = place<float>(ws, kHeader);
  r.piece = place<float2>(ws, p.off_piece);
  // the groups with the longest products first: their tiles are handed out in this order
  int order[MUON_GROUPS];
  for (int g = 0; g < p.n_groups; ++g) {
    int at = g;
    auto before = [&](const MuonGroup& a, const MuonGroup& b) {
      return a.r != b.r ? a.r > b.r : a.k > b.k;
    };
    for (; at > 0 && before(p.g[g], p.g[order[at - 1]]); --at) order[at] = order[at - 1];
    order[at] = g;
  }
  // the products' tiles: the cheapest of the eight ways
  bool pair[3] = {true, true, true};
  // Whether product w stores the blocks around the diagonal whole: where a later one of the same
  // symmetric factor has pairs' tiles. (P's tiles read S at their own places too.)
  auto whole = [](const bool* by, int w) {
    return (w < MUON_POLY && by[MUON_POLY]) || (w < MUON_APPLY && by[MUON_APPLY]);
  };
  double least = 0;
  for (int way = 0; way < 8; ++way) {
    const bool by[3] = {(way & 1) != 0, (way & 2) != 0, (way & 4) != 0};
    double cost = 0;
    for (int w = MUON_GRAM; w <= MUON_APPLY; ++w)
      cost += muon_cost(p.g, p.n_groups, (MuonProduct)w, by[w], whole(by, w), num_sms);
    if (way == 0 || cost <= least) {
      least = cost;
      std::copy(by, by + 3, pair);
    }
  }
  for (int w = MUON_GRAM; w <= MUON_POLY; ++w) r.whole[w] = whole(pair, w);
  int first = 0, part0 = 0, blocks = 0, tiles = 0, units[3] = {0, 0, 0}, next[MUON_GROUPS];
  for (int i = 0; i < p.n_groups; ++i) {
    MuonGroup& g = r.g[i];
    const int from = order[i];
    g = p.g[from];
    g.first = next[from] = first;
    first += g.count;
    g.part0 = part0;
    part0 += g.parts * g.count;
    g.blocks0 = blocks;
    blocks += g.parts * g.count;
    g.tiles0 = tiles;
    const int rows = g.tall ? g.k : g.r, cols = g.tall ? g.r : g.k;
    tiles += (rows + MUON_TILE - 1) / MUON_TILE * ((cols + MUON_TILE - 1) / MUON_TILE) * g.count;
    for (int w = MUON_GRAM; w <= MUON_APPLY; ++w) {
      g.units0[w] = units[w];
      g.units[w] = muon_units(g.r, g.k, (MuonProduct)w, pair[w], whole(pair, w));
      units[w] += g.units[w] * g.count;
    }
    const size_t x = pad256(p.x_bytes[from] * g.count), s = pad256(p.s_bytes[from] * g.count);
    g.X[0] = place<__half>(ws, p.off[from]);
    g.X[1] = place<__half>(ws, p.off[from] + x);
    g.S = place<__half>(ws, p.off[from] + 2 * x);
    g.P = place<__half>(ws, p.off[from] + 2 * x + s);
    const bool ok =
        encode_f16_boxes(&maps[0].m[i], g.X[0], g.k, g.r, 2ull * g.count, g.ldk) &&
        encode_f16_boxes(&maps[1].m[i], g.X[1], g.k, g.r, 2ull * g.count, g.ldk) &&
        encode_f16_boxes(&maps[2].m[i], g.S, g.r, g.r, 2ull * g.count, g.ldr) &&
        encode_f16_boxes(&maps[3].m[i], g.P, g.r, g.r, 2ull * g.count, g.ldr);
    if (!ok) return KD_ERR_CUDA;
  }
  r.fours = 1;
  for (int i = begin; i < p.end; ++i) {
    const kd_muon_matrix& x = m[i];
    l.m[next[p.group_of[i - begin]]++] = muon_matrix(x, o);
    if (x.cols % 4 != 0 || !aligned_to(x.param, o.param_bf16 ? 8 : 16) || !aligned_to(x.copy, 8))
      r.fours = 0;
  }
  int* status = place<int>(ws, 0);
  const bool g16 = o.grad_bf16 != 0, p16 = o.param_bf16 != 0;
  cudaError_t e = launch_muon_momentum(r, l, g16, blocks, stream);
  if (e == cudaSuccess) e = launch_muon_layout(r, l, g16, tiles, stream);
  for (int s = 0; s < o.steps && e == cudaSuccess; ++s) {
    const MuonMaps& X = maps[s & 1];
    auto product = [&](MuonProduct what, int w, const MuonMaps& a, const MuonMaps& b) {
      if (e == cudaSuccess)
        e = launch_muon_product(what, r, l, s & 1, a, b, p16, pair[w], units[w], status, num_sms,
                                stream);
    };
    product(MUON_GRAM, MUON_GRAM, X, X);
    product(MUON_POLY, MUON_POLY, maps[2], maps[2]);
    product(s + 1 < o.steps ? MUON_APPLY : MUON_UPDATE, MUON_APPLY, maps[3], X);
  }
  return e == cudaSuccess ? KD_OK : KD_ERR_CUDA;
}

}  // namespace
}  // namespace kdkl

using namespace kdkl;

extern "C" {

size_t kd_embedding_workspace_size(const kd_embedding_problem* prob, int which) {
  if (embed_check(prob) != KD_OK || which < 0 || which > 1) return 0;
  return embed_layout(*prob, which).total;
}

kd_status kd_embedding_forward(const kd_embedding_problem* prob, const void* W, const int32_t* ids,
                               const uint8_t* mask, void* Y, void* workspace,
                               size_t workspace_bytes, void* stream_ptr) {
  kd_status st = embed_check(prob);
  if (st != KD_OK) return st;
  const kd_embedding_problem& p = *prob;
  if (workspace && workspace_bytes < embed_layout(p, 0).total) return KD_ERR_WORKSPACE;
  if (p.T > 0 && (!W || !ids || !Y)) return KD_ERR_INVALID_ARG;
  if (!aligned_to(W, p.table_bf16 ? 2 : 4) || !aligned_to(ids, 4) ||
      !aligned_to(Y, p.rows_bf16 ? 2 : 4) || !aligned_to(workspace, 16))
    return KD_ERR_ALIGNMENT;
  int sms = 0;
  if ((st = (kd_status)current_device(&sms)) != KD_OK) return st;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
  if (workspace) forget_forward(workspace);
  if (p.T == 0 && !workspace) return KD_OK;
  if (p.T == 0)
    return cudaMemsetAsync(workspace, 0, kHeader, stream) == cudaSuccess ? KD_OK : KD_ERR_CUDA;
  EmbedArgs a{};
  a.W = W;
  a.ids = ids;
  a.mask = mask;
  a.Y = Y;
  a.T = (int)p.T;
  a.d = (int)p.d;
  a.V = (int)p.V;
  a.vec = p.d % 8 == 0 && aligned_to(W, 16) && aligned_to(Y, 16);
  a.scale = p.scale;
  a.status = static_cast<int*>(workspace);
  return launch_embedding_forward(a, p.table_bf16 != 0, p.rows_bf16 != 0, stream) == cudaSuccess
             ? KD_OK
             : KD_ERR_CUDA;
}

kd_status kd_embedding_backward(const kd_embedding_problem* prob, const void* dY,
                                const int32_t* ids, const uint8_t* mask, float* dW,
                                int accumulate_dW, void* workspace, size_t workspace_bytes,
                                void* stream_ptr) {
  kd_status st = embed_check(prob);
  if (st != KD_OK) return st;
  const kd_embedding_problem& p = *prob;
  const EmbedLayout L = embed_layout(p, 1);
  if (!workspace || workspace_bytes < L.total) return KD_ERR_WORKSPACE;
  if (!dW || (p.T > 0 && (!dY || !ids))) return KD_ERR_INVALID_ARG;
  if (!aligned_to(dY, p.rows_bf16 ? 2 : 4) || !aligned_to(ids, 4) || !aligned_to(dW, 4) ||
      !aligned_to(workspace, 16))
    return KD_ERR_ALIGNMENT;
  int sms = 0;
  if ((st = (kd_status)current_device(&sms)) != KD_OK) return st;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
  forget_forward(workspace);
  if (p.T == 0) {
    if (cudaMemsetAsync(workspace, 0, kHeader, stream) != cudaSuccess) return KD_ERR_CUDA;
    if (!accumulate_dW &&
        cudaMemsetAsync(dW, 0, (size_t)p.V * p.d * 4, stream) != cudaSuccess)
      return KD_ERR_CUDA;
    return KD_OK;
  }
  EmbedArgs a{};
  a.dY = dY;
  a.ids = ids;
  a.mask = mask;
  a.dW = dW;
  a.T = (int)p.T;
  a.d = (int)p.d;
  a.V = (int)p.V;
  a.accumulate = accumulate_dW != 0;
  a.vec = p.d % 8 == 0 && aligned_to(dY, 16) && aligned_to(dW, 16);
  a.scale = p.scale;
  a.status = place<int>(workspace, 0);
  a.clear_bytes = accumulate_dW ? sizeof(int) : L.off_pairs[0];
  a.met = accumulate_dW ? nullptr : place<unsigned>(workspace, L.off_met);
  for (int i = 0; i < 2; ++i) a.pairs[i] = place<int2>(workspace, L.off_pairs[i]);
  a.hist = place<unsigned>(workspace, L.off_hist);
  a.part = place<float>(workspace, L.off_part);
  return launch_embedding_backward(a, p.rows_bf16 != 0, sms, stream) == cudaSuccess ? KD_OK
                                                                                    : KD_ERR_CUDA;
}

kd_status kd_norm_forward(const kd_norm_problem* prob, const void* x, const void* residual,
                          const void* weight, const void* bias, void* y, void* h, float* mean,
                          float* rstd, void* stream_ptr) {
  kd_status st = norm_check(prob);
  if (st != KD_OK) return st;
  const kd_norm_problem& p = *prob;
  if (p.T > 0 && (!x || !y || (residual && !h))) return KD_ERR_INVALID_ARG;
  if (p.kind == KD_NORM_RMS && (bias || mean)) return KD_ERR_INVALID_ARG;
  if (residual && y == h && p.T > 0) return KD_ERR_INVALID_ARG;
  const size_t ra = p.rows_bf16 ? 2 : 4, wa = p.weight_bf16 ? 2 : 4;
  if (!aligned_to(x, ra) || !aligned_to(residual, ra) || !aligned_to(y, ra) || !aligned_to(h, ra) ||
      !aligned_to(weight, wa) || !aligned_to(bias, wa) || !aligned_to(mean, 4) ||
      !aligned_to(rstd, 4))
    return KD_ERR_ALIGNMENT;
  int sms = 0;
  if ((st = (kd_status)current_device(&sms)) != KD_OK) return st;
  if (p.T == 0) return KD_OK;
  NormArgs a{};
  a.x = x;
  a.residual = residual;
  a.weight = weight;
  a.bias = bias;
  a.y = y;
  a.h = h;
  a.mean_out = mean;
  a.rstd_out = rstd;
  a.T = (int)p.T;
  a.d = (int)p.d;
  a.kind = p.kind;
  a.w_bf16 = p.weight_bf16 != 0;
  a.vec = aligned_to(x, 16) && aligned_to(residual, 16) && aligned_to(y, 16) &&
          (!residual || aligned_to(h, 16));
  a.classes = a.vec ? row_classes((int)p.d, (int)ra) : 1;
  a.eps = (float)p.eps;
  a.width = (float)p.d;
  return launch_norm_forward(a, p.rows_bf16 != 0, sms, static_cast<cudaStream_t>(stream_ptr)) ==
                 cudaSuccess
             ? KD_OK
             : KD_ERR_CUDA;
}

size_t kd_norm_workspace_size(const kd_norm_problem* prob) {
  return norm_check(prob) == KD_OK ? norm_bytes(*prob) : 0;
}

kd_status kd_norm_backward(const kd_norm_problem* prob, const void* dy, const void* h,
                           const void* weight, const float* mean, const float* rstd, const void* dh,
                           void* dx, float* dweight, float* dbias, int accumulate, void* workspace,
                           size_t workspace_bytes, void* stream_ptr) {
  kd_status st = norm_check(prob);
  if (st != KD_OK) return st;
  const kd_norm_problem& p = *prob;
  if (!workspace || workspace_bytes < norm_bytes(p)) return KD_ERR_WORKSPACE;
  const bool layer = p.kind == KD_NORM_LAYER;
  if (p.T > 0 && (!dy || !h || !rstd || !dx || (layer && !mean))) return KD_ERR_INVALID_ARG;
  if (!layer && dbias) return KD_ERR_INVALID_ARG;
  const size_t ra = p.rows_bf16 ? 2 : 4;
  if (!aligned_to(dy, ra) || !aligned_to(h, ra) || !aligned_to(dh, ra) || !aligned_to(dx, ra) ||
      !aligned_to(weight, p.weight_bf16 ? 2 : 4) || !aligned_to(mean, 4) || !aligned_to(rstd, 4) ||
      !aligned_to(dweight, 4) || !aligned_to(dbias, 4) || !aligned_to(workspace, 16))
    return KD_ERR_ALIGNMENT;
  int sms = 0;
  if ((st = (kd_status)current_device(&sms)) != KD_OK) return st;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
  forget_forward(workspace);
  if (p.T == 0) {
    if (cudaMemsetAsync(workspace, 0, kHeader, stream) != cudaSuccess) return KD_ERR_CUDA;
    for (float* sum : {dweight, dbias})
      if (sum && !accumulate &&
          cudaMemsetAsync(sum, 0, (size_t)p.d * 4, stream) != cudaSuccess)
        return KD_ERR_CUDA;
    return KD_OK;
  }
  NormArgs a{};
  a.x = h;
  a.weight = weight;
  a.dy = dy;
  a.dh = dh;
  a.mean = mean;
  a.rstd = rstd;
  a.dx = dx;
  a.part = dweight || dbias ? place<float>(workspace, kHeader) : nullptr;
  a.status = place<int>(workspace, 0);
  if (!a.part && cudaMemsetAsync(a.status, 0, sizeof(int), stream) != cudaSuccess) return KD_ERR_CUDA;
  a.dweight = dweight;
  a.dbias = dbias;
  a.T = (int)p.T;
  a.d = (int)p.d;
  a.kind = p.kind;
  a.w_bf16 = p.weight_bf16 != 0;
  a.accumulate = accumulate != 0;
  a.vec = aligned_to(dy, 16) && aligned_to(h, 16) && aligned_to(dh, 16) && aligned_to(dx, 16);
  a.classes = a.vec ? row_classes((int)p.d, (int)ra) : 1;
  a.width = (float)p.d;
  return launch_norm_backward(a, p.rows_bf16 != 0, std::min(sms, kMaxSms), stream) == cudaSuccess
             ? KD_OK
             : KD_ERR_CUDA;
}

size_t kd_muon_workspace_size(const kd_muon_matrix* matrices, int32_t n_matrices) {
  return muon_sizes(matrices, n_matrices) == KD_OK ? muon_bytes(matrices, n_matrices) : 0;
}

kd_status kd_muon_step(const kd_muon_matrix* matrices, int32_t n_matrices,
                       const kd_muon_options* opts, void* workspace, size_t workspace_bytes,
                       void* stream_ptr) {
  kd_status st = muon_sizes(matrices, n_matrices);
  if (st != KD_OK) return st;
  if (!opts) return KD_ERR_INVALID_ARG;
  const kd_muon_options& o = *opts;
  if (!fits32(o.lr) || !(o.momentum >= 0.0 && (float)o.momentum < 1.f) || !fits32(o.weight_decay) ||
      !fits32(o.lr * o.weight_decay) || !((float)o.eps >= 1e-30f) || !fits32(o.eps) ||
      !isfinite(o.grad_scale) || o.steps < 1 || o.steps > 10 ||
      (o.scale != KD_MUON_SPECTRAL && o.scale != KD_MUON_RMS))
    return KD_ERR_INVALID_ARG;
  if (!aligned_to(o.grad_scale_dev, 4) || !aligned_to(workspace, 16)) return KD_ERR_ALIGNMENT;
  for (int i = 0; i < n_matrices; ++i) {
    const kd_muon_matrix& m = matrices[i];
    if (!m.param || !m.grad || !m.momentum) return KD_ERR_INVALID_ARG;
    if (!aligned_to(m.param, o.param_bf16 ? 2 : 4) || !aligned_to(m.grad, o.grad_bf16 ? 2 : 4) ||
        !aligned_to(m.momentum, 4) || !aligned_to(m.copy, 2))
      return KD_ERR_ALIGNMENT;
  }
  if (!workspace || workspace_bytes < muon_bytes(matrices, n_matrices)) return KD_ERR_WORKSPACE;
  int sms = 0;
  if ((st = (kd_status)current_device(&sms)) != KD_OK) return st;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
  forget_forward(workspace);
  if (cudaMemsetAsync(workspace, 0, kHeader, stream) != cudaSuccess) return KD_ERR_CUDA;
  if (all_small(matrices, n_matrices))
    return muon_small(matrices, n_matrices, o, place<int>(workspace, 0), stream);
  RoundPlan p;
  const size_t full = round_bytes(matrices, n_matrices);
  for (int at = 0; at < n_matrices; at = p.end) {
    plan_round(matrices, n_matrices, at, full, &p);
    if ((st = muon_round(matrices, at, p, o, workspace, sms, stream)) != KD_OK) return st;
  }
  return KD_OK;
}

}  // extern "C"
