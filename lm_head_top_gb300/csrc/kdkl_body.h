// Declarations shared by the embedding, the norms and the Muon step: kernels_embed.cu,
// kernels_norm.cu, kernels_muon.cu, and kdkl_body.cu, which calls them.
#pragma once

#include <cuda.h>
#include <cuda_fp16.h>

#include "kdkl_internal.h"

namespace kdkl {

// kernels_norm.cu
struct NormArgs {
  const void *x, *residual, *weight, *bias;  // forward
  void *y, *h;
  float *mean_out, *rstd_out;
  const void *dy, *dh;  // backward (x: what was normed)
  const float *mean, *rstd;
  void* dx;
  float* part;  // [blocks][2][d]: each block's sums for the weight and the bias
  int* status;  // backward
  float *dweight, *dbias;
  int T, d, kind, w_bf16, accumulate;
  int vec;      // every array of rows starts on 16 bytes
  int classes;  // with vec: how many rows after a row the next starts as it does within 16 bytes
  float eps, width;  // width: d
};
constexpr int NORM_MAX_D = 16384;
// Thread blocks of the backward at most (each leaves a row of partial sums).
int norm_backward_blocks(int T, int d, int num_sms);
cudaError_t launch_norm_forward(const NormArgs& a, bool rows_bf16, int num_sms, cudaStream_t stream);
cudaError_t launch_norm_backward(const NormArgs& a, bool rows_bf16, int num_sms,
                                 cudaStream_t stream);

// kernels_embed.cu
struct EmbedArgs {
  const void *W, *dY;
  const int32_t* ids;
  const uint8_t* mask;
  void* Y;
  float* dW;
  int T, d, V, accumulate;
  int vec;  // rows start on 16 bytes in every array, and d is a multiple of 8
  float scale;
  int* status;               // forward: or null
  size_t clear_bytes;        // backward: from `status` on, to be zero at the start
  unsigned* met;             // a bit for every row of the table that is named, or null
  int2* pairs[2];            // backward: (id, token), sorted from one into the other
  unsigned* hist;
  float* part;  // [pieces][2][d]
};
constexpr int EMBED_PIECE = 32;  // sorted tokens that are added up together
// Bytes of the counters of a sort of T ids.
size_t embed_sort_bytes(int T);
cudaError_t launch_embedding_forward(const EmbedArgs& a, bool table_bf16, bool rows_bf16,
                                     cudaStream_t stream);
cudaError_t launch_embedding_backward(const EmbedArgs& a, bool rows_bf16, int num_sms,
                                      cudaStream_t stream);

// kernels_muon.cu
struct MuonMatrix {
  void* param;
  const void* grad;
  float* momentum;
  uint16_t* copy;
  float step;  // lr * scale of its shape
  float keep;  // 1 - lr * weight_decay, or 1
};
// Matrices of one shape, worked on together. r <= k: the sizes after transposing.
// Every matrix is held as its high and its low halves, one after the other, rows of `ldk`
// (X) or `ldr` (X X^T and the polynomial) fp16 values.
struct MuonGroup {
  int first, count;  // in the list of matrices
  int r, k, ldk, ldr;
  int tall;          // rows > cols: X is the transposed matrix
  int part0, parts;  // sums of squares of a matrix: its first, how many
  int blocks0;       // first thread block of the elementwise launches' grids
  int tiles0;
  int units0[3], units[3];  // of each product: its first tile, tiles of a matrix
  __half *X[2], *S, *P;
};
constexpr int MUON_GROUPS = 16;
constexpr int MUON_LIST = 384;  // 15 KB of the 32,764 bytes a kernel's parameters may take
struct MuonRound {
  MuonGroup g[MUON_GROUPS];
  int n_groups;
  int whole[2];  // of the symmetric products: see muon_units
  int fours;     // rows of all parameters and copies start on four elements
  float momentum, eps, grad_scale;
  int nesterov;
  const float* grad_scale_dev;
  float* part;    // sums of squares by pieces, or -inf: see `piece`
  float2* piece;  // sums of squares of u / unit, and the unit
};
struct MuonList {
  MuonMatrix m[MUON_LIST];
};
// Maps of the groups' X[0], X[1], S and P, each [count][2][r][columns].
struct MuonMaps {
  CUtensorMap m[MUON_GROUPS];
};
constexpr int MUON_BOX = 64;            // rows and columns of a copied box
constexpr int MUON_CHUNK = 16384;       // elements of a thread block's sum of squares
constexpr int MUON_TILE = 64;           // of the pass that lays X out
// Matrices that a thread block takes through the whole step by itself.
struct MuonSmall {
  MuonMatrix m[MUON_LIST];
  unsigned short rows[MUON_LIST], cols[MUON_LIST];
  float momentum, eps, grad_scale;
  int nesterov, steps;
  const float* grad_scale_dev;
};
inline bool muon_is_small(long long rows, long long cols) {
  return rows * cols <= 128 * 256 && (rows < cols ? rows <= 128 && cols <= 256
                                                  : cols <= 128 && rows <= 256);
}
cudaError_t launch_muon_small(const MuonSmall& a, int count, bool grad_bf16, bool param_bf16,
                              int* status, cudaStream_t stream);
cudaError_t launch_muon_momentum(const MuonRound& r, const MuonList& l, bool grad_bf16, int blocks,
                                 cudaStream_t stream);
cudaError_t launch_muon_layout(const MuonRound& r, const MuonList& l, bool grad_bf16, int blocks,
                               cudaStream_t stream);
enum MuonProduct { MUON_GRAM = 0, MUON_POLY = 1, MUON_APPLY = 2, MUON_UPDATE = 3 };
// Tiles of a product of one matrix, of 256 x 256 (a pair of SMs) or 128 x 128; of a symmetric one
// those that later products read (whole: by pairs' tiles). And what they cost for a round's.
int muon_units(int r, int k, MuonProduct what, bool pair, bool whole);
double muon_cost(const MuonGroup* g, int n_groups, MuonProduct what, bool pair, bool whole,
                 int num_sms);
// S = X[from] X[from]^T; P = B S + C S^2; X[1 - from] = A X[from] + P X[from]; or that as the
// update of the parameters.
cudaError_t launch_muon_product(MuonProduct what, const MuonRound& r, const MuonList& l, int from,
                                const MuonMaps& a, const MuonMaps& b, bool param_bf16, bool pair,
                                int units, int* status, int num_sms, cudaStream_t stream);

}  // namespace kdkl
