// C ABI of the losses over token log-probabilities and of the optimizer's
// step: argument checks, workspace plans and launches. (The log-probabilities
// themselves share the planning of the KL path, in kdkl_api.cu.)
#include <math.h>

#include <algorithm>

#include "kdkl.h"
#include "kdkl_internal.h"

namespace kdkl {
namespace {

constexpr size_t kHeader = 256;  // int status; two counts; a ticket
// Bound on the SM count that sizes workspaces (the same with and without a device).
constexpr int kMaxSms = 256;
constexpr int64_t kMaxTokens = (1ll << 31) - 4096;  // a block's token indexes stay in 31 bits
// The searches among the sequences double a step of at most S, and round S up to 32s: in
// 31 bits up to here.
constexpr int64_t kMaxSequences = 1ll << 30;

inline size_t pad256(size_t x) { return (x + 255) & ~(size_t)255; }
inline bool aligned_to(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

template <typename T>
T* place(void* ws, size_t off) {
  return reinterpret_cast<T*>(static_cast<char*>(ws) + off);
}

// Vector accesses: 16 bytes of every array.
bool vectors(const void* a, const void* b, const void* c, const void* d, const void* e,
             const uint8_t* mask) {
  return aligned_to(a, 16) && aligned_to(b, 16) && aligned_to(c, 16) && aligned_to(d, 16) &&
         aligned_to(e, 16) && aligned_to(mask, 16);
}

// Finite as the kernels take it. (An infinite weight times the zero of a token that is
// not counted would be a NaN.)
bool fits32(double x) { return isfinite((float)x); }

// A border in 48 bits: the nearest float and the remainder.
void split_border(double x, float* hi, float* lo) {
  *hi = (float)x;
  *lo = (float)(x - (double)*hi);
}

struct PolicyLayout {
  size_t off_seq, off_part, off_clips, total;
};
PolicyLayout policy_layout(const kd_policy_problem& p) {
  PolicyLayout L{};
  L.off_seq = kHeader;
  L.off_part = pad256(L.off_seq + (size_t)p.S * 4);
  L.off_clips = pad256(L.off_part + (size_t)seq_blocks((int)p.T, kMaxSms) * 16);
  L.total = pad256(L.off_clips + (size_t)seq_blocks((int)p.T, kMaxSms) * 4);
  return L;
}

kd_status policy_check(const kd_policy_problem* p) {
  if (!p) return KD_ERR_INVALID_ARG;
  if (p->T < 0 || p->T >= kMaxTokens || p->S < 0 || p->S > kMaxSequences) return KD_ERR_SHAPE;
  if (!(p->clip_low >= 0.0 && p->clip_low <= 1.0) || !(p->clip_high >= 0.0))
    return KD_ERR_INVALID_ARG;
  if (!(p->dual_clip == 0.0 || p->dual_clip > 1.0) || !isfinite(p->dual_clip))
    return KD_ERR_INVALID_ARG;
  if (!fits32(p->kl_coef)) return KD_ERR_INVALID_ARG;
  if (p->reduction < KD_REDUCE_TOKEN || p->reduction > KD_REDUCE_SUM) return KD_ERR_INVALID_ARG;
  if (p->reduction == KD_REDUCE_SUM &&
      !(p->norm > 0.0 && isfinite(p->norm) && fits32(1.0 / p->norm)))
    return KD_ERR_INVALID_ARG;
  if ((p->reduction == KD_REDUCE_SEQUENCE || p->advantage_per_sequence) && p->T > 0 && p->S < 1)
    return KD_ERR_SHAPE;
  return KD_OK;
}

struct PrefLayout {
  size_t off_sum, off_n, off_pair, off_coef, total;
};
PrefLayout pref_layout(const kd_pref_problem& p) {
  PrefLayout L{};
  const size_t slots = std::max<size_t>(seq_warps((int)p.T, kMaxSms), 64) + 2 * (size_t)p.P;
  L.off_sum = kHeader;
  L.off_n = pad256(L.off_sum + slots * 8);
  L.off_pair = pad256(L.off_n + slots * 4);
  L.off_coef = pad256(L.off_pair + (size_t)p.P * 4);
  L.total = pad256(L.off_coef + 2 * (size_t)p.P * 4);
  return L;
}

kd_status pref_check(const kd_pref_problem* p) {
  if (!p) return KD_ERR_INVALID_ARG;
  if (p->T < 0 || p->T >= kMaxTokens || p->P < 0 || p->P > kMaxSequences / 2) return KD_ERR_SHAPE;
  if (p->T > 0 && p->P < 1) return KD_ERR_SHAPE;
  if (!((float)p->beta > 0.f) || !fits32(p->beta) || !fits32(0.5 / p->beta) || !fits32(p->margin))
    return KD_ERR_INVALID_ARG;
  if (!(p->label_smoothing >= 0.0 && p->label_smoothing < 1.0)) return KD_ERR_INVALID_ARG;
  if (p->kind < KD_PREF_SIGMOID || p->kind > KD_PREF_HINGE) return KD_ERR_INVALID_ARG;
  return KD_OK;
}

}  // namespace
}  // namespace kdkl

using namespace kdkl;

extern "C" {

size_t kd_policy_workspace_size(const kd_policy_problem* prob) {
  return policy_check(prob) == KD_OK ? policy_layout(*prob).total : 0;
}

kd_status kd_policy_loss(const kd_policy_problem* prob, const float* logp, const float* old_logp,
                         const float* ref_logp, const float* advantages, const uint8_t* mask,
                         const int32_t* cu_seqlens, float grad_loss, float* loss, float* stats,
                         float* grad_logp, void* workspace, size_t workspace_bytes,
                         void* stream_ptr) {
  kd_status st = policy_check(prob);
  if (st != KD_OK) return st;
  const kd_policy_problem& p = *prob;
  if (!workspace) return KD_ERR_WORKSPACE;
  if (!loss || (p.T > 0 && (!logp || !advantages))) return KD_ERR_INVALID_ARG;
  const bool per_seq = p.reduction == KD_REDUCE_SEQUENCE || p.advantage_per_sequence;
  if (per_seq && p.T > 0 && !cu_seqlens) return KD_ERR_INVALID_ARG;
  if (!ref_logp && p.kl_coef != 0.0 && p.T > 0) return KD_ERR_INVALID_ARG;
  if (!isfinite(grad_loss) ||
      (p.reduction == KD_REDUCE_SUM && !fits32((double)grad_loss / p.norm)))
    return KD_ERR_INVALID_ARG;
  if (!aligned_to(logp, 4) || !aligned_to(old_logp, 4) || !aligned_to(ref_logp, 4) ||
      !aligned_to(advantages, 4) || !aligned_to(cu_seqlens, 4) || !aligned_to(loss, 4) ||
      !aligned_to(stats, 4) || !aligned_to(grad_logp, 4) || !aligned_to(workspace, 16))
    return KD_ERR_ALIGNMENT;
  const PolicyLayout L = policy_layout(p);
  if (workspace_bytes < L.total) return KD_ERR_WORKSPACE;
  int sms = 0;
  if ((st = (kd_status)current_device(&sms)) != KD_OK) return st;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
  forget_forward(workspace);
  sms = std::min(sms, kMaxSms);
  // status, counts, ticket and the sequences' counts start at zero
  const size_t zeros = p.reduction == KD_REDUCE_SEQUENCE ? L.off_part : kHeader;
  if ((p.T == 0 || !policy_one_block((int)p.T, p.reduction)) &&
      cudaMemsetAsync(workspace, 0, zeros, stream) != cudaSuccess)
    return KD_ERR_CUDA;
  if (p.T == 0) {
    if (cudaMemsetAsync(loss, 0, 4, stream) != cudaSuccess) return KD_ERR_CUDA;
    if (stats && cudaMemsetAsync(stats, 0, 12, stream) != cudaSuccess) return KD_ERR_CUDA;
    return KD_OK;
  }
  int* status = place<int>(workspace, 0);
  PolicyArgs a{};
  a.logp = logp;
  a.old_logp = old_logp;
  a.ref_logp = ref_logp;
  a.advantages = advantages;
  a.mask = mask;
  a.cu = per_seq ? cu_seqlens : nullptr;
  a.T = (int)p.T;
  a.S = (int)p.S;
  a.vec = vectors(logp, old_logp, ref_logp, p.advantage_per_sequence ? nullptr : advantages,
                  grad_logp, mask);
  a.reduction = p.reduction;
  a.adv_per_seq = p.advantage_per_sequence ? 1 : 0;
  a.count_here = p.reduction != KD_REDUCE_SEQUENCE && p.T <= kPolicyCountHere;
  a.dual = p.dual_clip > 0.0;
  a.inv_norm = p.reduction == KD_REDUCE_SUM ? (float)(1.0 / p.norm) : 0.f;
  a.kl_coef = (float)p.kl_coef;
  a.grad_loss = grad_loss;
  a.r_low = (float)(1.0 - p.clip_low);
  a.r_high = (float)(1.0 + p.clip_high);
  a.r_dual = (float)p.dual_clip;
  split_border(log1p(-p.clip_low), &a.low_hi, &a.low_lo);
  split_border(log1p(p.clip_high), &a.high_hi, &a.high_lo);
  if (a.dual) split_border(log(p.dual_clip), &a.dual_hi, &a.dual_lo);
  a.n_count = status + 1;
  a.n_seq = place<int>(workspace, L.off_seq);
  a.ticket = status + 4;
  a.block_part = place<float4>(workspace, L.off_part);
  a.block_clips = place<int>(workspace, L.off_clips);
  a.loss = loss;
  a.stats = stats;
  a.grad = grad_logp;
  return launch_policy_loss(a, sms, status, stream) == cudaSuccess ? KD_OK : KD_ERR_CUDA;
}

size_t kd_pref_workspace_size(const kd_pref_problem* prob) {
  return pref_check(prob) == KD_OK ? pref_layout(*prob).total : 0;
}

kd_status kd_pref_loss(const kd_pref_problem* prob, const float* logp, const float* ref_logp,
                       const uint8_t* mask, const int32_t* cu_seqlens, float grad_loss, float* loss,
                       float* rewards, float* grad_logp, void* workspace, size_t workspace_bytes,
                       void* stream_ptr) {
  kd_status st = pref_check(prob);
  if (st != KD_OK) return st;
  const kd_pref_problem& p = *prob;
  if (!workspace) return KD_ERR_WORKSPACE;
  if (!loss || (p.P > 0 && (!rewards || !cu_seqlens)) || (p.T > 0 && !logp))
    return KD_ERR_INVALID_ARG;
  if (!isfinite(grad_loss)) return KD_ERR_INVALID_ARG;
  if (!aligned_to(logp, 4) || !aligned_to(ref_logp, 4) || !aligned_to(cu_seqlens, 4) ||
      !aligned_to(loss, 4) || !aligned_to(rewards, 4) || !aligned_to(grad_logp, 4) ||
      !aligned_to(workspace, 16))
    return KD_ERR_ALIGNMENT;
  const PrefLayout L = pref_layout(p);
  if (workspace_bytes < L.total) return KD_ERR_WORKSPACE;
  int sms = 0;
  if ((st = (kd_status)current_device(&sms)) != KD_OK) return st;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
  forget_forward(workspace);
  sms = std::min(sms, kMaxSms);
  if (p.P == 0) {
    if (cudaMemsetAsync(workspace, 0, kHeader, stream) != cudaSuccess) return KD_ERR_CUDA;
    return cudaMemsetAsync(loss, 0, 4, stream) == cudaSuccess ? KD_OK : KD_ERR_CUDA;
  }
  int* status = place<int>(workspace, 0);
  PrefArgs a{};
  a.logp = logp;
  a.ref_logp = ref_logp;
  a.mask = mask;
  a.cu = cu_seqlens;
  a.T = (int)p.T;
  a.P = (int)p.P;
  a.vec = vectors(logp, ref_logp, grad_logp, nullptr, nullptr, mask);
  a.kind = p.kind;
  a.average = p.average;
  a.halves = p.halves;
  a.beta = (float)p.beta;
  a.label_smoothing = (float)p.label_smoothing;
  a.margin = (float)p.margin;
  a.half_inv_beta = (float)(0.5 / p.beta);
  a.grad_over_P = (float)((double)grad_loss / (double)p.P);
  a.slot_sum = place<float2>(workspace, L.off_sum);
  a.slot_n = place<int>(workspace, L.off_n);
  a.pair_loss = place<float>(workspace, L.off_pair);
  a.coef = place<float>(workspace, L.off_coef);
  a.loss = loss;
  a.rewards = rewards;
  a.grad = grad_logp;
  return launch_pref_loss(a, sms, status, stream) == cudaSuccess ? KD_OK : KD_ERR_CUDA;
}

kd_status kd_adamw_step(const kd_adamw_tensor* tensors, int32_t n_tensors,
                        const kd_adamw_options* opts, void* stream_ptr) {
  if (!opts || n_tensors < 0 || (n_tensors > 0 && !tensors)) return KD_ERR_INVALID_ARG;
  const kd_adamw_options& o = *opts;
  if (!isfinite(o.lr) || !(o.beta1 >= 0.0 && o.beta1 < 1.0) || !(o.beta2 >= 0.0 && o.beta2 < 1.0) ||
      !(o.eps >= 0.0) || !isfinite(o.eps) || !isfinite(o.weight_decay) || o.step < 1 ||
      !isfinite(o.grad_scale))
    return KD_ERR_INVALID_ARG;
  if (!aligned_to(o.grad_scale_dev, 4)) return KD_ERR_ALIGNMENT;
  const bool s8 = o.state_8bit != 0;
  const size_t pa = o.param_bf16 ? 2 : 4, ga = o.grad_bf16 ? 2 : 4, sa = s8 ? 1 : 4;
  long long elements = 0;
  for (int i = 0; i < n_tensors; ++i) {
    const kd_adamw_tensor& t = tensors[i];
    if (t.n < 0 || t.n >= (1ll << 40)) return KD_ERR_SHAPE;  // 2^31 blocks of a pass at most
    if (t.n == 0) continue;
    elements += t.n;
    if (!t.param || !t.grad || !t.exp_avg || !t.exp_avg_sq || (s8 && (!t.m_scale || !t.v_scale)))
      return KD_ERR_INVALID_ARG;
    if (!aligned_to(t.param, pa) || !aligned_to(t.grad, ga) || !aligned_to(t.exp_avg, sa) ||
        !aligned_to(t.exp_avg_sq, sa) || !aligned_to(t.copy, 2) || !aligned_to(t.m_scale, 4) ||
        !aligned_to(t.v_scale, 4))
      return KD_ERR_ALIGNMENT;
  }
  int sms = 0;
  const kd_status st = (kd_status)current_device(&sms);
  if (st != KD_OK) return st;
  AdamScalars s{};
  s.b1 = (float)o.beta1;
  s.one_b1 = (float)(1.0 - o.beta1);
  s.b2 = (float)o.beta2;
  s.one_b2 = (float)(1.0 - o.beta2);
  s.inv_root_bc2 = (float)(1.0 / sqrt(1.0 - pow(o.beta2, (double)o.step)));
  s.eps = (float)o.eps;
  s.step = (float)(o.lr / (1.0 - pow(o.beta1, (double)o.step)));
  s.keep = (float)(1.0 - o.lr * o.weight_decay);
  s.grad_scale = o.grad_scale;
  s.grad_scale_dev = o.grad_scale_dev;
  s.passes = adamw_passes(elements, s8, sms);
  cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
  AdamTensor list[ADAMW_LIST];
  int n = 0;
  int64_t blocks = 0;
  auto flush = [&]() {
    if (n == 0) return true;
    const bool ok = launch_adamw(list, n, (int)blocks, o.param_bf16 != 0, o.grad_bf16 != 0, s8, s,
                                 stream) == cudaSuccess;
    n = 0;
    blocks = 0;
    return ok;
  };
  for (int i = 0; i < n_tensors; ++i) {
    const kd_adamw_tensor& t = tensors[i];
    if (t.n == 0) continue;
    const int64_t nb = adamw_blocks(t.n, s.passes);
    if ((n == ADAMW_LIST || blocks + nb >= (1ll << 31) - 1) && !flush()) return KD_ERR_CUDA;
    AdamTensor& x = list[n++];
    x = AdamTensor{};
    x.param = t.param;
    x.grad = t.grad;
    x.exp_avg = t.exp_avg;
    x.exp_avg_sq = t.exp_avg_sq;
    x.copy = t.copy;
    x.m_scale = t.m_scale;
    x.v_scale = t.v_scale;
    x.n = t.n;
    x.block0 = (int)blocks;
    x.decay = t.decay;
    x.vec = aligned_to(t.param, 16) && aligned_to(t.grad, 16) &&
            aligned_to(t.exp_avg, s8 ? 8 : 16) && aligned_to(t.exp_avg_sq, s8 ? 8 : 16) &&
            aligned_to(t.copy, 16);
    blocks += nb;
  }
  return flush() ? KD_OK : KD_ERR_CUDA;
}

}  // extern "C"
