"""fp64 CPU oracle of the calls that tune the head: token log-probabilities,
the clipped policy loss, the preference loss, and the AdamW step.

TEST INFRASTRUCTURE ONLY, as oracle/kl_oracle.py: plain numpy loops over the
definitions, no code shared with the library, checked against finite
differences by the tests.
"""
from __future__ import annotations

import numpy as np


def _softmax_rows(z):
    e = np.exp(z - z.max(axis=1, keepdims=True))
    return e / e.sum(axis=1, keepdims=True)


def logprob_forward(H, W, ids, mask, tau):
    """(logp, lse): zeros where not wanted."""
    T = H.shape[0]
    logp, lse = np.zeros(T), np.zeros(T)
    for t in range(T):
        if mask is not None and mask[t] == 0:
            continue
        z = W @ H[t] / tau
        top = z.max()
        lse[t] = top + np.log(np.exp(z - top).sum())
        logp[t] = z[ids[t]] - lse[t]
    return logp, lse


def logprob_backward(H, W, ids, grad, tau):
    """Gradients of sum_t grad[t] logp[t]."""
    dH, dW = np.zeros_like(H), np.zeros_like(W)
    for t in np.nonzero(grad)[0]:
        slope = -_softmax_rows((W @ H[t] / tau)[None])[0]
        slope[ids[t]] += 1.0
        slope *= grad[t] / tau
        dH[t] = slope @ W
        dW += slope[:, None] * H[t][None, :]
    return dH, dW


def sequence_of(cu, T):
    out = np.full(T, -1, dtype=np.int64)
    for s in range(len(cu) - 1):
        out[cu[s]:cu[s + 1]] = s
    return out


def policy_weights(mask, cu, T, reduction, norm):
    on = np.ones(T, dtype=bool) if mask is None else mask != 0
    w = np.zeros(T)
    if reduction == "token":
        w[on] = 1.0 / max(1, on.sum())
    elif reduction == "sum":
        w[on] = 1.0 / norm
    else:
        seq = sequence_of(cu, T)
        counts = np.bincount(seq[on], minlength=len(cu) - 1)
        w[on] = 1.0 / (counts[seq[on]] * (counts > 0).sum())
    return w, on


def policy_loss(logp, old, ref, adv, mask, cu, *, clip_low, clip_high, dual_clip, kl_coef,
                reduction, norm):
    """(loss, [policy part, KL part, clipped share], dloss/dlogp, clipped [T])."""
    T = len(logp)
    w, on = policy_weights(mask, cu, T, reduction, norm)
    A = adv if len(adv) == T else adv[sequence_of(cu, T)]
    pg = kl = 0.0
    grad, clipped = np.zeros(T), np.zeros(T, dtype=bool)
    for t in np.nonzero(on)[0]:
        d = logp[t] - old[t] if old is not None else 0.0
        if A[t] >= 0:
            clip = d > np.log1p(clip_high)
            r = 1.0 + clip_high if clip else np.exp(d)
        else:
            clip = d < np.log1p(-clip_low) if clip_low < 1 else False
            r = 1.0 - clip_low if clip else np.exp(d)
            if dual_clip and d > np.log(dual_clip):
                clip, r = True, dual_clip
        clipped[t] = clip
        pg -= w[t] * r * A[t]
        grad[t] = 0.0 if clip else -r * A[t]
        if ref is not None:
            x = ref[t] - logp[t]
            kl += w[t] * (np.expm1(x) - x)
            grad[t] -= kl_coef * np.expm1(x)
        grad[t] *= w[t]
    share = clipped.sum() / max(1, on.sum())
    return pg + kl_coef * kl, np.array([pg, kl, share]), grad, clipped


def pref_loss(logp, ref, mask, cu, *, beta, kind, label_smoothing, margin, average, halves):
    """(loss, rewards [P, 2], dloss/dlogp)."""
    T, P = len(logp), (len(cu) - 1) // 2
    on = np.ones(T, dtype=bool) if mask is None else mask != 0
    gap = np.zeros(T)
    gap[on] = logp[on] - (ref[on] if ref is not None else 0.0)
    grad, rewards, loss = np.zeros(T), np.zeros((P, 2)), 0.0
    for i in range(P):
        pair = (i, P + i) if halves else (2 * i, 2 * i + 1)
        q, n = [], []
        for s in pair:
            a, b = cu[s], cu[s + 1]
            n.append(max(1, on[a:b].sum()) if average else 1)
            q.append(gap[a:b].sum() / n[-1])
        rewards[i] = beta * q[0], beta * q[1]
        h = q[0] - q[1] - margin
        if kind == "sigmoid":
            e = label_smoothing
            loss += ((1 - e) * np.logaddexp(0, -beta * h) + e * np.logaddexp(0, beta * h)) / P
            up = 1.0 / (1.0 + np.exp(-beta * h))
            slope = beta * (e * up - (1 - e) * (1 - up))
        elif kind == "ipo":
            loss += (h - 0.5 / beta) ** 2 / P
            slope = 2 * (h - 0.5 / beta)
        else:
            loss += max(0.0, 1 - beta * h) / P
            slope = -beta if beta * h < 1 else 0.0
        for s, sign, k in ((pair[0], 1, 0), (pair[1], -1, 1)):
            grad[cu[s]:cu[s + 1]] = sign * slope / (P * n[k])
    return loss, rewards, np.where(on, grad, 0.0)


def adamw(p, g, m, v, *, lr, betas, eps, weight_decay, step, grad_scale, decay=True):
    """(p', m', v') of one step, fp64."""
    g = g * grad_scale
    m = betas[0] * m + (1 - betas[0]) * g
    v = betas[1] * v + (1 - betas[1]) * g * g
    hat = m / (1 - betas[0] ** step)
    root = np.sqrt(v / (1 - betas[1] ** step))
    return p - lr * weight_decay * p * bool(decay) - lr * hat / (root + eps), m, v


def e4m3_values():
    """All finite non-negative e4m3 values: 4 exponent bits (bias 7), 3 of mantissa."""
    out = []
    for code in range(127):  # 0x7f is NaN
        e, f = code >> 3, code & 7
        out.append(f * 2.0 ** -9 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7))
    return np.array(out)


def to_e4m3(x):
    """Nearest e4m3 value, ties to the even code (448 beyond it)."""
    grid = e4m3_values()
    a = np.minimum(np.abs(x), 448.0)
    hi = np.clip(np.searchsorted(grid, a), 1, len(grid) - 1)
    lo = hi - 1
    mid = (grid[lo] + grid[hi]) / 2
    pick = np.where(a > mid, hi, np.where(a < mid, lo, np.where(lo % 2 == 0, lo, hi)))
    return np.copysign(grid[pick], x)
