"""Tunes a language-model head on synthetic data, by preferences or by a policy loss.

    python examples/tune_head.py                 # preferences (pairs of answers)
    python examples/tune_head.py --loss policy   # sampled answers with advantages
    python examples/tune_head.py --state-bits 8  # 8-bit optimizer states

Every step: log-probabilities of the answers' tokens from the head (the logits are
never stored), the loss over them with its gradient, that gradient back to dW, and
one AdamW step on the head's fp32 weights, which writes the bf16 copy that the next
step reads. The hidden states stand in for a frozen trunk's output.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from lm_head_top_gb300 import kdkl  # noqa: E402


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--loss", choices=("preference", "policy"), default="preference")
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--answers", type=int, default=32, help="sequences, two to a pair")
    ap.add_argument("--length", type=int, default=64, help="tokens of each, the first quarter a prompt")
    ap.add_argument("--d", type=int, default=512)
    ap.add_argument("--vocabulary", type=int, default=8192)
    ap.add_argument("--state-bits", type=int, choices=(8, 32), default=32)
    ap.add_argument("--lr", type=float, default=2e-3)
    a = ap.parse_args()

    torch.manual_seed(0)
    dev, S, T, V, d = "cuda", a.answers, a.answers * a.length, a.vocabulary, a.d
    H = torch.randn(T, d, device=dev).bfloat16()
    master = torch.randn(V, d, device=dev) / d ** 0.5
    W = master.bfloat16()
    ids = torch.randint(0, V, (T,), device=dev, dtype=torch.int32)
    cu_seqlens = torch.arange(0, T + 1, a.length, device=dev, dtype=torch.int32)
    mask = (torch.arange(T, device=dev) % a.length >= a.length // 4).to(torch.uint8)
    advantages = torch.randn(S, device=dev)

    dW = torch.empty(V, d, device=dev)
    if a.state_bits == 32:
        m, v, scales = torch.zeros_like(master), torch.zeros_like(master), {}
    else:
        m, v = (torch.zeros(V, d, device=dev).to(torch.float8_e4m3fn) for _ in range(2))
        blocks = -(-V * d // kdkl.KD_ADAMW_BLOCK)
        scales = {k: [torch.ones(blocks, device=dev)] for k in ("m_scales", "v_scales")}
    tensors = kdkl.kd_adamw_tensors([master], [dW], [m], [v], copies=[W], **scales)

    # the frozen reference, and the policy that "sampled" the answers
    ref_logp, _ = kdkl.kd_logprob_forward(H, W, ids, mask)
    old_logp = ref_logp.clone()
    first = last = None
    for step in range(1, a.steps + 1):
        logp, lse = kdkl.kd_logprob_forward(H, W, ids, mask)
        if a.loss == "preference":
            loss, rewards, grad = kdkl.kd_pref_loss(logp, ref_logp, cu_seqlens, mask, beta=0.1)
            note = "chosen above rejected %.2f" % (rewards[:, 0] > rewards[:, 1]).float().mean().item()
        else:
            loss, stats, grad = kdkl.kd_policy_loss(logp, old_logp, ref_logp, advantages, mask, cu_seqlens,
                                                    advantage_per_sequence=True, clip_high=0.28, kl_coef=0.02,
                                                    reduction="sequence")
            note = "KL %.4f, clipped %.2f" % (stats[1].item(), stats[2].item())
        kdkl.kd_logprob_backward(H, W, ids, lse, grad, dW=dW)
        kdkl.kd_adamw_step(tensors, lr=a.lr, betas=(0.9, 0.95), step=step)
        last = loss.item()
        first = last if first is None else first
        print("step %2d  loss %.4f  %s" % (step, last, note))
    print("loss %.4f -> %.4f" % (first, last))
    return first, last


if __name__ == "__main__":
    first, last = main()
    sys.exit(0 if last < first else 1)
