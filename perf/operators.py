"""Cases of the operators that tune a language-model head by preferences or by a policy.

Four operators, in the order in which a training step calls them:

* ``logprob``: log-probabilities of given tokens under softmax(H W^T / tau) and
  their backward pass (dH, dW from one upstream gradient per token);
* ``policy``: the clipped policy loss with a KL term over packed sequences,
  with its gradient;
* ``pref``: the preference loss over pairs of packed sequences, with its gradient;
* ``adamw``: one AdamW step over a list of tensors, states in 32 or in 8 bits.
"""
import math

import torch

own = False

BLOCK = 256  # elements that share one scale of an 8-bit state
# A block's largest magnitude stays within 512 times this, which rounds to 448, e4m3's largest value. A fraction of no few
# bits: sums of 8-bit states and bf16 gradients meet 448 or 460.8 exactly, and then its last bit would set the scale.
BORDER = 0.904383


# ------------------------------------------------------------------- cases


def listed():
    return [
        # The repository's small test size, forward and backward: latency counts.
        dict(name="logprob_small", op="logprob", T=256, d=256, V=4096, tau=1.0, prompt=0, seq=64, backward=True),
        # Odd sizes (vocabulary not a multiple of any tile, partial token tile), a sampling temperature.
        dict(name="logprob_odd", op="logprob", T=999, d=1000, V=32003, tau=0.7, prompt=40, seq=111, backward=True),
        # Scoring by an old or a reference policy: forward alone, a quarter of each sequence is prompt.
        dict(name="logprob_score", op="logprob", T=4000, d=2880, V=201088, tau=1.0, prompt=125, seq=500, backward=False),
        # A training step's head, half of each sequence is prompt.
        dict(name="logprob_train", op="logprob", T=6000, d=2880, V=201088, tau=1.0, prompt=300, seq=600, backward=True),
        # One micro-batch of short answers: latency counts.
        dict(name="policy_small", op="policy", T=2048, S=8, reduction="token", per_sequence=False, dual_clip=0.0, kl_coef=0.02, dirty=False),
        # A batch of 64 answers of about 4K tokens, padding with garbage under the mask.
        dict(name="policy_batch", op="policy", T=262144, S=64, reduction="token", per_sequence=False, dual_clip=0.0, kl_coef=0.04, dirty=True),
        # A whole rollout of ragged sequences: one advantage each, every sequence weighs the same.
        dict(name="policy_rollout", op="policy", T=8388593, S=2048, reduction="sequence", per_sequence=True, dual_clip=3.0, kl_coef=0.01, dirty=True),
        # Four pairs of short answers: latency counts.
        dict(name="pref_small", op="pref", T=2000, P=4, kind="sigmoid", average=False, label_smoothing=0.0, margin=0.0, halves=False, dirty=False),
        # A large batch of ragged pairs, chosen sequences first, then the rejected ones.
        dict(name="pref_batch", op="pref", T=4194301, P=512, kind="sigmoid", average=True, label_smoothing=0.1, margin=0.3, halves=True, dirty=True),
        # A small model's or an adapter's tensors, states in 32 bits.
        dict(name="adamw_small", op="adamw", layers=2, d=96, f=250, V=999, state_bits=32, grad="fp32", param="fp32", copy=False),
        # Many tensors, fp32 gradients (what the head's backward accumulates), fp32 weights with a bf16 copy.
        dict(name="adamw_32bit", op="adamw", layers=24, d=1024, f=2816, V=32000, state_bits=32, grad="fp32", param="fp32", copy=True),
        # The same tensors with 8-bit states and bf16 gradients.
        dict(name="adamw_8bit", op="adamw", layers=24, d=1024, f=2816, V=32000, state_bits=8, grad="bf16", param="fp32", copy=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["logprob", "policy", "pref", "adamw"])
    if op == "logprob":
        T, d = _log(rng, 64, 4000), 8 * _log(rng, 16, 360)
        V = _log(rng, 2000, min(201088, int(6e11 / (T * d))))
        seq = _log(rng, 16, T)
        return dict(op=op, T=T, d=d, V=V, tau=rng.choice([1.0, 0.7, 1.3]), prompt=rng.choice([0, seq // 3, seq // 2]),
                    seq=seq, backward=rng.random() < 0.7)
    if op == "policy":
        T = _log(rng, 100, 8000000)
        return dict(op=op, T=T, S=_log(rng, 1, max(1, min(4096, T // 16))), reduction=rng.choice(["token", "sequence", "sum"]),
                    per_sequence=rng.random() < 0.5, dual_clip=rng.choice([0.0, 3.0]), kl_coef=rng.choice([0.0, 0.01, 0.1]),
                    dirty=rng.random() < 0.5)
    if op == "pref":
        T = _log(rng, 100, 8000000)
        return dict(op=op, T=T, P=_log(rng, 1, max(1, min(2048, T // 32))), kind=rng.choice(["sigmoid", "ipo", "hinge"]),
                    average=rng.random() < 0.5, label_smoothing=rng.choice([0.0, 0.1]), margin=rng.choice([0.0, 0.3]),
                    halves=rng.random() < 0.5, dirty=rng.random() < 0.5)
    param = rng.choice(["fp32", "fp32", "bf16"])
    return dict(op=op, layers=_log(rng, 1, 24), d=_log(rng, 32, 1000), f=_log(rng, 64, 2800), V=_log(rng, 100, 32000),
                state_bits=rng.choice([32, 8]), grad=rng.choice(["fp32", "bf16"]), param=param,
                copy=param == "fp32" and rng.random() < 0.5)


# ------------------------------------------------------------------ inputs


def _counted(case):
    """Counted tokens of a logprob case: those past each sequence's prompt."""
    full, rest = divmod(case["T"], case["seq"])
    return full * (case["seq"] - case["prompt"]) + max(0, rest - case["prompt"])


def _shapes(case):
    """The tensors of a stack of layers, those with weight decay first."""
    d, f = case["d"], case["f"]
    decay = [(case["V"], d)] + [s for _ in range(case["layers"]) for s in ((d, d),) * 4 + ((f, d),) * 3]
    return decay, [(d,)] * (2 * case["layers"] + 1)


def _offsets(shapes):
    """Each tensor's start in a flat buffer, at multiples of the scale block, and the length."""
    at, n = [], 0
    for s in shapes:
        at.append(n)
        n += -(-math.prod(s) // BLOCK) * BLOCK
    return at, n


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    rand = lambda *s: torch.rand(*s, generator=g, device="cuda")  # noqa: E731
    s = {"case": case}
    if case["op"] == "logprob":
        T, d, V = case["T"], case["d"], case["V"]
        # A trained head: frequent ids repeat, and hidden states lean towards their token's row.
        s["ids"] = (V * rand(T) ** 3).int().clamp_(max=V - 1)
        s["W"] = (randn(V, d) / math.sqrt(d)).bfloat16()
        lean = 14 * rand(T, 1) * case["tau"]
        s["H"] = (randn(T, d) + lean * s["W"][s["ids"].long()].float()).bfloat16()
        s["mask"] = (torch.arange(T, device="cuda") % case["seq"] >= case["prompt"]).to(torch.uint8)
        s["grad_logp"] = torch.where(s["mask"] != 0, randn(T) / max(1, _counted(case)), 0.0)
    elif case["op"] in ("policy", "pref"):
        T = case["T"]
        S = case["S"] if case["op"] == "policy" else 2 * case["P"]
        # Ragged lengths; now and then a sequence without a token.
        w = rand(S) * 1.8 + 0.2
        w[5::37] = 0
        ends = (torch.cumsum(w.double(), 0) / w.double().sum() * T).round().int()
        ends[-1] = T
        s["cu_seqlens"] = torch.cat([torch.zeros(1, dtype=torch.int32, device="cuda"), ends])
        at = torch.arange(T, device="cuda")
        # Prompts are not counted, and some sequences not at all.
        s["mask"] = ((at % 97 > 24) & (at // 1031 % 23 != 3)).to(torch.uint8)
        s["logp"] = -2.0 * randn(T).abs()
        s["ref_logp"] = s["logp"] + 0.3 * randn(T)
        if case["op"] == "policy":
            s["old_logp"] = s["logp"] + 0.15 * randn(T)
            s["advantages"] = randn(S if case["per_sequence"] else T)
        if case["dirty"]:  # what padded positions hold
            s["logp"][s["mask"] == 0] = float("nan")
            s["ref_logp"][s["mask"] == 0] = float("-inf")
    else:
        decay, plain = _shapes(case)
        at, n = _offsets(decay + plain)
        s["decayed"] = at[len(decay)]  # elements of the flat buffers that decay
        real = torch.zeros(n, device="cuda")
        for a, sh in zip(at, decay + plain):
            real[a:a + math.prod(sh)] = 1
        s["grad"] = (randn(n) * 1e-3 * 10 ** (2 * rand(n) - 1) * real).to(torch.float32 if case["grad"] == "fp32" else torch.bfloat16)
        s["param"] = (randn(n) * 0.02 * real).to(torch.float32 if case["param"] == "fp32" else torch.bfloat16)
        s["copy"] = s["param"].bfloat16() if case["copy"] else None
        m, r = randn(n) * 5e-4 * real, (rand(n) * 1e-3 + 1e-5) * real
        if case["state_bits"] == 32:
            s["exp_avg"], s["exp_avg_sq"], s["m_scale"], s["v_scale"] = m, r * r, None, None
        else:
            s["exp_avg"], s["m_scale"] = _quantise(m)
            s["exp_avg_sq"], s["v_scale"] = _quantise(r)
        s["hyper"] = dict(lr=3e-4, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1, step=7, grad_scale=0.5)
        if own:  # the handle that a program makes once for its tensors
            from lm_head_top_gb300 import kdkl
            cut = lambda t: None if t is None else [t[a:a + math.prod(x)] for a, x in zip(at, decay + plain)]  # noqa: E731
            part = lambda t: None if t is None else [t[a // BLOCK:(a + math.prod(x) + BLOCK - 1) // BLOCK]  # noqa: E731
                                                     for a, x in zip(at, decay + plain)]
            s["handle"] = kdkl.kd_adamw_tensors(
                cut(s["param"]), cut(s["grad"]), cut(s["exp_avg"]), cut(s["exp_avg_sq"]), copies=cut(s["copy"]),
                m_scales=part(s["m_scale"]), v_scales=part(s["v_scale"]),
                decay=[True] * len(decay) + [False] * len(plain))
    return s


# --------------------------------------------------------------------- run


def run(state):
    return {"logprob": _run_logprob, "policy": _run_policy, "pref": _run_pref, "adamw": _run_adamw}[state["case"]["op"]](state)


def _run_logprob(s):
    c = s["case"]
    if own:
        from lm_head_top_gb300 import kdkl
        logp, lse = kdkl.kd_logprob_forward(s["H"], s["W"], s["ids"], s["mask"], temperature=c["tau"])
        if not c["backward"]:
            return {"logp": logp, "lse": lse}
        dH, dW = kdkl.kd_logprob_backward(s["H"], s["W"], s["ids"], lse, s["grad_logp"], temperature=c["tau"],
                                          dW_dtype=torch.bfloat16)
        return {"logp": logp, "lse": lse, "dH": dH, "dW": dW}
    rows = s["mask"].nonzero().squeeze(1)
    ids = s["ids"].long()[rows, None]
    H, W = s["H"][rows].float(), s["W"].float()
    z = H @ W.t()
    z *= 1 / c["tau"]
    top = z.amax(1, keepdim=True)
    picked = z.gather(1, ids)
    e = z.sub_(top).exp_()
    total = e.sum(1, keepdim=True)
    row_lse = top + total.log()
    out = {}
    for name, v in (("logp", picked - row_lse), ("lse", row_lse)):
        out[name] = torch.zeros_like(s["grad_logp"])
        out[name][rows] = v.squeeze(1)
    if c["backward"]:
        gr = s["grad_logp"][rows, None] / c["tau"]
        G = e.mul_(-gr / total).scatter_add_(1, ids, gr)
        out["dH"] = torch.zeros_like(s["H"])
        out["dH"][rows] = (G @ W).bfloat16()
        out["dW"] = (G.t() @ H).bfloat16()
    return out


CLIP_LOW, CLIP_HIGH, GRAD_LOSS, NORM = 0.2, 0.28, 0.5, 4096.0


def _run_policy(s):
    c = s["case"]
    if own:
        from lm_head_top_gb300 import kdkl
        loss, stats, grad = kdkl.kd_policy_loss(
            s["logp"], s["old_logp"], s["ref_logp"], s["advantages"], s["mask"], s["cu_seqlens"], clip_low=CLIP_LOW,
            clip_high=CLIP_HIGH, dual_clip=c["dual_clip"], kl_coef=c["kl_coef"], reduction=c["reduction"], norm=NORM,
            grad_loss=GRAD_LOSS)
        return {"loss": loss, "stats": stats, "grad": grad}
    cu = s["cu_seqlens"].long()
    lens = cu[1:] - cu[:-1]
    seq = torch.repeat_interleave(torch.arange(lens.numel(), device=cu.device), lens, output_size=c["T"])
    on = s["mask"] != 0
    counts = torch.cumsum(torch.cat([on.new_zeros(1), on]), 0)
    per_seq = counts[cu[1:]] - counts[cu[:-1]]
    n = counts[-1]
    adv = s["advantages"][seq] if c["per_sequence"] else s["advantages"]
    # which side of a border a ratio is on takes 64 bits, and so does e^x - 1 - x for small x
    delta = torch.where(on, s["logp"].double() - s["old_logp"].double(), 0.0)
    x = torch.where(on, s["ref_logp"].double() - s["logp"].double(), 0.0)
    pos = adv >= 0
    clipped = torch.where(pos, delta > math.log(1 + CLIP_HIGH), delta < math.log(1 - CLIP_LOW))
    bound = torch.where(pos, 1 + CLIP_HIGH, 1 - CLIP_LOW)
    if c["dual_clip"]:
        over = ~pos & (delta > math.log(c["dual_clip"]))
        bound = torch.where(over, c["dual_clip"], bound)
        clipped = clipped | over
    ratio = torch.where(clipped, bound, delta.float().exp())
    rise = torch.expm1(x)
    if c["reduction"] == "token":
        weight = on / n.clamp(min=1).float()
    elif c["reduction"] == "sequence":
        weight = on / (per_seq * (per_seq > 0).sum()).clamp(min=1).float()[seq]
    else:
        weight = on / NORM
    pg = -(weight * torch.where(on, ratio * adv, 0.0)).double().sum()
    kl = (weight * (rise - x)).sum()
    grad = weight * (torch.where(clipped, 0.0, -ratio * adv) - c["kl_coef"] * rise).float() * GRAD_LOSS
    share = (clipped & on).sum() / n.clamp(min=1)
    return {"loss": (pg + c["kl_coef"] * kl).float().reshape(1), "stats": torch.stack([pg, kl, share.double()]).float(),
            "grad": torch.where(on, grad, 0.0)}


BETA = 0.1


def _run_pref(s):
    c = s["case"]
    if own:
        from lm_head_top_gb300 import kdkl
        loss, rewards, grad = kdkl.kd_pref_loss(
            s["logp"], s["ref_logp"], s["cu_seqlens"], s["mask"], beta=BETA, kind=c["kind"], average=c["average"],
            label_smoothing=c["label_smoothing"], margin=c["margin"], halves=c["halves"], grad_loss=GRAD_LOSS)
        return {"loss": loss, "rewards": rewards, "grad": grad}
    cu, P = s["cu_seqlens"].long(), c["P"]
    on = s["mask"] != 0
    gap = torch.where(on, s["logp"] - s["ref_logp"], 0.0)
    sums = torch.cumsum(torch.cat([gap.new_zeros(1), gap]).double(), 0)  # a long sum
    counts = torch.cumsum(torch.cat([on.new_zeros(1), on]), 0)
    share = 1 / (counts[cu[1:]] - counts[cu[:-1]]).clamp(min=1).double() if c["average"] else torch.ones(2 * P, dtype=torch.double, device=cu.device)
    ratios = (sums[cu[1:]] - sums[cu[:-1]]) * share
    pair = ratios.view(2, P) if c["halves"] else ratios.view(P, 2).t()
    h = pair[0] - pair[1] - c["margin"]
    b, eps = BETA * h, c["label_smoothing"]
    if c["kind"] == "sigmoid":
        soft = torch.log1p(torch.exp(-b.abs()))
        each = (1 - eps) * (soft + (-b).clamp(min=0)) + eps * (soft + b.clamp(min=0))
        slope = BETA * (eps - 1 / (1 + torch.exp(b)))
    elif c["kind"] == "ipo":
        each, slope = (h - 0.5 / BETA) ** 2, 2 * (h - 0.5 / BETA)
    else:
        each, slope = (1 - b).clamp(min=0), torch.where(b < 1, -BETA, 0.0).double()
    slope = slope * GRAD_LOSS / P
    both = torch.stack([slope, -slope], 0 if c["halves"] else 1).reshape(-1) * share
    seq = torch.repeat_interleave(torch.arange(2 * P, device=cu.device), cu[1:] - cu[:-1], output_size=c["T"])
    return {"loss": each.mean().float().reshape(1), "rewards": (BETA * pair.t()).float().contiguous(),
            "grad": torch.where(on, both.float()[seq], 0.0)}


def _quantise(x):
    """x in e4m3, and one power of two for each block of elements: the least that keeps the block within the border."""
    x = x.view(-1, BLOCK)
    half, e = torch.frexp(x.abs().amax(1))
    scale = torch.where(half > 0, torch.ldexp(torch.ones_like(half), (e - 9 + (half > BORDER)).clamp(min=-126)), 1.0)
    return (x / scale[:, None]).view(-1).to(torch.float8_e4m3fn), scale


def _run_adamw(s):
    c, h = s["case"], s["hyper"]
    if own:
        from lm_head_top_gb300 import kdkl
        kdkl.kd_adamw_step(s["handle"], **h)
        out = {"param": s["param"], "exp_avg": s["exp_avg"], "exp_avg_sq": s["exp_avg_sq"]}
    else:
        (b1, b2), lr, t = h["betas"], h["lr"], h["step"]
        g = s["grad"].float() * h["grad_scale"]
        if c["state_bits"] == 32:
            m, v = s["exp_avg"], s["exp_avg_sq"]
        else:
            m = (s["exp_avg"].float().view(-1, BLOCK) * s["m_scale"][:, None]).view(-1)
            v = (s["exp_avg_sq"].float().view(-1, BLOCK) * s["v_scale"][:, None]).view(-1) ** 2
        m = m * b1 + g * (1 - b1)
        v = v * b2 + g * g * (1 - b2)
        root = v.sqrt()
        p = s["param"].float()
        p[:s["decayed"]] *= 1 - lr * h["weight_decay"]
        p -= m / (root * (1 / math.sqrt(1 - b2 ** t)) + h["eps"]) * (lr / (1 - b1 ** t))
        s["param"].copy_(p)
        if c["copy"]:
            s["copy"].copy_(p)
        if c["state_bits"] == 32:
            s["exp_avg"].copy_(m)
            s["exp_avg_sq"].copy_(v)
        else:
            q, scale = _quantise(m)
            s["exp_avg"].copy_(q)
            s["m_scale"].copy_(scale)
            q, scale = _quantise(root)  # the root is held; what is not zero stays so
            q = torch.where((root > 0) & (q.float() == 0), 2.0 ** -9, q.float()).to(torch.float8_e4m3fn)
            s["exp_avg_sq"].copy_(q)
            s["v_scale"].copy_(scale)
        out = {"param": s["param"], "exp_avg": s["exp_avg"], "exp_avg_sq": s["exp_avg_sq"]}
    if c["copy"]:
        out["copy"] = s["copy"]
    if c["state_bits"] == 8:
        out["m_scale"], out["v_scale"] = s["m_scale"], s["v_scale"]
    return out


# -------------------------------------------------------------------- work


def work(case):
    """Each input read once, each output written once; the products a pass cannot do without."""
    if case["op"] == "logprob":
        N, T, d, V = _counted(case), case["T"], case["d"], case["V"]
        b, f = 2 * N * d + 2 * V * d + 5 * T + 8 * T, 2 * N * V * d
        return {"bytes": b + (2 * T * d + 2 * V * d + 4 * T if case["backward"] else 0), "flops": f * (3 if case["backward"] else 1)}
    if case["op"] == "policy":
        T = case["T"]
        return {"bytes": T * (4 * 3 + 1 + 4) + 4 * (case["S"] if case["per_sequence"] else T) + 4 * case["S"], "flops": 40 * T}
    if case["op"] == "pref":
        return {"bytes": case["T"] * (4 * 2 + 1 + 4) + 16 * case["P"], "flops": 4 * case["T"]}
    n = sum(math.prod(x) for group in _shapes(case) for x in group)
    each = (4 if case["grad"] == "fp32" else 2) + 2 * (4 if case["param"] == "fp32" else 2) + (2 if case["copy"] else 0)
    return {"bytes": n * (each + (16 if case["state_bits"] == 32 else 4 + 16 / BLOCK)), "flops": 20 * n}


# ------------------------------------------------------------------- exact


def exact(case, seed):
    s = prepare(case, seed)
    return {"logprob": _exact_logprob, "policy": _exact_policy, "pref": _exact_pref, "adamw": _exact_adamw}[case["op"]](s, case)


def _exact_logprob(s, c):
    if 2 * _counted(c) * c["V"] * c["d"] * (3 if c["backward"] else 1) > 1.3e13:
        return None
    T, dev = c["T"], s["H"].device
    W = s["W"].double()
    out = {"logp": torch.zeros(T, dtype=torch.double, device=dev), "lse": torch.zeros(T, dtype=torch.double, device=dev)}
    if c["backward"]:
        out["dH"] = torch.zeros(T, c["d"], dtype=torch.double, device=dev)
        out["dW"] = torch.zeros(c["V"], c["d"], dtype=torch.double, device=dev)
    rows = (s["mask"] != 0).nonzero().squeeze(1)
    for some in rows.split(1024):
        H = s["H"][some].double()
        logs = torch.log_softmax(torch.matmul(H, W.t()) / c["tau"], 1)
        mine = torch.nn.functional.one_hot(s["ids"][some].long(), c["V"]).bool()
        out["logp"][some] = logs[mine]
        out["lse"][some] = (H * W[s["ids"][some].long()]).sum(1) / c["tau"] - logs[mine]
        if c["backward"]:
            slope = (mine.double() - logs.exp()) * (s["grad_logp"][some].double() / c["tau"])[:, None]
            out["dH"][some] = slope @ W
            out["dW"] += slope.t() @ H
    return out


def _exact_policy(s, c):
    cu, on = s["cu_seqlens"].tolist(), s["mask"] != 0
    lens = torch.tensor([b - a for a, b in zip(cu, cu[1:])], device=on.device)
    which = torch.bucketize(torch.arange(c["T"], device=on.device), s["cu_seqlens"][1:].long(), right=True)
    hold = torch.zeros(lens.numel(), dtype=torch.double, device=on.device).index_add_(0, which, on.double())
    adv = s["advantages"].double()
    adv = adv[which] if c["per_sequence"] else adv
    idx = on.nonzero().squeeze(1)
    a, lp = adv[idx], s["logp"].double()[idx]
    lp_old, lp_ref = s["old_logp"].double()[idx], s["ref_logp"].double()[idx]
    r = torch.exp(lp - lp_old)
    free = r * a
    held = r.clamp(1 - CLIP_LOW, 1 + CLIP_HIGH) * a
    best = torch.minimum(free, held)
    if c["dual_clip"]:
        best = torch.where(a < 0, torch.maximum(best, c["dual_clip"] * a), best)
    moves = best == free
    k = torch.expm1(lp_ref - lp) - (lp_ref - lp)
    if c["reduction"] == "token":
        w = torch.full_like(a, 1 / max(1, idx.numel()))
    elif c["reduction"] == "sequence":
        w = 1 / (hold[which[idx]] * (hold > 0).sum())
    else:
        w = torch.full_like(a, 1 / NORM)
    pg, kl = -(w * best).sum(), (w * k).sum()
    grad = torch.zeros(c["T"], dtype=torch.double, device=on.device)
    grad[idx] = GRAD_LOSS * w * (-free * moves - c["kl_coef"] * torch.expm1(lp_ref - lp))
    share = (~moves).double().sum() / max(1, idx.numel())
    return {"loss": (pg + c["kl_coef"] * kl).reshape(1), "stats": torch.stack([pg, kl, share]), "grad": grad}


def _exact_pref(s, c):
    P, on = c["P"], (s["mask"] != 0)
    which = torch.bucketize(torch.arange(c["T"], device=on.device), s["cu_seqlens"][1:].long(), right=True)
    idx = on.nonzero().squeeze(1)
    zero = torch.zeros(2 * P, dtype=torch.double, device=on.device)
    total = zero.index_add(0, which[idx], s["logp"].double()[idx] - s["ref_logp"].double()[idx])
    n = zero.index_add(0, which[idx], torch.ones_like(idx, dtype=torch.double))
    per = n.clamp(min=1) if c["average"] else torch.ones_like(n)
    one = torch.arange(P, device=on.device) * (1 if c["halves"] else 2)
    two = one + (P if c["halves"] else 1)
    y = torch.stack([total[one] / per[one], total[two] / per[two]], 1).requires_grad_()
    h = y[:, 0] - y[:, 1] - c["margin"]
    ls = torch.nn.functional.logsigmoid
    if c["kind"] == "sigmoid":
        each = -(1 - c["label_smoothing"]) * ls(BETA * h) - c["label_smoothing"] * ls(-BETA * h)
    elif c["kind"] == "ipo":
        each = (h - 1 / (2 * BETA)).square()
    else:
        each = torch.relu(1 - BETA * h)
    loss = each.mean()
    (dy,) = torch.autograd.grad(loss, y)
    slope = zero.clone()
    slope[one], slope[two] = dy[:, 0], dy[:, 1]
    grad = torch.zeros(c["T"], dtype=torch.double, device=on.device)
    grad[idx] = GRAD_LOSS * (slope / per)[which[idx]]
    return {"loss": loss.detach().reshape(1), "rewards": BETA * y.detach(), "grad": grad}


def _exact_e4m3(x, least):
    """Nearest e4m3 values (ties to even) of x in units of its block's power of two, and those powers; `least`: no value but 0 becomes 0."""
    x = x.reshape(-1, BLOCK)
    top = x.abs().amax(1, keepdim=True)
    e = torch.ceil(torch.log2(top / (512 * BORDER))).clamp(min=-126)
    scale = torch.where(top > 0, 2 ** e, 1.0)
    y = x / scale
    unit = 2 ** (torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    q = (torch.round(y / unit) * unit).clamp(-448, 448)
    if least:
        q = torch.where((y > 0) & (q == 0), 2.0 ** -9, q)
    return q.reshape(-1), scale.reshape(-1)


def _exact_adamw(s, c):
    h = s["hyper"]
    beta1, beta2 = h["betas"]
    grad = s["grad"].double() * h["grad_scale"]
    mean, square = s["exp_avg"].to(torch.float32).double(), s["exp_avg_sq"].to(torch.float32).double()
    if c["state_bits"] == 8:
        mean = mean * s["m_scale"].double().repeat_interleave(BLOCK)
        square = (square * s["v_scale"].double().repeat_interleave(BLOCK)).square()
    mean = mean + (1 - beta1) * (grad - mean)
    square = square + (1 - beta2) * (grad.square() - square)
    fade = torch.ones_like(grad)
    fade[:s["decayed"]] = 1 - h["lr"] * h["weight_decay"]
    mhat, vhat = mean / (1 - beta1 ** h["step"]), square / (1 - beta2 ** h["step"])
    p = s["param"].double() * fade - h["lr"] * mhat / (vhat.sqrt() + h["eps"])
    out = {"param": p}
    if c["copy"]:
        out["copy"] = p
    if c["state_bits"] == 8:
        out["exp_avg"], out["m_scale"] = _exact_e4m3(mean, False)
        out["exp_avg_sq"], out["v_scale"] = _exact_e4m3(square.sqrt(), True)
    else:
        out["exp_avg"], out["exp_avg_sq"] = mean, square
    return out
