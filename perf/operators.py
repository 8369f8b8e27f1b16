"""The operators between a model's last block and the optimizer step, as measurable cases.

Four operators that a fine-tuning loop runs right before ``muon_step`` and
``muon_adamw_step``: the norms around a block with its gate and residual scale
("norm"), the log-probabilities of the target tokens under a vocabulary head
("head"), the preference loss over pairs of sequences ("preference") and the
clipped policy loss with a KL term ("policy"), each with its gradients.

``run`` computes an operator in its plain form (elementary torch operations in
32 bits, rounded once at the end) when ``own`` is false, and calls the
framework's entry point when it is true; ``exact`` is the definition in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ----------------------------------------------------------------------------
# Cases
# ----------------------------------------------------------------------------

def listed():
    return [
        # one token of a d = 2048 model, as a scoring or serving loop calls it
        dict(name="norm_one_token", op="norm", dtype="bf16", rows=1, cols=2048, gate="channel", direction="fwd"),
        # a training batch of the d = 2048 transformer, sandwich norms and a channel gate
        dict(name="norm_train", op="norm", dtype="bf16", rows=8192, cols=2048, gate="channel", direction="both"),
        # odd width, a gate per element, single precision
        dict(name="norm_odd_f32", op="norm", dtype="f32", rows=1003, cols=1407, gate="full", direction="both"),
        # one token scored against the 32000-entry head
        dict(name="head_one_token", op="head", dtype="bf16", tokens=1, cols=2048, vocab=32000, ignored=0.0,
             direction="fwd"),
        # the head of the d = 2048 transformer in a training step, a quarter of the tokens prompt
        dict(name="head_train", op="head", dtype="bf16", tokens=8192, cols=2048, vocab=32000, ignored=0.25,
             direction="both"),
        # odd sizes throughout, as after a change of vocabulary
        dict(name="head_odd", op="head", dtype="bf16", tokens=777, cols=1000, vocab=32003, ignored=0.3,
             direction="both"),
        # single precision, a small model
        dict(name="head_f32", op="head", dtype="f32", tokens=512, cols=1024, vocab=8192, ignored=0.0,
             direction="both"),
        # a micro-batch of four short pairs
        dict(name="preference_small", op="preference", dtype="f32", pairs=4, longest=64, kind="sigmoid",
             reference=True, average=False, masked=0.3),
        # a large batch of pairs with ragged answers
        dict(name="preference_batch", op="preference", dtype="f32", pairs=256, longest=4096, kind="sigmoid",
             reference=True, average=False, masked=0.3),
        # a few short answers
        dict(name="policy_small", op="policy", dtype="f32", sequences=8, longest=128, kl="k3", reduction="token",
             per_sequence=True, masked=0.2),
        # a rollout batch
        dict(name="policy_batch", op="policy", dtype="f32", sequences=2048, longest=2048, kl="k3",
             reduction="token", per_sequence=True, masked=0.2),
        # few, very long answers, a mean within each
        dict(name="policy_long", op="policy", dtype="f32", sequences=6, longest=400000, kl="k2",
             reduction="sequence", per_sequence=False, masked=0.1),
    ]


def _log_int(rng, lo, hi):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["norm", "head", "head", "preference", "policy"])
    if op == "norm":
        cols = rng.choice([rng.randint(64, 1000), rng.choice([1024, 2048, 4096, 8192]), rng.randint(1001, 8192)])
        rows = _log_int(rng, 1, max(1, 8192 * 2048 // cols))
        return dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]), rows=rows, cols=cols,
                    gate=rng.choice(["channel", "full", "none"]), direction=rng.choice(["fwd", "both"]))
    if op == "head":
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        cols = rng.choice([64 * rng.randint(2, 64), rng.choice([1024, 2048, 4096]), rng.randint(100, 4096)])
        vocab = rng.choice([_log_int(rng, 1000, 65536), rng.choice([8192, 32000, 65536])])
        most = (8192 * 2048 * 32000 if dtype == "bf16" else 1024 * 2048 * 16384) // (cols * vocab)
        tokens = _log_int(rng, 1, max(1, min(8192, most)))
        return dict(op=op, dtype=dtype, tokens=tokens, cols=cols, vocab=vocab,
                    ignored=rng.choice([0.0, 0.2, 0.5]) if tokens > 8 else 0.0,
                    direction=rng.choice(["fwd", "both", "both"]))
    if op == "preference":
        longest = _log_int(rng, 8, 65536)
        return dict(op=op, dtype=rng.choice(["f32", "f32", "bf16"]), pairs=_log_int(rng, 1, max(1, 1000000 // longest)),
                    longest=longest, kind=rng.choice(["sigmoid", "hinge", "squared"]),
                    reference=rng.random() < 0.7, average=rng.random() < 0.5, masked=rng.choice([0.0, 0.3]))
    longest = _log_int(rng, 8, 400000)
    return dict(op=op, dtype=rng.choice(["f32", "f32", "bf16"]), sequences=_log_int(rng, 1, max(1, 2400000 // longest)),
                longest=longest, kl=rng.choice(["k1", "k2", "k3", "none"]),
                reduction=rng.choice(["token", "sequence"]), per_sequence=rng.random() < 0.5,
                masked=rng.choice([0.0, 0.2]))


# ----------------------------------------------------------------------------
# Inputs
# ----------------------------------------------------------------------------

def _generator(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _normal(shape, g, std=1.0, mean=0.0, dtype=torch.float32):
    return (torch.randn(shape, generator=g, device=DEV) * std + mean).to(dtype)


def _ragged(count, longest, g):
    """Offsets of `count` sequences whose lengths spread over a factor of eight, up to about `longest`;
    the total is the case's own, whatever the seed."""
    u = 0.125 + 0.875 * torch.rand(count, generator=g, device=DEV, dtype=torch.float64)
    total = _total(count, longest)
    ends = (u.cumsum(0) * (total / u.sum())).round().long().clamp(0, total)
    ends[-1] = total
    return torch.cat([torch.zeros(1, dtype=torch.long, device=DEV), ends])


def _total(count, longest):
    return max(count, round(count * longest * 0.5625))


def _dead_tokens(offsets, n, share, g):
    """Mask (1: counts) that takes out about `share` of every sequence: its prompt, at the front."""
    if share == 0.0:
        return None
    count = offsets.numel() - 1
    lengths = offsets[1:] - offsets[:-1]
    cut = (lengths * (2.0 * share * torch.rand(count, generator=g, device=DEV))).long()
    seg = torch.searchsorted(offsets[1:], torch.arange(n, device=DEV), right=True)
    return (torch.arange(n, device=DEV) - offsets[seg] >= cut[seg]).to(torch.uint8)


def _norm_inputs(case, seed):
    g = _generator(seed)
    dt, t, d = DTYPES[case["dtype"]], case["rows"], case["cols"]
    s = dict(x=_normal((t, d), g, dtype=dt), residual=_normal((t, d), g, 2.0, dtype=dt),
             post_weight=_normal((d,), g, 0.1, 1.0, dt), pre_weight=_normal((d,), g, 0.1, 1.0, dt),
             gate=None, residual_scale=0.9, eps=1e-6)
    if case["gate"] != "none":
        s["gate"] = _normal((d,) if case["gate"] == "channel" else (t, d), g, 0.2, 0.5, dt)
    if case["direction"] == "both":
        s["grad_norm"] = _normal((t, d), g, 1e-3, dtype=dt)
        s["grad_out_residual"] = _normal((t, d), g, 1e-3, dtype=dt)
    return s


def _head_inputs(case, seed):
    g = _generator(seed)
    dt, t, d, v = DTYPES[case["dtype"]], case["tokens"], case["cols"], case["vocab"]
    head = _normal((v, d), g, d ** -0.5, dtype=dt)
    targets = torch.randint(0, v, (t,), generator=g, device=DEV)
    # logits of standard deviation one; the target's is raised by 0 .. 20, from unsure tokens to certain ones
    lift = 20.0 * torch.rand((t, 1), generator=g, device=DEV)
    hidden = (torch.randn((t, d), generator=g, device=DEV) + lift * head[targets].float()).to(dt)
    if case["ignored"] > 0.0:
        # prompts: runs of tokens that are not scored
        run = 64
        dead = torch.rand((t + run - 1) // run, generator=g, device=DEV) < case["ignored"]
        targets[dead.repeat_interleave(run)[:t]] = -100
    s = dict(hidden=hidden, head=head, targets=targets, scale=1.0)
    if case["direction"] == "both":
        s["grad_logp"] = _normal((t,), g, 1.0 / t)
    return s


def _preference_inputs(case, seed):
    g = _generator(seed)
    dt = DTYPES[case["dtype"]]
    offsets = _ragged(2 * case["pairs"], case["longest"], g)
    n = int(offsets[-1])
    ref = torch.rand(n, generator=g, device=DEV).mul_(0.98).add_(0.01).log_()
    s = dict(offsets=offsets, logp=(ref + _normal((n,), g, 0.1)).to(dt), ref_logp=None,
             mask=_dead_tokens(offsets, n, case["masked"], g), beta=0.1, label_smoothing=0.05, margin=0.1)
    if case["reference"]:
        s["ref_logp"] = ref.to(dt)
    return s


def _policy_inputs(case, seed):
    g = _generator(seed)
    dt = DTYPES[case["dtype"]]
    offsets = _ragged(case["sequences"], case["longest"], g)
    n = int(offsets[-1])
    old = torch.rand(n, generator=g, device=DEV).mul_(0.98).add_(0.01).log_()
    # log ratios in steps of 1/256, none of which falls on a clipping bound, where the gradient jumps
    step = (_normal((n,), g, 0.15) * 256).round() / 256
    s = dict(offsets=offsets, old_logp=old.to(dt), logp=(old + step).to(dt), ref_logp=None,
             advantages=_normal((case["sequences"] if case["per_sequence"] else n,), g),
             mask=_dead_tokens(offsets, n, case["masked"], g), clip_low=0.2, clip_high=0.28, dual_clip=3.0,
             kl_coef=0.0)
    if case["kl"] != "none":
        s["ref_logp"] = (old + _normal((n,), g, 0.2)).to(dt)
        s["kl_coef"] = 0.05
    return s


_INPUTS = {"norm": _norm_inputs, "head": _head_inputs, "preference": _preference_inputs, "policy": _policy_inputs}


def _own_buffers(case, s):
    """Outputs and workspaces that a program allocates once and passes to every call."""
    import matrix_aware_optimizer_amd as mao
    f32 = dict(dtype=torch.float32, device=DEV)
    if case["op"] == "norm":
        b = dict(out_residual=torch.empty_like(s["x"]), out_norm=torch.empty_like(s["x"]))
        if case["direction"] == "both":
            b.update(rstd=torch.empty((2, case["rows"]), **f32), grad_x=torch.empty_like(s["x"]),
                     grad_residual=torch.empty_like(s["x"]), grad_post_weight=torch.empty_like(s["post_weight"]),
                     grad_pre_weight=torch.empty_like(s["pre_weight"]),
                     grad_gate=None if s["gate"] is None else torch.empty_like(s["gate"]))
            b["workspace"] = mao.allocate_workspace(mao.muon_block_norm_backward_workspace_bytes(
                s["x"], post_weight=s["post_weight"], gate=s["gate"], pre_weight=s["pre_weight"]), DEV)
        return b
    if case["op"] == "head":
        t = case["tokens"]
        b = dict(logp=torch.empty(t, **f32), lse=torch.empty(t, **f32), saved=None)
        need = mao.muon_token_logp_workspace_bytes(s["hidden"], s["head"])
        if case["direction"] == "both":
            need = max(need, mao.muon_token_logp_backward_workspace_bytes(s["hidden"], s["head"], use_saved=True))
            b["saved"] = mao.allocate_workspace(mao.muon_token_logp_saved_bytes(s["hidden"], s["head"]), DEV)
            b.update(grad_hidden=torch.empty_like(s["hidden"]), grad_head=torch.empty_like(s["head"]))
        b["workspace"] = mao.allocate_workspace(need, DEV)
        return b
    b = dict(loss=torch.empty(1, **f32), grad_logp=torch.empty_like(s["logp"]))
    if case["op"] == "preference":
        b["rewards"] = torch.empty(s["offsets"].numel() - 1, **f32)
        b["workspace"] = mao.allocate_workspace(mao.muon_preference_loss_workspace_bytes(s["logp"], s["offsets"]), DEV)
    else:
        b["stats"] = torch.empty(4, **f32)
        b["workspace"] = mao.allocate_workspace(mao.muon_policy_loss_workspace_bytes(s["logp"], s["offsets"]), DEV)
    return b


def prepare(case, seed):
    state = _INPUTS[case["op"]](case, seed)
    state["case"] = dict(case)
    if own:
        state["buffers"] = _own_buffers(case, state)
    return state


# ----------------------------------------------------------------------------
# The framework's calls
# ----------------------------------------------------------------------------

def _own_norm(c, s, b):
    import matrix_aware_optimizer_amd as mao
    weights = dict(post_weight=s["post_weight"], gate=s["gate"], pre_weight=s["pre_weight"],
                   residual_scale=s["residual_scale"])
    mao.muon_block_norm(s["x"], s["residual"], b["out_residual"], b["out_norm"], rstd=b.get("rstd"), eps=s["eps"],
                        **weights)
    out = dict(out_residual=b["out_residual"], out_norm=b["out_norm"])
    if c["direction"] == "both":
        mao.muon_block_norm_backward(s["x"], b["out_residual"], b["rstd"], s["grad_norm"], b["grad_x"],
                                     b["grad_residual"], grad_out_residual=s["grad_out_residual"],
                                     grad_post_weight=b["grad_post_weight"], grad_gate=b["grad_gate"],
                                     grad_pre_weight=b["grad_pre_weight"], workspace=b["workspace"], **weights)
        for k in ("grad_x", "grad_residual", "grad_post_weight", "grad_pre_weight"):
            out[k] = b[k]
        if s["gate"] is not None:
            out["grad_gate"] = b["grad_gate"]
    return out


def _own_head(c, s, b):
    import matrix_aware_optimizer_amd as mao
    mao.muon_token_logp(s["hidden"], s["head"], s["targets"], b["logp"], b["lse"], scale=s["scale"],
                        saved=b["saved"], workspace=b["workspace"])
    out = dict(logp=b["logp"])
    if c["direction"] == "both":
        mao.muon_token_logp_backward(s["hidden"], s["head"], s["targets"], b["lse"], s["grad_logp"], b["grad_hidden"],
                                     b["grad_head"], scale=s["scale"], saved=b["saved"], workspace=b["workspace"])
        out.update(grad_hidden=b["grad_hidden"], grad_head=b["grad_head"])
    return out


def _own_preference(c, s, b):
    import matrix_aware_optimizer_amd as mao
    mao.muon_preference_loss(s["logp"], s["offsets"], b["loss"], b["grad_logp"], ref_logp=s["ref_logp"],
                             mask=s["mask"], beta=s["beta"], kind=c["kind"], label_smoothing=s["label_smoothing"],
                             margin=s["margin"], average=c["average"], rewards=b["rewards"], workspace=b["workspace"])
    return dict(loss=b["loss"], rewards=b["rewards"], grad_logp=b["grad_logp"])


def _own_policy(c, s, b):
    import matrix_aware_optimizer_amd as mao
    mao.muon_policy_loss(s["logp"], s["old_logp"], s["advantages"], s["offsets"], b["loss"], b["grad_logp"],
                         ref_logp=s["ref_logp"], mask=s["mask"], clip_low=s["clip_low"], clip_high=s["clip_high"],
                         dual_clip=s["dual_clip"], kl_coef=s["kl_coef"], kl=c["kl"], reduction=c["reduction"],
                         per_sequence=c["per_sequence"], stats=b["stats"], workspace=b["workspace"])
    return dict(loss=b["loss"], stats=b["stats"], grad_logp=b["grad_logp"])


# ----------------------------------------------------------------------------
# The plain forms
# ----------------------------------------------------------------------------

def _plain_norm(c, s):
    dt = s["x"].dtype
    x, r = s["x"].float(), s["residual"].float()
    wp, wq, eps, alpha = s["post_weight"].float(), s["pre_weight"].float(), s["eps"], s["residual_scale"]
    gate = None if s["gate"] is None else s["gate"].float()
    s1 = torch.rsqrt((x * x).mean(1, keepdim=True) + eps)
    xh = x * s1
    a = xh * wp
    y = alpha * r + (a if gate is None else gate * a)
    s2 = torch.rsqrt((y * y).mean(1, keepdim=True) + eps)
    h = y * s2
    out = dict(out_residual=y.to(dt), out_norm=(h * wq).to(dt))
    if c["direction"] == "both":
        dn, dy = s["grad_norm"].float(), s["grad_out_residual"].float()
        dh = dn * wq
        dy = dy + s2 * (dh - h * (dh * h).mean(1, keepdim=True))
        da = dy if gate is None else dy * gate
        dxh = da * wp
        out["grad_x"] = (s1 * (dxh - xh * (dxh * xh).mean(1, keepdim=True))).to(dt)
        out["grad_residual"] = (alpha * dy).to(dt)
        out["grad_post_weight"] = (da * xh).sum(0).to(dt)
        out["grad_pre_weight"] = (dn * h).sum(0).to(dt)
        if gate is not None:
            dg = dy * a
            out["grad_gate"] = (dg.sum(0) if gate.dim() == 1 else dg).to(dt)
    return out


def _plain_head(c, s):
    h, w, y = s["hidden"].float(), s["head"].float(), s["targets"]
    live = y >= 0
    z = h @ w.t()
    if s["scale"] != 1.0:
        z = z * s["scale"]
    m = z.max(1, keepdim=True).values
    lse = m + (z - m).exp().sum(1, keepdim=True).log()
    pick = y.clamp(min=0).unsqueeze(1)
    logp = torch.where(live, (z.gather(1, pick) - lse).squeeze(1), 0.0)
    out = dict(logp=logp)
    if c["direction"] == "both":
        coef = torch.where(live, s["grad_logp"], 0.0).unsqueeze(1) * s["scale"]
        dz = (z - lse).exp() * -coef
        dz.scatter_add_(1, pick, coef)
        out["grad_hidden"] = (dz @ w).to(s["hidden"].dtype)
        out["grad_head"] = (dz.t() @ h).to(s["head"].dtype)
    return out


def _segments(offsets, n):
    return torch.searchsorted(offsets[1:], torch.arange(n, device=offsets.device), right=True)


def _softplus(x):
    return x.clamp(min=0) + (1 + (-x.abs()).exp()).log()


def _plain_preference(c, s):
    lp = s["logp"].float()
    n, count = lp.numel(), s["offsets"].numel() - 1
    seg = _segments(s["offsets"], n)
    live = torch.ones(n, dtype=torch.bool, device=lp.device) if s["mask"] is None else s["mask"] != 0
    diff = lp if s["ref_logp"] is None else lp - s["ref_logp"].float()
    r = torch.zeros(count, device=lp.device).index_add_(0, seg, torch.where(live, diff, 0.0))
    weight = torch.ones(count, device=lp.device)
    if c["average"]:
        weight = 1 / torch.zeros(count, device=lp.device).index_add_(0, seg, live.float()).clamp(min=1)
        r = r * weight
    beta, ls = s["beta"], s["label_smoothing"]
    u = r[0::2] - r[1::2]
    h = beta * u - s["margin"]
    if c["kind"] == "sigmoid":
        loss = (1 - ls) * _softplus(-h) + ls * _softplus(h)
        du = beta * (1 / (1 + (-h).exp()) - (1 - ls))
    elif c["kind"] == "hinge":
        loss = (1 - h).clamp(min=0)
        du = torch.where(h < 1, -beta, 0.0)
    else:
        loss = (u - 1 / (2 * beta)) ** 2
        du = 2 * (u - 1 / (2 * beta))
    per_seq = torch.stack([du, -du], 1).reshape(-1) * weight / (count // 2)
    grad = torch.where(live, per_seq[seg], 0.0)
    return dict(loss=loss.mean().reshape(1), rewards=beta * r, grad_logp=grad.to(s["logp"].dtype))


def _plain_policy(c, s):
    lp, old = s["logp"].float(), s["old_logp"].float()
    n, count = lp.numel(), s["offsets"].numel() - 1
    seg = _segments(s["offsets"], n)
    live = torch.ones(n, dtype=torch.bool, device=lp.device) if s["mask"] is None else s["mask"] != 0
    adv = s["advantages"][seg] if c["per_sequence"] else s["advantages"]
    lo, hi, dual = 1 - s["clip_low"], 1 + s["clip_high"], s["dual_clip"]
    ratio = (lp - old).exp()
    gain = torch.minimum(ratio * adv, ratio.clamp(lo, hi) * adv)
    clipped = ((adv > 0) & (ratio > hi)) | ((adv < 0) & (ratio < lo))
    floor = (adv < 0) & (ratio > dual)
    gain = torch.where(floor, dual * adv, gain)
    clipped = clipped | floor
    token = -gain
    d = torch.where(clipped, 0.0, -ratio * adv)
    kl = torch.zeros_like(lp)
    if c["kl"] != "none":
        delta = s["ref_logp"].float() - lp
        if c["kl"] == "k1":
            kl, dkl = -delta, torch.ones_like(lp)
        elif c["kl"] == "k2":
            kl, dkl = 0.5 * delta * delta, -delta
        else:
            kl, dkl = delta.exp() - delta - 1, 1 - delta.exp()
        token = token + s["kl_coef"] * kl
        d = d + s["kl_coef"] * dkl
    lf = live.float()
    active = lf.sum()
    per_token = 1 / active.clamp(min=1)
    if c["reduction"] == "token":
        weight = lf * per_token
    else:
        lengths = torch.zeros(count, device=lp.device).index_add_(0, seg, lf).clamp(min=1)
        weight = lf / (lengths[seg] * count)
    loss = (torch.where(live, token, 0.0) * weight).sum()
    stats = torch.stack([torch.where(live, kl, 0.0).sum() * per_token, (clipped & live).float().sum() * per_token,
                         torch.where(live, ratio, 0.0).sum() * per_token, active])
    return dict(loss=loss.reshape(1), stats=stats, grad_logp=torch.where(live, d * weight, 0.0).to(s["logp"].dtype))


_PLAIN = {"norm": _plain_norm, "head": _plain_head, "preference": _plain_preference, "policy": _plain_policy}
_OWN = {"norm": _own_norm, "head": _own_head, "preference": _own_preference, "policy": _own_policy}


def run(state):
    case = state["case"]
    if own:
        return _OWN[case["op"]](case, state, state["buffers"])
    return _PLAIN[case["op"]](case, state)


# ----------------------------------------------------------------------------
# What a pass cannot do without
# ----------------------------------------------------------------------------

def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "norm":
        td, d = case["rows"] * case["cols"], case["cols"]
        gate = {"none": 0, "channel": d, "full": td}[case["gate"]]
        byt, fl = 4 * td + 2 * d + gate, 12 * td
        if case["direction"] == "both":
            # backward: x, the new residual and two gradients read, two gradients and the weights' written
            byt, fl = byt + 6 * td + 4 * d + 2 * gate, fl + 24 * td
        return dict(bytes=es * byt, flops=fl)
    if case["op"] == "head":
        t, d, v = case["tokens"], case["cols"], case["vocab"]
        live = max(1, round(t * (1 - case["ignored"])))
        byt, fl = es * (live * d + v * d) + 12 * t, 2 * live * d * v + 4 * live * v
        if case["direction"] == "both":
            byt += es * (live * d + v * d + t * d + v * d) + 12 * t
            fl += 4 * live * d * v + 3 * live * v
        return dict(bytes=byt, flops=fl)
    if case["op"] == "preference":
        n = _total(2 * case["pairs"], case["longest"])
        per = es * (3 if case["reference"] else 2) + (1 if case["masked"] else 0)
        return dict(bytes=n * per + 24 * case["pairs"], flops=4 * n)
    n = _total(case["sequences"], case["longest"])
    per = es * (4 if case["kl"] != "none" else 3) + (1 if case["masked"] else 0) + (0 if case["per_sequence"] else 4)
    return dict(bytes=n * per + 12 * case["sequences"], flops=20 * n)


# ----------------------------------------------------------------------------
# The definitions in 64 bits
# ----------------------------------------------------------------------------

def _exact_norm(c, s):
    f = torch.float64
    x, r, wp, wq = (s[k].to(f) for k in ("x", "residual", "post_weight", "pre_weight"))
    gate = torch.ones_like(wp) if s["gate"] is None else s["gate"].to(f)
    d = x.shape[1]
    inv1 = ((x.square().sum(1) / d + s["eps"]) ** -0.5)[:, None]
    post = wp * x * inv1
    res = s["residual_scale"] * r + gate * post
    inv2 = ((res.square().sum(1) / d + s["eps"]) ** -0.5)[:, None]
    out = dict(out_residual=res, out_norm=wq * res * inv2)
    if c["direction"] == "both":
        gn, gr = s["grad_norm"].to(f), s["grad_out_residual"].to(f)
        # d/dv of v / rms(v): (I - v v^T / (d rms^2)) / rms
        t = gn * wq
        total = gr + inv2 * t - res * inv2 ** 3 * ((t * res).sum(1, keepdim=True) / d)
        t = total * gate * wp
        out["grad_x"] = inv1 * t - x * inv1 ** 3 * ((t * x).sum(1, keepdim=True) / d)
        out["grad_residual"] = s["residual_scale"] * total
        out["grad_post_weight"] = (total * gate * x * inv1).sum(0)
        out["grad_pre_weight"] = (gn * res * inv2).sum(0)
        if s["gate"] is not None:
            out["grad_gate"] = (total * post).sum(0) if s["gate"].dim() == 1 else total * post
    return out


def _exact_head(c, s):
    f = torch.float64
    w, y = s["head"].to(f), s["targets"]
    t = y.numel()
    logp = torch.zeros(t, dtype=f, device=w.device)
    both = c["direction"] == "both"
    if both:
        gh = torch.zeros(s["hidden"].shape, dtype=f, device=w.device)
        gw = torch.zeros_like(w)
    live = torch.nonzero(y >= 0).squeeze(1)
    for rows in live.split(2048):
        h = s["hidden"][rows].to(f)
        logits = s["scale"] * torch.matmul(h, w.T.contiguous())
        logits -= torch.logsumexp(logits, 1, keepdim=True)
        at = torch.arange(rows.numel(), device=w.device)
        logp[rows] = logits[at, y[rows]]
        if both:
            g = s["grad_logp"][rows].to(f) * s["scale"]
            e = -logits.exp_()
            e[at, y[rows]] += 1
            e *= g[:, None]
            gh[rows] = torch.matmul(e, w)
            gw += torch.matmul(e.T.contiguous(), h)
    out = dict(logp=logp)
    if both:
        out.update(grad_hidden=gh, grad_head=gw)
    return out


def _live_values(s, name):
    v = s[name].to(torch.float64)
    return v if s["mask"] is None else v.masked_fill(s["mask"] == 0, 0.0)


def _span_sums(v, offsets):
    run = torch.cat([torch.zeros(1, dtype=v.dtype, device=v.device), v.cumsum(0)])
    return run[offsets[1:]] - run[offsets[:-1]]


def _counts(s, n):
    ones = torch.ones(n, dtype=torch.float64, device=s["logp"].device)
    return ones if s["mask"] is None else (s["mask"] != 0).to(torch.float64)


def _exact_preference(c, s):
    offsets = s["offsets"]
    lengths = offsets[1:] - offsets[:-1]
    m = _counts(s, s["logp"].numel())
    score = _live_values(s, "logp")
    if s["ref_logp"] is not None:
        score = score - _live_values(s, "ref_logp")
    r = _span_sums(score, offsets)
    share = torch.ones_like(r)
    if c["average"]:
        share = _span_sums(m, offsets).clamp(min=1).reciprocal()
    r = r * share
    pairs = r.numel() // 2
    u = r.reshape(pairs, 2)[:, 0] - r.reshape(pairs, 2)[:, 1]
    beta, ls = s["beta"], s["label_smoothing"]
    x = beta * u - s["margin"]
    if c["kind"] == "sigmoid":
        loss = -(1 - ls) * torch.nn.functional.logsigmoid(x) - ls * torch.nn.functional.logsigmoid(-x)
        slope = -beta * ((1 - ls) * torch.sigmoid(-x) - ls * torch.sigmoid(x))
    elif c["kind"] == "hinge":
        loss = torch.relu(1 - x)
        slope = -beta * (x < 1).to(torch.float64)
    else:
        loss = torch.square(u - 0.5 / beta)
        slope = 2 * u - 1 / beta
    each = torch.repeat_interleave(torch.stack((slope, -slope), 1).flatten() * share / pairs, lengths)
    return dict(loss=loss.sum().reshape(1) / pairs, rewards=beta * r, grad_logp=each * m)


def _exact_policy(c, s):
    offsets = s["offsets"]
    lengths = offsets[1:] - offsets[:-1]
    m = _counts(s, s["logp"].numel())
    lp, old = _live_values(s, "logp"), _live_values(s, "old_logp")
    a = s["advantages"].to(torch.float64)
    if c["per_sequence"]:
        a = torch.repeat_interleave(a, lengths)
    rho = torch.exp(lp - old)
    low, high = 1 - s["clip_low"], 1 + s["clip_high"]
    # where the gain is flat in rho: above `high` for a gain, below `low` or above the dual bound for a loss
    flat_value = torch.where(a > 0, torch.full_like(rho, high),
                             torch.where(rho > s["dual_clip"], torch.full_like(rho, s["dual_clip"]),
                                         torch.full_like(rho, low)))
    flat = torch.where(a > 0, rho > high, (a < 0) & ((rho < low) | (rho > s["dual_clip"])))
    term = -a * torch.where(flat, flat_value, rho)
    slope = torch.where(flat, torch.zeros_like(rho), -a * rho)
    kl = torch.zeros_like(rho)
    if c["kl"] != "none":
        x = lp - _live_values(s, "ref_logp")
        if c["kl"] == "k1":
            kl, dk = x, torch.ones_like(x)
        elif c["kl"] == "k2":
            kl, dk = x * x / 2, x
        else:
            kl, dk = torch.expm1(-x) + x, -torch.expm1(-x)
        term, slope = term + s["kl_coef"] * kl, slope + s["kl_coef"] * dk
    total = m.sum()
    per = 1 / total.clamp(min=1)
    if c["reduction"] == "token":
        wt = m * per
    else:
        wt = m * torch.repeat_interleave(1 / (_span_sums(m, offsets).clamp(min=1) * lengths.numel()), lengths)
    stats = torch.stack(((kl * m).sum() * per, (flat.to(m.dtype) * m).sum() * per, (rho * m).sum() * per, total))
    return dict(loss=(term * wt).sum().reshape(1), stats=stats, grad_logp=slope * wt)


_EXACT = {"norm": _exact_norm, "head": _exact_head, "preference": _exact_preference, "policy": _exact_policy}


def exact(case, seed):
    return _EXACT[case["op"]](case, _INPUTS[case["op"]](case, seed))
