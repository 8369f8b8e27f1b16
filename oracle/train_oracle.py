"""The training operators in fp64, from their definitions: norms around a block, token
log-probabilities over a vocabulary head, the preference loss and the clipped policy loss,
each with its gradients.  Test infrastructure; shares no code with the HIP path.
"""
from __future__ import annotations

import numpy as np


def _f(x):
    return None if x is None else np.asarray(x, np.float64)


# ---- norms around a block -----------------------------------------------------

def block_norm(x, residual, *, post_weight=None, gate=None, pre_weight=None, residual_scale=1.0, eps=1e-6):
    """dict(r, n, rstd0, rstd1): r' = alpha residual + gate (x rstd0 post_weight), n = r' rstd1 pre_weight."""
    x, r, wp, g, wq = map(_f, (x, residual, post_weight, gate, pre_weight))
    rows = x.shape[0]
    s0 = np.ones(rows) if wp is None else 1.0 / np.sqrt((x * x).mean(1) + eps)
    a = x if wp is None else x * s0[:, None] * wp
    y = residual_scale * r + (a if g is None else g * a)
    s1 = np.ones(rows) if wq is None else 1.0 / np.sqrt((y * y).mean(1) + eps)
    return dict(r=y, n=None if wq is None else y * s1[:, None] * wq, rstd0=s0, rstd1=s1)


def block_norm_backward(x, r, rstd0, rstd1, grad_n, grad_r, *, post_weight=None, gate=None, pre_weight=None,
                        residual_scale=1.0):
    """Gradients from the forward pass's r' and inverse rms; grad_n or grad_r may be None."""
    x, r, wp, g, wq, dn, dr = map(_f, (x, r, post_weight, gate, pre_weight, grad_n, grad_r))
    s0, s1 = np.asarray(rstd0, np.float64)[:, None], np.asarray(rstd1, np.float64)[:, None]
    total = np.zeros_like(x) if dr is None else dr.copy()
    out = dict(post_weight=None, gate=None, pre_weight=None)
    if wq is not None:
        out["pre_weight"] = np.zeros_like(wq)
    if dn is not None:
        h = r * s1
        dh = dn * wq
        total += s1 * (dh - h * (dh * h).mean(1, keepdims=True))
        out["pre_weight"] = (dn * h).sum(0)
    xh = x * s0 if wp is not None else x
    a = xh if wp is None else xh * wp
    da = total if g is None else total * g
    if g is not None:
        out["gate"] = (total * a).sum(0) if g.ndim == 1 else total * a
    if wp is None:
        out["x"] = da
    else:
        dxh = da * wp
        out["x"] = s0 * (dxh - xh * (dxh * xh).mean(1, keepdims=True))
        out["post_weight"] = (da * xh).sum(0)
    out["residual"] = residual_scale * total
    return out


# ---- token log-probabilities ----------------------------------------------------

def token_logp(hidden, head, targets, *, scale=1.0):
    """(logp, lse, z): negative targets give logp = lse = 0, targets beyond the vocabulary logp = NaN."""
    h, w, y = _f(hidden), _f(head), np.asarray(targets)
    live = y >= 0
    z = np.zeros((h.shape[0], w.shape[0]))
    z[live] = scale * (h[live] @ w.T)
    m = z.max(1, keepdims=True)
    lse = (m + np.log(np.exp(z - m).sum(1, keepdims=True)))[:, 0]
    logp = np.full(len(y), np.nan)
    ok = live & (y < w.shape[0])
    logp[ok] = z[ok, y[ok]] - lse[ok]
    logp[~live] = 0.0
    return logp, np.where(live, lse, 0.0), z


def token_logp_backward(hidden, head, targets, grad_logp, *, scale=1.0):
    """(grad_hidden, grad_head, dz, p)."""
    h, w, y, c = _f(hidden), _f(head), np.asarray(targets), _f(grad_logp)
    live = y >= 0
    _, lse, z = token_logp(h, w, y, scale=scale)
    p = np.where(live[:, None], np.exp(z - lse[:, None]), 0.0)
    dz = -p
    ok = np.nonzero(live & (y < w.shape[0]))[0]
    dz[ok, y[ok]] += 1.0
    dz *= np.where(live, scale * c, 0.0)[:, None]
    h = np.where(live[:, None], h, 0.0)
    return dz @ w, dz.T @ h, dz, p


# ---- losses -----------------------------------------------------------------------

def _spans(offsets, n):
    """(first, end) of every sequence, clamped to the tokens there are."""
    o = np.clip(np.asarray(offsets, np.int64), 0, n)
    return [(int(a), int(max(a, b))) for a, b in zip(o[:-1], o[1:])]


def _softplus(x):
    return np.logaddexp(0.0, x)


def preference_loss(logp, offsets, *, ref_logp=None, mask=None, beta=0.1, kind="sigmoid", label_smoothing=0.0,
                    margin=0.0, average=False, grad_scale=1.0):
    """dict(loss, rewards, grad, size): size is the sum of |terms| of each sequence's log ratio."""
    lp, ref = _f(logp), _f(ref_logp)
    n = lp.shape[0]
    live = np.ones(n, bool) if mask is None else np.asarray(mask) != 0
    spans = _spans(offsets, n)
    r, wt, size = np.zeros(len(spans)), np.ones(len(spans)), np.zeros(len(spans))
    for s, (a, b) in enumerate(spans):
        on = live[a:b]
        d = lp[a:b][on] - (ref[a:b][on] if ref is not None else 0.0)
        if average:
            wt[s] = 1.0 / max(1, int(on.sum()))
        r[s] = d.sum() * wt[s]
        size[s] = np.abs(d).sum() * wt[s]
    pairs = len(spans) // 2
    u = r[0::2] - r[1::2]
    h = beta * u - margin
    e = label_smoothing
    if kind == "sigmoid":
        loss = (1 - e) * _softplus(-h) + e * _softplus(h)
        du = beta * (e / (1 + np.exp(-h)) - (1 - e) / (1 + np.exp(h)))
    elif kind == "hinge":
        loss, du = np.maximum(0.0, 1 - h), np.where(h < 1, -beta, 0.0)
    else:
        loss, du = (u - 0.5 / beta) ** 2, 2 * (u - 0.5 / beta)
    grad = np.zeros(n)
    for s, (a, b) in enumerate(spans):
        f = du[s // 2] * (1.0 if s % 2 == 0 else -1.0) * wt[s] / pairs * grad_scale
        grad[a:b] = np.where(live[a:b], f, 0.0)
    return dict(loss=loss.mean() if pairs else 0.0, losses=loss, rewards=beta * r, grad=grad, size=size, h=h, u=u)


def policy_loss(logp, old_logp, advantages, offsets, *, ref_logp=None, mask=None, clip_low=0.2, clip_high=0.2,
                dual_clip=0.0, kl_coef=0.0, kl="none", reduction="token", per_sequence=False, grad_scale=1.0):
    """dict(loss, stats, grad, size, grad_size): the sizes are sums of |terms| (for error bounds)."""
    lp, old, ref, adv = map(_f, (logp, old_logp, ref_logp, advantages))
    n = lp.shape[0]
    live = np.ones(n, bool) if mask is None else np.asarray(mask) != 0
    spans = _spans(offsets, n)
    inside = np.zeros(n, bool)
    a_tok, per_seq_count, seq_of = np.zeros(n), np.zeros(len(spans)), np.zeros(n, np.int64)
    for s, (a, b) in enumerate(spans):
        inside[a:b] = True
        seq_of[a:b] = s
        a_tok[a:b] = adv[s] if per_sequence else adv[a:b]
        per_seq_count[s] = live[a:b].sum()
    live = live & inside
    t = np.nonzero(live)[0]
    A, rho = a_tok[t], np.exp(lp[t] - old[t])
    lo, hi = 1 - clip_low, 1 + clip_high
    gain = np.minimum(rho * A, np.clip(rho, lo, hi) * A)
    held = ((A > 0) & (rho > hi)) | ((A < 0) & (rho < lo))
    if dual_clip > 0:
        dual = (A < 0) & (rho > dual_clip)
        gain = np.where(dual, dual_clip * A, gain)
        held = held | dual
    d = np.where(held, 0.0, -rho * A)
    k, dk, ksize = np.zeros_like(rho), np.zeros_like(rho), np.zeros_like(rho)
    if kl != "none":
        q = ref[t] - lp[t]
        if kl == "k1":
            k, dk, ksize = -q, np.ones_like(q), np.abs(q)
        elif kl == "k2":
            k, dk, ksize = 0.5 * q * q, -q, q * q
        else:
            k, dk, ksize = np.expm1(q) - q, -np.expm1(q), np.abs(np.expm1(q)) + np.abs(q)
    l = -gain + kl_coef * k
    count = max(1, len(t))
    if reduction == "token":
        w = np.full(len(t), 1.0 / count)
    else:
        w = 1.0 / (np.maximum(per_seq_count[seq_of[t]], 1.0) * max(1, len(spans)))
    grad, gsize = np.zeros(n), np.zeros(n)
    grad[t] = (d + kl_coef * dk) * w * grad_scale
    gsize[t] = (np.abs(d) + abs(kl_coef) * (np.abs(dk) + 1e-30)) * w * abs(grad_scale)
    stats = np.array([k.sum() / count, held.sum() / count, rho.sum() / count, len(t)])
    return dict(loss=float((l * w).sum()), stats=stats, grad=grad, rho=rho, live=live,
                size=float(((np.abs(gain) + abs(kl_coef) * ksize) * w).sum()), grad_size=gsize, ksize=ksize.sum() / count)
