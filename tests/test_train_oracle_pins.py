"""The training operators' fp64 oracle against things other than itself: autograd in fp64,
central differences, closed forms, and the cases where a definition has to be chosen."""
import numpy as np
import pytest
import torch

from oracle import train_oracle as to

RNG = np.random.default_rng


def _t(x):
    return None if x is None else torch.tensor(x, dtype=torch.float64, requires_grad=True)


@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("gate", ["none", "channel", "full"])
@pytest.mark.parametrize("pre", [True, False])
def test_block_norm_gradients_match_autograd(post, gate, pre):
    rng = RNG(3)
    t, d, alpha, eps = 5, 7, 0.7, 1e-3
    x, r = rng.standard_normal((t, d)), rng.standard_normal((t, d))
    wp = rng.standard_normal(d) if post else None
    wq = rng.standard_normal(d) if pre else None
    g = {"none": None, "channel": rng.standard_normal(d), "full": rng.standard_normal((t, d))}[gate]
    gn = rng.standard_normal((t, d)) if pre else None
    gr = rng.standard_normal((t, d))
    kw = dict(post_weight=wp, gate=g, pre_weight=wq, residual_scale=alpha)
    f = to.block_norm(x, r, eps=eps, **kw)
    b = to.block_norm_backward(x, f["r"], f["rstd0"], f["rstd1"], gn, gr, **kw)
    X, R, WP, WQ, GT = map(_t, (x, r, wp, wq, g))
    a = X if WP is None else X / torch.sqrt((X * X).mean(1, keepdim=True) + eps) * WP
    y = alpha * R + (a if GT is None else GT * a)
    loss = (y * torch.tensor(gr)).sum()
    assert np.allclose(y.detach().numpy(), f["r"])
    if pre:
        n = y / torch.sqrt((y * y).mean(1, keepdim=True) + eps) * WQ
        assert np.allclose(n.detach().numpy(), f["n"])
        loss = loss + (n * torch.tensor(gn)).sum()
    loss.backward()
    for leaf, key in ((X, "x"), (R, "residual"), (WP, "post_weight"), (GT, "gate"), (WQ, "pre_weight")):
        if leaf is not None:
            assert np.allclose(leaf.grad.numpy(), b[key], rtol=1e-10, atol=1e-12), key


def test_token_logp_gradients_match_autograd_and_ignored_tokens_are_out():
    rng = RNG(4)
    t, d, v = 6, 5, 9
    h, w, c = rng.standard_normal((t, d)), rng.standard_normal((v, d)), rng.standard_normal(t)
    y = np.array([0, 8, -100, 3, 3, -1])
    logp, lse, _ = to.token_logp(h, w, y, scale=0.5)
    H, W = _t(h), _t(w)
    full = torch.log_softmax(0.5 * H @ W.T, 1)
    live = y >= 0
    assert np.allclose(logp[live], full.detach().numpy()[live, y[live]])
    assert np.all(logp[~live] == 0) and np.all(lse[~live] == 0)
    (full[torch.tensor(live), torch.tensor(y[live])] * torch.tensor(c[live])).sum().backward()
    gh, gw, dz, _ = to.token_logp_backward(h, w, y, c, scale=0.5)
    assert np.allclose(gh, H.grad.numpy()) and np.allclose(gw, W.grad.numpy())
    assert np.allclose(dz.sum(1), 0.0)
    # what an ignored token holds does not matter
    h2 = h.copy()
    h2[~live] = np.nan
    assert np.array_equal(to.token_logp_backward(h2, w, y, c, scale=0.5)[1], gw)


def _difference(fn, x, eps=1e-6):
    g = np.zeros_like(x)
    for i in range(x.size):
        up, dn = x.copy(), x.copy()
        up[i] += eps
        dn[i] -= eps
        g[i] = (fn(up) - fn(dn)) / (2 * eps)
    return g


@pytest.mark.parametrize("kind", ["sigmoid", "hinge", "squared"])
@pytest.mark.parametrize("average", [False, True])
def test_preference_gradient_matches_differences(kind, average):
    rng = RNG(5)
    offsets = np.array([1, 4, 4, 9, 12])           # a token before the first, an empty sequence, two after
    n = 14
    lp, ref = -rng.random(n), -rng.random(n)
    mask = np.ones(n, np.uint8)
    mask[[2, 7]] = 0
    kw = dict(ref_logp=ref, mask=mask, beta=0.7, kind=kind, label_smoothing=0.1, margin=0.2, average=average)
    out = to.preference_loss(lp, offsets, **kw)
    num = _difference(lambda v: to.preference_loss(v, offsets, **kw)["loss"], lp)
    assert np.allclose(out["grad"], num, atol=1e-8)
    assert out["grad"][0] == 0 and out["grad"][2] == 0 and np.all(out["grad"][12:] == 0)


def test_preference_closed_forms():
    # equal sequences: log 2; a hinge that is met: 0 with no gradient; no pairs: 0
    o = np.array([0, 3, 6])
    lp = np.array([-1.0, -2.0, -3.0] * 2)
    assert np.isclose(to.preference_loss(lp, o)["loss"], np.log(2.0))
    far = np.array([0.0, 0, 0, -9, -9, -9])
    h = to.preference_loss(far, o, beta=1.0, kind="hinge")
    assert h["loss"] == 0 and not h["grad"].any()
    assert to.preference_loss(np.zeros(3), np.array([0]))["loss"] == 0.0


@pytest.mark.parametrize("kl", ["none", "k1", "k2", "k3"])
@pytest.mark.parametrize("reduction", ["token", "sequence"])
@pytest.mark.parametrize("per_sequence", [True, False])
def test_policy_gradient_matches_differences(kl, reduction, per_sequence):
    rng = RNG(6)
    offsets = np.array([0, 5, 5, 11, 16])
    n = 18
    old = -rng.random(n)
    lp = old + 0.3 * rng.standard_normal(n)
    ref = None if kl == "none" else old + 0.2 * rng.standard_normal(n)
    adv = rng.standard_normal(4 if per_sequence else n)
    mask = np.ones(n, np.uint8)
    mask[[1, 12]] = 0
    kw = dict(ref_logp=ref, mask=mask, clip_low=0.2, clip_high=0.3, dual_clip=1.5, kl_coef=0.0 if kl == "none" else 0.1,
              kl=kl, reduction=reduction, per_sequence=per_sequence)
    out = to.policy_loss(lp, old, adv, offsets, **kw)
    num = _difference(lambda v: to.policy_loss(v, old, adv, offsets, **kw)["loss"], lp)
    assert np.allclose(out["grad"], num, atol=1e-8)
    assert 0 < out["stats"][1] < 1 and out["stats"][3] == 14


def test_policy_closed_forms():
    # rho = 1 everywhere: the loss is minus the mean advantage, KL 0; nothing counted: 0
    o, adv = np.array([0, 2, 4]), np.array([1.0, -3.0])
    lp = np.full(4, -1.5)
    out = to.policy_loss(lp, lp, adv, o, per_sequence=True, ref_logp=lp, kl="k3", kl_coef=1.0)
    assert np.isclose(out["loss"], 1.0) and np.allclose(out["stats"], [0, 0, 1, 4])
    none = to.policy_loss(lp, lp, adv, o, per_sequence=True, mask=np.zeros(4))
    assert none["loss"] == 0 and not none["grad"].any()


@pytest.mark.parametrize("mistake", ["no_mean_term", "target_sign", "pair_order", "clip_both"])
def test_planted_mistakes_are_caught(mistake):
    rng = RNG(8)
    if mistake == "no_mean_term":           # the norm's gradient without its projection
        x = rng.standard_normal((3, 4))
        f = to.block_norm(x, x, post_weight=np.ones(4))
        b = to.block_norm_backward(x, f["r"], f["rstd0"], f["rstd1"], None, x, post_weight=np.ones(4))
        assert np.abs((b["x"] * x).sum(1)).max() < 1e-5          # dx is orthogonal to x up to eps
        assert np.abs((x * f["rstd0"][:, None] * x).sum(1)).max() > 1.0
    elif mistake == "target_sign":
        h, w = rng.standard_normal((2, 3)), rng.standard_normal((4, 3))
        dz = to.token_logp_backward(h, w, np.array([1, 2]), np.ones(2))[2]
        assert dz[0, 1] > 0 and dz[1, 2] > 0 and (np.delete(dz[0], 1) < 0).all()
    elif mistake == "pair_order":
        g = to.preference_loss(np.zeros(4), np.array([0, 2, 4]))["grad"]
        assert (g[:2] < 0).all() and (g[2:] > 0).all()           # descent raises the preferred sequence
    else:
        # a gain is bounded above only: rho < lo with A > 0 keeps its gradient
        o = np.array([0, 1])
        g = to.policy_loss(np.array([-2.0]), np.array([-1.0]), np.array([1.0]), o)["grad"]
        assert g[0] < 0
