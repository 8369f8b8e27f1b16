"""The fp64 oracle of the operators inside a block against things other than itself: autograd in fp64, central differences,
closed forms, and the cases where a definition has to be chosen."""
import numpy as np
import pytest
import torch

from oracle import block_oracle as bo

RNG = np.random.default_rng


def _inputs(seed, nq, nk, heads, kv, width):
    r = RNG(seed)
    return (r.standard_normal((sum(nq), heads, width)), r.standard_normal((sum(nk), kv, width)),
            r.standard_normal((sum(nk), kv, width)), r.standard_normal((sum(nq), heads, width)))


@pytest.mark.parametrize("causal,window,masked", [(False, 0, False), (True, 0, True), (True, 3, False), (False, 4, True)])
def test_attention_matches_autograd(causal, window, masked):
    nq, nk = [5, 0, 3, 1], [5, 2, 6, 0]
    q, k, v, g = _inputs(1, nq, nk, 4, 2, 3)
    r = RNG(2)
    bias, bmap = r.standard_normal((5, 4)), r.integers(0, 5, 7)
    mask = r.random(sum(nk)) > 0.3 if masked else None
    off, koff = np.cumsum([0] + nq), np.cumsum([0] + nk)
    got = bo.attention(q, k, v, offsets=off, key_offsets=koff, mask=mask, bias=bias, bucket_map=bmap, scale=0.7, causal=causal,
                       window=window, grad_out=g)
    Q, K, V, B = (torch.tensor(t, requires_grad=True) for t in (q, k, v, bias))
    loss = 0.0
    for s in range(4):
        for h in range(4):
            for i in range(nq[s]):
                zs, at = [], []
                for j in range(nk[s]):
                    d = j - (i + nk[s] - nq[s])
                    if (causal and d > 0) or (window and abs(d) >= window) or (masked and not mask[koff[s] + j]):
                        continue
                    zs.append(0.7 * (Q[off[s] + i, h] * K[koff[s] + j, h // 2]).sum() + B[int(bmap[min(max(d, -3), 3) + 3]), h])
                    at.append(koff[s] + j)
                if not zs:
                    assert got["lse"][off[s] + i, h] == -np.inf and not got["out"][off[s] + i, h].any()
                    continue
                z = torch.stack(zs)
                o = (torch.softmax(z, 0)[:, None] * V[at, h // 2]).sum(0)
                assert np.allclose(o.detach(), got["out"][off[s] + i, h])
                assert np.isclose(float(torch.logsumexp(z, 0).detach()), got["lse"][off[s] + i, h])
                loss = loss + (o * torch.tensor(g[off[s] + i, h])).sum()
    loss.backward()
    for leaf, key in ((Q, "q"), (K, "k"), (V, "v"), (B, "bias")):
        assert np.allclose(leaf.grad.numpy(), got[key], rtol=1e-10, atol=1e-12), key


def test_attention_gradients_match_differences():
    nq, nk = [4], [7]
    q, k, v, g = _inputs(3, nq, nk, 2, 1, 3)
    bias, bmap = RNG(4).standard_normal((3, 2)), np.array([0, 1, 2, 1, 0])
    kw = dict(bucket_map=bmap, scale=0.5, causal=True)
    grads = bo.attention(q, k, v, bias=bias, grad_out=g, **kw)
    for name, t in (("q", q), ("k", k), ("v", v), ("bias", bias)):
        d = RNG(5).standard_normal(t.shape)
        step = 1e-5
        ends = []
        for sign in (1, -1):
            args = dict(q=q, k=k, v=v, bias=bias)
            args[name] = t + sign * step * d
            ends.append((bo.attention(args["q"], args["k"], args["v"], bias=args["bias"], **kw)["out"] * g).sum())
        assert np.isclose((ends[0] - ends[1]) / (2 * step), (grads[name] * d).sum(), rtol=1e-7)


def test_attention_sees_one_key_or_all_alike():
    q, k, v, g = _inputs(6, [3], [3], 1, 1, 4)
    one = bo.attention(q, k, v, window=1, grad_out=g)             # each query its own key
    assert np.allclose(one["out"], v) and np.allclose(one["v"], g) and np.allclose(one["q"], 0) and np.allclose(one["k"], 0)
    flat = bo.attention(q * 0, k, v)
    assert np.allclose(flat["out"], v.mean(0)) and np.allclose(flat["lse"], np.log(3))
    buckets = bo.attention(q * 0, k, v, bias=np.array([[0.0], [-np.inf]]), bucket_map=np.array([1, 0, 1]))
    assert np.allclose(buckets["out"], v)                          # a bucket of -infinity hides its distances


def test_masked_keys_and_rows_of_no_sequence_reach_nothing():
    q, k, v, g = _inputs(7, [6], [6], 2, 2, 4)
    mask = np.array([1, 0, 1, 1, 0, 1])
    off = np.array([1, 5])
    a = bo.attention(q, k, v, offsets=off, mask=mask, grad_out=g)
    k2, v2, q2, g2 = k.copy(), v.copy(), q.copy(), g.copy()
    for t in (k2, v2):
        t[[0, 1, 4, 5]] = np.nan
    q2[[0, 5]] = np.nan
    g2[[0, 5]] = np.nan
    b = bo.attention(q2, k2, v2, offsets=off, mask=mask, grad_out=g2)
    for key in ("out", "lse", "q", "k", "v"):
        assert np.array_equal(a[key], b[key]), key
    assert not a["k"][[0, 1, 4, 5]].any() and not a["q"][[0, 5]].any() and np.isinf(a["lse"][0]).all()


def test_expert_calls_match_autograd_and_indexing():
    r = RNG(8)
    experts = np.array([[2, 0], [0, 0], [-1, 3], [1, 2], [7, 2]])
    x, w, g = r.standard_normal((5, 3)), r.standard_normal((5, 2)), r.standard_normal((5, 3))
    s, slots, off = bo.expert_sort(x, experts, 4)
    assert off.tolist() == [0, 3, 4, 7, 8]
    assert slots.tolist() == [[4, 0], [1, 2], [-1, 7], [3, 5], [-1, 6]]
    assert np.array_equal(s[:8], x[[0, 1, 1, 3, 0, 3, 4, 2]]) and not s[8:].any()
    X, W = torch.tensor(x, requires_grad=True), torch.tensor(w, requires_grad=True)
    rows = torch.cat([X[[0, 1, 1, 3, 0, 3, 4, 2]], torch.zeros(2, 3, dtype=torch.float64)])
    Y = (rows * torch.arange(1.0, 11.0)[:, None].double()).detach().requires_grad_()
    out = torch.stack([sum((W[t, c] * Y[slots[t, c]] for c in range(2) if slots[t, c] >= 0), torch.zeros(3, dtype=torch.float64)) for t in range(5)])
    assert np.allclose(out.detach(), bo.expert_combine(Y.detach(), slots, w))
    (out * torch.tensor(g)).sum().backward()
    gy, gw = bo.expert_combine_backward(g, Y.detach().numpy(), slots, w)
    assert np.allclose(Y.grad, gy) and np.allclose(W.grad, gw)
    gs = r.standard_normal((10, 3))
    (rows * torch.tensor(gs)).sum().backward()
    assert np.allclose(X.grad, bo.expert_sort_backward(gs, slots))
