"""The block's step as one path (attention with its bias, norms, experts, head): gradients against torch's autograd in fp64 on the CPU.

In fp32 each operator and product adds rounding of a few 2^-24 relative to its terms, with sums over at most 500 terms; a block
of a dozen of them comes to some 1e-5 of a gradient's norm, and softmax and router carry it on by factors of a few: 3e-4.
"""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "block_step.py")


@pytest.fixture(scope="module")
def example(gpu_lib):
    spec = importlib.util.spec_from_file_location("block_step", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def _reference(b, x, offsets, targets):
    """(loss, gradients by name, gradient of x) with the experts that the block chose."""
    import torch
    w = {k: v.detach().double().cpu().requires_grad_() for k, v in {**b.matrices, **b.small}.items()}
    x = x.double().cpu().requires_grad_()
    rms = lambda v: v * torch.rsqrt((v * v).mean(1, keepdim=True) + 1e-6)
    hw, group = b.head_width, b.heads // b.kv_heads
    qkv = (x @ w["qkv"].t()).unflatten(1, (-1, hw))
    q, k, v = qkv[:, :b.heads], qkv[:, b.heads:b.heads + b.kv_heads], qkv[:, b.heads + b.kv_heads:]
    bmap = b.map.cpu().long()
    reach, out = len(bmap) // 2, []
    off = offsets.tolist()
    for s, e in zip(off, off[1:]):
        i = torch.arange(e - s)
        d = i[None] - i[:, None]
        heads = []
        for h in range(b.heads):
            z = q[s:e, h] @ k[s:e, h // group].t() * hw ** -0.5 + w["bias"][bmap[d.clamp(-reach, reach) + reach], h]
            heads.append(torch.softmax(z.masked_fill(d > 0, -float("inf")), 1) @ v[s:e, h // group])
        out.append(torch.stack(heads, 1))
    a = torch.cat(out).flatten(1)
    r1 = x + w["gate0"] * (rms(a @ w["o"].t()) * w["post0"])
    n1 = rms(r1) * w["pre0"]
    ids = b.experts.cpu()
    weights = torch.softmax((n1 @ w["router"].t()).gather(1, ids), 1)
    m = torch.zeros_like(n1)
    for e in range(b.num_experts):
        y = torch.nn.functional.silu(n1 @ w[f"up{e}"].t()) @ w[f"down{e}"].t()
        m = m + ((ids == e) * weights).sum(1, keepdim=True) * y
    n2 = rms(r1 + w["gate1"] * (rms(m) * w["post1"])) * w["pre1"]
    t = targets.cpu()
    live = t >= 0
    logp = torch.log_softmax(n2 @ w["head"].t(), 1).gather(1, t.clamp(min=0)[:, None])[:, 0]
    loss = -logp[live].mean()
    loss.backward()
    return float(loss.detach()), {k: v.grad for k, v in w.items()}, x.grad


def test_block_gradients_against_autograd(example):
    x, offsets, targets = example.batch(5, 50, 48, 211)
    b = example.Block(x.shape[0], 48, 4, 2, 5, 2, 40, 211)
    loss = b.step(x, offsets, targets, lr=(0.0, 0.0))
    want, grads, gx = _reference(b, x, offsets, targets)
    assert abs(float(loss) - want) <= 1e-5 * abs(want)
    for k, g in list(grads.items()) + [("x", gx)]:
        got = (b.gx if k == "x" else b.grads[k]).double().cpu()
        assert float((got - g).norm()) <= 3e-4 * float(g.norm()), k


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_block_example_runs(example, dtype):
    losses = example.main(["--steps", "3", "--sequences", "4", "--longest", "80", "--width", "128", "--heads", "4", "--experts", "4", "--hidden",
                           "96", "--vocab", "500", "--dtype", dtype])
    assert len(losses) == 3 and all(v == v and abs(v) < 100 for v in losses)
