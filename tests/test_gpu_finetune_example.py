"""The example's step: gradients of the whole path against torch's autograd in fp64, and losses that go down.

In fp32 a block norm, a product of width d and the head's products each add rounding of a few 2^-24 (the head's operands 2^-21)
relative to their terms, with sums over at most 500 terms: 1e-4 of a gradient's norm is some thirty times what they come to.
"""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "finetune_step.py")


@pytest.fixture(scope="module")
def example(gpu_lib):
    spec = importlib.util.spec_from_file_location("finetune_step", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def _reference(stack, x, targets, mask, offsets, loss_of):
    """loss and gradients of (matrices, head, norms) by autograd on the CPU in fp64."""
    import torch
    par = lambda t: t.detach().double().cpu().requires_grad_()
    ms, head, norms = [par(w) for w in stack.matrices], par(stack.head), [{k: par(w) for k, w in n.items()} for n in stack.norms]
    rms = lambda v: v * torch.rsqrt((v * v).mean(1, keepdim=True) + 1e-6)
    n = r = x.double().cpu()
    for w, p in zip(ms, norms):
        r = r + p["gate"] * (rms(n @ w.t()) * p["post_weight"])
        n = rms(r) * p["pre_weight"]
    t = targets.cpu()
    live = t >= 0
    logp = torch.zeros(len(t), dtype=torch.float64)
    logp = torch.where(live, torch.log_softmax(n @ head.t(), 1).gather(1, t.clamp(min=0)[:, None])[:, 0], logp)
    loss = loss_of(logp, mask.cpu().double(), [int(v) for v in offsets])
    loss.backward()
    return float(loss.detach()), [w.grad for w in ms], head.grad, [{k: w.grad for k, w in p.items()} for p in norms]


@pytest.mark.parametrize("loss", ["preference", "policy"])
def test_finetune_gradients_against_autograd(example, loss):
    import torch
    width, vocab, sequences = 72, 333, 6
    x, targets, mask, offsets = example.batch(sequences, 20, width, vocab)
    stack = example.Stack(x.shape[0], width, vocab, 2)
    start = stack.forward(x, targets).clone()
    ref = start + 0.3 * torch.randn(start.shape, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda")
    adv = torch.linspace(-1.0, 1.0, sequences, device="cuda")
    old, rf, av = start.double().cpu() + 0.01, ref.double().cpu(), adv.double().cpu()

    def preference(logp, m, off):
        s = [((logp - rf) * m)[a:b].sum() for a, b in zip(off, off[1:])]
        return torch.stack([torch.nn.functional.softplus(-0.1 * (s[k] - s[k + 1])) for k in range(0, len(s), 2)]).mean()

    def policy(logp, m, off):
        a = torch.cat([av[k].expand(off[k + 1] - off[k]) for k in range(sequences)])
        rho = torch.exp(logp - old.float().double())
        q = rf - logp
        term = -torch.minimum(rho * a, rho.clamp(0.8, 1.2) * a) + 0.05 * (torch.expm1(q) - q)
        return (term * m).sum() / m.sum()
    want = _reference(stack, x, targets, mask, offsets, preference if loss == "preference" else policy)
    kw = dict(mask=mask, lr=(0.0, 0.0))
    got = (stack.preference_step(x, targets, offsets, ref, **kw) if loss == "preference" else
           stack.policy_step(x, targets, offsets, old.float().cuda(), ref, adv, **kw))
    assert abs(float(got) - want[0]) <= 1e-5 * max(1.0, abs(want[0]))
    pairs = list(zip(stack.matrix_grads, want[1])) + [(stack.head_grad, want[2])]
    pairs += [(g[f"grad_{k}"], w[k]) for g, w in zip(stack.norm_grads, want[3]) for k in w]
    for g, w in pairs:
        assert float((g.double().cpu() - w).norm()) <= 1e-4 * float(w.norm())


@pytest.mark.parametrize("loss,dtype", [("preference", "f32"), ("policy", "f32"), ("preference", "bf16")])
def test_finetune_loss_goes_down(example, loss, dtype):
    losses = example.main(["--loss", loss, "--steps", "8", "--sequences", "8", "--longest", "64", "--width", "256", "--vocab", "1000",
                           "--dtype", dtype])
    assert losses[-1] < losses[0]


def test_token_logp_workspace_serves_both_forms(gpu_lib):
    import torch
    for dtype in (torch.float32, torch.bfloat16):
        for t in (3, 64, 65):
            h, w = torch.randn(t, 40, device="cuda").to(dtype), torch.randn(300, 40, device="cuda").to(dtype)
            y = torch.zeros(t, dtype=torch.int64, device="cuda")
            ws = torch.empty(gpu_lib.muon_token_logp_workspace_bytes(h, w), dtype=torch.uint8, device="cuda")
            saved = torch.empty(gpu_lib.muon_token_logp_saved_bytes(h, w), dtype=torch.uint8, device="cuda")
            logp, lse = torch.empty(t, device="cuda"), torch.empty(t, device="cuda")
            for keep in (None, saved):
                gpu_lib.muon_token_logp(h, w, y, logp, lse, saved=keep, workspace=ws)
            torch.cuda.synchronize()
