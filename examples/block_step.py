"""Fine-tuning steps of one transformer block with experts, every operator, gradient and update by this library.

    q, k, v = x Wqkv^T;  a = attention(q, k, v) with a learned relative position bias        muon_attention
    r1 = x + gate0 * rms_norm(a Wo^T) * post0;  n1 = rms_norm(r1) * pre0                      muon_block_norm
    each token to the experts with its largest scores n1 Wr^T, in the order of the experts    muon_expert_sort
    y = silu(rows W1_e^T) W2_e^T, expert by expert (torch)
    m = the experts' outputs, weighted, back in the order of the tokens                       muon_expert_combine
    r2 = r1 + gate1 * rms_norm(m) * post1;  n2 = rms_norm(r2) * pre1                          muon_block_norm
    mean negative log-probability of the next tokens under the vocabulary head                muon_token_logp
    the way back                                                  the operators' backward calls
    Wqkv, Wo and the experts' matrices by the Muon step; head, router, norms, gates and the bias by AdamW

    python examples/block_step.py --steps 10
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import matrix_aware_optimizer_amd as mao  # noqa: E402

SCHEDULE = [(3.4445, -4.7750, 2.0315)] * 5


def distance_buckets(buckets, reach, device):
    """int32 map of the distances -reach .. reach (key - query, none in front of the query): one bucket each for the near half
    of the buckets, then by factors up to `reach`."""
    near = buckets // 2
    out = []
    for back in range(reach, -reach - 1, -1):
        far = near + int(math.log(max(back, 1) / near) / math.log(reach / near) * (buckets - near)) if back >= near else 0
        out.append(max(back, 0) if back < near else min(buckets - 1, far))
    return torch.tensor(out, dtype=torch.int32, device=device)


class Block:
    """The parameters, their gradients and optimizer states, and one step's buffers (allocated once, reused by every step)."""

    def __init__(self, tokens, width, heads, kv_heads, experts, chosen, hidden, vocab, buckets=8, reach=16, dtype=torch.float32,
                 device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)

        def randn(*shape, std=1.0):
            return (torch.randn(shape, generator=g, device=device) * std).to(dtype)

        def empty(*shape, like=dtype):
            return torch.empty(shape, device=device, dtype=like)
        f32 = torch.float32
        self.heads, self.kv_heads, self.head_width, self.chosen, self.num_experts = heads, kv_heads, width // heads, chosen, experts
        rows = (heads + 2 * kv_heads) * self.head_width
        s = width ** -0.5
        self.matrices = dict(qkv=randn(rows, width, std=s), o=randn(width, width, std=s))
        for e in range(experts):
            self.matrices[f"up{e}"], self.matrices[f"down{e}"] = randn(hidden, width, std=s), randn(width, hidden, std=hidden ** -0.5)
        ones = lambda: torch.ones(width, device=device, dtype=dtype)
        self.small = dict(bias=randn(buckets, heads, std=0.5), router=randn(experts, width, std=s), head=randn(vocab, width, std=s))
        for i in range(2):
            self.small.update({f"post{i}": ones(), f"gate{i}": ones() * 0.5, f"pre{i}": ones()})
        self.map = distance_buckets(buckets, reach, device)
        self.grads = {k: torch.zeros_like(w) for k, w in {**self.matrices, **self.small}.items()}
        self.moms = {k: torch.zeros_like(w) for k, w in self.matrices.items()}
        self.states = [[torch.zeros(w.shape, device=device) for w in self.small.values()] for _ in range(2)]
        self.count = 0

        t, n = tokens, tokens * chosen
        self.qkv, self.gqkv = empty(t, rows), empty(t, rows)
        self.att, self.low, self.gatt = (empty(t, heads, self.head_width) for _ in range(3))
        self.lse_att, self.lse_att_low = empty(t, heads, like=f32), empty(t, heads, like=f32)
        self.o, self.m, self.r1, self.n1, self.r2, self.n2 = (empty(t, width) for _ in range(6))
        self.gn2, self.gm, self.gr1, self.gn1, self.go, self.gx = (empty(t, width) for _ in range(6))
        self.rstd = [empty(2, t, like=f32) for _ in range(2)]
        self.sorted, self.y, self.gy, self.gsorted = (empty(n, width) for _ in range(4))
        self.up = empty(n, hidden)
        self.slots, self.offsets = empty(t, chosen, like=torch.int32), empty(experts + 1, like=torch.int64)
        self.gweights, self.logp, self.lse = empty(t, chosen, like=f32), empty(t, like=f32), empty(t, like=f32)
        self.saved = mao.allocate_workspace(mao.muon_token_logp_saved_bytes(self.n2, self.small["head"]), device)

    def parts(self, qkv):
        """q, k and v as views of the rows that one product makes (or their gradients)."""
        w, h, kv = self.head_width, self.heads, self.kv_heads
        cut = lambda a, n: qkv[:, a * w:(a + n) * w].unflatten(1, (n, w))
        return cut(0, h), cut(h, kv), cut(h + kv, kv)

    def norm(self, i):
        return {k + "_weight" if k != "gate" else k: self.small[f"{k}{i}"] for k in ("post", "gate", "pre")}

    def norm_grads(self, i):
        return {f"grad_{k}_weight" if k != "gate" else "grad_gate": self.grads[f"{k}{i}"] for k in ("post", "gate", "pre")}

    def attention_form(self, offsets):
        return dict(offsets=offsets, bias=self.small["bias"], bucket_map=self.map, causal=True, out_low=self.low,
                    lse_low=self.lse_att_low)

    def forward(self, x, offsets, targets):
        """logp of the targets (< 0: not scored) for sequences packed one after the other."""
        torch.mm(x, self.matrices["qkv"].t(), out=self.qkv)
        mao.muon_attention(*self.parts(self.qkv), self.att, self.lse_att, **self.attention_form(offsets))
        torch.mm(self.att.flatten(1), self.matrices["o"].t(), out=self.o)
        mao.muon_block_norm(self.o, x, self.r1, self.n1, rstd=self.rstd[0], **self.norm(0))
        scores = (self.n1 @ self.small["router"].t()).float()
        self.experts = scores.topk(self.chosen, 1).indices
        self.weights = torch.softmax(scores.gather(1, self.experts), 1)
        mao.muon_expert_sort(self.n1, self.experts, self.sorted, self.slots, self.offsets)
        self.spans = self.offsets.tolist()
        for e, (a, b) in enumerate(zip(self.spans, self.spans[1:])):
            torch.mm(self.sorted[a:b], self.matrices[f"up{e}"].t(), out=self.up[a:b])
            torch.mm(torch.nn.functional.silu(self.up[a:b]), self.matrices[f"down{e}"].t(), out=self.y[a:b])
        mao.muon_expert_combine(self.y, self.slots, self.weights, self.m)
        mao.muon_block_norm(self.m, self.r1, self.r2, self.n2, rstd=self.rstd[1], **self.norm(1))
        mao.muon_token_logp(self.n2, self.small["head"], targets, self.logp, self.lse, saved=self.saved)
        return self.logp

    def backward(self, x, offsets, targets, grad_logp):
        """Every parameter's gradient, and x's in gx."""
        mao.muon_token_logp_backward(self.n2, self.small["head"], targets, self.lse, grad_logp, self.gn2, self.grads["head"], saved=self.saved)
        mao.muon_block_norm_backward(self.m, self.r2, self.rstd[1], self.gn2, self.gm, self.gr1, **self.norm(1), **self.norm_grads(1))
        mao.muon_expert_combine_backward(self.gm, self.y, self.slots, self.weights, self.offsets, self.gy, self.gweights)
        for e, (a, b) in enumerate(zip(self.spans, self.spans[1:])):
            h, s = self.up[a:b], torch.sigmoid(self.up[a:b])
            torch.mm(self.gy[a:b].t(), h * s, out=self.grads[f"down{e}"])
            gh = (self.gy[a:b] @ self.matrices[f"down{e}"]) * (s * (1 + h * (1 - s)))
            torch.mm(gh.t(), self.sorted[a:b], out=self.grads[f"up{e}"])
            torch.mm(gh, self.matrices[f"up{e}"], out=self.gsorted[a:b])
        mao.muon_expert_sort_backward(self.gsorted, self.slots, self.gn1)
        gs = self.weights * (self.gweights - (self.weights * self.gweights).sum(1, keepdim=True))
        gscores = torch.zeros((x.shape[0], self.num_experts), device=x.device).scatter_(1, self.experts, gs).to(x.dtype)
        torch.mm(gscores.t(), self.n1, out=self.grads["router"])
        self.gn1 += gscores @ self.small["router"]
        mao.muon_block_norm_backward(self.o, self.r1, self.rstd[0], self.gn1, self.go, self.gx, grad_out_residual=self.gr1, **self.norm(0),
                                     **self.norm_grads(0))
        torch.mm(self.go.t(), self.att.flatten(1), out=self.grads["o"])
        torch.mm(self.go, self.matrices["o"], out=self.gatt.flatten(1))
        mao.muon_attention_backward(*self.parts(self.qkv), self.att, self.lse_att, self.gatt, *self.parts(self.gqkv),
                                    grad_bias=self.grads["bias"], **self.attention_form(offsets))
        torch.mm(self.gqkv.t(), x, out=self.grads["qkv"])
        self.gx += self.gqkv @ self.matrices["qkv"]

    def step(self, x, offsets, targets, lr=(1e-3, 1e-3)):
        """One step on the mean negative log-probability; returns it."""
        logp = self.forward(x, offsets, targets)
        scored = (targets >= 0).float()
        grad = -scored / scored.sum()
        self.backward(x, offsets, targets, grad)
        self.count += 1
        names = list(self.matrices)
        mao.muon_step([self.matrices[k] for k in names], [self.grads[k] for k in names], [self.moms[k] for k in names], lr=lr[0], beta=0.95,
                      schedule=SCHEDULE, scale_rule="moonlight")
        mao.muon_adamw_step(list(self.small.values()), [self.grads[k] for k in self.small], *self.states, lr=lr[1], step=self.count)
        return (logp * grad).sum()


def batch(sequences, longest, width, vocab, dtype=torch.float32, device="cuda", seed=1):
    """Inputs, next tokens (the last of a sequence has none) and offsets of sequences packed one after the other."""
    g = torch.Generator(device=device).manual_seed(seed)
    lengths = torch.randint(2, longest + 1, (sequences,), generator=g, device=device)
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64, device=device), lengths.cumsum(0)])
    x = torch.randn((int(offsets[-1]), width), generator=g, device=device).to(dtype)
    targets = torch.randint(0, vocab, (x.shape[0],), generator=g, device=device)
    targets[offsets[1:] - 1] = -100
    return x, offsets, targets


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("steps", 10), ("sequences", 8), ("longest", 256), ("width", 512), ("heads", 8), ("kv-heads", 2), ("experts", 8),
                        ("chosen", 2), ("hidden", 1024), ("vocab", 4000)):
        p.add_argument(f"--{name}", type=int, default=value)
    p.add_argument("--dtype", choices=["bf16", "f32"], default="bf16")
    a = p.parse_args(argv)
    dtype = {"bf16": torch.bfloat16, "f32": torch.float32}[a.dtype]
    x, offsets, targets = batch(a.sequences, a.longest, a.width, a.vocab, dtype)
    block = Block(x.shape[0], a.width, a.heads, a.kv_heads, a.experts, a.chosen, a.hidden, a.vocab, dtype=dtype)
    losses = [float(block.step(x, offsets, targets)) for _ in range(a.steps)]
    print(f"loss over {a.steps} steps: " + " ".join(f"{v:.4f}" for v in losses))
    return losses


if __name__ == "__main__":
    main()
