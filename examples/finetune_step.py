"""Fine-tuning steps on sequences of tokens with a preference or a policy loss, every gradient and update by this library.

A stack of blocks, each a matrix product (torch) between norms:

    y_l = n_l W_l^T;   r_l+1 = r_l + gate_l * rms_norm(y_l) * post_l;   n_l+1 = rms_norm(r_l+1) * pre_l     muon_block_norm
    logp, lse of the target tokens under the vocabulary head, from the last n                               muon_token_logp
    the loss over sequences and its gradient with respect to logp               muon_preference_loss / muon_policy_loss
    back through the head and the norms                          muon_token_logp_backward, muon_block_norm_backward
    W_l by the Muon step; head, norm weights and gates by AdamW                       muon_step, muon_adamw_step

    python examples/finetune_step.py --loss preference --steps 20
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import matrix_aware_optimizer_amd as mao  # noqa: E402

SCHEDULE = [(3.4445, -4.7750, 2.0315)] * 5


class Stack:
    """The parameters, their gradients and optimizer states, and one step's buffers (allocated once, reused by every step)."""

    def __init__(self, tokens, width, vocab, blocks, dtype=torch.float32, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)

        def randn(*shape, std=1.0):
            return (torch.randn(shape, generator=g, device=device) * std).to(dtype)
        self.matrices = [randn(width, width, std=width ** -0.5) for _ in range(blocks)]
        self.head = randn(vocab, width, std=width ** -0.5)
        self.norms = [dict(post_weight=torch.ones(width, device=device, dtype=dtype),
                           gate=torch.full((width,), 0.5, device=device, dtype=dtype),
                           pre_weight=torch.ones(width, device=device, dtype=dtype)) for _ in range(blocks)]
        self.moms = [torch.zeros_like(w) for w in self.matrices]
        self.small = [self.head] + [w for n in self.norms for w in n.values()]
        self.states = [[torch.zeros(w.shape, device=device) for w in self.small] for _ in range(2)]
        self.matrix_grads = [torch.empty_like(w) for w in self.matrices]
        self.head_grad = torch.empty_like(self.head)
        self.norm_grads = [{f"grad_{k}": torch.empty_like(w) for k, w in n.items()} for n in self.norms]

        rows = [torch.empty((tokens, width), device=device, dtype=dtype) for _ in range(3 * blocks + 3)]
        self.y, self.r, self.n = rows[:blocks], rows[blocks:2 * blocks], rows[2 * blocks:3 * blocks]
        self.grad_n, self.grad_y, self.grad_r = rows[3 * blocks:]
        self.rstd = [torch.empty((2, tokens), device=device) for _ in range(blocks)]
        self.logp, self.lse = torch.empty(tokens, device=device), torch.empty(tokens, device=device)
        self.grad_logp, self.loss = torch.empty(tokens, device=device), torch.empty(1, device=device)
        self.saved = mao.allocate_workspace(mao.muon_token_logp_saved_bytes(self.n[-1], self.head), device)
        self.count = 0

    def forward(self, x, targets):
        """logp of the targets; x is both the first block's input and the residual it adds to."""
        n = r = x
        for k, w in enumerate(self.matrices):
            torch.mm(n, w.t(), out=self.y[k])
            mao.muon_block_norm(self.y[k], r, self.r[k], self.n[k], rstd=self.rstd[k], **self.norms[k])
            n, r = self.n[k], self.r[k]
        mao.muon_token_logp(n, self.head, targets, self.logp, self.lse, saved=self.saved)
        return self.logp

    def backward(self, x, targets):
        """Every parameter's gradient from grad_logp."""
        mao.muon_token_logp_backward(self.n[-1], self.head, targets, self.lse, self.grad_logp, self.grad_n,
                                     self.head_grad, saved=self.saved)
        above = None                                    # the gradient that comes down the residual
        for k in reversed(range(len(self.matrices))):
            mao.muon_block_norm_backward(self.y[k], self.r[k], self.rstd[k], self.grad_n, self.grad_y, self.grad_r,
                                         grad_out_residual=above, **self.norms[k], **self.norm_grads[k])
            above = self.grad_r
            torch.mm(self.grad_y.t(), self.n[k - 1] if k else x, out=self.matrix_grads[k])
            torch.mm(self.grad_y, self.matrices[k], out=self.grad_n)

    def update(self, lr_muon, lr_adamw):
        self.count += 1
        mao.muon_step(self.matrices, self.matrix_grads, self.moms, lr=lr_muon, beta=0.95, schedule=SCHEDULE, scale_rule="moonlight")
        grads = [self.head_grad] + [g for n in self.norm_grads for g in n.values()]
        mao.muon_adamw_step(self.small, grads, *self.states, lr=lr_adamw, step=self.count)

    def preference_step(self, x, targets, offsets, ref_logp, mask=None, lr=(1e-3, 1e-3)):
        logp = self.forward(x, targets)
        mao.muon_preference_loss(logp, offsets, self.loss, grad_logp=self.grad_logp, ref_logp=ref_logp, mask=mask, beta=0.1)
        self.backward(x, targets)
        self.update(*lr)
        return self.loss

    def policy_step(self, x, targets, offsets, old_logp, ref_logp, advantages, mask=None, lr=(1e-3, 1e-3)):
        logp = self.forward(x, targets)
        mao.muon_policy_loss(logp, old_logp, advantages, offsets, self.loss, grad_logp=self.grad_logp, ref_logp=ref_logp,
                             mask=mask, kl="k3", kl_coef=0.05, per_sequence=True)
        self.backward(x, targets)
        self.update(*lr)
        return self.loss


def batch(sequences, longest, width, vocab, dtype=torch.float32, device="cuda", seed=1):
    """Inputs, targets (the first quarter of every sequence is prompt, which is not scored), the scored tokens' mask, offsets."""
    g = torch.Generator(device=device).manual_seed(seed)
    lengths = torch.randint(4, longest + 1, (sequences,), generator=g, device=device)
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64, device=device), lengths.cumsum(0)])
    tokens = int(offsets[-1])
    x = torch.randn((tokens, width), generator=g, device=device).to(dtype)
    targets = torch.randint(0, vocab, (tokens,), generator=g, device=device)
    place = torch.arange(tokens, device=device) - torch.repeat_interleave(offsets[:-1], lengths)
    mask = place >= torch.repeat_interleave(lengths // 4, lengths)
    return x, torch.where(mask, targets, -100), mask, offsets


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--loss", choices=["preference", "policy"], default="preference")
    p.add_argument("--steps", type=int, default=10)
    p.add_argument("--sequences", type=int, default=16)
    p.add_argument("--longest", type=int, default=128)
    p.add_argument("--width", type=int, default=512)
    p.add_argument("--vocab", type=int, default=4000)
    p.add_argument("--blocks", type=int, default=2)
    p.add_argument("--dtype", choices=["bf16", "f32"], default="f32")
    a = p.parse_args(argv)
    dtype = {"bf16": torch.bfloat16, "f32": torch.float32}[a.dtype]
    x, targets, mask, offsets = batch(a.sequences, a.longest, a.width, a.vocab, dtype)
    stack = Stack(x.shape[0], a.width, a.vocab, a.blocks, dtype)
    start = stack.forward(x, targets).clone()           # the frozen reference, and the policy that answered
    advantages = torch.linspace(-1.0, 1.0, a.sequences, device=x.device)
    losses = []
    for _ in range(a.steps):
        if a.loss == "preference":
            loss = stack.preference_step(x, targets, offsets, start, mask)
        else:
            loss = stack.policy_step(x, targets, offsets, start, start, advantages, mask)
        losses.append(loss.clone())
    losses = [float(v) for v in losses]
    print(f"{a.loss} loss over {a.steps} steps: " + " ".join(f"{v:.4f}" for v in losses))
    return losses


if __name__ == "__main__":
    main()
