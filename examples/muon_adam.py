"""Trains a small two-layer network on two data-parallel replicas: its matrices
with dpg_muon_step, its biases and gains with dpg_step (Adam), as the two are
meant to be used side by side.  Needs a GB300 and the built library:

    python examples/muon_adam.py
"""
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import zero_optimizer_step_gb300 as dpg  # noqa: E402

R, STEPS, BATCH = 2, 60, 512
CAP = 1 << 20


class Group:
    """Flat buffers of some parameters: fp32 masters, bf16 views, R gradients."""

    def __init__(self, params):
        self.params = params
        self.plan = dpg.dpg_plan_buckets([p.numel() for p in params], CAP, R)
        n = self.plan.total_padded
        self.master = torch.zeros(n, device="cuda")
        self.view = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
        self.grads = [torch.zeros(n, dtype=torch.bfloat16, device="cuda") for _ in range(R)]
        for p, o in zip(params, self.plan.param_offset):
            at = slice(int(o), int(o) + p.numel())
            self.master[at] = p.detach().reshape(-1)
            self.view[at] = self.master[at].to(torch.bfloat16)
            p.data = self.view[at].view(p.shape)      # the model reads what the step writes

    def take_grads(self, r):
        for p, o in zip(self.params, self.plan.param_offset):
            self.grads[r][int(o):int(o) + p.numel()] = p.grad.reshape(-1)
            p.grad = None


def main():
    torch.manual_seed(0)
    d, h = 256, 768
    make = lambda *s: (torch.randn(*s, device="cuda") / s[-1] ** 0.5).to(torch.bfloat16).requires_grad_()  # noqa: E731
    flat = lambda n, x: torch.full((n,), x, dtype=torch.bfloat16, device="cuda").requires_grad_()          # noqa: E731
    w1, w2, bias, gain = make(h, d), make(d, h), flat(h, 0.0), flat(d, 1.0)
    target = torch.randn(d, d, device="cuda") / d ** 0.5

    matrices, vectors = Group([w1, w2]), Group([bias, gain])
    shapes = dpg.dpg_plan_matrices(matrices.plan, [h, d], [d, h])
    dpg.dpg_matrices_upload(shapes)                     # tables and workspace now, not in the first step
    momentum = torch.zeros_like(matrices.master)
    update = torch.zeros_like(matrices.view)
    exp_avg, exp_avg_sq = torch.zeros_like(vectors.master), torch.zeros_like(vectors.master)

    for t in range(1, STEPS + 1):
        total = 0.0
        for r in range(R):                              # a replica's share of the batch
            x = torch.randn(BATCH, d, device="cuda")
            y = F.gelu(x.to(torch.bfloat16) @ w1.t() + bias) @ w2.t() * gain
            loss = (y.float() - torch.tanh(x @ target)).square().sum(1).sum()   # sums: the step divides
            loss.backward()
            matrices.take_grads(r)
            vectors.take_grads(r)
            total += float(loss.detach())
        tokens = [BATCH] * R
        lr = 0.02 * (1 - t / (STEPS + 1))
        dpg.dpg_muon_step(matrices.plan, shapes, matrices.grads, tokens, dpg.MuonHParams(lr=lr),
                          matrices.master, momentum, update, [matrices.view])
        dpg.dpg_step(vectors.plan, vectors.grads, tokens, dpg.HParams(lr=1e-3, step=t), vectors.master,
                     exp_avg, exp_avg_sq, [vectors.view])
        if t == 1 or t % 20 == 0:
            print(f"step {t:3d}  loss {total / sum(tokens):.3f}")
    dpg.dpg_matrices_status(shapes)                     # no wait of the steps ran out


if __name__ == "__main__":
    main()
