"""Trains a small two-layer network on two data-parallel replicas: its matrices
with dpg_muon_step, its biases and gains with dpg_step (Adam), as the two are
meant to be used side by side.  Needs a GB300 and the built library:

    python examples/muon_adam.py [--fp4]

With --fp4 the inputs are normalised by dpg_layer_norm, and both layers multiply
4-bit forms of activations, weights and gradients (dpg_fp4_product); every operator
leaves its parameters' gradients in the flat buffers that the steps take.
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

    def slot(self, k, r):
        """Where the gradient of parameter k of replica r belongs."""
        o, p = int(self.plan.param_offset[k]), self.params[k]
        return self.grads[r][o:o + p.numel()].view(p.shape)

    def take_grads(self, r):
        for p, o in zip(self.params, self.plan.param_offset):
            if p.grad is not None:                    # (others are where they belong)
                self.grads[r][int(o):int(o) + p.numel()] = p.grad.reshape(-1)
                p.grad = None


class Norm(torch.autograd.Function):
    """Layer norm of rows x; gain's and bias's gradients go to dgain and dbias."""

    @staticmethod
    def forward(ctx, x, gain, bias, dgain, dbias):
        rows, cols = x.shape
        y, mean, rstd = torch.empty_like(x), torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
        dpg.dpg_layer_norm(x, gain, bias, 1e-5, y, mean, rstd)
        ctx.save_for_backward(x, gain, mean, rstd)
        ctx.slots = dgain, dbias
        return y

    @staticmethod
    def backward(ctx, dy):
        x, gain, mean, rstd = ctx.saved_tensors
        dx = torch.empty_like(x) if ctx.needs_input_grad[0] else None
        work = torch.empty(dpg.dpg_layer_norm_workspace(*x.shape), dtype=torch.uint8, device="cuda")
        dpg.dpg_layer_norm_backward(dy.contiguous(), x, gain, mean, rstd, dx, *ctx.slots, work)
        return dx, None, None, None, None


class Linear4(torch.autograd.Function):
    """x W^T with everything in 4 bits.  w: W's forms by row and by column; W's
    gradient goes to dw; the output's gradient is rounded stochastically."""

    @staticmethod
    def forward(ctx, x, w, dw, seed):
        row, ctx.col = dpg.Fp4(*x.shape), dpg.Fp4(*x.shape[::-1])
        dpg.dpg_fp4_quantize(x, row, ctx.col)
        y = torch.empty(x.shape[0], w[0].rows, dtype=x.dtype, device="cuda")
        dpg.dpg_fp4_product(row, w[0], y)
        ctx.w, ctx.dw, ctx.seed = w, dw, seed
        return y

    @staticmethod
    def backward(ctx, dy):
        row, col = dpg.Fp4(*dy.shape), dpg.Fp4(*dy.shape[::-1])
        dpg.dpg_fp4_quantize(dy.contiguous(), row, col, seed=ctx.seed)
        dx = torch.empty(dy.shape[0], ctx.w[1].rows, dtype=dy.dtype, device="cuda")
        dpg.dpg_fp4_product(row, ctx.w[1], dx)
        dpg.dpg_fp4_product(col, ctx.col, ctx.dw)
        return dx, None, None, None


def main(fp4=False):
    torch.manual_seed(0)
    d, h = 256, 768
    make = lambda *s: (torch.randn(*s, device="cuda") / s[-1] ** 0.5).to(torch.bfloat16).requires_grad_()  # noqa: E731
    flat = lambda n, x: torch.full((n,), x, dtype=torch.bfloat16, device="cuda").requires_grad_()          # noqa: E731
    w1, w2, bias, gain = make(h, d), make(d, h), flat(h, 0.0), flat(d, 1.0)
    target = torch.randn(d, d, device="cuda") / d ** 0.5

    norm = [flat(d, 1.0), flat(d, 0.0)] if fp4 else []

    matrices, vectors = Group([w1, w2]), Group([bias, gain] + norm)
    shapes = dpg.dpg_plan_matrices(matrices.plan, [h, d], [d, h])
    dpg.dpg_matrices_upload(shapes)                     # tables and workspace now, not in the first step
    momentum = torch.zeros_like(matrices.master)
    update = torch.zeros_like(matrices.view)
    exp_avg, exp_avg_sq = torch.zeros_like(vectors.master), torch.zeros_like(vectors.master)
    if fp4:
        rows, cols = [dpg.Fp4(h, d), dpg.Fp4(d, h)], [dpg.Fp4(d, h), dpg.Fp4(h, d)]
        dpg.dpg_allgather_params_fp4(shapes, matrices.master, rows, cols)
        # each layer's own, far from the other's: equal seeds would give their gradients equal bits
        seeds = torch.arange(2, dtype=torch.int64, device="cuda") << 32

    for t in range(1, STEPS + 1):
        total = 0.0
        for r in range(R):                              # a replica's share of the batch
            x = torch.randn(BATCH, d, device="cuda")
            if fp4:
                seeds += 1
                n = Norm.apply(x.to(torch.bfloat16).requires_grad_(), *norm, vectors.slot(2, r), vectors.slot(3, r))
                a = F.gelu(Linear4.apply(n, (rows[0], cols[0]), matrices.slot(0, r), seeds[:1]) + bias)
                y = Linear4.apply(a, (rows[1], cols[1]), matrices.slot(1, r), seeds[1:]) * gain
            else:
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
        if fp4:                                         # the next step's weights
            dpg.dpg_allgather_params_fp4(shapes, matrices.master, rows, cols)
        if t == 1 or t % 20 == 0:
            print(f"step {t:3d}  loss {total / sum(tokens):.3f}")
    dpg.dpg_matrices_status(shapes)                     # no wait of the steps ran out
    dpg.dpg_fp4_status()                                # nor of the products


if __name__ == "__main__":
    main("--fp4" in sys.argv[1:])
