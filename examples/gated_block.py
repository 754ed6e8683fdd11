"""Language model blocks on a gated linear recurrence, trained and served.

    x, r, i, z = in(y);  h = scan(x, r, i);  o = out(norm(h) act(z))
    s = s + scale norm(o);  y = norm(s)

Training runs with the library's kernels under torch's autograd: the gated scan
and the norms around a block, each with its gradient.  Serving keeps the weights
of both products in 4 bits: a long prompt multiplies by the values that they
stand for and fills the recurrence's states, and then each token takes one step
on them, with products on the 4 bits themselves.

    python examples/gated_block.py
"""
import os
import sys

import torch
import torch.nn.functional as F
from torch.autograd.function import once_differentiable

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from nonlinear_rnn_evaluation_newton_amd import binding as bd  # noqa: E402

BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8


def like(t, *shape, dtype=None):
    return torch.empty(*shape, dtype=dtype or t.dtype, device=t.device)


def workspace(n):
    return torch.empty(n, dtype=U8, device="cuda")


class Scan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, r, i, decay, r_bias, i_bias):
        y, states = like(x, *x.shape), like(decay, *bd.gated_states_shape(*x.shape))
        ws = workspace(bd.gated_workspace_bytes(x.dtype, *x.shape, with_adjoint=False))
        bd.gated_scan(x, r, i, decay, y, ws, r_bias=r_bias, i_bias=i_bias, states=states)
        ctx.save_for_backward(x, r, i, decay, r_bias, i_bias, states)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, r, i, decay, r_bias, i_bias, states = ctx.saved_tensors
        new = lambda t: like(t, *t.shape)  # noqa: E731
        g = dict(dx=new(x), dr=new(r), di=new(i), ddecay=new(decay), dr_bias=new(r_bias), di_bias=new(i_bias))
        bd.gated_scan_adjoint(x, r, i, decay, states, dy.contiguous(), workspace(bd.gated_workspace_bytes(x.dtype, *x.shape)),
                              r_bias=r_bias, i_bias=i_bias, **g)
        return tuple(g.values())


class Norm(torch.autograd.Function):
    """norm(x) w act(z): the norm at a block's start (no gate) and the one after the recurrence."""
    @staticmethod
    def forward(ctx, x, w, z):
        t, n = like(x, *x.shape), x.shape[-1]
        bd.block_norm(x.view(-1, n), w, t.view(-1, n), z=None if z is None else rows(z))
        ctx.save_for_backward(x, w, z)
        return t

    @staticmethod
    @once_differentiable
    def backward(ctx, dt):
        x, w, z = ctx.saved_tensors
        n, count = x.shape[-1], x.numel() // x.shape[-1]
        dx, dw, dz = like(x, count, n), like(w, n, dtype=F32), None if z is None else like(x, count, n)
        bd.block_norm_adjoint(x.view(-1, n), w, dx, workspace(bd.block_norm_workspace_bytes(x.dtype, count, n)),
                              z=None if z is None else rows(z), dt=dt.contiguous().view(-1, n), dz=dz, dw=dw)
        return dx.view(x.shape), dw.to(w.dtype), None if z is None else dz.view(z.shape)


class Join(torch.autograd.Function):
    """The stream that goes on, t = s + norm(x) w scale, and norm(t) w_next for the next block."""
    @staticmethod
    def forward(ctx, x, w, scale, s, w_next):
        n, t, y = x.shape[-1], like(x, *x.shape), like(x, *x.shape)
        bd.block_norm(x.view(-1, n), w, t.view(-1, n), scale=scale, residual=s.view(-1, n), y=y.view(-1, n), w_next=w_next)
        ctx.save_for_backward(x, w, scale, w_next, t)
        return t, y

    @staticmethod
    @once_differentiable
    def backward(ctx, dt, dy):
        x, w, scale, w_next, t = ctx.saved_tensors
        n, count = x.shape[-1], x.numel() // x.shape[-1]
        g = dict(dres=like(x, count, n), dw=like(w, n, dtype=F32), dscale=like(w, n, dtype=F32), dw_next=like(w, n, dtype=F32))
        dx = like(x, count, n)
        bd.block_norm_adjoint(x.view(-1, n), w, dx, workspace(bd.block_norm_workspace_bytes(x.dtype, count, n)),
                              scale=scale, w_next=w_next, t=t.view(-1, n), dt=dt.contiguous().view(-1, n),
                              dy=dy.contiguous().view(-1, n), **g)
        return (dx.view(x.shape), g["dw"].to(w.dtype), g["dscale"].to(w.dtype), g["dres"].view(x.shape),
                g["dw_next"].to(w.dtype))


def rows(z):
    """[.., n] as [rows, n]: in place where the rows lie at one stride, as slices of a wider projection do."""
    n = z.shape[-1]
    if z.dim() == 2 and z.stride(1) == 1:
        return z
    if z.dim() == 3 and z.stride(2) == 1 and z.stride(0) == z.shape[1] * z.stride(1):
        return z.as_strided((z.shape[0] * z.shape[1], n), (z.stride(1), 1), z.storage_offset())
    return z.reshape(-1, n).contiguous()


class Model:
    """A few blocks; y [B, T, dim], normed, for whatever reads it."""

    def __init__(self, dim=256, width=512, blocks=2, group=64, dtype=BF, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.dim, self.width, self.group = dim, width, group

        def normal(*shape, std=1.0, mean=0.0, to=dtype):
            return (torch.randn(*shape, generator=g) * std + mean).to(to).cuda().requires_grad_()

        self.first = normal(dim, std=0.1, mean=1.0)
        self.blocks = [dict(
            inp=normal(4 * width, dim, std=dim ** -0.5), out=normal(dim, width, std=width ** -0.5),
            decay=(torch.rand(width, generator=g) * 0.8 + 0.05).cuda().requires_grad_(),
            r_bias=normal(width, to=F32), i_bias=normal(width, to=F32), norm=normal(width, std=0.1, mean=1.0),
            post=normal(dim, std=0.1, mean=1.0), scale=normal(dim, std=0.02, mean=0.3), after=normal(dim, std=0.1, mean=1.0))
            for _ in range(blocks)]

    def parameters(self):
        return [self.first] + [v for b in self.blocks for v in b.values()]

    def forward(self, s):
        y, c = Norm.apply(s, self.first, None), self.width
        for w in self.blocks:
            p = F.linear(y, w["inp"])
            h = Scan.apply(p[..., :c], p[..., c:2 * c], p[..., 2 * c:3 * c], w["decay"], w["r_bias"], w["i_bias"])
            o = F.linear(Norm.apply(h, w["norm"], p[..., 3 * c:]), w["out"])
            s, y = Join.apply(o, w["post"], w["scale"], s, w["after"])
        return y

    # ---- serving -------------------------------------------------------
    @torch.no_grad()
    def freeze(self):
        """The products' weights in 4 bits, with a scale and a zero point for each group of columns."""
        self.q = []
        for w in self.blocks:
            packed = {}
            for k in ("inp", "out"):
                N, K = w[k].shape
                q, scale, zero = (like(w[k], N, (K + 1) // 2, dtype=U8), like(w[k], N, -(-K // self.group)),
                                  like(w[k], N, -(-K // self.group)))
                bd.quant_w4(w[k].detach(), q, scale, self.group, zero=zero)
                packed[k] = q, scale, zero
            self.q.append(packed)

    def product(self, k, j, y):
        q, scale, zero = self.q[k][j]
        if y.shape[0] > 64:  # a prompt: the values that the 4 bits stand for, once
            w = like(y, q.shape[0], y.shape[1])
            bd.dequant_w4(q, scale, w, self.group, zero=zero)
            return F.linear(y, w)
        out = like(y, y.shape[0], q.shape[0])
        bd.gemm_w4(y, q, scale, out, self.group, zero=zero)
        return out

    def run(self, s, recur):
        """The blocks on rows s [rows, dim]; recur(block, x, r, i) is the recurrence."""
        y, c = like(s, *s.shape), self.width
        bd.block_norm(s, self.first.detach(), y)
        for k, w in enumerate(self.blocks):
            w = {name: v.detach() for name, v in w.items()}
            p = self.product(k, "inp", y)
            h = recur(k, w, p[:, :c], p[:, c:2 * c], p[:, 2 * c:3 * c])
            g = like(h, *h.shape)
            bd.block_norm(h, w["norm"], g, z=p[:, 3 * c:])
            o, t, y = self.product(k, "out", g), like(s, *s.shape), like(s, *s.shape)
            bd.block_norm(o, w["post"], t, scale=w["scale"], residual=s, y=y, w_next=w["after"])
            s = t
        return y

    @torch.no_grad()
    def prompt(self, s, lengths=None):
        """s [B, T, dim]: the outputs and each block's states after the sequences."""
        B, T, _ = s.shape
        states = [torch.empty(B, self.width, device="cuda") for _ in self.blocks]

        def recur(k, w, x, r, i):
            y = like(x, B, T, self.width)
            ws = workspace(bd.gated_workspace_bytes(x.dtype, B, T, self.width, with_adjoint=False))
            bd.gated_scan(*(v.as_strided((B, T, self.width), (T * v.stride(0), v.stride(0), 1), v.storage_offset())
                            for v in (x, r, i)), w["decay"], y, ws, r_bias=w["r_bias"], i_bias=w["i_bias"],
                          h_last=states[k], lengths=lengths)
            return y.view(B * T, self.width)

        return self.run(s.reshape(B * T, -1), recur).view(B, T, -1), states

    @torch.no_grad()
    def token(self, s, states):
        """One token s [B, dim] of each sequence; the states move on in place."""
        def recur(k, w, x, r, i):
            y = like(x, x.shape[0], self.width)
            bd.gated_step(x, r, i, w["decay"], states[k], y, r_bias=w["r_bias"], i_bias=w["i_bias"])
            return y

        return self.run(s, recur)


def train(model, steps=8, B=2, T=96, lr=2e-3, seed=1):
    """The losses of a few steps towards a delayed copy of the input."""
    g = torch.Generator().manual_seed(seed)
    s = torch.randn(B, T, model.dim, generator=g).to(model.first.dtype).cuda()
    target = torch.roll(s, 2, 1)
    optimizer = torch.optim.Adam(model.parameters(), lr=lr)
    losses = []
    for _ in range(steps):
        loss = (model.forward(s).float() - target.float()).square().mean()
        optimizer.zero_grad()
        loss.backward()
        optimizer.step()
        with torch.no_grad():
            for w in model.blocks:
                w["decay"].clamp_(min=1e-4)  # below 0 the recurrence is not defined
        losses.append(float(loss.detach()))
    return losses


def serve(model, B=3, T=70, tokens=9, seed=2):
    """The last outputs from a prompt and single tokens, and from the whole sequence at once."""
    g = torch.Generator().manual_seed(seed)
    s = torch.randn(B, T + tokens, model.dim, generator=g).to(model.first.dtype).cuda()
    model.freeze()
    _, states = model.prompt(s[:, :T].contiguous())
    got = torch.stack([model.token(s[:, T + i].contiguous(), states) for i in range(tokens)], 1)
    return got, model.prompt(s)[0][:, T:]


if __name__ == "__main__":
    model = Model()
    print("training loss:", " ".join("%.4f" % v for v in train(model)))
    got, whole = serve(model)
    print("single tokens against the whole sequence: largest difference %.4f of %.2f"
          % (float((got.float() - whole.float()).abs().max()), float(whole.float().abs().max())))
