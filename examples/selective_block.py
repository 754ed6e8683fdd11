"""A language model block on a selective state space, trained and served.

    s = s + out(scan(conv(in(norm(s)))))

Training runs in bf16 with the library's kernels under torch's autograd: the
residual RMS norm, the short causal convolution and the selective scan, each
with its gradient.  Serving keeps the weights of both large products in 8 bits:
a prompt fills the convolution's and the scan's states, and then each token
takes one step on them.

    python examples/selective_block.py
"""
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from nonlinear_rnn_evaluation_newton_amd import binding as bd  # noqa: E402

BF, F32, I8 = torch.bfloat16, torch.float32, torch.int8


def like(t, *shape, dtype=None):
    return torch.empty(*shape, dtype=dtype or t.dtype, device=t.device)


def workspace(n):
    return torch.empty(n, dtype=torch.uint8, device="cuda")


class Norm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w):
        rows, n = x.numel() // x.shape[-1], x.shape[-1]
        y = torch.empty_like(x)
        bd.rmsnorm(x.view(rows, n), w, y.view(rows, n))
        ctx.save_for_backward(x, w)
        return y

    @staticmethod
    def backward(ctx, dy):
        x, w = ctx.saved_tensors
        rows, n = x.numel() // x.shape[-1], x.shape[-1]
        dx, dw = torch.empty_like(x), like(w, n, dtype=F32)
        bd.rmsnorm_adjoint(x.view(rows, n), w, dy.contiguous().view(rows, n), dx.view(rows, n), dw,
                           workspace(bd.rmsnorm_workspace_bytes(x.dtype, rows, n)))
        return dx, dw.to(w.dtype)


class Conv(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, bias):
        y = like(x, *x.shape)
        bd.conv(x, w, bias, y)
        ctx.save_for_backward(x, w, bias)
        return y

    @staticmethod
    def backward(ctx, dy):
        x, w, bias = ctx.saved_tensors
        dx, dw, db = like(x, *x.shape), like(w, *w.shape, dtype=F32), like(bias, *bias.shape, dtype=F32)
        bd.conv_adjoint(x, w, bias, dy.contiguous(), dx, dw, db,
                        workspace(bd.conv_workspace_bytes(x.dtype, *x.shape, w.shape[1])))
        return dx, dw.to(w.dtype), db.to(bias.dtype)


class Scan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, u, dt, A, Bm, Cm, D, z, dt_bias):
        B, T, ch = u.shape
        y = like(u, B, T, ch)
        states = like(A, *bd.ssm_states_shape(B, T, ch, A.shape[1]))
        ws = workspace(bd.ssm_workspace_bytes(u.dtype, B, T, ch, A.shape[1]))
        bd.ssm_scan(u, dt, A, Bm, Cm, y, ws, D=D, z=z, dt_bias=dt_bias, states=states)
        ctx.save_for_backward(u, dt, A, Bm, Cm, D, z, dt_bias, states)
        return y

    @staticmethod
    def backward(ctx, dy):
        u, dt, A, Bm, Cm, D, z, dt_bias, states = ctx.saved_tensors
        new = lambda t: like(t, *t.shape)  # noqa: E731
        g = dict(du=new(u), ddt=new(dt), dA=new(A), dB=new(Bm), dC=new(Cm), dD=new(D), dz=new(z), ddt_bias=new(dt_bias))
        ws = workspace(bd.ssm_workspace_bytes(u.dtype, *u.shape, A.shape[1]))
        bd.ssm_scan_adjoint(u, dt, A, Bm, Cm, states, dy.contiguous(), ws, D=D, z=z, dt_bias=dt_bias, **g)
        return tuple(g[k] for k in ("du", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias"))


class Block:
    def __init__(self, dim=256, states=16, taps=4, rank=16, seed=0):
        g = torch.Generator().manual_seed(seed)
        ch = 2 * dim
        self.dim, self.ch, self.states, self.taps, self.rank = dim, ch, states, taps, rank

        def normal(*shape, std=1.0, dtype=F32):
            return (torch.randn(*shape, generator=g) * std).to(dtype).cuda().requires_grad_()

        self.w = dict(
            norm=torch.ones(dim, dtype=BF, device="cuda", requires_grad=True),
            inp=normal(2 * ch, dim, std=dim ** -0.5, dtype=BF), out=normal(dim, ch, std=ch ** -0.5, dtype=BF),
            conv=normal(ch, taps, std=0.5, dtype=BF), conv_bias=normal(ch, std=0.1, dtype=BF),
            mix=normal(rank + 2 * states, ch, std=ch ** -0.5, dtype=BF), dt=normal(ch, rank, std=rank ** -0.5, dtype=BF),
            dt_bias=(torch.rand(ch, generator=g) * 3 - 5).cuda().requires_grad_(),
            A=-torch.arange(1, states + 1, dtype=F32).repeat(ch, 1).cuda(), D=normal(ch))
        self.w["A"].requires_grad_()

    def mixing(self, x):
        """Step size, B and C of the scan from the convolution's output."""
        m = F.linear(x, self.w["mix"])
        r, n = self.rank, self.states
        return F.linear(m[..., :r], self.w["dt"]), m[..., r:r + n], m[..., r + n:]

    def train_forward(self, s):
        w = self.w
        p = F.linear(Norm.apply(s, w["norm"]), w["inp"])
        x = Conv.apply(p[..., :self.ch], w["conv"], w["conv_bias"])
        dt, Bm, Cm = self.mixing(x)
        y = Scan.apply(x, dt, w["A"], Bm, Cm, w["D"], p[..., self.ch:], w["dt_bias"])
        return s + F.linear(y, w["out"])

    # ---- serving -------------------------------------------------------
    @torch.no_grad()
    def freeze(self):
        """The two large products' weights in 8 bits, a scale for each output channel."""
        self.q = {}
        for k in ("inp", "out"):
            w = self.w[k].detach()
            q, scale = like(w, *w.shape, dtype=I8), like(w, w.shape[0], dtype=F32)
            bd.quant_rows(w, q, scale)
            self.q[k] = q, scale

    def product(self, k, q, scale):
        w, ws = self.q[k]
        M, N = q.shape[0], w.shape[0]
        out = torch.empty(M, N, dtype=BF, device="cuda")
        bd.gemm_i8(q, scale, w, ws, out, workspace(bd.gemm_i8_workspace_bytes(M, N, q.shape[1])))
        return out

    def enter(self, s):
        q, scale = like(s, *s.shape, dtype=I8), like(s, s.shape[0], dtype=F32)
        bd.rmsnorm(s, self.w["norm"].detach(), q=q, scale=scale)
        return self.product("inp", q, scale)

    def leave(self, s, y):
        q, scale = like(y, *y.shape, dtype=I8), like(y, y.shape[0], dtype=F32)
        bd.quant_rows(y, q, scale)
        return s + self.product("out", q, scale)

    @torch.no_grad()
    def prompt(self, s, lengths=None):
        """s [B, T, dim]: the block's output and the states after each sequence."""
        w, (B, T, _) = {k: v.detach() for k, v in self.w.items()}, s.shape
        p = self.enter(s.reshape(B * T, -1)).view(B, T, -1)
        x, y = like(p, B, T, self.ch), like(p, B, T, self.ch)
        taps = torch.zeros(B, self.taps - 1, self.ch, dtype=BF, device="cuda")
        h = like(p, B, self.ch, self.states, dtype=F32)
        bd.conv(p[..., :self.ch], w["conv"], w["conv_bias"], x, state_out=taps, lengths=lengths)
        dt, Bm, Cm = self.mixing(x)
        ws = workspace(bd.ssm_workspace_bytes(BF, B, T, self.ch, self.states, with_adjoint=False))
        bd.ssm_scan(x, dt, w["A"], Bm, Cm, y, ws, D=w["D"], z=p[..., self.ch:], dt_bias=w["dt_bias"], h_last=h,
                    lengths=lengths)
        return self.leave(s.reshape(B * T, -1), y.view(B * T, -1)).view(B, T, -1), (taps, h)

    @torch.no_grad()
    def token(self, s, state):
        """One token s [B, dim] of each sequence; the states move on in place."""
        w, (taps, h) = {k: v.detach() for k, v in self.w.items()}, state
        p = self.enter(s)
        x, y = like(p, s.shape[0], self.ch), like(p, s.shape[0], self.ch)
        bd.conv_step(p[:, :self.ch], w["conv"], w["conv_bias"], taps, x)
        dt, Bm, Cm = self.mixing(x)
        bd.ssm_step(x, dt, w["A"], Bm, Cm, h, y, D=w["D"], z=p[:, self.ch:], dt_bias=w["dt_bias"])
        return self.leave(s, y)


def train(block, steps=12, B=2, T=64, lr=3e-3, seed=1):
    """The losses of a few steps towards a delayed copy of the input."""
    g = torch.Generator().manual_seed(seed)
    s = torch.randn(B, T, block.dim, generator=g).to(BF).cuda()
    target = torch.roll(s, 2, 1)
    optimizer = torch.optim.Adam(block.w.values(), lr=lr)
    losses = []
    for _ in range(steps):
        loss = (block.train_forward(s).float() - target.float()).square().mean()
        optimizer.zero_grad()
        loss.backward()
        optimizer.step()
        losses.append(float(loss.detach()))
    return losses


def serve(block, B=3, T=40, tokens=9, seed=2):
    """The last outputs from a prompt and single tokens, and from the whole sequence at once."""
    g = torch.Generator().manual_seed(seed)
    s = torch.randn(B, T + tokens, block.dim, generator=g).to(BF).cuda()
    block.freeze()
    _, state = block.prompt(s[:, :T].contiguous())
    got = torch.stack([block.token(s[:, T + i].contiguous(), state) for i in range(tokens)], 1)
    return got, block.prompt(s)[0][:, T:]


if __name__ == "__main__":
    block = Block()
    losses = train(block)
    print("training loss:", " ".join("%.4f" % v for v in losses))
    got, whole = serve(block)
    print("single tokens against the whole sequence: largest difference %.4f of %.2f"
          % (float((got - whole).abs().max()), float(whole.abs().max())))
