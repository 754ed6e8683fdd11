"""Plain 64-bit forms of the gated block's operators, one step after another, on
the CPU: what the GPU tests compare with.  Gradients are written out from the
formulas; test_gated_reference.py holds them to differences."""
import torch

F64 = torch.float64


def _steps(lengths, B, T):
    return torch.full((B,), T) if lengths is None else lengths.clamp(0, T)


def _gates(r, i, decay, rb, ib):
    r = torch.sigmoid(r.double() + (0 if rb is None else rb.double()))
    i = torch.sigmoid(i.double() + (0 if ib is None else ib.double()))
    v = decay.double() * r
    return r, i, torch.exp(-v), torch.sqrt(-torch.expm1(-2 * v))


def gated(x, r, i, decay, r_bias=None, i_bias=None, h0=None, lengths=None, keep=False):
    """y, the last state and, with keep, every state (h_{-1} first)."""
    B, T, D = x.shape
    h = torch.zeros(B, D, dtype=F64) if h0 is None else h0.double().clone()
    y, hs, n = torch.zeros(B, T, D, dtype=F64), [h], _steps(lengths, B, T)
    for t in range(T):
        on = (t < n)[:, None]
        _, gi, a, m = _gates(r[:, t], i[:, t], decay, r_bias, i_bias)
        h = torch.where(on, a * h + m * gi * x[:, t].double(), h)
        y[:, t] = torch.where(on, h, torch.zeros_like(h))
        hs.append(h)
    return (y, h, hs) if keep else (y, h)


def gated_grads(x, r, i, decay, dy, r_bias=None, i_bias=None, h0=None, lengths=None, dh_last=None):
    B, T, D = x.shape
    _, _, hs = gated(x, r, i, decay, r_bias, i_bias, h0, lengths, keep=True)
    n = _steps(lengths, B, T)
    g = torch.zeros(B, D, dtype=F64) if dh_last is None else dh_last.double().clone()
    o = {k: torch.zeros(B, T, D, dtype=F64) for k in ("dx", "dr", "di")}
    o["ddecay"] = torch.zeros(D, dtype=F64)
    zero = torch.zeros((), dtype=F64)
    for t in reversed(range(T)):
        on = (t < n)[:, None]
        gr, gi, a, m = _gates(r[:, t], i[:, t], decay, r_bias, i_bias)
        xt = x[:, t].double()
        full = g + dy[:, t].double()
        inv = torch.where(m > 0, 1 / m, zero)
        dv = full * (a * a * inv * gi * xt - a * hs[t])  # through v = decay r
        o["dx"][:, t] = torch.where(on, full * m * gi, zero)
        o["di"][:, t] = torch.where(on, full * m * xt * gi * (1 - gi), zero)
        o["dr"][:, t] = torch.where(on, dv * decay.double() * gr * (1 - gr), zero)
        o["ddecay"] += torch.where(on, dv * gr, zero).sum(0)
        g = torch.where(on, full * a, g)
    o["dr_bias"], o["di_bias"], o["dh0"] = o["dr"].sum((0, 1)), o["di"].sum((0, 1)), g
    return o


def act(z, gate):
    """The gate's value and its derivative."""
    if z is None:
        return torch.ones((), dtype=F64), torch.zeros((), dtype=F64)
    z = z.double()
    p = torch.sigmoid(z)
    return (p, p * (1 - p)) if gate == "sigmoid" else (z * p, p + z * p * (1 - p))


def _or1(w):
    return torch.ones((), dtype=F64) if w is None else w.double()


def _rstd(x, eps):
    return 1 / torch.sqrt((x * x).mean(1, keepdim=True) + eps)


def block_norm(x, w=None, z=None, gate="silu", scale=None, residual=None, eps=1e-5):
    """t before it is rounded."""
    x = x.double()
    u = x * _rstd(x, eps) * _or1(w) * _or1(scale) * act(z, gate)[0]
    return u if residual is None else residual.double() + u


def norm_next(t, w_next=None, eps=1e-5):
    t = t.double()
    return t * _rstd(t, eps) * _or1(w_next)


def block_norm_grads(x, w=None, z=None, gate="silu", scale=None, w_next=None, t=None, dt=None, dy=None, eps=1e-5):
    x = x.double()
    gt, o = torch.zeros_like(x) if dt is None else dt.double(), {}
    if dy is not None:
        t, dy = t.double(), dy.double()
        rs, e = _rstd(t, eps), dy * _or1(w_next)
        gt = gt + rs * (e - t * rs ** 2 * (e * t).mean(1, keepdim=True))
        o["dw_next"] = (dy * t * rs).sum(0)
    rs, (av, ad) = _rstd(x, eps), act(z, gate)
    f = _or1(w) * _or1(scale)
    e = gt * f * av
    o.update(dres=gt, dx=rs * (e - x * rs ** 2 * (e * x).mean(1, keepdim=True)))
    if z is not None:
        o["dz"] = gt * f * x * rs * ad
    q = (gt * av * x * rs).sum(0)
    o.update(dw=q * _or1(scale), dscale=q * _or1(w))
    return o


def unpack(q, K):
    """The 4-bit numbers [N, K] of packed bytes."""
    return torch.stack([q & 15, q >> 4], -1).reshape(q.shape[0], -1)[:, :K]


def weights(q, scale, K, group, zero=None, to=F64):
    wide = lambda v: v.to(to).repeat_interleave(group, 1)[:, :K]  # noqa: E731
    return (unpack(q, K).to(to) - (8 if zero is None else wide(zero))) * wide(scale)


def quant(w, group, zero=False):
    """q [N, K], scale and zero in w's type: 32-bit arithmetic, as it is defined."""
    N, K = w.shape
    f = torch.nn.functional.pad(w.float(), (0, -K % group)).reshape(N, -1, group)
    if zero:
        lo, hi = f.amin(-1).clamp(max=0), f.amax(-1).clamp(min=0)
        scale = ((hi - lo) * torch.tensor(1 / 15, dtype=torch.float32)).to(w.dtype)
    else:
        scale = (f.abs().amax(-1) * torch.tensor(1 / 7, dtype=torch.float32)).to(w.dtype)
    s = torch.where(scale.float() > 0, scale.float(), torch.ones(()))
    z = torch.round(-lo / s).clamp(0, 15) if zero else torch.full_like(s, 8)
    q = (torch.round(f / s[..., None]) + z[..., None]).clamp(0, 15)
    return q.reshape(N, -1)[:, :K].to(torch.uint8), scale, z.to(w.dtype)
