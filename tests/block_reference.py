"""Plain 64-bit forms of the selective block's operators, one step after
another, on the CPU: what the GPU tests compare with.  Gradients are written
out from the formulas; test_block_reference.py holds them to differences."""
import torch

F64 = torch.float64


def silu(x):
    return x * torch.sigmoid(x)


def dsilu(x):
    p = torch.sigmoid(x)
    return p + x * p * (1 - p)


def softplus(v):
    return torch.logaddexp(v, torch.zeros_like(v))


def conv(x, w, bias=None, state=None, lengths=None, act=True):
    """y and the state after the last step; x [B, T, D], w [D, W], state [B, W-1, D]."""
    B, T, D = x.shape
    W = w.shape[1]
    y = torch.zeros(B, T, D, dtype=F64)
    out = torch.zeros(B, W - 1, D, dtype=F64)
    for b in range(B):
        n = T if lengths is None else min(max(int(lengths[b]), 0), T)
        past = torch.zeros(W - 1, D, dtype=F64) if state is None else state[b].double()
        full = torch.cat([past, x[b, :n].double()])
        for t in range(n):
            a = (full[t:t + W] * w.double().t()).sum(0)
            a = a if bias is None else a + bias.double()
            y[b, t] = silu(a) if act else a
        out[b] = full[n:n + W - 1]
    return y, out


def conv_grads(x, w, dy, bias=None, state=None, dstate_out=None, lengths=None, act=True):
    B, T, D = x.shape
    W = w.shape[1]
    dx, ds = torch.zeros(B, T, D, dtype=F64), torch.zeros(B, W - 1, D, dtype=F64)
    dw, db = torch.zeros(D, W, dtype=F64), torch.zeros(D, dtype=F64)
    for b in range(B):
        n = T if lengths is None else min(max(int(lengths[b]), 0), T)
        past = torch.zeros(W - 1, D, dtype=F64) if state is None else state[b].double()
        full = torch.cat([past, x[b, :n].double()])
        g = torch.zeros_like(full)
        for t in range(n):
            a = (full[t:t + W] * w.double().t()).sum(0)
            a = a if bias is None else a + bias.double()
            da = dy[b, t].double() * (dsilu(a) if act else 1.0)
            g[t:t + W] += da * w.double().t()
            dw += (da * full[t:t + W]).t()
            db += da
        if dstate_out is not None:
            g[n:n + W - 1] += dstate_out[b].double()
        ds[b], dx[b, :n] = g[:W - 1], g[W - 1:]
    return dict(dx=dx, dw=dw, dbias=db, dstate=ds)


def _wide(m, D, G):
    return m.double().reshape(-1, G, m.shape[-1] // G).repeat_interleave(D // G, 1)  # [B, D, N]


def scan(u, dt, A, Bm, Cm, D=None, z=None, dt_bias=None, h0=None, lengths=None, sp=True, keep=False):
    """y, the last state and, with keep, every state (h_{-1} first)."""
    B, T, ch = u.shape
    N = A.shape[1]
    G = Bm.shape[-1] // N
    h = torch.zeros(B, ch, N, dtype=F64) if h0 is None else h0.double().clone()
    y = torch.zeros(B, T, ch, dtype=F64)
    hs = [h]
    n = torch.full((B,), T) if lengths is None else lengths.clamp(0, T)
    for t in range(T):
        v = dt[:, t].double() + (0 if dt_bias is None else dt_bias.double())
        delta = softplus(v) if sp else v
        x = delta * u[:, t].double()
        new = torch.exp(delta[..., None] * A.double()) * h + x[..., None] * _wide(Bm[:, t], ch, G)
        on = (t < n)[:, None]
        h = torch.where(on[..., None], new, h)
        o = (h * _wide(Cm[:, t], ch, G)).sum(-1) + (0 if D is None else D.double() * u[:, t].double())
        if z is not None:
            o = o * silu(z[:, t].double())
        y[:, t] = torch.where(on, o, torch.zeros_like(o))
        if keep:
            hs.append(h)
    return (y, h, hs) if keep else (y, h)


def scan_grads(u, dt, A, Bm, Cm, dy, D=None, z=None, dt_bias=None, h0=None, lengths=None, dh_last=None, sp=True):
    B, T, ch = u.shape
    N = A.shape[1]
    G = Bm.shape[-1] // N
    y, _, hs = scan(u, dt, A, Bm, Cm, D, None, dt_bias, h0, lengths, sp, keep=True)
    n = torch.full((B,), T) if lengths is None else lengths.clamp(0, T)
    g = torch.zeros(B, ch, N, dtype=F64) if dh_last is None else dh_last.double().clone()
    o = {k: torch.zeros(B, T, ch, dtype=F64) for k in ("du", "ddt", "dz")}
    o["dB"], o["dC"] = torch.zeros(Bm.shape, dtype=F64), torch.zeros(Cm.shape, dtype=F64)
    o["dA"], o["dD"] = torch.zeros(ch, N, dtype=F64), torch.zeros(ch, dtype=F64)
    zero = torch.zeros((), dtype=F64)
    for t in reversed(range(T)):
        on = (t < n)[:, None]
        uu = torch.where(on, u[:, t].double(), zero)
        v = torch.where(on, dt[:, t].double(), zero) + (0 if dt_bias is None else dt_bias.double())
        delta = softplus(v) if sp else v
        gy = torch.where(on, dy[:, t].double(), zero)
        e = gy
        if z is not None:
            zz = torch.where(on, z[:, t].double(), zero)
            e = gy * silu(zz)
            o["dz"][:, t] = gy * y[:, t] * dsilu(zz)
        Bt, Ct = (torch.where(on[..., None], _wide(m[:, t], ch, G), zero) for m in (Bm, Cm))
        a = torch.exp(delta[..., None] * A.double())
        at = g + Ct * e[..., None]
        gb = (at * Bt).sum(-1)
        q = at * a * hs[t]
        dd = uu * gb + (q * A.double()).sum(-1)
        dd = dd * torch.sigmoid(v) if sp else dd
        o["ddt"][:, t] = torch.where(on, dd, zero)
        o["du"][:, t] = torch.where(on, delta * gb + (0 if D is None else D.double() * e), zero)
        o["dA"] += torch.where(on[..., None], q * delta[..., None], zero).sum(0)
        o["dD"] += (e * uu).sum(0)
        xb = torch.where(on[..., None], (delta * uu)[..., None] * at, zero)
        xc = torch.where(on[..., None], e[..., None] * hs[t + 1], zero)
        o["dB"][:, t] = xb.reshape(B, G, ch // G, N).sum(2).reshape(B, G * N)
        o["dC"][:, t] = xc.reshape(B, G, ch // G, N).sum(2).reshape(B, G * N)
        g = torch.where(on[..., None], at * a, g)
    o["dbias"], o["dh0"] = o["ddt"].sum((0, 1)), g
    if z is None:
        del o["dz"]
    return o


def norm(s, w, eps):
    s = s.double()
    return s / torch.sqrt((s * s).mean(1, keepdim=True) + eps) * (1 if w is None else w.double())


def norm_grads(s, w, dy, eps, ds=None):
    s, g = s.double(), dy.double()
    rstd = 1 / torch.sqrt((s * s).mean(1, keepdim=True) + eps)
    t = g if w is None else g * w.double()
    dx = rstd * (t - s * rstd ** 2 * (t * s).mean(1, keepdim=True)) + (0 if ds is None else ds.double())
    return dx, (g * s * rstd).sum(0)


def quant(y):
    scale = y.double().abs().amax(1) / 127
    safe = torch.where(scale > 0, scale, torch.ones_like(scale))
    return torch.round(y.double() / safe[:, None]), scale
