"""Operators of a selective state space block: the cases they are measured on.

The block mixes a sequence with a short causal convolution and a linear
recurrence whose decay depends on the input; its projections run in 8-bit
integers when it serves, and a root-mean-square norm with the residual's
addition stands before each of them.  Four operators, each in the directions
in which a program calls it:

  conv     y_t = silu(b + sum_k w_k x_{t-W+1+k}) per channel; its gradient;
           single tokens on a pool of states
  scan     h_t = exp(delta_t A) h_{t-1} + delta_t u_t B_t,
           y_t = (C_t h_t + D u_t) silu(z_t), delta = softplus(dt + bias);
           its gradient; single tokens on a pool of states
  norm     s = x + r, y = s / sqrt(mean s^2 + eps) * w, in the storage type or
           in 8 bits with a scale for each row; its gradient
  product  C = (Aq Wq^T) sa sw + b on 8-bit integers, with rows quantised on
           the way or given

`run` computes them with elementary torch operations in 32 bits, or with the
package's calls where `own` is set.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one training step's convolution: the input is the first half of the projection that also holds the gate
        dict(name="conv train", op="conv", mode="train", dtype="bf16", B=8, T=4096, D=2048, W=4, ragged=False),
        # a decoding batch: one token for each of 48 sequences, states in a pool, some rows idle
        dict(name="conv step", op="conv", mode="step", dtype="bf16", B=48, T=1, D=2048, W=4, ragged=True),
        # a batch of long prompts
        dict(name="scan prompt", op="scan", mode="prompt", dtype="bf16", B=8, T=4096, D=2048, N=16, G=1, gate=True,
             ragged=False),
        # one very long sequence of few channels: only the time axis is wide
        dict(name="scan long", op="scan", mode="prompt", dtype="f32", B=1, T=32768, D=256, N=16, G=1, gate=False,
             ragged=False),
        # a training step: outputs and all gradients
        dict(name="scan train", op="scan", mode="train", dtype="bf16", B=4, T=2048, D=2048, N=16, G=1, gate=True,
             ragged=False),
        # a small model's training batch of sequences of unequal length, one of them empty, two groups of B and C
        dict(name="scan train ragged", op="scan", mode="train", dtype="f32", B=3, T=777, D=200, N=8, G=2, gate=True,
             ragged=True),
        # a decoding batch
        dict(name="scan step", op="scan", mode="step", dtype="bf16", B=64, T=1, D=2048, N=16, G=1, gate=True,
             ragged=True),
        # a prompt's norm before an 8-bit product
        dict(name="norm to 8 bits", op="norm", mode="serve", dtype="bf16", rows=8192, n=2048),
        # a training step's norm and its gradient
        dict(name="norm train", op="norm", mode="train", dtype="bf16", rows=16384, n=2048),
        # a decoding batch's projection
        dict(name="product decode", op="product", given=False, dtype="bf16", M=16, N=4096, K=2048),
        # the input projection of a batch of prompts
        dict(name="product prompt", op="product", given=False, dtype="bf16", M=16384, N=8192, K=2048),
        # sizes that end inside every tile, rows that are quantised already, 32-bit output
        dict(name="product odd", op="product", given=True, dtype="f32", M=301, N=1030, K=1000),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A number of channels: a power of two, an odd multiple of 16, or any odd number."""
    v = _log(rng, lo, hi)
    how = rng.randrange(3)
    if how == 0:
        return max(lo, min(hi, 1 << int(round(math.log2(v)))))
    if how == 1:
        return max(16, min(hi, 16 * (v // 16 | 1)))
    return min(hi - 1, v | 1)


def draw(rng):
    kind = rng.choice(["conv train", "conv step", "scan prompt", "scan prompt", "scan train", "scan train",
                       "scan step", "norm serve", "norm train", "product", "product"])
    op, _, mode = kind.partition(" ")
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "conv":
        D = _width(rng, 64, 4096)
        if mode == "step":
            return dict(op=op, mode=mode, dtype=dtype, B=_log(rng, 1, 256), T=1, D=D, W=rng.choice([2, 3, 4, 4]),
                        ragged=rng.random() < 0.5)
        B = _log(rng, 1, 16)
        T = _log(rng, 1, max(1, min(16384, (8 * 4096 * 2048 // (2 if dtype == "f32" else 1)) // (B * D))))
        return dict(op=op, mode=mode, dtype=dtype, B=B, T=T, D=D, W=rng.choice([2, 3, 4, 4]),
                    ragged=rng.random() < 0.4)
    if op == "scan":
        N = rng.choice([1, 5, 8, 16, 16, 16, 24, 32, 64])
        D = _width(rng, 64, 4096)
        G = rng.choice([1, 1, 2]) if D % 2 == 0 else 1
        if mode == "step":
            return dict(op=op, mode=mode, dtype=dtype, B=max(1, min(_log(rng, 1, 256), 64 * 2048 * 64 // (D * N))),
                        T=1, D=D, N=N, G=G, gate=rng.random() < 0.7, ragged=rng.random() < 0.5)
        most = (8 * 4096 if mode == "prompt" else 4 * 2048) * 2048 * 16
        B = _log(rng, 1, 8)
        T = _log(rng, 1, max(1, min(32768, most // (B * D * N))))
        return dict(op=op, mode=mode, dtype=dtype, B=B, T=T, D=D, N=N, G=G, gate=rng.random() < 0.7,
                    ragged=rng.random() < 0.4)
    if op == "norm":
        n = _width(rng, 64, 8192)
        return dict(op=op, mode=mode, dtype=dtype, rows=_log(rng, 1, 16384 * 2048 // (n * (2 if dtype == "f32" else 1))),
                    n=n)
    N, K = _width(rng, 64, 8192), _width(rng, 64, 8192)
    most = 16384 * 8192 * 2048 // (N * K)
    return dict(op=op, given=rng.random() < 0.5, dtype=dtype, M=_log(rng, 1, max(1, min(16384, most))), N=N, K=K)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _lengths(case, g):
    """Lengths of a ragged batch, from none to all of T; the last sequence is empty where there are several."""
    B, T = case["B"], case["T"]
    n = (torch.rand(B, generator=g, device=DEV) * (T + 1)).to(torch.int32).clamp_(max=T)
    n[0] = T
    if B > 1:
        n[-1] = 0
    return n


def _slots(case, g):
    """Rows of the state pool for a decoding batch; -1 marks an idle row."""
    B = case["B"]
    s = torch.randperm(B + 3, generator=g, device=DEV)[:B].to(torch.int32)
    if B > 4:
        s[B // 2] = -1
    return s


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]
    f32 = dict(dtype=torch.float32, device=DEV)

    def normal(*shape, std=1.0, to=dt):
        return (torch.randn(*shape, generator=g, **f32) * std).to(to)

    def uniform(*shape, lo=0.0, hi=1.0):
        return torch.rand(*shape, generator=g, **f32) * (hi - lo) + lo

    s = dict(case=case)
    if case["op"] == "conv":
        B, T, D, W = case["B"], case["T"], case["D"], case["W"]
        s["x"] = normal(B, T, 2 * D)[..., :D]  # the other half is the gate
        s["w"] = uniform(D, W, lo=-W ** -0.5, hi=W ** -0.5).to(dt)
        s["bias"] = uniform(D, lo=-W ** -0.5, hi=W ** -0.5).to(dt)
        if case["mode"] == "step":
            s["state"] = normal(B + 3, W - 1, D)
            s["slots"] = _slots(case, g) if case["ragged"] else None
        else:
            s["dy"] = normal(B, T, D)
            s["lengths"] = _lengths(case, g) if case["ragged"] else None
    elif case["op"] == "scan":
        B, T, D, N, G = case["B"], case["T"], case["D"], case["N"], case["G"]
        rank = max(1, D // 32)  # width of the low-rank step size in the projection that also holds B and C
        s["u"] = torch.nn.functional.silu(torch.randn(B, T, D, generator=g, **f32)).to(dt)
        s["dt"] = normal(B, T, D, std=0.5)
        # step sizes from 0.001 to 0.1 at dt = 0, spread over their logarithm
        step = torch.exp(uniform(D, lo=math.log(1e-3), hi=math.log(1e-1)))
        s["dt_bias"] = step + torch.log(-torch.expm1(-step))
        s["A"] = -torch.arange(1, N + 1, **f32) * torch.exp(0.1 * torch.randn(D, N, generator=g, **f32))
        proj = normal(B, T, rank + 2 * G * N)
        s["Bm"], s["Cm"] = proj[..., rank:rank + G * N], proj[..., rank + G * N:]
        s["D"] = 1.0 + 0.1 * torch.randn(D, generator=g, **f32)
        s["z"] = normal(B, T, 2 * D)[..., D:] if case["gate"] else None
        if case["mode"] == "step":
            s["state"] = torch.randn(B + 3, D, N, generator=g, **f32)
            s["slots"] = _slots(case, g) if case["ragged"] else None
        else:
            s["lengths"] = _lengths(case, g) if case["ragged"] else None
            if case["mode"] == "train":
                s["dy"] = normal(B, T, D)
            else:
                s["h0"] = torch.randn(B, D, N, generator=g, **f32) * 0.1  # what an earlier piece of the prompt left
    elif case["op"] == "norm":
        rows, n = case["rows"], case["n"]
        outlier = torch.exp(0.5 * torch.randn(n, generator=g, **f32))  # a stream's channels differ in size
        s["x"] = normal(rows, n)
        s["r"] = (torch.randn(rows, n, generator=g, **f32) * outlier).to(dt)
        s["w"] = normal(n, std=0.1) + 1
        if case["mode"] == "train":
            s["dy"], s["ds"] = normal(rows, n), normal(rows, n)
    else:
        M, N, K = case["M"], case["N"], case["K"]
        s["wq"] = torch.randint(-127, 128, (N, K), generator=g, device=DEV, dtype=torch.int8)
        s["ws"] = uniform(N, lo=0.5, hi=1.5) / (127 * K ** 0.5)
        s["bias"] = normal(N, std=0.1)
        if case["given"]:
            s["xq"] = torch.randint(-127, 128, (M, K), generator=g, device=DEV, dtype=torch.int8)
            s["xs"] = uniform(M, lo=0.01, hi=0.03)
        else:
            s["x"] = normal(M, K)
    if case.get("mode") == "step":  # one token: [B, channels]
        for k in ("x", "u", "dt", "Bm", "Cm", "z"):
            if s.get(k) is not None:
                s[k] = s[k][:, 0]
    if own:
        s["plan"] = _plan(s)
    return s


# ---------------------------------------------------------------------------
# the plain forms: elementary operations in 32 bits, one rounding at the end
# ---------------------------------------------------------------------------
def _silu(x):
    return x * torch.sigmoid(x)


def _dsilu(x):
    p = torch.sigmoid(x)
    return p * (1 + x * (1 - p))


def _keep(lengths, T, shape):
    """True at the steps that a sequence has, as a [B, T, 1, ...] mask."""
    m = torch.arange(T, device=DEV)[None] < lengths[:, None]
    return m.reshape(m.shape + (1,) * (len(shape) - 2))


def _masked(x, lengths):
    return x if lengths is None else torch.where(_keep(lengths, x.shape[1], x.shape), x, torch.zeros_like(x))


def _conv_train(s):
    x, w, bias, dy, lengths = s["x"].float(), s["w"].float(), s["bias"].float(), s["dy"].float(), s["lengths"]
    T, W = x.shape[1], w.shape[1]
    x, dy = _masked(x, lengths), _masked(dy, lengths)
    taps = torch.nn.functional.pad(x, (0, 0, W - 1, 0)).unfold(1, W, 1)  # [B, T, D, W]
    a = (taps * w).sum(-1) + bias
    y = _masked(_silu(a), lengths)
    da = dy * _dsilu(a)
    back = torch.nn.functional.pad(da, (0, 0, 0, W - 1)).unfold(1, W, 1)  # da_t .. da_{t+W-1}
    dx = _masked((back * w.flip(1)).sum(-1), lengths)
    dt = s["x"].dtype
    return dict(y=y.to(dt), dx=dx.to(dt), dw=(da[..., None] * taps).sum((0, 1)), dbias=da.sum((0, 1)))


def _conv_step(s):
    x, w, bias, state, slots = s["x"], s["w"].float(), s["bias"].float(), s["state"], s["slots"]
    B = x.shape[0]
    at = torch.arange(B, device=DEV) if slots is None else slots.long()
    live = at >= 0
    row = at.clamp(min=0)
    taps = torch.cat([state[row], x[:, None]], 1)  # [B, W, D]
    y = _silu((taps.float() * w.t()).sum(1) + bias)
    y = torch.where(live[:, None], y, torch.zeros_like(y)).to(x.dtype)
    spare = torch.cat([state, torch.empty_like(state[:1])])  # idle rows are written to a row that is dropped
    spare[torch.where(live, at, torch.full_like(at, state.shape[0]))] = taps[:, 1:]
    state.copy_(spare[:-1])
    return dict(y=y, state=state)


def _recurrence(a, b):
    """h_t = a_t h_{t-1} + b_t along axis 1, by doubling: after the pass at distance s every entry holds s steps more."""
    s = 1
    while s < a.shape[1]:
        b = torch.cat([b[:, :s], b[:, s:] + a[:, s:] * b[:, :-s]], 1)
        a = torch.cat([a[:, :s], a[:, s:] * a[:, :-s]], 1)
        s *= 2
    return b


def _per_channel(x, D, N, G):
    """B or C [B, T, G N] for each channel: [B, T, D, N]."""
    return x.float().reshape(x.shape[0], x.shape[1], G, 1, N).expand(-1, -1, G, D // G, N).reshape(
        x.shape[0], x.shape[1], D, N)


def _delta(s):
    v = s["dt"].float() + s["dt_bias"]
    return v, torch.clamp(v, min=0) + torch.log1p(torch.exp(-torch.abs(v)))


def _scan_states(s, h0):
    c, lengths = s["case"], s.get("lengths")
    D, N, G = c["D"], c["N"], c["G"]
    v, delta = _delta(s)
    delta = _masked(delta, lengths)
    u, Bm, Cm = _masked(s["u"].float(), lengths), _masked(s["Bm"].float(), lengths), _masked(s["Cm"].float(), lengths)
    a = torch.exp(delta[..., None] * s["A"])
    b = (delta * u)[..., None] * _per_channel(Bm, D, N, G)
    if h0 is not None:
        b[:, 0] += a[:, 0] * h0
    return v, delta, u, Bm, Cm, a, _recurrence(a, b)


def _scan_prompt(s):
    c, lengths = s["case"], s["lengths"]
    _, _, u, _, Cm, _, h = _scan_states(s, s["h0"])
    y = (h * _per_channel(Cm, c["D"], c["N"], c["G"])).sum(-1) + s["D"] * u
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    return dict(y=_masked(y, lengths).to(s["u"].dtype), h=h[:, -1].contiguous())


def _scan_train(s):
    c, lengths = s["case"], s["lengths"]
    B, T, D, N, G = c["B"], c["T"], c["D"], c["N"], c["G"]
    v, delta, u, Bm, Cm, a, h = _scan_states(s, None)
    Bc, Cc = _per_channel(Bm, D, N, G), _per_channel(Cm, D, N, G)
    dy = _masked(s["dy"].float(), lengths)
    y0 = (h * Cc).sum(-1) + s["D"] * u
    y, e, dz = y0, dy, None
    if s["z"] is not None:
        z = _masked(s["z"].float(), lengths)
        y, e, dz = y0 * _silu(z), dy * _silu(z), dy * y0 * _dsilu(z)
    # the adjoint state, backwards in time: g_t = C_t e_t + a_{t+1} g_{t+1}
    later = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1)
    g = _recurrence(later.flip(1), (Cc * e[..., None]).flip(1)).flip(1)
    before = torch.cat([torch.zeros_like(h[:, :1]), h[:, :-1]], 1)
    through = g * a * before
    gb = (g * Bc).sum(-1)
    ddelta = u * gb + (through * s["A"]).sum(-1)
    ddt = _masked(ddelta * torch.sigmoid(v), lengths)
    split = (B, T, G, D // G, N)
    dt = s["u"].dtype
    out = dict(y=_masked(y, lengths).to(dt), du=(delta * gb + s["D"] * e).to(dt), ddt=ddt.to(dt),
               dB=((delta * u)[..., None] * g).reshape(split).sum(3).reshape(B, T, G * N).to(dt),
               dC=(e[..., None] * h).reshape(split).sum(3).reshape(B, T, G * N).to(dt),
               dA=(delta[..., None] * through).sum((0, 1)), dD=(e * u).sum((0, 1)), dbias=ddt.sum((0, 1)))
    if dz is not None:
        out["dz"] = dz.to(dt)
    return out


def _scan_step(s):
    c, state, slots = s["case"], s["state"], s["slots"]
    D, N, G = c["D"], c["N"], c["G"]
    at = torch.arange(c["B"], device=DEV) if slots is None else slots.long()
    live = at >= 0
    _, delta = _delta(s)
    u = s["u"].float()
    Bc, Cc = _per_channel(s["Bm"][:, None], D, N, G)[:, 0], _per_channel(s["Cm"][:, None], D, N, G)[:, 0]
    h = torch.exp(delta[..., None] * s["A"]) * state[at.clamp(min=0)] + (delta * u)[..., None] * Bc
    y = (h * Cc).sum(-1) + s["D"] * u
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    y = torch.where(live[:, None], y, torch.zeros_like(y))
    spare = torch.cat([state, torch.empty_like(state[:1])])  # idle rows are written to a row that is dropped
    spare[torch.where(live, at, torch.full_like(at, state.shape[0]))] = h
    state.copy_(spare[:-1])
    return dict(y=y.to(s["u"].dtype), state=state)


def _quantise(y):
    scale = y.abs().amax(-1, keepdim=True) * (1 / 127)
    return torch.round(y / torch.where(scale > 0, scale, torch.ones_like(scale))), scale


def _norm(s):
    dt, n = s["x"].dtype, s["x"].shape[1]
    total = (s["x"].float() + s["r"].float()).to(dt)  # the stream as it is stored is what the norm sees
    t, w = total.float(), s["w"].float()
    rstd = torch.rsqrt((t * t).mean(-1, keepdim=True) + EPS)
    if s["case"]["mode"] == "serve":
        q, scale = _quantise(t * rstd * w)
        return dict(sum=total, y=(q * scale).to(torch.bfloat16), scale=scale[:, 0])
    xhat, dy = t * rstd, s["dy"].float()
    dxhat = dy * w
    dx = rstd * (dxhat - xhat * (dxhat * xhat).sum(-1, keepdim=True) / n) + s["ds"].float()
    return dict(sum=total, y=(xhat * w).to(dt), dx=dx.to(dt), dw=(dy * xhat).sum(0))


def _product(s):
    q, scale = (s["xq"].float(), s["xs"][:, None]) if s["case"]["given"] else _quantise(s["x"].float())
    return (q @ s["wq"].float().t() * scale * s["ws"] + s["bias"].float()).to(DTYPES[s["case"]["dtype"]])


# ---------------------------------------------------------------------------
# the package's operators
# ---------------------------------------------------------------------------
def _plan(s):
    """Outputs and workspaces that a program allocates once."""
    from nonlinear_rnn_evaluation_newton_amd import binding as bd
    c = s["case"]
    dt = DTYPES[c["dtype"]]

    def new(*shape, dtype=dt):
        return torch.empty(*shape, dtype=dtype, device=DEV)

    def work(nbytes):
        return torch.empty(nbytes, dtype=torch.uint8, device=DEV)

    if c["op"] == "conv":
        B, T, D, W = c["B"], c["T"], c["D"], c["W"]
        if c["mode"] == "step":
            return dict(y=new(B, D))
        p = dict(y=new(B, T, D))
        if c["mode"] == "train":
            p.update(dx=new(B, T, D), dw=new(D, W, dtype=torch.float32), dbias=new(D, dtype=torch.float32),
                     ws=work(bd.conv_workspace_bytes(dt, B, T, D, W)))
        return p
    if c["op"] == "scan":
        B, T, D, N, G = c["B"], c["T"], c["D"], c["N"], c["G"]
        if c["mode"] == "step":
            return dict(y=new(B, D))
        p = dict(y=new(B, T, D))
        train = c["mode"] == "train"
        p["ws"] = work(bd.ssm_workspace_bytes(dt, B, T, D, N, G, with_adjoint=train))
        if train:
            p.update(states=new(*bd.ssm_states_shape(B, T, D, N), dtype=torch.float32), du=new(B, T, D),
                     ddt=new(B, T, D), dB=new(B, T, G * N), dC=new(B, T, G * N),
                     dA=new(D, N, dtype=torch.float32), dD=new(D, dtype=torch.float32),
                     dbias=new(D, dtype=torch.float32), dz=new(B, T, D) if c["gate"] else None)
        else:
            p["h"] = new(B, D, N, dtype=torch.float32)
        return p
    if c["op"] == "norm":
        rows, n = c["rows"], c["n"]
        p = dict(sum=new(rows, n))
        if c["mode"] == "serve":
            p.update(q=new(rows, n, dtype=torch.int8), scale=new(rows, dtype=torch.float32),
                     y=new(rows, n, dtype=torch.bfloat16))
        else:
            p.update(y=new(rows, n), dx=new(rows, n), dw=new(n, dtype=torch.float32),
                     ws=work(bd.rmsnorm_workspace_bytes(dt, rows, n)))
        return p
    M, N, K = c["M"], c["N"], c["K"]
    p = dict(out=new(M, N), ws=work(bd.gemm_i8_workspace_bytes(M, N, K)))
    if not c["given"]:
        p.update(q=new(M, K, dtype=torch.int8), scale=new(M, dtype=torch.float32))
    return p


def _run_own(s):
    from nonlinear_rnn_evaluation_newton_amd import binding as bd
    c, p = s["case"], s["plan"]
    if c["op"] == "conv":
        if c["mode"] == "step":
            bd.conv_step(s["x"], s["w"], s["bias"], s["state"], p["y"], slots=s["slots"])
            return dict(y=p["y"], state=s["state"])
        bd.conv(s["x"], s["w"], s["bias"], p["y"], lengths=s["lengths"])
        bd.conv_adjoint(s["x"], s["w"], s["bias"], s["dy"], p["dx"], p["dw"], p["dbias"], p["ws"],
                        lengths=s["lengths"])
        return dict(y=p["y"], dx=p["dx"], dw=p["dw"], dbias=p["dbias"])
    if c["op"] == "scan":
        if c["mode"] == "step":
            bd.ssm_step(s["u"], s["dt"], s["A"], s["Bm"], s["Cm"], s["state"], p["y"], D=s["D"], z=s["z"],
                        dt_bias=s["dt_bias"], slots=s["slots"])
            return dict(y=p["y"], state=s["state"])
        if c["mode"] == "prompt":
            bd.ssm_scan(s["u"], s["dt"], s["A"], s["Bm"], s["Cm"], p["y"], p["ws"], D=s["D"], z=s["z"],
                        dt_bias=s["dt_bias"], h0=s["h0"], h_last=p["h"], lengths=s["lengths"])
            return dict(y=p["y"], h=p["h"])
        bd.ssm_scan(s["u"], s["dt"], s["A"], s["Bm"], s["Cm"], p["y"], p["ws"], D=s["D"], z=s["z"],
                    dt_bias=s["dt_bias"], states=p["states"], lengths=s["lengths"])
        bd.ssm_scan_adjoint(s["u"], s["dt"], s["A"], s["Bm"], s["Cm"], p["states"], s["dy"], p["ws"], D=s["D"],
                            z=s["z"], dt_bias=s["dt_bias"], lengths=s["lengths"], du=p["du"], ddt=p["ddt"],
                            dB=p["dB"], dC=p["dC"], dz=p["dz"], dA=p["dA"], dD=p["dD"], ddt_bias=p["dbias"])
        out = dict(y=p["y"], du=p["du"], ddt=p["ddt"], dB=p["dB"], dC=p["dC"], dA=p["dA"], dD=p["dD"],
                   dbias=p["dbias"])
        if c["gate"]:
            out["dz"] = p["dz"]
        return out
    if c["op"] == "norm":
        if c["mode"] == "serve":
            bd.rmsnorm(s["x"], s["w"], residual=s["r"], sum_out=p["sum"], q=p["q"], scale=p["scale"], eps=EPS)
            # what the 8 bits stand for
            return dict(sum=p["sum"], y=torch.mul(p["q"], p["scale"][:, None], out=p["y"]), scale=p["scale"])
        bd.rmsnorm(s["x"], s["w"], residual=s["r"], sum_out=p["sum"], y=p["y"], eps=EPS)
        bd.rmsnorm_adjoint(p["sum"], s["w"], s["dy"], p["dx"], p["dw"], p["ws"], dsum=s["ds"], eps=EPS)
        return dict(sum=p["sum"], y=p["y"], dx=p["dx"], dw=p["dw"])
    q, scale = (s["xq"], s["xs"]) if c["given"] else (p["q"], p["scale"])
    if not c["given"]:
        bd.quant_rows(s["x"], q, scale)
    bd.gemm_i8(q, scale, s["wq"], s["ws"], p["out"], p["ws"], bias=s["bias"])
    return p["out"]


def run(state):
    if own:
        return _run_own(state)
    c = state["case"]
    if c["op"] == "norm":
        return _norm(state)
    if c["op"] == "product":
        return _product(state)
    return {"conv train": _conv_train, "conv step": _conv_step, "scan prompt": _scan_prompt,
            "scan train": _scan_train, "scan step": _scan_step}[c["op"] + " " + c["mode"]](state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "conv":
        B, T, D, W = case["B"], case["T"], case["D"], case["W"]
        if case["mode"] == "step":  # token, output, state in and out, weights
            return dict(bytes=e * D * (2 * B + 2 * B * (W - 1) + W + 1), flops=B * D * (2 * W + 6))
        # x and dy read, y and dx written
        return dict(bytes=4 * e * B * T * D + (e + 4) * D * (W + 1), flops=B * T * D * (6 * W + 20))
    if case["op"] == "scan":
        B, T, D, N, G = case["B"], case["T"], case["D"], case["N"], case["G"]
        rows, z = B * T, 1 if case["gate"] else 0
        shared = 4 * D * (N + 2)
        if case["mode"] == "step":  # the state is read and written, in 32 bits
            return dict(bytes=e * rows * (D * (3 + z) + 2 * G * N) + 8 * B * D * N + shared,
                        flops=rows * D * (7 * N + 25))
        if case["mode"] == "prompt":
            return dict(bytes=e * rows * (D * (3 + z) + 2 * G * N) + 8 * B * D * N + shared,
                        flops=rows * D * (7 * N + 25))
        # u, dt, dy, (z), B, C read; y, du, ddt, (dz), dB, dC written
        return dict(bytes=e * rows * (D * (6 + 2 * z) + 4 * G * N) + 2 * shared, flops=rows * D * (24 * N + 60))
    if case["op"] == "norm":
        rows, n = case["rows"], case["n"]
        if case["mode"] == "serve":  # x, r read, s written, 8 bits and their scale
            return dict(bytes=rows * n * (3 * e + 1) + 4 * rows + e * n, flops=rows * n * 8)
        # x, r, dy, ds read; s, y, dx written
        return dict(bytes=7 * e * rows * n + (e + 4) * n, flops=rows * n * 16)
    M, N, K = case["M"], case["N"], case["K"]
    return dict(bytes=M * K * (1 if case["given"] else e) + N * K + (4 + e) * N + 4 * M + e * M * N,
                flops=2.0 * M * N * K)


# ---------------------------------------------------------------------------
# the definitions in 64 bits, one step after another
# ---------------------------------------------------------------------------
def _sig(x):
    return 1 / (1 + torch.exp(-x))


def exact(case, seed):
    s = prepare(case, seed)
    d = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v for k, v in s.items()}
    with torch.no_grad():
        if case["op"] == "conv":
            return _exact_conv_step(case, d) if case["mode"] == "step" else _exact_conv_train(case, d)
        if case["op"] == "scan":
            return _exact_scan_step(case, d) if case["mode"] == "step" else _exact_scan(case, d)
        return _exact_norm(case, d, s) if case["op"] == "norm" else _exact_product(case, d)


def _exact_conv_train(case, d):
    B, T, D, W = case["B"], case["T"], case["D"], case["W"]
    out = dict(y=torch.zeros(B, T, D, dtype=torch.float64, device=DEV),
               dx=torch.zeros(B, T, D, dtype=torch.float64, device=DEV),
               dw=torch.zeros(D, W, dtype=torch.float64, device=DEV),
               dbias=torch.zeros(D, dtype=torch.float64, device=DEV))
    for b in range(B):
        n = T if d["lengths"] is None else int(d["lengths"][b])
        if n == 0:
            continue
        x, dy = d["x"][b, :n], d["dy"][b, :n]
        a = d["bias"].expand(n, D).clone()
        for k in range(W):  # tap k reaches back W - 1 - k steps
            back = W - 1 - k
            if back < n:
                a[back:] += d["w"][:, k] * x[:n - back]
        p = _sig(a)
        out["y"][b, :n] = a * p
        da = dy * (p + a * p * (1 - p))
        out["dbias"] += da.sum(0)
        for k in range(W):
            back = W - 1 - k
            if back < n:
                out["dx"][b, :n - back] += d["w"][:, k] * da[back:]
                out["dw"][:, k] += (da[back:] * x[:n - back]).sum(0)
    return out


def _exact_conv_step(case, d):
    B, W = case["B"], case["W"]
    y = torch.zeros(B, case["D"], dtype=torch.float64, device=DEV)
    state = d["state"].clone()
    for b in range(B):
        at = b if d["slots"] is None else int(d["slots"][b])
        if at < 0:
            continue
        a = d["bias"] + d["w"][:, W - 1] * d["x"][b]
        for k in range(W - 1):
            a = a + d["w"][:, k] * d["state"][at, k]
        y[b] = a * _sig(a)
        state[at] = torch.cat([d["state"][at, 1:], d["x"][b][None]])
    return dict(y=y, state=state)


def _exact_scan(case, d):
    B, T, D, N, G = case["B"], case["T"], case["D"], case["N"], case["G"]
    train = case["mode"] == "train"
    if B * T * D * N * 8 * (2 if train else 0) > 40e9:
        return None
    f64 = dict(dtype=torch.float64, device=DEV)
    length = torch.full((B,), T, device=DEV) if d["lengths"] is None else d["lengths"]
    v = d["dt"] + d["dt_bias"]
    delta = torch.logaddexp(v, torch.zeros_like(v))
    A = d["A"]
    h = torch.zeros(B, D, N, **f64) if train else d["h0"].clone()
    y = torch.zeros(B, T, D, **f64)
    kept = torch.empty(B, T + 1, D, N, **f64) if train else None
    if train:
        kept[:, 0] = h

    def wide(m, t):
        return m[:, t].reshape(B, G, N).repeat_interleave(D // G, 1)

    for t in range(T):
        on = t < length
        if not train and bool(d["lengths"] is not None) and t % 64 == 0 and not bool(on.any()):
            break
        new = torch.exp(delta[:, t, :, None] * A) * h + (delta[:, t] * d["u"][:, t])[..., None] * wide(d["Bm"], t)
        h = torch.where(on[:, None, None], new, h)
        y[:, t] = ((h * wide(d["Cm"], t)).sum(-1) + d["D"] * d["u"][:, t]) * on[:, None]
        if train:
            kept[:, t + 1] = h
    gate = 1.0 if d["z"] is None else d["z"] * _sig(d["z"])
    if not train:
        return dict(y=y * gate, h=h)
    on = (torch.arange(T, device=DEV)[None] < length[:, None])[..., None].double()
    e = d["dy"] * gate * on
    out = dict(y=y * gate, du=torch.zeros(B, T, D, **f64), ddt=torch.zeros(B, T, D, **f64),
               dB=torch.zeros(B, T, G * N, **f64), dC=torch.zeros(B, T, G * N, **f64),
               dA=torch.zeros(D, N, **f64), dD=(e * d["u"]).sum((0, 1)))
    g = torch.zeros(B, D, N, **f64)
    for t in reversed(range(T)):
        live = on[:, t, :, None]
        a = torch.exp(delta[:, t, :, None] * A)
        at = (g + wide(d["Cm"], t) * e[:, t, :, None]) * live
        gb = (at * wide(d["Bm"], t)).sum(-1)
        q = at * a * kept[:, t]
        out["du"][:, t] = delta[:, t] * gb + d["D"] * e[:, t]
        out["ddt"][:, t] = (d["u"][:, t] * gb + (q * A).sum(-1)) * _sig(v[:, t])
        out["dA"] += (q * delta[:, t, :, None]).sum(0)
        x = (delta[:, t] * d["u"][:, t])[..., None] * at
        out["dB"][:, t] = x.reshape(B, G, D // G, N).sum(2).reshape(B, G * N)
        out["dC"][:, t] = (e[:, t, :, None] * kept[:, t + 1]).reshape(B, G, D // G, N).sum(2).reshape(B, G * N)
        g = torch.where(live > 0, at * a, g)
    out["dbias"] = out["ddt"].sum((0, 1))
    if d["z"] is not None:
        p = _sig(d["z"])
        out["dz"] = d["dy"] * y * (p + d["z"] * p * (1 - p))
    return out


def _exact_scan_step(case, d):
    B, D, N, G = case["B"], case["D"], case["N"], case["G"]
    y = torch.zeros(B, D, dtype=torch.float64, device=DEV)
    state = d["state"].clone()
    for b in range(B):
        at = b if d["slots"] is None else int(d["slots"][b])
        if at < 0:
            continue
        v = d["dt"][b] + d["dt_bias"]
        delta = torch.logaddexp(v, torch.zeros_like(v))[:, None]
        bm = d["Bm"][b].reshape(G, 1, N).expand(G, D // G, N).reshape(D, N)
        cm = d["Cm"][b].reshape(G, 1, N).expand(G, D // G, N).reshape(D, N)
        state[at] = torch.exp(delta * d["A"]) * d["state"][at] + delta * d["u"][b][:, None] * bm
        y[b] = (state[at] * cm).sum(1) + d["D"] * d["u"][b]
        if d["z"] is not None:
            y[b] *= d["z"][b] * _sig(d["z"][b])
    return dict(y=y, state=state)


def _exact_norm(case, d, s):
    n = case["n"]
    total = (d["x"] + d["r"]).to(s["x"].dtype).double()
    norm = torch.sqrt((total ** 2).sum(1, keepdim=True) / n + EPS)
    y = total / norm * d["w"]
    if case["mode"] == "serve":
        scale = y.abs().amax(1) / 127
        q = torch.round(y / torch.where(scale > 0, scale, torch.ones_like(scale))[:, None])
        return dict(sum=total, y=q * scale[:, None], scale=scale)
    t = d["dy"] * d["w"]
    dx = t / norm - total * (t * total).sum(1, keepdim=True) / (n * norm ** 3) + d["ds"]
    return dict(sum=total, y=y, dx=dx, dw=(d["dy"] * total / norm).sum(0))


def _exact_product(case, d):
    if case["M"] * case["N"] * case["K"] > 3e11:
        return None
    if case["given"]:
        q, scale = d["xq"].double(), d["xs"]
    else:
        scale = d["x"].abs().amax(1) / 127
        q = torch.round(d["x"] / torch.where(scale > 0, scale, torch.ones_like(scale))[:, None])
    return (q @ d["wq"].double().t()) * (scale[:, None] * d["ws"]) + d["bias"]
