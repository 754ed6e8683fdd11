"""GPU parity of the gated block's operators (gated scan, norms around a block,
products on 4-bit weights) against the 64-bit forms in gated_reference.py,
through the binding.

Tolerances:
  arithmetic in 32 bits   5e-5 of the output's largest value: a state keeps its
                          past for up to 250 steps here, with 1.8e-7 (three
                          roundings of 2^-24 in the decay and the sum) each
  sums over all steps or rows (weights' gradients)   1e-4 of the largest value
  bf16 outputs            2^-8 of the value itself beside that: one rounding to
                          8 significant bits, to the nearest
  products                4 sqrt(K) 2^-24 sum |x| (31 scale): the roundings of K
                          partial sums of terms up to 31 steps add like a random
                          walk, at four deviations
  4-bit forms             equal, bit for bit
Outputs are filled with NaN first, so that a value that is not written shows.
Values past a sequence's length are NaN in the inputs and must not be read."""
import pytest
import torch

import gated_reference as R
from nonlinear_rnn_evaluation_newton_amd import binding as bd

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32
TOL = 5e-5
SUM_TOL = 1e-4


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    bd.lib()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rnd(g, *shape, dtype=F, std=1.0):
    return (torch.randn(*shape, generator=g) * std).to(dtype)


def nan(*shape, dtype=F):
    return torch.full(shape, float("nan"), dtype=dtype, device="cuda")


def work(nbytes):
    return torch.empty(nbytes, dtype=torch.uint8, device="cuda").fill_(255)


def near(got, ref, tol, what):
    unit = 2.0 ** -8 if got.dtype == BF else 0.0
    got = got.double().cpu()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert torch.isfinite(got).all(), (what, "not finite at", torch.nonzero(~torch.isfinite(got))[:4].tolist())
    if ref.numel():
        err, top = (got - ref).abs() - unit * ref.abs(), max(1.0, float(ref.abs().max()))
        assert float(err.max()) <= tol * top, (what, float(err.max()), top)


def cut(x, lengths):
    """x with NaN past each sequence's length."""
    if lengths is None:
        return x
    x = x.clone()
    for b, n in enumerate(lengths.tolist()):
        x[b, max(n, 0):] = float("nan")
    return x


def slot_in(x, left, right):
    """x as a slice of a wider tensor on the GPU, left and right columns around it."""
    wide = torch.zeros(x.shape[:-1] + (left + x.shape[-1] + right,), dtype=x.dtype)
    wide[..., left:left + x.shape[-1]] = x
    return wide.cuda()[..., left:left + x.shape[-1]]


# ---------------------------------------------------------------------------
def gated_problem(g, dtype, B, T, D):
    return dict(x=rnd(g, B, T, D, dtype=dtype), r=rnd(g, B, T, D, dtype=dtype), i=rnd(g, B, T, D, dtype=dtype),
                decay=torch.rand(D, generator=g) * 0.8 + 0.05, r_bias=rnd(g, D), i_bias=rnd(g, D))


GATED = [  # B, T, D, ragged, columns around the slices
    (1, 1, 1, False, (0, 0)), (2, 5, 3, True, (1, 2)), (3, 16, 64, False, (0, 64)), (3, 17, 65, True, (0, 1)),
    (2, 127, 40, True, (8, 0)), (2, 128, 66, False, (0, 0)), (2, 129, 67, True, (0, 5)), (1, 256, 130, False, (0, 0)),
    (4, 257, 33, True, (3, 0)), (2, 1000, 24, True, (0, 24)), (1, 4100, 7, False, (0, 0)), (33, 70, 4, True, (0, 0)),
    (1, 640, 256, True, (0, 0)), (5, 384, 2, False, (2, 0))]


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("case", GATED)
def test_gated(dtype, case):
    B, T, D, ragged, pad = case
    print("gated", dtype, case, flush=True)
    g = gen(B * 1000 + T + D)
    p = gated_problem(g, dtype, B, T, D)
    n = None
    if ragged:
        n = torch.randint(-2, T + 3, (B,), generator=g).int()
        n[0] = T
        if B > 1:
            n[-1] = 0
    h0, dh, dy = rnd(g, B, D), rnd(g, B, D), rnd(g, B, T, D, dtype=dtype)
    dev = {k: v.cuda() for k, v in p.items()}
    for k in ("x", "r", "i"):
        dev[k] = slot_in(cut(p[k], n), *pad)
    main, kw = (dev["x"], dev["r"], dev["i"], dev["decay"]), dict(r_bias=dev["r_bias"], i_bias=dev["i_bias"],
                                                                  lengths=None if n is None else n.cuda())
    ws = work(bd.gated_workspace_bytes(dtype, B, T, D))
    y, hl, states = nan(B, T, D, dtype=dtype), nan(B, D), nan(*bd.gated_states_shape(B, T, D))
    bd.gated_scan(*main, y, ws, h0=h0.cuda(), h_last=hl, states=states, **kw)
    ry, rh, hs = R.gated(**p, h0=h0, lengths=n, keep=True)
    near(y, ry, TOL, "y")
    near(hl, rh, TOL, "h")
    want, on = torch.stack(hs[:-1][::bd.GATED_STATE_STEPS], 1), torch.ones(B, states.shape[1], dtype=torch.bool)
    if n is not None:
        on = torch.arange(states.shape[1])[None] * bd.GATED_STATE_STEPS < n[:, None]
    near(states.cpu()[on], want[on], TOL, "states")
    same = h0.cuda()  # the state in place
    ws.fill_(255)
    bd.gated_scan(*main, y, ws, h0=same, h_last=same, **kw)
    assert torch.equal(same, hl)
    o = dict(dx=nan(B, T, D, dtype=dtype), dr=nan(B, T, D, dtype=dtype), di=nan(B, T, D, dtype=dtype), ddecay=nan(D),
             dr_bias=nan(D), di_bias=nan(D), dh0=nan(B, D))
    ws.fill_(255)
    bd.gated_scan_adjoint(*main, states, slot_in(cut(dy, n), *pad), ws, dh_last=dh.cuda(), **kw, **o)
    r = R.gated_grads(**p, dy=dy, h0=h0, lengths=n, dh_last=dh)
    for k, v in o.items():
        near(v, r[k], SUM_TOL if k in ("ddecay", "dr_bias", "di_bias") else TOL, k)
    # any subset of the outputs, the same bits
    few, fx = nan(D), nan(B, T, D, dtype=dtype)
    bd.gated_scan_adjoint(*main, states, slot_in(cut(dy, n), *pad), ws, dh_last=dh.cuda(), **kw, dr_bias=few, dx=fx)
    assert torch.equal(few, o["dr_bias"]) and torch.equal(fx, o["dx"])
    bd.gated_scan_adjoint(*main, states, slot_in(cut(dy, n), *pad), ws, **kw, di=fx)
    near(fx, R.gated_grads(**p, dy=dy, h0=h0, lengths=n)["di"], TOL, "di")


@pytest.mark.parametrize("dtype", [BF, F])
def test_gated_pieces_and_bare(dtype):
    """No biases and no first state; a second piece that goes on from the first one's state."""
    g = gen(4)
    B, T, D = 2, 900, 70
    p = gated_problem(g, dtype, B, T, D)
    p["r_bias"] = p["i_bias"] = None
    dev = {k: None if v is None else v.cuda() for k, v in p.items()}
    ws = work(bd.gated_workspace_bytes(dtype, B, T, D))
    y, h, y2 = nan(B, T, D, dtype=dtype), nan(B, D), nan(B, T, D, dtype=dtype)
    bd.gated_scan(dev["x"], dev["r"], dev["i"], dev["decay"], y, ws)
    ry, rh = R.gated(**p)
    near(y, ry, TOL, "y")
    for t0, t1, h0 in ((0, 401, None), (401, T, h)):
        bd.gated_scan(dev["x"][:, t0:t1], dev["r"][:, t0:t1], dev["i"][:, t0:t1], dev["decay"], y2[:, t0:t1], ws, h0=h0,
                      h_last=h)
    near(y2, ry, TOL, "two pieces")
    near(h, rh, TOL, "two pieces' state")


@pytest.mark.parametrize("dtype", [BF, F])
def test_gated_ends_of_the_range(dtype):
    """Gates that are open, closed or far beyond, a decay of 0 and a large one:
    finite outputs and gradients, equal to the definition's limits."""
    g = gen(6)
    B, T, D = 1, 300, 16
    p = gated_problem(g, dtype, B, T, D)
    p["r_bias"] = p["i_bias"] = None
    inf = float("inf")
    for d, v in enumerate((-inf, inf, -1000.0, 1000.0, -90.0, 90.0, -30.0, 30.0)):
        p["r"][:, :, d] = v
        p["i"][:, :, 8 + d] = v
    p["decay"][10], p["decay"][11] = 0.0, 60.0
    dy = rnd(g, B, T, D, dtype=dtype)
    dev = {k: None if v is None else v.cuda() for k, v in p.items()}
    ws = work(bd.gated_workspace_bytes(dtype, B, T, D))
    y, states = nan(B, T, D, dtype=dtype), nan(*bd.gated_states_shape(B, T, D))
    main = (dev["x"], dev["r"], dev["i"], dev["decay"])
    bd.gated_scan(*main, y, ws, states=states)
    near(y, R.gated(**p)[0], TOL, "y")
    o = dict(dx=nan(B, T, D, dtype=dtype), dr=nan(B, T, D, dtype=dtype), di=nan(B, T, D, dtype=dtype))
    bd.gated_scan_adjoint(*main, states, dy.cuda(), ws, **o)
    r = R.gated_grads(**p, dy=dy)
    for k, v in o.items():
        near(v, r[k], TOL, k)


def test_gated_gradient_against_differences():
    """The kernels' gradients against central differences of the kernels' own
    outputs (fp32): steps of 1e-2 along the gradient, a loss of order 1e2 known
    to about 1e-5 of itself gives 1e-3 / 1e-2 of a gradient of order 10;
    compared to 1 per cent."""
    g = gen(11)
    B, T, D = 2, 300, 70
    p = gated_problem(g, F, B, T, D)
    dy, dev = rnd(g, B, T, D).cuda(), {k: v.cuda() for k, v in p.items()}
    ws = work(bd.gated_workspace_bytes(F, B, T, D))

    def loss(q, states=None):
        y = nan(B, T, D)
        bd.gated_scan(q["x"], q["r"], q["i"], q["decay"], y, ws, r_bias=q["r_bias"], i_bias=q["i_bias"], states=states)
        return float((y.double() * dy.double()).sum())

    states = nan(*bd.gated_states_shape(B, T, D))
    loss(dev, states)
    o = {"d" + k: nan(*v.shape) for k, v in dev.items()}
    bd.gated_scan_adjoint(dev["x"], dev["r"], dev["i"], dev["decay"], states, dy, ws, r_bias=dev["r_bias"],
                          i_bias=dev["i_bias"], **o)
    for k in dev:
        d = o["d" + k] / o["d" + k].norm()
        h = 1e-2
        num = (loss({**dev, k: dev[k] + h * d}) - loss({**dev, k: dev[k] - h * d})) / (2 * h)
        ana = float(o["d" + k].double().norm())
        assert abs(num - ana) <= 1e-2 * ana, (k, num, ana)


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("B,D", [(1, 1), (5, 40), (4, 33), (3, 1030), (7, 2048)])
def test_gated_step(dtype, B, D):
    g = gen(B + D)
    pool = B + 2
    p = gated_problem(g, dtype, B, 1, D)
    st = rnd(g, pool, D)
    some = torch.randperm(pool, generator=g)[:B].int()
    if B > 2:
        some[1], some[2] = -1, pool  # idle: below and above the pool
    dev = {k: v.cuda() for k, v in p.items()}
    tok = [slot_in(p[k][:, 0], 1, D) for k in ("x", "r", "i")]
    for slots, bias in ((None, True), (some, True), (some, False)):
        state, y = st.cuda(), nan(B, D, dtype=dtype)
        rb, ib = (dev["r_bias"], dev["i_bias"]) if bias else (None, None)
        bd.gated_step(*tok, dev["decay"], state, y, r_bias=rb, i_bias=ib, slots=None if slots is None else slots.cuda())
        ry, rs = torch.zeros(B, D, dtype=R.F64), st.double().clone()
        for b, k in enumerate(range(B) if slots is None else slots.tolist()):
            if 0 <= k < pool:
                yy, hh = R.gated(p["x"][b][None], p["r"][b][None], p["i"][b][None], p["decay"],
                                 p["r_bias"] if bias else None, p["i_bias"] if bias else None, st[k][None])
                ry[b], rs[k] = yy[0, 0], hh[0]
        near(y, ry, TOL, "y")
        near(state, rs, TOL, "state")


# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("rows,n", [(1, 1), (3, 5), (5, 64), (7, 512), (9, 257), (4, 1024), (3, 2049), (6, 2048),
                                    (2, 4104), (2, 8192), (2, 9001), (2, 16384), (2, 20001), (300, 72), (2100, 40)])
@pytest.mark.parametrize("gate", [None, "silu", "sigmoid"])
def test_block_norm(dtype, rows, n, gate):
    print("block norm", dtype, rows, n, gate, flush=True)
    g = gen(rows + n)
    x, z, res, dt, dy = (rnd(g, rows, n, dtype=dtype) for _ in range(5))
    w, scale, wn = (rnd(g, n, dtype=dtype) for _ in range(3))
    c = lambda v: None if v is None else v.cuda()  # noqa: E731
    z = z if gate else None
    kw = dict(gate=gate) if gate else {}
    ws = work(bd.block_norm_workspace_bytes(dtype, rows, n))
    for full in (True, False):
        if not full:
            scale = wn = res = dy = None
            w = w if gate == "silu" else None
        pad = (0, 0) if full else (1, 3)
        xs, zs = slot_in(x, *pad), None if z is None else slot_in(z, *pad)
        t, y = nan(rows, n, dtype=dtype), nan(rows, n, dtype=dtype) if full else None
        bd.block_norm(xs, c(w), t, z=zs, scale=c(scale), residual=c(res), y=y, w_next=c(wn), **kw)
        near(t, R.block_norm(x, w, z, gate, scale, res), TOL, "t")
        if full:
            near(y, R.norm_next(t.cpu(), wn), TOL, "y")
            same = res.cuda()  # the stream in place
            bd.block_norm(xs, c(w), same, z=zs, scale=c(scale), residual=same, y=y, w_next=c(wn), **kw)
            assert torch.equal(same, t)
        o = dict(dx=nan(rows, n, dtype=dtype), dres=nan(rows, n, dtype=dtype), dw=nan(n), dscale=nan(n),
                 dz=nan(rows, n, dtype=dtype) if gate else None, dw_next=nan(n) if full else None)
        kw2 = dict(z=zs, scale=c(scale), w_next=c(wn), t=t, **kw)
        bd.block_norm_adjoint(xs, c(w), workspace=ws, dt=slot_in(dt, *pad), dy=c(dy), **kw2, **o)
        r = R.block_norm_grads(x, w, z, gate, scale, wn, t.cpu(), dt, dy)
        for k, v in o.items():
            if v is not None:
                near(v, r[k], SUM_TOL if v.dim() == 1 else TOL, k)
        # the gradient that arrives, in place; any subset of the outputs
        same, few = dt.cuda(), nan(n)
        bd.block_norm_adjoint(xs, c(w), None, ws, dt=same, dy=c(dy), dres=same, dscale=few, **kw2)
        assert torch.equal(same, o["dres"]) and torch.equal(few, o["dscale"])
    # the norm after it alone has a gradient too
    wn, dy = rnd(g, n, dtype=dtype), rnd(g, rows, n, dtype=dtype)
    dx = nan(rows, n, dtype=dtype)
    bd.block_norm_adjoint(xs, c(w), dx, ws, z=zs, t=t, dy=dy.cuda(), w_next=wn.cuda(), **kw)
    near(dx, R.block_norm_grads(x, w, z, gate, None, wn, t.cpu(), None, dy)["dx"], TOL, "dx")


@pytest.mark.parametrize("dtype,n", [(BF, 513), (BF, 2049), (BF, 4099), (BF, 8193), (BF, 8199), (BF, 8705), (F, 257),
                                     (F, 1025), (F, 4097), (F, 4099), (F, 4353), (F, 6146), (BF, 12297), (F, 8193)])
def test_block_norm_in_place_at_row_ends(dtype, n):
    """The last vector of a row overlaps the one before: where it lies in another
    wavefront, or is taken later, a result over its input must not reach it."""
    g, rows = gen(n), 5
    x, z, res, dt, dy = (rnd(g, rows, n, dtype=dtype).cuda() for _ in range(5))
    w, scale, wn = (rnd(g, n, dtype=dtype).cuda() for _ in range(3))
    parts = dict(z=z, scale=scale, w_next=wn)
    ws = work(bd.block_norm_workspace_bytes(dtype, rows, n))
    t, y = nan(rows, n, dtype=dtype), nan(rows, n, dtype=dtype)
    bd.block_norm(x, w, t, residual=res, y=y, **parts)
    near(t, R.block_norm(x.cpu(), w.cpu(), z.cpu(), "silu", scale.cpu(), res.cpu()), TOL, "t")
    r = R.block_norm_grads(x.cpu(), w.cpu(), z.cpu(), "silu", scale.cpu(), wn.cpu(), t.cpu(), dt.cpu(), dy.cpu())
    for k in range(3):
        same = res.clone()
        bd.block_norm(x, w, same, residual=same, y=y, **parts)
        assert torch.equal(same, t)
        same = dt.clone()
        o = dict(dx=nan(rows, n, dtype=dtype), dz=nan(rows, n, dtype=dtype), dw=nan(n), dscale=nan(n), dw_next=nan(n))
        bd.block_norm_adjoint(x, w, workspace=ws, t=t, dt=same, dy=dy, dres=same, **parts, **o)
        near(same, r["dres"], TOL, "dres")
        for key, v in o.items():
            near(v, r[key], SUM_TOL if v.dim() == 1 else TOL, key)


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("n", [2, 64, 700])
def test_block_norm_of_tiny_rows(dtype, n):
    """Rows of +-2^-66 without eps: the squares, 2^-132, are denormal and exact, so
    the norm is +-1 up to the roundings of 1/n, of the mean, of the root (one place,
    2^-23) and of the product: 2^-22 with room; 1 is exact in bf16.  The gradient
    of a row along itself is 0, of any other dt it is dt 2^66 less that part."""
    x = torch.where(torch.arange(n) % 2 == 0, 1.0, -1.0).to(dtype).repeat(3, 1) * 2.0 ** -66
    t, y, dx = nan(3, n, dtype=dtype), nan(3, n, dtype=dtype), nan(3, n, dtype=dtype)
    bd.block_norm(x.cuda(), None, t, y=y, eps=0.0)
    sign = x.double().sign()
    for got in (t, y):
        assert float((got.double().cpu() - sign).abs().max()) <= (2.0 ** -22 if dtype == F else 0.0)
    dt = torch.ones(3, n, dtype=dtype)
    bd.block_norm_adjoint(x.cuda(), None, dx, work(bd.block_norm_workspace_bytes(dtype, 3, n)), dt=dt.cuda(), eps=0.0)
    ref = 2.0 ** 66 * (1 - sign * sign.mean(1, keepdim=True))  # (n is even: the mean is 0)
    assert float((dx.double().cpu() - ref).abs().max()) <= 2.0 ** 66 * (2.0 ** -22 if dtype == F else 2.0 ** -8)


def test_block_norm_zero_rows_and_far_gates():
    """A row of zeros, and gates beyond the exponential's range."""
    inf = float("inf")
    x = torch.zeros(2, 72, device="cuda")
    x[1] = 1.0
    z = torch.tensor([-inf, -200.0, -100.0, 0.0, 100.0, 200.0, inf, 5.0], device="cuda").repeat(2, 9)
    t = nan(2, 72)
    bd.block_norm(x, None, t, z=z, gate="sigmoid")
    near(t, R.block_norm(x.cpu(), None, z.cpu(), "sigmoid"), TOL, "t")
    z[:, 0::8] = -300.0
    z[:, 6::8] = 300.0
    ws, dx, dz = work(bd.block_norm_workspace_bytes(F, 2, 72)), nan(2, 72), nan(2, 72)
    for gate in ("sigmoid", "silu"):
        bd.block_norm(x, None, t, z=z, gate=gate, eps=1e-3)
        near(t, R.block_norm(x.cpu(), None, z.cpu(), gate, eps=1e-3), TOL, "t")
        bd.block_norm_adjoint(x, None, dx, ws, z=z, gate=gate, dt=torch.ones_like(x), dz=dz, eps=1e-3)
        r = R.block_norm_grads(x.cpu(), None, z.cpu(), gate, dt=torch.ones(2, 72), eps=1e-3)
        near(dx, r["dx"], TOL, "dx")
        near(dz, r["dz"], TOL, "dz")


# ---------------------------------------------------------------------------
def packed(g, N, K, left=0, right=0):
    """Random 4-bit numbers [N, (K + 1) / 2] as a slice of wider rows on the CPU."""
    wide = torch.randint(0, 256, (N, left + (K + 1) // 2 + right), generator=g, dtype=torch.uint8)
    return wide, slice(left, left + (K + 1) // 2)


PRODUCTS = [  # M, N, K, group, bytes around the rows of q, columns around x
    (1, 1, 1, 32, (0, 0), (0, 0)), (1, 16, 32, 32, (0, 0), (0, 0)), (2, 17, 33, 32, (1, 0), (0, 1)),
    (1, 40, 127, 64, (0, 3), (0, 0)), (3, 33, 128, 128, (0, 0), (8, 0)), (16, 64, 1000, 32, (0, 0), (0, 0)),
    (17, 50, 1001, 64, (0, 0), (1, 0)), (31, 16, 2048, 128, (0, 0), (0, 0)), (32, 100, 513, 96, (2, 3), (0, 0)),
    (33, 7, 700, 128, (0, 0), (0, 0)), (64, 130, 1500, 160, (0, 0), (0, 2)), (65, 20, 300, 32, (0, 0), (0, 0)),
    (150, 35, 260, 64, (0, 0), (0, 0)), (5, 300, 4096, 4096, (0, 0), (0, 0)), (1, 2000, 640, 1 << 20, (0, 0), (0, 0)),
    (4, 19, 9000, 256, (5, 0), (3, 3)),
    # two and four tiles of columns, two of rows by two and by four; long rows with every number of groups in 128 columns
    (3, 8201, 130, 32, (0, 0), (0, 0)), (16, 16400, 260, 64, (0, 0), (0, 0)), (33, 8300, 300, 128, (0, 0), (0, 0)),
    (20, 16390, 270, 64, (0, 0), (0, 0)), (40, 16400, 513, 32, (0, 0), (0, 0)), (2, 40, 5000, 64, (0, 0), (0, 0)),
    (2, 40, 5003, 32, (0, 0), (0, 0)), (2, 40, 7000, 384, (0, 0), (0, 0))]


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("zero", [True, False])
@pytest.mark.parametrize("case", PRODUCTS)
def test_product(dtype, zero, case):
    M, N, K, group, qpad, xpad = case
    print("4-bit product", dtype, zero, case, flush=True)
    g = gen(M + N + K)
    G = -(-K // group)
    wide, at = packed(g, N, K, *qpad)
    x, bias = rnd(g, M, K, dtype=dtype), rnd(g, N, dtype=dtype)
    scale = (torch.rand(N, G, generator=g) + 0.5).to(dtype)
    z = (torch.rand(N, G, generator=g) * 15).to(dtype) if zero else None  # between the numbers too
    out = nan(M, N + 5, dtype=dtype)
    args = (slot_in(x, *xpad), wide.cuda()[:, at], scale.cuda(), out[:, 2:N + 2], group)
    for b in (bias, None):
        out.fill_(float("nan"))
        bd.gemm_w4(*args, zero=None if z is None else z.cuda(), bias=None if b is None else b.cuda())
        assert torch.isnan(out[:, :2]).all() and torch.isnan(out[:, N + 2:]).all()
        ref = x.double() @ R.weights(wide[:, at], scale, K, group, z).t() + (0 if b is None else b.double())
        got = out[:, 2:N + 2].double().cpu()
        assert torch.isfinite(got).all()
        steps = scale.double().repeat_interleave(group, 1)[:, :K] if G > 1 else scale.double().expand(N, K)
        room = 4 * K ** 0.5 * 2.0 ** -24 * (x.double().abs() @ (31 * steps).t()) + 2.0 ** -24 * ref.abs()
        if dtype == BF:
            room = room + 2.0 ** -8 * ref.abs()
        assert bool(((got - ref).abs() <= room).all()), float(((got - ref).abs() / room).max())


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("zero", [True, False])
@pytest.mark.parametrize("N,K,group,qpad,wpad", [
    (1, 1, 32, (0, 0), (0, 0)), (3, 31, 32, (0, 0), (0, 1)), (5, 77, 32, (1, 0), (3, 0)), (4, 130, 64, (0, 0), (0, 0)),
    (7, 1001, 128, (0, 2), (0, 0)), (3, 500, 96, (0, 0), (0, 0)), (2, 3000, 256, (0, 0), (0, 0)),
    (2, 5000, 1024, (3, 0), (0, 0)), (300, 64, 4096, (0, 0), (0, 0))])
def test_four_bits(dtype, zero, N, K, group, qpad, wpad):
    g = gen(N + K)
    w = rnd(g, N, K, dtype=dtype)
    w[:, :group] *= 100
    if N > 2:
        w[1], w[2] = w[1].abs(), 0  # one sign only; nothing
    G = -(-K // group)
    rq, rs, rz = R.quant(w, group, zero)
    wide = torch.full((N, qpad[0] + (K + 1) // 2 + qpad[1]), 85, dtype=torch.uint8, device="cuda")
    q = wide[:, qpad[0]:qpad[0] + (K + 1) // 2]
    scale, z = nan(N, G, dtype=dtype), nan(N, G, dtype=dtype) if zero else None
    bd.quant_w4(slot_in(w, *wpad), q, scale, group, zero=z)
    assert torch.equal(R.unpack(q.cpu(), K), rq)
    assert torch.equal(scale.cpu(), rs) and (z is None or torch.equal(z.cpu(), rz))
    assert bool((wide[:, :qpad[0]] == 85).all()) and bool((wide[:, qpad[0] + (K + 1) // 2:] == 85).all())
    out = nan(N, K + 4, dtype=dtype)
    bd.dequant_w4(q, scale, out[:, 1:K + 1], group, zero=z)
    ref = R.weights(q.cpu(), rs, K, group, rz if zero else None, to=F).to(dtype)
    assert torch.equal(out[:, 1:K + 1].cpu(), ref)
    assert torch.isnan(out[:, 0]).all() and torch.isnan(out[:, K + 1:]).all()


def test_four_bits_of_infinite_groups():
    w = torch.ones(2, 96, device="cuda")
    w[0, 3], w[0, 40] = float("inf"), float("nan")
    q, s, z = torch.zeros(2, 48, dtype=torch.uint8, device="cuda"), nan(2, 3), nan(2, 3)
    bd.quant_w4(w, q, s, 32)
    assert bool(torch.isinf(s[0, 0])) and bool(torch.isnan(s[0, 1])) and bool(torch.isfinite(s[0, 2:]).all())
    assert bool((R.unpack(q.cpu(), 96)[0, :64] == 8).all()) and bool((R.unpack(q.cpu(), 96)[1] == 15).all())
    bd.quant_w4(w, q, s, 32, zero=z)
    assert bool((z[0, :2] == 8).all()) and bool((R.unpack(q.cpu(), 96)[0, :64] == 8).all())


# ---------------------------------------------------------------------------
def test_run_of_all_on_another_stream_and_in_a_graph():
    """The operators one after another as a block uses them: on a side stream,
    captured, and replayed on new inputs with eager work between the replays."""
    g = gen(21)
    B, T, D = 2, 1300, 136
    dt = BF
    p = gated_problem(g, dt, B, T, D)
    dev = {k: v.cuda() for k, v in p.items()}
    z, s, dy, ds = (rnd(g, B * T, D, dtype=dt).cuda() for _ in range(4))
    w, scale, wn = (rnd(g, D, dtype=dt).cuda() for _ in range(3))
    new = lambda *shape, to=dt: nan(*shape, dtype=to)  # noqa: E731
    o = dict(h=new(B, T, D), states=new(*bd.gated_states_shape(B, T, D), to=F), t=new(B * T, D), y=new(B * T, D),
             dx=new(B * T, D), dz=new(B * T, D), dres=new(B * T, D), dw=new(D, to=F), dn=new(D, to=F), dv=new(B, T, D),
             dr=new(B, T, D), di=new(B, T, D), dd=new(D, to=F), out=new(64, 48), q=None)
    wf = rnd(g, 48, D, dtype=dt).cuda()
    q4, s4 = torch.zeros(48, D // 2, dtype=torch.uint8, device="cuda"), new(48, 2)
    pool = rnd(g, 4, D).cuda()
    start = pool.clone()
    ws, ws2 = work(bd.gated_workspace_bytes(dt, B, T, D)), work(bd.block_norm_workspace_bytes(dt, B * T, D))
    main = (dev["x"], dev["r"], dev["i"], dev["decay"])
    kw = dict(r_bias=dev["r_bias"], i_bias=dev["i_bias"])

    def run():
        bd.gated_scan(*main, o["h"], ws, states=o["states"], **kw)
        h = o["h"].view(B * T, D)
        parts = dict(z=z, scale=scale, w_next=wn)
        bd.block_norm(h, w, o["t"], residual=s, y=o["y"], **parts)
        bd.block_norm_adjoint(h, w, o["dx"], ws2, t=o["t"], dt=ds, dy=dy, dz=o["dz"], dres=o["dres"], dw=o["dw"],
                              dw_next=o["dn"], **parts)
        bd.gated_scan_adjoint(*main, o["states"], o["dx"].view(B, T, D), ws, dx=o["dv"], dr=o["dr"], di=o["di"],
                              ddecay=o["dd"], **kw)
        bd.quant_w4(wf, q4, s4, 96)
        bd.gemm_w4(o["y"][:64], q4, s4, o["out"], 96)
        bd.gated_step(*(v[:, 0] for v in main[:3]), dev["decay"], pool, o["h"][:, 0], **kw)

    def results():
        torch.cuda.synchronize()
        return {k: v.clone() for k, v in {**o, "pool": pool, "q4": q4, "s4": s4}.items() if v is not None}

    run()
    first = results()
    pool.copy_(start)
    for v in o.values():
        if v is not None:
            v.fill_(float("nan"))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    again = results()
    for k in first:
        assert torch.equal(first[k], again[k]), k
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for k in range(4):
        dev["x"].copy_(rnd(gen(100 + k), B, T, D, dtype=dt))
        s.copy_(rnd(gen(200 + k), B * T, D, dtype=dt))
        pool.copy_(start)
        run()
        want = results()
        pool.copy_(start)
        for v in o.values():
            if v is not None:
                v.fill_(float("nan"))
        graph.replay()
        got = results()
        for key in want:
            assert torch.equal(want[key], got[key]), (k, key)


# ---------------------------------------------------------------------------
# far offsets, many tiles, many rows
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("B,T,D,ragged", [(1, 20000, 66, False), (3, 3000, 5, True), (9, 1100, 515, True)])
def test_gated_many_tiles(dtype, B, T, D, ragged):
    """Sequences of several hundred tiles, and many columns of tiles at once;
    calls that repeat give the same bits, however the tiles met."""
    g = gen(T + D)
    p = gated_problem(g, dtype, B, T, D)
    n = None
    if ragged:
        n = torch.randint(0, T + 1, (B,), generator=g).int()
        n[0], n[-1] = T, 1
    h0, dh, dy = rnd(g, B, D), rnd(g, B, D), rnd(g, B, T, D, dtype=dtype)
    dev = {k: v.cuda() for k, v in p.items()}
    main, kw = (dev["x"], dev["r"], dev["i"], dev["decay"]), dict(r_bias=dev["r_bias"], i_bias=dev["i_bias"],
                                                                  lengths=None if n is None else n.cuda())
    ws = work(bd.gated_workspace_bytes(dtype, B, T, D))
    ry, rh = R.gated(**p, h0=h0, lengths=n)
    r = R.gated_grads(**p, dy=dy, h0=h0, lengths=n, dh_last=dh)
    first = None
    for _ in range(4):
        o = dict(y=nan(B, T, D, dtype=dtype), h=nan(B, D), dx=nan(B, T, D, dtype=dtype), dr=nan(B, T, D, dtype=dtype),
                 di=nan(B, T, D, dtype=dtype), ddecay=nan(D), dr_bias=nan(D), di_bias=nan(D), dh0=nan(B, D))
        states = nan(*bd.gated_states_shape(B, T, D))
        bd.gated_scan(*main, o["y"], ws, h0=h0.cuda(), h_last=o["h"], states=states, **kw)
        bd.gated_scan_adjoint(*main, states, dy.cuda(), ws, dh_last=dh.cuda(), **kw,
                              **{k: v for k, v in o.items() if k not in ("y", "h")})
        if first is None:
            first = o
            near(o["y"], ry, TOL, "y")
            near(o["h"], rh, TOL, "h")
            for k in ("dx", "dr", "di", "ddecay", "dr_bias", "di_bias", "dh0"):
                near(o[k], r[k], SUM_TOL if o[k].dim() == 1 else TOL, k)
        for k, v in o.items():
            assert torch.equal(v, first[k]), k


@pytest.mark.parametrize("dtype", [BF, F])
def test_gated_of_far_steps(dtype):
    """Time strides whose products with the steps pass 2^32 bytes."""
    g = gen(8)
    B, T, D, st = 1, 1300, 37, 1 << 21 if dtype == BF else 1 << 20
    p = gated_problem(g, dtype, B, T, D)
    base = torch.empty(T * st, dtype=dtype, device="cuda")
    far = {}
    for k, at in (("x", 0), ("r", 1000), ("i", 2001), ("y", 3000), ("dx", 4001)):
        far[k] = base.as_strided((B, T, D), (T * st, st, 1), at)
        far[k].copy_(p[k].cuda() if k in p else torch.full((B, T, D), float("nan"), dtype=dtype, device="cuda"))
    dev = {k: p[k].cuda() for k in ("decay", "r_bias", "i_bias")}
    ws, states = work(bd.gated_workspace_bytes(dtype, B, T, D)), nan(*bd.gated_states_shape(B, T, D))
    kw = dict(r_bias=dev["r_bias"], i_bias=dev["i_bias"])
    bd.gated_scan(far["x"], far["r"], far["i"], dev["decay"], far["y"], ws, states=states, **kw)
    near(far["y"].contiguous(), R.gated(**p)[0], TOL, "y")
    dy = rnd(g, B, T, D, dtype=dtype)
    bd.gated_scan_adjoint(far["x"], far["r"], far["i"], dev["decay"], states, dy.cuda(), ws, dx=far["dx"], **kw)
    near(far["dx"].contiguous(), R.gated_grads(**p, dy=dy)["dx"], TOL, "dx")


def test_gated_step_on_a_large_pool():
    """States past 2^32 bytes of the pool."""
    g = gen(9)
    B, D, pool = 3, 1001, 1_200_000
    p = gated_problem(g, F, B, 1, D)
    dev = {k: v.cuda() for k, v in p.items()}
    state, st = torch.empty(pool, D, device="cuda"), rnd(g, B, D)
    at = torch.tensor([pool - 1, 0, pool - 2])
    state[at.cuda()] = st.cuda()
    y = nan(B, D)
    bd.gated_step(dev["x"][:, 0], dev["r"][:, 0], dev["i"][:, 0], dev["decay"], state, y, r_bias=dev["r_bias"],
                  i_bias=dev["i_bias"], slots=at.int().cuda())
    ry, rh = R.gated(**p, h0=st)
    near(y, ry[:, 0], TOL, "y")
    near(state[at.cuda()], rh, TOL, "state")


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("n", [5, 300, 2051, 20000])
def test_block_norm_of_far_rows(dtype, n):
    """Rows that lie more than 2^32 bytes apart."""
    g, rows, ld = gen(n), 3, (1 << 31) + 40 if dtype == BF else (1 << 30) + 24
    base = torch.empty(ld * (rows - 1) + 8 * n, dtype=dtype, device="cuda")
    names = ("x", "z", "res", "dt", "dy")
    v = {k: rnd(g, rows, n, dtype=dtype) for k in names}
    far = {k: base.as_strided((rows, n), (ld, 1), i * n) for i, k in enumerate(names + ("t", "y", "dx"))}
    for k in far:
        far[k].copy_(v[k].cuda() if k in v else torch.full((rows, n), float("nan"), dtype=dtype, device="cuda"))
    bd.block_norm(far["x"], None, far["t"], z=far["z"], residual=far["res"], y=far["y"])
    near(far["t"].contiguous(), R.block_norm(v["x"], None, v["z"], "silu", None, v["res"]), TOL, "t")
    near(far["y"].contiguous(), R.norm_next(far["t"].cpu()), TOL, "y")
    ws = work(bd.block_norm_workspace_bytes(dtype, rows, n))
    bd.block_norm_adjoint(far["x"], None, far["dx"], ws, z=far["z"], t=far["t"], dt=far["dt"], dy=far["dy"])
    r = R.block_norm_grads(v["x"], None, v["z"], "silu", None, None, far["t"].cpu(), v["dt"], v["dy"])
    near(far["dx"].contiguous(), r["dx"], TOL, "dx")


@pytest.mark.parametrize("n", [3, 8])
def test_block_norm_of_very_many_rows(n):
    """More rows than one grid dimension has blocks for: the first and the last ones."""
    rows = (1 << 24) + 300
    x = torch.randn(rows, n, device="cuda", dtype=BF)
    t, y = torch.full_like(x, float("nan")), torch.full_like(x, float("nan"))
    bd.block_norm(x, None, t, y=y)
    dx = torch.full_like(x, float("nan"))
    bd.block_norm_adjoint(x, None, dx, work(bd.block_norm_workspace_bytes(BF, rows, n)), dt=t)
    for s in (slice(0, 400), slice(rows - 400, rows)):
        near(t[s], R.block_norm(x[s].cpu()), TOL, "t")
        near(y[s], R.norm_next(t[s].cpu()), TOL, "y")
        near(dx[s], R.block_norm_grads(x[s].cpu(), dt=t[s].cpu())["dx"], TOL, "dx")
    assert not torch.isnan(t).any() and not torch.isnan(dx).any()


@pytest.mark.parametrize("dtype", [BF, F])
def test_four_bits_of_far_rows(dtype):
    """Packed rows and rows of weights past 2^32 bytes; very many rows of x."""
    g, N, K, ld = gen(3), 40, 131, 120_000_000
    w = rnd(g, N, K, dtype=dtype)
    base = torch.empty(N * ld, dtype=torch.uint8, device="cuda")
    q = base.as_strided((N, (K + 1) // 2), (ld, 1), 7)
    scale = nan(N, 5, dtype=dtype)
    bd.quant_w4(w.cuda(), q, scale, 32)
    rq, rs, _ = R.quant(w, 32)
    assert torch.equal(R.unpack(q.cpu(), K), rq) and torch.equal(scale.cpu(), rs)
    x, out = rnd(g, 70000, K, dtype=dtype), nan(70000, N, dtype=dtype)
    bd.gemm_w4(x.cuda(), q, scale, out, 32)
    ws = R.weights(q.cpu(), rs, K, 32)
    ref = x.double() @ ws.t()
    room = 4 * K ** 0.5 * 2.0 ** -24 * (x.double().abs() @ (31 * rs.double().repeat_interleave(32, 1)[:, :K]).t())
    room = room + (2.0 ** -8 if dtype == BF else 2.0 ** -24) * ref.abs()
    assert bool(((out.double().cpu() - ref).abs() <= room).all())
    back = torch.empty(N * ld // 2, dtype=dtype, device="cuda").as_strided((N, K), (ld // 2, 1), 3)
    bd.dequant_w4(q, scale, back, 32)
    assert torch.equal(back.cpu(), R.weights(q.cpu(), rs, K, 32, to=F).to(dtype))


# ---------------------------------------------------------------------------
# the operators as a model calls them
# ---------------------------------------------------------------------------
def example():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "gated_block.py")
    spec = importlib.util.spec_from_file_location("gated_block", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    return ex


def plain_model(first, blocks, s, c):
    """The example's forward pass in elementary operations (any type, any device)."""
    def norm(v, w):
        return v / torch.sqrt((v * v).mean(-1, keepdim=True) + 1e-5) * w

    y = norm(s, first)
    for w in blocks:
        x, r, i, z = (y @ w["inp"].t()).split(c, -1)
        v = w["decay"] * torch.sigmoid(r + w["r_bias"])
        a, u = torch.exp(-v), torch.sqrt(-torch.expm1(-2 * v)) * torch.sigmoid(i + w["i_bias"]) * x
        h, hs = torch.zeros_like(u[:, 0]), []
        for t in range(s.shape[1]):
            h = a[:, t] * h + u[:, t]
            hs.append(h)
        o = (norm(torch.stack(hs, 1), w["norm"]) * z * torch.sigmoid(z)) @ w["out"].t()
        s = s + norm(o, w["post"]) * w["scale"]
        y = norm(s, w["after"])
    return y


def test_example_gradients():
    """The example's model in fp32: output and gradients of all weights against
    torch's autograd in 64 bits.  The products and the scans are off by 5e-5 at
    most; each of the five norms behind them passes an error on at no more than
    about twice its size: 32 x 5e-5, compared to 2e-3 of the largest value."""
    ex = example()
    model = ex.Model(dim=48, width=80, dtype=F, seed=4)
    s = torch.randn(2, 150, 48, generator=gen(5))
    dy = torch.randn(2, 150, 48, generator=gen(6))
    y = model.forward(s.cuda())
    y.backward(dy.cuda())
    first, blocks = model.first.detach().double().cpu().requires_grad_(), [
        {k: v.detach().double().cpu().requires_grad_() for k, v in b.items()} for b in model.blocks]
    ref = plain_model(first, blocks, s.double(), 80)
    ref.backward(dy.double())
    near(y.detach(), ref.detach(), 2e-3, "y")
    near(model.first.grad, first.grad, 2e-3, "first")
    for mine, theirs in zip(model.blocks, blocks):
        for k in mine:
            near(mine[k].grad, theirs[k].grad, 2e-3, k)


def test_example_runs():
    """A few training steps have finite losses; single tokens continue a prompt as
    the whole sequence does.  A prompt's products take the weights rounded to
    bf16 (2^-8 each), and a dozen values on the way are rounded to bf16 in both
    (half a step is 2^-8 of the value): 20 roundings in all, which go either way and
    stand for half of their sum at most, 10 2^-8 of the largest output."""
    ex = example()
    model = ex.Model(dim=64, width=96, seed=3)
    losses = ex.train(model, steps=3)
    assert all(v == v and v < 1e3 for v in losses), losses
    got, whole = ex.serve(model)
    assert torch.isfinite(got).all()
    assert float((got.float() - whole.float()).abs().max()) <= 10 * 2.0 ** -8 * float(whole.float().abs().max())


def test_two_streams_at_once():
    """Scans on two streams, each with its workspace, at the same time: the same bits as alone."""
    g, dt, B, T, D = gen(31), BF, 2, 6000, 192
    sets = []
    for _ in range(2):
        p = {k: v.cuda() for k, v in gated_problem(g, dt, B, T, D).items()}
        sets.append(dict(p=p, dy=rnd(g, B, T, D, dtype=dt).cuda(), ws=work(bd.gated_workspace_bytes(dt, B, T, D)),
                         states=nan(*bd.gated_states_shape(B, T, D))))

    def run(s, y, dx):
        p, kw = s["p"], dict(r_bias=s["p"]["r_bias"], i_bias=s["p"]["i_bias"])
        bd.gated_scan(p["x"], p["r"], p["i"], p["decay"], y, s["ws"], states=s["states"], **kw)
        bd.gated_scan_adjoint(p["x"], p["r"], p["i"], p["decay"], s["states"], s["dy"], s["ws"], dx=dx, **kw)

    alone = [(nan(B, T, D, dtype=dt), nan(B, T, D, dtype=dt)) for _ in sets]
    for s, (y, dx) in zip(sets, alone):
        run(s, y, dx)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    together = [(nan(B, T, D, dtype=dt), nan(B, T, D, dtype=dt)) for _ in sets]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, (y, dx), st in zip(sets, together, streams):
            with torch.cuda.stream(st):
                run(s, y, dx)
    torch.cuda.synchronize()
    for one, two in zip(alone, together):
        assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1])


def test_host_workspace_is_refused():
    """Every call that takes a workspace refuses one in host memory before it launches anything."""
    z = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    host, x, d = torch.empty(1 << 20, dtype=torch.uint8), z(2, 32, 16), z(16)
    states, rows = z(*bd.gated_states_shape(2, 32, 16)), z(64, 16)
    for name, call in (("gated_scan", lambda: bd.gated_scan(x, x, x, d, z(2, 32, 16), host)),
                       ("gated_scan_adjoint", lambda: bd.gated_scan_adjoint(x, x, x, d, states, x, host, dx=z(2, 32, 16))),
                       ("block_norm_adjoint", lambda: bd.block_norm_adjoint(rows, None, z(64, 16), host, dt=rows))):
        with pytest.raises(ValueError, match=name + ": the workspace must be on the GPU"):
            call()
