"""The gated block's operators at the ends of their ranges: far gates, large
values, long memories, exact operands, long sums.  Every tolerance counts
roundings: U = 2^-24 is half a step of fp32 relative to the value, and the
device's exponential, root and reciprocal are good to one step, 2 U."""
import pytest
import torch

import gated_reference as R
from nonlinear_rnn_evaluation_newton_amd import binding as bd
from test_gpu_gated import BF, F, example, gated_problem, gen, nan, near, rnd, work

pytestmark = pytest.mark.gpu
TOL = 5e-5  # of an output's largest value, for arithmetic in 32 bits over up to 250 steps
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    bd.lib()


# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [BF, F])
def test_gates_past_the_exponentials_range(dtype):
    """Gates whose e^-x passes fp32 (x below -88.7) and its logarithm's sum, from the
    gate itself and from the bias: closed gates, with finite outputs and gradients."""
    g = gen(40)
    B, T = 1, 70
    far = torch.linspace(-131, -86, 181)
    D = 2 * far.numel()
    p = gated_problem(g, dtype, B, T, D)
    p["r_bias"].zero_(), p["i_bias"].zero_()
    for k, some in (("r", slice(0, far.numel())), ("i", slice(far.numel(), D))):
        p[k][:, ::2, some] = far.to(dtype)
        p[k][:, 1::2, some] += far.to(dtype) / 2
        p[k + "_bias"][some][::2] = far[::2] / 2
        p[k][:, ::2, some][..., ::2] = far[::2].to(dtype) / 2  # every other channel: half from the bias
    dy = rnd(g, B, T, D, dtype=dtype)
    dev = {k: v.cuda() for k, v in p.items()}
    main, kw = (dev["x"], dev["r"], dev["i"], dev["decay"]), dict(r_bias=dev["r_bias"], i_bias=dev["i_bias"])
    ws = work(bd.gated_workspace_bytes(dtype, B, T, D))
    y, states = nan(B, T, D, dtype=dtype), nan(*bd.gated_states_shape(B, T, D))
    bd.gated_scan(*main, y, ws, states=states, **kw)
    near(y, R.gated(**p)[0], TOL, "y")
    o = dict(dx=nan(B, T, D, dtype=dtype), dr=nan(B, T, D, dtype=dtype), di=nan(B, T, D, dtype=dtype))
    bd.gated_scan_adjoint(*main, states, dy.cuda(), ws, **kw, **o)
    r = R.gated_grads(**p, dy=dy)
    for k, v in o.items():
        near(v, r[k], TOL, k)
    for t in (0, 1):
        state, h0 = rnd(g, B, D), nan(B, D, dtype=dtype)
        pool = state.cuda()
        bd.gated_step(*(v[:, t] for v in main[:3]), dev["decay"], pool, h0, **kw)
        one = {k: v[:, t:t + 1] if v.dim() == 3 else v for k, v in p.items()}
        near(pool, R.gated(**one, h0=state)[1], TOL, "state")


# ---------------------------------------------------------------------------
PRODUCT_SIZES = [  # M, N, K, group: one, two and four tiles of columns, one and two of rows, every number of groups in 128 columns
    (1, 40, 300, 128), (3, 33, 1001, 64), (17, 50, 700, 32), (5, 20, 513, 96), (3, 8201, 130, 32), (16, 16400, 260, 64),
    (33, 8300, 300, 128), (40, 16400, 513, 32)]


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("zero", [True, False])
@pytest.mark.parametrize("case", PRODUCT_SIZES)
def test_product_of_large_rows(dtype, zero, case):
    """Rows up to 1e36, of one sign and of both, by the largest and the smallest
    numbers: sums of K terms of up to 31 steps, each sum rounded K times at most."""
    M, N, K, group = case
    print("large rows", dtype, zero, case, flush=True)
    g = gen(M + N + K)
    G = -(-K // group)
    scale = (2.0 ** -20 * (torch.rand(N, G, generator=g) + 0.5)).to(dtype)
    z = torch.randint(0, 16, (N, G), generator=g).to(dtype) if zero else None
    q = torch.randint(0, 256, (N, (K + 1) // 2), generator=g, dtype=torch.uint8)
    q[0::3], q[1::3] = 255, 0
    top = torch.tensor(0.99e36).to(dtype)
    x = torch.where(torch.rand(M, K, generator=g) < 0.5, top, -top)
    x[0] = top
    if M > 1:
        x[1] = -top
    out = nan(M, N, dtype=dtype)
    bd.gemm_w4(x.cuda(), q.cuda(), scale.cuda(), out, group, zero=None if z is None else z.cuda())
    ref = x.double() @ R.weights(q, scale, K, group, z).t()
    got = out.double().cpu()
    assert torch.isfinite(got).all(), torch.nonzero(~torch.isfinite(got))[:4].tolist()
    steps = scale.double().repeat_interleave(group, 1)[:, :K]
    room = 4 * K ** 0.5 * U * (x.double().abs() @ (31 * steps).t()) + (2.0 ** -8 if dtype == BF else U) * ref.abs()
    assert bool(((got - ref).abs() <= room).all()), float(((got - ref).abs() / room).max())


@pytest.mark.parametrize("zero", [True, False])
@pytest.mark.parametrize("case", PRODUCT_SIZES)
def test_product_has_every_bit_of_fp32_rows(zero, case):
    """One column with a weight other than 0 for each output: the result is x times
    a power of two, bit for bit.  All 24 bits of x are random: two operands of eight
    bits instead of three would miss nearly every one."""
    M, N, K, group = case
    g = gen(M + N + K + 1)
    G = -(-K // group)
    bits = torch.randint(1 << 23, 1 << 24, (M, K), generator=g).float()
    x = bits * 2.0 ** torch.randint(-40, 10, (M, K), generator=g).float()
    col, up = torch.randint(0, K, (N,), generator=g), torch.rand(N, generator=g) < 0.5
    q = torch.full((N, K + K % 2), 8, dtype=torch.uint8)
    step = torch.where(up, 4, -2)  # q - 8
    q[torch.arange(N), col] = (8 + step).to(torch.uint8)
    power = torch.randint(-3, 4, (N, G), generator=g).float()
    scale = 2.0 ** power
    out = nan(M, N)
    bd.gemm_w4(x.cuda(), (q[:, ::2] | q[:, 1::2] << 4).cuda(), scale.cuda(), out, group,
               zero=torch.full((N, G), 8.0, device="cuda") if zero else None)
    assert torch.equal(out.cpu(), x[:, col] * (step.float() * scale[torch.arange(N), col // group]))


# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [BF, F])
def test_long_memories(dtype):
    """Channels that remember most of a long sequence (a decay of 0.008 behind nearly
    closed gates, inputs of one sign).  States and their gradients are within 256 U of
    the largest: their decay is the sum of v over 1024 steps at a time, known to
    some 40 U of itself with the gates' far exponents (0.37 of that in e^-V), the input's
    factor to 20 U; inside those 1024 steps a value passes at most 30 factors of 2 U, and
    the 24 pieces of 1024 steps round it once each, without a factor's error."""
    g = gen(50)
    B, T = 1, 24601
    gate = torch.tensor([-3.0, -6.0, -9.0, -12.0]).repeat(9)
    D = gate.numel()
    p = dict(x=(1 + 0.5 * rnd(g, B, T, D)).to(dtype), r=rnd(g, B, T, D, std=0.1).to(dtype), i=rnd(g, B, T, D, dtype=dtype),
             decay=0.008 * (1 + 0.2 * torch.rand(D, generator=g)), r_bias=gate, i_bias=rnd(g, D))
    p["r"][..., ::2] = 0  # every other channel has a constant gate
    h0, dh, dy = 100 * rnd(g, B, D), 10 * rnd(g, B, D), (0.5 + rnd(g, B, T, D)).to(dtype)
    dev = {k: v.cuda() for k, v in p.items()}
    main, kw = (dev["x"], dev["r"], dev["i"], dev["decay"]), dict(r_bias=dev["r_bias"], i_bias=dev["i_bias"])
    ws = work(bd.gated_workspace_bytes(dtype, B, T, D))
    y, hl, states = nan(B, T, D, dtype=dtype), nan(B, D), nan(*bd.gated_states_shape(B, T, D))
    bd.gated_scan(*main, y, ws, h0=h0.cuda(), h_last=hl, states=states, **kw)
    ry, rh, hs = R.gated(**p, h0=h0, keep=True)

    def close(got, ref, k, dim):  # each channel by its own largest value
        off = (got.double().cpu() - ref).abs() - (2.0 ** -8 * ref.abs() if got.dtype == BF else 0)
        off = (off / ref.abs().amax(dim, keepdim=True)).max()
        assert float(off) <= 256 * U, (k, float(off) / U)

    close(hl, rh, "h", 0)
    close(states, torch.stack(hs[:-1][::bd.GATED_STATE_STEPS], 1), "states", (0, 1))
    close(y, ry, "y", (0, 1))
    o = dict(dx=nan(B, T, D, dtype=dtype), dr=nan(B, T, D, dtype=dtype), di=nan(B, T, D, dtype=dtype), dh0=nan(B, D),
             ddecay=nan(D))
    bd.gated_scan_adjoint(*main, states, dy.cuda(), ws, dh_last=dh.cuda(), **kw, **o)
    r = R.gated_grads(**p, dy=dy, h0=h0, dh_last=dh)
    for k in ("dx", "di", "dh0"):
        close(o[k], r[k], k, 0 if k == "dh0" else (0, 1))
    # g a^2 / m i x and g a h are each off by twice that of their own size; the sum over
    # the steps by that of the sum of the sizes
    gr, gi, a, m = R._gates(p["r"], p["i"], p["decay"], p["r_bias"], p["i_bias"])
    grad = (r["dx"] / (m * gi)).abs()  # |g|
    size = grad * (a * a / m * gi * p["x"].double().abs() + a * torch.stack(hs[:-1], 1).abs())
    part = p["decay"].double() * gr * (1 - gr)
    off = (o["dr"].double().cpu() - r["dr"]).abs() - (2.0 ** -8 * r["dr"].abs() if dtype == BF else 0)
    assert float((off / (size * part).amax((0, 1))).max()) <= 512 * U
    off = (o["ddecay"].double().cpu() - r["ddecay"]).abs() / (size * gr).sum((0, 1))
    assert float(off.max()) <= 512 * U, float(off.max()) / U


@pytest.mark.parametrize("dtype", [BF, F])
def test_long_memories_by_single_tokens(dtype):
    """The same with a step for each token: the state is rounded to fp32 at each, by U of
    it at most, to either side: 4 sqrt(T) U, beside the 60 U of decay and input."""
    g = gen(51)
    B, T = 1, 20000
    gate = torch.tensor([-3.0, -6.0, -9.0]).repeat(12)
    D = gate.numel()
    p = dict(x=(1 + 0.5 * rnd(g, B, T, D)).to(dtype), r=torch.zeros(B, T, D, dtype=dtype), i=rnd(g, B, T, D, dtype=dtype),
             decay=0.008 * (1 + 0.2 * torch.rand(D, generator=g)), r_bias=gate, i_bias=rnd(g, D))
    h0 = 100 * rnd(g, B, D)
    dev = {k: v.cuda() for k, v in p.items()}
    state, y = h0.cuda(), nan(B, D, dtype=dtype)
    for t in range(T):
        bd.gated_step(dev["x"][:, t], dev["r"][:, t], dev["i"][:, t], dev["decay"], state, y, r_bias=dev["r_bias"],
                      i_bias=dev["i_bias"])
    _, rh, hs = R.gated(**p, h0=h0, keep=True)
    off = (state.double().cpu() - rh).abs() / torch.stack(hs).abs().amax((0, 1))
    assert float(off.max()) <= (4 * T ** 0.5 + 60) * U, float(off.max()) / U


# ---------------------------------------------------------------------------
@pytest.mark.parametrize("n", [1, 3, 7, 64, 100, 257, 700, 1111, 2049, 5003, 9001, 20001])
def test_block_norm_factor(n):
    """Rows of powers of two without eps: the sum of squares is exact (below 2^24), the
    mean's rounding (U) counts half under the root, the factor is rounded once (U, and a
    hundredth for what its making leaves), and its product with a power of two is exact."""
    g, rows = gen(n), max(4, min(4000, 2_000_000 // n))
    x = 2.0 ** torch.randint(0, 4, (rows, n), generator=g).float() * torch.where(torch.rand(rows, n, generator=g) < 0.5, 1, -1)
    t, y = nan(rows, n), nan(rows, n)
    bd.block_norm(x.cuda(), None, t, y=y, eps=0.0)
    ref = R.block_norm(x, eps=0.0)
    off = ((t.double().cpu() - ref).abs() / ref.abs()).max()
    assert float(off) <= 1.51 * U, float(off) / U


@pytest.mark.parametrize("scale", [2.0 ** -70, 2.0 ** -20, 2.0 ** 20, 2.0 ** 55])
def test_block_norm_factor_of_far_rows(scale):
    """The same where the mean is denormal or near fp32's largest; and rows whose squares
    pass it, whose factor is 0, and rows of zeros with an eps."""
    x = torch.full((4, 40), scale)
    x[:, ::2] *= 2
    t = nan(4, 40)
    bd.block_norm(x.cuda(), None, t, eps=0.0)
    ref = R.block_norm(x, eps=0.0)
    assert float(((t.double().cpu() - ref).abs() / ref).max()) <= (1.51 * U if scale > 2.0 ** -60 else 2.0 ** -9)
    bd.block_norm(torch.full((4, 40), 1e30, device="cuda"), None, t)
    assert bool((t == 0).all())
    bd.block_norm(torch.zeros(4, 40, device="cuda"), None, t)
    assert bool((t == 0).all())


@pytest.mark.parametrize("n", [3, 80, 1111, 9001])
@pytest.mark.parametrize("gate", ["silu", "sigmoid"])
def test_block_norm_gates_in_fp32(n, gate):
    """Rows of ones, whose factor is 1: t is the gate itself.  e^-z: one step of the
    exponential and two roundings (4 U), the sum (U), the reciprocal (2 U) and the
    product with z (U): 8 U of the value.  Its derivative is a sum of two such terms,
    p and z p (1 - p), where 1 - p is off by the 7 U of p: 12 U of their sizes with
    the products, and 8 U |z| p more for 1 - p."""
    z = torch.linspace(-86, 86, n * 5).view(5, n)
    x, t = torch.ones(5, n), nan(5, n)
    bd.block_norm(x.cuda(), None, t, z=z.cuda(), gate=gate, eps=0.0)
    ref, p = R.act(z, gate), torch.sigmoid(z.double())
    assert float(((t.double().cpu() - ref[0]).abs() / ref[0].abs().clamp(min=1e-300)).nan_to_num(0).max()) <= 8 * U
    dz = nan(5, n)
    bd.block_norm_adjoint(x.cuda(), None, None, work(bd.block_norm_workspace_bytes(F, 5, n)), z=z.cuda(), gate=gate,
                          dt=torch.ones(5, n, device="cuda"), dz=dz, eps=0.0)
    size = p * (1 - p) if gate == "sigmoid" else p + z.double().abs() * p * (1 - p)
    room = 12 * U * size + 8 * U * p * (1 if gate == "sigmoid" else z.double().abs())
    assert bool(((dz.double().cpu() - ref[1]).abs() <= room).all())


def test_block_norm_sums_of_long_rows():
    """A row of 2^25 values: its squares are added 256 at a time in fp32 (256 U at most,
    half of it under the root), then in 64 bits; a gradient takes three such sums."""
    n = (1 << 25) + 40
    g = torch.Generator(device="cuda").manual_seed(71)
    x, dt, dy = (torch.randn(1, n, generator=g, device="cuda") for _ in range(3))
    t, y, dx = (torch.full_like(x, float("nan")) for _ in range(3))
    bd.block_norm(x, None, t, y=y)
    ref = R.block_norm(x)
    assert bool(((t.double() - ref).abs() <= 130 * U * ref.abs()).all())
    ref = R.norm_next(t)
    assert bool(((y.double() - ref).abs() <= 130 * U * ref.abs()).all())
    dt += x  # a gradient along the row, which the norm takes off
    bd.block_norm_adjoint(x, None, dx, work(bd.block_norm_workspace_bytes(F, 1, n)), t=t, dt=dt, dy=dy)
    ref = R.block_norm_grads(x, t=t, dt=dt, dy=dy)["dx"]
    assert float((dx.double() - ref).abs().max()) <= 520 * U * float(ref.abs().max())


@pytest.mark.parametrize("dtype", [BF, F])
def test_block_norm_of_very_long_rows(dtype):
    """More columns than one grid dimension has threads for in the weights' sums."""
    rows, n = 2, (1 << 26) + 40
    g = torch.Generator(device="cuda").manual_seed(70)
    x, res, dt, dy = (torch.randn(rows, n, generator=g, device="cuda", dtype=dtype) for _ in range(4))
    w, wn = (1 + 0.1 * torch.randn(n, generator=g, device="cuda", dtype=dtype) for _ in range(2))
    t, y = (torch.full_like(x, float("nan")) for _ in range(2))
    bd.block_norm(x, w, t, residual=res, y=y, w_next=wn)
    o = dict(dx=torch.full_like(x, float("nan")), dw=nan(n), dscale=nan(n), dw_next=nan(n))
    bd.block_norm_adjoint(x, w, workspace=work(bd.block_norm_workspace_bytes(dtype, rows, n)), t=t, dt=dt, dy=dy,
                          w_next=wn, **o)
    r = R.block_norm_grads(x, w, w_next=wn, t=t, dt=dt, dy=dy)
    r.update(t=R.block_norm(x, w, residual=res), y=R.norm_next(t, wn))
    for k, v in dict(o, t=t, y=y).items():
        off = (v.double() - r[k]).abs() - (2.0 ** -8 * r[k].abs() if v.dtype == BF else 0)
        assert float(off.max()) <= TOL * max(1.0, float(r[k].abs().max())), k


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("n", [3, 12, 300])
def test_block_norm_weights_gradients_of_very_many_rows(dtype, n):
    """2^26 equal rows (of stride 0): every addition of a sum rounds to the same side
    while the sum's exponent stays.  512 of them in fp32 lose 256 U at most, as the sum
    grows from nothing; a term itself has some 12 roundings."""
    g, rows = gen(80 + n), 1 << 26
    x, dt, dy, t = (1 + torch.rand(1, n, generator=g).to(dtype) for _ in range(4))
    w, scale, wn = (1 + torch.rand(n, generator=g).to(dtype) for _ in range(3))
    wide = lambda v: v.cuda().expand(rows, n)  # noqa: E731
    o = dict(dw=nan(n), dscale=nan(n), dw_next=nan(n))
    bd.block_norm_adjoint(wide(x), w.cuda(), None, work(bd.block_norm_workspace_bytes(dtype, rows, n)), scale=scale.cuda(),
                          w_next=wn.cuda(), t=wide(t), dt=wide(dt), dy=wide(dy), **o)
    r = R.block_norm_grads(x, w, scale=scale, w_next=wn, t=t, dt=dt, dy=dy)
    # (of the gradient at t the norm takes off what lies along t: the size of dt is left of it and more)
    size = x.double() * R._rstd(x.double(), 1e-5) * (dt.double() + 2 * dy.double() * wn.double() * R._rstd(t.double(), 1e-5))
    for k, f in (("dw", scale), ("dscale", w), ("dw_next", None)):
        top = r[k].abs() if f is None else (size * f.double())[0]
        off = ((o[k].double().cpu() - rows * r[k]).abs() / (rows * top)).max()
        assert float(off) <= 270 * U, (k, float(off) / U)


# ---------------------------------------------------------------------------
def test_example_rows_of_any_view():
    """Gates that are views cut in time or transposed keep their rows."""
    ex = example()
    g = gen(60)
    x, w = rnd(g, 3, 5, 24).cuda(), rnd(g, 24).cuda()
    whole = rnd(g, 3, 9, 48).cuda()
    for z in (whole[:, 2:7, 3:27], whole[:, :5, :24].contiguous(), whole.transpose(1, 2)[:, :5, :9].repeat(1, 1, 3)[..., :24],
              rnd(g, 5, 3, 24).cuda().transpose(0, 1)):
        near(ex.Norm.apply(x, w, z).view(15, 24), R.block_norm(x.view(15, 24).cpu(), w.cpu(), z.reshape(15, 24).cpu()), TOL, "t")


def test_example_keeps_its_decays():
    """Large steps do not take a decay below 0, where the recurrence is not defined."""
    ex = example()
    model = ex.Model(dim=32, width=64, blocks=1, seed=5)
    losses = ex.train(model, steps=40, lr=0.1)
    assert all(v == v for v in losses), losses
    for b in model.blocks:
        assert float(b["decay"].detach().min()) > 0


def test_example_does_not_differentiate_twice():
    """The operators have no second derivatives: asking for one is an error, not a zero."""
    ex = example()
    model = ex.Model(dim=16, width=32, blocks=1, dtype=F)
    s = torch.randn(1, 20, 16, device="cuda", requires_grad=True)
    first, = torch.autograd.grad(model.forward(s).square().sum(), s, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        first.sum().backward()


# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [BF, F])
def test_decays_of_any_size(dtype):
    """Decays from 0 to 1e38 over many tiles, each channel held to its own largest value:
    a state that is only kept, one that hardly fades, one that is gone at once.  A decay
    of 1e-38 leaves 1 - a^2 below 2^-126 at some steps, whose inputs' terms (1e-19 of x)
    may be 0: its outputs are finite and its state is the first one."""
    g = gen(90)
    B, T = 2, 1500
    each = torch.tensor([0.0, 1e-38, 1e-30, 1e-12, 1e-7, 1e-5, 1e-3, 0.03, 0.0624, 0.126, 1.0, 20.0, 80.0, 150.0, 1e10, 1e38])
    D = each.numel() * 5
    p = gated_problem(g, dtype, B, T, D)
    p["decay"] = each.repeat(5)
    h0, dh, dy = rnd(g, B, D), rnd(g, B, D), rnd(g, B, T, D, dtype=dtype)
    dev = {k: v.cuda() for k, v in p.items()}
    main, kw = (dev["x"], dev["r"], dev["i"], dev["decay"]), dict(r_bias=dev["r_bias"], i_bias=dev["i_bias"])
    ws = work(bd.gated_workspace_bytes(dtype, B, T, D))
    o = dict(y=nan(B, T, D, dtype=dtype), h=nan(B, D), dx=nan(B, T, D, dtype=dtype), dr=nan(B, T, D, dtype=dtype),
             di=nan(B, T, D, dtype=dtype), ddecay=nan(D), dh0=nan(B, D))
    states = nan(*bd.gated_states_shape(B, T, D))
    bd.gated_scan(*main, o["y"], ws, h0=h0.cuda(), h_last=o["h"], states=states, **kw)
    bd.gated_scan_adjoint(*main, states, dy.cuda(), ws, dh_last=dh.cuda(), **kw,
                          **{k: o[k] for k in ("dx", "dr", "di", "ddecay", "dh0")})
    y, h, hs = R.gated(**p, h0=h0, keep=True)
    r = R.gated_grads(**p, dy=dy, h0=h0, dh_last=dh)
    r.update(y=y, h=h)
    gr, gi, a, m = R._gates(p["r"], p["i"], p["decay"], p["r_bias"], p["i_bias"])
    inv = torch.where(m > 0, 1 / m, torch.zeros((), dtype=R.F64))
    grad = R.gated_grads(**{**p, "i": torch.full_like(p["i"], 1e4)}, dy=dy, h0=h0, dh_last=dh)["dx"] * inv  # g, where m > 0
    # at a decay of 0, g is the sum of all that follows
    grad = torch.where(m > 0, grad, (dy.double().flip(1).cumsum(1).flip(1) + dh.double()[:, None])).abs()
    size = grad * (a * a * inv * gi * p["x"].double().abs() + a * torch.stack(hs[:-1], 1).abs())
    size = dict(dr=(size * p["decay"].double() * gr * (1 - gr)).amax((0, 1)), ddecay=(size * gr).sum((0, 1)))
    near(o["h"][:, 1::each.numel()], h0.double()[:, 1::each.numel()], TOL, "h")
    for k, v in o.items():
        assert torch.isfinite(v).all(), k
        top = size[k] if k in size else r[k].abs().amax(tuple(range(v.dim() - 1)))
        off = (v.double().cpu() - r[k]).abs() - (2.0 ** -8 * r[k].abs() if v.dtype == BF else 0)
        room = TOL * top
        if k == "dh0":  # a_0 = e^-v times the rest: v, of 16 roundings at most (two gates' terms, sigmoid, product), counts v times
            room = room + 16 * U * p["decay"].double() * gr[:, 0].amax(0) * top
        bad = off > room
        bad[..., 1::each.numel()] = False  # (1e-38)
        assert not bad.any(), (k, p["decay"][torch.nonzero(bad)[0, -1]], float((off / top).nan_to_num(0).max()))


def test_infinite_inputs_stay_in_their_channel():
    """From an infinite input on its channel's states are infinite or NaN (its tiles' factors
    may be 0, and 0 times infinity is a NaN), by scan and by step, and no other's are."""
    g = gen(91)
    B, T, D = 1, 2500, 20
    p = gated_problem(g, F, B, T, D)
    p["x"][0, 700, 3], p["x"][0, 900, 7] = float("inf"), float("-inf")
    dev = {k: v.cuda() for k, v in p.items()}
    kw = dict(r_bias=dev["r_bias"], i_bias=dev["i_bias"])
    y, h = nan(B, T, D), nan(B, D)
    bd.gated_scan(dev["x"], dev["r"], dev["i"], dev["decay"], y, work(bd.gated_workspace_bytes(F, B, T, D)), h_last=h, **kw)
    ref = R.gated(**p)[0]
    assert torch.equal(torch.isfinite(y).cpu(), torch.isfinite(ref))
    near(y[..., 8:], ref[..., 8:], TOL, "y")
    one = nan(B, D)
    bd.gated_step(*(dev[k][:, 0] for k in ("x", "r", "i")), dev["decay"], h, one, **kw)
    assert torch.equal(torch.isfinite(one).cpu(), torch.isfinite(ref[:, -1]))


@pytest.mark.parametrize("dtype", [BF, F])
def test_two_million_steps(dtype):
    """A chain of thousands of tiles of 8, against the recurrence by doubling in 64 bits:
    256 U as for long memories, and 4096 roundings to either side beside them, 4 x 64 U."""
    B, T, D = 1, 2 ** 21 + 77, 6
    g = torch.Generator(device="cuda").manual_seed(95)
    x, r, i, dy = (torch.randn(B, T, D, generator=g, device="cuda").add_(0.5).to(dtype) for _ in range(4))
    decay = torch.tensor([1e-5, 1e-3, 0.008, 0.05, 0.3, 2.0], device="cuda")
    rb = torch.tensor([-2.0, -6.0, -9.0, -3.0, 0.0, 1.0], device="cuda")
    ws = work(bd.gated_workspace_bytes(dtype, B, T, D))
    y, dx = (torch.full_like(x, float("nan")) for _ in range(2))
    h, dh0, states = nan(B, D), nan(B, D), nan(*bd.gated_states_shape(B, T, D))
    bd.gated_scan(x, r, i, decay, y, ws, r_bias=rb, h_last=h, states=states)
    bd.gated_scan_adjoint(x, r, i, decay, states, dy, ws, r_bias=rb, dx=dx, dh0=dh0)
    gi, v = torch.sigmoid(i.double()), decay.double() * torch.sigmoid(r.double() + rb.double())
    m = torch.sqrt(-torch.expm1(-2 * v))

    def recurrence(a, b):  # along axis 1
        a, s = a.clone(), 1
        while s < T:
            b = torch.cat([b[:, :s], b[:, s:] + a[:, s:] * b[:, :-s]], 1)
            a = torch.cat([a[:, :s], a[:, s:] * a[:, :-s]], 1)
            s *= 2
        return b

    ry = recurrence(torch.exp(-v), m * gi * x.double())
    later = torch.cat([torch.exp(-v)[:, 1:], torch.zeros(B, 1, D, dtype=R.F64, device="cuda")], 1)
    rg = recurrence(later.flip(1), dy.double().flip(1)).flip(1)
    for k, got, ref in (("h", h, ry[:, -1]), ("states", states[:, 1:], ry[:, 63::64][:, :states.shape[1] - 1]), ("y", y, ry),
                        ("dx", dx, rg * m * gi), ("dh0", dh0, rg[:, 0] * torch.exp(-v[:, 0]))):
        dims = tuple(range(got.dim() - 1))
        off = (got.double() - ref).abs() - (2.0 ** -8 * ref.abs() if got.dtype == BF else 0)
        off = off.amax(dims) / (ry if k in ("h", "states") else ref if k != "dh0" else rg).abs().amax((0, 1) if k != "dx" else dims)
        assert float(off.max()) <= 512 * U, (k, (off / U).tolist())


# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("zero", [True, False])
@pytest.mark.parametrize("group", [32, 64, 1024])
def test_four_bits_of_every_size(dtype, zero, group):
    """Groups from fp32's denormals to its largest values, and values that lie between two
    numbers: the 4-bit form is the definition's, bit for bit."""
    g, N, K = gen(group), 260, 1030
    size = 2.0 ** torch.linspace(-147, 126, N, dtype=R.F64)[:, None]
    w = (torch.randn(N, K, generator=g).clamp(-1.9, 1.9).double() * size).to(dtype)
    half = (torch.randint(-15, 16, (N, K), generator=g) * 0.5).double() * size.clamp(2.0 ** -140, 2.0 ** 120)
    w[::2] = half.to(dtype)[::2]  # a group's scale is a power of two over 7 or 15: ties and what lies next to them
    rq, rs, rz = R.quant(w, group, zero)
    q = torch.zeros(N, (K + 1) // 2, dtype=torch.uint8, device="cuda")
    G = -(-K // group)
    scale, z, back = nan(N, G, dtype=dtype), nan(N, G, dtype=dtype) if zero else None, nan(N, K, dtype=dtype)
    bd.quant_w4(w.cuda(), q, scale, group, zero=z)
    assert torch.equal(scale.cpu(), rs), torch.nonzero(scale.cpu() != rs)[:5].tolist()
    assert not zero or torch.equal(z.cpu(), rz), torch.nonzero(z.cpu() != rz)[:5].tolist()
    live = (rs.float() > 0).repeat_interleave(group, 1)[:, :K]  # a scale that rounds to 0 stands for zeros, whatever q is
    bad = (R.unpack(q.cpu(), K) != rq) & live
    assert not bad.any(), (int(bad.sum()), torch.nonzero(bad)[:5].tolist())
    bd.dequant_w4(q, scale, back, group, zero=z)
    assert torch.equal(back.cpu(), R.weights(q.cpu(), rs, K, group, rz if zero else None, to=F).to(dtype))


def test_product_of_tiny_fp32_rows():
    """From 2^-109 on every bit of x counts; below it what lies above 2^-133 does."""
    g, N, K, M = gen(97), 64, 128, 60
    x = (torch.randint(1 << 23, 1 << 24, (M, K), generator=g).double() * 2.0 ** (-23 - 140 + torch.arange(M)[:, None])).float()
    col = torch.randint(0, K, (N,), generator=g)
    q = torch.full((N, K), 8, dtype=torch.uint8)
    q[torch.arange(N), col] = 12
    out = nan(M, N)
    bd.gemm_w4(x.cuda(), (q[:, ::2] | q[:, 1::2] << 4).cuda(), torch.full((N, 4), 2.0 ** 60, device="cuda"), out, 32)
    off = (out.double().cpu() - x[:, col].double() * 2.0 ** 62).abs()
    assert float(off[31:].max()) == 0 and float(off.max()) <= 2.0 ** (62 - 133)
