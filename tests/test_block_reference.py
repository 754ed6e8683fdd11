"""The 64-bit gradients that the GPU tests compare with, against central
differences of the 64-bit forward forms (CPU).

A central difference with step h has an error of h^2 / 6 times the third
derivative plus 2^-53 |f| / h; at h = 1e-5 and values of order 1 to 100 both
are below 1e-9, so 1e-6 of the gradient's size leaves room for the third
derivative and for long sums."""
import pytest
import torch

import block_reference as R

TOL, H = 1e-6, 1e-5


def check(f, grads, args, gen):
    """f(**args) is a number; grads: {name: gradient}; one random direction for each."""
    for name, g in grads.items():
        d = torch.randn(args[name].shape, generator=gen, dtype=R.F64)
        hi, lo = (f(**{**args, name: args[name] + s * H * d}) for s in (1, -1))
        num, ana = float((hi - lo) / (2 * H)), float((g * d).sum())
        assert abs(num - ana) <= TOL * max(1.0, abs(ana)), (name, num, ana)


def rnd(gen, *shape, std=1.0):
    return torch.randn(*shape, generator=gen, dtype=R.F64) * std


@pytest.mark.parametrize("W", [1, 2, 4])
@pytest.mark.parametrize("act", [True, False])
@pytest.mark.parametrize("lengths", [None, [7, 0, 2]])
def test_conv(W, act, lengths):
    gen = torch.Generator().manual_seed(W)
    B, T, D = 3, 7, 5
    n = None if lengths is None else torch.tensor(lengths)
    a = dict(x=rnd(gen, B, T, D), w=rnd(gen, D, W), bias=rnd(gen, D), state=rnd(gen, B, W - 1, D))
    dy, ds = rnd(gen, B, T, D), rnd(gen, B, W - 1, D)

    def f(**k):
        y, s = R.conv(**k, lengths=n, act=act)
        return (y * dy).sum() + (s * ds).sum()

    g = R.conv_grads(**a, dy=dy, dstate_out=ds, lengths=n, act=act)
    check(f, dict(x=g["dx"], w=g["dw"], bias=g["dbias"], state=g["dstate"]), a, gen)


@pytest.mark.parametrize("N,G,gate,sp", [(1, 1, True, True), (3, 2, True, False), (4, 1, False, True)])
@pytest.mark.parametrize("lengths", [None, [9, 0, 4]])
def test_scan(N, G, gate, sp, lengths):
    gen = torch.Generator().manual_seed(N)
    B, T, ch = 3, 9, 6
    n = None if lengths is None else torch.tensor(lengths)
    a = dict(u=rnd(gen, B, T, ch), dt=rnd(gen, B, T, ch, std=0.3) + (0 if sp else 0.5),
             A=-torch.rand(ch, N, generator=gen, dtype=R.F64) - 0.1, Bm=rnd(gen, B, T, G * N), Cm=rnd(gen, B, T, G * N),
             D=rnd(gen, ch), dt_bias=rnd(gen, ch, std=0.2), h0=rnd(gen, B, ch, N))
    if gate:
        a["z"] = rnd(gen, B, T, ch)
    dy, dh = rnd(gen, B, T, ch), rnd(gen, B, ch, N)

    def f(**k):
        y, h = R.scan(**k, lengths=n, sp=sp)
        return (y * dy).sum() + (h * dh).sum()

    g = R.scan_grads(**a, dy=dy, dh_last=dh, lengths=n, sp=sp)
    names = dict(u="du", dt="ddt", A="dA", Bm="dB", Cm="dC", D="dD", dt_bias="dbias", h0="dh0", z="dz")
    check(f, {k: g[v] for k, v in names.items() if k in a}, a, gen)


def test_norm():
    gen = torch.Generator().manual_seed(3)
    a = dict(s=rnd(gen, 4, 11), w=rnd(gen, 11))
    dy = rnd(gen, 4, 11)
    dx, dw = R.norm_grads(a["s"], a["w"], dy, 1e-3)
    check(lambda s, w: (R.norm(s, w, 1e-3) * dy).sum(), dict(s=dx, w=dw), a, gen)
