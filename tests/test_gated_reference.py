"""The 64-bit gradients that the GPU tests compare with, against central
differences of the 64-bit forward forms (CPU).

A central difference with step h has an error of h^2 / 6 times the third
derivative plus 2^-53 |f| / h; at h = 1e-5 and values of order 1 to 100 both
are below 1e-9, so 1e-6 of the gradient's size leaves room for the third
derivative and for long sums."""
import pytest
import torch

import gated_reference as R

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


@pytest.mark.parametrize("lengths", [None, [9, 0, 4]])
def test_gated(lengths):
    gen = torch.Generator().manual_seed(3)
    B, T, D = 3, 9, 5
    n = None if lengths is None else torch.tensor(lengths)
    a = dict(x=rnd(gen, B, T, D), r=rnd(gen, B, T, D), i=rnd(gen, B, T, D),
             decay=torch.rand(D, generator=gen, dtype=R.F64) + 0.1, r_bias=rnd(gen, D), i_bias=rnd(gen, D),
             h0=rnd(gen, B, D))
    dy, dh = rnd(gen, B, T, D), rnd(gen, B, D)

    def f(**k):
        y, h = R.gated(**k, lengths=n)
        return (y * dy).sum() + (h * dh).sum()

    g = R.gated_grads(**a, dy=dy, lengths=n, dh_last=dh)
    check(f, {k: g["d" + k] for k in a}, a, gen)


@pytest.mark.parametrize("gate", [None, "silu", "sigmoid"])
@pytest.mark.parametrize("join", [True, False])
def test_block_norm(gate, join):
    gen = torch.Generator().manual_seed(5)
    rows, n = 4, 7
    a = dict(x=rnd(gen, rows, n), w=rnd(gen, n))
    if gate:
        a["z"] = rnd(gen, rows, n)
    if join:
        a.update(res=rnd(gen, rows, n), scale=rnd(gen, n), w_next=rnd(gen, n))
    dt, dy = rnd(gen, rows, n), rnd(gen, rows, n) if join else None

    def t_of(x, w, z=None, res=None, scale=None, w_next=None):
        return R.block_norm(x, w, z, gate, scale, res)

    def f(**k):
        t = t_of(**k)
        return (t * dt).sum() + ((R.norm_next(t, k["w_next"]) * dy).sum() if join else 0)

    g = R.block_norm_grads(a["x"], a["w"], a.get("z"), gate, a.get("scale"), a.get("w_next"), t_of(**a), dt, dy)
    check(f, {k: g["d" + k] for k in a}, a, gen)


def test_four_bits_there_and_back():
    """Every number is off by half a step at most, and the ends of a group are kept."""
    gen = torch.Generator().manual_seed(7)
    w = rnd(gen, 5, 77).float()
    for zero in (False, True):
        q, s, z = R.quant(w, 32, zero)
        packed = torch.nn.functional.pad(q, (0, 1))
        packed = packed[:, ::2] | (packed[:, 1::2] << 4)
        back = R.weights(packed, s, 77, 32, z if zero else None)
        step = s.double().repeat_interleave(32, 1)[:, :77]
        assert float(((back - w).abs() / step).max()) <= (1.0 if zero else 0.5) + 1e-5
        assert int(q.max()) == 15 and int(q.min()) <= 1
