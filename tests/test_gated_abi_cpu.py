"""The gated block's entry points without a GPU: bad arguments are refused
before any HIP call, by the library and by the binding."""
import ctypes as C

import pytest
import torch

from nonlinear_rnn_evaluation_newton_amd import binding as bd

V = C.c_void_p(256)
VIEW = bd.View(256, 4096, 64)
NOVIEW = bd.View(None, 0, 0)
ROWS, NOROWS = bd.Rows(256, 64), bd.Rows(None, 0)
BIG = 1 << 45


def ref(x):
    return None if x is None else C.byref(x)


def gated_inputs(**kw):
    f = dict(x=VIEW, r=VIEW, i=VIEW, decay=256, r_bias=None, i_bias=None, h0=None, lengths=None)
    f.update(kw)
    return bd.GatedInputs(*f.values())


@pytest.mark.parametrize("bad,code", [
    (dict(dtype=9), bd.PR_EINVAL), (dict(B=0), bd.PR_EINVAL), (dict(T=0), bd.PR_EINVAL), (dict(D=-1), bd.PR_EINVAL),
    (dict(T=(1 << 30) + 1), bd.PR_EUNSUPPORTED), (dict(D=(1 << 22) + 1), bd.PR_EUNSUPPORTED),
    (dict(B=1 << 30, T=1 << 30), bd.PR_EUNSUPPORTED)])
def test_gated_problems(bad, code):
    L = bd.lib()
    f = dict(dtype=bd.PR_BF16, B=2, T=64, D=32)
    f.update(bad)
    pb, inp = bd.GatedProblem(*f.values()), gated_inputs()
    assert L.pararnn_gated_workspace_bytes(ref(pb), 1) == 0
    assert L.pararnn_gated_scan(ref(pb), ref(inp), ref(VIEW), None, None, V, BIG, None) == code
    assert L.pararnn_gated_adjoint(ref(pb), ref(inp), V, ref(VIEW), None, ref(bd.GatedGrads()), V, BIG, None) == code
    if "T" not in bad:  # a single token
        assert L.pararnn_gated_step(ref(pb), ref(inp), ref(VIEW), V, 8, None, None) == code
    assert bd.last_error() != ""


def test_gated_arguments():
    L = bd.lib()
    pb = bd.GatedProblem(bd.PR_F32, 2, 640, 32)
    fw, ad = (L.pararnn_gated_workspace_bytes(ref(pb), k) for k in (0, 1))
    assert 0 < fw <= ad

    def scan(inp=gated_inputs(), y=VIEW, n=fw, ws=V):
        return L.pararnn_gated_scan(ref(pb), ref(inp), ref(y), None, None, ws, n, None)

    for k in ("x", "r", "i"):
        assert scan(inp=gated_inputs(**{k: NOVIEW})) == bd.PR_EINVAL, k
    assert scan(inp=gated_inputs(decay=None)) == bd.PR_EINVAL and scan(inp=None) == bd.PR_EINVAL
    assert scan(y=None) == bd.PR_EINVAL and scan(y=NOVIEW) == bd.PR_EINVAL
    far = bd.View(256, 4096, (1 << 22) + 1)
    for v in (far, bd.View(256, 4096, -64)):
        assert scan(inp=gated_inputs(r=v)) == bd.PR_EUNSUPPORTED and scan(y=v) == bd.PR_EUNSUPPORTED
    assert scan(n=fw - 1) == bd.PR_EWORKSPACE and scan(ws=None) == bd.PR_EWORKSPACE
    assert scan(ws=C.c_void_p(264)) == bd.PR_EINVAL

    def adj(states=V, dy=VIEW, gr=bd.GatedGrads(), n=ad):
        return L.pararnn_gated_adjoint(ref(pb), ref(gated_inputs()), states, ref(dy), None, ref(gr), V, n, None)

    assert adj(states=None) == bd.PR_EINVAL and adj(dy=None) == bd.PR_EINVAL and adj(gr=None) == bd.PR_EINVAL
    assert adj(n=ad - 1) == bd.PR_EWORKSPACE
    assert adj(dy=far) == bd.PR_EUNSUPPORTED and adj(gr=bd.GatedGrads(i=far)) == bd.PR_EUNSUPPORTED

    def step(p=pb, inp=gated_inputs(), y=VIEW, state=V, pool=4, slots=None):
        return L.pararnn_gated_step(ref(p), ref(inp), ref(y), state, pool, slots, None)

    assert step(state=None) == bd.PR_EINVAL and step(pool=0) == bd.PR_EINVAL and step(y=None) == bd.PR_EINVAL
    assert step(pool=1) == bd.PR_EINVAL  # two sequences, one state
    assert step(inp=gated_inputs(r=NOVIEW)) == bd.PR_EINVAL
    assert step(p=bd.GatedProblem(bd.PR_F32, 65536, 1, 32)) == bd.PR_EUNSUPPORTED


def test_block_norm_arguments():
    L = bd.lib()
    good = (bd.PR_F32, 64, 8, 1e-5, 1)

    def call(p=good, x=ROWS, z=None, t=ROWS, y=None):
        pb = None if p is None else bd.BlockNormProblem(*p)
        return L.pararnn_block_norm(ref(pb), ref(x), ref(z), None, None, None, None, ref(t), ref(y), None)

    assert call(p=None) == bd.PR_EINVAL and call(x=NOROWS) == bd.PR_EINVAL and call(x=None) == bd.PR_EINVAL
    assert call(t=None) == bd.PR_EINVAL and call(t=NOROWS) == bd.PR_EINVAL
    for p in ((3, 64, 8, 0.0, 1), (0, 0, 8, 0.0, 1), (0, 64, 0, 0.0, 1), (0, 64, 8, -1.0, 1),
              (0, 64, 8, float("nan"), 1), (0, 64, 8, float("inf"), 1)):
        assert call(p=p) == bd.PR_EINVAL, p
    for gate in (0, 3, -1):
        assert call(p=(0, 64, 8, 0.0, gate), z=ROWS) == bd.PR_EINVAL, gate
    assert call(p=(0, 64, 1 << 31, 0.0, 1)) == bd.PR_EUNSUPPORTED
    pb = bd.BlockNormProblem(*good)
    ws = L.pararnn_block_norm_workspace_bytes(ref(pb))
    assert ws > 0 and L.pararnn_block_norm_workspace_bytes(ref(bd.BlockNormProblem(0, 64, 0, 0.0, 1))) == 0

    def adj(x=ROWS, z=None, t=ROWS, dt=ROWS, dy=ROWS, gr=bd.BlockNormGrads(), w=V, n=ws):
        return L.pararnn_block_norm_adjoint(ref(pb), ref(x), ref(z), None, None, None, ref(t), ref(dt), ref(dy),
                                            ref(gr), w, n, None)

    assert adj(x=None) == bd.PR_EINVAL and adj(gr=None) == bd.PR_EINVAL
    assert adj(dt=None, dy=None) == bd.PR_EINVAL and adj(t=None) == bd.PR_EINVAL
    assert adj(gr=bd.BlockNormGrads(z=ROWS)) == bd.PR_EINVAL  # a gradient of a gate that is not there
    assert adj(dy=None, gr=bd.BlockNormGrads(w_next=256)) == bd.PR_EINVAL
    assert adj(n=ws - 1) == bd.PR_EWORKSPACE and adj(w=None) == bd.PR_EWORKSPACE
    assert adj(w=C.c_void_p(300)) == bd.PR_EINVAL


def test_four_bit_arguments():
    L = bd.lib()

    def gemm(dtype=0, M=8, N=64, K=100, group=32, x=V, ldx=100, q=V, ldq=50, scale=V, out=V, ldo=64):
        return L.pararnn_gemm_w4(dtype, M, N, K, group, x, ldx, q, ldq, scale, None, None, out, ldo, None)

    def quant(dtype=0, N=64, K=100, group=32, w=V, ldw=100, q=V, ldq=50, scale=V):
        return L.pararnn_quant_w4(dtype, N, K, group, w, ldw, q, ldq, scale, None, None)

    def dequant(dtype=0, N=64, K=100, group=32, q=V, ldq=50, scale=V, w=V, ldw=100):
        return L.pararnn_dequant_w4(dtype, N, K, group, q, ldq, scale, None, w, ldw, None)

    for k in ("x", "q", "scale", "out"):
        assert gemm(**{k: None}) == bd.PR_EINVAL, k
    for f in (gemm, quant, dequant):
        assert f(dtype=4) == bd.PR_EINVAL and f(N=0) == bd.PR_EINVAL and f(K=-1) == bd.PR_EINVAL
        assert f(group=0) == bd.PR_EINVAL and f(group=-32) == bd.PR_EINVAL and f(ldq=49) == bd.PR_EINVAL
        for g in (1, 16, 48, 100):
            assert f(group=g) == bd.PR_EUNSUPPORTED, g
        assert f(N=(1 << 24) + 1) == bd.PR_EUNSUPPORTED
        assert f(q=None) == bd.PR_EINVAL and f(scale=None) == bd.PR_EINVAL
    assert gemm(M=0) == bd.PR_EINVAL and gemm(ldx=99) == bd.PR_EINVAL and gemm(ldo=63) == bd.PR_EINVAL
    assert gemm(M=(1 << 21) + 1) == bd.PR_EUNSUPPORTED
    assert gemm(M=1 << 21, N=1 << 24, ldo=1 << 24) == bd.PR_EUNSUPPORTED
    assert quant(w=None) == bd.PR_EINVAL and dequant(w=None) == bd.PR_EINVAL and dequant(ldw=99) == bd.PR_EINVAL


def test_packed_structures_have_the_header_layout():
    """The binding packs these as bytes; ctypes lays the same fields out by the C rules."""
    view, rows = [7, 8, 9], [5, 6]
    for cls, pack, v in ((bd.GatedProblem, bd._PACK_GATED, [1, 2, 3, 4]), (bd.View, bd._PACK_VIEW, view),
                         (bd.Rows, bd._PACK_ROWS, rows), (bd.BlockNormProblem, bd._PACK_BLOCK_NORM, [1, 2, 3, 0.5, 4])):
        assert pack(*v) == bytes(cls(*v)), cls
    V3, R2 = bd.View(*view), bd.Rows(*rows)
    assert bd._PACK_GATED_IN(*view * 3, 1, 2, 3, 4, 5) == bytes(bd.GatedInputs(V3, V3, V3, 1, 2, 3, 4, 5))
    assert bd._PACK_GATED_GRADS(*view * 3, 1, 2, 3, 4) == bytes(bd.GatedGrads(V3, V3, V3, 1, 2, 3, 4))
    assert bd._PACK_BLOCK_NORM_GRADS(*rows * 3, 1, 2, 3) == bytes(bd.BlockNormGrads(R2, R2, R2, 1, 2, 3))


def test_binding_refuses_what_the_library_cannot_see():
    x, z = torch.zeros(2, 8, 16), torch.zeros(2, 16)
    f16, ws = torch.zeros(16), torch.empty(1 << 10, dtype=torch.uint8)
    with pytest.raises(ValueError, match="on the GPU"):
        bd.gated_scan(x, x, x, f16, torch.zeros_like(x), ws)
    with pytest.raises(ValueError, match="storage"):
        bd.gated_scan(x.half(), x.half(), x.half(), f16, x.half(), ws)
    with pytest.raises(ValueError, match=r"gated_scan: x must be \[B, T, channels\]"):
        bd.gated_scan(z, z, z, f16, z, ws)
    with pytest.raises(ValueError, match=r"gated_scan_adjoint: x must be \[B, T, channels\]"):
        bd.gated_scan_adjoint(z, z, z, f16, torch.zeros(2, 1, 16), z, ws)
    with pytest.raises(ValueError, match=r"gated_step: x must be \[B, channels\]"):
        bd.gated_step(x, x, x, f16, torch.zeros(2, 16), x)
    with pytest.raises(ValueError, match="gate must be"):
        bd.block_norm(z, None, z, z=z, gate="relu")
    with pytest.raises(ValueError, match="gate must be"):
        bd.block_norm_adjoint(z, None, z, ws, z=z, gate="gelu", dt=z)
    with pytest.raises(ValueError, match="on the GPU"):
        bd.block_norm(z, None, z)
    q, s = torch.zeros(4, 8, dtype=torch.uint8), torch.zeros(4, 1)
    with pytest.raises(ValueError, match="on the GPU"):
        bd.gemm_w4(z, q, s, torch.zeros(2, 4), 32)
    with pytest.raises(ValueError, match="at least one column"):
        bd._w4("quant_w4", q, s, None, 4, 16, 0, torch.float32)
