"""The selective block's entry points without a GPU: bad arguments are refused
before any HIP call, by the library and by the binding."""
import ctypes as C

import pytest
import torch

from nonlinear_rnn_evaluation_newton_amd import binding as bd

V = C.c_void_p(256)
VIEW = bd.View(256, 4096, 64)
NOVIEW = bd.View(None, 0, 0)
BIG = 1 << 40


def ref(x):
    return None if x is None else C.byref(x)


def ssm_inputs(**kw):
    f = dict(u=VIEW, dt=VIEW, z=NOVIEW, B=VIEW, C=VIEW, A=256, D=None, dt_bias=None, h0=None, lengths=None)
    f.update(kw)
    return bd.SsmInputs(*f.values())


@pytest.mark.parametrize("bad,code", [
    (dict(dtype=9), bd.PR_EINVAL), (dict(B=0), bd.PR_EINVAL), (dict(T=0), bd.PR_EINVAL), (dict(D=-1), bd.PR_EINVAL),
    (dict(W=0), bd.PR_EINVAL), (dict(W=5), bd.PR_EUNSUPPORTED), (dict(T=(1 << 30) + 1), bd.PR_EUNSUPPORTED),
    (dict(B=1 << 30, T=1 << 30), bd.PR_EUNSUPPORTED)])
def test_conv_problems(bad, code):
    L = bd.lib()
    f = dict(dtype=bd.PR_BF16, B=2, T=64, D=32, W=4, silu=1)
    f.update(bad)
    pb = bd.ConvProblem(*f.values())
    assert L.pararnn_conv(ref(pb), ref(VIEW), V, None, None, None, ref(VIEW), None, None) == code
    if "B" not in bad or bad["B"] == 0:
        assert L.pararnn_conv_workspace_bytes(ref(pb)) == 0
    assert bd.last_error() != ""


def test_conv_arguments():
    L = bd.lib()
    pb = bd.ConvProblem(bd.PR_F32, 2, 64, 32, 4, 1)
    ws = L.pararnn_conv_workspace_bytes(ref(pb))
    assert ws > 0

    def fwd(p=pb, x=VIEW, w=V, y=VIEW):
        return L.pararnn_conv(ref(p), ref(x), w, None, None, None, ref(y), None, None)

    for k in ("p", "x", "w", "y"):
        assert fwd(**{k: None}) == bd.PR_EINVAL, k
    assert fwd(x=NOVIEW) == bd.PR_EINVAL

    def adj(dy=VIEW, ws_p=V, n=ws):
        return L.pararnn_conv_adjoint(ref(pb), ref(VIEW), V, None, None, None, ref(dy), None, None, V, V, None, ws_p,
                                      n, None)

    assert adj(dy=None) == bd.PR_EINVAL
    assert adj(n=ws - 1) == bd.PR_EWORKSPACE and adj(ws_p=None) == bd.PR_EWORKSPACE
    assert adj(ws_p=C.c_void_p(264)) == bd.PR_EINVAL

    def step(state=V, slots=V, pool=4, p=pb):
        return L.pararnn_conv_step(ref(p), ref(VIEW), V, None, state, pool, slots, ref(VIEW), None)

    assert step(state=None) == bd.PR_EINVAL and step(pool=0) == bd.PR_EINVAL
    assert step(slots=None, pool=1) == bd.PR_EINVAL  # two sequences, one state
    assert step(p=bd.ConvProblem(bd.PR_F32, 65536, 1, 32, 4, 1)) == bd.PR_EUNSUPPORTED


@pytest.mark.parametrize("bad,code", [
    (dict(dtype=2), bd.PR_EINVAL), (dict(B=0), bd.PR_EINVAL), (dict(T=-4), bd.PR_EINVAL), (dict(D=0), bd.PR_EINVAL),
    (dict(N=0), bd.PR_EINVAL), (dict(G=0), bd.PR_EINVAL), (dict(G=5), bd.PR_EINVAL), (dict(N=65), bd.PR_EUNSUPPORTED),
    (dict(T=(1 << 30) + 1), bd.PR_EUNSUPPORTED), (dict(B=1 << 26), bd.PR_EUNSUPPORTED)])
def test_scan_problems(bad, code):
    L = bd.lib()
    f = dict(dtype=bd.PR_BF16, B=2, T=64, D=32, N=16, G=1, softplus=1)
    f.update(bad)
    pb = bd.SsmProblem(*f.values())
    inp = ssm_inputs()
    assert L.pararnn_ssm_workspace_bytes(ref(pb), 1) == 0
    assert L.pararnn_ssm_scan(ref(pb), ref(inp), ref(VIEW), None, None, V, BIG, None) == code
    assert L.pararnn_ssm_adjoint(ref(pb), ref(inp), V, ref(VIEW), None, ref(bd.SsmGrads()), V, BIG, None) == code
    assert L.pararnn_ssm_step(ref(pb), ref(inp), ref(VIEW), V, 8, None, None) == code
    assert bd.last_error() != ""


def test_scan_arguments():
    L = bd.lib()
    pb = bd.SsmProblem(bd.PR_F32, 2, 64, 32, 16, 2, 1)
    fw, ad = (L.pararnn_ssm_workspace_bytes(ref(pb), k) for k in (0, 1))
    assert 0 < fw <= ad

    def scan(inp=ssm_inputs(), y=VIEW, n=fw, ws=V, hl=None):
        return L.pararnn_ssm_scan(ref(pb), ref(inp), ref(y), hl, None, ws, n, None)

    for k in ("u", "dt", "B", "C"):
        assert scan(inp=ssm_inputs(**{k: NOVIEW})) == bd.PR_EINVAL, k
    assert scan(inp=ssm_inputs(A=None)) == bd.PR_EINVAL and scan(inp=None) == bd.PR_EINVAL
    assert scan(y=None) == bd.PR_EINVAL and scan(y=NOVIEW) == bd.PR_EINVAL
    assert scan(n=fw - 1) == bd.PR_EWORKSPACE and scan(ws=None) == bd.PR_EWORKSPACE
    assert scan(ws=C.c_void_p(264)) == bd.PR_EINVAL
    assert scan(inp=ssm_inputs(A=260)) == bd.PR_EINVAL and scan(hl=C.c_void_p(260)) == bd.PR_EINVAL  # alignment

    def adj(states=V, dy=VIEW, gr=bd.SsmGrads(), n=ad):
        return L.pararnn_ssm_adjoint(ref(pb), ref(ssm_inputs()), states, ref(dy), None, ref(gr), V, n, None)

    assert adj(states=None) == bd.PR_EINVAL and adj(dy=None) == bd.PR_EINVAL and adj(gr=None) == bd.PR_EINVAL
    assert adj(gr=bd.SsmGrads(z=VIEW)) == bd.PR_EINVAL  # a gradient of a gate that is not there
    assert adj(n=ad - 1) == bd.PR_EWORKSPACE
    inp = ssm_inputs()
    step = L.pararnn_ssm_step
    assert step(ref(pb), ref(inp), ref(VIEW), None, 4, None, None) == bd.PR_EINVAL
    assert step(ref(pb), ref(inp), ref(VIEW), V, 1, None, None) == bd.PR_EINVAL
    assert step(ref(pb), ref(inp), ref(VIEW), C.c_void_p(264), 4, None, None) == bd.PR_EINVAL


def test_norm_arguments():
    L = bd.lib()
    rows, none = bd.Rows(256, 64), bd.Rows(None, 0)

    def call(p=bd.NormProblem(bd.PR_F32, 64, 8, 1e-5), x=rows, y=rows, q=None, scale=None):
        return L.pararnn_rmsnorm(ref(p), ref(x), None, None, None, ref(y), ref(q), scale, None)

    assert call(p=None) == bd.PR_EINVAL and call(x=none) == bd.PR_EINVAL
    assert call(y=None) == bd.PR_EINVAL and call(q=rows, scale=V) == bd.PR_EINVAL  # exactly one output form
    assert call(y=None, q=rows) == bd.PR_EINVAL
    for p in ((3, 64, 8, 0.0), (0, 0, 8, 0.0), (0, 64, 0, 0.0), (0, 64, 8, -1.0), (0, 64, 8, float("nan")),
              (0, 64, 8, float("inf"))):
        assert call(p=bd.NormProblem(*p)) == bd.PR_EINVAL, p
    assert call(p=bd.NormProblem(0, 64, 1 << 31, 0.0)) == bd.PR_EUNSUPPORTED
    pb = bd.NormProblem(bd.PR_F32, 64, 8, 1e-5)
    assert L.pararnn_quant_rows(ref(pb), ref(rows), None, V, None) == bd.PR_EINVAL
    assert L.pararnn_quant_rows(ref(pb), ref(rows), ref(rows), None, None) == bd.PR_EINVAL
    ws = L.pararnn_rmsnorm_workspace_bytes(ref(pb))

    def adj(s=rows, dy=rows, n=ws, w=V):
        return L.pararnn_rmsnorm_adjoint(ref(pb), ref(s), None, ref(dy), None, None, V, w, n, None)

    assert ws > 0 and adj(s=None) == bd.PR_EINVAL and adj(dy=None) == bd.PR_EINVAL
    assert adj(n=ws - 1) == bd.PR_EWORKSPACE and adj(w=C.c_void_p(300)) == bd.PR_EINVAL


def test_product_arguments():
    L = bd.lib()
    ws = bd.gemm_i8_workspace_bytes(100, 200, 300)
    assert ws > 0
    for mnk in ((0, 1, 1), (1, 0, 1), (1, 1, -2), (1, 1, 131072)):
        assert bd.gemm_i8_workspace_bytes(*mnk) == 0

    def call(dtype=0, M=100, N=200, K=300, a=V, lda=300, sa=V, w=V, ldw=300, sw=V, out=V, ldo=200, wsp=V, n=ws):
        return L.pararnn_gemm_i8(dtype, M, N, K, a, lda, sa, w, ldw, sw, None, out, ldo, wsp, n, None)

    for k in ("a", "sa", "w", "sw", "out"):
        assert call(**{k: None}) == bd.PR_EINVAL, k
    assert call(dtype=5) == bd.PR_EINVAL and call(M=0) == bd.PR_EINVAL
    assert call(K=131072, lda=131072, ldw=131072) == bd.PR_EUNSUPPORTED
    assert call(lda=299) == bd.PR_EINVAL and call(ldw=1) == bd.PR_EINVAL and call(ldo=199) == bd.PR_EINVAL
    assert call(n=ws - 1) == bd.PR_EWORKSPACE and call(wsp=C.c_void_p(264)) == bd.PR_EINVAL


def test_binding_refuses_what_the_library_cannot_see():
    """Types, shapes and devices of tensors are checked in Python."""
    x, w = torch.zeros(2, 8, 16), torch.zeros(16, 4)
    ws = torch.empty(1 << 20, dtype=torch.uint8)
    with pytest.raises(ValueError, match="on the GPU"):
        bd.conv(x, w, None, torch.zeros_like(x))
    with pytest.raises(ValueError, match="storage"):
        bd.conv(x.half(), w.half(), None, torch.zeros_like(x.half()))
    with pytest.raises(ValueError, match="int32|int64"):
        bd._dense("f", "lengths", torch.zeros(2, dtype=torch.int64), (2,), torch.int32)
    with pytest.raises(ValueError, match="multiple"):
        bd.ssm_scan(x, x, torch.zeros(16, 5), torch.zeros(2, 8, 16), torch.zeros(2, 8, 16), x, ws)
    with pytest.raises(ValueError, match="shape"):
        bd._need("f", "w", torch.zeros(3, 7), (3, 8), torch.float32)
    with pytest.raises(ValueError, match="contiguous"):
        bd._strides("f", "w", torch.zeros(8, 3).t(), (3, 8), 1)


def test_workspace_is_checked_in_python():
    """Kernels write through the workspace's address: one in host memory, or
    one whose bytes are not all its own, is refused."""
    with pytest.raises(ValueError, match="ssm_scan: the workspace must be on the GPU"):
        bd._ws("ssm_scan", torch.empty(1 << 10, dtype=torch.uint8))
    with pytest.raises(ValueError, match="contiguous"):
        bd._ws("ssm_scan", torch.empty(1, dtype=torch.uint8).expand(1 << 20))
    with pytest.raises(ValueError, match="contiguous"):
        bd._ws("ssm_scan", torch.empty(64, 64, dtype=torch.uint8)[:, ::2])


def test_scan_takes_sequences_and_its_step_takes_tokens():
    """Sequences given to the step would have had their first token computed and
    the rest of y left as it was; a batch of tokens given to the scan is not one sequence."""
    A, seq, tok, ws = torch.zeros(16, 8), torch.zeros(2, 5, 16), torch.zeros(2, 16), torch.empty(1 << 10, dtype=torch.uint8)
    bc, bt = torch.zeros(2, 5, 8), torch.zeros(2, 8)
    with pytest.raises(ValueError, match=r"ssm_step: u must be \[B, channels\]"):
        bd.ssm_step(seq, seq, A, bc, bc, torch.zeros(2, 16, 8), seq)
    with pytest.raises(ValueError, match=r"ssm_scan: u must be \[B, T, channels\]"):
        bd.ssm_scan(tok, tok, A, bt, bt, tok, ws)
    with pytest.raises(ValueError, match=r"ssm_scan_adjoint: u must be \[B, T, channels\]"):
        bd.ssm_scan_adjoint(tok, tok, A, bt, bt, torch.zeros(2, 1, 16, 8), tok, ws)


class OnGpu:
    """Stands for a contiguous tensor on GPU `at`, of which the checks only look at this."""

    def __init__(self, t, at):
        self.t, self.at, self.is_cuda, self.dtype, self.shape = t, at, True, t.dtype, t.shape

    def get_device(self):
        return self.at

    def __getattr__(self, name):
        return getattr(self.t, name)


@pytest.mark.parametrize("what", ["_need", "_dense", "_ws"])
def test_tensors_of_another_gpu_are_refused(what, monkeypatch):
    """With several GPUs, a tensor of one that is not current would be reached
    from the current one, or launched on the wrong stream."""
    bd.lib()
    monkeypatch.setattr(bd, "_several_gpus", True)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    t = torch.zeros(4, 8)

    def call(at):
        x = OnGpu(t, at)
        return bd._ws("f", x) if what == "_ws" else getattr(bd, what)("f", "x", x, (4, 8), torch.float32)

    with pytest.raises(ValueError, match="is on GPU 0, the current one is 1"):
        call(0)
    got = call(1)
    assert got == ((t.data_ptr(), 128) if what == "_ws" else t.data_ptr())


def test_scan_time_strides():
    """Strides that 16 steps and the tiles fetched ahead cannot be reached with, and negative ones, are refused."""
    L = bd.lib()
    for dtype, most in ((bd.PR_F32, 2147483000 // (144 * 4)), (bd.PR_BF16, 2147483000 // (144 * 2))):
        pb = bd.SsmProblem(dtype, 2, 64, 32, 16, 2, 1)
        fw, ad = (L.pararnn_ssm_workspace_bytes(ref(pb), k) for k in (0, 1))
        for st in (most + 1, 1 << 40, -32):
            far = bd.View(256, 64, st)
            for k in ("u", "dt", "z", "B", "C"):
                assert L.pararnn_ssm_scan(ref(pb), ref(ssm_inputs(**{k: far})), ref(VIEW), None, None, V, fw,
                                          None) == bd.PR_EUNSUPPORTED, (k, st)
            assert L.pararnn_ssm_scan(ref(pb), ref(ssm_inputs()), ref(far), None, None, V, fw, None) == bd.PR_EUNSUPPORTED
            for k in ("u", "dt", "z"):
                gr = bd.SsmGrads(**{k: far})
                assert L.pararnn_ssm_adjoint(ref(pb), ref(ssm_inputs(z=VIEW)), V, ref(VIEW), None, ref(gr), V, ad,
                                             None) == bd.PR_EUNSUPPORTED, (k, st)
        assert "stride" in bd.last_error()


def test_scan_launches_that_no_grid_takes():
    """One grid dimension takes 2^32 threads: 2^23 blocks of channels of all sequences are refused."""
    L = bd.lib()

    def size(B, D, G=1):
        return L.pararnn_ssm_workspace_bytes(ref(bd.SsmProblem(bd.PR_BF16, B, 16, D, 16, G, 1)), 0)

    assert size(1 << 18, 31 * 64) > 0 and size(1 << 18, 31, 31) > 0
    assert size(1 << 18, 32 * 64) == 0 and size(1 << 18, 32, 32) == 0
    assert "blocks" in bd.last_error()


def test_products_that_no_grid_takes():
    """A launch has 2^32 threads at most; more were cut without an error: few
    rows of 2^27 columns, and more of them where there are 2^24 tiles of 128 x 128."""
    size = bd.gemm_i8_workspace_bytes
    assert size(64, (1 << 27) - 16, 16) > 0 and size(1 << 20, (1 << 18) - 128, 16) > 0
    for M, N in ((64, (1 << 27) - 15), (1, 1 << 30), (1 << 20, 1 << 18), (1 << 30, 1 << 18)):
        assert size(M, N, 16) == 0 and "large" in bd.last_error(), (M, N)
    assert size(100, (1 << 30) + 1, 16) == 0 and size((1 << 31) - 1, 1, 16) == 0
