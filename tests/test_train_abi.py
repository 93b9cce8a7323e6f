"""CPU checks of the training operators: refusals before any device work, sizes, the binding's argument checks,
and the float64 references themselves (gradients against central differences)."""
import ctypes
import os

import pytest
import torch

import train_ref as R


@pytest.fixture(scope="module")
def M():
    import moe_expert_ffn_sqrt_gb300 as M
    if not os.path.exists(M.LIB_PATH):
        from moe_expert_ffn_sqrt_gb300 import build
        build.build()
    M.lib()
    return M


P = ctypes.c_void_p(0x10000)      # never dereferenced: validation fails first
ODD = ctypes.c_void_p(0x10008)
BIG = 1 << 40


def rows(M, ld, ptr=0x10000):
    return M._Rows(ptr, ld)


def test_workspace_sizes(M):
    n = ctypes.c_size_t(0)
    L = M.lib()
    assert M.workspace_size_rows(8, 6, 256) >= 256
    assert M.workspace_size_rows(16384, 6, 256) > M.workspace_size_rows(8, 6, 256)
    for T, K, E in ((-1, 2, 4), (4, 0, 4), (4, 5, 4), (4, 33, 64), (1 << 28, 32, 64)):
        assert L.moe_workspace_size_rows(T, K, E, ctypes.byref(n)) == M.ERR_INVALID_ARG
    assert L.moe_workspace_size_rows(4, 2, 4, None) == M.ERR_INVALID_ARG
    # dz is kept in the workspace only where there is an activation
    assert M.workspace_size_linear(4096, 2048, 512, 0, "silu") >= M.workspace_size_linear(4096, 2048, 512, 0, "none") + 4096 * 2048 * 2
    for a in ((-1, 64, 64, 0, 0), (4, 0, 64, 0, 0), (4, 63, 64, 0, 0), (4, 64, 60, 0, 0), (4, 64, 64, 1025, 0), (4, 64, 64, 0, 5),
              (4, 72, 64, 0, 4), (4, 64, 64, -1, 0)):
        assert L.moe_workspace_size_linear(*a, ctypes.byref(n)) == M.ERR_INVALID_ARG, a


def test_dispatch_refusals(M):
    L = M.lib()

    def call(dt=0, ids=P, x=None, T=4, H=64, E=8, K=2, align=16, xp=None, inv=P, ws=P, n=BIG):
        return L.moe_dispatch(dt, ids, x or rows(M, 64), T, H, E, K, align, xp or rows(M, 64), P, P, inv, P, None, ws, n, None)

    assert call(dt=3) == M.ERR_INVALID_ARG
    assert call(align=3) == M.ERR_INVALID_ARG and call(align=512) == M.ERR_INVALID_ARG
    assert call(K=9) == M.ERR_INVALID_ARG and call(K=0) == M.ERR_INVALID_ARG and call(T=-1) == M.ERR_INVALID_ARG
    assert call(H=0) == M.ERR_INVALID_ARG
    assert call(E=2000) == M.ERR_UNSUPPORTED
    assert call(x=rows(M, 63)) == M.ERR_INVALID_ARG            # rows that overlap
    assert call(x=rows(M, 64, 0x10001)) == M.ERR_INVALID_ARG   # not element-aligned
    assert call(xp=rows(M, 64, None)) == M.ERR_INVALID_ARG
    assert call(ids=None) == M.ERR_INVALID_ARG and call(inv=None) == M.ERR_INVALID_ARG
    assert call(ws=None) == M.ERR_WORKSPACE and call(n=100) == M.ERR_WORKSPACE


def test_combine_refusals(M):
    L = M.lib()
    none = rows(M, 0, None)

    def fwd(dt=2, y=None, inv=P, res=none, T=4, H=64, K=2, U=16, out=None, ws=P, n=256):
        return L.moe_combine(dt, y or rows(M, 64), inv, P, res, T, H, K, U, out or rows(M, 64), ws, n, None)

    assert fwd(dt=-1) == M.ERR_INVALID_ARG and fwd(K=33) == M.ERR_INVALID_ARG and fwd(U=-1) == M.ERR_INVALID_ARG
    assert fwd(inv=None) == M.ERR_INVALID_ARG and fwd(res=rows(M, 10)) == M.ERR_INVALID_ARG
    assert fwd(out=rows(M, 64, 0x10002)) == M.ERR_INVALID_ARG
    assert fwd(ws=None) == M.ERR_WORKSPACE and fwd(n=255) == M.ERR_WORKSPACE
    assert L.moe_dispatch_backward(0, rows(M, 8), P, none, 4, 64, 2, 16, rows(M, 64), P, 256, None) == M.ERR_INVALID_ARG

    def bwd(y=None, w=P, dw=P, dy=None):
        return L.moe_combine_backward(0, rows(M, 64), y or rows(M, 64), P, w, 4, 64, 2, 16, dy or rows(M, 64), dw, P, 255, None)

    assert bwd(dw=None) == M.ERR_INVALID_ARG and bwd(y=none) == M.ERR_INVALID_ARG      # both or neither
    assert bwd(w=None) == M.ERR_INVALID_ARG                                            # a plain sum has no weight gradient
    assert bwd(dy=none) == M.ERR_INVALID_ARG
    assert bwd() == M.ERR_WORKSPACE


def test_route_backward_refusals(M):
    L = M.lib()

    def call(l=P, T=4, E=8, K=2, fn=0, dt=2, d=P, n=256):
        return L.moe_route_backward(l, P, P, P, T, E, K, fn, 1, dt, d, P, n, None)

    assert call(fn=2) == M.ERR_INVALID_ARG and call(K=9) == M.ERR_INVALID_ARG and call(E=1025) == M.ERR_INVALID_ARG
    assert call(dt=7) == M.ERR_INVALID_ARG and call(l=None) == M.ERR_INVALID_ARG and call(d=ODD) == M.ERR_INVALID_ARG
    assert call(n=10) == M.ERR_WORKSPACE


def test_linear_refusals(M):
    L = M.lib()
    none = rows(M, 0, None)

    def fwd(dt=0, x=None, w=P, bias=None, res=none, act=0, counts=None, m=4, N=64, K=64, E=0, align=0, y=None, z=none, ws=P, n=256):
        return L.moe_linear(dt, x or rows(M, 64), w, bias, res, act, counts, m, N, K, E, align, y or rows(M, 64), z, ws, n, None)

    assert fwd(dt=2) == M.ERR_UNSUPPORTED
    assert fwd(dt=9) == M.ERR_INVALID_ARG and fwd(act=5) == M.ERR_INVALID_ARG and fwd(act=-1) == M.ERR_INVALID_ARG
    assert fwd(N=60) == M.ERR_INVALID_ARG and fwd(K=4) == M.ERR_INVALID_ARG and fwd(N=72, act=4, y=rows(M, 72)) == M.ERR_INVALID_ARG
    assert fwd(E=4) == M.ERR_INVALID_ARG and fwd(counts=P) == M.ERR_INVALID_ARG          # counts and experts go together
    assert fwd(E=4, counts=P, align=3) == M.ERR_INVALID_ARG and fwd(E=1025, counts=P, align=1) == M.ERR_INVALID_ARG
    assert fwd(x=rows(M, 68)) == M.ERR_INVALID_ARG and fwd(x=rows(M, 64, 0x10008)) == M.ERR_INVALID_ARG
    assert fwd(x=rows(M, 56)) == M.ERR_INVALID_ARG and fwd(y=none) == M.ERR_INVALID_ARG and fwd(w=ODD) == M.ERR_INVALID_ARG
    assert fwd(res=rows(M, 60)) == M.ERR_INVALID_ARG and fwd(z=rows(M, 8)) == M.ERR_INVALID_ARG and fwd(bias=ODD) == M.ERR_INVALID_ARG
    assert fwd(m=-1) == M.ERR_INVALID_ARG
    assert fwd(ws=None) == M.ERR_WORKSPACE and fwd(n=0) == M.ERR_WORKSPACE
    assert fwd(m=0) == M.OK

    def bwd(dy=None, x=None, w=P, z=none, act=0, res=none, dx=None, dw=P, db=None, n=BIG):
        return L.moe_linear_backward(0, dy or rows(M, 64), x or rows(M, 64), w, z, act, None, 4, 64, 64, 0, 0, res,
                                     dx or rows(M, 64), dw, db, P, n, None)

    assert bwd(dx=none, dw=None) == M.ERR_INVALID_ARG                      # nothing asked for
    assert bwd(act=2) == M.ERR_INVALID_ARG and bwd(z=rows(M, 64)) == M.ERR_INVALID_ARG     # z with, and only with, an activation
    assert bwd(w=None) == M.ERR_INVALID_ARG and bwd(x=none) == M.ERR_INVALID_ARG
    assert bwd(dx=none, res=rows(M, 64)) == M.ERR_INVALID_ARG and bwd(dw=ODD) == M.ERR_INVALID_ARG and bwd(db=ODD) == M.ERR_INVALID_ARG
    assert bwd(n=300) == M.ERR_WORKSPACE
    # the dense call's workspace is enough for it, one byte less is not
    assert bwd(n=M.workspace_size_linear(4, 64, 64) - 1) == M.ERR_WORKSPACE


def test_the_binding_checks_its_arguments(M):
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        M._rows(x, torch.bfloat16, (4, 64), "x")
    assert M._rows(None, torch.bfloat16, (4, 64), "x").ptr is None
    with pytest.raises(TypeError, match="torch.Tensor"):
        M._rows([1], torch.bfloat16, (4, 64), "x")
    with pytest.raises(TypeError, match="bfloat16, float16 or float32"):
        M._dtype(torch.zeros(1, dtype=torch.int32), "x")
    with pytest.raises(ValueError, match="CUDA tensor"):
        M._full(torch.zeros(3), torch.float32, (4,), "bias")
    with pytest.raises(ValueError, match="w must have shape"):
        M._linear_dims(x, torch.zeros(2, 8, 64), "none", None)


# ------------------------------------------------------------------------------------- the references

def central(f, v, d, h):
    return (f(v + h * d) - f(v - h * d)) / (2 * h)


@pytest.mark.parametrize("fn", ["softmax", "sqrt_softplus"])
@pytest.mark.parametrize("renorm", [True, False])
def test_reference_route_gradient_against_differences(fn, renorm):
    g = torch.Generator().manual_seed(5)
    l = torch.randn(9, 12, generator=g, dtype=R.F64)
    ids = torch.rand(9, 12, generator=g).topk(3, 1).indices
    c, d = torch.randn(9, 3, generator=g, dtype=R.F64), torch.randn(9, 12, generator=g, dtype=R.F64)
    num = central(lambda v: (R.route_weights(v, ids, fn, renorm) * c).sum(), l, d, 1e-5)
    # truncation h^2 times third derivatives of order one, rounding 1e-16 / h: far below 1e-7
    assert abs(float(num - (R.route_grad(l, ids, c, fn, renorm) * d).sum())) < 1e-7


@pytest.mark.parametrize("act", ["none", "silu", "gelu", "swiglu", "relu"])
def test_reference_linear_gradients_against_differences(act):
    g = torch.Generator().manual_seed(6)

    def rnd(*s):
        return torch.randn(*s, generator=g, dtype=R.F64)

    x, w, b = rnd(5, 8), rnd(12, 8), rnd(12)
    c = rnd(5, 6 if act == "swiglu" else 12)

    def f(x_, w_, b_):
        return (R.act(x_ @ w_.t() + b_, act) * c).sum()

    z = x @ w.t() + b
    (dx, _), (dw, _), (db, _) = R.linear_grad(c, x, w, z, act, None, torch.float32)
    assert float(z.abs().min()) > 1e-3           # no relu kink inside the differences
    for v, grad, ff in ((x, dx, lambda v: f(v, w, b)), (w, dw, lambda v: f(x, v, b)), (b, db, lambda v: f(x, w, v))):
        d = rnd(*v.shape)
        assert abs(float(central(ff, v, d, 1e-5) - (grad * d).sum())) < 1e-6
