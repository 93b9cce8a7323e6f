"""CPU checks of the norm, the routing by groups and the 8-bit rows: refusals before any device work, sizes, the
binding's argument checks, and the float64 references themselves."""
import ctypes
import os

import pytest
import torch

import around_ref as A
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


def rows8(M, ldq, lds, q=0x10000, sf=0x20000):
    return M._Rows8(q, sf, ldq, lds)


def test_norm_refusals(M):
    L = M.lib()
    none, none8 = rows(M, 0, None), rows8(M, 0, 0, None, None)

    def fwd(dt=0, x=None, res=none, w=P, eps=1e-6, T=4, H=200, s=none, y=None, y8=none8):
        return L.moe_rms_norm(dt, x or rows(M, 200), res, w, eps, T, H, s, y or rows(M, 200), y8, None)

    bad = M.ERR_INVALID_ARG
    assert fwd(dt=3) == bad and fwd(T=-1) == bad and fwd(H=0) == bad and fwd(H=1 << 25) == bad
    assert fwd(eps=-1.0) == bad and fwd(eps=float("nan")) == bad and fwd(eps=float("inf")) == bad
    assert fwd(x=rows(M, 199)) == bad and fwd(x=rows(M, 200, 0x10001)) == bad and fwd(x=none) == bad
    assert fwd(res=rows(M, 10)) == bad and fwd(s=rows(M, 10)) == bad and fwd(y=rows(M, 10)) == bad
    assert fwd(w=None) == bad and fwd(w=ODD) == bad
    assert fwd(y=none) == bad                                              # no output at all
    assert fwd(s=rows(M, 200, 0x40000), y=rows(M, 200, 0x40000)) == bad    # two outputs in one place
    assert fwd(y8=rows8(M, 199, 2)) == bad and fwd(y8=rows8(M, 200, 1)) == bad
    assert fwd(y8=rows8(M, 200, 2, None)) == bad and fwd(y8=rows8(M, 200, 2, 0x10000, None)) == bad
    assert fwd(T=0, x=none) == M.OK

    def bwd(dt=0, dy=None, x=None, w=P, eps=0.0, ds=none, T=4, dx=None, dw=P, ws=P, n=BIG):
        return L.moe_rms_norm_backward(dt, dy or rows(M, 200), x or rows(M, 200), w, eps, ds, T, 200, dx or rows(M, 200), dw, ws, n, None)

    assert bwd(dt=-1) == bad and bwd(dy=none) == bad and bwd(x=rows(M, 20)) == bad and bwd(w=ODD) == bad and bwd(dw=ODD) == bad
    assert bwd(dx=none, dw=None) == bad and bwd(dx=none, ds=rows(M, 200)) == bad and bwd(eps=-0.5) == bad
    assert bwd(ws=None) == M.ERR_WORKSPACE and bwd(n=M.workspace_size_norm(4, 200) - 1) == M.ERR_WORKSPACE
    assert bwd(T=0, dw=None) == M.OK
    n = ctypes.c_size_t(0)
    for a in ((-1, 4), (4, 0), (4, 1 << 25)):
        assert L.moe_workspace_size_norm(*a, ctypes.byref(n)) == bad
    assert L.moe_workspace_size_norm(4, 4, None) == bad


def test_select_refusals(M):
    L, bad = M.lib(), M.ERR_INVALID_ARG

    def call(dt=2, l=None, T=4, E=64, K=6, fn=2, G=8, KG=4, best=2, scale=1.0, ids=P, w=P):
        return L.moe_select(dt, l or rows(M, 64), None, T, E, K, M._SelectRule(fn, G, KG, best, 1, scale), ids, w, None)

    assert call(dt=4) == bad and call(T=-1) == bad and call(E=0) == bad and call(E=2048, l=rows(M, 2048)) == bad
    assert call(K=0) == bad and call(K=33) == bad and call(K=33, G=1, KG=1) == bad and call(fn=3) == bad and call(fn=-1) == bad
    assert call(G=0) == bad and call(G=7) == bad and call(G=64) == bad and call(KG=0) == bad and call(KG=9) == bad
    assert call(K=9, KG=1) == bad                                      # more experts than the groups have
    assert call(best=0) == bad and call(best=3) == bad
    assert call(scale=0.0) == bad and call(scale=float("nan")) == bad and call(scale=float("inf")) == bad
    assert call(l=rows(M, 63)) == bad and call(l=rows(M, 64, None)) == bad and call(ids=None) == bad and call(w=None) == bad
    assert call(T=0, l=rows(M, 0, None)) == M.OK

    def bwd(dt=2, gdt=2, l=None, E=64, K=6, fn=2, scale=1.0, d=None, w=P, ws=P, n=256):
        return L.moe_select_backward(dt, l or rows(M, 64), P, w, P, 4, E, K, fn, 1, scale, gdt, d or rows(M, 64), ws, n, None)

    assert bwd(dt=5) == bad and bwd(gdt=5) == bad and bwd(K=65) == bad and bwd(E=1025) == bad and bwd(fn=3) == bad
    assert bwd(scale=0.0) == bad and bwd(l=rows(M, 10)) == bad and bwd(d=rows(M, 64, None)) == bad and bwd(w=None) == bad
    assert bwd(dt=0, gdt=2) == M.ERR_UNSUPPORTED and bwd(dt=0, gdt=1) == M.ERR_UNSUPPORTED
    assert bwd(ws=None) == M.ERR_WORKSPACE and bwd(n=255) == M.ERR_WORKSPACE
    # the calls that were there take no sigmoid
    assert L.moe_route(P, P, None, None, 4, 128, 8, 2, 2, 1, None, P, P, None, None, P, BIG, None) == bad
    assert L.moe_route_backward(P, P, P, P, 4, 8, 2, 2, 1, 2, P, P, 256, None) == bad


def test_rows8_refusals(M):
    L, bad = M.lib(), M.ERR_INVALID_ARG
    none, none8 = rows(M, 0, None), rows8(M, 0, 0, None, None)

    def pack(dt=0, x=None, counts=None, n=4, c=200, E=0, align=0, x8=None, ws=None, b=0):
        return L.moe_pack_rows8(dt, x or rows(M, 200), counts, n, c, E, align, x8 or rows8(M, 200, 2), ws, b, None)

    assert pack(dt=3) == bad and pack(n=-1) == bad and pack(c=0) == bad and pack(c=1 << 25) == bad
    assert pack(E=2) == bad and pack(counts=P) == bad and pack(E=-1) == bad
    assert pack(counts=P, E=2, align=3, ws=P, b=256) == bad and pack(counts=P, E=1025, align=1, ws=P, b=256) == bad
    assert pack(x=rows(M, 100)) == bad and pack(x=none) == bad and pack(x8=none8) == bad and pack(x8=rows8(M, 200, 1)) == bad
    assert pack(counts=P, E=2, align=4) == M.ERR_WORKSPACE
    assert pack(n=0, x=none) == M.OK

    def unpack(dt=0, x8=None, ids=None, div=1, src=4, n=4, c=200, x=None, ws=None, b=0):
        return L.moe_unpack_rows8(dt, x8 or rows8(M, 200, 2), ids, div, src, None, n, c, 0, 0, x or rows(M, 200), ws, b, None)

    assert unpack(dt=3) == bad and unpack(n=-1) == bad and unpack(x8=none8) == bad and unpack(x=rows(M, 100)) == bad
    assert unpack(ids=P, div=0, ws=P, b=256) == bad and unpack(ids=P, src=-1, ws=P, b=256) == bad
    assert unpack(ids=P) == M.ERR_WORKSPACE and unpack(ids=P, ws=P, b=255) == M.ERR_WORKSPACE

    def bwd(dt=0, dy=None, x=none, x8=None, ids=None, div=1, src=4, z=none, z8=none8, act=0, dx=None, dw=P, n=BIG, ws=P):
        return L.moe_linear_backward8(dt, dy or rows(M, 64), x, x8 or rows8(M, 64, 1), ids, div, src, P, z, z8, act, None, 4, 64, 64,
                                      0, 0, none, dx or rows(M, 64), dw, None, ws, n, None)

    assert bwd(dt=2) == M.ERR_UNSUPPORTED and bwd(act=5) == bad
    assert bwd(x=rows(M, 64)) == bad and bwd(x8=none8) == bad                        # x or x8, one of them
    assert bwd(x8=rows8(M, 63, 1)) == bad and bwd(x8=rows8(M, 64, 0)) == bad
    assert bwd(ids=P, div=0) == bad and bwd(ids=P, src=-1) == bad and bwd(ids=P, x8=none8, x=rows(M, 64)) == bad
    assert bwd(z8=rows8(M, 64, 1)) == bad                                            # no activation, no z
    assert bwd(act=2) == bad and bwd(act=2, z=rows(M, 64), z8=rows8(M, 64, 1)) == bad and bwd(act=2, z8=rows8(M, 64, 0)) == bad
    assert bwd(ws=None) == M.ERR_WORKSPACE and bwd(n=M.workspace_size_linear8(4, 64, 64) - 1) == M.ERR_WORKSPACE
    n = ctypes.c_size_t(0)
    assert L.moe_workspace_size_linear8(4, 63, 64, 0, 0, ctypes.byref(n)) == bad and L.moe_workspace_size_linear8(4, 64, 64, 0, 0, None) == bad
    assert M.workspace_size_linear8(4096, 64, 512) >= M.workspace_size_linear(4096, 64, 512) + 4096 * 512 * 2


def test_the_binding_checks_its_arguments(M):
    q, s = torch.zeros(4, 200, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8)
    assert M._rows8(None, 4, 200, "y8").q is None
    with pytest.raises(ValueError, match="CUDA tensor"):
        M._rows8((q, s), 4, 200, "y8")
    a, b = M.new_rows8(3, 129, device="cpu")
    assert a.shape == (3, 129) and b.shape == (3, 2)


# ------------------------------------------------------------------------------------- the references

CPU_CALLS = """
import torch
import moe_expert_ffn_sqrt_gb300 as M
x, w, ws = torch.ones(4, 256, dtype=torch.bfloat16), torch.ones(256), torch.zeros(4096, dtype=torch.uint8)
ids, tw, w2, q = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2), torch.ones(256, 256, dtype=torch.bfloat16), M.new_rows8(4, 256, "cpu")
for f in (lambda: M.rms_norm(x, w, 1e-6, y=x), lambda: M.rms_norm_backward(x, x, w, 1e-6, x, ws),
          lambda: M.select(x, ids, tw, "sigmoid"), lambda: M.select_backward(x, ids, tw, tw, x, ws, "sigmoid"),
          lambda: M.pack_rows8(x, q), lambda: M.unpack_rows8(q, x),
          lambda: M.linear_backward8(x, w2, ws, x8=q, dw=w2)):
    try:
        f()
    except Exception:
        continue
    raise SystemExit("not refused")
print("refused all")
"""


def test_tensors_of_the_host_raise(M):
    """Every call with tensors outside a GPU, on a machine without one too: an exception, and the process lives."""
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", CPU_CALLS], cwd=root, capture_output=True, text=True, timeout=300,
                       env={**os.environ, "CUDA_VISIBLE_DEVICES": ""})
    assert r.returncode == 0 and r.stdout.strip() == "refused all", r.stderr[-2000:]


def test_reference_norm_gradient_against_differences():
    g = torch.Generator().manual_seed(5)
    x, d, c = (torch.randn(5, 12, generator=g, dtype=R.F64) for _ in range(3))
    w, v = (torch.randn(12, generator=g, dtype=R.F64) for _ in range(2))
    f = lambda x_, w_: (A.norm(x_, None, w_, 1e-3, R.F64)[1] * c).sum()   # noqa: E731
    (dx, _), (dw, _) = A.norm_grad(c, x, w, 1e-3, None, torch.float32)
    h = 1e-5
    assert abs(float((f(x + h * d, w) - f(x - h * d, w)) / (2 * h) - (dx * d).sum())) < 1e-7
    assert abs(float((f(x, w + h * v) - f(x, w - h * v)) / (2 * h) - (dw * v).sum())) < 1e-7


@pytest.mark.parametrize("fn", ["softmax", "sqrt_softplus", "sigmoid"])
def test_reference_select(fn):
    l = torch.tensor([[1.0, 3.0, 2.0, 2.0, 0.0, 5.0, -1.0, 0.5]])
    ids, w = A.select(l, None, 3, fn)
    assert ids.tolist() == [[5, 1, 2]] and abs(float(w.sum()) - 1) < 1e-12
    # groups of two by their two best: {1,3} and {2,2} beat {0,5} only where the sum of scores says so
    s = A.score(l, fn)[0]
    worth = [float(s[2 * i] + s[2 * i + 1]) for i in range(4)]
    g = max(range(4), key=lambda i: worth[i])
    ids, _ = A.select(l, None, 2, fn, G=4, KG=1)
    assert sorted(ids[0].tolist()) == [2 * g, 2 * g + 1]
    assert A.select(l, None, 1, fn, G=4, KG=1, best=1)[0].tolist() == [[5]]
    b = torch.zeros(8)
    b[6] = 10.0
    assert A.select(l, b, 2, fn)[0].tolist() == [[6, 5]]
    assert A.select(torch.full((1, 8), -float("inf")), None, 2, fn)[1].tolist() == [[0.0, 0.0]]


def test_reference_rows8():
    x = torch.tensor([[448.0, 449.0, -1.0, 0.0], [0.0, 0.0, 0.0, 0.0], [float("inf"), 2.0, float("nan"), -2.0]])
    q, sf = A.pack8(x)
    assert sf[:, 0].tolist() == [128, 127, 120]
    v = A.values8(q, sf)
    assert v[0].tolist() == [448.0, 448.0, -1.0, 0.0] and torch.isnan(v[2, [0, 2]]).all() and v[2, 1] == 2.0
