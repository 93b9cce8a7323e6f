"""The two ways that arguments of the calls around the layer are checked and passed on (_native.so, and Python and ctypes
where it does not load) give the same results and the same refusals."""
import ctypes

import pytest
import torch

from gpu_util import ensure_lib

pytestmark = pytest.mark.gpu

BF, HF, FP = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def M():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return ensure_lib()


def outcome(M, fast, f):
    """What the call gives with this marshalling: its outputs, or the exception's type (and status)."""
    kept, M._fast = M._fast, fast
    try:
        return [t.clone() for t in f()]
    except M.MoeError as e:
        return ("MoeError", e.status)
    except (TypeError, ValueError, AttributeError, ctypes.ArgumentError) as e:
        return type(e).__name__
    finally:
        M._fast = kept


def same(M, f):
    M._load_native()
    assert not isinstance(M._fast, M._NoNative)
    a, b = outcome(M, M._fast, f), outcome(M, M._NoNative(), f)
    torch.cuda.synchronize()
    if isinstance(a, list):
        assert isinstance(b, list) and len(a) == len(b) and all(torch.equal(u.view(torch.uint8), v.view(torch.uint8)) for u, v in zip(a, b))
    else:
        assert a == b
    return a


def rn(*s, dt=BF, seed=0):
    return torch.randn(*s, generator=torch.Generator().manual_seed(seed + sum(s))).to(dt).cuda()


def test_norm(M):
    T, H = 12, 264
    w = rn(H, dt=FP)
    for dt in (BF, HF, FP):
        x, r = rn(T, H, dt=dt), rn(T, H, dt=dt, seed=1)

        def fwd(x=x, w=w, eps=1e-5, r=r, **kw):
            s, y, y8 = torch.zeros_like(x), torch.zeros_like(x), tuple(t.zero_() for t in M.new_rows8(T, H))
            kw = {**dict(residual=r, sum_out=s, y=y, y8=y8), **kw}
            M.rms_norm(x, w, eps, **kw)
            return [s, y, *y8]

        def bwd(dy=x, x=r, w=w, eps=1e-5, ws=M.new_workspace_norm(T, H), **kw):
            dx, dw = torch.zeros_like(r), torch.zeros(H, device="cuda")
            kw = {**dict(dx=dx, ws=ws, dweight=dw, dsum=x), **kw}
            M.rms_norm_backward(dy, x, w, eps, **kw)
            return [dx, dw]

        assert isinstance(same(M, fwd), list) and isinstance(same(M, bwd), list)
        for good in (dict(eps=0), dict(eps=1), dict(r=None), dict(sum_out=None), dict(y8=None), dict(x=rn(T, H + 4, dt=dt)[:, :H])):
            assert isinstance(same(M, lambda: fwd(**good)), list), good
        other = BF if dt != BF else HF
        for bad in (dict(eps=-1.0), dict(eps=float("nan")), dict(w=w[:-1]), dict(w=w.half()), dict(w=w.cpu()), dict(x=x.cpu()), dict(x=x[0]),
                    dict(x=x.to(torch.float64)), dict(r=r[:-1]), dict(r=r.to(other)), dict(y=x.t()), dict(y=x[:, ::2]), dict(y=3),
                    dict(y8=M.new_rows8(T, H + 1)), dict(y8=M.new_rows8(T, H)[:1]), dict(y8=tuple(t.int() for t in M.new_rows8(T, H))),
                    dict(sum_out=None, y=None, y8=None), dict(sum_out=x, y=x), dict(eps="1"), dict(x=x[:1].expand(T, H)), dict(w=w[1:]),
                    dict(y8=5)):
            assert not isinstance(same(M, lambda: fwd(**bad)), list), bad
        for bad in (dict(ws=None), dict(ws=torch.zeros(256, dtype=torch.uint8, device="cuda")), dict(ws=torch.zeros(99999, device="cuda")),
                    dict(dx=None, dweight=None), dict(dx=None), dict(dy=x[:-1]), dict(dsum=x.to(other)), dict(dweight=w[:-1]), dict(eps=-1.0)):
            assert not isinstance(same(M, lambda: bwd(**bad)), list), bad


def test_select(M):
    T, E, K = 9, 64, 6
    for dt in (FP, BF, HF):
        l, b = rn(T, E, dt=dt), rn(E, dt=FP)

        def fwd(l=l, b=b, fn="sigmoid", k=K, ids=None, w=None, **kw):
            ids = torch.zeros(T, k, dtype=torch.int32, device="cuda") if ids is None else ids
            w = torch.zeros(T, k, device="cuda") if w is None else w
            M.select(l, ids, w, fn, e_score_bias=b, **kw)
            return [ids, w]

        ids, w = fwd()
        dw = rn(T, K, dt=FP, seed=2)

        def bwd(l=l, ids=ids, w=w, dw=dw, out=None, ws=M.new_workspace_rows(T, K, E), fn="sigmoid", **kw):
            out = torch.zeros_like(l) if out is None else out
            M.select_backward(l, ids, w, dw, out, ws, fn, **kw)
            return [out]

        for good in (dict(), dict(fn=0), dict(fn="softmax", b=None), dict(n_groups=8, topk_groups=4), dict(renormalize=False, scale=2),
                     dict(scale=-0.5, group_best=1), dict(l=rn(T, E + 3, dt=dt)[:, :E])):
            assert isinstance(same(M, lambda: fwd(**good)), list), good
        for bad in (dict(fn="tanh"), dict(fn=7), dict(k=33), dict(n_groups=7), dict(n_groups=8, topk_groups=9), dict(scale=0.0), dict(b=b[:-1]),
                    dict(b=b.half()), dict(l=l.cpu()), dict(l=l[:-1]), dict(ids=torch.zeros(T, K, device="cuda")), dict(w=torch.zeros(T, 5, device="cuda")),
                    dict(ids=torch.zeros(T, K, dtype=torch.int32)), dict(n_groups=1.5), dict(group_best=3), dict(l=l.double())):
            assert not isinstance(same(M, lambda: fwd(**bad)), list), bad
        for good in (dict(), dict(fn="softmax", renormalize=False, scale=1), dict(out=torch.zeros(T, E + 5, dtype=dt, device="cuda")[:, :E])):
            assert isinstance(same(M, lambda: bwd(**good)), list), good
        for bad in (dict(ws=None), dict(ws=torch.zeros(99, dtype=torch.uint8, device="cuda")), dict(fn=5), dict(scale=0), dict(w=w[:-1]),
                    dict(out=torch.zeros(T, E - 1, device="cuda")), dict(dw=dw.cpu()), dict(out=torch.zeros(T, E, dtype=torch.int32, device="cuda")),
                    *([] if dt == FP else [dict(out=torch.zeros(T, E, device="cuda"))])):
            assert not isinstance(same(M, lambda: bwd(**bad)), list), bad


def test_rows8_and_linear(M):
    rows, N, K, E, align = 64, 48, 72, 3, 16
    counts = torch.tensor([5, 16, 20], dtype=torch.int32, device="cuda")
    ws256 = torch.zeros(256, dtype=torch.uint8, device="cuda")
    x = rn(rows, K)

    def pack(x=x, cols=K, **kw):
        x8 = tuple(t.zero_() for t in M.new_rows8(rows, cols))
        M.pack_rows8(x, x8, **kw)
        return list(x8)

    assert isinstance(same(M, pack), list)
    assert isinstance(same(M, lambda: pack(expert_counts=counts, align=align, ws=ws256)), list)
    for bad in (dict(cols=K + 1), dict(x=x.cpu()), dict(x=x.double()), dict(expert_counts=counts, align=3, ws=ws256),
                dict(expert_counts=counts, align=16), dict(expert_counts=counts[:0], align=16, ws=ws256), dict(expert_counts=counts.long()),
                dict(expert_counts=counts, align=16, ws=ws256[:99]), dict(align="a")):
        assert not isinstance(same(M, lambda: pack(**bad)), list), bad
    x8 = pack()
    for act, experts in (("silu", False), ("swiglu", True), ("none", False)):
        w = rn(*([E] if experts else []), N, K)
        cols = N // 2 if act == "swiglu" else N
        dy, z, res = rn(rows, cols, seed=3), rn(rows, N, seed=4), rn(rows, K, seed=5)
        z8 = tuple(t.zero_() for t in M.new_rows8(rows, N))
        M.pack_rows8(z, z8)
        ids = torch.randint(0, 2 * rows, (rows,), generator=torch.Generator().manual_seed(1), dtype=torch.int32).cuda()

        def bwd(dy=dy, w=w, ws=M.new_workspace_linear8(rows, N, K, E, act), **kw):
            dx, dw = torch.zeros(rows, K, dtype=BF, device="cuda"), torch.zeros_like(w)
            db = torch.zeros(w.shape[:-1], device="cuda")
            kw = {**dict(x8=tuple(x8), z8=None if act == "none" else z8, x_ids=ids, x_div=2, dx=dx, dw=dw, dbias=db, act=act, dx_residual=res,
                         expert_counts=counts if experts else None, align=align), **kw}
            M.linear_backward8(dy, w, ws, **kw)
            return [dx, dw, db]

        assert isinstance(same(M, bwd), list)
        for good in (dict(x8=None, x=x, x_ids=None), dict(dx=None, dx_residual=None), dict(dbias=None), dict(x_ids=None)):
            assert isinstance(same(M, lambda: bwd(**good)), list), good
        if act != "none":
            assert isinstance(same(M, lambda: bwd(z8=None, z=z)), list)
        for bad in (dict(x=x), dict(x8=None), dict(z8=z8, act="none") if act != "none" else dict(z=z), dict(dx=None), dict(x_div=0), dict(w=w[..., :-8]),
                    dict(dy=dy[:-1]), dict(ws=ws256), dict(dw=w[..., :8]), dict(dbias=w), dict(act="tanh"), dict(x_ids=ids[:-1]), dict(align=5) if experts
                    else dict(expert_counts=counts), dict(x8=(x8[0], x8[0])), dict(dy=dy.float()), dict(ws=None)):
            assert not isinstance(same(M, lambda: bwd(**bad)), list), bad
