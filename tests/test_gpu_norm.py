"""RMS norm with the residual's addition and 8-bit rows, and its gradients, against float64."""
import pytest
import torch

import around_ref as A
import train_ref as R
from gpu_util import ensure_lib

pytestmark = pytest.mark.gpu

BF, HF, FP = torch.bfloat16, torch.float16, torch.float32
SENTINEL = 7.25
EPS = 1e-5


@pytest.fixture(scope="module")
def M():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return ensure_lib()


def mat(n, c, dt, seed, pitch=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    v = (torch.randn(n, c, generator=g) * torch.exp(torch.randn(n, 1, generator=g)) * scale).to(dt)
    wide = torch.full((n, c + pitch), SENTINEL, dtype=dt, device="cuda")
    wide[:, :c] = v.cuda()
    return v, wide[:, :c]


def room(n, c, dt, pitch=0):
    return torch.full((n, c + pitch), SENTINEL, dtype=dt, device="cuda")


def weight(H, seed=9):
    w = torch.rand(H, generator=torch.Generator().manual_seed(seed)) * 2 - 0.5
    return w, w.cuda()


def room8(n, c, pitch=0, spitch=0):
    q = torch.full((n, c + pitch), 0x55, dtype=torch.uint8, device="cuda")
    s = torch.full((n, -(-c // 128) + spitch), 0x55, dtype=torch.uint8, device="cuda")
    return q, s


CASES = [  # T, H, dtype, extra pitch
    (1, 7168, BF, 0), (8, 7168, BF, 8), (3, 1, FP, 0), (2, 1, BF, 0), (5, 33, HF, 0), (37, 129, BF, 3), (64, 1000, HF, 0),
    (130, 24, FP, 0), (257, 520, BF, 4), (333, 1001, FP, 0), (700, 128, HF, 0), (9, 2048, FP, 4), (3, 8200, BF, 0),
    (2, 16384, FP, 0), (3, 16392, BF, 0), (2, 33000, BF, 0), (2, 40001, HF, 0), (1, 70000, FP, 0), (1500, 64, BF, 0),
    (400, 256, BF, 8), (5, 7168, HF, 1), (40, 4099, BF, 0), (300, 3001, HF, 0), (17, 384, BF, 0), (6, 1024, BF, 0),
]


# rows through the ring: groups of several sizes, rows that start anywhere, rows of more than 1024 packs, few rows at a time
CASES += [(200, 7168, BF, 0), (160, 8192, BF, 0), (155, 15360, BF, 0), (400, 5001, FP, 0), (170, 4472, HF, 0), (700, 945, HF, 0),
          (2500, 264, BF, 0), (620, 1001, FP, 3), (333, 2521, BF, 1), (1000, 4096, FP, 0), (5000, 72, FP, 0), (310, 1032, HF, 8),
          (153, 9700, HF, 0), (153, 9733, BF, 0), (8, 7168, FP, 0), (9, 7168, BF, 0), (10, 7168, BF, 0)]
# many short rows that start anywhere: groups of one warp, and of two
CASES += [(700, 155, FP, 0), (3000, 300, BF, 0), (6500, 301, HF, 1), (5000, 265, BF, 0), (800, 509, HF, 0), (900, 254, FP, 2),
          (4000, 545, HF, 0), (640, 257, FP, 0)]


@pytest.mark.parametrize("T,H,dt,extra", CASES)
def test_norm(M, T, H, dt, extra):
    x, xd = mat(T, H, dt, T + H, extra)
    r, rd = mat(T, H, dt, T + H + 1)
    w, wd = weight(H)
    for res in (None, r):
        s, y, e = A.norm(x, res, w, EPS, dt)
        bound = e + R.half_step(dt) * (y.abs() + e) + R.tiny(dt)
        so, yo, y8 = room(T, H, dt, extra), room(T, H, dt, extra), room8(T, H, extra)
        M.rms_norm(xd, wd, EPS, residual=None if res is None else rd, sum_out=so[:, :H], y=yo[:, :H],
                   y8=(y8[0][:, :H], y8[1]))
        assert torch.equal(so[:, :H].cpu().to(A.F64), s)
        R.check(yo[:, :H], y, bound, "y")
        A.check8(y8[0][:, :H], y8[1], y, e, "y8")
        assert (so[:, H:] == SENTINEL).all() and (yo[:, H:] == SENTINEL).all() and (y8[0][:, H:] == 0x55).all()
        # each output alone is the same
        for kw in (dict(sum_out=torch.empty_like(so[:, :H])), dict(y=torch.empty_like(yo[:, :H])),
                   dict(y8=room8(T, H, 0, 1))):
            if "y8" in kw:
                kw["y8"] = (kw["y8"][0], kw["y8"][1][:, :-1])
            M.rms_norm(xd, wd, EPS, residual=None if res is None else rd, **kw)
            for k, v in kw.items():
                if k == "y8":
                    assert torch.equal(v[0], y8[0][:, :H]) and torch.equal(v[1], y8[1])
                else:
                    assert torch.equal(v, (so if k == "sum_out" else yo)[:, :H])
    # in place: the stream into x or into the residual, y over the other.  (A row's sum is taken in an order that goes by
    # the rows' alignment, so y's last bits may differ from those of rows with a pitch: the same bits are asked of a call
    # out of place on rows like these.)
    xc, rc = xd.clone(), rd.clone()
    so, yo = torch.empty_like(xc), torch.empty_like(xc)
    M.rms_norm(xc, wd, EPS, residual=rc, sum_out=so, y=yo)
    assert torch.equal(so.cpu().to(A.F64), s)
    R.check(yo, y, bound, "y of contiguous rows")
    for a, b in ((0, 1), (1, 0)):
        buf = [xd.clone(), rd.clone()]
        M.rms_norm(buf[0], wd, EPS, residual=buf[1], sum_out=buf[a], y=buf[b])
        assert torch.equal(buf[a], so) and torch.equal(buf[b], yo)
    buf = xd.clone()
    M.rms_norm(buf, wd, EPS, residual=rc, y=buf)
    assert torch.equal(buf, yo)


@pytest.mark.parametrize("T,H,dt,extra", CASES)
def test_norm_gradients(M, T, H, dt, extra):
    x, xd = mat(T, H, dt, T + H, extra)
    dy, dyd = mat(T, H, dt, T + H + 2)
    ds, dsd = mat(T, H, dt, T + H + 3, extra)
    w, wd = weight(H)
    ws = M.new_workspace_norm(T, H)
    for d in (None, ds):
        (dx, ex), (dw, ew) = A.norm_grad(dy, x, w, EPS, d, dt)
        out, dwo = room(T, H, dt, extra), torch.full((H,), float("nan"), device="cuda")
        dd = None if d is None else dsd
        M.rms_norm_backward(dyd, xd, wd, EPS, out[:, :H], ws, dweight=dwo, dsum=dd)
        R.check(out[:, :H], dx, ex, "dx")
        R.check(dwo, dw, ew, "dweight")
        assert (out[:, H:] == SENTINEL).all()
        # either alone; and again, on contiguous rows: the same bits (their order goes by the rows' alignment)
        o2, w2 = torch.empty_like(xd), torch.empty_like(dwo)
        M.rms_norm_backward(dyd, xd, wd, EPS, o2, ws, dsum=dd)
        M.rms_norm_backward(dyd, xd, wd, EPS, None, ws, dweight=w2)
        R.check(o2, dx, ex, "dx alone")
        R.check(w2, dw, ew, "dweight alone")
        full = [t if t is None else t.clone() for t in (dyd, xd, dd)]
        o3, w3, o4, w4 = (f(v) for f in (torch.empty_like,) for v in (full[0], w2, full[0], w2))
        for o, v in ((o3, w3), (o4, w4)):
            M.rms_norm_backward(full[0], full[1], wd, EPS, o, ws, dweight=v, dsum=full[2])
        R.check(o3, dx, ex, "dx of contiguous rows")
        R.check(w3, dw, ew, "dweight of contiguous rows")
        assert torch.equal(o3, o4) and torch.equal(w3, w4)
    # in place of each input
    for k in range(3):
        buf = [dyd.clone(), xd.clone(), dsd.clone()]
        M.rms_norm_backward(buf[0], buf[1], wd, EPS, buf[k], ws, dweight=w2, dsum=buf[2])
        assert torch.equal(buf[k], o3) and torch.equal(w2, w3)
    assert M.get_error(ws) == M.OK


def test_norm_gradient_against_differences(M):
    """dL/dx along a direction, L = sum(c y + c2 sum), in fp32: central differences of the kernel's own forward."""
    T, H, h = 6, 96, 2.0 ** -6
    g = torch.Generator().manual_seed(3)
    x, d, c, c2 = (torch.randn(T, H, generator=g).cuda() for _ in range(4))
    w = (torch.rand(H, generator=g) + 0.5).cuda()
    y1, y2, dx = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    M.rms_norm(x + h * d, w, EPS, y=y1)
    M.rms_norm(x - h * d, w, EPS, y=y2)
    M.rms_norm_backward(c, x, w, EPS, dx, M.new_workspace_norm(T, H), dsum=c2)
    num = ((y1.double() - y2.double()) * c.double()).sum() / (2 * h) + (c2.double() * d.double()).sum()
    # truncation h^2 / 6 = 4e-5 times a third derivative along d (of order |d / rms|^3, a few) per term of 576 with signs
    # at random: 24 * 4e-5 * 10 = 0.01; rounding 576 * 2^-22 / h: 0.01
    assert abs(float(num - (dx.double() * d.double()).sum())) < 0.02


def test_rows_of_zeros_and_what_is_not_finite(M):
    w = torch.ones(256, device="cuda")
    x = torch.zeros(5, 256, device="cuda", dtype=BF)
    x[1] = 1
    x[2, 7] = float("inf")
    x[2, 8] = 1
    x[3, 9] = float("nan")
    x[4] = 1e-30
    y, y8 = torch.empty_like(x), room8(5, 256)
    M.rms_norm(x, w, 1e-6, y=y, y8=y8)
    v = A.values8(y8[0].cpu(), y8[1].cpu())
    assert (y[0] == 0).all() and (v[0] == 0).all() and (y8[1][0] == 127).all()
    assert (y[1] == 1).all() and (v[1] == 1).all()
    assert torch.isnan(y[2, 7]) and y[2, 8] == 0 and torch.isnan(v[2, 7]) and (v[2, 8:] == 0).all()   # inf * 0
    assert torch.isnan(y[3]).all() and torch.isnan(v[3]).all()
    assert (y[4].float() - 1e-27).abs().max() < 1e-29
    M.rms_norm(x, w, 0.0, y=y)                    # no eps: 0 * inf
    assert torch.isnan(y[0]).all() and (y[1] == 1).all()


def test_one_workspace_for_many_sizes(M):
    """Calls of different sizes in turn on one workspace: what one leaves there does not reach the next."""
    ws = M.new_workspace_norm(700, 945)
    for T, H, dt in ((5, 300, BF), (700, 945, HF), (9, 512, FP), (1, 64, BF), (5, 300, BF), (300, 128, FP), (40, 600, BF)) * 2:
        x, xd = mat(T, H, dt, T)
        dy, dyd = mat(T, H, dt, T + 1)
        w, wd = weight(H)
        dw = torch.full((H,), float("nan"), device="cuda")
        M.rms_norm_backward(dyd, xd, wd, EPS, None, ws, dweight=dw)
        _, (ref, ew) = A.norm_grad(dy, x, w, EPS, None, dt)
        R.check(dw, ref, ew, "dweight")
    assert M.get_error(ws) == M.OK


def test_no_rows(M):
    x, w = torch.empty(0, 64, device="cuda", dtype=BF), torch.ones(64, device="cuda")
    M.rms_norm(x, w, EPS, y=x)
    dw = torch.ones(64, device="cuda")
    M.rms_norm_backward(x, x, w, EPS, x, M.new_workspace_norm(0, 64), dweight=dw)
    assert (dw == 0).all()


def test_capture_and_streams(M):
    """Forward and backward captured into a graph, replayed on new inputs, beside eager calls on another stream."""
    T, H = 65, 1024
    w, wd = weight(H)
    x, xd = mat(T, H, BF, 1)
    dy, dyd = mat(T, H, BF, 2)
    s, y, dx = torch.empty_like(xd), torch.empty_like(xd), torch.empty_like(xd)
    dw, ws, y8 = torch.empty(H, device="cuda"), M.new_workspace_norm(T, H), M.new_rows8(T, H)

    def call(ws, s, y, y8, dx, dw):
        M.rms_norm(xd, wd, EPS, residual=dyd, sum_out=s, y=y, y8=y8)
        M.rms_norm_backward(dyd, s, wd, EPS, dx, ws, dweight=dw)

    call(ws, s, y, y8, dx, dw)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(ws, s, y, y8, dx, dw)
    for seed in (3, 4):
        xd.copy_(mat(T, H, BF, seed)[0])
        for t in (s, y, dx, dw, *y8):
            t.zero_()
        torch.cuda.synchronize()
        g.replay()
        other = [torch.empty_like(t) for t in (s, y, dx, dw)]
        o8, ows = M.new_rows8(T, H), M.new_workspace_norm(T, H)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            call(ows, other[0], other[1], o8, other[2], other[3])
        torch.cuda.synchronize()
        for a, b in zip((s, y, dx, dw, *y8), (*other, *o8)):
            assert torch.equal(a, b)
