"""Norm and gradients where some of the matrices have their rows on 16-byte boundaries and others have not, through every way
that rows are run (a warp each, a few CTAs, the ring, wide rows)."""
import pytest
import torch

import around_ref as A
import train_ref as R
from gpu_util import ensure_lib
from test_gpu_norm import EPS, SENTINEL, mat, room, room8, weight

pytestmark = pytest.mark.gpu

BF, HF, FP = torch.bfloat16, torch.float16, torch.float32
SHAPES = [(40, 64, BF), (3, 1024, HF), (400, 512, BF), (200, 7168, BF), (700, 1024, FP), (160, 4096, FP), (5, 16392, BF), (160, 24576, BF)]


@pytest.fixture(scope="module")
def M():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return ensure_lib()


@pytest.mark.parametrize("T,H,dt", SHAPES)
@pytest.mark.parametrize("residual", [False, True])
def test_outputs_off_boundaries_of_inputs_on_them(M, T, H, dt, residual):
    x, xd = mat(T, H, dt, T + H)
    r, rd = mat(T, H, dt, T + H + 1)
    w, wd = weight(H)
    s, y, e = A.norm(x, r if residual else None, w, EPS, dt)
    bound = e + R.half_step(dt) * (y.abs() + e) + R.tiny(dt)
    for so, yo, q in ((1, 0, 0), (0, 1, 3), (1, 3, 1)):
        for start in (0, 1):                  # rows off by their pitch, and by where the first one starts too
            cut = slice(start, start + H)
            sb, yb, y8 = room(T, H, dt, so + 1), room(T, H, dt, yo + 1), room8(T, H, q)
            M.rms_norm(xd, wd, EPS, residual=rd if residual else None, sum_out=sb[:, cut], y=yb[:, cut], y8=(y8[0][:, :H], y8[1]))
            assert torch.equal(sb[:, cut].cpu().to(A.F64), s)
            R.check(yb[:, cut], y, bound, "y")
            A.check8(y8[0][:, :H], y8[1], y, e, "y8")
            for b in (sb, yb):
                assert (b[:, :start] == SENTINEL).all() and (b[:, start + H:] == SENTINEL).all()
            assert (y8[0][:, H:] == 0x55).all()


@pytest.mark.parametrize("T,H,dt", SHAPES)
@pytest.mark.parametrize("which", [0, 1, 2, 3])
def test_gradients_with_one_matrix_off_boundaries(M, T, H, dt, which):
    pitch = [1 if i == which else 0 for i in range(4)]
    x, xd = mat(T, H, dt, T + H, pitch[0])
    dy, dyd = mat(T, H, dt, T + H + 2, pitch[1])
    ds, dsd = mat(T, H, dt, T + H + 3, pitch[2])
    w, wd = weight(H)
    out, dw, ws = room(T, H, dt, pitch[3]), torch.full((H,), float("nan"), device="cuda"), M.new_workspace_norm(T, H)
    for d in (None, ds):
        (dx, ex), (dwr, ew) = A.norm_grad(dy, x, w, EPS, d, dt)
        M.rms_norm_backward(dyd, xd, wd, EPS, out[:, :H], ws, dweight=dw, dsum=None if d is None else dsd)
        R.check(out[:, :H], dx, ex, "dx")
        R.check(dw, dwr, ew, "dweight")
        assert (out[:, H:] == SENTINEL).all()
    assert M.get_error(ws) == M.OK


# rows past the ring, many of them: every loop over rows goes round more than once, with and without a dsum and in place
@pytest.mark.parametrize("T,H,dt", [(400, 8704, BF), (310, 9009, HF), (333, 7168, FP), (330, 17000, BF), (300, 17001, HF), (200, 9000, FP),
                                    (170, 33000, BF)])
def test_gradients_of_many_wide_rows(M, T, H, dt):
    x, xd = mat(T, H, dt, T + H)
    dy, dyd = mat(T, H, dt, T + H + 2)
    ds, dsd = mat(T, H, dt, T + H + 3)
    w, wd = weight(H)
    ws = M.new_workspace_norm(T, H)
    for d in (None, ds):
        (dx, ex), (dwr, ew) = A.norm_grad(dy, x, w, EPS, d, dt)
        out, dw = room(T, H, dt), torch.full((H,), float("nan"), device="cuda")
        M.rms_norm_backward(dyd, xd, wd, EPS, out, ws, dweight=dw, dsum=None if d is None else dsd)
        R.check(out, dx, ex, "dx")
        R.check(dw, dwr, ew, "dweight")
        for k in range(3 if d is not None else 2):
            buf, dw2 = [dyd.clone(), xd.clone(), dsd.clone()], torch.empty_like(dw)
            M.rms_norm_backward(buf[0], buf[1], wd, EPS, buf[k], ws, dweight=dw2, dsum=None if d is None else buf[2])
            assert torch.equal(buf[k], out) and torch.equal(dw2, dw)
    assert M.get_error(ws) == M.OK


@pytest.mark.parametrize("T,H,dt", [(300, 9000, FP), (400, 17000, BF), (310, 17001, HF), (320, 33000, BF)])
def test_many_wide_rows(M, T, H, dt):
    x, xd = mat(T, H, dt, T + H)
    r, rd = mat(T, H, dt, T + H + 1)
    w, wd = weight(H)
    for res in (None, r):
        s, y, e = A.norm(x, res, w, EPS, dt)
        so, yo, y8 = room(T, H, dt), room(T, H, dt), room8(T, H)
        M.rms_norm(xd, wd, EPS, residual=None if res is None else rd, sum_out=so, y=yo, y8=y8)
        assert torch.equal(so.cpu().to(A.F64), s)
        R.check(yo, y, e + R.half_step(dt) * (y.abs() + e) + R.tiny(dt), "y")
        A.check8(*y8, y, e, "y8")
