"""Matrix products with bias, activation and residual, dense and per expert, and their gradients, against float64."""
import pytest
import torch

import train_ref as R
from gpu_util import ensure_lib

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16
SENTINEL = 7.25


@pytest.fixture(scope="module")
def M():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return ensure_lib()


def mat(n, c, dt, seed, pitch=0, scale=1.0):
    v = (torch.randn(n, c, generator=torch.Generator().manual_seed(seed)) * scale).to(dt)
    wide = torch.full((n, c + pitch), SENTINEL, dtype=dt, device="cuda")
    wide[:, :c] = v.cuda()
    return v, wide[:, :c]


def operands(rows, N, K, E, counts, align, dt, pitch=0):
    x, xd = mat(rows, K, dt, 1, pitch)
    n = max(E, 1)
    w, wd = mat(n * N, K, dt, 2, 0, K ** -0.5)
    if E:
        wd = wd.reshape(E, N, K)
    bias = torch.randn((E, N) if E else (N,), generator=torch.Generator().manual_seed(3))
    live = torch.zeros(rows, dtype=torch.bool)
    for _, r, c in R.segments(counts, align, rows):
        live[r:r + c] = True
    return x, xd, w.reshape(n, N, K), wd.contiguous(), bias, live


def poison(t, live):
    t[~live.cuda()] = float("nan")


# rows (dense) or counts, N, K, align
DENSE = [(1, 64, 64), (1, 2048, 1000), (8, 4096, 520), (7, 8, 8), (16, 200, 72), (31, 136, 264), (128, 1024, 512),
         (129, 264, 1032), (255, 128, 64), (256, 256, 192), (300, 520, 328), (1000, 776, 200), (2500, 640, 448)]
EXPERTS = [([3, 0, 130, 1], 16, 144, 200), ([0, 0, 5], 1, 64, 64), ([300, 17, 256, 0, 64], 128, 272, 136),
           ([1], 256, 2048, 72), ([0, 0], 64, 80, 80), ([700, 3, 90], 1, 528, 264), ([1] * 40, 16, 96, 128),
           # some hundred rows each (pairs of 256-row tiles): sums of 2, 5 and 13 slabs in the forward
           ([513, 0, 512, 31, 256, 257, 1000], 16, 272, 128), ([300, 290, 1], 1, 336, 264), ([1100, 600], 256, 784, 800)]
ACTS = ["none", "relu", "silu", "gelu", "swiglu"]


def cases():
    for i, (rows, N, K) in enumerate(DENSE):
        for a in (ACTS if i in (2, 5, 10) else [ACTS[i % 5], ACTS[(i + 2) % 5]]):
            if a != "swiglu" or N % 16 == 0:
                yield rows, None, 0, N, K, a
    for i, (counts, align, N, K) in enumerate(EXPERTS):
        rows = sum(-(-c // align) * align for c in counts) + (5 if i % 2 else 0)
        for a in ("none", "swiglu", ACTS[1 + i % 3]):
            yield max(rows, 1), counts, align, N, K, a


@pytest.mark.parametrize("rows,counts,align,N,K,act", list(cases()))
def test_linear_and_its_gradients(M, rows, counts, align, N, K, act):
    E = len(counts) if counts else 0
    for dt, pitch in ((BF, 0), (HF, 24)):
        x, xd, w, wd, bias, live = operands(rows, N, K, E, counts, align, dt, pitch)
        cols = N // 2 if act == "swiglu" else N
        cd = torch.tensor(counts, dtype=torch.int32, device="cuda") if E else None
        kw = dict(act=act, expert_counts=cd, align=align)
        ws = M.new_workspace_linear(rows, N, K, E, act)
        res, resd = mat(rows, cols, dt, 4, pitch)
        poison(xd, live)
        poison(resd, live)
        # forward: with everything, and bare
        for full in (True, False):
            y = torch.full((rows, cols + pitch), SENTINEL, dtype=dt, device="cuda")
            z = torch.full((rows, N + pitch), SENTINEL, dtype=dt, device="cuda")
            M.linear(xd, wd, y[:, :cols], ws, bias=bias.cuda() if full else None, residual=resd if full else None,
                     z=z[:, :N] if full else None, **kw)
            assert M.get_error(ws) == M.OK
            for e, r, c in R.segments(counts, align, rows):
                b = (bias[e] if E else bias) if full else None
                yr, ey, zr, ez = R.linear(x[r:r + c], w[e], b, act, res[r:r + c] if full else None, dt)
                R.check(y[r:r + c, :cols], yr, ey, f"y of expert {e}")
                if full:
                    R.check(z[r:r + c, :N], zr, ez, f"z of expert {e}")
            dead = ~live.cuda()
            assert (y[dead] == SENTINEL).all() and (y[:, cols:] == SENTINEL).all(), "only the rows' own columns are written"
            assert (z[dead] == SENTINEL).all() and (z[:, N:] == SENTINEL).all()
        # gradients
        dy, dyd = mat(rows, cols, dt, 5, pitch)
        zz, zzd = mat(rows, N, dt, 6, pitch)
        dres, dresd = mat(rows, K, dt, 7, pitch)
        for t in (dyd, zzd, dresd):
            poison(t, live)
        for r_ in (None, dres):
            dx = torch.full((rows, K + pitch), SENTINEL, dtype=dt, device="cuda")
            dw = torch.full(wd.shape, SENTINEL, dtype=dt, device="cuda")
            db = torch.full(bias.shape, SENTINEL, device="cuda")
            M.linear_backward(dyd, xd, wd, ws, dx=dx[:, :K], dw=dw, dbias=db, z=None if act == "none" else zzd,
                              dx_residual=None if r_ is None else dresd, **kw)
            assert M.get_error(ws) == M.OK
            for e, r, c in R.segments(counts, align, rows):
                (dxr, ex), (dwr, ew), (dbr, eb) = R.linear_grad(dy[r:r + c], x[r:r + c], w[e], zz[r:r + c], act,
                                                                None if r_ is None else dres[r:r + c], dt)
                R.check(dx[r:r + c, :K], dxr, ex, f"dx of expert {e}")
                R.check(dw[e] if E else dw, dwr, ew, f"dw of expert {e}")
                R.check(db[e] if E else db, dbr, eb, f"dbias of expert {e}")
                if c == 0:
                    assert (dw[e] == 0).all() and (db[e] == 0).all()
            assert (dx[~live.cuda()] == SENTINEL).all() and (dx[:, K:] == SENTINEL).all()
        # each gradient alone gives the same bits
        for one in ("dx", "dw", "dbias"):
            o = {"dx": torch.zeros(rows, K, dtype=dt, device="cuda"), "dw": torch.zeros_like(dw), "dbias": torch.zeros_like(db)}
            M.linear_backward(dyd, xd if one == "dw" else None, wd, ws, **{one: o[one]}, z=None if act == "none" else zzd,
                              dx_residual=dresd if one == "dx" else None, **kw)
            full_ = {"dx": dx[:, :K], "dw": dw, "dbias": db}[one]
            m = live.cuda() if one == "dx" else slice(None)
            assert torch.equal(o[one][m], full_[m]), one
        assert M.get_error(ws) == M.OK


@pytest.mark.parametrize("rows,N,K,act", [(4096, 1024, 2048, "gelu"), (5000, 2064, 1544, "swiglu"), (1, 7168, 2048, "none"),
                                          (200, 4096, 7168, "swiglu"), (64, 256, 7168, "silu")])
def test_linear_large(M, rows, N, K, act):
    # the reference in float64 on the GPU; the same bounds
    dt = BF
    x, xd, w, wd, bias, _ = operands(rows, N, K, 0, None, 0, dt)
    cols = N // 2 if act == "swiglu" else N
    res, resd = mat(rows, cols, dt, 4)
    ws = M.new_workspace_linear(rows, N, K, 0, act)
    y = torch.empty(rows, cols, dtype=dt, device="cuda")
    z = torch.empty(rows, N, dtype=dt, device="cuda")
    M.linear(xd, wd, y, ws, bias=bias.cuda(), residual=resd, z=z, act=act)
    yr, ey, zr, ez = (t.cpu() for t in R.linear(xd, wd, bias.cuda(), act, resd, dt))
    R.check(y, yr, ey, "y")
    R.check(z, zr, ez, "z")
    dy, dyd = mat(rows, cols, dt, 5)
    dx = torch.empty(rows, K, dtype=dt, device="cuda")
    dw = torch.empty_like(wd)
    db = torch.empty(N, device="cuda")
    M.linear_backward(dyd, xd, wd, ws, dx=dx, dw=dw, dbias=db, act=act, z=None if act == "none" else z)
    (a, ea), (b, eb), (c, ec) = R.linear_grad(dyd, xd, wd, None if act == "none" else z, act, None, dt)
    for got, ref, e, n in ((dx, a, ea, "dx"), (dw, b, eb, "dw"), (db, c, ec, "dbias")):
        R.check(got, ref.cpu(), e.cpu(), n)
    # equal inputs give equal bits
    y2 = torch.empty_like(y)
    M.linear(xd, wd, y2, ws, bias=bias.cuda(), residual=resd, act=act)
    assert torch.equal(y, y2)
    assert M.get_error(ws) == M.OK


UNEVEN = [0 if e % 5 == 3 else 1 + (e * 37) % 90 for e in range(70)]


@pytest.mark.parametrize("counts,align,N,K,act", [
    ([20, 0, 9], 16, 64, 4096, "silu"), ([20, 0, 9], 64, 4096, 72, "none"),            # long sums, few tiles
    ([33, 1, 0, 64, 500, 7, 0, 2], 8, 320, 1400, "swiglu"), (UNEVEN, 4, 96, 328, "gelu"), (UNEVEN, 64, 208, 200, "swiglu"),
    ([1500, 0, 2, 1], 1, 176, 1032, "relu"), ([0] * 40 + [5] + [0] * 23, 256, 96, 264, "none"),   # one expert has them
    ([500, 610, 0, 433, 256, 512, 1, 300, 470, 555, 128, 390], 32, 1536, 648, "swiglu"),
    ([310, 200, 0, 513, 256, 333, 640, 301], 16, 4096, 9640, "swiglu")])               # long enough for maps of its own
def test_experts_every_way(M, counts, align, N, K, act):
    # the reference in float64 on the GPU; padding rows are NaN
    E, dt = len(counts), BF
    rows = sum(-(-c // align) * align for c in counts)
    g = torch.Generator(device="cuda").manual_seed(rows + N)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")
    cols = N // 2 if act == "swiglu" else N
    x, w, bias, res = rand(rows, K).to(dt), (rand(E, N, K) * K ** -0.5).to(dt), rand(E, N), rand(rows, cols).to(dt)
    live = torch.zeros(rows, dtype=torch.bool, device="cuda")
    for _, r, c in R.segments(counts, align, rows):
        live[r:r + c] = True
    dy, dres = rand(rows, cols).to(dt), rand(rows, K).to(dt)
    for t in (x, res, dy, dres):
        t[~live] = float("nan")
    kw = dict(act=act, expert_counts=torch.tensor(counts, dtype=torch.int32, device="cuda"), align=align)
    ws = M.new_workspace_linear(rows, N, K, E, act)
    y = torch.full((rows, cols), SENTINEL, dtype=dt, device="cuda")
    z = torch.full((rows, N), SENTINEL, dtype=dt, device="cuda")
    M.linear(x, w, y, ws, bias=bias, residual=res, z=z, **kw)
    dx = torch.full((rows, K), SENTINEL, dtype=dt, device="cuda")
    M.linear_backward(dy, x, w, ws, dx=dx, z=None if act == "none" else z, dx_residual=dres, **kw)
    assert M.get_error(ws) == M.OK
    for e, r, c in R.segments(counts, align, rows):
        s = slice(r, r + c)
        yr, ey, zr, ez = R.linear(x[s], w[e], bias[e], act, res[s], dt)
        R.check(y[s], yr.cpu(), ey.cpu(), f"y of expert {e}")
        R.check(z[s], zr.cpu(), ez.cpu(), f"z of expert {e}")
        (a, ea), _, _ = R.linear_grad(dy[s], x[s], w[e], z[s], act, dres[s], dt)
        R.check(dx[s], a.cpu(), ea.cpu(), f"dx of expert {e}")
    assert (y[~live] == SENTINEL).all() and (z[~live] == SENTINEL).all() and (dx[~live] == SENTINEL).all()


def test_special_values(M):
    # relu keeps NaN, large negative arguments vanish, infinities stay where they are
    x = torch.eye(8, dtype=BF)
    w = torch.zeros(8, 8, dtype=BF)
    w[:, 0] = torch.tensor([float("nan"), float("inf"), -200.0, 200.0, -1e30, 0.0, -0.0, 1.0])
    ws = M.new_workspace_linear(8, 8, 8)
    x[1:] = 0                     # row 0 picks column 0 of w; the other rows are zero rows
    for act in ("relu", "silu", "gelu"):
        y = torch.empty(8, 8, dtype=BF, device="cuda")
        M.linear(x.cuda(), w.cuda(), y, ws, act=act)
        v = y[0].float().cpu()
        assert torch.isnan(v[0]) and v[1] == float("inf") and v[2] == 0 and v[3] == 200 and v[4] == 0 and v[5] == 0
        assert torch.isnan(y[1, 0]) and torch.isnan(y[1, 1]) and (y[1, 2:] == 0).all()     # 0 * NaN, 0 * inf


def test_no_rows(M):
    w = torch.randn(32, 16, device="cuda").to(BF)
    ws = M.new_workspace_linear(0, 32, 16)
    x, y = torch.zeros(0, 16, dtype=BF, device="cuda"), torch.zeros(0, 32, dtype=BF, device="cuda")
    M.linear(x, w, y, ws)
    dw, db = torch.full_like(w, 3), torch.full((32,), 3.0, device="cuda")
    M.linear_backward(y, x, w, ws, dx=x, dw=dw, dbias=db)
    assert (dw == 0).all() and (db == 0).all()


def test_segments_past_the_buffers_are_reported(M):
    # the counts ask for more rows than the buffers hold: reported, and nothing outside is touched
    rows, N, K = 40, 64, 64
    x = torch.randn(rows, K, device="cuda").to(BF)
    w = torch.randn(3, N, K, device="cuda").to(BF)
    ws = M.new_workspace_linear(rows, N, K, 3)
    for counts in ([16, 30, 5], [-3, 8, 8], [1000, 1, 1], [2 ** 31 - 1, 2 ** 31 - 1, 7]):
        buf = torch.full((rows + 64, N), SENTINEL, dtype=BF, device="cuda")
        c = torch.tensor(counts, dtype=torch.int32, device="cuda")
        M.linear(x, w, buf[:rows], ws, expert_counts=c, align=16)
        assert M.get_error(ws) == M.ERR_DEVICE_INDEX
        assert (buf[rows:] == SENTINEL).all()
        dw, db = torch.empty_like(w), torch.empty(3, N, device="cuda")
        M.linear_backward(buf[:rows], x, w, ws, dx=torch.empty_like(x), dw=dw, dbias=db, expert_counts=c, align=16)
        assert M.get_error(ws) == M.ERR_DEVICE_INDEX


def test_segments_past_large_buffers_are_reported(M):
    # the same where the tiles are many, and the rows that do exist are still right
    rows, N, K = 2000, 4096, 512
    x = torch.randn(rows, K, device="cuda").to(BF)
    w = (torch.randn(4, N, K, device="cuda") * K ** -0.5).to(BF)
    ws = M.new_workspace_linear(rows, N, K, 4)
    for counts in ([500, 1000, 480, 700], [300, -7, 4000, 5], [2 ** 31 - 1, 2 ** 31 - 1, 7, 0]):
        buf = torch.full((rows + 300, N), SENTINEL, dtype=BF, device="cuda")
        c = torch.tensor(counts, dtype=torch.int32, device="cuda")
        M.linear(x, w, buf[:rows], ws, expert_counts=c, align=16)
        assert M.get_error(ws) == M.ERR_DEVICE_INDEX
        assert (buf[rows:] == SENTINEL).all()
        n = min(counts[0], rows)
        yr, ey, _, _ = R.linear(x[:n], w[0], None, "none", None, BF)
        R.check(buf[:n], yr.cpu(), ey.cpu(), "y of expert 0")
        M.linear_backward(buf[:rows], x, w, ws, dx=torch.empty_like(x), dw=torch.empty_like(w), expert_counts=c, align=16)
        assert M.get_error(ws) == M.ERR_DEVICE_INDEX


def test_linear_on_another_stream_and_in_a_graph(M):
    rows, N, K = 96, 256, 320
    x = torch.randn(rows, K, device="cuda").to(BF)
    w = torch.randn(N, K, device="cuda").to(BF) * 0.05
    bias = torch.randn(N, device="cuda")
    ws = M.new_workspace_linear(rows, N, K, 0, "silu")
    y, z = torch.empty(rows, N, dtype=BF, device="cuda"), torch.empty(rows, N, dtype=BF, device="cuda")
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty(N, device="cuda")

    def step():
        M.linear(x, w, y, ws, bias=bias, act="silu", z=z)
        M.linear_backward(y, x, w, ws, dx=dx, dw=dw, dbias=db, act="silu", z=z)

    step()
    torch.cuda.synchronize()
    want = [t.clone() for t in (y, z, dx, dw, db)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, (y, z, dx, dw, db)))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for k in range(3):
        x.copy_(torch.randn(rows, K, device="cuda").to(BF))
        step()
        want = [t.clone() for t in (y, z, dx, dw, db)]
        for t in (y, z, dx, dw, db):
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, (y, z, dx, dw, db)))
    assert M.get_error(ws) == M.OK


@pytest.mark.parametrize("rows,N,act", [(40, 64, "none"), (40, 64, "swiglu"), (2000, 4096, "gelu")])
def test_a_bias_gradient_alone_reports_bad_counts(M, rows, N, act):
    # only the activation's pass runs: it reports what the products report, and nothing where the counts fit
    dy = torch.randn(rows, N // 2 if act == "swiglu" else N, device="cuda").to(BF)
    z = None if act == "none" else torch.randn(rows, N, device="cuda").to(BF)
    w = torch.zeros(4, N, 64, dtype=BF, device="cuda")
    ws = M.new_workspace_linear(rows, N, 64, 4, act)
    db = torch.empty(4, N, device="cuda")
    n = rows // 4
    bad = [[n, n, -1, 0], [n, n, n, 3 * n], [rows + 1, 0, 0, 0], [0, 0, 0, -7], [rows, 1, 0, 0], [2 ** 31 - 1, 2 ** 31 - 1, 7, 0]]
    good = [[n // 2, 0, n, 1], [rows, 0, 0, 0], [0, 0, 0, rows], [0, 0, 0, 0], [rows - 1, 0, 0, 0]]
    for counts, want in [(c, M.ERR_DEVICE_INDEX) for c in bad] + [(c, M.OK) for c in good]:
        c = torch.tensor(counts, dtype=torch.int32, device="cuda")
        M.linear_backward(dy, None, w, ws, dbias=db, act=act, z=z, expert_counts=c, align=8)
        assert M.get_error(ws) == want, counts
        # the same as with the products
        M.linear_backward(dy, dy.new_zeros(rows, 64), w, ws, dw=torch.empty_like(w), act=act, z=z, expert_counts=c, align=8)
        assert M.get_error(ws) == want, counts


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("rows,counts,align,N,K", [
    (1, None, 0, 4096, 1000), (7, None, 0, 16, 8), (200, None, 0, 4096, 2048), (300, None, 0, 528, 328), (129, None, 0, 272, 4096),
    (4109, None, 0, 2064, 1544), (2500, None, 0, 4096, 64), (0, [3, 0, 130, 1], 16, 144, 200), (0, [20, 0, 9], 64, 4096, 72),
    (0, [1500, 0, 2, 1], 1, 176, 1032), (0, [700, 3, 90, 513, 256, 31], 32, 2064, 1544),
    (0, [310, 200, 0, 513, 256, 333, 640, 301], 16, 4096, 9640)])
def test_a_residual_in_place(M, dt, rows, counts, align, N, K):
    # the residual may be the output itself: the bits are those of a residual of its own
    E = len(counts) if counts else 0
    rows = rows or sum(-(-c // align) * align for c in counts) + 3
    g = torch.Generator(device="cuda").manual_seed(rows + N)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dt)
    x, w = rand(rows, K), rand(*((E, N, K) if E else (N, K))) * K ** -0.5
    kw = dict(expert_counts=torch.tensor(counts, dtype=torch.int32, device="cuda") if E else None, align=align)
    for act in ("none", "silu", "gelu", "swiglu"):
        cols = N // 2 if act == "swiglu" else N
        ws = M.new_workspace_linear(rows, N, K, E, act)
        res, z = rand(rows, cols), torch.empty(rows, N, dtype=dt, device="cuda")
        apart, same = res.clone(), res.clone()
        M.linear(x, w, apart, ws, act=act, residual=res, z=z, **kw)
        M.linear(x, w, same, ws, act=act, residual=same, z=z, **kw)
        assert torch.equal(apart, same), act
        assert not torch.equal(apart, res)
        dres, dy = rand(rows, K), rand(rows, cols)
        dx, dsame = dres.clone(), dres.clone()
        zz = None if act == "none" else z
        M.linear_backward(dy, None, w, ws, dx=dx, act=act, z=zz, dx_residual=dres, **kw)
        M.linear_backward(dy, None, w, ws, dx=dsame, act=act, z=zz, dx_residual=dsame, **kw)
        assert torch.equal(dx, dsame), act
        assert M.get_error(ws) == M.OK


def sample(rows, n=300):
    return [slice(0, n), slice(rows // 2, rows // 2 + n), slice(rows - n, rows)]


@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_outputs_beyond_32_bit_offsets(M, act):
    # y, z, the residual and dx with more than 2^31 elements
    rows, N, K, dt = 270_003, 8192, 64, BF
    g = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=dt)
    cols = N // 2 if act == "swiglu" else N
    x, w, bias, res = rand(rows, K), rand(N, K) * K ** -0.5, torch.randn(N, generator=g, device="cuda"), rand(rows, cols)
    ws = M.new_workspace_linear(rows, N, K, 0, "none")
    y, z = torch.empty(rows, cols, dtype=dt, device="cuda"), torch.empty(rows, N, dtype=dt, device="cuda")
    M.linear(x, w, y, ws, bias=bias, act=act, residual=res, z=z)
    for s in sample(rows):
        yr, ey, zr, ez = R.linear(x[s], w, bias, act, res[s], dt)
        R.check(y[s], yr.cpu(), ey.cpu(), "y")
        R.check(z[s], zr.cpu(), ez.cpu(), "z")
    assert M.get_error(ws) == M.OK


def test_input_and_weight_gradients_beyond_32_bit_offsets(M):
    rows, N, K, dt = 270_003, 64, 8192, BF
    g = torch.Generator(device="cuda").manual_seed(2)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=dt)
    x, w, dy = rand(rows, K), rand(N, K), rand(rows, N)
    ws = M.new_workspace_linear(rows, N, K)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty(N, device="cuda")
    M.linear_backward(dy, x, w, ws, dx=dx, dw=dw, dbias=db, dx_residual=x)
    for s in sample(rows):
        (a, ea), _, _ = R.linear_grad(dy[s], x[s], w, None, "none", x[s], dt)
        R.check(dx[s], a.cpu(), ea.cpu(), "dx")
    ref, bound = torch.zeros(N, K, dtype=R.F64, device="cuda"), torch.zeros(N, K, dtype=R.F64, device="cuda")
    for r in range(0, rows, 30_000):
        d, v = dy[r:r + 30_000].double(), x[r:r + 30_000].double()
        ref += d.t() @ v
        bound += d.abs().t() @ v.abs()
    h = R.half_step(dt)
    bound *= R.mma_err(rows)
    R.check(dw, ref.cpu(), (bound + h * (ref.abs() + bound) + R.tiny(dt)).cpu(), "dw")
    assert M.get_error(ws) == M.OK


def test_expert_weights_beyond_32_bit_offsets(M):
    E, N, K, dt = 40, 8192, 6656, BF                    # 2.18e9 weights
    counts = [0] * E
    counts[0], counts[1], counts[E - 2], counts[E - 1] = 70, 300, 1, 200
    rows = sum(-(-c // 8) * 8 for c in counts)
    g = torch.Generator(device="cuda").manual_seed(3)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=dt)
    x, w, bias, dy = rand(rows, K), rand(E, N, K), torch.randn(E, N, generator=g, device="cuda"), rand(rows, N)
    w *= K ** -0.5
    kw = dict(expert_counts=torch.tensor(counts, dtype=torch.int32, device="cuda"), align=8)
    ws = M.new_workspace_linear(rows, N, K, E)
    y, dx = torch.zeros(rows, N, dtype=dt, device="cuda"), torch.zeros(rows, K, dtype=dt, device="cuda")
    dw, db = torch.full_like(w, 3), torch.empty(E, N, device="cuda")
    M.linear(x, w, y, ws, bias=bias, **kw)
    M.linear_backward(dy, x, w, ws, dx=dx, dw=dw, dbias=db, **kw)
    assert M.get_error(ws) == M.OK
    for e, r, c in R.segments(counts, 8, rows):
        s = slice(r, r + c)
        if c == 0:
            assert (dw[e] == 0).all() and (db[e] == 0).all()
            continue
        yr, ey, _, _ = R.linear(x[s], w[e], bias[e], "none", None, dt)
        R.check(y[s], yr.cpu(), ey.cpu(), f"y of expert {e}")
        (a, ea), (b, eb), (v, ev) = R.linear_grad(dy[s], x[s], w[e], None, "none", None, dt)
        for got, ref, bound, n in ((dx[s], a, ea, "dx"), (dw[e], b, eb, "dw"), (db[e], v, ev, "dbias")):
            R.check(got, ref.cpu(), bound.cpu(), f"{n} of expert {e}")


@pytest.mark.parametrize("counts,align,N,K,act", [
    ([20, 0, 9], 16, 64, 4096, "silu"), ([33, 1, 0, 64, 500, 7, 0, 2], 8, 320, 1400, "swiglu"), ([1500, 0, 2, 1], 1, 176, 1032, "relu"),
    ([500, 610, 0, 433, 256, 512, 1, 300, 470, 555, 128, 390], 32, 1536, 648, "gelu"),
    ([310, 200, 0, 513, 256, 333, 640, 301], 16, 4096, 9640, "swiglu"), ([4109], 1, 2064, 1544, "none")])
def test_experts_in_fp16(M, counts, align, N, K, act):
    E, dt = len(counts), HF
    rows = sum(-(-c // align) * align for c in counts)
    g = torch.Generator(device="cuda").manual_seed(rows + N)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")
    cols = N // 2 if act == "swiglu" else N
    x, w, bias, res = rand(rows, K).to(dt), (rand(E, N, K) * K ** -0.5).to(dt), rand(E, N), rand(rows, cols).to(dt)
    dy, dres = rand(rows, cols).to(dt), rand(rows, K).to(dt)
    live = torch.zeros(rows, dtype=torch.bool, device="cuda")
    for _, r, c in R.segments(counts, align, rows):
        live[r:r + c] = True
    for t in (x, res, dy, dres):
        t[~live] = float("nan")
    kw = dict(act=act, expert_counts=torch.tensor(counts, dtype=torch.int32, device="cuda"), align=align)
    ws = M.new_workspace_linear(rows, N, K, E, act)
    y, z = torch.empty(rows, cols, dtype=dt, device="cuda"), torch.zeros(rows, N, dtype=dt, device="cuda")
    M.linear(x, w, y, ws, bias=bias, residual=res, z=z, **kw)
    dx, dw, db = torch.empty(rows, K, dtype=dt, device="cuda"), torch.empty_like(w), torch.empty(E, N, device="cuda")
    M.linear_backward(dy, x, w, ws, dx=dx, dw=dw, dbias=db, z=None if act == "none" else z, dx_residual=dres, **kw)
    assert M.get_error(ws) == M.OK
    for e, r, c in R.segments(counts, align, rows):
        s = slice(r, r + c)
        yr, ey, zr, ez = R.linear(x[s], w[e], bias[e], act, res[s], dt)
        R.check(y[s], yr.cpu(), ey.cpu(), f"y of expert {e}")
        R.check(z[s], zr.cpu(), ez.cpu(), f"z of expert {e}")
        (a, ea), (b, eb), (v, ev) = R.linear_grad(dy[s], x[s], w[e], z[s], act, dres[s], dt)
        for got, ref, bound, n in ((dx[s], a, ea, "dx"), (dw[e], b, eb, "dw"), (db[e], v, ev, "dbias")):
            R.check(got, ref.cpu(), bound.cpu(), f"{n} of expert {e}")


def test_range_of_dz(M):
    # dz is an operand of the products in the rows' type: past its range it is infinite, the bias' sum (in fp32) is not
    N, K = 64, 64
    z = torch.ones(8, N)
    dy = torch.full((8, N // 2), 400.0)
    z[:, N // 2:] = 400.0
    w = torch.full((N, K), 2.0 ** -12)
    for dt, finite in ((HF, False), (BF, True)):
        ws = M.new_workspace_linear(8, N, K, 0, "swiglu")
        dx, db = torch.empty(8, K, dtype=dt, device="cuda"), torch.empty(N, device="cuda")
        M.linear_backward(dy.to(dt).cuda(), None, w.to(dt).cuda(), ws, dx=dx, dbias=db, act="swiglu", z=z.to(dt).cuda())
        assert bool(torch.isfinite(dx).all()) == finite
        s = 1 / (1 + 2.718281828459045 ** -1)
        ref = torch.cat([torch.full((N // 2,), 8 * 160000.0 * (s + s * (1 - s))), torch.full((N // 2,), 8 * 400.0 * s)]).double()
        R.check(db, ref, 2.0 ** -16 * ref, "dbias")
