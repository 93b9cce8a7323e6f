"""Dispatch, combine, their gradients and the router gradient against float64."""
import numpy as np
import pytest
import torch

import train_ref as R
from gpu_util import ensure_lib
from oracle import moe as O

pytestmark = pytest.mark.gpu

BF, HF, FP = torch.bfloat16, torch.float16, torch.float32
SENTINEL = 7.25      # exact in every type; marks what a call must not write


@pytest.fixture(scope="module")
def M():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return ensure_lib()


def routing(T, E, K, seed, skew=0.0):
    g = torch.Generator().manual_seed(seed)
    keys = torch.rand(T, E, generator=g) + skew * torch.linspace(1, 0, E)
    ids = keys.topk(K, 1).indices.to(torch.int32)
    w = torch.rand(T, K, generator=g) + 0.05
    return ids, w


def rows(n, H, dt, seed, pitch=0):
    """A [n, H] CPU matrix and its CUDA copy, the latter a slice of a wider buffer when pitch > H."""
    v = torch.randn(n, H, generator=torch.Generator().manual_seed(seed)).to(dt)
    if not pitch:
        return v, v.cuda()
    wide = torch.full((n, pitch), SENTINEL, dtype=dt, device="cuda")
    wide[:, :H] = v.cuda()
    return v, wide[:, :H]


CASES = [  # T, H, E, K, align, dtype, extra pitch
    (1, 7168, 256, 6, 16, BF, 0), (8, 7168, 256, 6, 16, BF, 8), (3, 1, 2, 1, 1, FP, 0), (5, 33, 4, 4, 1, HF, 0),
    (37, 129, 7, 3, 64, BF, 3), (64, 1000, 16, 4, 128, HF, 0), (130, 24, 300, 8, 16, FP, 0), (257, 520, 16, 5, 256, FP, 4),
    (1111, 136, 16, 4, 1, HF, 0), (700, 7168, 64, 2, 32, BF, 0), (5, 264, 40, 32, 16, BF, 0), (40, 8200, 8, 3, 16, FP, 0),
    # around the borders between the ways to work the layout out (pairs and experts), wide odd rows
    (64, 72, 4, 4, 16, BF, 0), (65, 72, 256, 4, 16, BF, 0), (682, 40, 256, 6, 1, BF, 0), (683, 40, 256, 6, 64, HF, 0),
    (341, 40, 64, 6, 16, BF, 0), (342, 40, 64, 6, 16, BF, 0), (256, 24, 512, 8, 64, FP, 0), (256, 24, 513, 8, 64, FP, 0),
    (128, 24, 1024, 8, 16, FP, 0), (129, 24, 1024, 8, 16, FP, 0), (300, 3001, 16, 2, 32, HF, 0), (90, 4099, 5, 5, 8, FP, 1),
]


@pytest.mark.parametrize("T,H,E,K,align,dt,extra", CASES)
def test_dispatch_and_its_gradient(M, T, H, E, K, align, dt, extra):
    ids, _ = routing(T, E, K, T + H, skew=0.5)
    U = M.msum_upper(T, K, E, align)
    x, xd = rows(T, H, dt, 1, H + extra if extra else 0)
    xp = torch.full((U, H + extra), SENTINEL, dtype=dt, device="cuda")[:, :H]
    out = {n: torch.full((s,), -7, dtype=torch.int32, device="cuda")
           for n, s in (("sorted", U), ("experts", U), ("m_sum", 1), ("counts", E))}
    inv = torch.full((T, K), -7, dtype=torch.int32, device="cuda")
    ws = M.new_workspace_rows(T, K, E)
    M.dispatch(ids.cuda(), xd, E, align, xp, out["sorted"], out["experts"], inv, out["m_sum"], ws,
               expert_counts=out["counts"])
    assert M.get_error(ws) == M.OK
    p = O.permute(ids.numpy(), E, align)
    assert np.array_equal(inv.cpu().numpy(), p["inv_perm"])
    assert np.array_equal(out["sorted"].cpu().numpy(), p["sorted_token_ids"])
    assert np.array_equal(out["experts"].cpu().numpy(), p["expert_ids"])
    assert int(out["m_sum"]) == p["m_sum"]
    assert np.array_equal(out["counts"].cpu().numpy(), np.bincount(ids.numpy().reshape(-1), minlength=E))
    ref = torch.full((U, H), SENTINEL, dtype=dt)
    ref[inv.cpu().reshape(-1).long()] = x.repeat_interleave(K, 0)
    assert torch.equal(xp.cpu(), ref), "rows moved exactly, padding rows untouched"
    # gradient: padding rows hold NaN and must not be read; with and without a residual, and in place
    g, gd = rows(U, H, dt, 2, H + extra if extra else 0)
    pad = torch.ones(U, dtype=torch.bool)
    pad[inv.cpu().reshape(-1).long()] = False
    gd[pad.cuda()] = float("nan")
    res, resd = rows(T, H, dt, 3)
    for r in (None, res):
        ref, mag = R.combine(g, inv.cpu(), None, r)
        dx = torch.full((T, H + extra), SENTINEL, dtype=dt, device="cuda")
        M.dispatch_backward(gd, inv, dx[:, :H], ws, residual=None if r is None else resd)
        bound = R.half_step(dt) * ref.abs() * 1.01 + (K + 2) * R.U32 * mag + R.tiny(dt)
        R.check(dx[:, :H], ref, bound, "dx")
        assert (dx[:, H:] == SENTINEL).all()
    first = dx[:, :H].clone()
    M.dispatch_backward(gd, inv, resd, ws, residual=resd)
    assert torch.equal(resd, first)
    assert M.get_error(ws) == M.OK


@pytest.mark.parametrize("T,H,E,K,align,dt,extra", CASES)
def test_combine_and_its_gradients(M, T, H, E, K, align, dt, extra):
    ids, w = routing(T, E, K, T * 3 + H)
    inv, _ = R.positions(ids, E, align)
    U = M.msum_upper(T, K, E, align)
    if T > 4:
        inv[1, 0] = -1                                   # dropped pairs, one token without any row
        inv[T - 1] = -1
    y, yd = rows(U, H, dt, 4, H + extra if extra else 0)
    pad = torch.ones(U, dtype=torch.bool)
    pad[inv[inv >= 0].long()] = False
    yd[pad.cuda()] = float("nan")
    res, resd = rows(T, H, dt, 5)
    ws = M.new_workspace_rows(T, K, E)
    for ww in (w, None):
        for r in (None, res):
            ref, mag = R.combine(y, inv, ww, r)
            out = torch.full((T, H + extra), SENTINEL, dtype=dt, device="cuda")
            M.combine(yd, inv.cuda(), None if ww is None else w.cuda(), out[:, :H], ws, residual=None if r is None else resd)
            R.check(out[:, :H], ref, R.half_step(dt) * ref.abs() * 1.01 + (K + 2) * R.U32 * mag + R.tiny(dt), "out")
            assert (out[:, H:] == SENTINEL).all()
    d, dd = rows(T, H, dt, 6, H + extra if extra else 0)
    ref, dwref, mag = R.combine_grad(d, y, inv, w, U)
    dy = torch.full((U, H + extra), SENTINEL, dtype=dt, device="cuda")
    dw = torch.full((T, K), float("nan"), device="cuda")
    M.combine_backward(dd, yd, inv.cuda(), w.cuda(), dy[:, :H], dw, ws)
    live = ~pad
    R.check(dy[:, :H][live.cuda()], ref[live], (R.half_step(dt) * 1.01 + R.U32) * ref[live].abs() + R.tiny(dt), "dy")
    assert (dy[:, :H][pad.cuda()] == SENTINEL).all() and (dy[:, H:] == SENTINEL).all()
    R.check(dw, dwref, (H + 2) * R.U32 * mag + 1e-30, "dw")
    assert (dw.cpu()[inv < 0] == 0).all()
    # the rows' gradient alone gives the same rows; of the plain sum, dout's rows
    dy2 = torch.full((U, H), SENTINEL, dtype=dt, device="cuda")
    M.combine_backward(dd, None, inv.cuda(), w.cuda(), dy2, None, ws)
    assert torch.equal(dy2, dy[:, :H])
    M.combine_backward(dd, None, inv.cuda(), None, dy2, None, ws)
    assert torch.equal(dy2[int(inv[0, 0])], dd[0])
    assert M.get_error(ws) == M.OK


def at(v, off, pitch):
    """v's CUDA copy with rows `pitch` apart and row 0 `off` elements into its buffer, which ends with the last row;
    all the rest is NaN."""
    n, H = v.shape
    flat = torch.full((off + (n - 1) * pitch + H,), float("nan"), dtype=v.dtype, device="cuda")
    m = flat.as_strided((n, H), (pitch, 1), off)
    m.copy_(v)
    return flat, m


@pytest.mark.parametrize("dt", [BF, HF, FP])
@pytest.mark.parametrize("T,H,off,gap", [(70, 1, 1, 0), (70, 7, 3, 1), (70, 8, 1, 8), (70, 9, 0, 0), (70, 16, 5, 0), (70, 19, 2, 6),
                                         (70, 64, 0, 1), (70, 261, 7, 2), (3, 23, 1, 1), (700, 1027, 1, 0)])
def test_rows_at_any_alignment(M, dt, T, H, off, gap):
    # every matrix starts off its 16-byte boundary by another number of elements, has its own pitch, and NaN around it
    E, K, align = 6, 4, 8
    ids, w = routing(T, E, K, H)
    inv, _ = R.positions(ids, E, align)
    U = M.msum_upper(T, K, E, align)
    g = torch.Generator().manual_seed(H + off)
    v = {n: torch.randn(r, H, generator=g).to(dt) for n, r in (("x", T), ("d", T), ("res", T), ("y", U))}
    pad = torch.ones(U, dtype=torch.bool)
    pad[inv.reshape(-1).long()] = False
    v["y"][pad] = float("nan")
    m = {n: at(a, off + i, H + gap + i)[1] for i, (n, a) in enumerate(v.items())}
    new = lambda i, rows: at(torch.full((rows, H), SENTINEL, dtype=dt), off + i, H + gap + i)
    ws = M.new_workspace_rows(T, K, E)
    idx = [torch.empty(s, dtype=torch.int32, device="cuda") for s in (U, U, 1)]
    invd, wd = inv.cuda(), w.cuda()
    flat, xp = new(2, U)
    M.dispatch(ids.cuda(), m["x"], E, align, xp, idx[0], idx[1], torch.empty_like(invd), idx[2], ws)
    ref = torch.full((U, H), SENTINEL, dtype=dt)
    ref[inv.reshape(-1).long()] = v["x"].repeat_interleave(K, 0)
    assert torch.equal(xp.cpu(), ref)
    assert int(flat.isnan().sum()) == flat.numel() - U * H
    y = torch.where(pad[:, None], torch.zeros((), dtype=dt), v["y"])
    for ww, fn in ((w, M.combine), (None, M.dispatch_backward)):
        ref, mag = R.combine(y, inv, ww, v["res"])
        bound = R.half_step(dt) * ref.abs() * 1.01 + (K + 2) * R.U32 * mag + R.tiny(dt)
        flat, out = new(1, T)
        if ww is None:
            fn(m["y"], invd, out, ws, residual=m["res"])
        else:
            fn(m["y"], invd, wd, out, ws, residual=m["res"])
        R.check(out, ref, bound, "sum")
        assert int(flat.isnan().sum()) == flat.numel() - T * H
    ref, dwref, mag = R.combine_grad(v["d"], y, inv, w, U)
    flat, dy = new(5, U)
    dw = torch.empty(T, K, device="cuda")
    M.combine_backward(m["d"], m["y"], invd, wd, dy, dw, ws)
    R.check(dy[~pad.cuda()], ref[~pad], (R.half_step(dt) * 1.01 + R.U32) * ref[~pad].abs() + R.tiny(dt), "dy")
    R.check(dw, dwref, (H + 2) * R.U32 * mag + 1e-30, "dw")
    assert (dy[pad.cuda()] == SENTINEL).all() and int(flat.isnan().sum()) == flat.numel() - U * H
    assert M.get_error(ws) == M.OK


@pytest.mark.parametrize("dt", [BF, HF, FP])
@pytest.mark.parametrize("T,H,off,gap", [(70, 1, 1, 0), (70, 7, 3, 1), (70, 9, 0, 0), (70, 64, 0, 1), (70, 261, 7, 2), (3, 23, 1, 1),
                                         (700, 1027, 1, 0), (70, 256, 0, 0)])
def test_combine_gradient_over_the_rows_themselves(M, dt, T, H, off, gap):
    # dy_perm may be y_perm, whatever the rows' alignment; padding rows and what is between rows stay
    E, K, align = 6, 4, 8
    ids, w = routing(T, E, K, H)
    inv, _ = R.positions(ids, E, align)
    inv[0, 1] = -1
    U = M.msum_upper(T, K, E, align)
    g = torch.Generator().manual_seed(H + off)
    y, d = (torch.randn(r, H, generator=g).to(dt) for r in (U, T))
    _, dd = at(d, off + 1, H + gap)
    _, yd = at(y, off, H + gap)
    ws = M.new_workspace_rows(T, K, E)
    flat, dy = at(y, off, H + gap)
    dw, dw2 = torch.empty(T, K, device="cuda"), torch.empty(T, K, device="cuda")
    M.combine_backward(dd, yd, inv.cuda(), w.cuda(), dy, dw, ws)
    flat2, both = at(y, off, H + gap)
    M.combine_backward(dd, both, inv.cuda(), w.cuda(), both, dw2, ws)
    assert torch.equal(dw, dw2) and torch.equal(dy, both)
    assert int(flat2.isnan().sum()) == flat2.numel() - U * H
    assert M.get_error(ws) == M.OK


def test_combine_gradient_against_differences(M):
    # fp32 rows: the directional derivative of <c, combine(y, w)> by central differences of the kernel itself.
    # The function is linear in y and in w, so the difference has no truncation error, only rounding.
    T, H, E, K = 6, 96, 5, 3
    ids, w = routing(T, E, K, 11)
    inv, _ = R.positions(ids, E, 4)
    U = M.msum_upper(T, K, E, 4)
    y, c = torch.randn(U, H), torch.randn(T, H)
    vy, vw = torch.randn(U, H), torch.randn(T, K)
    ws = M.new_workspace_rows(T, K, E)
    dy, dw = torch.zeros(U, H, device="cuda"), torch.zeros(T, K, device="cuda")
    M.combine_backward(c.cuda(), y.cuda(), inv.cuda(), w.cuda(), dy, dw, ws)

    def f(yy, ww):
        out = torch.empty(T, H, device="cuda")
        M.combine(yy.cuda(), inv.cuda(), ww.cuda(), out, ws)
        return float((out.double().cpu() * c.double()).sum())

    mag = float((c.abs().double()).sum() * K * 20)       # magnitudes in the sums below
    tol = 64 * R.U32 * mag
    assert abs((f(y + vy, w) - f(y - vy, w)) / 2 - float((dy.cpu().double() * vy.double()).sum())) <= tol
    assert abs((f(y, w + vw) - f(y, w - vw)) / 2 - float((dw.cpu().double() * vw.double()).sum())) <= tol


def test_bad_rows_are_reported_and_skipped(M):
    T, H, E, K, U = 4, 64, 3, 2, 8
    inv = torch.tensor([[0, 1], [2, 99], [-5, 3], [4, 5]], dtype=torch.int32)
    y = torch.randn(U, H)
    ws = M.new_workspace_rows(T, K, E)
    out = torch.empty(T, H, device="cuda")
    M.combine(y.cuda(), inv.cuda(), None, out, ws)
    assert M.get_error(ws) == M.ERR_DEVICE_INDEX
    good = torch.where((inv >= 0) & (inv < U), inv, torch.full_like(inv, -1))
    ref, mag = R.combine(y, good, None)
    R.check(out, ref, 8 * R.U32 * mag, "out")
    dy, dw = torch.zeros(U, H, device="cuda"), torch.full((T, K), 5.0, device="cuda")
    M.combine_backward(out, y.cuda(), inv.cuda(), torch.ones(T, K, device="cuda"), dy, dw, ws)
    assert M.get_error(ws) == M.ERR_DEVICE_INDEX
    assert (dw.cpu()[good < 0] == 0).all() and (dy[6:] == 0).all()
    # an expert id out of range
    ids = torch.tensor([[0, 1], [2, 3], [0, 2], [1, 0]], dtype=torch.int32)
    n = M.msum_upper(T, K, E, 1)
    i = [torch.empty(s, dtype=torch.int32, device="cuda") for s in (n, n, 1)]
    M.dispatch(ids.cuda(), y[:T].cuda(), E, 1, torch.zeros(n, H, device="cuda"), i[0], i[1],
               torch.zeros(T, K, dtype=torch.int32, device="cuda"), i[2], ws)
    assert M.get_error(ws) == M.ERR_DEVICE_INDEX
    assert M.get_error(ws) == M.OK


def test_no_tokens(M):
    ws = M.new_workspace_rows(0, 2, 4)
    z = torch.zeros(0, 64, dtype=BF, device="cuda")
    e = torch.zeros(0, 2, dtype=torch.int32, device="cuda")
    U = M.msum_upper(0, 2, 4, 16)
    s = [torch.full((n,), 3, dtype=torch.int32, device="cuda") for n in (U, U, 1, 4)]
    M.dispatch(e, z, 4, 16, torch.zeros(U, 64, dtype=BF, device="cuda"), s[0], s[1], e, s[2], ws, expert_counts=s[3])
    assert (s[0] == 0).all() and (s[1] == -1).all() and int(s[2]) == 0 and (s[3] == 0).all()
    M.combine(torch.zeros(U, 64, dtype=BF, device="cuda"), e, None, z, ws)
    M.combine_backward(z, None, e, None, torch.zeros(U, 64, dtype=BF, device="cuda"), None, ws)
    f = torch.zeros(0, 2, device="cuda")
    M.route_backward(torch.zeros(0, 4, device="cuda"), e, f, f, "softmax", True, torch.zeros(0, 4, device="cuda"), ws)
    assert M.get_error(ws) == M.OK


def test_rows_beyond_32_bit_offsets(M):
    # row offsets past 2^31 elements: a sorted buffer of 2^31 + elements with the live rows at its end
    H, U = 65536, 32800                                   # 2.15e9 elements, 4.3 GB
    y = torch.empty(U, H, dtype=BF, device="cuda")
    last = torch.randn(2, H, device="cuda").to(BF)
    y[U - 2:] = last
    inv = torch.tensor([[U - 1, U - 2]], dtype=torch.int32, device="cuda")
    ws = M.new_workspace_rows(1, 2, 4)
    out = torch.empty(1, H, dtype=BF, device="cuda")
    w = torch.tensor([[0.5, 2.0]], device="cuda")
    M.combine(y, inv, w, out, ws)
    ref = 0.5 * last[1].double() + 2 * last[0].double()
    R.check(out[0], ref.cpu(), (R.half_step(BF) * 1.01 * ref.abs() + 4 * R.U32 * (last.double().abs().sum(0) * 2)).cpu(), "out")
    dw = torch.empty(1, 2, device="cuda")
    M.combine_backward(out, y, inv, w, y, dw, ws)          # the gradient over the rows themselves
    assert torch.equal(y[U - 2], (out[0].float() * 2).to(BF)) and torch.equal(y[U - 1], (out[0].float() * 0.5).to(BF))
    assert M.get_error(ws) == M.OK


# ------------------------------------------------------------------------------------- router gradient

@pytest.mark.parametrize("fn", ["softmax", "sqrt_softplus"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,K,dt", [(1, 256, 6, FP), (8, 256, 6, BF), (33, 4, 4, FP), (77, 1024, 8, FP), (500, 33, 1, FP),
                                      (3, 1, 1, FP), (20, 70, 32, HF), (2049, 64, 6, FP)])
def test_route_gradient(M, fn, renorm, T, E, K, dt):
    g = torch.Generator().manual_seed(T + E + K)
    logits = torch.randn(T, E, generator=g) * 3
    ids = torch.rand(T, E, generator=g).topk(K, 1).indices.to(torch.int32)       # any selection, not only the best
    w = R.route_weights(logits, ids, fn, renorm).float()
    dw = torch.randn(T, K, generator=g)
    ref = R.route_grad(logits, ids, dw, fn, renorm)
    ws = M.new_workspace_rows(T, K, E)
    out = torch.full((T, E), float("nan"), dtype=dt, device="cuda")
    M.route_backward(logits.cuda(), ids.cuda(), w.cuda(), dw.cuda(), fn, renorm, out, ws)
    assert M.get_error(ws) == M.OK
    terms = (w.double() * dw.double()).abs()
    scale = terms + w.double() * terms.sum(1, keepdim=True)          # what each w (dw - c) is made of
    bound = torch.zeros(T, E, dtype=R.F64).scatter_(1, ids.long(), scale)
    if fn == "softmax":
        bound = bound + torch.softmax(logits.double(), 1) * terms.sum(1, keepdim=True)
    # sums of up to E terms, an exponential whose argument is off by |l| half steps, about 64 roundings in all
    bound = bound * (E + 64 + 2 * logits.abs().max()) * R.U32
    R.check(out, ref, bound + R.half_step(dt) * ref.abs() * 1.01 + R.tiny(dt), "dlogits")


@pytest.mark.parametrize("T,E,K,dt", [(64, 256, 6, FP), (64, 64, 8, BF), (64, 33, 5, FP), (64, 5, 5, FP), (64, 1024, 32, HF),
                                      (64, 256, 1, FP)])
def test_route_gradient_of_one_likely_expert(M, T, E, K, dt):
    # softmax weights as they are, one logit 4 to 67 above the rest: a selected expert's gradient is
    # w_k ((1 - p_k) dw_k - sum of the other w_j dw_j), held to the magnitudes of these terms, which are as small as 1 - p_k
    g = torch.Generator().manual_seed(T + E + K)
    logits = torch.randn(T, E, generator=g)
    top = torch.randint(0, E, (T, 1), generator=g)
    logits.scatter_(1, top, torch.arange(T)[:, None] + 4.0)
    keys = torch.rand(T, E, generator=g)
    keys[: T - 8].scatter_(1, top[: T - 8], 2.0)             # (in the last rows it may be left out)
    ids = keys.topk(K, 1).indices.to(torch.int32)
    w = R.route_weights(logits, ids, "softmax", False)
    dw = torch.randn(T, K, generator=g)
    p = torch.softmax(logits.double(), 1)
    x = torch.exp(logits.double() - logits.double().amax(1, keepdim=True))
    rest = torch.stack([x[:, :e].sum(1) + x[:, e + 1:].sum(1) for e in range(E)], 1) / x.sum(1, keepdim=True)   # 1 - p
    q = rest.gather(1, ids.long())
    terms = w * dw.double()
    others = torch.stack([terms[:, :k].sum(1) + terms[:, k + 1:].sum(1) for k in range(K)], 1)
    others_abs = torch.stack([terms[:, :k].abs().sum(1) + terms[:, k + 1:].abs().sum(1) for k in range(K)], 1)
    ref = (-p * terms.sum(1, keepdim=True)).scatter(1, ids.long(), terms * q - w * others)
    mag = (p * terms.abs().sum(1, keepdim=True)).scatter(1, ids.long(), terms.abs() * q + w * others_abs)
    ws = M.new_workspace_rows(T, K, E)
    out = torch.full((T, E), float("nan"), dtype=dt, device="cuda")
    M.route_backward(logits.cuda(), ids.cuda(), w.float().cuda(), dw.cuda(), "softmax", False, out, ws)
    assert M.get_error(ws) == M.OK
    # sums of up to E terms, exponentials whose argument is off by |l| half steps, about 64 roundings in all; below
    # the smallest normal number, whole steps of it
    bound = mag * (E + 64 + 2 * logits.abs().max()) * R.U32 + 2.0 ** -126
    R.check(out, ref, bound + R.half_step(dt) * ref.abs() * 1.01 + R.tiny(dt), "dlogits")


def test_route_gradient_of_equal_logits(M):
    # several largest logits: none of them is left out of 1 - p
    logits = torch.tensor([[3.0, 3.0, -40.0, 3.0], [0.0, 0.0, 0.0, 0.0], [50.0, 50.0, 0.0, 49.0]])
    ids = torch.tensor([[0, 3], [2, 1], [1, 3]], dtype=torch.int32)
    w = R.route_weights(logits, ids, "softmax", False).float()
    dw = torch.tensor([[1.0, -2.0], [0.5, 0.25], [-1.0, 3.0]])
    ws = M.new_workspace_rows(3, 2, 4)
    out = torch.empty(3, 4, device="cuda")
    M.route_backward(logits.cuda(), ids.cuda(), w.cuda(), dw.cuda(), "softmax", False, out, ws)
    ref = R.route_grad(logits, ids, dw, "softmax", False)
    scale = torch.softmax(logits.double(), 1) * 4
    R.check(out, ref, scale * (64 + 100) * R.U32 + 1e-30, "dlogits")


def test_route_gradient_of_underflowing_scores(M):
    # logits so low that every sqrt(softplus) score underflows in the formula s'(l) = sigmoid / (2 s): the
    # gradient of the normalised weights is still w_k (dw_k - c) / 2; masked experts (-inf) get none
    logits = torch.tensor([[-150.0, -150.0, -160.0, float("-inf")], [-30.0, 0.0, 60.0, float("-inf")]])
    ids = torch.tensor([[0, 1], [2, 0]], dtype=torch.int32)
    l = logits.double().gather(1, ids.long())
    s = torch.where(l < -20, (l / 2).exp(), torch.nn.functional.softplus(l, threshold=1e9).sqrt())
    w = (s / s.sum(1, keepdim=True)).float()
    dw = torch.tensor([[1.0, -0.5], [0.25, 2.0]])
    ws = M.new_workspace_rows(2, 2, 4)
    out = torch.empty(2, 4, device="cuda")
    M.route_backward(logits.cuda(), ids.cuda(), w.cuda(), dw.cuda(), "sqrt_softplus", True, out, ws)
    c = (w.double() * dw.double()).sum(1, keepdim=True)
    ratio = torch.where(l < -20, torch.ones_like(l), torch.sigmoid(l) / torch.nn.functional.softplus(l, threshold=1e9))
    ref = torch.zeros(2, 4, dtype=R.F64).scatter_(1, ids.long(), w.double() * (dw.double() - c) * ratio / 2)
    part = torch.zeros(2, 4, dtype=R.F64).scatter_(1, ids.long(), w.double() * (dw.double().abs() + c.abs()) * ratio / 2)
    R.check(out, ref, 64 * R.U32 * part + 1e-30, "dlogits")
    M.route_backward(logits.cuda(), ids.cuda(), w.cuda(), dw.cuda(), "softmax", False, out, ws)
    assert torch.isfinite(out).all() and (out[:, 3] == 0).all()


def test_route_gradient_reports_bad_ids_and_adds_repeated_ones(M):
    logits = torch.randn(2, 8)
    ids = torch.tensor([[3, 3], [1, 8]], dtype=torch.int32)
    w, dw = torch.tensor([[0.5, 0.25], [0.5, 0.5]]), torch.tensor([[1.0, 2.0], [1.0, 1.0]])
    ws = M.new_workspace_rows(2, 2, 8)
    out = torch.empty(2, 8, device="cuda")
    M.route_backward(logits.cuda(), ids.cuda(), w.cuda(), dw.cuda(), "sqrt_softplus", False, out, ws)
    assert M.get_error(ws) == M.ERR_DEVICE_INDEX
    l = logits.double()
    r = torch.sigmoid(l) / torch.nn.functional.softplus(l) / 2
    assert abs(float(out[0, 3]) - float(1.0 * r[0, 3])) < 1e-5 and int((out[0] != 0).sum()) == 1
    assert abs(float(out[1, 1]) - float(0.5 * r[1, 1])) < 1e-5 and int((out[1] != 0).sum()) == 1


def test_rows_on_another_stream_and_in_a_graph(M):
    T, H, E, K, align = 50, 256, 8, 3, 16
    ids, w = routing(T, E, K, 3)
    inv, _ = R.positions(ids, E, align)
    U = M.msum_upper(T, K, E, align)
    y = torch.zeros(U, H, dtype=BF, device="cuda")
    idd, wd, invd = ids.cuda(), w.cuda(), inv.cuda()
    ws = M.new_workspace_rows(T, K, E)
    x = torch.randn(T, H, device="cuda").to(BF)
    out = torch.zeros(T, H, dtype=BF, device="cuda")
    i = [torch.zeros(n, dtype=torch.int32, device="cuda") for n in (U, U, 1)]

    def step():
        M.dispatch(idd, x, E, align, y, i[0], i[1], invd, i[2], ws)
        M.combine(y, invd, wd, out, ws, residual=x)

    step()
    torch.cuda.synchronize()
    want = out.clone()
    s = torch.cuda.Stream()
    out.zero_()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    assert torch.equal(out, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for k in range(3):
        x.copy_(torch.randn(T, H, device="cuda").to(BF))
        step()
        want = out.clone()
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert M.get_error(ws) == M.OK


def test_the_binding_refuses_wrong_tensors(M):
    T, H, E, K = 4, 64, 3, 2
    inv = torch.zeros(T, K, dtype=torch.int32, device="cuda")
    y, out = torch.zeros(8, H, device="cuda"), torch.zeros(T, H, device="cuda")
    ws = M.new_workspace_rows(T, K, E)
    with pytest.raises(TypeError, match="y_perm must have dtype"):
        M.combine(y.half(), inv, None, out, ws)
    with pytest.raises(ValueError, match="residual must have shape"):
        M.combine(y, inv, None, out, ws, residual=out[:2])
    with pytest.raises(ValueError, match="unit column stride"):
        M.combine(torch.zeros(H, 8, device="cuda").t(), inv, None, out, ws)
    with pytest.raises(ValueError, match="do not overlap"):
        M.combine(y[0].expand(8, H), inv, None, out, ws)
    with pytest.raises(ValueError, match="inv_perm must be contiguous"):
        M.combine(y, torch.zeros(K, T, dtype=torch.int32, device="cuda").t(), None, out, ws)
    with pytest.raises(ValueError, match="CUDA tensor"):
        M.combine(y, inv, torch.zeros(T, K), out, ws)
    with pytest.raises(TypeError, match="torch.Tensor"):
        M.combine(y, inv, [1.0], out, ws)
    with pytest.raises(M.MoeError):
        M.linear(y, torch.zeros(H, H, device="cuda"), torch.zeros(8, H, device="cuda"), M.new_workspace_linear(8, H, H))
