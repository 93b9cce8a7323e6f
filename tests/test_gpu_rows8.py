"""Rows in 8 bits and the linear layer's gradients from them, against float64 and against the 16-bit call."""
import pytest
import torch

import around_ref as A
import train_ref as R
from gpu_util import ensure_lib

pytestmark = pytest.mark.gpu

BF, HF, FP = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def M():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return ensure_lib()


def values(n, c, dt, seed):
    """Rows whose groups differ by many powers of two, zeros, subnormals and the type's largest values among them."""
    g = torch.Generator().manual_seed(seed)
    v = torch.randn(n, c, generator=g, dtype=torch.float64) * 2.0 ** torch.randint(-12, 12, (n, -(-c // 32)), generator=g).double(
    ).repeat_interleave(32, 1)[:, :c]
    v[0, :] = 0
    f = torch.finfo(dt)
    if n > 3:
        v[1] = torch.linspace(-1, 1, c) * f.max
        v[2] = torch.linspace(-1, 1, c) * f.tiny
        v[3, ::3] = f.smallest_normal * f.eps
        v[3, 1::3] = 448.0
    return v.clamp(-f.max, f.max).to(dt)


CASES = [(1, 7168, BF, 0), (5, 128, FP, 0), (7, 1, HF, 0), (33, 129, BF, 3), (64, 1000, HF, 0), (9, 264, FP, 4), (200, 40, BF, 0),
         (12, 2001, BF, 0), (6, 515, FP, 0), (70, 384, HF, 8), (4, 20000, BF, 0), (1000, 64, BF, 0), (301, 520, BF, 0)]


@pytest.mark.parametrize("n,c,dt,pitch", CASES)
def test_pack_and_unpack(M, n, c, dt, pitch):
    x = values(n, c, dt, n + c)
    wide = torch.full((n, c + pitch), float("nan"), dtype=dt, device="cuda")
    wide[:, :c] = x.cuda()
    q, sf = A.pack8(x)
    for qp, sp in ((0, 0), (8, 0), (3, 2)):
        qd = torch.full((n, c + qp), 0x55, dtype=torch.uint8, device="cuda")
        sd = torch.full((n, sf.shape[1] + sp), 0x55, dtype=torch.uint8, device="cuda")
        x8 = (qd[:, :c], sd[:, :sf.shape[1]])
        M.pack_rows8(wide[:, :c], x8)
        assert torch.equal(x8[1].cpu(), sf)
        assert torch.equal(A.values8(x8[0].cpu(), sf), A.values8(q, sf))
        assert (qd[:, c:] == 0x55).all() and (sd[:, sf.shape[1]:] == 0x55).all()
        for to in (BF, HF, FP):
            out = torch.full((n, c + pitch), 7.25, dtype=to, device="cuda")
            M.unpack_rows8(x8, out[:, :c])
            assert torch.equal(out[:, :c].cpu(), A.unpacked(q, sf, to)), to
            assert (out[:, c:] == 7.25).all()
    # a value's own type holds it exactly
    assert torch.equal(A.unpacked(q, sf, dt).double(), A.values8(q, sf).clamp(-A.largest(dt), A.largest(dt)))


def test_what_is_not_finite(M):
    x = torch.ones(2, 256, device="cuda", dtype=BF)
    x[0, 3], x[0, 4], x[0, 5], x[1] = float("inf"), -float("inf"), float("nan"), float("nan")
    x8 = M.new_rows8(2, 256)
    M.pack_rows8(x, x8)
    out = torch.empty_like(x)
    M.unpack_rows8(x8, out)
    assert torch.isnan(out[0, 3:6]).all() and (out[0, 6:] == 1).all() and (out[0, :3] == 1).all() and torch.isnan(out[1]).all()
    assert (x8[1][1] == 127).all()


@pytest.mark.parametrize("counts,align,c", [([3, 0, 130, 1], 16, 200), ([0, 0, 5], 1, 64), ([300, 17, 0, 64], 128, 136),
                                            ([0, 0], 64, 80), ([1] * 40, 16, 96)])
def test_rows_of_experts(M, counts, align, c):
    U = sum(-(-n // align) * align for n in counts) + 5
    x = torch.randn(U, c, generator=torch.Generator().manual_seed(U)).to(BF)
    live = torch.zeros(U, dtype=torch.bool)
    for _, r, n in R.segments(counts, align, U):
        live[r:r + n] = True
    xd, cd = x.cuda(), torch.tensor(counts, dtype=torch.int32, device="cuda")
    xd[~live.cuda()] = float("nan")
    x8 = (torch.full((U, c), 0x55, dtype=torch.uint8, device="cuda"), torch.full((U, -(-c // 128)), 0x55, dtype=torch.uint8, device="cuda"))
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    M.pack_rows8(xd, x8, expert_counts=cd, align=align, ws=ws)
    q, sf = A.pack8(x)
    assert torch.equal(x8[1].cpu()[live], sf[live]) and torch.equal(A.values8(*(t.cpu()[live] for t in x8)), A.values8(q[live], sf[live]))
    assert (x8[0].cpu()[~live] == 0x55).all() and (x8[1].cpu()[~live] == 0x55).all()
    out = torch.full((U, c), 7.25, dtype=BF, device="cuda")
    M.unpack_rows8(x8, out, expert_counts=cd, align=align, ws=ws)
    ref = torch.full((U, c), 7.25, dtype=BF)
    ref[live] = A.unpacked(q, sf, BF)[live]
    assert torch.equal(out.cpu(), ref)
    # through an index, three sorted rows to a token row; ids on padding rows are never read
    ids = torch.randint(0, 3 * U, (U,), generator=torch.Generator().manual_seed(1), dtype=torch.int32)
    M.pack_rows8(x.cuda(), x8)
    ids[~live] = 3 * U
    M.unpack_rows8(x8, out, x_ids=ids.cuda(), x_div=3, expert_counts=cd, align=align, ws=ws)
    ref[live] = A.unpacked(q, sf, BF)[ids[live].long() // 3]
    assert torch.equal(out.cpu(), ref)
    assert M.get_error(ws) == M.OK
    if live.any():
        first = int(live.nonzero()[0])
        for bad in (-1, 3 * U):
            ids[first] = bad
            M.unpack_rows8(x8, out, x_ids=ids.cuda(), x_div=3, expert_counts=cd, align=align, ws=ws)
            assert (out[first] == 0).all()
            assert M.get_error(ws) == M.ERR_DEVICE_INDEX


def test_counts_that_leave_the_buffer_are_reported(M):
    x, ws = torch.ones(8, 64, device="cuda", dtype=BF), torch.zeros(256, dtype=torch.uint8, device="cuda")
    x8 = (torch.zeros(8, 64, dtype=torch.uint8, device="cuda"), torch.zeros(8, 1, dtype=torch.uint8, device="cuda"))
    for bad in ([4, 5], [-1, 4], [100, 1]):
        M.pack_rows8(x, x8, expert_counts=torch.tensor(bad, dtype=torch.int32, device="cuda"), align=4, ws=ws)
        assert M.get_error(ws) == M.ERR_DEVICE_INDEX


# rows or counts, align, N, K
LINEAR = [(1, 0, 64, 64), (7, 0, 8, 8), (31, 0, 144, 264), (129, 0, 272, 1032), (300, 0, 528, 328), (1000, 0, 784, 200),
          (2500, 0, 640, 448), ([3, 0, 130, 1], 16, 144, 200), ([0, 0, 5], 1, 64, 64), ([300, 17, 256, 0, 64], 128, 272, 136),
          ([0, 0], 64, 80, 80), ([1] * 40, 16, 96, 128), ([700, 3, 90], 1, 528, 264)]
ACTS = ["none", "relu", "silu", "gelu", "swiglu"]


@pytest.mark.parametrize("i", range(len(LINEAR)))
@pytest.mark.parametrize("dt", [BF, HF])
def test_linear_gradients_from_8_bits(M, i, dt):
    counts, align, N, K = LINEAR[i]
    E = 0 if isinstance(counts, int) else len(counts)
    rows = sum(-(-n // align) * align for n in counts) + 3 if E else counts
    segs = R.segments(counts if E else None, align, rows)
    g = torch.Generator().manual_seed(i)
    live = torch.zeros(rows, dtype=torch.bool)
    for _, r, n in segs:
        live[r:r + n] = True
    w = (torch.randn(max(E, 1), N, K, generator=g) * K ** -0.5).to(dt)
    wd = (w if E else w[0]).contiguous().cuda()
    cd = torch.tensor(counts, dtype=torch.int32, device="cuda") if E else None
    for act in (ACTS if i in (2, 9) else [ACTS[i % 5], "swiglu"]):
        if act == "swiglu" and N % 16:
            continue
        cols = N // 2 if act == "swiglu" else N
        dy = torch.randn(rows, cols, generator=g).to(dt)
        for div in (0, 1, 3):
            tokens = rows if not div else max(1, rows // div)
            x8 = tuple(t.cuda() for t in A.pack8(torch.randn(tokens, K, generator=g).to(dt)))
            z8 = tuple(t.cuda() for t in A.pack8(torch.randn(rows, N, generator=g).to(dt))) if act != "none" else None
            ids = torch.randint(0, tokens * max(div, 1), (rows,), generator=g, dtype=torch.int32)
            if not div:
                ids = torch.arange(rows, dtype=torch.int32)
            x = A.unpacked(*(t.cpu() for t in x8), dt)[ids.long() // max(div, 1)]
            z = None if z8 is None else A.unpacked(*(t.cpu() for t in z8), dt)
            res = torch.randn(rows, K, generator=g).to(dt)
            dyd, resd = dy.cuda(), res.cuda()
            dyd[~live.cuda()] = float("nan")
            ids[~live] = -5
            ws = M.new_workspace_linear8(rows, N, K, E, act)
            kw = dict(act=act, expert_counts=cd, align=align, dx_residual=resd)
            idx = dict(x_ids=ids.cuda(), x_div=div) if div else {}

            def out():
                return (torch.full((rows, K), 7.25, dtype=dt, device="cuda"), torch.empty_like(wd),
                        torch.empty((E, N) if E else (N,), device="cuda"))

            a, b = out(), out()
            M.linear_backward8(dyd, wd, ws, x8=x8, z8=z8, dx=a[0], dw=a[1], dbias=a[2], **idx, **kw)
            # the 16-bit call on the unpacked rows: the same bits
            M.linear_backward(dyd, x.cuda(), wd, ws, z=None if z is None else z.cuda(), dx=b[0], dw=b[1], dbias=b[2], **kw)
            for u, v, name in zip(a, b, ("dx", "dw", "dbias")):
                assert torch.equal(u, v), (name, act, div)
            if div == 1:          # one of the two in 16 bits
                c = out()
                M.linear_backward8(dyd, wd, ws, x=x.cuda(), z8=z8, dx=c[0], dw=c[1], dbias=c[2], **kw)
                assert all(torch.equal(u, v) for u, v in zip(c, b))
                M.linear_backward8(dyd, wd, ws, x8=x8, z=None if z is None else z.cuda(), dw=c[1], act=act, expert_counts=cd,
                                   align=align, **idx)
                assert torch.equal(c[1], b[1])
            assert M.get_error(ws) == M.OK
            for e, r, n in segs:
                s = slice(r, r + n)
                (dx, ex), (dw, ew), (db, eb) = R.linear_grad(dy[s], x[s], w[e], None if z is None else z[s], act, res[s], dt)
                R.check(a[0][s], dx, ex, "dx")
                R.check(a[1][e] if E else a[1], dw, ew, "dw")
                R.check(a[2][e] if E else a[2], db, eb, "dbias")
            assert (a[0].cpu()[~live] == 7.25).all()


def test_a_bad_id_counts_as_a_row_of_zeros(M):
    g = torch.Generator().manual_seed(1)
    x = torch.randn(4, 64, generator=g).to(BF)
    x8 = tuple(t.cuda() for t in A.pack8(x))
    dy, w = torch.randn(6, 32, generator=g).to(BF).cuda(), torch.randn(32, 64, generator=g).to(BF).cuda()
    ws = M.new_workspace_linear8(6, 32, 64)
    dw, ref = torch.empty_like(w), torch.empty_like(w)
    M.linear_backward8(dy, w, ws, x8=x8, x_ids=torch.tensor([0, 1, 9, 3, -2, 2], dtype=torch.int32, device="cuda"), dw=dw)
    assert M.get_error(ws) == M.ERR_DEVICE_INDEX
    rows = A.unpacked(*(t.cpu() for t in x8), BF)[[0, 1, 0, 3, 0, 2]]
    rows[2] = rows[4] = 0
    M.linear_backward(dy, rows.cuda(), w, ws, dw=ref)
    assert torch.equal(dw, ref) and M.get_error(ws) == M.OK
