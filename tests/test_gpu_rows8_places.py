"""The linear layer's gradients from 8-bit rows wherever those start: codes off 8-byte boundaries, pitches, fewer scales between
rows than a row has.  Equal, bit for bit, to the same call with contiguous 8-bit rows and to the 16-bit call."""
import pytest
import torch

import around_ref as A
import train_ref as R
from gpu_util import ensure_lib

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def M():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return ensure_lib()


def placed(q, sf, start, pitch, spitch):
    """The same rows in wider buffers, from column `start` on."""
    n, c = q.shape
    wide = torch.full((n, c + start + pitch), 0x7F, dtype=torch.uint8, device="cuda")
    scales = torch.full((n, sf.shape[1] + spitch), 255, dtype=torch.uint8, device="cuda")
    wide[:, start:start + c] = q.cuda()
    scales[:, :sf.shape[1]] = sf.cuda()
    return wide[:, start:start + c], scales[:, :sf.shape[1]]


@pytest.mark.parametrize("act", ["relu", "silu", "gelu", "swiglu"])
@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("counts,align,N,K", [(70, 0, 144, 264), (333, 0, 272, 136), ([40, 0, 130, 1], 16, 144, 200)])
def test_codes_anywhere(M, act, dt, counts, align, N, K):
    E = 0 if isinstance(counts, int) else len(counts)
    rows = sum(-(-n // align) * align for n in counts) + 3 if E else counts
    segs = R.segments(counts if E else None, align, rows)
    live = torch.zeros(rows, dtype=torch.bool)
    for _, r, n in segs:
        live[r:r + n] = True
    g = torch.Generator().manual_seed(N + K)
    tokens = rows // 2
    xq, zq = A.pack8(torch.randn(tokens, K, generator=g).to(dt)), A.pack8(torch.randn(rows, N, generator=g).to(dt))
    ids = torch.randint(0, 2 * tokens, (rows,), generator=g, dtype=torch.int32)
    cols = N // 2 if act == "swiglu" else N
    dy = torch.randn(rows, cols, generator=g).to(dt).cuda()
    w = (torch.randn(max(E, 1), N, K, generator=g) * K ** -0.5).to(dt)
    wd = (w if E else w[0]).contiguous().cuda()
    kw = dict(act=act, expert_counts=torch.tensor(counts, dtype=torch.int32, device="cuda") if E else None, align=align)
    ws = M.new_workspace_linear8(rows, N, K, E, act)

    def out():
        return torch.full((rows, K), 7.25, dtype=dt, device="cuda"), torch.empty_like(wd), torch.empty(wd.shape[:-1], device="cuda")

    ref = out()
    x, z = A.unpacked(*xq, dt)[ids.long() // 2], A.unpacked(*zq, dt)
    M.linear_backward(dy, x.cuda(), wd, ws, z=z.cuda(), dx=ref[0], dw=ref[1], dbias=ref[2], **kw)
    no_bias = out()
    M.linear_backward(dy, x.cuda(), wd, ws, z=z.cuda(), dx=no_bias[0], dw=no_bias[1], **kw)
    for start, pitch, spitch in ((0, 0, 0), (1, 0, 0), (3, 4, 1), (8, 0, 2), (4, 4, 0), (0, 5, 3)):
        x8, z8 = placed(*xq, start, pitch, spitch), placed(*zq, start, pitch, spitch)
        o = out()
        M.linear_backward8(dy, wd, ws, x8=x8, z8=z8, x_ids=ids.cuda(), x_div=2, dx=o[0], dw=o[1], dbias=o[2], **kw)
        assert all(torch.equal(u, v) for u, v in zip(o, ref)), (start, pitch)
        o = out()
        M.linear_backward8(dy, wd, ws, x8=x8, z8=z8, x_ids=ids.cuda(), x_div=2, dx=o[0], dw=o[1], **kw)
        assert all(torch.equal(u, v) for u, v in zip(o[:2], no_bias[:2])), (start, pitch, "without a bias")
    assert M.get_error(ws) == M.OK
    for e, r, n in segs:
        s = slice(r, r + n)
        (dx, ex), (dw, ew), (db, eb) = R.linear_grad(dy.cpu()[s], x[s], w[e], z[s], act, None, dt)
        R.check(ref[0][s], dx, ex, "dx")
        R.check(ref[1][e] if E else ref[1], dw, ew, "dw")
        R.check(ref[2][e] if E else ref[2], db, eb, "dbias")
    assert (ref[0].cpu()[~live] == 7.25).all()


@pytest.mark.parametrize("dt", [BF, HF])
def test_pack_and_unpack_anywhere(M, dt):
    for n, c in ((37, 264), (130, 1000), (5, 2521)):
        x = torch.randn(n, c, generator=torch.Generator().manual_seed(c)).to(dt)
        q, sf = A.pack8(x)
        for start, pitch, spitch in ((1, 0, 0), (3, 4, 1), (8, 0, 2), (5, 2, 0)):
            x8 = placed(torch.zeros_like(q), torch.zeros_like(sf), start, pitch, spitch)
            M.pack_rows8(x.cuda(), x8)
            assert torch.equal(x8[1].cpu(), sf) and torch.equal(A.values8(x8[0].cpu(), sf), A.values8(q, sf))
            out = torch.empty(n, c, dtype=dt, device="cuda")
            M.unpack_rows8(x8, out)
            assert torch.equal(out.cpu(), A.unpacked(q, sf, dt))
