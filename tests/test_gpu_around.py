"""The norm, the routing by groups and the 8-bit rows as they are used together with the layer's calls, on streams, in
captured graphs, from two host threads, and what the binding refuses."""
import threading

import numpy as np
import pytest
import torch

import around_ref as A
import synth
import train_ref as R
from gpu_util import OUT_TOL, device_weights, ensure_lib
from oracle import formats as F
from oracle import moe as O

pytestmark = pytest.mark.gpu

BF, HF, FP = torch.bfloat16, torch.float16, torch.float32
EPS = 1e-5


@pytest.fixture(scope="module")
def M():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return ensure_lib()


@pytest.mark.parametrize("T,align", [(40, 16), (1, 16), (300, 64)])
def test_in_front_of_the_serving_layer(M, T, align):
    """norm with 8-bit rows -> gate -> select -> permute -> experts -> reduce, against the oracle on the norm's own rows."""
    w = synth.custom(T=T, H=512, I=256, E=16, K=4, align=align, seed=T)
    stack = synth.all_expert_weights(w)
    w13, w2 = device_weights(M, stack, w.fmt)
    H, I, E, K = w.H, w.I, w.E, w.K
    g = torch.Generator().manual_seed(T)
    x, res = torch.randn(T, H, generator=g).to(BF), torch.randn(T, H, generator=g).to(BF)
    nw, gate = torch.rand(H, generator=g) + 0.5, torch.randn(E, H, generator=g) * H ** -0.5
    bias = torch.randn(E, generator=g) * 0.1
    i32, dev = torch.int32, "cuda"
    s, y = torch.empty(T, H, dtype=BF, device=dev), torch.empty(T, H, dtype=BF, device=dev)
    y8 = M.new_rows8(T, H)
    M.rms_norm(x.cuda(), nw.cuda(), EPS, residual=res.cuda(), sum_out=s, y=y, y8=y8)
    ws = M.new_workspace(T, H, I, E, K, align)
    ids, tw = torch.empty(T, K, dtype=i32, device=dev), torch.empty(T, K, device=dev)
    logits = torch.empty(T, E, device=dev)
    M.route(y, gate.cuda(), None, None, K, "softmax", True, ids, tw, ws, logits_out=logits)
    rule = dict(G=4, KG=2, best=2, renorm=True, scale=2.5)
    M.select(logits, ids, tw, "sigmoid", e_score_bias=bias.cuda(), n_groups=4, topk_groups=2, scale=2.5)
    ri, rw = A.select(logits.cpu(), bias, K, "sigmoid", **rule)
    assert torch.equal(ids.cpu(), ri)
    U = M.msum_upper(T, K, E, align)
    sorted_ids, eids = torch.empty(U, dtype=i32, device=dev), torch.empty(U, dtype=i32, device=dev)
    inv, m_sum = torch.empty(T, K, dtype=i32, device=dev), torch.empty(1, dtype=i32, device=dev)
    x_perm = torch.zeros(U, H, dtype=torch.uint8, device=dev)
    x_sf = torch.zeros(M.act_sf_tiled_bytes(U, H // 128, align), dtype=torch.uint8, device=dev)
    M.permute(ids, E, align, sorted_ids, eids, inv, m_sum, ws, x_q=y8[0], x_sf=y8[1], x_perm=x_perm, x_perm_sf=x_sf)
    h_q = torch.empty(U, I, dtype=torch.uint8, device=dev)
    h_sf = torch.empty(M.act_sf_tiled_bytes(U, I // 128, align), dtype=torch.uint8, device=dev)
    y_perm, out = torch.empty(U, H, dtype=BF, device=dev), torch.empty(T, H, dtype=BF, device=dev)
    M.grouped_ffn(x_perm, x_sf, eids, m_sum, T, K, H, I, E, align, w13, w2, h_q, h_sf, y_perm, ws)
    M.unpermute_reduce(y_perm, inv, tw, out)
    assert M.get_error(ws) == M.OK
    xd = A.values8(y8[0].cpu(), y8[1].cpu()).numpy()
    ref = np.zeros((T, H))
    for e in range(E):
        t, k = np.nonzero(ri.numpy() == e)
        if not len(t):
            continue
        hq, hs = O.expert_l1_swiglu(xd[t], O.dequant_weight(stack["w13_q"][e], stack["w13_sf"][e], None, w.fmt), I)[1:]
        yr = F.bf16_to_f64(O.expert_l2(hq, hs, O.dequant_weight(stack["w2_q"][e], stack["w2_sf"][e], None, w.fmt)))
        np.add.at(ref, t, yr * rw.numpy()[t, k][:, None])
    rms = float(np.sqrt(np.mean(ref * ref)))
    assert float(np.abs(out.cpu().double().numpy() - ref).max()) <= OUT_TOL * rms


class Block:
    """norm -> gate and routing by groups -> experts with SwiGLU -> combine onto the stream, forward and backward; x and z of
    the experts' first product kept in 8 bits, x once per token."""

    def __init__(self, M, T, H=256, I=64, E=16, K=4, align=16, seed=0):
        self.M, self.T, self.H, self.I, self.E, self.K, self.align = M, T, H, I, E, K, align
        g = torch.Generator().manual_seed(seed)
        rnd = lambda *s: (torch.randn(*s, generator=g) * s[-1] ** -0.5).to(BF).cuda()        # noqa: E731
        self.nw = (torch.rand(H, generator=g) + 0.5).cuda()
        self.gate, self.w13, self.w2 = rnd(E, H), rnd(E, 2 * I, H), rnd(E, H, I)
        self.U = U = M.msum_upper(T, K, E, align)
        i32 = torch.int32
        row = lambda n, c: torch.zeros(n, c, dtype=BF, device="cuda")                          # noqa: E731
        self.s, self.y, self.out, self.dy, self.dyg, self.dx = (row(T, H) for _ in range(6))
        self.y8, self.z8 = M.new_rows8(T, H), tuple(torch.zeros_like(t) for t in M.new_rows8(U, 2 * I))
        self.logits, self.dlogits = row(T, E), row(T, E)
        self.ids, self.tw, self.dtw = torch.zeros(T, K, dtype=i32, device="cuda"), torch.zeros(T, K, device="cuda"), torch.zeros(T, K, device="cuda")
        self.sorted, self.eids = (torch.zeros(U, dtype=i32, device="cuda") for _ in range(2))
        self.inv, self.m_sum, self.counts = torch.zeros_like(self.ids), torch.zeros(1, dtype=i32, device="cuda"), torch.zeros(E, dtype=i32, device="cuda")
        self.xp, self.z, self.h, self.yp, self.dyp, self.dh, self.dxp = (row(U, c) for c in (H, 2 * I, I, H, H, I, H))
        self.grads = [torch.zeros_like(t) for t in (self.w13, self.w2, self.gate)] + [torch.zeros(H, device="cuda")]
        self.wr, self.wn = M.new_workspace_rows(T, K, E), M.new_workspace_norm(T, H)
        self.wu, self.wd = M.new_workspace_linear8(U, 2 * I, H, E, "swiglu"), M.new_workspace_linear(U, H, I, E)
        self.wg = M.new_workspace_linear(T, E, H)
        self.ws = torch.zeros(256, dtype=torch.uint8, device="cuda")

    def run(self, x, dout, unpacked=False):
        M, exp = self.M, dict(expert_counts=self.counts, align=self.align)
        M.rms_norm(x, self.nw, EPS, y=self.y, y8=self.y8)
        M.linear(self.y, self.gate, self.logits, self.wg)
        M.select(self.logits, self.ids, self.tw, "sigmoid", n_groups=4, topk_groups=2, scale=2.5)
        M.dispatch(self.ids, self.y, self.E, self.align, self.xp, self.sorted, self.eids, self.inv, self.m_sum, self.wr,
                   expert_counts=self.counts)
        M.linear(self.xp, self.w13, self.h, self.wu, act="swiglu", z=self.z, **exp)
        M.pack_rows8(self.z, self.z8, ws=self.ws, **exp)
        M.linear(self.h, self.w2, self.yp, self.wd, **exp)
        M.combine(self.yp, self.inv, self.tw, self.out, self.wr, residual=x)
        # backward
        M.combine_backward(dout, self.yp, self.inv, self.tw, self.dyp, self.dtw, self.wr)
        M.linear_backward(self.dyp, self.h, self.w2, self.wd, dx=self.dh, dw=self.grads[1], **exp)
        if unpacked:
            xr, zr = torch.zeros_like(self.xp), torch.zeros_like(self.z)
            M.unpack_rows8(self.y8, xr, x_ids=self.sorted, x_div=self.K, ws=self.ws, **exp)
            M.unpack_rows8(self.z8, zr, ws=self.ws, **exp)
            M.linear_backward(self.dh, xr, self.w13, self.wu, dx=self.dxp, dw=self.grads[0], act="swiglu", z=zr, **exp)
        else:
            M.linear_backward8(self.dh, self.w13, self.wu, x8=self.y8, x_ids=self.sorted, x_div=self.K, z8=self.z8,
                               dx=self.dxp, dw=self.grads[0], act="swiglu", **exp)
        M.dispatch_backward(self.dxp, self.inv, self.dy, self.wr)
        M.select_backward(self.logits, self.ids, self.tw, self.dtw, self.dlogits, self.wr, "sigmoid", scale=2.5)
        M.linear_backward(self.dlogits, self.y, self.gate, self.wg, dx=self.dyg, dw=self.grads[2], dx_residual=self.dy)
        M.rms_norm_backward(self.dyg, x, self.nw, EPS, self.dx, self.wn, dweight=self.grads[3], dsum=dout)
        return [self.out, self.dx, *self.grads]

    def check(self):
        assert all(self.M.get_error(w) == self.M.OK for w in (self.wr, self.wn, self.wu, self.wd, self.wg, self.ws))


def inputs(T, H, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(T, H, generator=g).to(BF).cuda(), torch.randn(T, H, generator=g).to(BF).cuda()


@pytest.mark.parametrize("T", [1, 70, 513])
def test_in_a_training_block(M, T):
    b = Block(M, T, seed=T)
    x, dout = inputs(T, b.H, T)
    got = [t.clone() for t in b.run(x, dout)]
    b.check()
    for u, v in zip(got, b.run(x, dout, unpacked=True)):
        assert torch.equal(u, v)          # the 16-bit gradients of the unpacked rows
    b.check()
    # float64, the choice as it was made: forward in full, and the stream's gradient by autograd of the same formulas
    c = lambda t: t.detach().cpu().to(R.F64)          # noqa: E731
    xr, ids = c(x).requires_grad_(), b.ids.cpu().long()
    y = xr / torch.sqrt((xr * xr).mean(1, keepdim=True) + EPS) * c(b.nw)
    w = A.select_weights(y @ c(b.gate).t(), ids, "sigmoid", True, 2.5)
    out = xr
    for e in range(b.E):
        t, k = (ids == e).nonzero(as_tuple=True)
        out = out.index_add(0, t, (R.act(y[t] @ c(b.w13[e]).t(), "swiglu") @ c(b.w2[e]).t()) * w[t, k, None])
    out.backward(c(dout))
    # out: roundings to bf16 of y, logits, h, the experts' rows and out itself, each below 2^-8 of a value: 2^-5 of the norm
    # is above their sum.  dx: the same on the way back, and z off by up to 2^-4 of each value (x only enters dw)
    rel = lambda u, v: float((c(u) - v).norm() / v.norm())      # noqa: E731
    assert rel(got[0], out.detach()) < 2.0 ** -5
    assert rel(got[1], xr.grad) < 2.0 ** -5 + 2.0 ** -4


def test_captured_and_on_another_stream(M):
    b, o = Block(M, 70, seed=3), Block(M, 70, seed=3)
    x, dout = inputs(70, b.H, 1)
    b.run(x, dout)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = b.run(x, dout)
    for seed in (2, 3):
        xn, dn = inputs(70, b.H, seed)
        x.copy_(xn)
        dout.copy_(dn)
        for t in outs:
            t.zero_()
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        g.replay()
        with torch.cuda.stream(side):
            other = o.run(xn, dn)
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(outs, other))
    b.check()


def test_two_host_threads(M):
    blocks = [Block(M, T, seed=T) for T in (33, 160)]
    data = [inputs(b.T, b.H, 5) for b in blocks]
    alone = [[t.clone() for t in b.run(*d)] for b, d in zip(blocks, data)]
    torch.cuda.synchronize()
    errors, start = [], threading.Barrier(2)

    def work(b, d):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                start.wait()
                for _ in range(20):
                    b.run(*d)
        except Exception as e:      # noqa: BLE001 (any of them fails the test)
            errors.append(e)

    threads = [threading.Thread(target=work, args=a) for a in zip(blocks, data)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    for b, ref in zip(blocks, alone):
        assert all(torch.equal(u, v) for u, v in zip([b.out, b.dx, *b.grads], ref))


def test_rows_far_apart(M):
    """Pitches that put a row's place past 2^32 bytes and 2^31 elements."""
    ld, H, T = (1 << 30) + 8, 640, 4
    far = torch.empty(ld * (T - 1) + H, dtype=BF, device="cuda")
    x, dev = torch.randn(T, H, generator=torch.Generator().manual_seed(1)).to(BF), far.as_strided((T, H), (ld, 1))
    dev.copy_(x)
    w = torch.ones(H, device="cuda")
    y, z, y8, x8 = (torch.empty(T, H, dtype=BF, device="cuda") for _ in range(2)), None, M.new_rows8(T, H), M.new_rows8(T, H)
    y, z = y
    M.rms_norm(dev, w, EPS, y=y, y8=y8)
    M.rms_norm(x.cuda(), w, EPS, y=z)
    assert torch.equal(y, z)
    M.pack_rows8(dev, x8)
    q, sf = A.pack8(x)
    assert torch.equal(x8[1].cpu(), sf) and torch.equal(A.values8(x8[0].cpu(), sf), A.values8(q, sf))
    ids, tw, i2, t2 = (torch.empty(T, 4, dtype=t, device="cuda") for t in (torch.int32, FP, torch.int32, FP))
    M.select(dev, ids, tw, "softmax")
    M.select(x.cuda(), i2, t2, "softmax")
    assert torch.equal(ids, i2) and torch.equal(tw, t2)
    back = far.as_strided((T, H), (ld, 1))
    back.zero_()
    M.unpack_rows8(x8, back)
    assert torch.equal(back.cpu(), A.unpacked(q, sf, BF))


def test_the_binding_says_what_is_wrong(M):
    x, w = torch.zeros(4, 200, dtype=BF, device="cuda"), torch.ones(200, device="cuda")
    y8 = M.new_rows8(4, 200)
    for kw, err, text in ((dict(y=x[:3]), ValueError, "y must have shape"), (dict(y=x.float()), TypeError, "y must have dtype"),
                          (dict(y=x.cpu()), ValueError, "CUDA tensor|current device"), (dict(y=[1]), (TypeError, AttributeError), "torch.Tensor|attribute"),
                          (dict(y=x.t().contiguous().t()), ValueError, "row-major"), (dict(), M.MoeError, "invalid"),
                          (dict(y8=(y8[0][:3], y8[1])), ValueError, "y8 must have shape"), (dict(y8=(y8[0], y8[1][:, :1])), ValueError, "scales"),
                          (dict(sum_out=x, y=x), M.MoeError, "invalid")):
        with pytest.raises(err, match=text):
            M.rms_norm(x, w, EPS, **kw)
    with pytest.raises(ValueError, match="weight must have shape"):
        M.rms_norm(x, w[:100], EPS, y=x)
    with pytest.raises(TypeError):
        M.rms_norm(x, w.to(BF), EPS, y=x)
    with pytest.raises(M.MoeError):
        M.rms_norm(x, w, -1.0, y=x)
    with pytest.raises(M.MoeError):          # not on a 16-byte boundary
        M.rms_norm(x, torch.ones(201, device="cuda")[1:], EPS, y=x)
    with pytest.raises(TypeError, match="bfloat16, float16 or float32"):
        M.rms_norm(x.double(), w, EPS, y=x.double())
    with pytest.raises(M.MoeError, match="workspace"):
        M.rms_norm_backward(x, x, w, EPS, x, torch.zeros(256, dtype=torch.uint8, device="cuda"))
    ids, tw = torch.zeros(4, 6, dtype=torch.int32, device="cuda"), torch.zeros(4, 6, device="cuda")
    for kw in (dict(n_groups=7), dict(n_groups=8, topk_groups=9), dict(scale=0.0), dict(group_best=3), dict(n_groups=40, topk_groups=1)):
        with pytest.raises(M.MoeError):
            M.select(x, ids, tw, "sigmoid", **kw)
    with pytest.raises(ValueError, match="e_score_bias must have shape"):
        M.select(x, ids, tw, "sigmoid", e_score_bias=w[:10])
    with pytest.raises(TypeError, match="topk_ids must have dtype"):
        M.select(x, ids.long(), tw, "sigmoid")
    with pytest.raises(ValueError, match="topk_w must have shape"):
        M.select(x, ids, tw[:2], "sigmoid")
    with pytest.raises(ValueError, match="expert_counts is empty"):
        M.pack_rows8(x, y8, expert_counts=torch.zeros(0, dtype=torch.int32, device="cuda"))
    with pytest.raises(M.MoeError):          # the status needs a workspace
        M.pack_rows8(x, y8, expert_counts=torch.ones(2, dtype=torch.int32, device="cuda"), align=2)
    M.pack_rows8(x, list(y8))                # (a pair of any kind)
    with pytest.raises(ValueError, match="w must have shape"):
        M.linear_backward8(x, torch.zeros(2, 200, 64, dtype=BF, device="cuda"), y8[0])
    ws = M.new_workspace_linear8(4, 200, 64)
    with pytest.raises(M.MoeError):          # neither x nor x8
        M.linear_backward8(x, torch.zeros(200, 64, dtype=BF, device="cuda"), ws, dw=torch.zeros(200, 64, dtype=BF, device="cuda"))
    torch.cuda.synchronize()


def test_other_dtypes_of_numbers(M):
    """Arguments as numpy numbers go through the binding's own checks to the same call."""
    l = torch.randn(5, 32, generator=torch.Generator().manual_seed(1)).cuda()
    ids, tw, i2, t2 = (torch.empty(5, 4, dtype=t, device="cuda") for t in (torch.int32, FP, torch.int32, FP))
    M.select(l, ids, tw, "sigmoid", n_groups=4, topk_groups=2, scale=2)
    M.select(l, i2, t2, "sigmoid", n_groups=np.int64(4).item(), topk_groups=2, scale=np.float64(2.0), renormalize=np.bool_(True))
    assert torch.equal(ids, i2) and torch.equal(tw, t2)
