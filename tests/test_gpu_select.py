"""Routing from logits by groups of experts, and its gradient, against float64."""
import pytest
import torch

import around_ref as A
import train_ref as R
from gpu_util import ensure_lib

pytestmark = pytest.mark.gpu

BF, HF, FP = torch.bfloat16, torch.float16, torch.float32
FNS = ["softmax", "sqrt_softplus", "sigmoid"]
INF = float("inf")


@pytest.fixture(scope="module")
def M():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return ensure_lib()


def run(M, logits, bias, K, fn, G=1, KG=1, best=2, renorm=True, scale=1.0, pitch=0):
    T, E = logits.shape
    wide = torch.full((T, E + pitch), 50.0, dtype=logits.dtype, device="cuda")
    wide[:, :E] = logits.cuda()
    ids = torch.full((T + 1, K), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T + 1, K), -7.0, device="cuda")
    M.select(wide[:, :E], ids[:T], w[:T], fn, e_score_bias=None if bias is None else bias.cuda(), n_groups=G, topk_groups=KG,
             group_best=best, renormalize=renorm, scale=scale)
    assert (ids[T:] == -7).all() and (w[T:] == -7).all()
    return ids[:T].cpu(), w[:T].cpu()


def check(M, logits, bias, K, fn, **kw):
    ids, w = run(M, logits, bias, K, fn, **kw)
    kw.pop("pitch", None)
    ri, rw = A.select(logits, bias, K, fn, **kw)
    assert torch.equal(ids, ri), f"{(ids != ri).any(1).sum()} tokens differ"
    # a score within 2^-20 (softmax: its sum's additions too), the sum of K of them and two operations
    rel = (8 + (logits.shape[1] / 32 + 8 if fn == "softmax" else 0) + kw.get("renorm", True) * 16) * 2.0 ** -23
    R.check(w, rw, rel * 2 * rw.abs() + 1e-37, "w")


CASES = [  # T, E, K, G, KG, best, dtype, bias, renorm, scale, pitch
    (8, 256, 6, 8, 4, 2, FP, True, True, 2.5, 0), (1, 256, 8, 8, 4, 2, FP, True, True, 1.0, 4), (77, 256, 6, 1, 1, 2, FP, False, True, 1.0, 0),
    (33, 16, 4, 4, 2, 2, BF, True, False, 2.5, 0), (5, 1, 1, 1, 1, 1, FP, True, True, 1.0, 0), (9, 4, 4, 4, 4, 2, HF, False, True, 1.0, 1),
    (40, 160, 6, 8, 3, 1, FP, False, False, 16.0, 0), (21, 60, 5, 4, 1, 2, FP, True, True, 1.0, 3), (19, 1024, 32, 32, 32, 2, FP, True, True, 1.0, 0),
    (13, 1024, 32, 32, 7, 2, BF, True, True, 1.0, 0), (11, 1020, 8, 17, 5, 2, FP, True, True, 1.0, 0), (7, 1023, 8, 3, 1, 1, FP, True, False, 1.0, 0),
    (30, 33, 3, 11, 2, 2, HF, True, True, 1.0, 0), (30, 32, 2, 32, 2, 2, FP, True, True, 1.0, 0), (16, 72, 7, 9, 4, 2, BF, False, True, 0.5, 0),
    (500, 64, 8, 8, 4, 2, BF, True, True, 1.0, 0), (23, 512, 8, 16, 4, 2, FP, True, True, 1.0, 2), (3, 1000, 10, 5, 2, 2, FP, True, True, 1.0, 0),
    (6, 999, 9, 27, 3, 2, FP, False, True, 1.0, 0), (50, 128, 31, 2, 1, 2, FP, True, True, 1.0, 0), (50, 128, 32, 2, 1, 2, FP, True, True, 1.0, 0),
    (12, 7, 7, 1, 1, 2, BF, True, True, 1.0, 0), (64, 258, 6, 6, 3, 2, FP, True, True, -1.5, 0),
]


@pytest.mark.parametrize("fn", FNS)
@pytest.mark.parametrize("T,E,K,G,KG,best,dt,bias,renorm,scale,pitch", CASES)
def test_select(M, fn, T, E, K, G, KG, best, dt, bias, renorm, scale, pitch):
    g = torch.Generator().manual_seed(T * E + K)
    logits = (torch.randn(T, E, generator=g) * 2).to(dt)
    b = torch.randn(E, generator=g) * 0.1 if bias else None
    check(M, logits, b, K, fn, G=G, KG=KG, best=best, renorm=renorm, scale=scale, pitch=pitch)


@pytest.mark.parametrize("fn", FNS)
def test_exact_ties(M, fn):
    """Equal keys: the lower expert and the lower group, also with a bias of zeros, and on rows that are all equal."""
    g = torch.Generator().manual_seed(1)
    logits = (torch.randn(60, 64, generator=g) * 2).round()
    logits[:5] = 0.0
    for b in (None, torch.zeros(64), (torch.randn(64, generator=g) * 2).round()):
        for G, KG in ((1, 1), (8, 3), (16, 5)):
            for best in (1, 2):
                check(M, logits, b, 6, fn, G=G, KG=KG, best=best)
    check(M, logits.to(BF), torch.zeros(64), 6, fn, G=4, KG=2)


@pytest.mark.parametrize("fn", FNS)
def test_keys_that_fp32_cannot_tell_apart(M, fn):
    """Biases that bring every key of a token next to one value: keys differ by about 1e-9 (the biases' last place), far
    less than fp32 scores are good for; the order is that of 64 bits, of experts and of groups."""
    g = torch.Generator().manual_seed(2)
    E, told = 64, 0
    for seed in range(24):
        l = torch.randn(1, E, generator=g) * 0.3
        s = A.score(l, fn)[0]
        base = float(s.mean())
        bias = (base - s).float()            # |bias| is small, its rounding 2^-25 of it
        key = s + bias.double()
        assert float((key - base).abs().max()) < 1e-7 and key.unique().numel() == E
        if float(torch.diff(key.sort().values).min()) < 1e-15:
            continue                         # 64-bit evaluations, good to 1e-16, might not tell them apart either
        told += 1
        many = l.expand(9, E).contiguous()
        check(M, many, bias, 8, fn)
        check(M, many, bias, 8, fn, G=8, KG=3, best=1)
        check(M, many, bias, 8, fn, G=8, KG=3, best=2)
        check(M, many, bias, 32, fn, G=8, KG=4, best=2)
    assert told >= 16


@pytest.mark.parametrize("fn", FNS)
@pytest.mark.parametrize("dt", [FP, BF, HF])
def test_masked_experts(M, fn, dt):
    """Logits of -infinity or the type's lowest value, whole groups and whole rows of them; biases of -infinity."""
    g = torch.Generator().manual_seed(4)
    E, K = 40, 6
    l = (torch.randn(12, E, generator=g) * 2).to(dt)
    l[0, 5:] = -INF                       # fewer than K left
    l[1] = -INF
    l[2] = torch.finfo(dt).min
    l[3, ::2] = torch.finfo(dt).min
    l[4, 8:16] = -INF
    l[5, 1] = 80.0                        # one expert has nearly everything
    l[6] = 90.0 if fn != "softmax" else 3.0
    b = torch.randn(E, generator=g) * 0.1
    off = b.clone()
    off[3:20] = -INF
    for bias in (None, b, off, torch.full((E,), -INF)):
        for kw in (dict(), dict(G=5, KG=2), dict(G=5, KG=2, best=1), dict(renorm=False)):
            check(M, l, bias, K, fn, **kw)


def test_nan_and_infinite_logits_give_valid_ids(M):
    l = torch.randn(6, 32, generator=torch.Generator().manual_seed(5))
    l[0, 3] = float("nan")
    l[1] = float("nan")
    l[2, 4] = INF
    l[3, 4:6] = INF
    for fn in FNS:
        for bias in (None, torch.zeros(32)):
            for kw in (dict(), dict(G=4, KG=2)):
                ids, w = run(M, l, bias, 8, fn, **kw)
                for row in ids.tolist():
                    assert len(set(row)) == 8 and all(0 <= e < 32 for e in row), (fn, row)
                assert torch.isfinite(w[4:]).all()
                assert torch.isnan(w[1]).any()


@pytest.mark.parametrize("fn", FNS)
@pytest.mark.parametrize("E,G,KG,K,best", [(32, 8, 3, 6, 2), (32, 16, 4, 5, 2), (32, 16, 4, 5, 1), (12, 12, 5, 5, 2), (96, 6, 2, 8, 2),
                                           (256, 8, 4, 6, 2), (512, 4, 2, 9, 1)])
def test_nan_logits_without_a_bias_leave_their_groups_last(M, fn, E, G, KG, K, best):
    """A NaN's key is -infinity in what its group is worth too, not the score 0 of a masked expert."""
    g = torch.Generator().manual_seed(E + G)
    l = torch.randn(64, E, generator=g)
    l[torch.rand(64, E, generator=g) < torch.linspace(0, 1, 64)[:, None]] = float("nan")
    ids, _ = run(M, l, None, K, fn, G=G, KG=KG, best=best)
    ref, _ = A.select(l, None, K, fn, G, KG, best)
    assert torch.equal(ids.cpu(), ref)


@pytest.mark.parametrize("fn", FNS)
def test_masked_groups_without_a_bias(M, fn):
    """Groups whose logits are all -infinity score 0; equals go to the lower group and expert."""
    g = torch.Generator().manual_seed(3)
    l = torch.randn(40, 8, 8, generator=g)
    l[torch.rand(40, 8, generator=g) < torch.linspace(0, 0.95, 40)[:, None]] = -INF
    l = l.reshape(40, 64)
    ids, _ = run(M, l, None, 7, fn, G=8, KG=3)
    l64 = l.to(torch.float64)
    l64[(l == -INF).all(1)] = 0          # (a row of nothing: every score 0, so are these)
    ref, _ = A.select(l64, None, 7, fn, 8, 3)
    assert torch.equal(ids.cpu(), ref)


GRAD = [  # T, E, K, dtype, grad dtype, pitch
    (8, 256, 6, FP, FP, 0), (33, 64, 4, BF, BF, 0), (70, 100, 5, FP, BF, 4), (11, 7, 7, HF, HF, 1), (5, 1, 1, FP, FP, 0),
    (9, 1024, 32, FP, HF, 0), (100, 258, 3, BF, BF, 2), (40, 511, 8, FP, FP, 0), (300, 32, 2, HF, HF, 0),
]


@pytest.mark.parametrize("fn", FNS)
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,K,dt,gdt,pitch", GRAD)
def test_select_gradient(M, fn, renorm, T, E, K, dt, gdt, pitch):
    g = torch.Generator().manual_seed(T + E)
    l = (torch.randn(T, E, generator=g) * 2).to(dt)
    scale = 2.5
    wide = torch.full((T, E + pitch), 9.0, dtype=dt, device="cuda")
    wide[:, :E] = l.cuda()
    ids, w = torch.empty(T, K, dtype=torch.int32, device="cuda"), torch.empty(T, K, device="cuda")
    M.select(wide[:, :E], ids, w, fn, renormalize=renorm, scale=scale)
    dw = torch.randn(T, K, generator=g)
    out = torch.full((T, E + pitch), 9.0, dtype=gdt, device="cuda")
    ws = M.new_workspace_rows(T, K, E)
    M.select_backward(wide[:, :E], ids, w, dw.cuda(), out[:, :E], ws, fn, renormalize=renorm, scale=scale)
    ref = A.select_grad(l, ids.cpu(), dw, fn, renorm, scale)
    # each entry is a sum of terms w_k w_j dw (renormalised, or softmax's others) of which every factor is within a few
    # 2^-23 (softmax: its sum's additions too); 2^-16 of their magnitudes' sum covers K = 32 of them
    s = A.score(l, fn)
    wk = w.cpu().double().abs()
    size = (wk * dw.abs().double()).sum(1, keepdim=True)
    here = torch.zeros(T, E, dtype=R.F64).scatter_add_(1, ids.cpu().long(), wk * (dw.abs().double() + size / scale))
    # the reference's own rounding: with renormalised softmax weights an expert that is not selected has s_i sum_j g_j,
    # exactly zero, but g's and their sum are rounded in 64 bits, (K + E + 8) 2^-53 < 2^-42 of the terms' magnitudes, which
    # are at most w_k (|dw_k| + sum_j w_j |dw_j| / scale) each: their sum here is at most that of `here`
    own = s * here.sum(1, keepdim=True) * 2.0 ** -42 if fn == "softmax" else 0
    size = here + (s * size if fn == "softmax" and not renorm else 0)
    R.check(out[:, :E], ref, own + 2.0 ** -17 * size + R.half_step(gdt) * ref.abs() * 1.01 + R.tiny(gdt), "dlogits")
    assert (out[:, E:] == 9.0).all() and M.get_error(ws) == M.OK


def test_select_gradient_against_differences(M):
    """The kernel's own weights at l + h d and l - h d, for experts that stay the same."""
    T, E, K, h = 20, 32, 4, 2.0 ** -7
    g = torch.Generator().manual_seed(8)
    for fn in FNS:
        l, d = torch.randn(T, E, generator=g).cuda(), torch.randn(T, E, generator=g).cuda()
        c = torch.randn(T, K, generator=g).cuda()
        push = torch.zeros(E, device="cuda")
        push[:K] = torch.arange(K, 0, -1, device="cuda") * 10.0        # a bias that decides the choice and its order
        out = []
        for x in (l, l + h * d, l - h * d):
            ids, w = torch.empty(T, K, dtype=torch.int32, device="cuda"), torch.empty(T, K, device="cuda")
            M.select(x, ids, w, fn, e_score_bias=push, scale=1.5)
            assert (ids == torch.arange(K, device="cuda")).all()
            out.append((ids, w))
        dl = torch.empty(T, E, device="cuda")
        M.select_backward(l, out[0][0], out[0][1], c, dl, M.new_workspace_rows(T, K, E), fn, scale=1.5)
        num = ((out[1][1].double() - out[2][1].double()) * c.double()).sum() / (2 * h)
        # 80 terms: truncation h^2 / 6 = 1e-5 times a third derivative below 1 each, rounding 2^-23 / h = 1.5e-5 each
        assert abs(float(num - (dl.double() * d.double()).sum())) < 80 * 2.5e-5 * 4


def test_a_gradient_of_masked_rows_is_zero(M):
    l = torch.full((2, 16), -INF)
    l[1] = torch.randn(16)
    ids, w = run(M, l, None, 3, "softmax", renorm=False)
    assert (w[0] == 0).all()
    ws = M.new_workspace_rows(2, 3, 16)
    out = torch.full((2, 16), 9.0, device="cuda")
    for fn in FNS:
        for renorm in (True, False):
            ids, w = run(M, l, None, 3, fn, renorm=renorm)
            M.select_backward(l.cuda(), ids.cuda(), w.cuda(), torch.ones(2, 3, device="cuda"), out, ws, fn, renormalize=renorm)
            assert (out[0] == 0).all() and torch.isfinite(out).all()


def test_an_id_out_of_range_is_reported(M):
    ids = torch.tensor([[0, 99]], dtype=torch.int32, device="cuda")
    ws = M.new_workspace_rows(1, 2, 8)
    l, w, out = torch.zeros(1, 8, device="cuda"), torch.ones(1, 2, device="cuda"), torch.empty(1, 8, device="cuda")
    M.select_backward(l, ids, w, w, out, ws, "sigmoid", renormalize=False)
    assert M.get_error(ws) == M.ERR_DEVICE_INDEX
    assert M.get_error(ws) == M.OK
