"""Routing whose scores are tiny: weights, choice and gradient against float64."""
import pytest
import torch

import around_ref as A
import train_ref as R
from gpu_util import ensure_lib
from test_gpu_select import check, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def M():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return ensure_lib()


def rows(T, E, lo, hi, dt=torch.float32, seed=0):
    g = torch.Generator().manual_seed(seed)
    return (torch.rand(T, E, generator=g) * (hi - lo) + lo).to(dt)


# (to -170: the scores are normal fp32 numbers down to -174)
@pytest.mark.parametrize("lo,hi", [(-90, -86), (-106, -86), (-170, -88), (-170, -150), (-22, -18), (-60, -10), (-170, 20)])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_sqrt_softplus_of_far_negative_logits(M, lo, hi, dt):
    T, E, K = 24, 64, 6
    l = rows(T, E, lo, hi, dt, 1)
    g = torch.Generator().manual_seed(2)
    # biases of the scores' own size decide together with them; larger ones alone
    size = float(A.score(l, "sqrt_softplus").median())
    for bias in (None, torch.zeros(E), torch.randn(E, generator=g) * size, torch.randn(E, generator=g) * 0.1):
        for renorm in (True, False):
            for kw in (dict(), dict(G=8, KG=3), dict(G=8, KG=3, best=1)):
                check(M, l, bias, K, "sqrt_softplus", renorm=renorm, scale=2.5, **kw)


@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_of_far_negative_logits(M, renorm):
    T, E, K, scale = 24, 64, 6, 2.5
    l = rows(T, E, -170, -88, seed=3)
    ids, w = run(M, l, None, K, "sqrt_softplus", renorm=renorm, scale=scale)
    dw = torch.randn(T, K, generator=torch.Generator().manual_seed(4))
    out, ws = torch.full((T, E), 9.0, device="cuda"), M.new_workspace_rows(T, K, E)
    M.select_backward(l.cuda(), ids.cuda(), w.cuda(), dw.cuda(), out, ws, "sqrt_softplus", renormalize=renorm, scale=scale)
    ref = A.select_grad(l, ids, dw, "sqrt_softplus", renorm, scale)
    # as the gradients of ordinary logits: 2^-17 of the terms' magnitudes, w_k (|dw_k| + sum_j w_j |dw_j| / scale)
    wk = w.double().abs()
    size = (wk * dw.abs().double()).sum(1, keepdim=True)
    here = torch.zeros(T, E, dtype=R.F64).scatter_add_(1, ids.long(), wk * (dw.abs().double() + size / scale))
    R.check(out, ref, 2.0 ** -17 * here + R.tiny(torch.float32), "dlogits")
    assert M.get_error(ws) == M.OK


# logits whose scores fp32 holds in few bits or not at all, but 64 bits do: sigmoid e^l, softmax e^(l - the largest)
@pytest.mark.parametrize("fn,lo,hi", [("sigmoid", -700, -600), ("sigmoid", -104, -86), ("sigmoid", -89, -20), ("sigmoid", -120, 3),
                                      ("sqrt_softplus", -700, -600), ("sqrt_softplus", -208, -172), ("sqrt_softplus", -230, 3)])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_weights_of_scores_below_fp32(M, fn, lo, hi, dt):
    l = rows(24, 64, lo, hi, dt, 5)
    push = torch.zeros(64)
    push[::5] = 9.0                       # chooses experts of every score
    for bias in (None, push):
        for renorm in (True, False):
            for scale in (1.0, -2.5, 1e20):
                check(M, l, bias, 8, fn, renorm=renorm, scale=scale)
                check(M, l, bias, 8, fn, renorm=renorm, scale=scale, G=8, KG=4)


@pytest.mark.parametrize("drop", [60, 88, 104, 120, 600])
def test_softmax_weights_of_experts_far_below_the_largest(M, drop):
    """A bias may choose experts that have nearly nothing; their normalised weights are ordinary numbers."""
    l = rows(24, 64, -4, 4, seed=6)
    l[:, 7] += drop
    push = torch.zeros(64)
    push[20:40] = 9.0
    for renorm in (True, False):
        check(M, l, push, 8, "softmax", renorm=renorm)
    l[:, 20:30] += drop / 3
    for renorm in (True, False):
        check(M, l, push, 12, "softmax", renorm=renorm)


def test_a_row_that_64_bits_call_zero_has_no_weights(M):
    for fn in ("softmax", "sqrt_softplus", "sigmoid"):
        l = torch.full((3, 16), -2000.0)
        l[0] = -float("inf")
        l[1, 0] = 0.0
        check(M, l, None, 4, fn)
        check(M, l, None, 4, fn, renorm=False)


@pytest.mark.parametrize("E", [64, 256, 1000])
@pytest.mark.parametrize("spread", [2.0, 10.0])
def test_softmax_weights_as_they_are(M, E, spread):
    """Unnormalised weights e^(l - m) / sum: the exponential within 2 units in the last place (4 of 2^-24, its argument's own
    rounding made up for by one product), the sum's terms the same and |l - m| 2^-24 of theirs more, E / 32 + 5 additions, one
    division.  (An argument rounded alone: up to |l - m| 2^-24, past 40 of them here; fast exponentials in the sum: as much of
    each of its terms.)"""
    l = torch.randn(4096, E, generator=torch.Generator().manual_seed(E)) * spread
    ids, w = run(M, l, None, 8, "softmax", renorm=False)
    p = torch.softmax(l.double(), 1)
    d = l.double() - l.double().amax(1, keepdim=True)
    ref = p.gather(1, ids.long())
    units = 4 + 2 + 4 + (p * d.abs()).sum(1, keepdim=True) + E / 32 + 5 + 1
    R.check(w, ref, ref * units * 2.0 ** -24 * 1.001 + 1e-37, "w")
    # and not off to one side: the mean of 32768 of them is within a third of a unit
    assert abs(float((w.double() / ref - 1)[ref > 1e-30].mean())) < 2.0 ** -24 / 3


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16, torch.float16])
def test_logits_of_a_types_largest_and_lowest_value(M, dt):
    """Their difference is past fp32's range: a weight of zero, not NaN."""
    f = torch.finfo(dt)
    l = rows(12, 16, -2, 2, dt, 9)
    l[:4, 3], l[2:8, 5], l[:, 9] = f.max, f.max, f.min
    l[6:, 10:14] = f.max
    push = (torch.arange(16) == 9).float()
    for fn in ("softmax", "sqrt_softplus", "sigmoid"):
        for bias in (None, torch.zeros(16), push * (50 if fn != "sqrt_softplus" else 1e30)):
            for renorm in (True, False):
                for K in (3, 5):
                    check(M, l, bias, K, fn, renorm=renorm)
                    check(M, l, bias, K, fn, renorm=renorm, G=4, KG=2)
