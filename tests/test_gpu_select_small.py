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
