"""The training operators together: a layer with routed experts and a shared expert (examples/train_layer.py)
against float64 autograd of the same layer."""
import importlib.util
import os

import pytest
import torch

import train_ref as R
from gpu_util import ensure_lib

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ensure_lib()
    spec = importlib.util.spec_from_file_location("train_layer", os.path.join(ROOT, "examples", "train_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def reference(L, x, dout):
    """out, dx and the weights' gradients in float64, the selection as the layer made it; the gradient of the routing
    weights with the magnitudes in its sums."""
    p = {n: (L.w[n] if n in L.w else v).detach().cpu().to(R.F64).requires_grad_() for n, v in L.master.items()}
    xr = x.cpu().to(R.F64).requires_grad_()
    d = dout.cpu().to(R.F64)
    ids = L.ids.cpu().long()
    w = R.route_weights_autograd(xr @ p["gate"].t(), ids, L.score_fn)
    out = R.act(xr @ p["v13"].t(), "swiglu") @ p["v2"].t() + p["b"]
    dw, mag = torch.zeros(ids.shape, dtype=R.F64), torch.zeros(ids.shape, dtype=R.F64)
    for e in range(L.E):
        t, k = (ids == e).nonzero(as_tuple=True)
        h = R.act(xr[t] @ p["w13"][e].t(), "swiglu")
        y = h @ p["w2"][e].t()
        out = out.index_add(0, t, y * w[t, k, None])
        dw[t, k] = (d[t] * y).sum(1).detach()
        mag[t, k] = (d[t].abs() * (y.abs() + h.abs() @ p["w2"][e].abs().t())).sum(1).detach()
    out.backward(d)
    return out.detach(), xr.grad, {n: v.grad for n, v in p.items()}, dw, mag


@pytest.mark.parametrize("T,E,K,align,score", [(70, 16, 4, 16, "sqrt_softplus"), (300, 8, 2, 128, "softmax"), (1, 4, 2, 1, "softmax")])
def test_layer_gradients(example, T, E, K, align, score):
    L = example.TrainLayer(T, H=256, I=128, E=E, K=K, shared=64, align=align, score_fn=score, seed=T)
    g = torch.Generator().manual_seed(1)
    x = torch.randn(T, 256, generator=g).cuda().to(torch.bfloat16)
    dout = torch.randn(T, 256, generator=g).cuda().to(torch.bfloat16)
    out = L.forward(x).clone()
    dx = L.backward(x, dout).clone()
    L.check()
    ref, dxr, grads, dwr, mag = reference(L, x, dout)
    # Every tensor between two operators is rounded to bf16, which moves its norm by less than 2^-9 of it (a half
    # step is 2^-8 at most): out passes through four such roundings (h, y, the sums, out), dx and the weights'
    # gradients through at most eight (with z, dh, dz twice), which add up at worst linearly.
    def rel(a, b):
        return float((a.cpu().to(R.F64) - b).norm() / b.norm())

    bound = 8 * 2.0 ** -9
    assert rel(out, ref) < bound
    assert rel(dx, dxr) < bound
    for n, want in grads.items():
        if n != "gate":
            assert rel(L.grads[n], want) < bound, n
    # The routing weights' gradients are dot products of few or one token, whose errors are relative to the
    # magnitudes in them: y is rounded once, and so is each h in it (half a step each; 10% for everything else).
    h = R.half_step(torch.bfloat16)
    R.check(L.dtopk_w, dwr, 1.1 * h * mag, "dtopk_w")
    # From there on: the gate's gradient of what the kernels handed on.
    w, dw, logits = (t.cpu().to(R.F64) for t in (L.topk_w, L.dtopk_w, L.logits))
    dl = R.route_grad(logits, L.ids.cpu(), dw, score, True)
    terms = (w * dw).abs()
    scale = torch.zeros_like(dl).scatter_(1, L.ids.cpu().long(), terms + w * terms.sum(1, keepdim=True))
    if score == "softmax":
        scale = scale + torch.softmax(logits, 1) * terms.sum(1, keepdim=True)
    e_dl = scale * (E + 64 + 2 * logits.abs().max()) * R.U32 + h * 1.01 * dl.abs() + R.tiny(torch.bfloat16)
    xa = x.cpu().to(R.F64)
    want = dl.t() @ xa
    e = e_dl.t() @ xa.abs() * 1.01 + R.mma_err(T) * (dl.abs().t() @ xa.abs())
    R.check(L.grads["gate"], want, e + h * (want.abs() + e) + R.tiny(torch.bfloat16), "gate")


def test_layer_learns(example):
    torch.manual_seed(0)
    L = example.TrainLayer(512, H=256, I=128, E=8, K=2, shared=128)
    x = torch.randn(512, 256, device="cuda").to(torch.bfloat16)
    target = torch.tanh(x.float() @ torch.randn(256, 256, device="cuda") / 16)
    losses = []
    for _ in range(12):
        diff = L.forward(x).float() - target
        losses.append(float(diff.square().mean()))
        L.backward(x, (diff * (2.0 / 256)).to(torch.bfloat16))
        L.update(2.0 / 512)
    L.check()
    assert losses[-1] < 0.9 * losses[0] and all(b < a * 1.001 for a, b in zip(losses, losses[1:])), losses
