"""Float64 definitions of the norm, the routing by groups and the 8-bit rows, with the error bounds of their kernels
(how bounds count is in train_ref)."""
import numpy as np
import torch

import train_ref as R
from oracle import formats as F

F64, U32 = R.F64, R.U32


# ------------------------------------------------------------------------------------- 8-bit rows

def pack8(x):
    """Codes [M, C] and scales [M, ceil(C / 128)] (uint8) of x: exact, one rounding per code."""
    x = x.to(F64).numpy()
    M, C = x.shape
    q = np.zeros((M, C), np.uint8)
    sf = np.zeros((M, -(-C // 128)), np.uint8)
    for r in range(M):
        for g in range(sf.shape[1]):
            v = x[r, 128 * g:128 * (g + 1)]
            fine = np.isfinite(v)
            e = F.ue8m0_exponent_for_amax(float(np.abs(v[fine]).max()) if fine.any() else 0.0)
            c = F.encode_e4m3_rne(np.where(fine, v, 0.0) / 2.0 ** e)
            q[r, 128 * g:128 * (g + 1)] = np.where(fine, c, 0x7F)
            sf[r, g] = e + 127
    return torch.from_numpy(q), torch.from_numpy(sf)


def values8(q, sf):
    scale = torch.from_numpy(F.decode_ue8m0(sf.numpy())).repeat_interleave(128, 1)[:, :q.shape[1]]
    return torch.from_numpy(F.decode_e4m3(q.numpy())) * scale


def largest(dt):
    return torch.finfo(dt).max


def unpacked(q, sf, dt):
    """The values in type dt (exact up to its largest)."""
    v = values8(q, sf)
    return torch.where(v.abs() > largest(dt), torch.sign(v) * largest(dt), v).to(dt)


def check8(q, sf, ref, err, what):
    """8-bit rows of values that are known to within err: every scale is the rule's for some value within the bound, every
    code off by at most half a step more than that."""
    q, sf = q.cpu(), sf.cpu()
    got = values8(q, sf)
    assert torch.isfinite(got).all(), what
    C = ref.shape[1]
    for g in range(sf.shape[1]):
        s = slice(128 * g, min(128 * (g + 1), C))
        lo = (ref[:, s].abs() - err[:, s]).clamp(min=0).amax(1)
        hi = (ref[:, s].abs() + err[:, s]).amax(1)
        e = sf[:, g].to(F64) - 127
        assert (448 * 2 ** e >= lo).all(), f"{what}: a scale too small"
        assert ((448 * 2 ** (e - 1) < hi) | (e == -127) | ((e == 0) & (lo == 0))).all(), f"{what}: a scale too large"
        step = 2.0 ** (torch.floor(torch.log2((ref[:, s].abs() + err[:, s]).clamp(min=1e-300) / 2 ** e[:, None])).clamp(min=-6) - 3)
        over = (got[:, s] - ref[:, s]).abs() - (err[:, s] + step / 2 * 2 ** e[:, None])
        assert (over <= 0).all(), f"{what}: code off by {float(over.max()):.3e} more than half a step"


# ------------------------------------------------------------------------------------- norm

def sums_err(H):
    """Relative error of a sum of H positive fp32 terms: no term passes more than H / 32 + 16 additions."""
    return (H / 32 + 16) * U32


def norm(x, residual, w, eps, dt):
    """(sum as stored, y, bound of y before its rounding)."""
    s = x.to(F64)
    if residual is not None:
        s = (x.float() + residual.float()).to(dt).to(F64)      # one rounding: the fp32 sum of two 16-bit values and more
    r = 1 / torch.sqrt((s * s).mean(1, keepdim=True) + eps)
    y = s * r * w.to(F64)
    # half of the mean's error (sum, division, eps), a reciprocal root within 2^-22, two products
    return s, y, y.abs() * (sums_err(x.shape[1]) / 2 + 2 * U32 + 2.0 ** -22 + 3 * U32) + 1e-44


def norm_grad(dy, x, w, eps, dsum, dt):
    """(dx, its bound), (dw, its bound)"""
    dy, v, w = dy.to(F64), x.to(F64), w.to(F64)
    T, H = v.shape
    r = 1 / torch.sqrt((v * v).mean(1, keepdim=True) + eps)
    g = dy * w
    along = (v * g).mean(1, keepdim=True)
    dx = r * g - v * r ** 3 * along
    er = sums_err(H) / 2 + 2 * U32 + 2.0 ** -22
    size = r * g.abs() + v.abs() * r ** 3 * (v * g).abs().mean(1, keepdim=True)
    ex = size * (4 * er + sums_err(H) + 8 * U32)
    if dsum is not None:
        dx = dx + dsum.to(F64)
        ex = ex + U32 * (dx.abs() + dsum.to(F64).abs())
    ex = ex + R.half_step(dt) * (dx.abs() + ex) + R.tiny(dt)
    dw = (dy * v * r).sum(0)
    ew = (dy * v * r).abs().sum(0) * (er + (T + 4) * U32) + 1e-40
    return (dx, ex), (dw, ew)


# ------------------------------------------------------------------------------------- routing

def score(l, fn):
    l = l.to(F64)
    if fn == "softmax":
        m = l.amax(1, keepdim=True)
        e = torch.where(torch.isinf(l) & (l < 0), torch.zeros_like(l), torch.exp(l - m))
        s = e.sum(1, keepdim=True)
        return e / torch.where(s == 0, torch.ones_like(s), s)
    if fn == "sigmoid":
        return 1 / (1 + torch.exp(-l))
    return torch.sqrt(l.clamp(min=0) + torch.log1p(torch.exp(-l.abs())))


def select(logits, bias, K, fn, G=1, KG=1, best=2, renorm=True, scale=1.0):
    """ids and weights by sorting in plain Python."""
    s = score(logits, fn)
    key = s if bias is None else s + bias.to(F64)
    order = logits.to(F64) if bias is None else key
    clean = lambda t: torch.where(torch.isnan(t), torch.full_like(t, -float("inf")), t).tolist()   # noqa: E731
    key, order = clean(key), clean(order)
    T, E = logits.shape
    n = E // G
    ids = []
    for t in range(T):
        allowed = range(E)
        if KG < G:
            worth = []
            for g in range(G):
                top = sorted(key[t][g * n:(g + 1) * n], reverse=True)[:best]
                v = sum(top)
                worth.append(-float("inf") if v != v else v)
            groups = sorted(range(G), key=lambda g: (-worth[g], g))[:KG]
            allowed = [e for g in groups for e in range(g * n, (g + 1) * n)]
        ids.append(sorted(allowed, key=lambda e: (-order[t][e], e))[:K])
    ids = torch.tensor(ids, dtype=torch.int64).reshape(T, K)
    w = s.gather(1, ids)
    if renorm:
        total = w.sum(1, keepdim=True)
        w = torch.where(total == 0, torch.zeros_like(w), w / total)
    return ids.to(torch.int32), w * scale


def select_weights(l, ids, fn, renorm, scale):
    """Weights of given experts, differentiable."""
    s = {"softmax": lambda: torch.softmax(l, 1), "sigmoid": lambda: torch.sigmoid(l),
         "sqrt_softplus": lambda: torch.nn.functional.softplus(l, threshold=1e9).sqrt()}[fn]()
    w = s.gather(1, ids)
    return scale * (w / w.sum(1, keepdim=True) if renorm else w)


def select_grad(l, ids, dw, fn, renorm, scale):
    l = l.to(F64).clone().requires_grad_(True)
    (select_weights(l, ids.long(), fn, renorm, scale) * dw.to(F64)).sum().backward()
    return l.grad
