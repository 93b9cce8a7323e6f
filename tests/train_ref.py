"""Float64 definitions of the training operators, and the error bounds their kernels are held to.

Bounds count roundings: a value rounded to type t is off by at most eps(t)/2 relative; an fp32 sum of n
terms by at most n * 2^-24 times the sum of their magnitudes; a tensor-core sum adds 16 products at a
time and may drop bits below 2^-22 of the running sum at each of those steps.
"""
import math

import torch

U32 = 2.0 ** -24
F64 = torch.float64


def half_step(t):
    return torch.finfo(t).eps / 2


def tiny(t):
    return float(torch.finfo(t).smallest_normal) * torch.finfo(t).eps


def positions(ids, E, align):
    """(inv_perm [T, K], counts [E]) of the expert-contiguous layout, pairs in ascending t*K+k order."""
    counts = [0] * E
    for e in ids.reshape(-1).tolist():
        counts[e] += 1
    seg, row = [], 0
    for c in counts:
        seg.append(row)
        row += -(-c // align) * align
    inv, seen = [], [0] * E
    for e in ids.reshape(-1).tolist():
        inv.append(seg[e] + seen[e])
        seen[e] += 1
    return torch.tensor(inv, dtype=torch.int32).reshape(ids.shape), torch.tensor(counts, dtype=torch.int32)


def combine(y, inv, w, residual=None):
    """(out, sum of magnitudes); inv -1: nothing."""
    keep = (inv >= 0).to(F64)
    w = keep if w is None else keep * w.to(F64)
    rows = y.to(F64)[inv.clamp(min=0).long()]
    rows = torch.where(inv[..., None] >= 0, rows, torch.zeros_like(rows))
    out, mag = (rows * w[..., None]).sum(1), (rows * w[..., None]).abs().sum(1)
    if residual is not None:
        out, mag = out + residual.to(F64), mag + residual.to(F64).abs()
    return out, mag


def combine_grad(dout, y, inv, w, U):
    dy = torch.zeros(U, dout.shape[1], dtype=F64)
    dw, mag = torch.zeros(inv.shape, dtype=F64), torch.zeros(inv.shape, dtype=F64)
    d = dout.to(F64)
    for k in range(inv.shape[1]):
        t = (inv[:, k] >= 0).nonzero().reshape(-1)
        r = inv[t, k].long()
        dy[r] = d[t] if w is None else d[t] * w[t, k, None].to(F64)
        if y is not None:
            p = d[t] * y[r].to(F64)
            dw[t, k], mag[t, k] = p.sum(1), p.abs().sum(1)
    return dy, dw, mag


def route_weights(logits, ids, fn, renorm):
    l = logits.to(F64)
    s = torch.softmax(l, 1) if fn == "softmax" else torch.nn.functional.softplus(l, threshold=1e9).sqrt()
    w = s.gather(1, ids.long())
    return w / w.sum(1, keepdim=True) if renorm else w


def route_weights_autograd(logits, ids, fn):
    """Normalised weights of the selected experts, differentiable in the logits."""
    s = torch.softmax(logits, 1) if fn == "softmax" else torch.nn.functional.softplus(logits, threshold=1e9).sqrt()
    w = s.gather(1, ids)
    return w / w.sum(1, keepdim=True)


def route_grad(logits, ids, dw, fn, renorm):
    """dL/dlogits by the chain rule over the whole row."""
    l = logits.to(F64)
    ids, dw = ids.long(), dw.to(F64)
    s = torch.softmax(l, 1) if fn == "softmax" else torch.nn.functional.softplus(l, threshold=1e9).sqrt()
    sel = s.gather(1, ids)
    if renorm:
        n = sel.sum(1, keepdim=True)
        dsel = dw / n - (dw * sel).sum(1, keepdim=True) / n ** 2
    else:
        dsel = dw
    ds = torch.zeros_like(s).scatter_add_(1, ids, dsel)
    if fn == "softmax":
        return s * (ds - (ds * s).sum(1, keepdim=True))
    return ds * torch.sigmoid(l) / (2 * s)


def act(z, name):
    if name == "relu":
        return z.clamp(min=0)
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu":
        return z * 0.5 * torch.erfc(-z / math.sqrt(2))
    if name == "swiglu":
        g, u = z.chunk(2, -1)
        return g * torch.sigmoid(g) * u
    return z


def act_grad(dy, z, name):
    if name == "none":
        return dy
    if name == "relu":
        return dy * (z > 0)
    if name == "gelu":
        return dy * (0.5 * torch.erfc(-z / math.sqrt(2)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi))
    if name == "silu":
        s = torch.sigmoid(z)
        return dy * (s + z * s * (1 - s))
    g, u = z.chunk(2, -1)
    s = torch.sigmoid(g)
    return torch.cat([dy * u * (s + g * s * (1 - s)), dy * g * s], -1)


# Evaluating an activation (or its derivative) in fp32 with the fast exponential and division: relative
# error below 2^-17 of |z| + 1 times the factors it multiplies.
ACT_EVAL = 2.0 ** -17


def segments(counts, align, rows):
    """[(expert, first row, rows)]; counts None: one dense segment."""
    if counts is None:
        return [(0, 0, rows)]
    out, row = [], 0
    for e, c in enumerate(counts):
        out.append((e, row, c))
        row += -(-c // align) * align
    return out


def mma_err(q):
    """Relative (to the sum of magnitudes) error of a tensor-core sum of q products."""
    return (q / 16 + 16) * 2.0 ** -22


def linear(x, w, bias, name, residual, dt):
    """One segment: y, z and their error bounds before nothing but the kernel's arithmetic."""
    x, w = x.to(F64), w.to(F64)
    z, mag = x @ w.t(), x.abs() @ w.abs().t()
    if bias is not None:
        z, mag = z + bias.to(F64), mag + bias.to(F64).abs()
    ez = mma_err(x.shape[1]) * mag
    y = act(z, name)
    if name == "swiglu":
        g, u = z.chunk(2, -1)
        eg, eu = ez.chunk(2, -1)
        ey = 1.2 * eg * u.abs() + eu * act(g, "silu").abs() + eg * eu + ACT_EVAL * (g.abs() + 1) * y.abs()
    elif name == "none":
        ey = ez
    else:
        ey = 1.2 * ez + ACT_EVAL * (z.abs() + 1) * y.abs()
    if residual is not None:
        y = y + residual.to(F64)
        ey = ey + U32 * (y.abs() + residual.to(F64).abs())
    h = half_step(dt)
    return y, ey + h * (y.abs() + ey) + tiny(dt), z, ez + h * (z.abs() + ez) + tiny(dt)


def linear_grad(dy, x, w, z, name, residual, dt):
    """One segment: (dx, its bound), (dw, its bound), (dbias, its bound)."""
    dy, x, w = dy.to(F64), x.to(F64), w.to(F64)
    h = half_step(dt)
    dz = act_grad(dy, None if z is None else z.to(F64), name)
    if name == "none":
        ev = torch.zeros_like(dz)
        ed = ev
    else:
        zz = z.to(F64)
        if name == "swiglu":
            g, u = zz.chunk(2, -1)
            ev = ACT_EVAL * torch.cat([dy.abs() * u.abs() * (1 + g.abs()), dy.abs() * (1 + g.abs())], -1)
        else:
            ev = ACT_EVAL * dy.abs() * (1 + zz.abs())
        ed = ev + h * (dz.abs() + ev) + tiny(dt)
    dx = dz @ w
    ex = ed @ w.abs() + mma_err(w.shape[0]) * ((dz.abs() + ed) @ w.abs())
    if residual is not None:
        dx = dx + residual.to(F64)
        ex = ex + U32 * (dx.abs() + residual.to(F64).abs())
    dw = dz.t() @ x
    ew = ed.t() @ x.abs() + mma_err(x.shape[0]) * ((dz.abs() + ed).t() @ x.abs())
    db = dz.sum(0)
    eb = ev.sum(0) + (x.shape[0] + 2) * U32 * dz.abs().sum(0)
    return (dx, ex + h * (dx.abs() + ex) + tiny(dt)), (dw, ew + h * (dw.abs() + ew) + tiny(dt)), (db, eb + 1e-30)


def check(got, ref, bound, what):
    got = got.detach().to("cpu", F64)
    assert torch.isfinite(got).all(), f"{what}: not finite"
    over = (got - ref).abs() - bound
    worst = over.argmax() if over.numel() else None
    assert worst is None or over.reshape(-1)[worst] <= 0, (
        f"{what}: off by {(got - ref).abs().reshape(-1)[worst]:.3e}, allowed {bound.reshape(-1)[worst]:.3e} "
        f"at {int(worst)} (value {ref.reshape(-1)[worst]:.4e})")
