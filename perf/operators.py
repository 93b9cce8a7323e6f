"""Workloads of the training operators of the MoE layer, with their plain forms.

Four operators, in both directions:

* dispatch  rows of tokens, sorted by expert (and the gradient of the token rows)
* combine   the experts' rows back to their tokens, weighted (and both gradients)
* router    the gradient of the routing weights with respect to the logits
* linear    a matrix product with bias, activation and residual, dense or one weight per expert
            (and the gradients of its input, weight and bias)

``listed()`` names the workloads, ``draw(rng)`` gives others of the same ranges, ``prepare`` makes a
workload's inputs, ``run`` computes it (plain torch operations in 32 bits, or the package's kernels
where ``own`` is set), ``work`` counts what a pass cannot do without, and ``exact`` is the same result
in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}


# ------------------------------------------------------------------------------------- workloads

def listed():
    return [
        # one decode step of the layer's own decode shape: 8 tokens to 6 of 256 experts
        dict(name="dispatch-decode", op="dispatch", T=8, H=7168, E=256, K=6, align=16, dtype="bf16", skew=0.0),
        # the training or prefill batch of 16384 tokens with a Zipf-like expert load
        dict(name="dispatch-prefill", op="dispatch", T=16384, H=7168, E=256, K=6, align=128, dtype="bf16", skew=1.0),
        # gradient of the token rows in fp32, added to the gradient that the residual path brought
        dict(name="dispatch-grad", op="dispatch_grad", T=4096, H=7168, E=256, K=6, align=256, dtype="f32", skew=0.0,
             residual=True),
        # a ragged fp16 batch of a small layer, combined onto the residual stream
        dict(name="combine-ragged", op="combine", T=1111, H=1000, E=16, K=4, align=1, dtype="f16", skew=0.5,
             residual=True),
        # both gradients of the combine in a training step
        dict(name="combine-grad", op="combine_grad", T=8192, H=7168, E=256, K=6, align=128, dtype="bf16", skew=1.0),
        # routing-weight gradient of a handful of tokens
        dict(name="router-grad-few", op="router_grad", T=8, E=256, K=6, score="sqrt_softplus", renorm=True),
        # routing-weight gradient of a training batch, softmax weights left unnormalised
        dict(name="router-grad-batch", op="router_grad", T=16384, E=256, K=6, score="softmax", renorm=False),
        # one token through a shared expert's gate and up projection (decode)
        dict(name="linear-token", op="linear", M=1, N=4096, K=7168, E=0, align=0, act="swiglu", dtype="bf16", bias=False,
             residual=False, save=False),
        # prefill through a shared expert's down projection, added to the routed experts' output
        dict(name="linear-prefill", op="linear", M=4096, N=7168, K=2048, E=0, align=0, act="none", dtype="bf16",
             bias=True, residual=True, save=False),
        # training backward of a dense projection with a GELU
        dict(name="linear-grad", op="linear_grad", M=4096, N=2048, K=7168, E=0, align=0, act="gelu", dtype="f16",
             bias=True),
        # training forward of 32 experts (one of eight ranks' share of 256): gate and up with SwiGLU,
        # the products before the activation kept for the backward pass
        dict(name="experts", op="linear", M=12288, N=4096, K=7168, E=32, align=128, act="swiglu", dtype="bf16",
             bias=False, residual=False, save=True),
        # training backward of the same experts' down projection
        dict(name="experts-grad", op="linear_grad", M=12288, N=7168, K=2048, E=32, align=128, act="none", dtype="bf16",
             bias=False),
    ]


def _log_int(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], evenly spread over its logarithm."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi)))) / step)) * step
    return n + step if n == 3 * 1024 else max(n, step)      # (3 * 1024 is no size of this layer)


def draw(rng):
    op = rng.choice(["dispatch", "dispatch_grad", "combine", "combine_grad", "router_grad", "linear", "linear",
                     "linear_grad", "linear_grad"])
    if op == "router_grad":
        E = _log_int(rng, 4, 512)
        renorm = rng.random() < 0.5           # (one normalised weight is the constant 1)
        return dict(op=op, T=_log_int(rng, 1, 16384), E=E, K=rng.randint(2 if renorm else 1, min(8, E)),
                    score=rng.choice(["softmax", "sqrt_softplus"]), renorm=renorm)
    if op in ("linear", "linear_grad"):
        experts = rng.random() < 0.5
        act = rng.choice(["none", "relu", "silu", "gelu", "swiglu"])
        N = _log_int(rng, 64, 7168, 16)
        K = _log_int(rng, 32, 7168, 8)
        most = min(8192, int(4096 * 2048 * 7168 / (N * K)))
        M = _log_int(rng, 1, most)
        case = dict(op=op, M=M, N=N, K=K, E=_log_int(rng, 2, 32) if experts else 0,
                    align=rng.choice([1, 16, 64, 128, 256]) if experts else 0, act=act,
                    dtype=rng.choice(["bf16", "f16"]), bias=rng.random() < 0.5)
        if op == "linear":
            case.update(residual=rng.random() < 0.5, save=rng.random() < 0.5)
        return case
    E = _log_int(rng, 4, 256)
    K = rng.randint(1, min(8, E))
    H = _log_int(rng, 64, 7168, 8) if rng.random() < 0.8 else _log_int(rng, 64, 4200, 2) + 1
    T = _log_int(rng, 1, min(16384, int(16384 * 6 * 7168 / (2 * K * H))))
    case = dict(op=op, T=T, H=H, E=E, K=K, align=rng.choice([1, 16, 64, 128, 256]),
                dtype=rng.choice(["bf16", "f16", "f32"]), skew=rng.choice([0.0, 0.5, 1.0]))
    if op in ("dispatch_grad", "combine"):
        case["residual"] = rng.random() < 0.5
    return case


# ------------------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 11)
    return g


def _normal(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _routing(g, case):
    """topk_ids [T, K] int32 (distinct experts per token, popularity ~ rank^-skew) and topk_w [T, K] fp32."""
    T, E, K = case["T"], case["E"], case["K"]
    pop = -case.get("skew", 0.0) * torch.log(torch.arange(1, E + 1, device="cuda", dtype=torch.float32))
    pop = pop[torch.randperm(E, generator=g, device="cuda")]
    noise = torch.rand((T, E), generator=g, device="cuda").clamp_(1e-6, 1 - 1e-6)
    keys = pop - torch.log(-torch.log(noise))
    ids = keys.topk(K, dim=1).indices.to(torch.int32)
    w = torch.rand((T, K), generator=g, device="cuda") + 0.05
    return ids, w / w.sum(dim=1, keepdim=True)


def _positions(ids, E, align):
    """inv_perm [T, K] int32 and the counts [E]: row of each pair, experts' segments padded to `align` rows."""
    flat = ids.reshape(-1).long()
    counts = torch.bincount(flat, minlength=E)
    seg = torch.cumsum((counts + align - 1) // align * align, 0) - (counts + align - 1) // align * align
    order = torch.sort(flat, stable=True).indices
    first = torch.cumsum(counts, 0) - counts
    rank = torch.empty_like(flat)
    rank[order] = torch.arange(flat.numel(), device=flat.device) - first[flat[order]]
    return (seg[flat] + rank).to(torch.int32).reshape(ids.shape), counts


def _rows_upper(pairs, E, align):
    return pairs + E * (align - 1)


def _expert_counts(g, case):
    """Rows per expert [E] int32: uneven, about one expert in eight without any; their sum is M."""
    E, M = case["E"], case["M"]
    load = torch.rand(E, generator=g, device="cuda") + 0.5
    load[torch.rand(E, generator=g, device="cuda") < 0.125] = 0
    load[int(torch.randint(E, (1,), generator=g, device="cuda"))] += 0.5
    edge = torch.round(torch.cumsum(load, 0) / load.sum() * M).long()
    edge[-1] = M
    return torch.diff(edge, prepend=edge.new_zeros(1)).clamp_(min=0).to(torch.int32)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = {"case": case}
    if op == "router_grad":
        T, E, K = case["T"], case["E"], case["K"]
        s["logits"] = torch.randn((T, E), generator=g, device="cuda") * 2.0
        score = _scores(s["logits"], case["score"])
        top = score.topk(K, dim=1)
        s["ids"] = top.indices.to(torch.int32)
        s["w"] = top.values / top.values.sum(1, keepdim=True) if case["renorm"] else top.values.contiguous()
        s["dw"] = torch.randn((T, K), generator=g, device="cuda")
        s["dlogits"] = torch.zeros((T, E), device="cuda")
        return s
    dt = DTYPES[case["dtype"]]
    if op in ("linear", "linear_grad"):
        M, N, K, E, act = case["M"], case["N"], case["K"], case["E"], case["act"]
        rows = _rows_upper(M, E, case["align"]) if E else M
        out = N // 2 if act == "swiglu" else N
        s["counts"] = _expert_counts(g, case) if E else None
        s["most"] = int(s["counts"].max()) if E else M
        s["x"] = _normal(g, (rows, K), dt)
        s["w"] = _normal(g, (E, N, K) if E else (N, K), dt, 1.0 / math.sqrt(K))
        if op == "linear":
            shape = (E, N) if E else (N,)
            s["bias"] = torch.randn(shape, generator=g, device="cuda") * 0.5 if case["bias"] else None
            s["residual"] = _normal(g, (rows, out), dt) if case["residual"] else None
            s["y"] = torch.zeros((rows, out), dtype=dt, device="cuda")
            s["z"] = torch.zeros((rows, N), dtype=dt, device="cuda") if case["save"] else None
        else:
            s["dy"] = _normal(g, (rows, out), dt)
            s["z"] = _normal(g, (rows, N), dt) if act != "none" else None
            s["dx"] = torch.zeros((rows, K), dtype=dt, device="cuda")
            s["dweight"] = torch.zeros_like(s["w"])
            s["dbias"] = torch.zeros((E, N) if E else (N,), device="cuda") if case["bias"] else None
        return s
    T, H, E, K, align = case["T"], case["H"], case["E"], case["K"], case["align"]
    U = _rows_upper(T * K, E, align)
    s["ids"], s["w"] = _routing(g, case)
    if op == "dispatch":
        s["x"] = _normal(g, (T, H), dt)
        s["x_perm"] = torch.zeros((U, H), dtype=dt, device="cuda")
        for name, n in (("sorted", U), ("experts", U), ("m_sum", 1), ("counts", E)):
            s[name] = torch.zeros(n, dtype=torch.int32, device="cuda")
        s["inv"] = torch.zeros((T, K), dtype=torch.int32, device="cuda")
        return s
    s["inv"], _ = _positions(s["ids"], E, align)
    if op == "dispatch_grad":
        s["g_perm"] = _normal(g, (U, H), dt)
        s["out"] = torch.zeros((T, H), dtype=dt, device="cuda")
    elif op == "combine":
        s["y_perm"] = _normal(g, (U, H), dt)
        s["out"] = torch.zeros((T, H), dtype=dt, device="cuda")
    else:
        s["dout"] = _normal(g, (T, H), dt)
        s["y_perm"] = _normal(g, (U, H), dt)
        s["dy_perm"] = torch.zeros((U, H), dtype=dt, device="cuda")
        s["dw"] = torch.zeros((T, K), device="cuda")
    s["residual"] = _normal(g, (T, H), dt) if case.get("residual") else None
    return s


# ------------------------------------------------------------------------------------- plain forms

def _scores(logits, fn):
    if fn == "softmax":
        e = torch.exp(logits - logits.amax(dim=1, keepdim=True))
        return e / e.sum(dim=1, keepdim=True)
    return torch.sqrt(torch.clamp(logits, min=0) + torch.log1p(torch.exp(-logits.abs())))


def _plain_dispatch(s):
    c = s["case"]
    T, K, E, align = c["T"], c["K"], c["E"], c["align"]
    inv, counts = _positions(s["ids"], E, align)
    flat = inv.reshape(-1).long()
    s["sorted"].fill_(T * K)
    s["experts"].fill_(-1)
    s["sorted"][flat] = torch.arange(T * K, device="cuda", dtype=torch.int32)
    s["experts"][flat] = s["ids"].reshape(-1)
    s["inv"].copy_(inv)
    s["m_sum"].copy_(((counts + align - 1) // align * align).sum())
    s["counts"].copy_(counts)
    s["x_perm"][flat] = s["x"].repeat_interleave(K, dim=0)
    return [s[k] for k in ("sorted", "experts", "inv", "m_sum", "counts", "x_perm")]


def _plain_gather_sum(rows, inv, w, residual, out):
    picked = rows[inv.long()].float()
    total = picked.sum(dim=1) if w is None else (picked * w[:, :, None]).sum(dim=1)
    if residual is not None:
        total = total + residual.float()
    out.copy_(total)
    return out


def _plain_combine_grad(s):
    flat = s["inv"].long()
    dout = s["dout"].float()
    s["dw"].copy_((s["y_perm"][flat].float() * dout[:, None, :]).sum(dim=2))
    s["dy_perm"][flat] = (s["w"][:, :, None] * dout[:, None, :]).to(s["dy_perm"].dtype)
    return [s["dy_perm"], s["dw"]]


def _plain_router_grad(s):
    c = s["case"]
    ids, w, dw = s["ids"].long(), s["w"], s["dw"]
    if c["renorm"]:
        dscore_w = w * (dw - (dw * w).sum(dim=1, keepdim=True))      # w dL/ds * s of each selected score s
    else:
        dscore_w = w * dw
    if c["score"] == "softmax":
        g = torch.zeros_like(s["logits"]).scatter_(1, ids, dscore_w)
        if not c["renorm"]:
            g = g - _scores(s["logits"], "softmax") * dscore_w.sum(dim=1, keepdim=True)
    else:
        l = s["logits"].gather(1, ids)
        soft = torch.clamp(l, min=0) + torch.log1p(torch.exp(-l.abs()))
        g = torch.zeros_like(s["logits"]).scatter_(1, ids, dscore_w * 0.5 * torch.sigmoid(l) / soft)
    s["dlogits"].copy_(g)
    return s["dlogits"]


def _act(z, act):
    if act == "relu":
        return torch.clamp(z, min=0)
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return z * 0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "swiglu":
        gate, up = z.chunk(2, dim=-1)
        return gate * torch.sigmoid(gate) * up
    return z


def _act_grad(dy, z, act):
    if act == "none":
        return dy
    if act == "relu":
        return dy * (z > 0)
    if act == "gelu":
        return dy * (0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi))
    if act == "silu":
        sig = torch.sigmoid(z)
        return dy * sig * (1 + z * (1 - sig))
    gate, up = z.chunk(2, dim=-1)
    sig = torch.sigmoid(gate)
    return torch.cat([dy * up * sig * (1 + gate * (1 - sig)), dy * gate * sig], dim=-1)


def _slots(s):
    """Row of each expert's i-th slot [E, most] (one past the last row where the expert has fewer rows)."""
    c = s["case"]
    counts = s["counts"].long()
    padded = (counts + c["align"] - 1) // c["align"] * c["align"]
    i = torch.arange(s["most"], device="cuda")
    rows = (torch.cumsum(padded, 0) - padded)[:, None] + i
    return torch.where(i < counts[:, None], rows, s["x"].shape[0])


def _by_expert(t, rows):
    return torch.cat([t, t.new_zeros((1, t.shape[1]))])[rows].float()


def _to_rows(out, v, rows):
    full = torch.cat([out, out.new_zeros((1, out.shape[1]))])
    full[rows] = v.to(out.dtype)
    out.copy_(full[:-1])
    return out


def _plain_linear(s):
    c = s["case"]
    rows = _slots(s) if c["E"] else None
    x = _by_expert(s["x"], rows) if c["E"] else s["x"].float()
    z = x @ s["w"].float().transpose(-1, -2)
    if s["bias"] is not None:
        z = z + (s["bias"][:, None, :] if c["E"] else s["bias"])
    y = _act(z, c["act"])
    if s["residual"] is not None:
        y = y + (_by_expert(s["residual"], rows) if c["E"] else s["residual"].float())
    outs = [(s["y"], y)] + ([(s["z"], z)] if s["z"] is not None else [])
    return [_to_rows(o, v, rows) if c["E"] else o.copy_(v) for o, v in outs]


def _plain_linear_grad(s):
    c = s["case"]
    rows = _slots(s) if c["E"] else None
    x, dy, z = [None if t is None else _by_expert(t, rows) if c["E"] else t.float() for t in (s["x"], s["dy"], s["z"])]
    dz = _act_grad(dy, z, c["act"])
    dx = dz @ s["w"].float()
    s["dx"] = _to_rows(s["dx"], dx, rows) if c["E"] else s["dx"].copy_(dx)
    s["dweight"].copy_(dz.transpose(-1, -2) @ x)
    outs = [s["dx"], s["dweight"]]
    if s["dbias"] is not None:
        outs.append(s["dbias"].copy_(dz.sum(dim=-2)))
    return outs


# ------------------------------------------------------------------------------------- a pass

def _own(s):
    import moe_expert_ffn_sqrt_gb300 as M
    c = s["case"]
    op = c["op"]
    if op in ("linear", "linear_grad"):
        if "ws" not in s:     # kept by the caller from call to call
            s["ws"] = M.new_workspace_linear(s["x"].shape[0], c["N"], c["K"], c["E"], c["act"])
        if op == "linear":
            M.linear(s["x"], s["w"], s["y"], s["ws"], bias=s["bias"], act=c["act"], residual=s["residual"], z=s["z"],
                     expert_counts=s["counts"], align=c["align"])
            return [s["y"]] + ([s["z"]] if s["z"] is not None else [])
        M.linear_backward(s["dy"], s["x"], s["w"], s["ws"], dx=s["dx"], dw=s["dweight"], dbias=s["dbias"],
                          act=c["act"], z=s["z"], expert_counts=s["counts"], align=c["align"])
        return [s["dx"], s["dweight"]] + ([s["dbias"]] if s["dbias"] is not None else [])
    if "ws" not in s:
        s["ws"] = M.new_workspace_rows(c["T"], c["K"], c["E"])
    if op == "dispatch":
        M.dispatch(s["ids"], s["x"], c["E"], c["align"], s["x_perm"], s["sorted"], s["experts"], s["inv"], s["m_sum"],
                   s["ws"], expert_counts=s["counts"])
        return [s[k] for k in ("sorted", "experts", "inv", "m_sum", "counts", "x_perm")]
    if op == "dispatch_grad":
        M.dispatch_backward(s["g_perm"], s["inv"], s["out"], s["ws"], residual=s["residual"])
        return s["out"]
    if op == "combine":
        M.combine(s["y_perm"], s["inv"], s["w"], s["out"], s["ws"], residual=s["residual"])
        return s["out"]
    if op == "combine_grad":
        M.combine_backward(s["dout"], s["y_perm"], s["inv"], s["w"], s["dy_perm"], s["dw"], s["ws"])
        return [s["dy_perm"], s["dw"]]
    M.route_backward(s["logits"], s["ids"], s["w"], s["dw"], c["score"], c["renorm"], s["dlogits"], s["ws"])
    return s["dlogits"]


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "dispatch":
        return _plain_dispatch(state)
    if op == "dispatch_grad":
        return _plain_gather_sum(state["g_perm"], state["inv"], None, state["residual"], state["out"])
    if op == "combine":
        return _plain_gather_sum(state["y_perm"], state["inv"], state["w"], state["residual"], state["out"])
    if op == "combine_grad":
        return _plain_combine_grad(state)
    if op == "router_grad":
        return _plain_router_grad(state)
    return _plain_linear(state) if op == "linear" else _plain_linear_grad(state)


# ------------------------------------------------------------------------------------- what it takes

def work(case):
    op = case["op"]
    if op == "router_grad":
        T, E, K = case["T"], case["E"], case["K"]
        reads = T * E * 4 if case["score"] == "softmax" and not case["renorm"] else T * K * 4
        return {"bytes": reads + 3 * T * K * 4 + T * E * 4, "flops": 4 * T * E}
    b = SIZE[case["dtype"]]
    if op in ("linear", "linear_grad"):
        M, N, K, E, act = case["M"], case["N"], case["K"], case["E"], case["act"]
        out = N // 2 if act == "swiglu" else N
        weight = max(1, min(E, M)) * N * K * b       # of the experts that have rows
        if op == "linear":
            rows = M * (K + out + (out if case["residual"] else 0) + (N if case["save"] else 0)) * b
            return {"bytes": weight + rows + (N * 4 if case["bias"] else 0), "flops": 2 * M * N * K}
        rows = M * (2 * K + out + (N if act != "none" else 0)) * b
        return {"bytes": weight + max(1, E) * N * K * b + rows, "flops": 4 * M * N * K}
    T, H, K = case["T"], case["H"], case["K"]
    index = T * K * 4
    if op == "dispatch":
        return {"bytes": (T + T * K) * H * b + 4 * index, "flops": 0}
    if op == "combine_grad":
        return {"bytes": (T + 2 * T * K) * H * b + 3 * index, "flops": 3 * T * K * H}
    extra = T if case["residual"] else 0
    return {"bytes": (T * K + T + extra) * H * b + (2 if op == "combine" else 1) * index, "flops": 2 * T * K * H}


# ------------------------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    f64 = torch.float64
    if op == "router_grad":
        # the chain rule over the whole row: weights -> scores -> logits
        l, ids, dw = s["logits"].to(f64), s["ids"].long(), s["dw"].to(f64)
        soft = torch.logaddexp(l, torch.zeros_like(l))
        score = torch.softmax(l, dim=1) if case["score"] == "softmax" else soft.sqrt()
        sel = score.gather(1, ids)
        if case["renorm"]:
            total = sel.sum(dim=1, keepdim=True)
            dsel = dw / total - (dw * sel).sum(dim=1, keepdim=True) / total ** 2
        else:
            dsel = dw
        ds = torch.zeros_like(score).scatter_add_(1, ids, dsel)
        if case["score"] == "softmax":
            return score * (ds - (ds * score).sum(dim=1, keepdim=True))
        return ds * torch.sigmoid(l) / (2 * score)
    if op not in ("linear", "linear_grad"):
        T, H, E, K, align = case["T"], case["H"], case["E"], case["K"], case["align"]
        if op == "dispatch":
            x_perm = torch.zeros((s["x_perm"].shape[0], H), dtype=f64, device="cuda")
            row = 0
            for e in range(E):
                pairs = (s["ids"].reshape(-1) == e).nonzero().reshape(-1)
                n = pairs.numel()
                x_perm[row:row + n] = s["x"][pairs // K].to(f64)
                row += (n + align - 1) // align * align
            return [None, None, None, None, None, x_perm]
        if op == "combine_grad":
            dy = torch.zeros(s["dy_perm"].shape, dtype=f64, device="cuda")
            dw = torch.zeros((T, K), dtype=f64, device="cuda")
            dout = s["dout"].to(f64)
            for k in range(K):
                row = s["inv"][:, k].long()
                dy[row] = dout * s["w"][:, k, None].to(f64)
                dw[:, k] = torch.einsum("th,th->t", dout, s["y_perm"][row].to(f64))
            return [dy, dw]
        rows = s["g_perm"] if op == "dispatch_grad" else s["y_perm"]
        out = torch.zeros((T, H), dtype=f64, device="cuda")
        for k in range(K):
            part = rows[s["inv"][:, k].long()].to(f64)
            out += part if op == "dispatch_grad" else part * s["w"][:, k, None].to(f64)
        return out if s["residual"] is None else out + s["residual"].to(f64)
    E, act, align = case["E"], case["act"], case["align"]
    parts, row = [], 0
    if E:
        for n in s["counts"].tolist():
            parts.append((row, n))
            row += (n + align - 1) // align * align
    else:
        parts.append((0, case["M"]))

    def one(t, e):
        return t[e] if E else t

    def phi(z):
        return 0.5 * torch.erfc(-z / math.sqrt(2.0))

    if case["op"] == "linear":
        y = torch.zeros(s["y"].shape, dtype=f64, device="cuda")
        zs = torch.zeros((s["y"].shape[0], case["N"]), dtype=f64, device="cuda")
        for e, (r, n) in enumerate(parts):
            z = torch.matmul(s["x"][r:r + n].to(f64), one(s["w"], e).to(f64).t())
            if s["bias"] is not None:
                z += one(s["bias"], e).to(f64)
            h = case["N"] // 2
            v = {"none": lambda: z, "relu": lambda: z.relu(), "silu": lambda: z / (1 + torch.exp(-z)),
                 "gelu": lambda: z * phi(z), "swiglu": lambda: z[:, :h] / (1 + torch.exp(-z[:, :h])) * z[:, h:]}[act]()
            if s["residual"] is not None:
                v = v + s["residual"][r:r + n].to(f64)
            y[r:r + n], zs[r:r + n] = v, z
        return [y] + ([zs] if s["z"] is not None else [])
    dx = torch.zeros(s["dx"].shape, dtype=f64, device="cuda")
    dw = torch.zeros(s["dweight"].shape, dtype=f64, device="cuda")
    db = torch.zeros(s["dweight"].shape[:-1], dtype=f64, device="cuda")
    for e, (r, n) in enumerate(parts):
        dz = s["dy"][r:r + n].to(f64)
        if act != "none":
            z = s["z"][r:r + n].to(f64)
            h = case["N"] // 2
            if act == "relu":
                dz = torch.where(z > 0, dz, torch.zeros_like(dz))
            elif act == "gelu":
                dz = dz * (phi(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi))
            elif act == "silu":
                t = 1 / (1 + torch.exp(-z))
                dz = dz * (t + z * t * (1 - t))
            else:
                a, b = z[:, :h], z[:, h:]
                t = 1 / (1 + torch.exp(-a))
                dz = torch.cat([dz * b * (t + a * t * (1 - t)), dz * a * t], dim=1)
        dx[r:r + n] = torch.matmul(dz, one(s["w"], e).to(f64))
        grad = torch.matmul(dz.t(), s["x"][r:r + n].to(f64))
        if E:
            dw[e], db[e] = grad, dz.sum(dim=0)
        else:
            dw, db = grad, dz.sum(dim=0)
    return [dx, dw] + ([db] if s["dbias"] is not None else [])
