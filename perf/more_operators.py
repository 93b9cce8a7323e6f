"""Workloads of the operators around the MoE layer, with their plain forms.

Three pairs of operators:

* norm    root-mean-square norm of a residual stream, with the addition that precedes it and outputs of the
          stream's type and in 8 bits (E4M3 codes with one power-of-two scale per 128 columns), and its gradients
* select  routing from logits: scores, a bias for balance, groups of experts, top-k, weights, and its gradient
* pack8   activations kept for the backward pass in 8 bits, and the gradients of a linear layer computed from them

``listed()`` names the workloads, ``draw(rng)`` gives others of the same ranges, ``prepare`` makes a
workload's inputs, ``run`` computes it (plain torch operations in 32 bits, or the package's kernels
where ``own`` is set), ``work`` counts what a pass cannot do without, and ``exact`` is the same result
in 64 bits.  8-bit outputs are returned as torch's 8-bit float types, codes and scales apart.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
GROUP = 128          # columns per scale
EPS = 1e-6


# ------------------------------------------------------------------------------------- workloads

def listed():
    return [
        # the norm in front of the layer when one token is decoded: residual added, 8-bit rows for the experts
        dict(name="norm-token", op="norm", T=1, H=7168, dtype="bf16", residual=True, y=True, q=True),
        # the same for the largest prefill batch
        dict(name="norm-prefill", op="norm", T=16384, H=7168, dtype="bf16", residual=True, y=True, q=True),
        # a ragged fp16 batch of a small model, no residual and no 8-bit rows
        dict(name="norm-ragged", op="norm", T=1111, H=1000, dtype="f16", residual=False, y=True, q=False),
        # both gradients in a training step, added to the gradient that the residual stream brought
        dict(name="norm-grad", op="norm_grad", T=8192, H=7168, dtype="bf16", dsum=True),
        # a small ragged model trained in fp32
        dict(name="norm-grad-ragged", op="norm_grad", T=333, H=1001, dtype="f32", dsum=False),
        # one decode step of 8 tokens: 8 groups of 32 experts, 4 of them used
        dict(name="select-few", op="select", T=8, E=256, K=6, score="sigmoid", G=8, KG=4, best=2, bias=True, renorm=True,
             scale=2.5, dtype="f32"),
        # the largest prefill or training batch
        dict(name="select-batch", op="select", T=16384, E=256, K=6, score="sigmoid", G=8, KG=4, best=2, bias=True,
             renorm=True, scale=2.5, dtype="f32"),
        # routing gradient of a training batch, for 16-bit logits
        dict(name="select-grad", op="select_grad", T=16384, E=256, K=6, score="sigmoid", renorm=True, scale=2.5,
             dtype="bf16"),
        # the layer's input kept in 8 bits
        dict(name="pack8-tokens", op="pack8", M=16384, C=7168, dtype="bf16"),
        # gate and up products of a small shared expert, odd sizes
        dict(name="pack8-ragged", op="pack8", M=777, C=1000, dtype="f16"),
        # training backward of a shared expert's gate and up projection from 8-bit x and z
        dict(name="linear8-grad", op="linear8_grad", M=4096, N=4096, K=7168, E=0, topk=0, align=0, act="swiglu",
             dtype="bf16", bias=False),
        # training backward of 32 experts (one of eight ranks' share of 256); the 8-bit rows are the tokens', read
        # through the routing instead of being kept once per expert
        dict(name="experts8-grad", op="linear8_grad", M=12288, N=4096, K=7168, E=32, topk=6, align=128, act="swiglu",
             dtype="bf16", bias=False),
    ]


def _log_int(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], evenly spread over its logarithm."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi)))) / step)) * step
    return max(n, step)


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_grad", "norm_grad", "select", "select", "select_grad", "pack8",
                     "linear8_grad", "linear8_grad"])
    if op in ("select", "select_grad"):
        E = _log_int(rng, 8, 512)
        T = _log_int(rng, 1, 16384)
        score = rng.choice(["softmax", "sqrt_softplus", "sigmoid"])
        case = dict(op=op, T=T, E=E, score=score, renorm=rng.random() < 0.6, scale=rng.choice([1.0, 2.5]),
                    dtype=rng.choice(["f32", "f32", "bf16", "f16"]))
        if op == "select":
            G = rng.choice([g for g in range(1, 33) if E % g == 0])
            KG = rng.randint(1, G)
            case.update(G=G, KG=KG, best=rng.choice([1, 2]), bias=rng.random() < 0.6, K=rng.randint(1, min(8, KG * (E // G))))
        else:
            case["K"] = rng.randint(2 if case["renorm"] else 1, min(8, E))     # (one normalised weight is a constant)
        return case
    if op == "linear8_grad":
        experts = rng.random() < 0.5
        N, K = _log_int(rng, 64, 4096, 16), _log_int(rng, 32, 7168, 8)
        M = _log_int(rng, 1, min(8192, int(4096 * 2048 * 7168 / (N * K))))
        E = _log_int(rng, 4, 32) if experts else 0
        topk = rng.randint(1, 4) if experts and rng.random() < 0.6 else 0
        return dict(op=op, M=(M + topk - 1) // topk * topk if topk else M, N=N, K=K, E=E, topk=topk,
                    align=rng.choice([1, 16, 64, 128, 256]) if experts else 0,
                    act=rng.choice(["none", "relu", "silu", "gelu", "swiglu"]), dtype=rng.choice(["bf16", "f16"]),
                    bias=rng.random() < 0.5)
    H = _log_int(rng, 64, 7168, 8) if rng.random() < 0.7 else _log_int(rng, 64, 7000, 2) + 1
    T = _log_int(rng, 1, min(16384, int(16384 * 7168 / (2 * H))))
    dtype = rng.choice(["bf16", "f16", "f32"])
    if op == "pack8":
        return dict(op=op, M=T, C=H, dtype=dtype)
    if op == "norm_grad":
        return dict(op=op, T=T, H=H, dtype=dtype, dsum=rng.random() < 0.5)
    y, q = rng.choice([(True, False), (False, True), (True, True)])
    return dict(op=op, T=T, H=H, dtype=dtype, residual=rng.random() < 0.5, y=y, q=q)


# ------------------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 6007 + 29)
    return g


def _normal(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _stream(g, T, H, dtype):
    """Rows of a residual stream: magnitudes differ from row to row, and a few columns are much larger than the others."""
    rows = torch.exp(torch.randn((T, 1), generator=g, device="cuda") * 0.7)
    cols = torch.where(torch.rand((1, H), generator=g, device="cuda") < 0.005, 20.0, 1.0)
    return (torch.randn((T, H), generator=g, device="cuda") * rows * cols).to(dtype)


def _room8(M, C):
    groups = (C + GROUP - 1) // GROUP
    return (torch.zeros((M, C), dtype=torch.uint8, device="cuda"), torch.zeros((M, groups), dtype=torch.uint8, device="cuda"))


def _positions(ids, E, align):
    """sorted pair of each row [U] (T*K on padding rows) and the counts [E], experts' segments padded to `align` rows."""
    flat = ids.reshape(-1).long()
    counts = torch.bincount(flat, minlength=E)
    padded = (counts + align - 1) // align * align
    seg = torch.cumsum(padded, 0) - padded
    order = torch.sort(flat, stable=True).indices
    rank = torch.arange(flat.numel(), device=flat.device) - (torch.cumsum(counts, 0) - counts)[flat[order]]
    pairs = torch.full((flat.numel() + E * (align - 1),), flat.numel(), dtype=torch.int32, device="cuda")
    pairs[seg[flat[order]] + rank] = order.to(torch.int32)
    return pairs, counts.to(torch.int32)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = {"case": case}
    if op in ("norm", "norm_grad"):
        T, H, dt = case["T"], case["H"], DTYPES[case["dtype"]]
        s["x"] = _stream(g, T, H, dt)
        s["w"] = torch.rand(H, generator=g, device="cuda") + 0.5
        if op == "norm":
            s["residual"] = _stream(g, T, H, dt) if case["residual"] else None
            s["sum"] = torch.zeros_like(s["x"]) if case["residual"] else None
            s["y"] = torch.zeros_like(s["x"]) if case["y"] else None
            s["y8"] = _room8(T, H) if case["q"] else None
        else:
            s["dy"] = _normal(g, (T, H), dt)
            s["dsum"] = _normal(g, (T, H), dt) if case["dsum"] else None
            s["dx"] = torch.zeros_like(s["x"])
            s["dw"] = torch.zeros(H, device="cuda")
        return s
    if op in ("select", "select_grad"):
        T, E, K = case["T"], case["E"], case["K"]
        s["logits"] = _normal(g, (T, E), DTYPES[case["dtype"]], 2.0)
        if op == "select":
            s["bias"] = torch.randn(E, generator=g, device="cuda") * 0.1 if case["bias"] else None
            s["ids"] = torch.zeros((T, K), dtype=torch.int32, device="cuda")
            s["w"] = torch.zeros((T, K), device="cuda")
        else:
            score = _scores(s["logits"].float(), case["score"])
            top = torch.sort(score, dim=1, descending=True, stable=True)
            s["ids"] = top.indices[:, :K].to(torch.int32).contiguous()
            w = top.values[:, :K]
            s["w"] = (w * case["scale"] / (w.sum(1, keepdim=True) if case["renorm"] else 1.0)).contiguous()
            s["dw"] = torch.randn((T, K), generator=g, device="cuda")
            s["dlogits"] = torch.zeros_like(s["logits"])
        return s
    dt = DTYPES[case["dtype"]]
    if op == "pack8":
        s["x"] = _stream(g, case["M"], case["C"], dt)
        s["x8"] = _room8(case["M"], case["C"])
        return s
    M, N, K, E, act, topk = case["M"], case["N"], case["K"], case["E"], case["act"], case["topk"]
    s["pairs"] = s["counts"] = None
    rows = tokens = M
    if E:
        rows = M + E * (case["align"] - 1)
        if topk:                            # the routing of M / topk tokens
            tokens = M // topk
            ids = torch.rand((tokens, E), generator=g, device="cuda").argsort(dim=1)[:, :topk]
            s["pairs"], s["counts"] = _positions(ids, E, case["align"])
        else:                               # rows packed as they are sorted, an expert or two without any
            ids = (torch.rand((M, 1), generator=g, device="cuda") ** 1.5 * E).long().clamp_(max=E - 1)
            _, s["counts"] = _positions(ids, E, case["align"])
            tokens = rows
    s["most"] = int(s["counts"].max()) if E else M
    s["x8"] = _room8(tokens, K)
    _pack8(_normal(g, (tokens, K), dt), s["x8"])
    s["z8"] = _room8(rows, N) if act != "none" else None
    if act != "none":
        _pack8(_normal(g, (rows, N), dt), s["z8"])
    s["w"] = _normal(g, (E, N, K) if E else (N, K), dt, 1.0 / math.sqrt(K))
    s["dy"] = _normal(g, (rows, N // 2 if act == "swiglu" else N), dt)
    s["dx"] = torch.zeros((rows, K), dtype=dt, device="cuda")
    s["dweight"] = torch.zeros_like(s["w"])
    s["dbias"] = torch.zeros((E, N) if E else (N,), device="cuda") if case["bias"] else None
    return s


# ------------------------------------------------------------------------------------- plain forms

def _pack8(v, room):
    """v [M, C] into codes and scales: per 128 columns the smallest power of two 2^e with amax <= 448 * 2^e."""
    q, sf = room
    M, C = v.shape
    groups = sf.shape[1]
    f = v.float()
    if C % GROUP:
        f = torch.cat([f, f.new_zeros((M, groups * GROUP - C))], dim=1)
    f = f.reshape(M, groups, GROUP)
    amax = torch.where(torch.isfinite(f), f.abs(), torch.zeros_like(f)).amax(dim=2)
    m, ex = torch.frexp(amax)                                   # amax = m * 2^ex, m in [0.5, 1); 448 = 0.875 * 2^9
    e = torch.where(amax == 0, torch.zeros_like(ex), torch.clamp(ex - 9 + (m > 0.875).to(ex.dtype), -127, 127))
    codes = (f * torch.exp2(-e.float())[:, :, None]).to(torch.float8_e4m3fn)
    q.copy_(codes.view(torch.uint8).reshape(M, groups * GROUP)[:, :C])
    sf.copy_((e + 127).to(torch.uint8))


def _values8(room):
    return [room[0].view(torch.float8_e4m3fn), room[1].view(torch.float8_e8m0fnu)]


def _unpack8(room):
    q, sf = room
    scale = torch.exp2(sf.float() - 127.0).repeat_interleave(GROUP, dim=1)[:, :q.shape[1]]
    return q.view(torch.float8_e4m3fn).float() * scale


def _plain_norm(s):
    v = s["x"]
    out = {}
    if s["residual"] is not None:
        s["sum"].copy_(v.float() + s["residual"].float())
        v = out["sum"] = s["sum"]                # the norm is of the stream as it is stored
    f = v.float()
    y = f * torch.rsqrt((f * f).mean(dim=1, keepdim=True) + EPS) * s["w"]
    if s["y"] is not None:
        out["y"] = s["y"].copy_(y)
    if s["y8"] is not None:
        _pack8(y, s["y8"])
        out["y8"] = _values8(s["y8"])
    return out


def _plain_norm_grad(s):
    v, dy = s["x"].float(), s["dy"].float()
    r = torch.rsqrt((v * v).mean(dim=1, keepdim=True) + EPS)
    h, g = v * r, dy * s["w"]
    dx = (g - h * (g * h).mean(dim=1, keepdim=True)) * r
    if s["dsum"] is not None:
        dx = dx + s["dsum"].float()
    s["dw"].copy_((dy * h).sum(dim=0))
    return [s["dx"].copy_(dx), s["dw"]]


def _scores(l, fn):
    if fn == "softmax":
        e = torch.exp(l - l.amax(dim=1, keepdim=True))
        return e / e.sum(dim=1, keepdim=True)
    if fn == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-l))
    return torch.sqrt(torch.clamp(l, min=0) + torch.log1p(torch.exp(-l.abs())))


def _plain_select(s):
    c = s["case"]
    T, E, K, G = c["T"], c["E"], c["K"], c["G"]
    score = _scores(s["logits"].double(), c["score"])        # in 64 bits: neighbouring scores decide
    key = score if s["bias"] is None else score + s["bias"].double()
    if c["KG"] < G:
        by_group = torch.sort(key.reshape(T, G, E // G), dim=2, descending=True).values[:, :, :c["best"]].sum(dim=2)
        best = torch.sort(by_group, dim=1, descending=True, stable=True).indices[:, :c["KG"]]
        kept = torch.zeros((T, G), dtype=torch.bool, device="cuda").scatter_(1, best, True)
        key = torch.where(kept.repeat_interleave(E // G, dim=1), key, torch.full_like(key, -math.inf))
    ids = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :K]
    w = score.gather(1, ids)
    if c["renorm"]:
        w = w / w.sum(dim=1, keepdim=True)
    s["ids"].copy_(ids)
    s["w"].copy_(w * c["scale"])
    return [s["ids"], s["w"]]


def _plain_select_grad(s):
    c = s["case"]
    l, ids, w, dw = s["logits"].float(), s["ids"].long(), s["w"], s["dw"]
    if c["renorm"]:                                            # g = s dL/ds of each selected score s
        g = w * (dw - (dw * w).sum(dim=1, keepdim=True) / c["scale"])
    else:
        g = w * dw
    if c["score"] == "softmax":
        full = torch.zeros_like(l).scatter_(1, ids, g)
        if not c["renorm"]:
            full = full - _scores(l, "softmax") * g.sum(dim=1, keepdim=True)
    else:
        t = l.gather(1, ids)
        if c["score"] == "sigmoid":
            g = g / (1.0 + torch.exp(t))
        else:
            g = g * 0.5 / (1.0 + torch.exp(-t)) / (torch.clamp(t, min=0) + torch.log1p(torch.exp(-t.abs())))
        full = torch.zeros_like(l).scatter_(1, ids, g)
    return s["dlogits"].copy_(full)


def _act_grad(dy, z, act):
    if act == "none":
        return dy
    if act == "relu":
        return dy * (z > 0)
    if act == "gelu":
        return dy * (0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi))
    if act == "silu":
        sig = 1.0 / (1.0 + torch.exp(-z))
        return dy * sig * (1 + z * (1 - sig))
    gate, up = z.chunk(2, dim=-1)
    sig = 1.0 / (1.0 + torch.exp(-gate))
    return torch.cat([dy * up * sig * (1 + gate * (1 - sig)), dy * gate * sig], dim=-1)


def _slots(s):
    """Row of each expert's i-th slot [E, most] (one past the last row where the expert has fewer rows)."""
    c = s["case"]
    counts = s["counts"].long()
    padded = (counts + c["align"] - 1) // c["align"] * c["align"]
    i = torch.arange(s["most"], device="cuda")
    rows = (torch.cumsum(padded, 0) - padded)[:, None] + i
    return torch.where(i < counts[:, None], rows, s["dy"].shape[0])


def _by_expert(t, rows):
    return torch.cat([t, t.new_zeros((1, t.shape[1]))])[rows].float()


def _plain_linear8_grad(s):
    c = s["case"]
    x, z = _unpack8(s["x8"]), None if s["z8"] is None else _unpack8(s["z8"])
    dy, rows = s["dy"].float(), None
    if c["E"]:
        rows = _slots(s)
        if s["pairs"] is not None:          # a sorted row's token; none on padding rows
            x = torch.cat([x, x.new_zeros((1, x.shape[1]))])[s["pairs"].long() // c["topk"]]
        x, dy, z = [None if t is None else _by_expert(t, rows) for t in (x, dy, z)]
    dz = _act_grad(dy, z, c["act"])
    dx = dz @ s["w"].float()
    if rows is None:
        s["dx"].copy_(dx)
    else:
        full = torch.cat([s["dx"], s["dx"].new_zeros((1, c["K"]))])
        full[rows] = dx.to(full.dtype)
        s["dx"].copy_(full[:-1])
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
    if op == "norm":
        M.rms_norm(s["x"], s["w"], EPS, residual=s["residual"], sum_out=s["sum"], y=s["y"], y8=s["y8"])
        out = {k: s[k] for k in ("sum", "y") if s[k] is not None}
        if s["y8"] is not None:
            out["y8"] = _values8(s["y8"])
        return out
    if op == "norm_grad":
        if "ws" not in s:     # kept by the caller from call to call
            s["ws"] = M.new_workspace_norm(c["T"], c["H"])
        M.rms_norm_backward(s["dy"], s["x"], s["w"], EPS, s["dx"], s["ws"], dweight=s["dw"], dsum=s["dsum"])
        return [s["dx"], s["dw"]]
    if op == "select":
        M.select(s["logits"], s["ids"], s["w"], c["score"], e_score_bias=s["bias"], n_groups=c["G"], topk_groups=c["KG"],
                 group_best=c["best"], renormalize=c["renorm"], scale=c["scale"])
        return [s["ids"], s["w"]]
    if op == "select_grad":
        if "ws" not in s:
            s["ws"] = M.new_workspace_rows(c["T"], c["K"], c["E"])
        M.select_backward(s["logits"], s["ids"], s["w"], s["dw"], s["dlogits"], s["ws"], c["score"],
                          renormalize=c["renorm"], scale=c["scale"])
        return s["dlogits"]
    if op == "pack8":
        M.pack_rows8(s["x"], s["x8"])
        return _values8(s["x8"])
    if "ws" not in s:
        s["ws"] = M.new_workspace_linear8(s["dy"].shape[0], c["N"], c["K"], c["E"], c["act"])
    M.linear_backward8(s["dy"], s["w"], s["ws"], x8=s["x8"], z8=s["z8"], x_ids=s["pairs"], x_div=max(1, c["topk"]),
                       dx=s["dx"], dw=s["dweight"], dbias=s["dbias"], act=c["act"], expert_counts=s["counts"],
                       align=c["align"])
    return [s["dx"], s["dweight"]] + ([s["dbias"]] if s["dbias"] is not None else [])


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "norm":
        return _plain_norm(state)
    if op == "norm_grad":
        return _plain_norm_grad(state)
    if op == "select":
        return _plain_select(state)
    if op == "select_grad":
        return _plain_select_grad(state)
    if op == "pack8":
        _pack8(state["x"], state["x8"])
        return _values8(state["x8"])
    return _plain_linear8_grad(state)


# ------------------------------------------------------------------------------------- what it takes

def work(case):
    op = case["op"]
    b = SIZE[case["dtype"]]
    if op == "norm":
        T, H = case["T"], case["H"]
        row = H * b * (1 + 2 * case["residual"] + case["y"]) + (H + (H + GROUP - 1) // GROUP) * case["q"]
        return {"bytes": T * row + 4 * H, "flops": 6 * T * H}
    if op == "norm_grad":
        T, H = case["T"], case["H"]
        return {"bytes": T * H * b * (3 + case["dsum"]) + 8 * H, "flops": 12 * T * H}
    if op == "select":
        T, E, K = case["T"], case["E"], case["K"]
        return {"bytes": T * E * b + 8 * T * K + 4 * E * case["bias"], "flops": 8 * T * E}
    if op == "select_grad":
        T, E, K = case["T"], case["E"], case["K"]
        dense = case["score"] == "softmax" and not case["renorm"]
        read = T * E * b if dense else T * K * b * (case["score"] != "softmax")
        return {"bytes": read + 12 * T * K + T * E * b, "flops": 4 * T * K + 4 * T * E * dense}
    if op == "pack8":
        M, C = case["M"], case["C"]
        return {"bytes": M * (C * (b + 1) + (C + GROUP - 1) // GROUP), "flops": 2 * M * C}
    M, N, K, E, act, topk = case["M"], case["N"], case["K"], case["E"], case["act"], case["topk"]
    out = N // 2 if act == "swiglu" else N
    kept = (M // topk if topk else M) * (K + (K + GROUP - 1) // GROUP)        # x in 8 bits
    if act != "none":
        kept += M * (N + (N + GROUP - 1) // GROUP)                            # z in 8 bits
    weight = max(1, min(E, M)) * N * K * b       # of the experts that have rows
    grads = M * K * b + max(1, E) * N * K * b + 4 * max(1, E) * N * case["bias"]
    return {"bytes": kept + M * out * b + weight + grads + 4 * M * (topk > 0), "flops": 4 * M * N * K}


# ------------------------------------------------------------------------------------- in 64 bits

F64 = torch.float64


def _exact8(y):
    """Codes and scales of y (64 bits), as values: steps of the code's last place instead of a conversion."""
    M, C = y.shape
    groups = (C + GROUP - 1) // GROUP
    codes = torch.zeros((M, C), dtype=F64, device="cuda")
    scales = torch.zeros((M, groups), dtype=F64, device="cuda")
    for k in range(groups):
        part = y[:, k * GROUP:(k + 1) * GROUP]
        amax = part.abs().amax(dim=1)
        e = torch.ceil(torch.log2(amax / 448.0))
        e = torch.where(448.0 * torch.exp2(e) < amax, e + 1, e)               # (the logarithm's own rounding)
        e = torch.where(448.0 * torch.exp2(e - 1) >= amax, e - 1, e)
        e = torch.where(amax == 0, torch.zeros_like(e), e.clamp(-127, 127))
        v = part / torch.exp2(e)[:, None]
        last = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3      # three bits after the leading one
        codes[:, k * GROUP:(k + 1) * GROUP] = torch.round(v / torch.exp2(last)) * torch.exp2(last)
        scales[:, k] = torch.exp2(e)
    return [codes, scales]


def _table8(room):
    """The values of 8-bit rows, by a table of the 256 codes."""
    q, sf = room
    code = torch.arange(256, device="cuda")
    exp, man = (code >> 3) & 15, code & 7
    mag = torch.where(exp == 0, man * 2.0 ** -9, (8 + man) * torch.exp2((exp - 10).to(F64)))
    table = torch.where(code >= 128, -mag, mag).to(F64)
    out = table[q.long()]
    for k in range(sf.shape[1]):
        out[:, k * GROUP:(k + 1) * GROUP] *= torch.exp2(sf[:, k:k + 1].to(F64) - 127)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        out = {}
        v = s["x"].to(F64)
        if s["residual"] is not None:
            out["sum"] = v + s["residual"].to(F64)
            v = out["sum"].to(s["x"].dtype).to(F64)
        y = v * s["w"].to(F64) / torch.sqrt(torch.einsum("th,th->t", v, v) / case["H"] + EPS)[:, None]
        if s["y"] is not None:
            out["y"] = y
        if s["y8"] is not None:
            out["y8"] = _exact8(y)
        return out
    if op == "norm_grad":
        v, dy, w = s["x"].to(F64), s["dy"].to(F64), s["w"].to(F64)
        n = torch.sqrt(torch.einsum("th,th->t", v, v) / case["H"] + EPS)
        along = torch.einsum("th,th,h->t", v, dy, w) / case["H"]
        dx = dy * w / n[:, None] - v * (along / n ** 3)[:, None]
        if s["dsum"] is not None:
            dx += s["dsum"].to(F64)
        return [dx, torch.einsum("th,th,t->h", dy, v, 1 / n)]
    if op == "select":
        # expert by expert from the largest key down
        T, E, K, G = case["T"], case["E"], case["K"], case["G"]
        l = s["logits"].to(F64)
        score = {"softmax": lambda: torch.softmax(l, 1), "sigmoid": lambda: torch.sigmoid(l),
                 "sqrt_softplus": lambda: torch.logaddexp(l, torch.zeros_like(l)).sqrt()}[case["score"]]()
        key = score if s["bias"] is None else score + s["bias"].to(F64)
        parts = key.reshape(T, G, E // G)
        first = parts.amax(2)
        if case["best"] == 2 and E // G > 1:
            at = parts.argmax(2, keepdim=True)
            first = first + parts.scatter(2, at, -math.inf).amax(2)
        open_ = torch.zeros((T, G), dtype=torch.bool, device="cuda")
        for _ in range(case["KG"]):
            at = first.argmax(1, keepdim=True)
            open_.scatter_(1, at, True)
            first = first.scatter(1, at, -math.inf)
        key = torch.where(open_[:, :, None], parts, torch.full_like(parts, -math.inf)).reshape(T, E)
        picked = []
        for _ in range(K):
            at = key.argmax(1, keepdim=True)
            picked.append(score.gather(1, at))
            key = key.scatter(1, at, -math.inf)
        w = torch.cat(picked, dim=1)
        return [None, w * case["scale"] / (w.sum(1, keepdim=True) if case["renorm"] else 1.0)]
    if op == "select_grad":
        # the chain rule over the whole row: weights -> scores -> logits
        l, ids, dw = s["logits"].to(F64), s["ids"].long(), s["dw"].to(F64) * case["scale"]
        soft = torch.logaddexp(l, torch.zeros_like(l))
        score = {"softmax": lambda: torch.softmax(l, 1), "sigmoid": lambda: torch.sigmoid(l),
                 "sqrt_softplus": lambda: soft.sqrt()}[case["score"]]()
        sel = score.gather(1, ids)
        if case["renorm"]:
            total = sel.sum(dim=1, keepdim=True)
            dw = dw / total - (dw * sel).sum(dim=1, keepdim=True) / total ** 2
        ds = torch.zeros_like(score).scatter_add_(1, ids, dw)
        if case["score"] == "softmax":
            return score * (ds - (ds * score).sum(dim=1, keepdim=True))
        return ds * (score * torch.sigmoid(-l) if case["score"] == "sigmoid" else torch.sigmoid(l) / (2 * score))
    if op == "pack8":
        return _exact8(s["x"].to(F64))
    E, act, topk, align, h = case["E"], case["act"], case["topk"], case["align"], case["N"] // 2
    x8, z8 = _table8(s["x8"]), None if s["z8"] is None else _table8(s["z8"])
    dx = torch.zeros(s["dx"].shape, dtype=F64, device="cuda")
    dw = torch.zeros(s["dweight"].shape, dtype=F64, device="cuda")
    db = torch.zeros(s["dweight"].shape[:-1], dtype=F64, device="cuda")
    row = 0
    for e, n in enumerate(s["counts"].tolist() if E else [case["M"]]):
        part = slice(row, row + n)
        dz = s["dy"][part].to(F64)
        x = x8[s["pairs"][part].long() // topk] if topk else x8[part]
        if act != "none":
            z = z8[part]
            if act == "relu":
                dz = torch.where(z > 0, dz, torch.zeros_like(dz))
            elif act == "gelu":
                dz = dz * (0.5 * torch.erfc(-z / math.sqrt(2)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi))
            elif act == "silu":
                t = torch.sigmoid(z)
                dz = dz * (t + z * t * (1 - t))
            else:
                a, b = z[:, :h], z[:, h:]
                t = torch.sigmoid(a)
                dz = torch.cat([dz * b * (t + a * t * (1 - t)), dz * a * t], dim=1)
        wd, dd, bd = (s["w"][e], dw[e], db[e]) if E else (s["w"], dw, db)
        dx[part] = torch.matmul(dz, wd.to(F64))
        dd.copy_(torch.matmul(dz.t(), x))
        bd.copy_(dz.sum(dim=0))
        row += (n + align - 1) // align * align if E else n
    return [dx, dw] + ([db] if s["dbias"] is not None else [])
