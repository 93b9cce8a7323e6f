"""One MoE layer trained with the library's training operators: routed experts next to a shared expert.

    out[t] = sum_k w[t,k] * W2[e_k] . swiglu(W13[e_k] . x[t])  +  V2 . swiglu(V13 . x[t]) + b

The routing, the rows' way to the experts and back, all products and all gradients run on the library's
kernels; torch holds the tensors and does the weight update.  Weights are bf16 with fp32 master copies.

    python examples/train_layer.py [--tokens 2048] [--steps 20]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import moe_expert_ffn_sqrt_gb300 as M  # noqa: E402

BF16 = torch.bfloat16


class TrainLayer:
    """Weights, workspaces and buffers for batches of T tokens."""

    def __init__(self, T, H=512, I=256, E=16, K=4, shared=256, align=128, score_fn="sqrt_softplus", seed=0):
        self.T, self.H, self.I, self.E, self.K, self.align, self.score_fn = T, H, I, E, K, align, score_fn
        g = torch.Generator().manual_seed(seed)

        def weight(*shape):
            return (torch.randn(*shape, generator=g) * shape[-1] ** -0.5).cuda()

        self.master = {"gate": weight(E, H), "w13": weight(E, 2 * I, H), "w2": weight(E, H, I), "v13": weight(2 * shared, H),
                       "v2": weight(H, shared), "b": torch.zeros(H, device="cuda")}
        self.w = {n: v.to(BF16) for n, v in self.master.items() if n not in ("gate", "b")}
        self.U = U = M.msum_upper(T, K, E, align)
        i32, f32, dev = torch.int32, torch.float32, "cuda"

        def rows(n, cols):
            return torch.zeros(n, cols, dtype=BF16, device=dev)

        self.logits = torch.empty(T, E, dtype=f32, device=dev)
        self.ids, self.topk_w = torch.empty(T, K, dtype=i32, device=dev), torch.empty(T, K, dtype=f32, device=dev)
        self.sorted, self.experts = (torch.empty(U, dtype=i32, device=dev) for _ in range(2))
        self.inv, self.m_sum = torch.empty(T, K, dtype=i32, device=dev), torch.empty(1, dtype=i32, device=dev)
        self.counts = torch.empty(E, dtype=i32, device=dev)
        self.x_perm, self.y_perm, self.z, self.h = rows(U, H), rows(U, H), rows(U, 2 * I), rows(U, I)
        self.sz, self.sh, self.mid, self.out = rows(T, 2 * shared), rows(T, shared), rows(T, H), rows(T, H)
        self.dy, self.dh, self.dx_perm = rows(U, H), rows(U, I), rows(U, H)
        self.dsh, self.dx_gate, self.dx_shared, self.dx = rows(T, shared), rows(T, H), rows(T, H), rows(T, H)
        self.dtopk_w, self.dlogits = torch.empty(T, K, device=dev), torch.empty(T, E, dtype=BF16, device=dev)
        self.grads = {n: torch.empty_like(v) for n, v in self.w.items()}
        self.grads["gate"], self.grads["b"] = torch.empty(E, H, dtype=BF16, device=dev), torch.empty(H, device=dev)
        self.ws_route = M.new_workspace(T, H, 128, E, K, align)
        self.ws_rows = M.new_workspace_rows(T, K, E)
        self.ws = {n: M.new_workspace_linear(*a) for n, a in (("up", (U, 2 * I, H, E, "swiglu")), ("down", (U, H, I, E)),
                                                             ("sup", (T, 2 * shared, H, 0, "swiglu")),
                                                             ("sdown", (T, H, shared)))}
        if E % 8 == 0:
            self.ws["gate"] = M.new_workspace_linear(T, E, H)

    def forward(self, x):
        """x [T, H] bf16 -> out [T, H] bf16."""
        w, exp = self.w, dict(expert_counts=self.counts, align=self.align)
        M.route(x, self.master["gate"], None, None, self.K, self.score_fn, True, self.ids, self.topk_w, self.ws_route,
                logits_out=self.logits)
        M.dispatch(self.ids, x, self.E, self.align, self.x_perm, self.sorted, self.experts, self.inv, self.m_sum,
                   self.ws_rows, expert_counts=self.counts)
        M.linear(self.x_perm, w["w13"], self.h, self.ws["up"], act="swiglu", z=self.z, **exp)
        M.linear(self.h, w["w2"], self.y_perm, self.ws["down"], **exp)
        M.combine(self.y_perm, self.inv, self.topk_w, self.mid, self.ws_rows)
        # the shared expert's down projection adds the routed experts' output as its residual
        M.linear(x, w["v13"], self.sh, self.ws["sup"], act="swiglu", z=self.sz)
        M.linear(self.sh, w["v2"], self.out, self.ws["sdown"], bias=self.master["b"], residual=self.mid)
        return self.out

    def backward(self, x, dout):
        """Gradients of the weights into self.grads; returns dx [T, H]."""
        w, g, exp = self.w, self.grads, dict(expert_counts=self.counts, align=self.align)
        # shared expert; the residual's gradient is dout itself
        M.linear_backward(dout, self.sh, w["v2"], self.ws["sdown"], dx=self.dsh, dw=g["v2"], dbias=g["b"])
        M.linear_backward(self.dsh, x, w["v13"], self.ws["sup"], dx=self.dx_shared, dw=g["v13"], act="swiglu", z=self.sz)
        # routed experts
        M.combine_backward(dout, self.y_perm, self.inv, self.topk_w, self.dy, self.dtopk_w, self.ws_rows)
        M.linear_backward(self.dy, self.h, w["w2"], self.ws["down"], dx=self.dh, dw=g["w2"], **exp)
        M.linear_backward(self.dh, self.x_perm, w["w13"], self.ws["up"], dx=self.dx_perm, dw=g["w13"], act="swiglu", z=self.z,
                          **exp)
        # router: weights -> logits -> gate; its dx joins the shared expert's, the rows' come last
        M.route_backward(self.logits, self.ids, self.topk_w, self.dtopk_w, self.score_fn, True, self.dlogits, self.ws_rows)
        if self.E % 8 == 0:
            M.linear_backward(self.dlogits, x, self.master["gate"].to(BF16), self.ws["gate"], dx=self.dx_gate, dw=g["gate"],
                              dx_residual=self.dx_shared)
        else:                  # rows of logits that are no whole 16 bytes: a small product for torch
            d = self.dlogits.float()
            g["gate"].copy_(d.t() @ x.float())
            self.dx_gate.copy_(d @ self.master["gate"] + self.dx_shared.float())
        M.dispatch_backward(self.dx_perm, self.inv, self.dx, self.ws_rows, residual=self.dx_gate)
        return self.dx

    def update(self, lr):
        for n, m in self.master.items():
            m.sub_(self.grads[n].float(), alpha=lr)
            if n in self.w:
                self.w[n].copy_(m)

    def check(self):
        """Raises if a kernel recorded a device error."""
        for ws in (self.ws_route, self.ws_rows, *self.ws.values()):
            st = M.get_error(ws)
            if st != M.OK:
                raise RuntimeError(M.status_str(st))


def main():
    p = argparse.ArgumentParser()
    p.add_argument("--tokens", type=int, default=2048)
    p.add_argument("--steps", type=int, default=20)
    p.add_argument("--lr", type=float, default=2.0)
    a = p.parse_args()
    torch.manual_seed(0)
    layer = TrainLayer(a.tokens)
    x = torch.randn(a.tokens, layer.H, device="cuda").to(BF16)
    target = torch.tanh(x.float() @ torch.randn(layer.H, layer.H, device="cuda") * layer.H ** -0.5)
    for step in range(a.steps):
        diff = layer.forward(x).float() - target
        loss = diff.square().mean()
        layer.backward(x, (diff * (2.0 / layer.H)).to(BF16))        # per token: the mean over its columns
        layer.update(a.lr / a.tokens)
        print(f"step {step:3d}  loss {float(loss):.5f}", flush=True)
    layer.check()


if __name__ == "__main__":
    main()
