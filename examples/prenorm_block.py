"""A pre-norm expert block, x + experts(norm(x)), from the package's operators.

Block4Bit serves it with expert weights frozen in 4 bits:
  layer norm -> router, top-k and schedule (moe_route) -> the normalised rows
  quantised in expert order -> first product with SwiGLU -> quantised again ->
  second product -> rows back to token order, weighted, added to x.

train_step runs forward and backward of the same block around an expert function
of the program's own: rows sorted by expert (rows over an expert's capacity
dropped), moved to it and back, and every gradient of the moves and the norm.

  python examples/prenorm_block.py
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from mixture_experts_layer_stable_gb300 import binding as B, ops  # noqa: E402

EPS = 1e-5


def _bytes(n):
    return torch.empty(n, dtype=torch.uint8, device="cuda")


class Block4Bit:
    """norm_w, norm_b [d], w_router [E, d], W1 [E, d, 2f] and W2 [E, f, d] in bf16, for T tokens of
    k experts each.  The experts' weights are quantised here, once."""

    def __init__(self, norm_w, norm_b, w_router, W1, W2, T, k):
        E, d, f2 = W1.shape
        self.norm_w, self.norm_b, self.w_router, self.k = norm_w, norm_b, w_router, k
        self.w1, self.s1 = _bytes(E * f2 * d // 2).view(E, f2, d // 2), _bytes(ops.moe_mxfp4_weight_scale_bytes(E, d, f2))
        self.w2, self.s2 = _bytes(E * d * f2 // 4).view(E, d, f2 // 4), _bytes(ops.moe_mxfp4_weight_scale_bytes(E, f2 // 2, d))
        ops.moe_quantize_mxfp4(W1, self.w1, self.s1, paired=True)
        ops.moe_quantize_mxfp4(W2, self.w2, self.s2)
        self.cfg = B.make_config(T, d, f2 // 2, E, k)
        self.sched, self.route_ws = B.alloc_sched(self.cfg), B.alloc_workspace(self.cfg)
        self.logits = torch.empty(T, E, device="cuda")
        R, bf = T * k, dict(dtype=torch.bfloat16, device="cuda")
        self.xn, self.out = torch.empty(T, d, **bf), torch.empty(T, d, **bf)
        self.a, self.y = torch.empty(R, f2 // 2, **bf), torch.empty(R, d, **bf)
        self.xq, self.xs = _bytes(R * d // 2), _bytes(ops.moe_mxfp4_row_scale_bytes(R, d, E))
        self.aq, self.as_ = _bytes(R * f2 // 4), _bytes(ops.moe_mxfp4_row_scale_bytes(R, f2 // 2, E))
        # a workspace for each product: its status is that of the last call that was given it
        self.ws1 = _bytes(ops.moe_mxfp4_product_workspace_bytes(R, f2, d, E))
        self.ws = _bytes(ops.moe_mxfp4_product_workspace_bytes(R, d, f2 // 2, E))

    def status(self):
        """The first error of the last call's bounded waits, 0 if there was none (synchronises)."""
        return next((e for e in map(B.moe_read_status, (self.route_ws, self.ws1, self.ws)) if e), 0)

    def __call__(self, x):
        s, off = self.sched, self.sched["offsets"]
        ops.moe_layernorm_forward(x, self.norm_w, self.norm_b, EPS, self.xn)
        B.moe_route(self.cfg, self.xn, self.w_router, self.logits, s, self.route_ws)
        ops.moe_quantize_mxfp4_rows(self.xn, self.xq, self.xs, off, perm=s["perm"], k=self.k)
        ops.moe_mxfp4_product(self.xq, self.xs, off, self.w1, self.s1, ops.MOE_ACT_SWIGLU, self.a, self.ws1)
        ops.moe_quantize_mxfp4_rows(self.a, self.aq, self.as_, off)
        ops.moe_mxfp4_product(self.aq, self.as_, off, self.w2, self.s2, ops.MOE_ACT_NONE, self.y, self.ws)
        ops.moe_unpermute(self.y, s["topk_w"], self.k, s["inv"], off, self.out, base=x)
        return self.out


def cap_ids(ids, E, capacity):
    """ids with the rows past the first `capacity` of each expert marked -1 (they are dropped).
    An id outside [0, E) is dropped already and stays."""
    one = (ids[:, None] == torch.arange(E, device=ids.device)).int()
    rank = (one.cumsum(0) * one).sum(1) - 1
    return torch.where(rank < capacity, ids, torch.full_like(ids, -1))


def train_step(x, norm_w, norm_b, ids, weights, E, experts, experts_backward, dout):
    """out = x + sum_j weights[t, j] * expert(norm(x)[t]) and its gradients for dout.
    ids [T*k] int32, weights [T, k] fp32; experts(rows, offsets) -> y and
    experts_backward(dy, rows, offsets) -> drows work on rows in expert order."""
    T, d = x.shape
    k = weights.shape[1]
    R, like = T * k, dict(dtype=x.dtype, device=x.device)
    i32 = dict(dtype=torch.int32, device=x.device)
    xn, out, dxn, dx = (torch.empty(T, d, **like) for _ in range(4))
    mean, rstd = torch.empty(T, device=x.device), torch.empty(T, device=x.device)
    counts, offsets = torch.empty(E, **i32), torch.empty(E + 1, **i32)
    perm, inv = torch.empty(R, **i32), torch.empty(R, **i32)
    rows, dy = torch.empty(R, d, **like), torch.empty(R, d, **like)
    dweights = torch.empty(R, device=x.device)
    dnorm_w, dnorm_b = torch.empty_like(norm_w), torch.empty_like(norm_b)
    # forward
    ops.moe_layernorm_forward(x, norm_w, norm_b, EPS, xn, mean, rstd)
    ops.moe_sort_rows(ids, counts, offsets, perm, inv, _bytes(ops.moe_sort_workspace_bytes(R, E)))
    ops.moe_permute(xn, k, inv, offsets, rows)
    y = experts(rows, offsets)
    ops.moe_unpermute(y, weights, k, inv, offsets, out, base=x)
    # backward
    ops.moe_unpermute_backward(dout, y, weights, k, inv, offsets, dy, dweights)
    drows = experts_backward(dy, rows, offsets)
    ops.moe_unpermute(drows, None, k, inv, offsets, dxn)
    ops.moe_layernorm_backward(dxn, x, norm_w, mean, rstd, dx, dnorm_w, dnorm_b,
                               _bytes(ops.moe_layernorm_workspace_bytes(T, d)), dadd=dout)
    return out, dict(x=dx, norm_w=dnorm_w, norm_b=dnorm_b, weights=dweights.view(T, k))


def main():
    g = torch.Generator(device="cuda").manual_seed(0)

    def randn(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(torch.bfloat16)

    T, d, f, E, k = 256, 1024, 512, 16, 4
    norm_w, norm_b = randn(d, std=0.1) + 1, randn(d, std=0.1)
    block = Block4Bit(norm_w, norm_b, randn(E, d, std=d ** -0.5), randn(E, d, 2 * f, std=d ** -0.5),
                      randn(E, f, d, std=f ** -0.5), T, k)
    x = randn(T, d)
    out = block(x)
    assert block.status() == 0, B.moe_status_string(block.status())
    print("4-bit block: out - x has rms %.3f" % (out.float() - x.float()).square().mean().sqrt().item())

    scale = randn(E, d)

    def of_row(offsets):  # expert of every row, E past the last
        return torch.searchsorted(offsets[1:], torch.arange(T * k, device="cuda", dtype=torch.int32), right=True)

    def experts(rows, offsets):
        return rows * torch.cat((scale, torch.zeros_like(scale[:1])))[of_row(offsets)]

    def experts_backward(dy, rows, offsets):
        return experts(dy, offsets)

    ids = cap_ids(torch.rand(T, E, generator=g, device="cuda").topk(k).indices.to(torch.int32).reshape(-1), E, T * k // E)
    weights = torch.softmax(torch.randn(T, k, generator=g, device="cuda"), 1)
    out, grads = train_step(x, norm_w, norm_b, ids, weights, E, experts, experts_backward, randn(T, d))
    print("training step:", ", ".join("|d%s| %.2f" % (n, v.float().norm().item()) for n, v in grads.items()))


if __name__ == "__main__":
    main()
