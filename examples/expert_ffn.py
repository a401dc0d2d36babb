"""A training step around experts of the program's own: the pre-norm block of
prenorm_block.py with SwiGLU experts from the package's products.

  forward   rows -> product with W1 -> SwiGLU -> product with W2
  backward  dy -> product with W2 transposed -> SwiGLU's backward -> product with
            W1 transposed, and the weights' gradients

Between the two only 8 bits an element are kept: of the SwiGLU's input always (its
output is computed again in the backward), of the rows if keep_rows is false.

  python examples/expert_ffn.py
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from mixture_experts_layer_stable_gb300 import binding as B, ops  # noqa: E402
from prenorm_block import cap_ids, train_step  # noqa: E402


def _bytes(n):
    return torch.empty(n, dtype=torch.uint8, device="cuda")


class SwiGLUExperts:
    """W1 [E, d, 2f] (gate | up) and W2 [E, f, d] for up to `rows` rows in expert order; their gradients are
    added to dW1 and dW2 (fp32), from zero after reset()."""

    def __init__(self, W1, W2, rows, keep_rows=False):
        E, d, f2 = W1.shape
        f, like = f2 // 2, dict(dtype=W1.dtype, device="cuda")
        self.W1, self.W2, self.keep_rows, self.fresh = W1, W2, keep_rows, True
        self.dW1, self.dW2 = (torch.empty(w.shape, device="cuda") for w in (W1, W2))
        # work arrays: the product's results, the activation (computed again in the backward), the rows' gradient
        self.h, self.a = torch.empty(rows, f2, **like), torch.empty(rows, f, **like)
        self.y, self.dx = torch.empty(rows, d, **like), torch.empty(rows, d, **like)
        # kept from the forward to the backward
        self.hq, self.hs = torch.empty(rows, f2, dtype=torch.int8, device="cuda"), _bytes(ops.moe_mxint8_scale_bytes(2 * rows, f))
        if not keep_rows:
            self.xq, self.xs = torch.empty(rows, d, dtype=torch.int8, device="cuda"), _bytes(ops.moe_mxint8_scale_bytes(rows, d))
        self.ws1 = _bytes(ops.moe_grouped_product_workspace_bytes(rows, d, f2, E))
        self.ws2 = _bytes(ops.moe_grouped_product_workspace_bytes(rows, f, d, E))

    def reset(self):
        self.fresh = True

    def status(self):
        """The first error of the last calls' bounded waits, 0 if there was none (synchronises)."""
        return next((e for e in map(B.moe_read_status, (self.ws1, self.ws2)) if e), 0)

    def forward(self, rows, offsets):
        n = rows.shape[0]
        h, a, y = self.h[:n], self.a[:n], self.y[:n]
        ops.moe_grouped_product(rows, self.W1, offsets, h, self.ws1)
        ops.moe_swiglu_forward(h, a, self.hq[:n], self.hs)
        ops.moe_grouped_product(a, self.W2, offsets, y, self.ws2)
        if not self.keep_rows:
            ops.moe_quantize_mxint8_rows(rows, self.xq[:n], self.xs)
        return y

    def backward(self, dy, rows, offsets):
        """The rows' gradient; of `rows` nothing is read unless keep_rows."""
        n = dy.shape[0]
        # h's place takes dh, the activation's its gradient and then the activation again
        add, a, dh, dx = not self.fresh, self.a[:n], self.h[:n], self.dx[:n]
        ops.moe_grouped_product(dy, self.W2, offsets, a, self.ws2, transposed=True)
        ops.moe_swiglu_backward(a, None, dh, a, self.hq[:n], self.hs)
        ops.moe_grouped_product_dw(a, dy, offsets, self.dW2, self.ws2, accumulate=add)
        ops.moe_grouped_product(dh, self.W1, offsets, dx, self.ws1, transposed=True)
        if not self.keep_rows:
            rows = self.y[:n]
            ops.moe_dequantize_mxint8_rows(self.xq[:n], self.xs, rows)
        ops.moe_grouped_product_dw(rows, dh, offsets, self.dW1, self.ws1, accumulate=add)
        self.fresh = False
        return dx


def main():
    g = torch.Generator(device="cuda").manual_seed(0)

    def randn(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(torch.bfloat16)

    T, d, f, E, k = 1024, 1024, 512, 16, 4
    R = T * k
    experts = SwiGLUExperts(randn(E, d, 2 * f, std=d ** -0.5), randn(E, f, d, std=f ** -0.5), R)
    norm_w, norm_b = randn(d, std=0.1) + 1, randn(d, std=0.1)
    for _ in range(2):  # two batches' gradients
        x, dout = randn(T, d), randn(T, d)
        ids = cap_ids(torch.rand(T, E, generator=g, device="cuda").topk(k).indices.to(torch.int32).reshape(-1), E, 2 * R // E)
        weights = torch.softmax(torch.randn(T, k, generator=g, device="cuda"), 1)
        out, grads = train_step(x, norm_w, norm_b, ids, weights, E, experts.forward, experts.backward, dout)
    assert experts.status() == 0, B.moe_status_string(experts.status())
    kept = sum(t.nbytes for t in (experts.hq, experts.hs, experts.xq, experts.xs))
    print("kept between forward and backward: %.1f MB (in 16 bits, with the activation, %.1f)" % (
        kept / 1e6, R * (d + 3 * f) * 2 / 1e6))
    print("gradients:", ", ".join("|d%s| %.2f" % (n, v.float().norm().item()) for n, v in
                                  dict(grads, W1=experts.dW1, W2=experts.dW2).items()))


if __name__ == "__main__":
    main()
