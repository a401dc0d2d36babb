"""SwiGLU's backward in place on the GPU, over the ways in which rows move: vectors, words and single elements, with
strides, from h and from its checkpoint."""
import pytest
import torch

from mixture_experts_layer_stable_gb300 import ops

from ops_util import DT, gen, strided

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("f,pad,shift", [(512, 0, 0), (500, 0, 0), (500, 4, 4), (1002, 2, 2), (333, 0, 0), (333, 5, 3), (8200, 0, 0)])
def test_in_place(cuda_lib, dt, f, pad, shift):
    g = gen(f + pad)
    rows = 70
    h, da = strided(g, rows, 2 * f, DT[dt], pad, shift, std=2.0), strided(g, rows, f, DT[dt], pad, shift)
    q = torch.empty(rows, 2 * f, dtype=torch.int8, device="cuda")
    s = torch.empty(ops.moe_mxint8_scale_bytes(2 * rows, f), dtype=torch.uint8, device="cuda")
    a = torch.empty(rows, f, dtype=DT[dt], device="cuda")
    ops.moe_swiglu_forward(h, a, q, s)
    for kept in (True, False):
        src = (None, q, s) if kept else (h, None, None)
        dh, again = torch.empty(rows, 2 * f, dtype=DT[dt], device="cuda"), torch.empty_like(a)
        ops.moe_swiglu_backward(da, src[0], dh, again, src[1], src[2])
        for h_too, a_too in ((True, False), (False, True), (True, True)):
            h2, da2 = strided(g, rows, 2 * f, DT[dt], pad, shift), strided(g, rows, f, DT[dt], pad, shift)
            h2.copy_(h)
            da2.copy_(da)
            dh2 = h2 if h_too else torch.empty_like(dh)
            again2 = da2 if a_too else torch.empty_like(again)
            ops.moe_swiglu_backward(da2, None if kept else h2, dh2, again2, src[1], src[2])
            assert torch.equal(dh2, dh) and torch.equal(again2, again), (kept, h_too, a_too)
