"""SwiGLU over its gates on the GPU, with bounds relative to the results.

With s = sigmoid(g), c = 1 - s:  a = g s u,  dg = da u (s + g s c),  du = da g s.

fp32: t = exp(-|g|) is within 2 ulp, 1 / (1 + t) two roundings, s and c one product at most: each within
2^-21; two products and a sum: a and du within 2^-20 of themselves, dg within 2^-20 of |da u| s (1 + |g| c).

16 bits: the hardware exponential is within 2 + 1.173 |g| ulp (2^-23), a quotient within 2, two sums and products
half of one each, so s is within e = (8 + 1.173 |g|) 2^-23 of itself where g < 0; where g > 0 the exponential is
below 1 and its error's share in 1 + exp(-g) below one ulp: e = 8 2^-23.  c = 1 - s is off by e s + 2^-24, which
comes into dg times |g| s: together below |da u| ((e + 2^-22) s (1 + |g| c) + |g| s (e s + 2^-24))."""
import pytest
import torch

from mixture_experts_layer_stable_gb300 import ops

from ops_util import DT, U, close, gen

pytestmark = pytest.mark.gpu


def sweep(dt, lo, hi, rows=96, f=672):
    """Gates over [lo, hi] in order, up values and gradients that keep 16-bit results normal where it can be."""
    g = gen(21)
    gate = torch.linspace(lo, hi, rows * f, dtype=torch.float64, device="cuda").reshape(rows, f).to(DT[dt])
    rand = lambda: torch.rand(rows, f, generator=g, device="cuda") + 0.5  # noqa: E731
    up, da = rand(), rand()
    if dt == "f16":
        up = up * torch.where(gate < 0, 4e4, 4e2)
    up *= torch.where(rand() < 1, -1.0, 1.0)
    return torch.cat((gate, up.to(DT[dt])), 1), da.to(DT[dt])


def check(dt, got_a, got_dh, gate, up, da):
    f = gate.shape[1]
    s, c = torch.sigmoid(gate), torch.sigmoid(-gate)
    want = gate * s * up
    if dt == "f32":
        e = torch.full_like(gate, 2.0 ** -20)
        ea, eg = e * want.abs(), e * (da * up).abs() * s * (1 + gate.abs() * c)
        eu = e * (da * gate * s).abs()
    else:
        e = (8 + 1.173 * gate.abs() * (gate < 0)) * 2.0 ** -23
        ea = (e + 2.0 ** -22) * want.abs()
        eg = (da * up).abs() * ((e + 2.0 ** -22) * s * (1 + gate.abs() * c) + gate.abs() * s * (e * s + 2.0 ** -24))
        eu = (e + 2.0 ** -22) * (da * gate * s).abs()
    # (an error in front of the rounding moves it by up to half a step more of the moved value)
    close(got_a, want, dt, ea * (1 + U[dt]), "a")
    close(got_dh[:, :f], da * up * (s + gate * s * c), dt, eg * (1 + U[dt]), "dg")
    close(got_dh[:, f:], da * gate * s, dt, eu * (1 + U[dt]), "du")


@pytest.mark.parametrize("dt,lo,hi", [("f32", -86, 86), ("bf16", -86, 86), ("f16", -24, 86), ("f16", -86, -20), ("f32", -4, 4),
                                      ("bf16", -4, 4), ("f16", -4, 4), ("f32", 80, 3e4), ("bf16", 80, 3e4)])
@pytest.mark.parametrize("cut", [0, 1, 2])
def test_gates(cuda_lib, dt, lo, hi, cut):
    """Whole vectors, single elements and words; from h, and from its 8 bits with their values."""
    h, da = sweep(dt, lo, hi)
    rows, f = da.shape[0], da.shape[1] - cut
    h = torch.cat((h[:, :f], h[:, f + cut:2 * f + cut]), 1)
    da = da[:, :f].contiguous()
    a, dh, again = torch.empty_like(da), torch.empty_like(h), torch.empty_like(da)
    q = torch.empty(rows, 2 * f, dtype=torch.int8, device="cuda")
    sc = torch.empty(ops.moe_mxint8_scale_bytes(2 * rows, f), dtype=torch.uint8, device="cuda")
    ops.moe_swiglu_forward(h, a, q, sc)
    ops.moe_swiglu_backward(da, h, dh, again)
    assert torch.equal(a, again)
    check(dt, a, dh, h[:, :f].double(), h[:, f:].double(), da.double())
    kept = torch.empty(2 * rows, f, device="cuda")
    ops.moe_dequantize_mxint8_rows(q.reshape(2 * rows, f), sc, kept)
    kept = kept.reshape(rows, 2 * f).double()
    ops.moe_swiglu_backward(da, None, dh, again, q, sc)
    check(dt, again, dh, kept[:, :f], kept[:, f:], da.double())
