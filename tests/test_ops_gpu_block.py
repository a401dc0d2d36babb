"""The operators together, as examples/prenorm_block.py runs them, against the block in 64 bits.

The 4-bit block is compared with the same steps on the values the kernels themselves
quantised (read back), so that only roundings of bf16 are between the two: the norm's
output, the SwiGLU output and the second product are rounded once each (2^-8 relative,
random signs), which the products average; 2e-2 of the norm of out - x is four such
roundings.  Codes of the SwiGLU output come from the kernel's own bf16 values."""
import importlib.util
import os

import pytest
import torch

from mixture_experts_layer_stable_gb300 import binding as B
from mixture_experts_layer_stable_gb300 import ops

from ops_util import gen, randn

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def block(cuda_lib):
    spec = importlib.util.spec_from_file_location("prenorm_block", os.path.join(ROOT, "examples", "prenorm_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def norm64(x, w, b, eps=1e-5):
    x = x.double()
    xc = x - x.mean(1, keepdim=True)
    return xc / torch.sqrt((xc * xc).mean(1, keepdim=True) + eps) * w.double() + b.double()


@pytest.mark.parametrize("T,d,f,E,k", [(1, 256, 128, 8, 2), (37, 512, 192, 12, 3), (300, 1024, 512, 16, 4)])
def test_four_bit_block(block, T, d, f, E, k):
    g = gen(T)
    bf = torch.bfloat16
    nw, nb = randn(g, d, dtype=bf, std=0.1, mean=1.0), randn(g, d, dtype=bf, std=0.1)
    wr = randn(g, E, d, dtype=bf, std=d ** -0.5)
    W1, W2 = randn(g, E, d, 2 * f, dtype=bf, std=d ** -0.5), randn(g, E, f, d, dtype=bf, std=f ** -0.5)
    m = block.Block4Bit(nw, nb, wr, W1, W2, T, k)
    x = randn(g, T, d, dtype=bf)
    out = m(x)
    assert B.moe_read_status(m.route_ws) == 0 and B.moe_read_status(m.ws) == 0
    # the values behind the codes
    v1, v2 = torch.empty(E, d, 2 * f, device="cuda"), torch.empty(E, f, d, device="cuda")
    ops.moe_dequantize_mxfp4(m.w1, m.s1, v1, paired=True)
    ops.moe_dequantize_mxfp4(m.w2, m.s2, v2)
    off = m.sched["offsets"]
    xv, av = torch.empty(T * k, d, device="cuda"), torch.empty(T * k, f, device="cuda")
    ops.moe_dequantize_mxfp4_rows(m.xq, m.xs, xv, off)
    ops.moe_dequantize_mxfp4_rows(m.aq, m.as_, av, off)
    assert (m.xn.double() - norm64(x, nw, nb)).norm() <= 2.0 ** -8 * norm64(x, nw, nb).norm()
    perm = m.sched["perm"].long()
    # 4 bits of the normalised rows: a step of E2M1 is at most a third of the value above it
    assert (xv.double() - m.xn.double()[perm // k]).norm() <= 0.2 * m.xn.double().norm() * k ** 0.5
    y = torch.zeros(T * k, d, dtype=torch.float64, device="cuda")
    a = torch.zeros(T * k, f, dtype=torch.float64, device="cuda")
    o = off.tolist()
    for e in range(E):
        s = slice(o[e], o[e + 1])
        h = xv[s].double() @ v1[e].double()
        a[s] = torch.nn.functional.silu(h[:, :f]) * h[:, f:]
        y[s] = av[s].double() @ v2[e].double()
    assert (m.a.double() - a).norm() <= 2.0 ** -8 * a.norm() * 1.5
    want = torch.zeros(T, d, dtype=torch.float64, device="cuda")
    want.index_add_(0, perm // k, y * m.sched["topk_w"].double()[perm][:, None])
    assert (out.double() - x.double() - want).norm() <= 2e-2 * want.norm() + 2.0 ** -8 * x.double().norm()


@pytest.mark.parametrize("T,d,E,k,cap", [(1, 64, 4, 2, 8), (50, 96, 6, 3, 20), (200, 513, 9, 4, 1000)])
def test_training_step_against_autograd(block, T, d, E, k, cap):
    """fp32 operators against fp64 autograd of the same block; every sum has at most 4 d terms, whose
    fp32 error stays below 1e-5 of the gradients' norms."""
    g = gen(T + d)
    x, dout = randn(g, T, d), randn(g, T, d)
    nw, nb, scale = randn(g, d, mean=1.0, std=0.2), randn(g, d), randn(g, E, d)
    w = torch.softmax(randn(g, T, k), 1)
    ids = torch.rand(T, E, generator=g, device="cuda").topk(k).indices.to(torch.int32).reshape(-1)
    ids = block.cap_ids(ids, E, cap)
    table = torch.cat((scale, torch.zeros_like(scale[:1])))

    def of_row(off):
        return torch.searchsorted(off[1:], torch.arange(T * k, device="cuda", dtype=torch.int32), right=True)

    out, grads = block.train_step(x, nw, nb, ids, w, E, lambda r, o: r * table[of_row(o)],
                                  lambda dy, r, o: dy * table[of_row(o)], dout)
    px, pw, pb, pk = (t.double().requires_grad_() for t in (x, nw, nb, w))
    xn = norm64(px, pw, pb)
    kept = (ids >= 0).reshape(T, k)
    sel = table.double()[torch.where(ids >= 0, ids, E).long()].reshape(T, k, d)
    ref = px + (pk * kept)[:, :, None].mul(sel).mul(xn[:, None, :]).sum(1)
    ref.backward(dout.double())
    assert (out.double() - ref).norm() <= 1e-5 * ref.norm()
    for name, p in (("x", px), ("norm_w", pw), ("norm_b", pb), ("weights", pk)):
        assert (grads[name].double() - p.grad).norm() <= 1e-5 * p.grad.norm() + 1e-7, name


def test_graph_capture(block):
    """The serving block in a CUDA graph gives the same bits (every launch is capturable)."""
    g = gen(3)
    bf = torch.bfloat16
    T, d, f, E, k = 64, 512, 256, 8, 2
    m = block.Block4Bit(randn(g, d, dtype=bf), randn(g, d, dtype=bf), randn(g, E, d, dtype=bf, std=d ** -0.5),
                        randn(g, E, d, 2 * f, dtype=bf, std=d ** -0.5), randn(g, E, f, d, dtype=bf, std=f ** -0.5), T, k)
    x = randn(g, T, d, dtype=bf)
    want = m(x).clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m(x)
    m.out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(m.out, want)
    x.copy_(randn(g, T, d, dtype=bf))
    graph.replay()
    torch.cuda.synchronize()
    got = m.out.clone()
    assert torch.equal(m(x), got)


def test_every_product_s_status_is_seen(block):
    """An error that either product reported is not cleared by the other's call."""
    g = gen(4)
    bf = torch.bfloat16
    T, d, f, E, k = 16, 256, 128, 4, 2
    m = block.Block4Bit(randn(g, d, dtype=bf), randn(g, d, dtype=bf), randn(g, E, d, dtype=bf, std=d ** -0.5),
                        randn(g, E, d, 2 * f, dtype=bf, std=d ** -0.5), randn(g, E, f, d, dtype=bf, std=f ** -0.5), T, k)
    x = randn(g, T, d, dtype=bf)
    m(x)
    assert m.status() == 0
    for ws in (m.ws1, m.ws, m.route_ws):
        ws[:4].view(torch.int32).fill_(B.MOE_ERR_TIMEOUT)     # as a wait that ran out leaves it
        assert m.status() == B.MOE_ERR_TIMEOUT
        m(x)
        assert m.status() == 0
    # the second product alone does not touch the first one's
    m.ws1[:4].view(torch.int32).fill_(B.MOE_ERR_TIMEOUT)
    ops.moe_mxfp4_product(m.aq, m.as_, m.sched["offsets"], m.w2, m.s2, ops.MOE_ACT_NONE, m.y, m.ws)
    assert m.status() == B.MOE_ERR_TIMEOUT
