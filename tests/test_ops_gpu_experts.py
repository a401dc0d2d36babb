"""The products, SwiGLU and the checkpoints together on the GPU: the example's experts in a training step,
against 64 bits."""
import importlib.util
import os

import pytest
import torch

from mixture_experts_layer_stable_gb300 import ops

from ops_util import DT, gen, randn

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ffn(cuda_lib):
    spec = importlib.util.spec_from_file_location("expert_ffn", os.path.join(ROOT, "examples", "expert_ffn.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def problem(seed, T, d, f, E, k, dtype=torch.float32):
    g = gen(seed)
    x, dout = randn(g, T, d, dtype=dtype), randn(g, T, d, dtype=dtype)
    nw, nb = randn(g, d, dtype=dtype, mean=1.0, std=0.2), randn(g, d, dtype=dtype)
    W1, W2 = randn(g, E, d, 2 * f, dtype=dtype, std=d ** -0.5), randn(g, E, f, d, dtype=dtype, std=f ** -0.5)
    w = torch.softmax(randn(g, T, k), 1)
    ids = torch.rand(T, E, generator=g, device="cuda").topk(k).indices.to(torch.int32).reshape(-1)
    return x, dout, nw, nb, W1, W2, w, ids


def norm64(x, w, b):
    c = x - x.mean(1, keepdim=True)
    return c / torch.sqrt((c * c).mean(1, keepdim=True) + 1e-5) * w + b


class Kept(torch.autograd.Function):
    """The value in the forward, the one kept in 8 bits in the backward: passes its gradient on."""

    @staticmethod
    def forward(ctx, h, f, kept):
        ctx.save_for_backward(kept)
        ctx.f = f
        return torch.nn.functional.silu(h[:, :f]) * h[:, f:]

    @staticmethod
    def backward(ctx, da):
        (kept,), f = ctx.saved_tensors, ctx.f
        g, u = kept[:, :f], kept[:, f:]
        s = torch.sigmoid(g)
        return torch.cat((da * u * (s + g * s * (1 - s)), da * g * s), 1), None, None


@pytest.mark.parametrize("keep_rows", [True, False])
@pytest.mark.parametrize("T,d,f,E,k,cap", [(1, 64, 32, 4, 2, 8), (50, 96, 40, 6, 3, 20), (200, 130, 67, 9, 4, 1000)])
def test_training_step_in_fp32(ffn, T, d, f, E, k, cap, keep_rows):
    """fp32 operators against fp64 with the same 8-bit values in the backward: sums of at most 4 d or T k
    terms, whose fp32 error stays below 1e-5 of the gradients' norms."""
    x, dout, nw, nb, W1, W2, w, ids = problem(T + d, T, d, f, E, k)
    ids = ffn.cap_ids(ids, E, cap)
    R = T * k
    m = ffn.SwiGLUExperts(W1, W2, R, keep_rows)
    out, grads = ffn.train_step(x, nw, nb, ids, w, E, m.forward, m.backward, dout)
    assert m.status() == 0
    # the kept values, in expert order
    kh = torch.empty(2 * R, f, device="cuda")
    ops.moe_dequantize_mxint8_rows(m.hq.reshape(2 * R, f), m.hs, kh)
    kh = kh.reshape(R, 2 * f).double()
    px, pw, pb, pk, p1, p2 = (t.double().requires_grad_() for t in (x, nw, nb, w, W1, W2))
    xn = norm64(px, pw, pb)
    order = sorted(range(R), key=lambda r: (int(ids[r]) if ids[r] >= 0 else E))
    kept = int((ids >= 0).sum())
    perm = torch.tensor(order, device="cuda")[:kept]
    e = ids[perm].long()
    rows = xn[perm // k]
    if not keep_rows:  # the weights' gradient sees the rows in 8 bits, the rest the rows themselves
        kx = torch.empty(R, d, device="cuda")
        ops.moe_dequantize_mxint8_rows(m.xq, m.xs, kx)
        kx = kx[:kept].double()
        assert bool(((kx - rows).abs() <= rows.abs().amax(1, keepdim=True) / 127 + 1e-5).all())
    h = torch.einsum("pk,pkn->pn", rows, p1[e])
    tol = torch.cat((h[:, :f].abs().amax(1, keepdim=True).expand(-1, f), h[:, f:].abs().amax(1, keepdim=True).expand(-1, f)), 1)
    assert bool(((kh[:kept] - h).abs() <= tol / 127 + 1e-5).all())
    a = Kept.apply(h, f, kh[:kept])
    y = torch.einsum("pk,pkn->pn", a, p2[e])
    ref = px.index_add(0, perm // k, y * pk.reshape(-1)[perm][:, None])
    ref.backward(dout.double())
    assert (out.double() - ref).norm() <= 1e-5 * ref.norm()
    for name, p in (("x", px), ("norm_w", pw), ("norm_b", pb), ("weights", pk)):
        assert (grads[name].double() - p.grad).norm() <= 1e-5 * p.grad.norm() + 1e-6, name
    # the weights' gradients from the 8-bit activation (and rows)
    dy = (dout.double()[perm // k] * w.double().reshape(-1)[perm][:, None])
    g, u = kh[:kept, :f], kh[:kept, f:]
    s = torch.sigmoid(g)
    da = torch.einsum("pn,pkn->pk", dy, W2.double()[e])
    dh = torch.cat((da * u * (s + g * s * (1 - s)), da * g * s), 1)
    d2 = torch.zeros(E, f, d, dtype=torch.float64, device="cuda").index_add_(0, e, torch.einsum("pk,pn->pkn", g * s * u, dy))
    d1 = torch.zeros(E, d, 2 * f, dtype=torch.float64, device="cuda").index_add_(
        0, e, torch.einsum("pk,pn->pkn", rows.detach() if keep_rows else kx, dh))
    assert (m.dW2.double() - d2).norm() <= 1e-5 * d2.norm() + 1e-6
    assert (m.dW1.double() - d1).norm() <= 1e-5 * d1.norm() + 1e-6


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_16_bit_gradients_are_near_autograd(ffn, dt):
    """Against fp64 autograd without any rounding: the 8-bit values are off by at most 1/127 of their
    block's largest (norm-wise below 1 %), the 16-bit arrays by 2^-8 or less each; a handful of such factors
    stay below 5 % of the gradients' norms."""
    T, d, f, E, k = 300, 256, 128, 8, 2
    x, dout, nw, nb, W1, W2, w, ids = problem(5, T, d, f, E, k, DT[dt])
    m = ffn.SwiGLUExperts(W1, W2, T * k)
    out, grads = ffn.train_step(x, nw, nb, ids, w, E, m.forward, m.backward, dout)
    p = {n: t.double().requires_grad_() for n, t in dict(x=x, norm_w=nw, norm_b=nb, weights=w, W1=W1, W2=W2).items()}
    xn = norm64(p["x"], p["norm_w"], p["norm_b"])
    e = ids.long()
    h = torch.einsum("pk,pkn->pn", xn.repeat_interleave(k, 0), p["W1"][e])
    y = torch.einsum("pk,pkn->pn", torch.nn.functional.silu(h[:, :f]) * h[:, f:], p["W2"][e])
    ref = p["x"] + (y * p["weights"].reshape(-1, 1)).reshape(T, k, d).sum(1)
    ref.backward(dout.double())
    assert (out.double() - ref).norm() <= 0.02 * ref.norm()
    for n, v in dict(grads, W1=m.dW1, W2=m.dW2).items():
        assert (v.double() - p[n].grad).norm() <= 0.05 * p[n].grad.norm(), n


def test_gradients_add_up_and_a_captured_step_repeats(ffn):
    """Two batches' weight gradients are the sum of each alone, and a captured step gives the eager one's bits."""
    T, d, f, E, k = 64, 128, 64, 4, 2
    a, b = problem(1, T, d, f, E, k, torch.bfloat16), problem(2, T, d, f, E, k, torch.bfloat16)
    W1, W2 = a[4], a[5]

    def step(m, q):
        x, dout, nw, nb, _, _, w, ids = q
        return ffn.train_step(x, nw, nb, ids, w, E, m.forward, m.backward, dout)

    alone = []
    for q in (a, b):
        m = ffn.SwiGLUExperts(W1, W2, T * k)
        step(m, q)
        alone.append((m.dW1.clone(), m.dW2.clone()))
    m = ffn.SwiGLUExperts(W1, W2, T * k)
    step(m, a)
    step(m, b)
    for got, u, v in zip((m.dW1, m.dW2), *alone):
        # the second sum starts from the first: one more rounding of each
        assert bool(((got - (u + v)).abs() <= 2.0 ** -22 * (u.abs() + v.abs()) + 1e-7).all())
    m.reset()
    out, _ = step(m, a)
    want = [t.clone() for t in (out, m.dW1, m.dW2)]
    m.reset()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        out, _ = step(m, a)
    m.dW1.fill_(9)
    m.dW2.fill_(9)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for x, y in zip((out, m.dW1, m.dW2), want):
        assert torch.equal(x, y)
    assert m.status() == 0


def test_example_runs(ffn, capsys):
    ffn.main()
    assert "kept between" in capsys.readouterr().out
