"""The products, SwiGLU and the checkpoints without a GPU: sizes and refusals (argument errors return
before any CUDA call), and what the binding refuses."""
import pytest
import torch

INV, SMALL, OK = 1, 3, 0
P = 1 << 20  # a 128-byte aligned address that is never read


@pytest.fixture(scope="module")
def O():
    from mixture_experts_layer_stable_gb300 import build, ops
    build.build()
    ops.lib()
    return ops


def test_sizes(O):
    ws = O.moe_grouped_product_workspace_bytes
    assert ws(0, 8, 8, 1) >= 8 and ws(4096, 2048, 1536, 64) >= 8
    for bad in ((-1, 8, 8, 1), (4, 0, 8, 1), (4, 8, 0, 1), (4, 8, 8, 0), (4, 8, 8, 1025), ((1 << 28) + 1, 8, 8, 1),
                (4, (1 << 22) + 1, 8, 1), (1 << 28, 1 << 20, 8, 1), (4, 1 << 22, 1 << 22, 1)):
        assert ws(*bad) == 0, bad
    # K and N in each other's place need the same: one workspace serves the forward and both gradients
    for rows, K, N, G in ((8, 7168, 256, 1), (3636, 84, 6373, 1), (5000, 128, 256, 2), (1, 1, 1, 1), (100, 4096, 24, 3)):
        assert ws(rows, K, N, G) == ws(rows, N, K, G) >= 128
    s = O.moe_mxint8_scale_bytes
    assert s(3, 1) == 3 and s(3, 32) == 3 and s(3, 33) == 6 and s(0, 5) == 0
    assert s(-1, 32) == 0 and s(1, 0) == 0 and s(1, (1 << 22) + 1) == 0


def test_product_refusals(O):
    L = O.lib()

    def prod(dt=1, odt=1, n=4, K=8, N=16, G=2, off=P, x=P, ldx=8, w=P, t=0, out=P, ldo=16, ws=P, wsb=1 << 30):
        return L.moe_grouped_product(dt, odt, n, K, N, G, off, x, ldx, w, t, out, ldo, ws, wsb, None)

    for bad in (dict(dt=3), dict(dt=-1), dict(odt=2), dict(dt=0, odt=1), dict(n=-1), dict(n=(1 << 28) + 1), dict(K=0),
                dict(N=0), dict(G=0), dict(G=1025), dict(off=None), dict(off=P + 2), dict(x=None), dict(x=P + 1), dict(ldx=7),
                dict(w=None), dict(w=P + 1), dict(out=None), dict(out=P + 1), dict(odt=0, out=P + 2), dict(ldo=15),
                dict(ws=None), dict(ws=P + 64)):
        assert prod(**bad) == INV, bad
    assert prod(wsb=0) == SMALL
    assert prod(n=0, x=None, out=None, w=None) == OK

    def dw(dt=1, wdt=1, n=4, K=8, N=16, G=2, off=P, x=P, ldx=8, dy=P, lddy=16, dw=P, acc=0, ws=P, wsb=1 << 30):
        return L.moe_grouped_product_dw(dt, wdt, n, K, N, G, off, x, ldx, dy, lddy, dw, acc, ws, wsb, None)

    for bad in (dict(dt=3), dict(wdt=2), dict(dt=0, wdt=1), dict(n=-1), dict(K=0), dict(N=0), dict(G=0), dict(off=None),
                dict(x=None), dict(ldx=7), dict(dy=None), dict(dy=P + 1), dict(lddy=15), dict(dw=None), dict(wdt=0, dw=P + 2),
                dict(ws=None), dict(ws=P + 4)):
        assert dw(**bad) == INV, bad
    assert dw(wsb=8) == SMALL


def test_checkpoint_refusals(O):
    L = O.lib()

    def quant(dt=1, n=4, d=40, x=P, ldx=40, q=P, s=P):
        return L.moe_quantize_mxint8_rows(dt, n, d, x, ldx, q, s, None)

    for bad in (dict(dt=3), dict(n=-1), dict(n=(1 << 30) + 1), dict(d=0), dict(d=(1 << 22) + 1, ldx=1 << 23), dict(ldx=39),
                dict(x=None), dict(x=P + 1), dict(q=None), dict(s=None)):
        assert quant(**bad) == INV, bad
        b = dict(bad)
        assert L.moe_dequantize_mxint8_rows(b.get("dt", 1), b.get("n", 4), b.get("d", 40), b.get("q", P), b.get("s", P),
                                            b.get("x", P), b.get("ldx", 40), None) == INV, bad
    assert quant(n=0, x=None, q=None, s=None) == OK

    def fwd(dt=1, n=4, f=40, h=P, ldh=80, a=P, lda=40, q=P, s=P):
        return L.moe_swiglu_forward(dt, n, f, h, ldh, a, lda, q, s, None)

    for bad in (dict(dt=3), dict(n=-1), dict(f=0), dict(h=None), dict(h=P + 1), dict(ldh=79), dict(a=None), dict(lda=39),
                dict(q=None), dict(s=None)):
        assert fwd(**bad) == INV, bad
    assert fwd(n=0, h=None, a=None, q=None, s=None) == OK

    def bwd(dt=1, n=4, f=40, da=P, ldda=40, h=P, ldh=80, q=P, s=P, dh=P, lddh=80, a=P, lda=40):
        return L.moe_swiglu_backward(dt, n, f, da, ldda, h, ldh, q, s, dh, lddh, a, lda, None)

    for bad in (dict(dt=3), dict(n=-1), dict(f=0), dict(da=None), dict(ldda=39), dict(ldh=79), dict(h=None, q=None, s=None),
                dict(q=None), dict(s=None), dict(dh=None), dict(dh=P + 1), dict(lddh=79), dict(a=P + 1), dict(lda=39)):
        assert bwd(**bad) == INV, bad
    assert bwd(n=0, da=None, h=None, dh=None, a=None) == OK


def _calls(O, device):
    """(function, its tensors) of a small valid call of every operator."""
    def t(*shape, dtype=torch.float32):
        return torch.zeros(*shape, dtype=dtype, device=device)

    off = torch.tensor([0, 3, 4], dtype=torch.int32, device=device)
    ws = t(O.moe_grouped_product_workspace_bytes(4, 8, 16, 2), dtype=torch.uint8)
    q, s = t(4, 80, dtype=torch.int8), t(O.moe_mxint8_scale_bytes(8, 40), dtype=torch.uint8)
    return [
        (lambda *a: O.moe_grouped_product(*a, stream=0), [t(4, 8), t(2, 8, 16), off, t(4, 16), ws]),
        (lambda *a: O.moe_grouped_product(*a, transposed=True, stream=0), [t(4, 16), t(2, 8, 16), off, t(4, 8), ws]),
        (lambda *a: O.moe_grouped_product_dw(*a, stream=0), [t(4, 8), t(4, 16), off, t(2, 8, 16), ws]),
        (lambda *a: O.moe_quantize_mxint8_rows(*a, stream=0), [t(4, 80), q, t(4 * 3, dtype=torch.uint8)]),
        (lambda *a: O.moe_dequantize_mxint8_rows(*a, stream=0), [q, t(4 * 3, dtype=torch.uint8), t(4, 80)]),
        (lambda *a: O.moe_swiglu_forward(*a, stream=0), [t(4, 80), t(4, 40), q, s]),
        (lambda *a: O.moe_swiglu_backward(*a, stream=0), [t(4, 40), t(4, 80), t(4, 80), t(4, 40)]),
        (lambda *a: O.moe_swiglu_backward(a[0], None, *a[1:], stream=0), [t(4, 40), t(4, 80), t(4, 40), q, s]),
    ]


def _misfits(O, device):
    """Calls whose tensors do not fit together."""
    def t(*shape, dtype=torch.float32):
        return torch.zeros(*shape, dtype=dtype, device=device)

    off, ws, q, s = t(3, dtype=torch.int32), t(4096, dtype=torch.uint8), t(4, 80, dtype=torch.int8), t(16, dtype=torch.uint8)
    x, w, y = t(4, 8), t(2, 8, 16), t(4, 16)
    return [
        lambda: O.moe_grouped_product(x, w, off, t(3, 16), ws),
        lambda: O.moe_grouped_product(x, w, off, t(4, 15), ws),
        lambda: O.moe_grouped_product(x, t(2, 16, 8), off, y, ws),
        lambda: O.moe_grouped_product(x, w, off, y, ws, transposed=True),
        lambda: O.moe_grouped_product(x, w, t(4, dtype=torch.int32), y, ws),
        lambda: O.moe_grouped_product(x, w, off.long(), y, ws),
        lambda: O.moe_grouped_product(x, w.half(), off, y, ws),
        lambda: O.moe_grouped_product(x.half(), w.half(), off, y.bfloat16(), ws),
        lambda: O.moe_grouped_product(x.double(), w.double(), off, y.double(), ws),
        lambda: O.moe_grouped_product(t(8, 4).t(), w, off, y, ws),
        lambda: O.moe_grouped_product(x, w, None, y, ws),
        lambda: O.moe_grouped_product_dw(x, t(3, 16), off, w, ws),
        lambda: O.moe_grouped_product_dw(x, y.half(), off, w, ws),
        lambda: O.moe_grouped_product_dw(x, y, off, t(2, 16, 8), ws),
        lambda: O.moe_grouped_product_dw(x, y, off, w.half(), ws),
        lambda: O.moe_quantize_mxint8_rows(t(4, 81), q, s),
        lambda: O.moe_quantize_mxint8_rows(t(4, 80), q.byte(), s),
        lambda: O.moe_quantize_mxint8_rows(t(4, 80), q, s[:11]),
        lambda: O.moe_swiglu_forward(t(4, 79), t(4, 40)),
        lambda: O.moe_swiglu_forward(t(4, 80).half(), t(4, 40)),
        lambda: O.moe_swiglu_forward(t(4, 80), t(4, 40), q),
        lambda: O.moe_swiglu_forward(t(4, 80), t(4, 40), q, s[:15]),
        lambda: O.moe_swiglu_backward(t(4, 40), t(3, 80), t(4, 80)),
        lambda: O.moe_swiglu_backward(t(4, 40), None, t(4, 80)),
        lambda: O.moe_swiglu_backward(t(4, 40), t(4, 80), t(4, 80), t(4, 41)),
    ]


def test_binding_refuses_host_tensors(O):
    from mixture_experts_layer_stable_gb300.binding import MoeError
    for f, tensors in _calls(O, "cpu"):
        with pytest.raises(MoeError) as e:
            f(*tensors)
        assert e.value.code == INV
    for f in _misfits(O, "cpu"):
        with pytest.raises(MoeError):
            f()


@pytest.mark.gpu
def test_binding_refuses_what_does_not_fit_on_the_gpu(O, cuda_lib, monkeypatch):
    from mixture_experts_layer_stable_gb300.binding import MoeError
    calls = _calls(O, "cuda")
    torch.cuda.synchronize()
    for n, (f, tensors) in enumerate(calls):
        f(*tensors)
        for i in range(len(tensors)):
            mixed = list(tensors)
            mixed[i] = tensors[i].cpu()
            with pytest.raises(MoeError) as e:
                f(*mixed)
            assert e.value.code == INV, (n, i)
    torch.cuda.synchronize()
    for n, f in enumerate(_misfits(O, "cuda")):
        with pytest.raises(MoeError) as e:
            f()
        assert e.value.code == INV, n
    ws = torch.zeros(8, dtype=torch.uint8, device="cuda")
    f, tensors = calls[0]
    with pytest.raises(MoeError) as e:
        f(*tensors[:4], ws)
    assert e.value.code == SMALL
    monkeypatch.setattr(O, "_current_device", lambda: 1)
    for f, tensors in calls:
        with pytest.raises(MoeError) as e:
            f(*tensors)
        assert e.value.code == INV
