"""The operators of include/moe_ops.h without a GPU: exported symbols, sizes
and refusals (argument errors return before any CUDA call)."""
import ctypes
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INV, SMALL, OK = 1, 3, 0
P = 1 << 20  # a 128-byte aligned address that is never read


@pytest.fixture(scope="module")
def O():
    from mixture_experts_layer_stable_gb300 import build, ops
    build.build()
    ops.lib()
    return ops


def test_exports_every_declared_symbol(O):
    txt = open(os.path.join(ROOT, "include", "moe_ops.h")).read()
    txt = re.sub(r"/\*.*?\*/", "", txt, flags=re.S)
    names = sorted(set(re.findall(r"\b(moe_[a-z0-9_]+)\s*\(", txt)))
    assert names == sorted(O.EXPORTED)
    for n in names:
        assert hasattr(O.lib(), n), n


def test_sizes(O):
    assert O.moe_layernorm_workspace_bytes(100, 64) >= 2 * 64 * 4
    assert O.moe_layernorm_workspace_bytes(-1, 64) == 0 and O.moe_layernorm_workspace_bytes(1, 65537) == 0
    assert O.moe_sort_workspace_bytes(0, 1) > 0 and O.moe_sort_workspace_bytes(5, 1025) == 0
    assert O.moe_mxfp4_weight_scale_bytes(3, 160, 130) == 3 * 2 * 2 * 512
    assert O.moe_mxfp4_weight_scale_bytes(3, 48, 130) == 0
    # every expert's blocks fit, whatever the split of the rows
    for counts in ([0, 0, 1], [128, 128], [127, 1, 129], [1] * 9, [1000], [0] * 5 + [257]):
        off = [sum(counts[:i]) for i in range(len(counts) + 1)]
        t = 128
        end, last = 0, -1
        for g, c in enumerate(counts):
            first = off[g] // t + g
            assert first > last or c == 0 or last == -1
            if c:
                assert first >= end
                end = first + -(-c // t)
            last = first
        assert O.moe_mxfp4_row_scale_bytes(off[-1], 128, len(counts)) >= end * 512
    assert O.moe_mxfp4_row_scale_bytes(10, 33, 1) == 0 and O.moe_mxfp4_row_scale_bytes(10, 32, 0) == 0


def test_layernorm_refusals(O):
    L = O.lib()

    def fwd(dt=1, wt=1, n=4, d=8, x=P, ldx=8, w=P, b=P, eps=1e-5, y=P, ldy=8, m=P, r=P):
        return L.moe_layernorm_forward(dt, wt, n, d, x, ldx, w, b, eps, y, ldy, m, r, None)

    for bad in (dict(dt=3), dict(dt=-1), dict(dt=1, wt=2), dict(dt=0, wt=1), dict(n=-1), dict(d=0), dict(d=65537),
                dict(x=None), dict(y=None), dict(ldx=7), dict(ldy=7), dict(x=P + 1), dict(w=P + 1), dict(eps=-1.0),
                dict(eps=float("nan")), dict(eps=float("inf")), dict(m=None), dict(r=None), dict(r=P + 2)):
        assert fwd(**bad) == INV, bad
    assert fwd(n=0, x=None, y=None) == OK

    def bwd(dt=1, wt=1, n=4, d=8, dy=P, lddy=8, x=P, ldx=8, w=P, m=P, r=P, a=None, lda=0, dx=P, lddx=8, dw=P, db=P,
            ws=P, wsb=1 << 20):
        return L.moe_layernorm_backward(dt, wt, n, d, dy, lddy, x, ldx, w, m, r, a, lda, dx, lddx, dw, db, ws, wsb, None)

    for bad in (dict(dt=9), dict(wt=2), dict(n=-1), dict(d=0), dict(dy=None), dict(x=None), dict(dx=None), dict(m=None),
                dict(r=None), dict(lddy=7), dict(ldx=7), dict(lddx=7), dict(a=P, lda=7), dict(dw=P + 1), dict(ws=None),
                dict(ws=P + 64)):
        assert bwd(**bad) == INV, bad
    assert bwd(wsb=16) == SMALL
    assert bwd(n=0, dw=None, db=None, dy=None, x=None, dx=None, ws=None) == OK


def test_sort_and_permute_refusals(O):
    L = O.lib()

    def sort(ids=P, R=16, E=4, c=P, o=P, p=P, i=P, ws=P, n=1 << 20):
        return L.moe_sort_rows(ids, R, E, c, o, p, i, ws, n, None)

    for bad in (dict(R=-1), dict(R=(1 << 28) + 1), dict(E=0), dict(E=1025), dict(ids=None), dict(c=None), dict(o=None),
                dict(p=None), dict(i=None), dict(ws=None), dict(ws=P + 4), dict(ids=P + 2)):
        assert sort(**bad) == INV, bad
    assert sort(n=8) == SMALL

    def perm(dt=1, T=4, d=8, k=2, E=4, x=P, ldx=8, inv=P, off=P, xp=P):
        return L.moe_permute(dt, T, d, k, E, x, ldx, inv, off, xp, None)

    for bad in (dict(dt=3), dict(T=-1), dict(d=0), dict(k=0), dict(k=33), dict(E=0), dict(E=1025), dict(ldx=7),
                dict(x=None), dict(inv=None), dict(off=None), dict(xp=None), dict(x=P + 1), dict(T=1 << 28)):
        assert perm(**bad) == INV, bad
    assert perm(T=0, x=None, xp=None) == OK

    def unp(dt=1, T=4, d=8, k=2, E=4, y=P, w=P, inv=P, off=P, b=None, ldb=0, out=P, ldo=8):
        return L.moe_unpermute(dt, T, d, k, E, y, w, inv, off, b, ldb, out, ldo, None)

    for bad in (dict(dt=3), dict(y=None), dict(out=None), dict(ldo=7), dict(b=P, ldb=7), dict(w=P + 2), dict(k=0)):
        assert unp(**bad) == INV, bad

    def bwd(dt=1, T=4, d=8, k=2, E=4, g=P, ldg=8, y=P, w=P, inv=P, off=P, dy=P, dw=P):
        return L.moe_unpermute_backward(dt, T, d, k, E, g, ldg, y, w, inv, off, dy, dw, None)

    for bad in (dict(g=None), dict(ldg=7), dict(y=None), dict(dy=None), dict(dw=P + 1), dict(dt=-1)):
        assert bwd(**bad) == INV, bad


def test_mxfp4_refusals(O):
    L = O.lib()

    def qw(dt=1, w=P, b=2, K=64, N=8, p=0, q=P, s=P):
        return L.moe_quantize_mxfp4(dt, w, b, K, N, p, q, s, None)

    for bad in (dict(dt=3), dict(w=None), dict(b=-1), dict(K=0), dict(K=48), dict(N=0), dict(p=1, N=7), dict(q=P + 64),
                dict(s=None)):
        assert qw(**bad) == INV, bad
        b = dict(bad)
        assert L.moe_dequantize_mxfp4(b.get("dt", 1), b.get("q", P), b.get("s", P), b.get("b", 2), b.get("K", 64),
                                      b.get("N", 8), b.get("p", 0), b.get("w", P), None) == INV

    def qr(dt=1, n=4, K=64, x=P, ldx=64, G=2, off=P, perm=None, k=1, q=P, s=P):
        return L.moe_quantize_mxfp4_rows(dt, n, K, x, ldx, G, off, perm, k, q, s, None)

    for bad in (dict(dt=3), dict(n=-1), dict(K=40), dict(ldx=63), dict(G=0), dict(G=1025), dict(off=None), dict(k=0),
                dict(x=None), dict(q=None), dict(s=P + 8), dict(perm=P + 1)):
        assert qr(**bad) == INV, bad
    assert qr(n=0, x=None, q=None, s=None) == OK

    def prod(dt=1, n=4, N=8, K=64, G=2, off=P, x=P, xs=P, w=P, ws_=P, act=0, out=P, ldo=8, ws=P, wsb=1 << 30):
        return L.moe_mxfp4_product(dt, n, N, K, G, off, x, xs, w, ws_, act, out, ldo, ws, wsb, None)

    for bad in (dict(dt=3), dict(n=-1), dict(N=0), dict(K=16), dict(G=0), dict(off=None), dict(x=None), dict(xs=P + 16),
                dict(w=None), dict(ws_=None), dict(act=2), dict(act=1, N=7), dict(out=None), dict(ldo=7),
                dict(act=1, ldo=3), dict(ws=None)):
        assert prod(**bad) == INV, bad
    assert prod(wsb=0) == SMALL
    assert prod(n=0, x=None, out=None) == OK


def test_binding_refuses_tensors_that_do_not_fit(O):
    from mixture_experts_layer_stable_gb300.binding import MoeError
    x = torch.zeros(4, 8)
    with pytest.raises(MoeError):
        O.moe_layernorm_forward(x, None, None, 1e-5, torch.zeros(4, 7), stream=0)
    with pytest.raises(MoeError):
        O.moe_layernorm_forward(x.t(), None, None, 1e-5, torch.zeros(8, 4), stream=0)
    with pytest.raises(MoeError):
        O.moe_layernorm_forward(x.double(), None, None, 1e-5, x.double(), stream=0)
    with pytest.raises(MoeError):
        O.moe_permute(x, 2, torch.zeros(7, dtype=torch.int32), torch.zeros(3, dtype=torch.int32), torch.zeros(8, 8), stream=0)
    with pytest.raises(MoeError):
        O.moe_sort_rows(torch.zeros(4), *(torch.zeros(n, dtype=torch.int32) for n in (2, 3, 4, 4)),
                        torch.zeros(4096, dtype=torch.uint8), stream=0)
    u8 = torch.zeros(4096, dtype=torch.uint8)
    with pytest.raises(MoeError):
        O.moe_mxfp4_product(u8, u8, None, torch.zeros(2, 4, 32, dtype=torch.uint8), u8, 0, torch.zeros(4, 4), u8, stream=0)


def _calls(O, device):
    """(function, its tensors) of a small valid call of every operator."""
    def t(*shape, dtype=torch.float32):
        return torch.zeros(*shape, dtype=dtype, device=device)

    def i32(*shape):
        return t(*shape, dtype=torch.int32)

    def u8(n):
        return t(n, dtype=torch.uint8)

    x, v, w, ws = t(4, 32), t(4), t(32), u8(1 << 16)
    inv, off, q, sc = i32(8), i32(3), u8(8 * 16), u8(O.moe_mxfp4_row_scale_bytes(8, 32, 2))
    wq, wsc = t(2, 6, 16, dtype=torch.uint8), u8(O.moe_mxfp4_weight_scale_bytes(2, 32, 6))
    return [
        (lambda *a: O.moe_layernorm_forward(*a[:3], 1e-5, *a[3:], stream=0), [x, w, w.clone(), t(4, 32), v, v.clone()]),
        (lambda *a: O.moe_layernorm_backward(*a[:9], dadd=a[9], stream=0),
         [x, x.clone(), w, v, v.clone(), t(4, 32), t(32), t(32), ws, x.clone()]),
        (lambda *a: O.moe_sort_rows(*a, stream=0), [i32(8), i32(2), off, i32(8), inv, ws]),
        (lambda *a: O.moe_permute(a[0], 2, *a[1:], stream=0), [x, inv, off, t(8, 32)]),
        (lambda *a: O.moe_unpermute(a[0], a[1], 2, *a[2:5], base=a[5], stream=0), [t(8, 32), t(8), inv, off, t(4, 32), x]),
        (lambda *a: O.moe_unpermute_backward(*a[:3], 2, *a[3:], stream=0), [x, t(8, 32), t(8), inv, off, t(8, 32), t(8)]),
        (lambda *a: O.moe_quantize_mxfp4(*a, stream=0), [t(2, 32, 6), wq, wsc]),
        (lambda *a: O.moe_dequantize_mxfp4(*a, stream=0), [wq, wsc, t(2, 32, 6)]),
        (lambda *a: O.moe_quantize_mxfp4_rows(*a, k=2, stream=0), [x, q, sc, off, i32(8)]),
        (lambda *a: O.moe_dequantize_mxfp4_rows(a[0], a[1], a[2], a[3], stream=0), [q, sc, t(8, 32), off]),
        (lambda *a: O.moe_mxfp4_product(*a[:5], 0, *a[5:], stream=0), [q, sc, off, wq, wsc, t(8, 6), ws]),
    ]


def test_binding_refuses_host_tensors(O):
    """Refused as arguments, before the library sees their addresses."""
    from mixture_experts_layer_stable_gb300.binding import MoeError
    for f, tensors in _calls(O, "cpu"):
        with pytest.raises(MoeError) as e:
            f(*tensors)
        assert e.value.code == INV


@pytest.mark.gpu
def test_binding_refuses_tensors_off_the_current_gpu(O, cuda_lib, monkeypatch):
    from mixture_experts_layer_stable_gb300.binding import MoeError
    calls = _calls(O, "cuda")
    torch.cuda.synchronize()
    for n, (f, tensors) in enumerate(calls):
        f(*tensors)                               # all on the GPU: accepted
        for i in range(len(tensors)):
            mixed = list(tensors)
            mixed[i] = tensors[i].cpu()
            with pytest.raises(MoeError) as e:
                f(*mixed)
            assert e.value.code == INV, (n, i)
    torch.cuda.synchronize()
    # a workspace with gaps
    strided = torch.zeros(1 << 12, 32, dtype=torch.uint8, device="cuda")[:, :16]
    for n in (1, 2, 10):
        f, tensors = calls[n]
        at = next(i for i, t in enumerate(tensors) if t.numel() == 1 << 16)
        with pytest.raises(MoeError) as e:
            f(*[strided if i == at else t for i, t in enumerate(tensors)])
        assert e.value.code == INV, n
    # tensors on the GPU that do not fit together
    x, u8 = torch.zeros(4, 8, device="cuda"), torch.zeros(4096, dtype=torch.uint8, device="cuda")

    def i32(n):
        return torch.zeros(n, dtype=torch.int32, device="cuda")

    for f in (lambda: O.moe_layernorm_forward(x, None, None, 1e-5, torch.zeros(4, 7, device="cuda")),
              lambda: O.moe_layernorm_forward(x.t(), None, None, 1e-5, torch.zeros(8, 4, device="cuda")),
              lambda: O.moe_layernorm_forward(x.double(), None, None, 1e-5, x.double()),
              lambda: O.moe_permute(x, 2, i32(7), i32(3), torch.zeros(8, 8, device="cuda")),
              lambda: O.moe_sort_rows(torch.zeros(4, device="cuda"), i32(2), i32(3), i32(4), i32(4), u8),
              lambda: O.moe_sort_rows(i32(4), i32(2), i32(3), i32(4), i32(3), u8),
              lambda: O.moe_unpermute(torch.zeros(8, 8, device="cuda"), None, 2, i32(8), i32(3), x, base=x[:, :7]),
              lambda: O.moe_mxfp4_product(u8, u8, None, torch.zeros(2, 4, 32, dtype=torch.uint8, device="cuda"), u8, 0,
                                          torch.zeros(4, 4, device="cuda"), u8)):
        with pytest.raises(MoeError) as e:
            f()
        assert e.value.code == INV
    # another device is current
    monkeypatch.setattr(O, "_current_device", lambda: 1)
    for f, tensors in calls:
        with pytest.raises(MoeError) as e:
            f(*tensors)
        assert e.value.code == INV
