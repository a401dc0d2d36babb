"""Rows sorted by expert and back on the GPU: the order exactly, sums against
64 bits.  Bounds: an output is rounded once (u |want|) after at most k + 1 fp32
fused multiply-adds (each 2^-24 of the sum of magnitudes); the scalar products
over d terms are held to (16 + d / 256 + log2 d) 2^-24 of theirs (chains of at
most d / 256 or so terms, then trees)."""
import math

import numpy as np
import pytest
import torch

from mixture_experts_layer_stable_gb300 import binding as B
from mixture_experts_layer_stable_gb300 import ops

from ops_util import DT, close, empty_strided, gen, randn, strided

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_lib):
    yield


def sort(ids, E, stream=None):
    R = ids.numel()
    i32 = dict(dtype=torch.int32, device="cuda")
    s = dict(counts=torch.full((E,), -7, **i32), offsets=torch.full((E + 1,), -7, **i32), perm=torch.full((R,), -7, **i32),
             inv=torch.full((R,), -7, **i32))
    ws = torch.full((ops.moe_sort_workspace_bytes(R, E),), 255, dtype=torch.uint8, device="cuda")
    if stream is not None:
        torch.cuda.synchronize()  # the fills above run on the current stream
    ops.moe_sort_rows(ids, s["counts"], s["offsets"], s["perm"], s["inv"], ws, stream=stream)
    return s


def order(ids, E):
    key = np.where((ids >= 0) & (ids < E), ids, E)
    perm = np.argsort(key, kind="stable")
    inv = np.empty_like(perm)
    inv[perm] = np.arange(len(ids))
    counts = np.bincount(key, minlength=E + 1)[:E]
    return perm, inv, counts, np.concatenate([[0], np.cumsum(counts)])


def make_ids(g, R, E, drop, how="even"):
    if how == "one":
        ids = torch.full((R,), E - 1, dtype=torch.int32, device="cuda")
    elif how == "zipf":
        ids = (E * torch.rand(R, generator=g, device="cuda") ** 4).to(torch.int32).clamp(max=E - 1)
    else:
        ids = torch.randint(0, E, (R,), generator=g, device="cuda", dtype=torch.int32)
    if drop:
        odd = torch.tensor([-1, E, E + 5, -2 ** 31, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
        m = torch.rand(R, generator=g, device="cuda") < drop
        ids = torch.where(m, odd[torch.randint(0, 5, (R,), generator=g, device="cuda")], ids)
    return ids.contiguous()


@pytest.mark.parametrize("R,E", [(0, 3), (1, 1), (1, 1024), (8, 256), (31, 5), (32, 2), (33, 1), (257, 17), (1023, 64),
                                 (1024, 64), (1025, 64), (4095, 1024), (4097, 3), (8192, 255), (8193, 256), (20000, 37),
                                 (32768, 256), (100003, 1000), (1 << 20, 8), (3000001, 256)])
@pytest.mark.parametrize("drop", [0.0, 0.3, 1.0])
def test_order(R, E, drop):
    how = ("even", "zipf", "one")[(R + E) % 3]
    ids = make_ids(gen(R + E), R, E, drop, how)
    s = sort(ids, E)
    perm, inv, counts, off = order(ids.cpu().numpy().astype(np.int64), E)
    assert np.array_equal(s["counts"].cpu().numpy(), counts)
    assert np.array_equal(s["offsets"].cpu().numpy(), off)
    assert np.array_equal(s["perm"].cpu().numpy(), perm)
    assert np.array_equal(s["inv"].cpu().numpy(), inv)


def test_order_is_the_schedule_s():
    cfg = B.make_config(300, 128, 64, 40, 5)
    logits = randn(gen(1), 300, 40)
    sched, ws = B.alloc_sched(cfg), B.alloc_workspace(cfg)
    B.moe_schedule(cfg, logits, sched, ws)
    s = sort(sched["topk_ids"], 40)
    for k in ("counts", "offsets", "perm", "inv"):
        assert torch.equal(s[k], sched[k]), k


CASES = [(1, 1, 1, 1, 0.0), (1, 256, 8, 7168, 0.0), (5, 4, 4, 3, 0.5), (7, 9, 3, 33, 0.2), (64, 8, 2, 128, 0.0),
         (100, 37, 5, 333, 0.3), (33, 64, 32, 257, 0.1), (1000, 16, 6, 1024, 0.0), (777, 20, 8, 2049, 0.2),
         (6, 5, 2, 20001, 0.2), (300, 12, 1, 512, 0.0), (50, 3, 3, 64, 1.0), (2049, 256, 8, 4096, 0.0)]


def dots_bound(d):
    return (16 + d / 256 + math.log2(d)) * 2.0 ** -24


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,E,k,d,drop", CASES)
def test_permute_unpermute_and_gradients(T, E, k, d, drop, dt):
    g = gen(T + d)
    R, t = T * k, DT[dt]
    pad = (0, 8, 3)[T % 3]
    ids = make_ids(g, R, E, drop)
    s = sort(ids, E)
    kept, inv = int(s["offsets"][E]), s["inv"].long()
    live = inv < kept
    x = strided(g, T, d, t, pad)
    xp = torch.full((R, d), 9.0, dtype=t, device="cuda")
    ops.moe_permute(x, k, s["inv"], s["offsets"], xp)
    want = torch.zeros(R, d, dtype=t, device="cuda")
    tok = torch.arange(R, device="cuda") // k
    want[inv[live]] = x[tok[live]]
    assert torch.equal(xp, want)

    y, w = randn(g, R, d, dtype=t), randn(g, T, k)
    y[kept:] = float("nan")                       # rows of dropped slots are not read
    base = strided(g, T, d, t, pad)
    yt = torch.zeros(R, d, dtype=torch.float64, device="cuda")
    yt[live] = y[inv[live]].double()
    for ww in (w, None):
        wd = torch.ones(R, 1, dtype=torch.float64, device="cuda") if ww is None else w.reshape(R, 1).double()
        for bb in (None, base):
            out = empty_strided(T, d, t, pad, fill=9.0)
            ops.moe_unpermute(y, ww, k, s["inv"], s["offsets"], out, base=bb)
            prod = (wd * yt).reshape(T, k, d)
            b64 = 0.0 if bb is None else bb.double()
            mag = prod.abs().sum(1) + (0 if bb is None else b64.abs())
            close(out, prod.sum(1) + b64, dt, (k + 1) * 2.0 ** -24 * mag, "out")
            if bb is not None:
                same = base.clone(memory_format=torch.preserve_format)
                ops.moe_unpermute(y, ww, k, s["inv"], s["offsets"], same, base=same)
                assert torch.equal(same, out)
        dout = strided(g, T, d, t, pad)
        dy, dw = torch.full((R, d), 9.0, dtype=t, device="cuda"), torch.full((R,), 9.0, device="cuda")
        ops.moe_unpermute_backward(dout, y, ww, k, s["inv"], s["offsets"], dy, dw)
        gt = dout.double()[tok]
        wy = torch.zeros(R, d, dtype=torch.float64, device="cuda")
        wy[inv[live]] = (wd * gt)[live]
        close(dy, wy, dt, 2.0 ** -24 * wy.abs(), "dy")
        close(dw, (gt * yt).sum(1), "f32", dots_bound(d) * (gt * yt).abs().sum(1), "dw")
        dy2 = torch.empty_like(dy)
        ops.moe_unpermute_backward(dout, None, ww, k, s["inv"], s["offsets"], dy2, None)
        assert torch.equal(dy, dy2)


@pytest.mark.parametrize("shift", [1, 2, 4])
def test_misaligned_rows(shift):
    g = gen(3)
    T, E, k, d = 20, 6, 3, 200
    s = sort(make_ids(g, T * k, E, 0.2), E)
    x = strided(g, T, d, torch.bfloat16, 1, shift)
    xp = empty_strided(T * k, d, torch.bfloat16, 0, shift)
    ops.moe_permute(x, k, s["inv"], s["offsets"], xp)
    ref = torch.empty(T * k, d, dtype=torch.bfloat16, device="cuda")
    ops.moe_permute(x.contiguous(), k, s["inv"], s["offsets"], ref)
    assert torch.equal(xp, ref)
    w = randn(g, T, k)
    o1, o2 = empty_strided(T, d, torch.bfloat16, 3, shift), torch.empty(T, d, dtype=torch.bfloat16, device="cuda")
    ops.moe_unpermute(xp, w, k, s["inv"], s["offsets"], o1, base=x)
    ops.moe_unpermute(ref, w, k, s["inv"], s["offsets"], o2, base=x.contiguous())
    assert torch.equal(o1, o2)
    dy1, dy2 = empty_strided(T * k, d, torch.bfloat16, 0, shift), torch.empty_like(ref)
    dw1, dw2 = torch.empty(T * k, device="cuda"), torch.empty(T * k, device="cuda")
    ops.moe_unpermute_backward(x, xp, w, k, s["inv"], s["offsets"], dy1, dw1)
    ops.moe_unpermute_backward(x.contiguous(), ref, w, k, s["inv"], s["offsets"], dy2, dw2)
    assert torch.equal(dy1, dy2)
    mag = (xp.double().norm(dim=1).max() * x.double().norm(dim=1).max()).item()
    assert (dw1 - dw2).abs().max() <= 2 * dots_bound(d) * mag


def test_non_finite_rows_and_no_tokens():
    g = gen(4)
    T, E, k, d = 30, 4, 2, 96
    s = sort(make_ids(g, T * k, E, 0.0), E)
    y = randn(g, T * k, d)
    y[3] = float("inf")
    out = torch.empty(T, d, device="cuda")
    ops.moe_unpermute(y, None, k, s["inv"], s["offsets"], out)
    hit = int(s["perm"][3]) // k
    bad = ~out.isfinite().all(1)
    assert bad.nonzero().flatten().tolist() == [hit]
    e = torch.empty(0, d, device="cuda")
    z = sort(torch.empty(0, dtype=torch.int32, device="cuda"), E)
    assert not z["counts"].any() and not z["offsets"].any()
    ops.moe_permute(e, k, z["inv"], z["offsets"], e)
    ops.moe_unpermute(e, None, k, z["inv"], z["offsets"], e)
    ops.moe_unpermute_backward(e, e, None, k, z["inv"], z["offsets"], e, torch.empty(0, device="cuda"))


def test_offsets_past_32_bits():
    """More than 2^32 elements of expert-ordered rows: the last rows land where they belong."""
    T, E, k, d = 40000, 16, 16, 7168               # 4.6e9 elements, 9.2 GB
    g = gen(5)
    s = sort(make_ids(g, T * k, E, 0.0), E)
    x = randn(g, T, d, dtype=torch.bfloat16)
    xp = torch.empty(T * k, d, dtype=torch.bfloat16, device="cuda")
    ops.moe_permute(x, k, s["inv"], s["offsets"], xp)
    at = torch.cat((torch.arange(0, T * k, 9973, device="cuda"), torch.arange(T * k - 50, T * k, device="cuda")))
    assert torch.equal(xp[at], x[s["perm"][at].long() // k])
    out = torch.empty_like(x)
    ops.moe_unpermute(xp, None, k, s["inv"], s["offsets"], out)
    assert torch.equal(out, (x.float() * k).to(torch.bfloat16))


def test_same_bits_and_other_stream():
    g = gen(6)
    T, E, k, d = 3000, 64, 8, 1024
    ids = make_ids(g, T * k, E, 0.1)
    x, y, w = randn(g, T, d, dtype=torch.bfloat16), randn(g, T * k, d, dtype=torch.bfloat16), randn(g, T, k)

    def go(stream=None):
        s = sort(ids, E, stream)
        out, dy, dw = torch.empty_like(x), torch.empty_like(y), torch.empty(T * k, device="cuda")
        ops.moe_unpermute(y, w, k, s["inv"], s["offsets"], out, stream=stream)
        ops.moe_unpermute_backward(x, y, w, k, s["inv"], s["offsets"], dy, dw, stream=stream)
        return s["perm"], out, dy, dw

    a = go()
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    b = go(st)
    st.synchronize()
    for p, q in zip(a, b):
        assert torch.equal(p, q)


def test_gradients_against_differences():
    """out is linear in y, w and base: differences with a step of 1 in fp32 are off only by the
    rounding of out and of the sums (2^-20 of the magnitudes summed)."""
    g = gen(7)
    T, E, k, d = 20, 5, 3, 40
    s = sort(make_ids(g, T * k, E, 0.2), E)
    y, w, dout = randn(g, T * k, d), randn(g, T, k), randn(g, T, d)
    vy, vw = randn(g, T * k, d), randn(g, T, k)

    def L(y, w):
        out = torch.empty(T, d, device="cuda")
        ops.moe_unpermute(y, w, k, s["inv"], s["offsets"], out)
        return (out.double() * dout.double()).sum()

    dy, dw = torch.empty_like(y), torch.empty(T * k, device="cuda")
    ops.moe_unpermute_backward(dout, y, w, k, s["inv"], s["offsets"], dy, dw)
    scale = dout.double().norm() * (y.double().norm() + vy.double().norm()) * (w.double().abs().max() + vw.double().abs().max())
    assert abs(L(y + vy, w) - L(y, w) - (dy.double() * vy.double()).sum()) <= 2.0 ** -20 * scale
    assert abs(L(y, w + vw) - L(y, w) - (dw.double() * vw.double().reshape(-1)).sum()) <= 2.0 ** -20 * scale
    # the backward of permute is unpermute without weights: <xp(x), g> = <x, dx(g)>
    x, gx = randn(g, T, d), randn(g, T * k, d)
    xp, dx = torch.empty(T * k, d, device="cuda"), torch.empty(T, d, device="cuda")
    ops.moe_permute(x, k, s["inv"], s["offsets"], xp)
    ops.moe_unpermute(gx, None, k, s["inv"], s["offsets"], dx)
    lhs, rhs = (xp.double() * gx.double()).sum(), (x.double() * dx.double()).sum()
    assert abs(lhs - rhs) <= 2.0 ** -20 * x.double().norm() * gx.double().norm() * k
