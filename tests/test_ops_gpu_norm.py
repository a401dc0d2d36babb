"""Layer norm on the GPU against the formulas in 64 bits.

Bounds: outputs are rounded once to their type (u |want|); before that, fp32
arithmetic.  Sums of d terms are taken in some order with at most d roundings a
path, in fact in short chains joined as a tree: their error is held to
c = 32 + log2(d) units of 2^-24 of the sum of magnitudes.  The mean's error is
so c 2^-24 mean|x|, which moves xh by that times rstd; rstd itself is off by the
relative error of the variance, 2c 2^-24, plus the mean's error squared."""
import math

import pytest
import torch

from mixture_experts_layer_stable_gb300 import ops

from ops_util import DT, U, close, empty_strided, gen, randn, strided

pytestmark = pytest.mark.gpu
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_lib):
    yield


def plain(x, w, b, dy=None, dadd=None, eps=EPS):
    x, d = x.double(), x.shape[1]
    w = torch.ones(d, dtype=torch.float64, device="cuda") if w is None else w.double()
    b = torch.zeros(d, dtype=torch.float64, device="cuda") if b is None else b.double()
    mean = x.mean(1, keepdim=True)
    xc = x - mean
    rstd = 1 / torch.sqrt((xc * xc).mean(1, keepdim=True) + eps)
    xh = xc * rstd
    e = (32 + math.log2(d)) * 2.0 ** -24
    exh = e * (x.abs().mean(1, keepdim=True) + x.abs()) * rstd + 2 * e * xh.abs()   # error of xh
    out = dict(y=xh * w + b, ey=exh * w.abs() + 4 * 2.0 ** -24 * ((xh * w).abs() + b.abs()),
               mean=mean[:, 0], rstd=rstd[:, 0], emean=e * x.abs().mean(1),
               erstd=rstd[:, 0] * 3 * e * (1 + x.abs().mean(1) * rstd[:, 0]))
    if dy is not None:
        dy = dy.double()
        g = dy * w
        m1, m2 = g.mean(1, keepdim=True), (g * xh).mean(1, keepdim=True)
        dx = rstd * (g - m1 - xh * m2)
        a1, a2 = g.abs().mean(1, keepdim=True), (g * xh).abs().mean(1, keepdim=True)
        es = e * (g.abs() + a1 + xh.abs() * a2 * 2) + exh * a2 + xh.abs() * (g.abs() * exh).mean(1, keepdim=True)
        relr = 3 * e * (1 + x.abs().mean(1, keepdim=True) * rstd)
        out.update(dx=dx if dadd is None else dx + dadd.double(),
                   edx=rstd * es + relr * dx.abs() + (0 if dadd is None else 2.0 ** -23 * (dx.abs() + dadd.double().abs())),
                   dw=(dy * xh).sum(0), edw=(dy.abs() * (exh + (e + x.shape[0] * 2.0 ** -24) * xh.abs())).sum(0),
                   db=dy.sum(0), edb=(e + x.shape[0] * 2.0 ** -24) * dy.abs().sum(0))
    return out


def run(x, w, b, dy, dadd=None, ypad=0, stream=None, eps=EPS):
    n, d = x.shape
    wdt = x.dtype if w is None and b is None else (w if w is not None else b).dtype
    y, dx = empty_strided(n, d, x.dtype, ypad), empty_strided(n, d, x.dtype, ypad)
    mean, rstd = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    dw, db = torch.empty(d, dtype=wdt, device="cuda"), torch.empty(d, dtype=wdt, device="cuda")
    ws = torch.empty(ops.moe_layernorm_workspace_bytes(n, d), dtype=torch.uint8, device="cuda")
    ops.moe_layernorm_forward(x, w, b, eps, y, mean, rstd, stream=stream)
    ops.moe_layernorm_backward(dy, x, w, mean, rstd, dx, dw, db, ws, dadd=dadd, stream=stream)
    return dict(y=y, mean=mean, rstd=rstd, dx=dx, dw=dw, db=db)


SHAPES = [(1, 1), (2, 2), (3, 7), (1, 33), (5, 64), (1, 7168), (17, 100), (300, 257), (129, 1000), (1003, 1999),
          (64, 2048), (700, 4096), (31, 7168), (33, 8192), (3, 12289), (2, 16385), (3, 65536), (2500, 96)]


@pytest.mark.parametrize("dt,wdt", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32")])
@pytest.mark.parametrize("n,d", SHAPES)
def test_forward_and_backward(n, d, dt, wdt):
    g = gen(n * 7 + d)
    pad = (0, 3, 8)[(n + d) % 3]
    x, dy = strided(g, n, d, DT[dt], pad, std=1.5, mean=0.4), strided(g, n, d, DT[dt], pad)
    w, b = randn(g, d, dtype=DT[wdt], std=0.3, mean=1.0), randn(g, d, dtype=DT[wdt], std=0.3)
    got, want = run(x, w, b, dy, ypad=pad), plain(x, w, b, dy)
    close(got["mean"], want["mean"], "f32", want["emean"], "mean")
    close(got["rstd"], want["rstd"], "f32", want["erstd"], "rstd")
    close(got["y"], want["y"], dt, want["ey"], "y")
    close(got["dx"], want["dx"], dt, want["edx"], "dx")
    close(got["dw"], want["dw"], wdt, want["edw"], "dw")
    close(got["db"], want["db"], wdt, want["edb"], "db")


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("shift", [0, 1, 2, 4])
@pytest.mark.parametrize("d", [96, 101, 2048])
def test_misaligned_rows(d, shift, dt):
    g = gen(5)
    x, dy = strided(g, 37, d, DT[dt], 0, shift), strided(g, 37, d, DT[dt], 1, shift)
    w, b = randn(g, d + 1, dtype=DT[dt])[1:], randn(g, d + 1, dtype=DT[dt])[1:]
    got, want = run(x, w, b, dy, ypad=3), plain(x, w, b, dy)
    for k in ("y", "dx", "dw", "db"):
        close(got[k], want[k], dt, want["e" + k], k)


@pytest.mark.parametrize("d", [77, 1024])
def test_optional_arguments(d):
    g = gen(6)
    n = 50
    x, dy, dadd = (strided(g, n, d, torch.bfloat16, 8) for _ in range(3))
    w = randn(g, d, dtype=torch.bfloat16)
    for ww, bb in ((None, None), (w, None), (None, w)):
        got, want = run(x, ww, bb, dy, dadd=dadd), plain(x, ww, bb, dy, dadd)
        for k in ("y", "dx", "dw", "db"):
            close(got[k], want[k], "bf16", want["e" + k], k)
    # no statistics, no weight gradients, in place
    want = plain(x, w, None, dy, dadd)
    y = x.clone()
    ops.moe_layernorm_forward(y, w, None, EPS, y)
    close(y, want["y"], "bf16", want["ey"], "y in place")
    full = run(x, w, None, dy, dadd=dadd)
    for into in ("dy", "dadd"):
        a, c = dy.clone(), dadd.clone()
        t = a if into == "dy" else c
        ops.moe_layernorm_backward(a, x, w, full["mean"], full["rstd"], t, None, None, None, dadd=c)
        assert torch.equal(t, full["dx"])
    only = torch.empty(d, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(ops.moe_layernorm_workspace_bytes(n, d), dtype=torch.uint8, device="cuda")
    dx = torch.empty(n, d, dtype=torch.bfloat16, device="cuda")
    ops.moe_layernorm_backward(dy, x, w, full["mean"], full["rstd"], dx, only, None, ws)
    assert torch.equal(only, full["dw"])
    ops.moe_layernorm_backward(dy, x, w, full["mean"], full["rstd"], dx, None, only, ws)
    assert torch.equal(only, full["db"])


def test_in_place_dy_with_weight_gradients():
    """dx may be dy: the sums over the rows still see dy."""
    g = gen(8)
    x, dy = randn(g, 700, 512), randn(g, 700, 512)
    w = randn(g, 512)
    full = run(x, w, None, dy)
    dw, db = torch.empty_like(w), torch.empty_like(w)
    ws = torch.empty(ops.moe_layernorm_workspace_bytes(700, 512), dtype=torch.uint8, device="cuda")
    ops.moe_layernorm_backward(dy, x, w, full["mean"], full["rstd"], dy, dw, db, ws)
    assert torch.equal(dy, full["dx"]) and torch.equal(dw, full["dw"]) and torch.equal(db, full["db"])


def test_no_rows_and_constant_rows():
    x = torch.empty(0, 64, device="cuda")
    dw, db = torch.full((64,), 7.0, device="cuda"), torch.full((64,), 7.0, device="cuda")
    e = torch.empty(0, device="cuda")
    ws = torch.empty(ops.moe_layernorm_workspace_bytes(0, 64), dtype=torch.uint8, device="cuda")
    ops.moe_layernorm_forward(x, None, None, EPS, x, e, e)
    ops.moe_layernorm_backward(x, x, None, e, e, x, dw, db, ws)
    assert not dw.any() and not db.any()
    # a row of one value: variance 0, y = b exactly, whatever the value
    b = torch.arange(100, device="cuda", dtype=torch.float32)
    for v in (0.0, 3.0, 1024.0):
        y = torch.empty(2, 100, device="cuda")
        ops.moe_layernorm_forward(torch.full((2, 100), v, device="cuda"), None, b, EPS, y)
        assert torch.equal(y, b.expand(2, 100))


def test_large_mean_keeps_the_variance():
    """std 1 around 1000: a variance from the mean of squares would lose it."""
    g = gen(9)
    x = randn(g, 40, 4096, mean=1000.0)
    dy = randn(g, 40, 4096)
    got, want = run(x, None, None, dy), plain(x, None, None, dy)
    for k in ("y", "dx"):
        close(got[k], want[k], "f32", want["e" + k], k)
    assert (got["y"].double() - want["y"]).abs().max() < 0.01


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_non_finite_rows_stay_in_their_row(bad):
    g = gen(10)
    x, dy = randn(g, 12, 512, dtype=torch.bfloat16), randn(g, 12, 512, dtype=torch.bfloat16)
    clean = run(x, None, None, dy)
    x[5, 77] = bad
    got = run(x, None, None, dy)
    rest = [i for i in range(12) if i != 5]
    assert torch.equal(got["y"][rest], clean["y"][rest]) and torch.equal(got["dx"][rest], clean["dx"][rest])
    assert got["y"][5].isnan().all() and got["dx"][5].isnan().all()
    assert got["dw"].isnan().all() and torch.equal(got["db"], clean["db"])


def test_same_bits_and_other_stream():
    g = gen(11)
    x, dy = randn(g, 4000, 1024, dtype=torch.bfloat16), randn(g, 4000, 1024, dtype=torch.bfloat16)
    w = randn(g, 1024, dtype=torch.bfloat16)
    first = run(x, w, w, dy)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        second = run(x, w, w, dy)
    s.synchronize()
    third = run(x, w, w, dy, stream=s)
    s.synchronize()
    for k in first:
        assert torch.equal(first[k], second[k]) and torch.equal(first[k], third[k]), k


def test_gradient_against_differences():
    """<dL/dx, v> and <dL/dw, v> against central differences of the kernel's own fp32 forward,
    L = sum(dy * y).  Step 2^-6: the third derivative's term is below h^2 (2.5e-4) of the slope's
    scale ||dx|| ||v||, and the rounding of y (2^-24 an element, random) below 1e-4 of it."""
    g = gen(12)
    n, d = 6, 40
    x, dy, v = randn(g, n, d), randn(g, n, d), randn(g, n, d)
    w, vw = randn(g, d), randn(g, d)
    got = run(x, w, None, dy)

    def L(x, w):
        y = torch.empty(n, d, device="cuda")
        ops.moe_layernorm_forward(x, w, None, EPS, y)
        return (y.double() * dy.double()).sum()

    h = 2.0 ** -6
    num = (L(x + h * v, w) - L(x - h * v, w)) / (2 * h)
    assert abs(num - (got["dx"].double() * v.double()).sum()) <= 2e-3 * got["dx"].double().norm() * v.double().norm()
    num = (L(x, w + h * vw) - L(x, w - h * vw)) / (2 * h)
    assert abs(num - (got["dw"].double() * vw.double()).sum()) <= 2e-3 * got["dw"].double().norm() * vw.double().norm()


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("d,pad", [(96, 0), (97, 0), (500, 2), (512, 0), (2046, 0), (2047, 0), (2048, 0), (2048, 1), (7168, 0),
                                   (12289, 0)])
def test_backward_of_rows_far_from_zero(d, pad, dt):
    """xh = (x - mean) rstd of the given statistics: the difference is exact here (neighbouring values of
    the type), so xh is off by one rounding of the product, however large mean * rstd is.  The statistics
    are chosen so that mean * rstd itself is not near an fp32 number."""
    g = gen(d + pad)
    n, at, step = 3, {"f32": 65536.0, "bf16": 256.0, "f16": 1024.0}[dt], {"f32": 1.0, "bf16": 2.0, "f16": 1.0}[dt]
    x = strided(g, n, d, DT[dt], pad)
    x.copy_(at + step * torch.randint(0, 3, (n, d), generator=g, device="cuda"))
    mean = (at + step * (0.9 + 0.1 * torch.rand(n, generator=g, device="cuda"))).float()
    tries = (0.9 + 0.2 * torch.rand(n, 1000, generator=g, device="cuda")) / step
    off = ((mean[:, None] * tries).double() - mean[:, None].double() * tries.double()).abs()
    rstd = tries.gather(1, off.argmax(1, keepdim=True))[:, 0].contiguous()
    dy, w = strided(g, n, d, DT[dt], pad), randn(g, d, std=0.3, mean=1.0)
    dx = empty_strided(n, d, DT[dt], pad)
    dw, db = torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
    ws = torch.empty(ops.moe_layernorm_workspace_bytes(n, d), dtype=torch.uint8, device="cuda")
    ops.moe_layernorm_backward(dy, x, w, mean, rstd, dx, dw, db, ws)
    rs, t, e = rstd.double()[:, None], dy.double(), (32 + math.log2(d)) * 2.0 ** -24
    xh, gg = (x.double() - mean.double()[:, None]) * rs, dy.double() * w.double()
    exh = 2.0 ** -23 * xh.abs()
    m1, m2 = gg.mean(1, keepdim=True), (gg * xh).mean(1, keepdim=True)
    a1, a2 = gg.abs().mean(1, keepdim=True), (gg * xh).abs().mean(1, keepdim=True)
    edx = rs * (e * (gg.abs() + a1 + 2 * xh.abs() * a2) + exh * a2 + xh.abs() * (gg.abs() * exh).mean(1, keepdim=True))
    close(dw, (t * xh).sum(0), "f32", (t.abs() * (exh + (e + n * 2.0 ** -24) * xh.abs())).sum(0), "dw")
    close(db, t.sum(0), "f32", (e + n * 2.0 ** -24) * t.abs().sum(0), "db")
    close(dx, rs * (gg - m1 - xh * m2), dt, edx, "dx")
