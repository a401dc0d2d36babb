"""Activations kept in 8 bits and SwiGLU on the GPU, against 64 bits.

Codes, scales and values are exact: scales are powers of two, so nothing rounds but the
codes themselves.  SwiGLU's bounds: fp32 arithmetic of at most ten operations and an
exponential, each within 2^-22 of its result (expf: 2 ulp, the sums of the slope have no term
larger than 1 + |g|); 16-bit types use the hardware exponential and reciprocal, within 2^-18
of the sigmoid for |g| <= 64; then one rounding."""
import pytest
import torch

from mixture_experts_layer_stable_gb300 import ops

from ops_util import DT, close, empty_strided, gen, randn, strided

pytestmark = pytest.mark.gpu
EPS = {"f32": 2.0 ** -20, "bf16": 2.0 ** -17, "f16": 2.0 ** -17}
MARK = 7.0


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_lib):
    yield


def quantize(v):
    """fp64 rows -> (codes, scale bytes, values) by the definition: exponents tried upwards, nearest
    whole number by comparison, ties to even."""
    n, d = v.shape
    nb = -(-d // 32)
    b = torch.zeros(n, nb * 32, dtype=torch.float64, device=v.device)
    b[:, :d] = v
    b = b.reshape(n, nb, 32)
    top = b.abs().amax(-1, keepdim=True)
    fin = torch.isfinite(top)
    top = torch.where(fin, top, torch.ones_like(top))
    b = torch.where(fin, b, torch.zeros_like(b))
    s = torch.floor(torch.log2(top.clamp(min=2.0 ** -200) / 127)) - 1
    for _ in range(3):
        s = torch.where(top > 127 * torch.exp2(s), s + 1, s)
    s = s.clamp(min=-127)
    y = b * torch.exp2(-s)
    low = torch.floor(y)
    up = (y - low > 0.5) | ((y - low == 0.5) & (low % 2 != 0))
    c = low + up
    c = torch.where(s >= 122, c.clamp(-63, 63), c)
    val = torch.where(fin, c * torch.exp2(s), torch.full_like(c, float("nan")))
    byte = torch.where(fin, s + 127, torch.full_like(s, 255))
    cut = lambda t: t.reshape(n, -1)[:, :d]  # noqa: E731
    return cut(c).to(torch.int8), byte.reshape(n, nb).to(torch.uint8), cut(val)


def kept(rows, n, shift=0):
    q = torch.full((rows * n + shift,), 99, dtype=torch.int8, device="cuda")[shift:].reshape(rows, n)
    return q, torch.full((ops.moe_mxint8_scale_bytes(rows, n),), 9, dtype=torch.uint8, device="cuda")


SHAPES = [(1, 1, 0, 0), (3, 31, 0, 0), (2, 32, 0, 0), (5, 33, 1, 1), (64, 96, 8, 0), (17, 1000, 0, 0), (9, 1003, 0, 0),
          (300, 768, 0, 0), (40, 2048, 16, 8), (7, 2048, 3, 0), (33, 8200, 0, 0), (4, 20000, 8, 8), (6, 4099, 5, 3),
          (3, 2, 0, 0), (21, 34, 2, 2), (50, 1002, 0, 0), (5, 4690, 4, 2)]


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,n,pad,shift", SHAPES)
def test_rows_codes_scales_values(dt, rows, n, pad, shift):
    g = gen(rows + n)
    x = strided(g, rows, n, DT[dt], pad, shift, std=1.5, mean=0.2)
    x[rows // 2, : n // 2] *= 2.0 ** -10            # blocks of other sizes in a row
    x[0, n // 3:] = 0
    q, s = kept(rows, n, shift)
    ops.moe_quantize_mxint8_rows(x, q, s)
    code, byte, val = quantize(x.double())
    assert torch.equal(q, code) and torch.equal(s.reshape(byte.shape), byte)
    for ydt in ("f32", dt):
        buf = empty_strided(rows, n + 2, DT[ydt], pad, shift, MARK)  # y inside wider rows
        y = buf[:, :n]
        ops.moe_dequantize_mxint8_rows(q, s, y)
        assert torch.equal(y.double(), val.to(DT[ydt]).double())
        assert bool((buf[:, n:] == MARK).all())
    assert bool((val - x.double()).abs().le(x.double().abs().amax(1, keepdim=True) / 127).all())


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("n", [256, 259])
def test_ties_extremes_and_non_finite_blocks(dt, n):
    """Ties go to even, each scale's limit stays with it, the largest values come back finite, the
    smallest on a grid of 2^-127, and a block with a NaN or an infinity comes back as NaN alone."""
    t, fi = DT[dt], torch.finfo(DT[dt])
    x = torch.zeros(11, n, dtype=torch.float64)
    ramp = torch.arange(n, dtype=torch.float64) % 32
    x[0] = ramp + 0.5                               # ties of s = 0 where the block holds more than 63.5
    x[0, ::32] = 127
    x[1] = ramp - 15.5
    x[1, ::32] = -127
    x[2, ::32] = 127                                # the largest of its scale
    x[3, ::32] = 127.5                              # (128 in bf16) the next scale
    x[4] = fi.max
    x[5] = -fi.max
    x[5, 1::2] = fi.max / 3
    x[6] = fi.tiny * ramp
    x[7] = fi.smallest_normal / 2 * (ramp % 2)
    x[8, 40] = float("nan")
    x[9, 70] = float("-inf")
    x[10] = torch.linspace(-1, 1, n, dtype=torch.float64)
    x = x.to(t).cuda()
    q, s = kept(11, n)
    ops.moe_quantize_mxint8_rows(x, q, s)
    code, byte, val = quantize(x.double())
    assert torch.equal(s.reshape(byte.shape), byte)
    assert torch.equal(q, torch.where(torch.isnan(val), torch.zeros_like(code), code))
    y = torch.empty(11, n, dtype=t, device="cuda")
    ops.moe_dequantize_mxint8_rows(q, s, y)
    want = val.clamp(-fi.max, fi.max) if dt == "f16" else val
    want = torch.where(torch.isnan(val), val, want).to(t)
    assert torch.equal(torch.isnan(y), torch.isnan(want)) and torch.equal(torch.nan_to_num(y), torch.nan_to_num(want))
    bad = torch.isnan(y)
    assert int(bad.sum()) == 64 and bool(bad[8, 32:64].all()) and bool(bad[9, 64:96].all())
    assert bool(torch.isfinite(y[:8]).all())


def swiglu64(g, u, da=None):
    s = torch.sigmoid(g)
    a = g * s * u
    if da is None:
        return a
    return a, torch.cat((da * u * (s + g * s * torch.sigmoid(-g)), da * g * s), 1)


def bound_dh(g, u, da):
    return torch.cat((da.abs() * u.abs() * (1 + g.abs()), da.abs() * g.abs()), 1)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,f,pad,shift", SHAPES)
def test_swiglu_and_its_backward(dt, rows, f, pad, shift):
    g = gen(rows * 3 + f)
    t, e = DT[dt], EPS[dt]
    h, da = strided(g, rows, 2 * f, t, pad, shift, std=2.0), strided(g, rows, f, t, pad, shift)
    gate, up = h[:, :f].double(), h[:, f:].double()
    a = empty_strided(rows, f, t, pad, shift, MARK)
    ops.moe_swiglu_forward(h, a)
    close(a, swiglu64(gate, up), dt, e * (gate * up).abs())
    # with a checkpoint: the same bits, and the checkpoint of the halves
    q, s = kept(2 * rows, f, shift)
    a2 = empty_strided(rows, f, t, pad, shift, MARK)
    ops.moe_swiglu_forward(h, a2, q.reshape(rows, 2 * f), s)
    assert torch.equal(a, a2)
    halves = torch.cat((gate, up), 1).reshape(2 * rows, f)
    code, byte, val = quantize(halves)
    assert torch.equal(q, code) and torch.equal(s.reshape(byte.shape), byte)
    # the backward from h and from the checkpoint
    val = val.reshape(rows, 2 * f)
    for src, (vg, vu) in ((True, (gate, up)), (False, (val[:, :f], val[:, f:]))):
        dh, again = empty_strided(rows, 2 * f, t, pad, shift, MARK), empty_strided(rows, f, t, pad, shift, MARK)
        args = (da, h, dh, again) if src else (da, None, dh, again, q, s)
        ops.moe_swiglu_backward(*args)
        want_a, want = swiglu64(vg, vu, da.double())
        close(again, want_a, dt, e * (vg * vu).abs())
        close(dh, want, dt, e * bound_dh(vg, vu, da.double()))
        alone = empty_strided(rows, 2 * f, t, pad, shift, MARK)
        ops.moe_swiglu_backward(*((da, h, alone) if src else (da, None, alone, None, q, s)))
        assert torch.equal(alone, dh)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("f", [64, 67])
def test_swiglu_of_large_gates_and_non_finite_rows(dt, f):
    """Gates far out on both sides saturate without NaN; a NaN stays in its element (or its checkpoint's
    block), and rows keep to themselves."""
    t = DT[dt]
    h = torch.zeros(6, 2 * f, device="cuda")
    h[:, f:] = 1.5
    for r, v in enumerate((60.0, -60.0, 3e4, -3e4, 0.0)):
        h[r, :f] = v
    h[5, 40] = float("nan")
    h = h.to(t)
    da = torch.ones(6, f, dtype=t, device="cuda")
    a, dh = torch.empty(6, f, dtype=t, device="cuda"), torch.empty(6, 2 * f, dtype=t, device="cuda")
    q, s = kept(12, f)
    ops.moe_swiglu_forward(h, a, q, s)
    gate, up = h[:, :f].double(), h[:, f:].double()
    close(a[:5], swiglu64(gate, up)[:5], dt, EPS[dt] * (gate * up).abs()[:5])
    assert bool(torch.isnan(a[5, 40])) and int(torch.isnan(a).sum()) == 1
    for kw in (dict(), dict(q=q, scales=s)):
        ops.moe_swiglu_backward(da, None if kw else h, dh, **kw)
        v = quantize(torch.cat((gate, up), 1).reshape(12, f))[2].reshape(6, 2 * f) if kw else h.double()
        close(dh[:5], swiglu64(v[:5, :f], v[:5, f:], da[:5].double())[1], dt,
              EPS[dt] * bound_dh(v[:5, :f], v[:5, f:], da[:5].double()))
        bad = torch.isnan(dh)
        assert not bool(bad[:5].any())
        assert int(bad.sum()) == 2 * (min(64, f) - 32 if kw else 1)


@pytest.mark.parametrize("f", [96, 53])
def test_backward_against_differences(f):
    """fp32: (a(h + e v) - a(h - e v)) / 2e against <dh, v>, e = 2^-6: the third derivative's share is
    below e^2 of sums of magnitudes of order one, roundings 2^-20 / e."""
    g = gen(11)
    h, v, da = randn(g, 30, 2 * f), randn(g, 30, 2 * f), randn(g, 30, f)
    dh = torch.empty(30, 2 * f, device="cuda")
    ops.moe_swiglu_backward(da, h, dh)
    e = 2.0 ** -6

    def a(x):
        y = torch.empty(30, f, device="cuda")
        ops.moe_swiglu_forward(x, y)
        return y.double()

    got = (da.double() * (a(h + e * v) - a(h - e * v)) / (2 * e)).sum(1)
    want = (dh.double() * v.double()).sum(1)
    mag = (da.abs() * (1 + h[:, :f].abs()) * (1 + h[:, f:].abs()) * (1 + v[:, :f].abs()) ** 3 *
           (1 + v[:, f:].abs())).double().sum(1)
    assert bool(((got - want).abs() <= (e * e + 2.0 ** -20 / e) * mag).all())


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("f", [128, 77])
def test_in_place(dt, f):
    """dh in the place of h and a in the place of da."""
    g = gen(12)
    t = DT[dt]
    h, da = randn(g, 50, 2 * f, dtype=t), randn(g, 50, f, dtype=t)
    dh, again = torch.empty_like(h), torch.empty_like(da)
    ops.moe_swiglu_backward(da, h, dh, again)
    ops.moe_swiglu_backward(da, h, h, da)
    assert torch.equal(h, dh) and torch.equal(da, again)


def test_no_rows_and_streams():
    z = torch.empty(0, 16, device="cuda")
    ops.moe_quantize_mxint8_rows(z, torch.empty(0, 16, dtype=torch.int8, device="cuda"), torch.empty(0, dtype=torch.uint8, device="cuda"))
    ops.moe_swiglu_forward(torch.empty(0, 32, device="cuda"), z)
    g = gen(13)
    h = randn(g, 2000, 512, dtype=torch.bfloat16)
    a, b = (torch.empty(2000, 256, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ops.moe_swiglu_forward(h, a)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ops.moe_swiglu_forward(h, b, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(a, b)


def test_captured_chain():
    """Forward and backward from the checkpoint in a graph, replayed on other values."""
    g = gen(14)
    bf = torch.bfloat16
    h, da = randn(g, 300, 1536, dtype=bf), randn(g, 300, 768, dtype=bf)
    q, s = kept(600, 768)
    bufs = [torch.empty(300, n, dtype=bf, device="cuda") for n in (768, 1536, 768)]

    def chain(a, dh, again):
        ops.moe_swiglu_forward(h, a, q, s)
        ops.moe_swiglu_backward(da, None, dh, again, q, s)

    chain(*bufs)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain(*bufs)
    h.copy_(randn(g, 300, 1536, dtype=bf))
    graph.replay()
    torch.cuda.synchronize()
    got = [b.clone() for b in bufs]
    chain(*bufs)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, bufs))


def test_rows_past_32_bits_of_elements():
    if torch.cuda.mem_get_info()[0] < 40e9:
        pytest.skip("needs 40 GB")
    rows, f = 150_000, 14_336                       # h: 4.3e9 elements
    h = torch.zeros(rows, 2 * f, dtype=torch.bfloat16, device="cuda")
    g = gen(15)
    h[-3:] = randn(g, 3, 2 * f, dtype=torch.bfloat16)
    a, da = torch.empty(rows, f, dtype=torch.bfloat16, device="cuda"), torch.ones(rows, f, dtype=torch.bfloat16, device="cuda")
    q, s = kept(2 * rows, f)
    ops.moe_swiglu_forward(h, a, q, s)
    gate, up = h[-3:, :f].double(), h[-3:, f:].double()
    close(a[-3:], swiglu64(gate, up), "bf16", EPS["bf16"] * (gate * up).abs())
    assert not bool(a[:-3].any())
    val = quantize(h[-3:].double().reshape(6, f))[2].reshape(3, 2 * f)
    ops.moe_swiglu_backward(da, None, h, a, q, s)
    want_a, want = swiglu64(val[:, :f], val[:, f:], da[-3:].double())
    close(a[-3:], want_a, "bf16", EPS["bf16"] * (val[:, :f] * val[:, f:]).abs())
    close(h[-3:], want, "bf16", EPS["bf16"] * bound_dh(val[:, :f], val[:, f:], da[-3:].double()))
