"""MXFP4 on the GPU: codes and scales exactly, the experts' product against 64 bits.

Bounds of the product: the products of 4-bit values and power-of-two scales are
exact in fp32; a sum of K of them in fp32, whatever the order and even if every
addition truncates, is off by at most K 2^-23 of the sum of magnitudes; then one
rounding (u |want|).  The SwiGLU epilogue: |silu'| <= 1.1 carries that error of
the gate, |silu| that of the up product, and exp and the division cost at most
2^-18 of the result (the gates stay below 64 in magnitude)."""
import numpy as np
import pytest
import torch

from mixture_experts_layer_stable_gb300 import binding as B
from mixture_experts_layer_stable_gb300 import ops

from ops_util import DT, close, empty_strided, gen, randn, strided

pytestmark = pytest.mark.gpu
GRID = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_lib):
    yield


def quantize(v):
    """[n, K] fp64 on the CPU -> (codes [n, K], scale bytes [n, K/32], values): nearest by distance,
    ties to the even code; s from exact integer comparisons."""
    n, K = v.shape
    b = v.reshape(n, K // 32, 32)
    amax = b.abs().amax(-1)
    fin = torch.isfinite(amax)
    m, e = torch.frexp(torch.where(fin, amax, torch.ones_like(amax)))
    s = torch.where(m <= 0.75, e - 3, e - 2).to(torch.int64)
    s = torch.where(amax == 0, torch.full_like(s, -127), s).clamp(min=-127)
    y = torch.ldexp(torch.where(fin[..., None], b, torch.zeros_like(b)), -s[..., None])
    dist = (y.abs()[..., None] - GRID).abs()
    best = dist.min(-1).values[..., None]
    near = dist == best
    idx = torch.arange(8)
    code = torch.where(near & (idx % 2 == 0), idx, 99).amin(-1)
    code = torch.where(code == 99, torch.where(near, idx, 99).amin(-1), code)
    val = GRID[code] * torch.where(torch.signbit(y), -1.0, 1.0)
    val = torch.ldexp(val, s[..., None])
    code = code + 8 * torch.signbit(y)
    code = torch.where(fin[..., None], code, 0)
    val = torch.where(fin[..., None], val, torch.full_like(val, float("nan")))
    byte = torch.where(fin, s + 127, torch.full_like(s, 255))
    return code.reshape(n, K).to(torch.uint8), byte.to(torch.uint8), val.reshape(n, K)


def row_tiles(byte, offsets):
    """{offset: byte} of the documented layout for rows."""
    n, nb = byte.shape
    KT = -(-nb // 4)
    out = {}
    for g in range(len(offsets) - 1):
        for i in range(offsets[g + 1] - offsets[g]):
            run, r = offsets[g] // 128 + g + i // 128, i % 128
            for kb in range(KT * 4):
                at = (run * KT + kb // 4) * 512 + 16 * (r % 32) + 4 * (r // 32) + kb % 4
                assert at not in out
                out[at] = int(byte[offsets[g] + i, kb]) if kb < nb else 127
    return out


def tricky(g, n, K, dt):
    """Blocks of very different sizes, ties, zeros, signed zeros, extremes of the type."""
    x = randn(g, n, K)
    b = x.reshape(-1, 32)
    b *= torch.exp2(torch.randint(-20, 20, (b.shape[0], 1), generator=g, device="cuda").float())
    if dt != "f16":
        b[::7] *= 2.0 ** 90
        b[1::7] *= 2.0 ** -100
    b[2::11] = 0.0
    b[3::11] = -0.0
    ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], device="cuda").repeat(4)
    b[4::11] = ties * torch.where(torch.arange(32, device="cuda") % 3 == 0, -1.0, 1.0)
    b[5::11] = torch.tensor([0.0] * 31 + [1.0], device="cuda")
    x = x.clamp(-torch.finfo(DT[dt]).max, torch.finfo(DT[dt]).max).to(DT[dt])
    x.reshape(-1, 32)[6::11, 0] = torch.finfo(DT[dt]).max
    x.reshape(-1, 32)[8::11] = torch.finfo(DT[dt]).tiny * 0.5
    return x


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n,K,counts", [(1, 32, [1]), (3, 64, [0, 2, 1]), (5, 96, None), (9, 160, [4, 0, 0, 5]),
                                        (300, 256, [130, 170]), (700, 128, [224, 0, 225, 1, 250]), (40, 7168, [17, 23])])
def test_rows_exactly(n, K, counts, dt):
    g = gen(n + K)
    x = tricky(g, n, K, dt)
    xs = empty_strided(n, K, DT[dt], pad=(0, 8, 1)[n % 3])
    xs.copy_(x)
    off = None if counts is None else torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device="cuda")
    G = 1 if counts is None else len(counts)
    q = torch.full((n, K // 2), 77, dtype=torch.uint8, device="cuda")
    sc = torch.full((ops.moe_mxfp4_row_scale_bytes(n, K, G),), 77, dtype=torch.uint8, device="cuda")
    ops.moe_quantize_mxfp4_rows(xs, q, sc, off)
    code, byte, val = quantize(x.cpu().double())
    qc = q.cpu()
    assert torch.equal(qc & 15, code[:, 0::2]) and torch.equal(qc >> 4, code[:, 1::2])
    scc = sc.cpu().numpy()
    for at, b in row_tiles(byte, [0, n] if off is None else off.tolist()).items():
        assert scc[at] == b, at
    y = empty_strided(n, K, torch.float32, pad=3)
    ops.moe_dequantize_mxfp4_rows(q, sc, y, off)
    # the smallest values (below fp32's subnormal step) round to it
    assert torch.equal(y.cpu(), val.float())
    # gathered on the way: the same bytes as of gathered rows
    k = 3
    perm = torch.randperm(n * k, generator=g, device="cuda").to(torch.int32)[:n].contiguous()
    q1, s1, q2, s2 = torch.empty_like(q), torch.empty_like(sc).fill_(1), torch.empty_like(q), torch.empty_like(sc).fill_(1)
    ops.moe_quantize_mxfp4_rows(xs, q1, s1, off, perm=perm, k=k)
    ops.moe_quantize_mxfp4_rows(x[perm.long() // k].contiguous(), q2, s2, off)
    assert torch.equal(q1, q2) and torch.equal(s1, s2)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("b,K,N,paired", [(1, 32, 1, False), (2, 64, 6, True), (3, 160, 130, False), (2, 96, 258, True)])
def test_weights_exactly(b, K, N, paired, dt):
    g = gen(b + K + N)
    rows = tricky(g, b * N, K, dt)
    w = rows.reshape(b, N, K).transpose(1, 2).contiguous()        # [b, K, N]
    q = torch.empty(b, N, K // 2, dtype=torch.uint8, device="cuda")
    sc = torch.full((ops.moe_mxfp4_weight_scale_bytes(b, K, N),), 77, dtype=torch.uint8, device="cuda")
    ops.moe_quantize_mxfp4(w, q, sc, paired)
    ref = rows.reshape(b, N, K)
    if paired:
        ref = torch.stack((ref[:, :N // 2], ref[:, N // 2:]), 2).reshape(b, N, K)
    code, byte, val = quantize(ref.reshape(b * N, K).cpu().double())
    qc = q.cpu().reshape(b * N, K // 2)
    assert torch.equal(qc & 15, code[:, 0::2]) and torch.equal(qc >> 4, code[:, 1::2])
    NT, KT, scc = -(-N // 128), -(-K // 128), sc.cpu().numpy()
    for r in range(b * N):
        e, n = divmod(r, N)
        for kb in range(K // 32):
            at = ((e * NT + n // 128) * KT + kb // 4) * 512 + 16 * (n % 32) + 4 * (n % 128 // 32) + kb % 4
            assert scc[at] == byte[r, kb]
    back = torch.empty(b, K, N, device="cuda")
    ops.moe_dequantize_mxfp4(q, sc, back, paired)
    val = val.float().reshape(b, N, K)
    if paired:
        val = torch.cat((val[:, 0::2], val[:, 1::2]), 1)
    assert torch.equal(back.cpu(), val.transpose(1, 2))


def experts(g, G, K, N, paired=False):
    w = randn(g, G, K, N, dtype=torch.bfloat16, std=K ** -0.5)
    q = torch.empty(G, N, K // 2, dtype=torch.uint8, device="cuda")
    sc = torch.empty(ops.moe_mxfp4_weight_scale_bytes(G, K, N), dtype=torch.uint8, device="cuda")
    ops.moe_quantize_mxfp4(w, q, sc, paired)
    v = torch.empty(G, K, N, device="cuda")
    ops.moe_dequantize_mxfp4(q, sc, v, paired)
    return q, sc, v.double()


def rows_of(x, off):
    G = off.numel() - 1
    q = torch.full((x.shape[0], x.shape[1] // 2), 255, dtype=torch.uint8, device="cuda")
    sc = torch.full((ops.moe_mxfp4_row_scale_bytes(*x.shape, G),), 255, dtype=torch.uint8, device="cuda")
    ops.moe_quantize_mxfp4_rows(x, q, sc, off)
    v = torch.zeros(x.shape, device="cuda")
    ops.moe_dequantize_mxfp4_rows(q, sc, v, off)
    return q, sc, v.double()


def product(q, sc, off, wq, ws, act, out):
    rows, G = out.shape[0], wq.shape[0]
    w = torch.full((ops.moe_mxfp4_product_workspace_bytes(rows, wq.shape[1], wq.shape[2] * 2, G),), 255,
                   dtype=torch.uint8, device="cuda")
    ops.moe_mxfp4_product(q, sc, off, wq, ws, act, out, w)
    assert B.moe_read_status(w) == 0


def want_of(xv, wv, off, act):
    """(want, error of the fp32 arithmetic), wv [G, K, N] with gate and up halves."""
    K, N = wv.shape[1], wv.shape[2]
    h = torch.zeros(xv.shape[0], N, dtype=torch.float64, device="cuda")
    a = torch.zeros_like(h)
    for e in range(wv.shape[0]):
        s = slice(off[e], off[e + 1])
        h[s], a[s] = xv[s] @ wv[e], xv[s].abs() @ wv[e].abs()
    err = K * 2.0 ** -23 * a
    if not act:
        return h, err
    g, u, eg, eu = h[:, :N // 2], h[:, N // 2:], err[:, :N // 2], err[:, N // 2:]
    silu = g * torch.sigmoid(g)
    out = silu * u
    return out, 1.1 * eg * (u.abs() + eu) + silu.abs() * eu + 2.0 ** -18 * out.abs()


PRODUCTS = [([1], 32, 1), ([1], 64, 8), ([3], 96, 7), ([0, 5, 0], 128, 127), ([16, 1], 160, 128), ([17, 33], 256, 129),
            ([128], 288, 256), ([129, 0, 2], 512, 300), ([223, 224, 225], 224, 130), ([449, 1], 1056, 999),
            ([1] * 40, 512, 64), ([0] * 30 + [700], 992, 260), ([1, 1, 1, 1, 1, 1, 1, 1], 7168, 512),
            ([300, 40, 0, 90], 2048, 1536), ([13], 4096, 4096), ([8], 7168, 2048),
            # long K and many rows: CTA pairs
            ([160], 4096, 256), ([0, 449, 1, 300], 4128, 389), ([193, 200, 1025], 4224, 130), ([320, 0], 7168, 1000)]


@pytest.mark.parametrize("act", [False, True])
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("counts,K,N", PRODUCTS)
def test_product(counts, K, N, dt, act):
    if act and N % 2:
        N += 1
    g = gen(sum(counts) + K + N)
    n, G = sum(counts), len(counts)
    off = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device="cuda")
    x = randn(g, n, K, dtype=torch.bfloat16)
    q, sc, xv = rows_of(x, off)
    wq, ws, wv = experts(g, G, K, N, act)
    want, err = want_of(xv, wv, off.tolist(), act)
    nout = want.shape[1]
    out = empty_strided(n, nout, DT[dt], pad=(0, 8, 1)[n % 3], fill=float("nan"))
    product(q, sc, off, wq, ws, int(act), out)
    close(out, want, dt, err, "out")
    again = torch.empty(n, nout, dtype=DT[dt], device="cuda")
    product(q, sc, off, wq, ws, int(act), again)
    assert torch.equal(again, out)


def test_rows_behind_the_last_expert_are_left_alone():
    g = gen(3)
    K, N, n = 128, 72, 50
    off = torch.tensor([0, 10, 10, 31], dtype=torch.int32, device="cuda")
    x = randn(g, n, K, dtype=torch.bfloat16)
    x[31:] = float("nan")
    q, sc, xv = rows_of(x, off)
    assert (q[31:] == 255).all()
    wq, ws, wv = experts(g, 3, K, N)
    out = torch.full((n, N), 5.0, dtype=torch.bfloat16, device="cuda")
    product(q, sc, off, wq, ws, 0, out)
    want, err = want_of(xv, wv, off.tolist(), False)
    close(out[:31], want[:31], "bf16", err[:31], "out")
    assert (out[31:] == 5.0).all()
    # no rows at all
    z = torch.zeros(4, dtype=torch.int32, device="cuda")
    out.fill_(5.0)
    product(q, sc, z, wq, ws, 0, out)
    assert (out == 5.0).all()


def test_one_segment_without_offsets():
    g = gen(4)
    K, N, n = 320, 200, 77
    x = randn(g, n, K, dtype=torch.bfloat16)
    off = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    q, sc, xv = rows_of(x, off)
    wq, ws, wv = experts(g, 1, K, N)
    a, b = (torch.empty(n, N, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    product(q, sc, off, wq, ws, 0, a)
    product(q, sc, None, wq, ws, 0, b)
    assert torch.equal(a, b)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_non_finite_values_become_nan_in_their_rows_and_columns(bad):
    g = gen(5)
    K, N, counts = 256, 136, [20, 200]
    off = torch.tensor([0, 20, 220], dtype=torch.int32, device="cuda")
    x = randn(g, 220, K, dtype=torch.bfloat16)
    clean_q, clean_s, _ = rows_of(x, off)
    x[150, 40] = bad
    q, sc, _ = rows_of(x, off)
    w = randn(g, 2, K, N, dtype=torch.bfloat16)
    wq = torch.empty(2, N, K // 2, dtype=torch.uint8, device="cuda")
    ws, ws2 = (torch.empty(ops.moe_mxfp4_weight_scale_bytes(2, K, N), dtype=torch.uint8, device="cuda") for _ in range(2))
    ops.moe_quantize_mxfp4(w, wq, ws)
    ref, out = (torch.empty(220, N, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    product(clean_q, clean_s, off, wq, ws, 0, ref)
    product(q, sc, off, wq, ws, 0, out)
    assert out[150].isnan().all()
    rest = [i for i in range(220) if i != 150]
    assert torch.equal(out[rest], ref[rest])
    w[0, 99, 130] = bad
    wq2 = torch.empty_like(wq)
    ops.moe_quantize_mxfp4(w, wq2, ws2)
    product(clean_q, clean_s, off, wq2, ws2, 0, out)
    assert out[:20, 130].isnan().all()
    out[:20, 130] = ref[:20, 130]
    assert torch.equal(out, ref)


def test_extreme_scales():
    """Values far from 1 on one side met by the opposite on the other: nothing overflows on the way."""
    g = gen(6)
    K, N, n = 128, 64, 40
    off = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    for e in (-100, -60, 60, 100):
        x = (randn(g, n, K) * 2.0 ** e).to(torch.bfloat16)
        w = (randn(g, 1, K, N) * 2.0 ** -e).to(torch.bfloat16)
        q, sc, xv = rows_of(x, off)
        wq = torch.empty(1, N, K // 2, dtype=torch.uint8, device="cuda")
        ws = torch.empty(ops.moe_mxfp4_weight_scale_bytes(1, K, N), dtype=torch.uint8, device="cuda")
        ops.moe_quantize_mxfp4(w, wq, ws)
        wv = torch.empty(1, K, N, device="cuda")
        ops.moe_dequantize_mxfp4(wq, ws, wv)
        want, err = want_of(xv, wv.double(), [0, n], False)
        out = torch.empty(n, N, device="cuda")
        product(q, sc, off, wq, ws, 0, out)
        close(out, want, "f32", err, f"2^{e}")


def test_other_stream():
    g = gen(7)
    K, N, n = 512, 384, 300
    off = torch.tensor([0, 100, 300], dtype=torch.int32, device="cuda")
    x = randn(g, n, K, dtype=torch.bfloat16)
    q, sc, _ = rows_of(x, off)
    wq, ws, _ = experts(g, 2, K, N, True)
    a, b = (torch.empty(n, N // 2, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    product(q, sc, off, wq, ws, 1, a)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    w = torch.empty(ops.moe_mxfp4_product_workspace_bytes(n, N, K, 2), dtype=torch.uint8, device="cuda")
    q2, s2 = torch.empty_like(q), torch.empty_like(sc)
    torch.cuda.synchronize()
    ops.moe_quantize_mxfp4_rows(x, q2, s2, off, stream=st)
    ops.moe_mxfp4_product(q2, s2, off, wq, ws, 1, b, w, stream=st)
    st.synchronize()
    assert torch.equal(a, b)


@pytest.mark.parametrize("N,act", [(64, 0), (64, 1)])
def test_no_rows_clear_the_status(N, act):
    """A call without rows launches no kernel, and its status is its own all the same: not what the
    workspace held."""
    K, G = 128, 3
    off = torch.zeros(G + 1, dtype=torch.int32, device="cuda")
    empty = torch.empty(0, dtype=torch.uint8, device="cuda")
    wq, ws, _ = experts(gen(8), G, K, N, bool(act))
    out = torch.empty(0, N // 2 if act else N, dtype=torch.bfloat16, device="cuda")
    sc = torch.empty(ops.moe_mxfp4_row_scale_bytes(0, K, G), dtype=torch.uint8, device="cuda")
    for stream in (None, torch.cuda.Stream()):
        w = torch.full((ops.moe_mxfp4_product_workspace_bytes(0, N, K, G),), 255, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        ops.moe_mxfp4_product(empty, sc, off, wq, ws, act, out, w, stream=stream)
        assert B.moe_read_status(w, stream) == 0


@pytest.mark.parametrize("n,K,N", [(40, 32, 512), (7, 96, 130), (160, 4096, 512)])
def test_swiglu_in_fp32(n, K, N):
    """Results of 32 bits have the precision of fp32 throughout.  One value a row meets one a
    column, so that the products h are exact; of silu(g) u with g in [-72, 72] the exponential is off by
    at most 2 units in the last place (2^-22) and the sum, the two products and the division by 2^-24
    each: 2^-21 of the result."""
    g = gen(9 + K)

    def exact(count, low, high):  # +- 1 or 1.5 times a power of two: quantised without an error
        m = 1 + 0.5 * torch.randint(0, 2, (count,), generator=g, device="cuda")
        s = 1 - 2 * torch.randint(0, 2, (count,), generator=g, device="cuda")
        return m * s * torch.exp2(torch.randint(low, high + 1, (count,), generator=g, device="cuda").float())

    x, w = torch.zeros(n, K, device="cuda"), torch.zeros(1, K, N, device="cuda")
    x[:, 0], w[0, 0] = exact(n, -2, 2), exact(N, -6, 3)
    w[0, 0, N // 2:] = exact(N // 2, -3, 3)
    off = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    q, sc, xv = rows_of(x, off)
    assert torch.equal(xv, x.double())
    wq = torch.empty(1, N, K // 2, dtype=torch.uint8, device="cuda")
    ws = torch.empty(ops.moe_mxfp4_weight_scale_bytes(1, K, N), dtype=torch.uint8, device="cuda")
    ops.moe_quantize_mxfp4(w, wq, ws, True)
    h = x[:, :1].double() * w[0, :1].double()
    want = h[:, :N // 2] * torch.sigmoid(h[:, :N // 2]) * h[:, N // 2:]
    out = torch.empty(n, N // 2, device="cuda")
    product(q, sc, off, wq, ws, 1, out)
    close(out, want, "f32", 2.0 ** -21 * want.abs(), "out")


def test_swiglu_in_fp32_of_large_gates():
    """Gates far below zero met by large up products: exp(-g) would overflow, the result does not vanish."""
    gate = torch.tensor([-64.0, -80.0, -84.0, -96.0, 96.0, 192.0], dtype=torch.float64, device="cuda")
    up, K, n = 2.0 ** 100, 64, 4
    N = 2 * gate.numel()
    x, w = torch.zeros(n, K, device="cuda"), torch.zeros(1, K, N, device="cuda")
    x[:, 0], x[:, 32] = 1.0, 1.0        # a block for the gates, one for the up products
    # -80 and -84 as sums of two values that are exact in 4 bits
    for i, v in enumerate(gate.tolist()):
        a = {-80.0: -64.0, -84.0: -96.0}.get(v, v)
        w[0, 0, i], w[0, 32, i] = a, v - a
    w[0, 32, N // 2:] = up
    off = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    q, sc, _ = rows_of(x, off)
    wq = torch.empty(1, N, K // 2, dtype=torch.uint8, device="cuda")
    ws = torch.empty(ops.moe_mxfp4_weight_scale_bytes(1, K, N), dtype=torch.uint8, device="cuda")
    ops.moe_quantize_mxfp4(w, wq, ws, True)
    v = torch.empty(1, K, N, device="cuda")
    ops.moe_dequantize_mxfp4(wq, ws, v, True)
    assert torch.equal(v, w)
    want = (gate * torch.sigmoid(gate) * up).expand(n, -1)
    out = torch.empty(n, N // 2, device="cuda")
    product(q, sc, off, wq, ws, 1, out)
    # exp(-96) = 2^-138.5 is a subnormal number in fp32, of steps of 2^-149: two of them are 2^-9.5 of it
    close(out, want, "f32", (2.0 ** -21 + torch.where(gate < -87, 2.0 ** -9, 0.0)) * want.abs(), "out")


@pytest.mark.parametrize("K,n,bounds", [(128, 50, [10, 10, 31]), (96, 700, [1, 130, 258, 699]), (8224, 20, [5, 20])])
def test_rows_before_the_first_expert_are_left_alone(K, n, bounds):
    """The offsets of some of the experts: rows before theirs have no place among the scales."""
    g = gen(K)
    N, G = 72, len(bounds) - 1
    a, b = bounds[0], bounds[-1]
    off = torch.tensor(bounds, dtype=torch.int32, device="cuda")
    x = randn(g, n, K, dtype=torch.bfloat16)
    guard, size = 1 << 16, ops.moe_mxfp4_row_scale_bytes(n, K, G)
    buf = torch.full((size + 2 * guard,), 77, dtype=torch.uint8, device="cuda")
    sc = buf[guard:guard + size]
    q = torch.full((n, K // 2), 255, dtype=torch.uint8, device="cuda")
    ops.moe_quantize_mxfp4_rows(x, q, sc, off)
    assert (q[:a] == 255).all() and (q[b:] == 255).all()
    assert (buf[:guard] == 77).all() and (buf[guard + size:] == 77).all()
    # the rows between as with offsets that begin at 0 for them alone
    q0, s0, v0 = rows_of(x[a:b].contiguous(), off - a)
    assert torch.equal(q[a:b], q0)
    v = torch.full((n, K), 9.0, device="cuda")
    ops.moe_dequantize_mxfp4_rows(q, sc, v, off)
    assert torch.equal(v[a:b].double(), v0) and (v[:a] == 9.0).all() and (v[b:] == 9.0).all()
    wq, ws, wv = experts(g, G, K, N)
    out = torch.full((n, N), 5.0, dtype=torch.bfloat16, device="cuda")
    product(q, sc, off, wq, ws, 0, out)
    ref = torch.empty(b - a, N, dtype=torch.bfloat16, device="cuda")
    product(q0, s0, off - a, wq, ws, 0, ref)
    assert torch.equal(out[a:b], ref) and (out[:a] == 5.0).all() and (out[b:] == 5.0).all()


def test_no_rows_in_a_graph():
    """A call without rows is captured like any other."""
    K, N = 64, 8
    wq, ws, _ = experts(gen(10), 1, K, N)
    empty, sc = torch.empty(0, dtype=torch.uint8, device="cuda"), torch.empty(512, dtype=torch.uint8, device="cuda")
    out, w = torch.empty(0, N, device="cuda"), torch.full((128,), 255, dtype=torch.uint8, device="cuda")
    off = torch.zeros(2, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.moe_mxfp4_product(empty, sc, off, wq, ws, 0, out, w)
    graph.replay()
    assert B.moe_read_status(w) == 0
