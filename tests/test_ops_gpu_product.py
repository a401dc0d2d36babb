"""Products by expert and their gradients on the GPU, against 64 bits.

Bounds: a product of two 16-bit values is exact in fp32; one of fp32 values, in three parts of 8
bits each, misses terms of less than 2^-24 of it; a sum of n of them in fp32, whatever the order and even if every addition
truncates, is off by at most n 2^-23 of the sum of magnitudes (n + 1 with an initial value);
then one rounding (u |want|)."""
import pytest
import torch

from mixture_experts_layer_stable_gb300 import binding as B
from mixture_experts_layer_stable_gb300 import ops

from ops_util import DT, close, empty_strided, gen, randn, strided

pytestmark = pytest.mark.gpu
MARK = 7.0  # what rows hold that a call must not write


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_lib):
    yield


def workspace(rows, K, N, G, fill=255):
    return torch.full((ops.moe_grouped_product_workspace_bytes(rows, K, N, G),), fill, dtype=torch.uint8, device="cuda")


def offsets_of(counts, first=0):
    o = [first]
    for c in counts:
        o.append(o[-1] + c)
    return torch.tensor(o, dtype=torch.int32, device="cuda")


def check_rows(x, w, off, out, dt, transposed):
    """out of the rows of each expert against 64 bits; the others still hold MARK."""
    o = off.tolist()
    K = x.shape[1]
    for g in range(len(o) - 1):
        s = slice(o[g], o[g + 1])
        if s.start == s.stop:
            continue
        a, b = x[s].double(), w[g].double()
        b = b.t() if transposed else b
        close(out[s], a @ b, dt, K * 2.0 ** -23 * (a.abs() @ b.abs()), f"expert {g}")
    assert bool((out[:o[0]] == MARK).all()) and bool((out[o[-1]:] == MARK).all())


def check_dw(x, dy, off, dw, dt, was=None):
    o = off.tolist()
    for g in range(len(o) - 1):
        s = slice(o[g], o[g + 1])
        a, b = x[s].double().t(), dy[s].double()
        want, mag = a @ b, a.abs() @ b.abs()
        if was is not None:
            want, mag = want + was[g].double(), mag + was[g].double().abs()
        close(dw[g], want, dt, (s.stop - s.start + 1) * 2.0 ** -23 * mag, f"expert {g}")


def run_all(dt, odt, counts, K, N, pad=0, shift=0, first=0, behind=0, seed=0):
    """The forward, both gradients and the accumulating form on one set of rows; rows outside the
    experts hold NaN."""
    g = gen(seed + K * 31 + N)
    t, ot = DT[dt], DT[odt]
    off = offsets_of(counts, first)
    n, G = int(off[-1]) + behind, len(counts)
    x, dy = strided(g, n, K, t, pad, shift), strided(g, n, N, t, pad, shift)
    for r in (x, dy):
        r[:first] = float("nan")
        r[n - behind:] = float("nan")
    w = randn(g, G * K * N + shift, dtype=t, std=K ** -0.5)[shift:].reshape(G, K, N)
    ws = workspace(n, K, N, G)
    out = empty_strided(n, N, ot, pad, shift, MARK)
    ops.moe_grouped_product(x, w, off, out, ws)
    check_rows(x, w, off, out, odt, False)
    dx = empty_strided(n, K, ot, pad, shift, MARK)
    ops.moe_grouped_product(dy, w, off, dx, ws, transposed=True)
    check_rows(dy, w, off, dx, odt, True)
    dw = torch.full((G * K * N + shift,), MARK, dtype=ot, device="cuda")[shift:].reshape(G, K, N)
    ops.moe_grouped_product_dw(x, dy, off, dw, ws)
    check_dw(x, dy, off, dw, odt)
    was = randn(g, G, K, N, dtype=ot)
    more = torch.full((G * K * N + shift,), MARK, dtype=ot, device="cuda")[shift:].reshape(G, K, N)
    more.copy_(was)
    ops.moe_grouped_product_dw(x, dy, off, more, ws, accumulate=True)
    check_dw(x, dy, off, more, odt, was)
    assert B.moe_read_status(ws) == 0


TYPES = [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32"), ("f32", "f32")]


@pytest.mark.parametrize("dt,odt", TYPES)
@pytest.mark.parametrize("counts,K,N", [
    ([1], 1, 1), ([3], 8, 8), ([0, 5, 0], 16, 24), ([1, 1, 1, 1], 64, 64), ([127, 128, 129, 0, 1], 128, 136),
    ([255, 256, 257, 300], 192, 320), ([16], 72, 520), ([700], 64, 256), ([33, 64, 65], 1000, 8), ([2, 0, 0, 40], 8, 1000),
    ([128, 130], 256, 512), ([5, 70, 200], 2048, 264)])
def test_products_and_gradients(dt, odt, counts, K, N):
    run_all(dt, odt, counts, K, N)


@pytest.mark.parametrize("dt,odt", TYPES)
@pytest.mark.parametrize("counts,K,N,pad,shift", [
    ([40, 0, 9], 64, 64, 8, 0), ([40, 200], 72, 80, 16, 8), ([17, 3], 33, 47, 0, 0), ([130, 131], 65, 129, 3, 1),
    ([50], 127, 255, 1, 0), ([64, 64], 64, 128, 0, 1), ([64, 64], 64, 128, 2, 2), ([257], 130, 258, 4, 4), ([9, 300], 515, 77, 5, 3)])
def test_strides_and_alignment(dt, odt, counts, K, N, pad, shift):
    run_all(dt, odt, counts, K, N, pad, shift)


@pytest.mark.parametrize("dt,odt", TYPES)
@pytest.mark.parametrize("counts,K,N,first,behind", [
    ([8], 4096, 24, 0, 0), ([40, 3], 2048, 130, 7, 90), ([3000], 24, 136, 0, 0), ([1, 0, 2500, 17], 96, 40, 3, 1),
    ([130], 1100, 260, 0, 0), ([5], 1025, 1023, 2, 3), ([2049], 65, 33, 0, 0)])
def test_long_contractions_of_few_tiles(dt, odt, counts, K, N, first, behind):
    """Contractions cut into parts, those of experts that are shorter than the others too."""
    run_all(dt, odt, counts, K, N, first=first, behind=behind)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("K,N", [(64, 128), (61, 45)])
def test_rows_of_some_of_the_experts(dt, K, N):
    """Offsets that begin above 0 and end before the last row; the rows outside are neither used nor written."""
    run_all(dt, dt, [70, 0, 33], K, N, first=21, behind=150)
    run_all(dt, dt, [0, 0], K, N, first=5, behind=5)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_many_experts(dt):
    g = torch.Generator().manual_seed(5)
    counts = torch.randint(0, 4, (1024,), generator=g).tolist()
    run_all(dt, dt, counts, 24, 40)


@pytest.mark.parametrize("odt", ["bf16", "f32"])
@pytest.mark.parametrize("counts,K,N", [([1000, 40, 24], 16, 40_000), ([500, 7, 0, 9], 264, 10_000)])
def test_many_units_of_one_stage(odt, counts, K, N):
    """Contractions that end inside their only stage, several units of them under way in a block."""
    run_all("bf16", odt, counts, K, N)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_one_segment_and_long_contractions(dt):
    """offsets None, K long; and one expert's many rows into its weights' gradient."""
    g = gen(1)
    t = DT[dt]
    for rows, K, N in ((1, 7168, 512), (8, 7168, 136), (300, 4096, 256), (5000, 128, 256)):
        x, w, dy = randn(g, rows, K, dtype=t), randn(g, 1, K, N, dtype=t, std=K ** -0.5), randn(g, rows, N, dtype=t)
        ws = workspace(rows, K, N, 1)
        out = torch.empty(rows, N, dtype=t, device="cuda")
        ops.moe_grouped_product(x, w, None, out, ws)
        off = torch.tensor([0, rows])
        check_rows(x, w, off, out, dt, False)
        dw = torch.empty(1, K, N, device="cuda")
        ops.moe_grouped_product_dw(x, dy, None, dw, ws)
        check_dw(x, dy, off, dw, "f32")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_non_finite_values_stay_in_their_rows(dt):
    """A NaN or an infinity in a row reaches that row's results and its expert's weight gradient alone;
    so do those in an expert's weights."""
    g = gen(2)
    t = DT[dt]
    K, N, counts = 96, 72, [100, 30, 61]
    off = offsets_of(counts)
    x, dy, w = randn(g, 191, K, dtype=t), randn(g, 191, N, dtype=t), randn(g, 3, K, N, dtype=t)
    x[99, 3] = float("nan")
    x[100, 5] = float("inf")
    w[2, 7, 9] = float("nan")
    ws = workspace(191, K, N, 3)
    out, dw = torch.empty(191, N, dtype=t, device="cuda"), torch.empty(3, K, N, dtype=t, device="cuda")
    ops.moe_grouped_product(x, w, off, out, ws)
    bad = ~torch.isfinite(out)
    assert bool(bad[99].all()) and bool(bad[100].all()) and bool(bad[130:, 9].all())
    bad[99] = bad[100] = False
    bad[130:, 9] = False
    assert not bool(bad.any())
    ops.moe_grouped_product_dw(x, dy, off, dw, ws)
    bad = ~torch.isfinite(dw)
    assert bool(bad[0, 3].all()) and bool(bad[1, 5].all())
    bad[0, 3] = bad[1, 5] = False
    assert not bool(bad.any())


def test_fp32_values_over_their_range():
    """Rows and weights of very different sizes, the largest values (which the nearest 16-bit value is past)
    and an infinity, which stays in its row."""
    g = gen(9)
    K, N, n = 70, 50, 40
    x, w = randn(g, n, K), randn(g, 1, K, N)
    x *= torch.exp2(torch.randint(-60, 61, (n, K), generator=g, device="cuda").float())
    w *= torch.exp2(torch.randint(-30, 31, (1, K, N), generator=g, device="cuda").float())
    x[0] = torch.finfo(torch.float32).max
    x[1] = -torch.finfo(torch.float32).max
    w[0, 0] *= 2.0 ** -40
    x[0:2, 1:] = 0
    out, ws = torch.empty(n, N, device="cuda"), workspace(n, K, N, 1)
    off = torch.tensor([0, n])
    ops.moe_grouped_product(x, w, None, out, ws)
    check_rows(x, w, off, out, "f32", False)
    x[3, 4] = float("inf")
    ops.moe_grouped_product(x, w, None, out, ws)
    assert not bool(torch.isfinite(out[3]).any())
    out[3], x[3] = 0, 0
    check_rows(x, w, off, out, "f32", False)


def test_fp32_products_of_two_values():
    """A value's three parts leave out at most 2^-24 + 2^-34 of a product; its small parts' five sums truncate
    (each 2^-23 of less than 2^-7 of it), and the sum is rounded once (2^-24)."""
    g = gen(9)
    hard = torch.tensor([1.0, 1.0 + 2.0 ** -8 + 2.0 ** -17 + 2.0 ** -23, 1.0 + 2.0 ** -7 - 2.0 ** -16 + 2.0 ** -23,
                         2.0 - 2.0 ** -23, 1.0 + 2.0 ** -7 - 2.0 ** -23, 1.0 + 2.0 ** -8 - 2.0 ** -17 - 2.0 ** -23], device="cuda")
    x = torch.cat((hard, -hard, randn(g, 700))).reshape(-1, 1)
    w = torch.cat((hard, randn(g, 506))).reshape(1, 1, -1)
    R, N = x.shape[0], w.shape[2]
    out = torch.empty(R, N, device="cuda")
    ops.moe_grouped_product(x, w, offsets_of([R]), out, workspace(R, 1, N, 1))
    want = x.double() @ w[0].double()
    bound = 2.0 ** -23 + 2.0 ** -34 + 5 * 2.0 ** -30
    assert bool(((out.double() - want).abs() <= bound * want.abs()).all())


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_no_rows(dt):
    t = DT[dt]
    K, N = 64, 48
    off = offsets_of([0, 0])
    w = torch.ones(2, K, N, dtype=t, device="cuda")
    ws = workspace(0, K, N, 2)
    ops.moe_grouped_product(torch.empty(0, K, dtype=t, device="cuda"), w, off, torch.empty(0, N, dtype=t, device="cuda"), ws)
    assert B.moe_read_status(ws) == 0
    dw = torch.full((2, K, N), MARK, dtype=t, device="cuda")
    args = torch.empty(0, K, dtype=t, device="cuda"), torch.empty(0, N, dtype=t, device="cuda"), off, dw, ws
    ops.moe_grouped_product_dw(*args, accumulate=True)
    assert bool((dw == MARK).all())
    ops.moe_grouped_product_dw(*args)
    assert not bool(dw.any())


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_gradients_against_differences(dt):
    """<dout, out(x + h v) - out(x - h v)> / 2h against <dx, v>: the product is linear, so only roundings
    count.  In fp32 results the outputs are off by K 2^-23 of their magnitudes' sums."""
    g = gen(3)
    t = DT[dt]
    K, N, counts = 128, 64, [20, 45]
    off = offsets_of(counts)
    # values that both steps hold exactly: multiples of 1/4 below 8
    def quarter(*s):
        return (torch.randint(-16, 17, s, generator=g, device="cuda") / 4.0).to(t)

    x, w, v, dout = quarter(65, K), quarter(2, K, N), quarter(65, K), quarter(65, N)
    vw = quarter(2, K, N)
    ws = workspace(65, K, N, 2)

    def f(xx, ww):
        out = torch.empty(65, N, device="cuda")
        ops.moe_grouped_product(xx, ww, off, out, ws)
        return (out.double() * dout.double()).sum()

    dx, dw = torch.empty(65, K, device="cuda"), torch.empty(2, K, N, device="cuda")
    ops.moe_grouped_product(dout, w, off, dx, ws, transposed=True)
    ops.moe_grouped_product_dw(x, dout, off, dw, ws)
    # every product and sum is a multiple of 1/16 below 2^16: exact in fp32
    assert ((f(x + v, w) - f(x - v, w)) / 2).item() == (dx.double() * v.double()).sum().item()
    assert ((f(x, w + vw) - f(x, w - vw)) / 2).item() == (dw.double() * vw.double()).sum().item()


@pytest.mark.parametrize("dt,K,N", [("bf16", 2048, 512), ("f16", 333, 257), ("f32", 96, 200)])
def test_same_bits_each_run_and_on_another_stream(dt, K, N):
    g = gen(4)
    t = DT[dt]
    counts = [1, 300, 0, 128, 77]
    off = offsets_of(counts)
    n = sum(counts)
    x, dy, w = randn(g, n, K, dtype=t), randn(g, n, N, dtype=t), randn(g, 5, K, N, dtype=t)

    def both(stream=None):
        ws = workspace(n, K, N, 5)
        out, dw = torch.empty(n, N, dtype=t, device="cuda"), torch.empty(5, K, N, dtype=t, device="cuda")
        ops.moe_grouped_product(x, w, off, out, ws, stream=stream)
        ops.moe_grouped_product_dw(x, dy, off, dw, ws, stream=stream)
        return out, dw

    first = both()
    torch.cuda.synchronize()
    for _ in range(3):
        for a, b in zip(first, both()):
            assert torch.equal(a, b)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = both()
    given = both(s)
    torch.cuda.synchronize()
    for a, b, c in zip(first, other, given):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_captured_calls_follow_their_offsets():
    """A captured chain replayed with other rows and offsets of the same sizes."""
    g = gen(6)
    K, N, n = 256, 384, 500
    bf = torch.bfloat16
    x, dy, w = randn(g, n, K, dtype=bf), randn(g, n, N, dtype=bf), randn(g, 3, K, N, dtype=bf, std=K ** -0.5)
    off = offsets_of([100, 300, 100])
    out, dw = torch.empty(n, N, dtype=bf, device="cuda"), torch.empty(3, K, N, device="cuda")
    ws = workspace(n, K, N, 3)

    def both():
        ops.moe_grouped_product(x, w, off, out, ws)
        ops.moe_grouped_product_dw(x, dy, off, dw, ws)

    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for counts in ([100, 300, 100], [0, 500, 0], [490, 1, 0], [2, 130, 368]):
        off.copy_(offsets_of(counts))
        x.copy_(randn(g, n, K, dtype=bf))
        out.fill_(MARK)
        graph.replay()
        torch.cuda.synchronize()
        check_rows(x, w, off, out, "bf16", False)
        check_dw(x, dy, off, dw, "f32")
    assert B.moe_read_status(ws) == 0


def test_two_streams_at_once():
    """Calls that overlap, a workspace each."""
    g = gen(8)
    K, N, n = 512, 768, 600
    bf = torch.bfloat16
    x, w = randn(g, n, K, dtype=bf), randn(g, 2, K, N, dtype=bf, std=K ** -0.5)
    offs = [offsets_of([200, 400]), offsets_of([600, 0])]
    outs = [torch.empty(n, N, dtype=bf, device="cuda") for _ in offs]
    wss = [workspace(n, K, N, 2) for _ in offs]
    streams = [torch.cuda.Stream() for _ in offs]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, o, y, ws in zip(streams, offs, outs, wss):
            ops.moe_grouped_product(x, w, o, y, ws, stream=s)
    torch.cuda.synchronize()
    for o, y, ws in zip(offs, outs, wss):
        check_rows(x, w, o, y, "bf16", False)
        assert B.moe_read_status(ws) == 0


def test_rows_past_32_bits_of_elements():
    """Results and rows whose elements lie past 2^32: the last expert's, at the end."""
    n, K, N = 150_000, 16, 29_000                 # out: 4.35e9 elements
    free = torch.cuda.mem_get_info()[0]
    if free < 24e9:
        pytest.skip("needs 24 GB")
    g = gen(7)
    bf = torch.bfloat16
    x, w = randn(g, n, K, dtype=bf), randn(g, 2, K, N, dtype=bf)
    off = offsets_of([n - 40, 40])
    out = torch.empty(n, N, dtype=bf, device="cuda")
    ws = workspace(n, K, N, 2)
    ops.moe_grouped_product(x, w, off, out, ws)
    for r in (slice(0, 10), slice(n - 60, n - 40), slice(n - 40, n)):
        a, b = x[r].double(), w[0 if r.start < n - 40 else 1].double()
        close(out[r], a @ b, "bf16", K * 2.0 ** -23 * (a.abs() @ b.abs()))
    # dy is out: its last rows through the gradients
    dx, dw = torch.empty(n, K, device="cuda"), torch.empty(2, K, N, device="cuda")
    ops.moe_grouped_product(out, w, off, dx, ws, transposed=True)
    a, b = out[n - 40:].double(), w[1].double().t()
    close(dx[n - 40:], a @ b, "f32", N * 2.0 ** -23 * (a.abs() @ b.abs()))
    ops.moe_grouped_product_dw(x, out, off, dw, ws)
    a, b = x[n - 40:].double().t(), out[n - 40:].double()
    close(dw[1], a @ b, "f32", 40 * 2.0 ** -23 * (a.abs() @ b.abs()))
