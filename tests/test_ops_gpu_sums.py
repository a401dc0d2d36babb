"""The products' long sums on the GPU: what an accumulator that truncates would lose.

The tensor cores add 16 products at a time to an fp32 accumulator and cut the sum off, losing up to one last
place (2^-23) of it, half of one on average.  An accumulator takes 512 of the contraction (32 additions), 1024
(64) where results have 16 bits; accumulators are added rounded to nearest (2^-24 each).

Terms of one sign: no sum is larger than the result, so additions lose at most (64 + 1) 2^-23 of the result and
the c accumulators' sums at most c 2^-24.
Terms of random signs: after i of n additions the sum is of the order sqrt(i / n) of the result, so a chunk
of m additions loses on average 2^-24 sum_i sqrt(i / n) = 2^-24 (2/3) m sqrt(m / n), and the n / m chunks, whose
signs are independent, sqrt(n / m) times that: 2^-24 (2/3) m of the results' norm, whatever n."""
import pytest
import torch

from mixture_experts_layer_stable_gb300 import binding as B
from mixture_experts_layer_stable_gb300 import ops

from ops_util import DT, close, gen, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_lib):
    yield


def workspace(rows, K, N, G):
    return torch.full((ops.moe_grouped_product_workspace_bytes(rows, K, N, G),), 255, dtype=torch.uint8, device="cuda")


def same_sign(n):
    """Relative loss of n terms of one sign in accumulators of 1024 at most, before the last rounding."""
    return 65 * 2.0 ** -23 + (n // 512 + 1) * 2.0 ** -24


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("K,N", [(256, 256), (136, 128), (255, 253)])
def test_weight_gradients_of_many_rows_of_one_sign(dt, K, N):
    """262144 rows of one of 160 experts (so many that the contraction is not cut into parts), by pairs, single
    blocks and loading warps; two more experts whose sums are short."""
    rows, G, long = 1 << 18, 160, 1 << 18
    g = gen(1)
    x = torch.rand(rows + 1030, K, generator=g, device="cuda").to(DT[dt])
    dy = (torch.rand(rows + 1030, N, generator=g, device="cuda") / 16).to(DT[dt])
    off = torch.full((G + 1,), rows + 1030, dtype=torch.int32, device="cuda")
    off[0:4] = torch.tensor([0, 5, long + 5, long + 1030])
    dw = torch.empty(G, K, N, dtype=DT[dt], device="cuda")
    ws = workspace(rows + 1030, K, N, G)
    ops.moe_grouped_product_dw(x, dy, off, dw, ws)
    o = off.tolist()
    for e in range(5):
        s = slice(o[e], o[e + 1])
        want = x[s].double().t() @ dy[s].double()
        close(dw[e], want, dt, same_sign(o[e + 1] - o[e]) * want, f"expert {e}")
    assert not bool(dw[5:].any()) and B.moe_read_status(ws) == 0


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("shift", [0, 1])
def test_long_rows_of_one_sign(dt, transposed, shift):
    """Rows of 65536 into more columns than leave parts, with both kinds of operands."""
    rows, K, N = 70, 65536 + shift, 10_240
    g = gen(2)
    x = torch.rand(rows, K, generator=g, device="cuda").to(DT[dt])
    w = torch.empty(1, *((N, K) if transposed else (K, N)), dtype=DT[dt], device="cuda")
    for part in w[0].split(4096):
        part.copy_(torch.rand(*part.shape, generator=g, device="cuda") / 256)
    out = torch.empty(rows, N, dtype=DT[dt], device="cuda")
    ws = workspace(rows, K, N, 1)
    ops.moe_grouped_product(x, w, None, out, ws, transposed=transposed)
    for c in (slice(0, 300), slice(N - 140, N)):
        want = x.double() @ (w[0, c].double().t() if transposed else w[0, :, c].double())
        close(out[:, c], want, dt, same_sign(K) * want)
    assert B.moe_read_status(ws) == 0


@pytest.mark.parametrize("dt,m", [("bf16", 32), ("f16", 32), ("f32", 16)])
@pytest.mark.parametrize("shift", [0, 1])
def test_fp32_sums_of_random_signs(dt, m, shift):
    """Sums of 4096 terms into fp32, all three forms, in the norm.  (m additions an accumulator; of fp32 operands
    the parts leave out 2^-24 of a product and the accumulators' sums 2^-24 each, which the norm takes as it
    takes independent errors: below 2^-23 together.)"""
    n, R, N = 4096, 1500, 2000 + shift
    g = gen(3)
    lim = 2.0 ** -24 * m * 2 / 3 + 2.0 ** -23
    x, w = randn(g, R, n + shift, dtype=DT[dt])[:, :n], randn(g, 1, n, N, dtype=DT[dt])
    out, ws = torch.empty(R, N, device="cuda"), workspace(R, n, N, 1)
    want = x.double() @ w[0].double()
    ops.moe_grouped_product(x, w, None, out, ws)
    assert (out.double() - want).norm() <= lim * want.norm()
    wt = w.transpose(1, 2).contiguous()
    ops.moe_grouped_product(x, wt, None, out, ws, transposed=True)
    assert (out.double() - want).norm() <= lim * want.norm()
    xt = torch.empty(n, R + shift, dtype=DT[dt], device="cuda")[:, :R]
    xt.copy_(x.t())
    dw, ws = torch.empty(1, R, N, device="cuda"), workspace(n, R, N, 1)
    ops.moe_grouped_product_dw(xt, w[0], None, dw, ws)
    assert (dw[0].double() - want).norm() <= lim * want.norm()


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("counts,K,N", [([1030, 3, 0, 2100, 1024, 1025, 64, 5000] * 12, 40, 133),
                                        ([2048, 1, 1500] * 40, 264, 72)])
def test_long_and_short_sums_in_turn(dt, counts, K, N):
    """Units of one and of several accumulators behind one another in a block: whole numbers whose sums are
    exact in fp32, so that a sum of the wrong unit shows, rounded once."""
    g = gen(4)
    n, G = sum(counts), len(counts)
    x = torch.randint(-3, 4, (n, K), generator=g, device="cuda").to(DT[dt])
    dy = torch.randint(-3, 4, (n, N), generator=g, device="cuda").to(DT[dt])
    off = torch.tensor([0] + counts, dtype=torch.int32).cumsum(0).to(torch.int32).cuda()
    dw, ws = torch.empty(G, K, N, dtype=DT[dt], device="cuda"), workspace(n, K, N, G)
    ops.moe_grouped_product_dw(x, dy, off, dw, ws)
    o = off.tolist()
    for e in range(G):
        s = slice(o[e], o[e + 1])
        assert torch.equal(dw[e], (x[s].double().t() @ dy[s].double()).to(DT[dt])), e
    assert B.moe_read_status(ws) == 0
