"""The products' workspace: one allocated for the most rows serves every call of fewer."""
import pytest
import torch

from ops_util import DT, close

INV, SMALL = 1, 3
P = 1 << 20  # a 128-byte aligned address that is never read
ROWS = [0, 1, 2, 7, 8, 63, 100, 129, 512, 1000, 1024, 4096, 5000, 16384, 20000, 100_000, 1 << 20, 1 << 25]
SIZES = [(2048, 1024, 8), (2048, 512, 8), (7168, 256, 1), (7168, 4096, 32), (1024, 1024, 1), (6373, 84, 1), (960, 961, 2),
         (64, 64, 1024), (128, 16, 3), (1 << 15, 3, 1), (1, 1, 1), (4097, 129, 40)]


@pytest.fixture(scope="module")
def O():
    from mixture_experts_layer_stable_gb300 import build, ops
    build.build()
    ops.lib()
    return ops


@pytest.mark.parametrize("K,N,G", SIZES)
def test_size_grows_with_the_rows_and_serves_fewer(O, K, N, G):
    L = O.lib()
    sizes = [O.moe_grouped_product_workspace_bytes(r, K, N, G) for r in ROWS]
    assert sizes == sorted(sizes) and sizes[0] >= 128 and sizes[-1] <= 128 + 160 * 256 * 128 * 4
    for i, most in enumerate(sizes):
        for r in ROWS[1:i + 1]:
            # a missing operand is refused behind the size of the workspace, before any launch
            for t, k, n in ((0, K, N), (1, N, K)):
                assert L.moe_grouped_product(1, 1, r, k, n, G, P, None, k, P, t, P, n, P, most, None) == INV, (r, ROWS[i])
            assert L.moe_grouped_product_dw(1, 1, r, K, N, G, P, None, K, P, N, P, 0, P, most, None) == INV, (r, ROWS[i])
    assert L.moe_grouped_product(1, 1, 4, K, N, G, P, None, K, P, 0, P, N, P, 127, None) == SMALL
    assert L.moe_grouped_product_dw(1, 1, 4, K, N, G, P, None, K, P, N, P, 0, P, 127, None) == SMALL


@pytest.mark.gpu
@pytest.mark.parametrize("dt,pad", [("bf16", 0), ("bf16", 1), ("f32", 0)])
def test_one_workspace_for_every_batch(O, cuda_lib, dt, pad):
    """Batches of fewer rows than the workspace was made for, in parts and whole, right behind one another."""
    K, N, G, most = 2048, 520 + pad, 4, 8192
    g = torch.Generator(device="cuda").manual_seed(1)
    x, dy, w = (torch.randn(*s, generator=g, device="cuda").to(DT[dt]) for s in ((most, K + pad), (most, N), (G, K, N)))
    x = x[:, :K]
    ws = torch.full((O.moe_grouped_product_workspace_bytes(most, K, N, G),), 255, dtype=torch.uint8, device="cuda")
    calls = []
    for r in (most, 8, 1, 700, 4000, 100, 3):
        o = [0, r // 2, r // 2, r - r // 8, r]
        off = torch.tensor(o, dtype=torch.int32, device="cuda")
        out, dx = torch.empty(r, N, device="cuda"), torch.empty(r, K, device="cuda")
        dw = torch.empty(G, K, N, device="cuda")
        O.moe_grouped_product(x[:r], w, off, out, ws)
        O.moe_grouped_product(dy[:r], w, off, dx, ws, transposed=True)
        O.moe_grouped_product_dw(x[:r], dy[:r], off, dw, ws)
        calls.append((o, out, dx, dw))
    for o, out, dx, dw in calls:
        for e in range(G):
            s = slice(o[e], o[e + 1])
            a, b, c = x[s].double(), dy[s].double(), w[e].double()
            close(out[s], a @ c, "f32", K * 2.0 ** -23 * (a.abs() @ c.abs()))
            close(dx[s], b @ c.t(), "f32", N * 2.0 ** -23 * (b.abs() @ c.t().abs()))
            close(dw[e], a.t() @ b, "f32", (s.stop - s.start + 1) * 2.0 ** -23 * (a.t().abs() @ b.abs()))
