"""Products of rows with very wide strides on the GPU: a tile's rows lie 4 GiB and more apart.  Bounds as in
test_ops_gpu_product.py."""
import pytest
import torch

from mixture_experts_layer_stable_gb300 import binding as B
from mixture_experts_layer_stable_gb300 import ops

from ops_util import DT, close, gen, randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("ld,first", [((1 << 24) + 1, 0), ((1 << 24) + 1, 3), ((1 << 26) + 1, 0), (1 << 26, 8)])
def test_rows_far_apart(cuda_lib, dt, ld, first):
    """Rows and gradients in columns of one wide array, results in others: contractions of several whole stages
    and the end of one, over K and over the rows."""
    n, K, N, counts = 200, 520, 190, [1, 199]
    if torch.cuda.mem_get_info()[0] < 4.2 * n * ld * DT[dt].itemsize:
        ld = (ld >> 2) + (ld & 1)
    if torch.cuda.mem_get_info()[0] < 1.1 * n * ld * DT[dt].itemsize:
        pytest.skip("needs more memory")
    g = gen(1)
    buf = torch.empty(n * ld, dtype=DT[dt], device="cuda").reshape(n, ld)
    at, cols = first, []
    for d in (K, N, N, K):
        cols.append(buf[:, at:at + d])
        at += d + first
    x, dy, out, dx = cols
    x.copy_(randn(g, n, K))
    dy.copy_(randn(g, n, N))
    w = randn(g, 2, K, N, dtype=DT[dt])
    off = torch.tensor([0, 1, n], dtype=torch.int32, device="cuda")
    ws = torch.full((ops.moe_grouped_product_workspace_bytes(n, K, N, 2),), 255, dtype=torch.uint8, device="cuda")
    dw = torch.empty(2, K, N, dtype=DT[dt], device="cuda")
    ops.moe_grouped_product(x, w, off, out, ws)
    ops.moe_grouped_product(dy, w, off, dx, ws, transposed=True)
    ops.moe_grouped_product_dw(x, dy, off, dw, ws)
    for e, s in enumerate((slice(0, 1), slice(1, n))):
        a, b, c = x[s].double(), dy[s].double(), w[e].double()
        close(out[s], a @ c, dt, K * 2.0 ** -23 * (a.abs() @ c.abs()), "rows")
        close(dx[s], b @ c.t(), dt, N * 2.0 ** -23 * (b.abs() @ c.t().abs()), "their gradient")
        close(dw[e], a.t() @ b, dt, (n + 1) * 2.0 ** -23 * (a.t().abs() @ b.abs()), "weights' gradient")
    assert B.moe_read_status(ws) == 0


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("K,N", [(264, 136), (61, 45)])
@pytest.mark.parametrize("ld", [(1 << 62) + 1, 1 << 44, 1001])
def test_one_rows_stride_says_nothing(cuda_lib, dt, K, N, ld):
    g = gen(2)
    x, dy, w = randn(g, 1, K, dtype=DT[dt]), randn(g, 1, N, dtype=DT[dt]), randn(g, 1, K, N, dtype=DT[dt])
    out, dx, dw = torch.empty_like(dy), torch.empty_like(x), torch.empty_like(w)
    ws = torch.full((ops.moe_grouped_product_workspace_bytes(1, K, N, 1),), 255, dtype=torch.uint8, device="cuda")
    L, t, st = ops.lib(), {"f32": 0, "bf16": 1}[dt], torch.cuda.current_stream().cuda_stream
    at = [v.data_ptr() for v in (x, dy, w, out, dx, dw, ws)]
    assert L.moe_grouped_product(t, t, 1, K, N, 1, None, at[0], ld, at[2], 0, at[3], ld, at[6], ws.nbytes, st) == 0
    assert L.moe_grouped_product(t, t, 1, N, K, 1, None, at[1], ld, at[2], 1, at[4], ld, at[6], ws.nbytes, st) == 0
    assert L.moe_grouped_product_dw(t, t, 1, K, N, 1, None, at[0], ld, at[1], ld, at[5], 0, at[6], ws.nbytes, st) == 0
    a, b, c = x.double(), dy.double(), w[0].double()
    close(out, a @ c, dt, K * 2.0 ** -23 * (a.abs() @ c.abs()))
    close(dx, b @ c.t(), dt, N * 2.0 ** -23 * (b.abs() @ c.t().abs()))
    close(dw[0], a.t() @ b, dt, 2 * 2.0 ** -23 * (a.t().abs() @ b.abs()))
