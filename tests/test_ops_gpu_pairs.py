"""Weight gradients by CTA pairs on the GPU whose contraction ends inside a stage, beside rows that are NaN: the
zeros that each block of a pair puts behind an expert's last row have to be there for every unit under way."""
import pytest
import torch

from mixture_experts_layer_stable_gb300 import binding as B
from mixture_experts_layer_stable_gb300 import ops

from ops_util import DT, close, gen, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_lib):
    yield


def experts(counts, K, N, dt, odt, seed, apart=0):
    """Gradients of experts with `apart` NaN rows behind each one's rows: every second expert of the call is NaN."""
    g = gen(seed)
    t = DT[dt]
    sizes = [c for n in counts for c in ((n, apart) if apart else (n,))]
    off = torch.tensor([0] + sizes, dtype=torch.int32).cumsum(0).to(torch.int32).cuda()
    n, G = sum(sizes), len(sizes)
    x, dy = randn(g, n, K, dtype=t), randn(g, n, N, dtype=t)
    o = off.tolist()
    if apart:
        for e in range(1, G, 2):
            x[o[e]:o[e + 1]] = float("nan")
            dy[o[e]:o[e + 1]] = float("nan")
    dw = torch.empty(G, K, N, dtype=DT[odt], device="cuda")
    ws = torch.full((ops.moe_grouped_product_workspace_bytes(n, K, N, G),), 255, dtype=torch.uint8, device="cuda")
    return x, dy, off, dw, ws, o


@pytest.mark.parametrize("dt,odt", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32")])
@pytest.mark.parametrize("counts,K,N", [
    ([65, 127, 190, 3, 77], 192, 136), ([129] * 40, 520, 264), ([193, 71, 255, 1000, 8] * 8, 264, 392),
    ([1501, 1, 2049, 700], 776, 1032), ([64 * i + i % 16 for i in range(1, 17)] * 3, 136, 256)])
def test_ends_beside_nan_rows(dt, odt, counts, K, N):
    """N over 128 and 64 rows an expert on average take pairs; lengths that leave every rest of 16."""
    x, dy, off, dw, ws, o = experts(counts, K, N, dt, odt, K + N, apart=max(1, 128 - min(counts)))
    assert o[-1] >= 64 * (len(o) - 1)
    ops.moe_grouped_product_dw(x, dy, off, dw, ws)
    first = dw.clone()
    for e in range(0, len(o) - 1, 2):
        a, b = x[o[e]:o[e + 1]].double().t(), dy[o[e]:o[e + 1]].double()
        close(dw[e], a @ b, odt, (o[e + 1] - o[e] + 1) * 2.0 ** -23 * (a.abs() @ b.abs()), f"expert {e}")
    for _ in range(10):
        dw.fill_(7)
        ops.moe_grouped_product_dw(x, dy, off, dw, ws)
        assert torch.equal(dw[0::2], first[0::2])
    assert B.moe_read_status(ws) == 0


@pytest.mark.parametrize("odt", ["bf16", "f32"])
def test_ends_with_stores_under_way(odt):
    """Many units of one short stage each, so that ends, copies and stores of several are under way, beside the
    next expert's infinities."""
    counts = [33, 95] * 60
    x, dy, off, dw, ws, o = experts(counts, 1032, 1288, "bf16", odt, 9)
    x[o[1]:] *= 2.0 ** 100
    dy[o[1]:] *= 2.0 ** 100                       # products past fp32: infinities if one gets in
    ops.moe_grouped_product_dw(x, dy, off, dw, ws)
    a, b = x[:33].double().t(), dy[:33].double()
    close(dw[0], a @ b, odt, 34 * 2.0 ** -23 * (a.abs() @ b.abs()))
    first = dw.clone()
    for _ in range(20):
        ops.moe_grouped_product_dw(x, dy, off, dw, ws)
        assert torch.equal(dw.view(torch.int16), first.view(torch.int16))
    assert B.moe_read_status(ws) == 0
