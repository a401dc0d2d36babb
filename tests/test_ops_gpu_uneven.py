"""Products of very uneven experts on the GPU: with one expert over four times the average of those that have rows,
units are taken from both ends of their order in turns.  Bounds as in test_ops_gpu_product.py."""
import pytest
import torch

from mixture_experts_layer_stable_gb300 import binding as B
from mixture_experts_layer_stable_gb300 import ops

from ops_util import DT, close, empty_strided, gen, randn, strided

pytestmark = pytest.mark.gpu
MARK = 7.0


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_lib):
    yield


HEAVY = [3, 0, 1500, 1, 17, 0, 5, 2, 9, 33]                        # seven light experts, one heavy
LIGHT = [1, 0, 0, 2, 1, 200, 1, 0, 3, 1, 1, 0]                     # below 64 rows an expert: no pairs
MANY = [1 if i % 3 else 0 for i in range(150)] + [900] + [2] * 20  # the heavy one behind the light ones
FIRST = [2600] + [5, 0, 7, 130, 1, 0, 64]                          # and in front of them


@pytest.mark.parametrize("dt,odt", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f32", "f32")])
@pytest.mark.parametrize("counts,K,N,pad,shift", [
    (HEAVY, 264, 392, 0, 0),            # pairs (aligned, over 128 columns, 64 rows an expert)
    (HEAVY, 136, 1032, 8, 0),           # an odd number of units a tile
    (FIRST, 392, 264, 0, 0),
    (LIGHT, 264, 392, 0, 0),            # single blocks
    (LIGHT, 72, 1160, 0, 8),
    (MANY, 64, 520, 0, 0),
    (HEAVY, 129, 255, 0, 0),            # loading warps
    (LIGHT, 257, 131, 3, 1),
    (FIRST, 65, 387, 1, 0),
    (LIGHT, 4096, 24, 0, 0),            # contractions in parts
    (FIRST, 1100, 136, 0, 0),
    ([1] * 9 + [3000], 24, 40, 0, 0),
])
def test_units_from_both_ends(dt, odt, counts, K, N, pad, shift):
    some = [c for c in counts if c]
    assert max(some) > 4 * (sum(some) // len(some))
    g = gen(K + N)
    t, ot = DT[dt], DT[odt]
    first, behind = 2, 5
    off = torch.tensor([first] + counts, dtype=torch.int32).cumsum(0).to(torch.int32).cuda()
    o = off.tolist()
    n, G = o[-1] + behind, len(counts)
    x, dy = strided(g, n, K, t, pad, shift), strided(g, n, N, t, pad, shift)
    for r in (x, dy):
        r[:first] = float("nan")
        r[o[-1]:] = float("nan")
    w = randn(g, G * K * N + shift, dtype=t, std=K ** -0.5)[shift:].reshape(G, K, N)
    out, dx = empty_strided(n, N, ot, pad, shift, MARK), empty_strided(n, K, ot, pad, shift, MARK)
    dw = torch.full((G, K, N), MARK, dtype=ot, device="cuda")
    ws = torch.full((ops.moe_grouped_product_workspace_bytes(n, K, N, G),), 255, dtype=torch.uint8, device="cuda")
    ops.moe_grouped_product(x, w, off, out, ws)
    ops.moe_grouped_product(dy, w, off, dx, ws, transposed=True)
    ops.moe_grouped_product_dw(x, dy, off, dw, ws)
    for e in range(G):
        s = slice(o[e], o[e + 1])
        a, b, c = x[s].double(), dy[s].double(), w[e].double()
        close(out[s], a @ c, odt, K * 2.0 ** -23 * (a.abs() @ c.abs()), f"rows of {e}")
        close(dx[s], b @ c.t(), odt, N * 2.0 ** -23 * (b.abs() @ c.t().abs()), f"their gradient, {e}")
        close(dw[e], a.t() @ b, odt, (s.stop - s.start + 1) * 2.0 ** -23 * (a.t().abs() @ b.abs()), f"weights of {e}")
    for r in (out, dx):
        assert bool((r[:first] == MARK).all()) and bool((r[o[-1]:] == MARK).all())
    more = dw.clone()
    ops.moe_grouped_product_dw(x, dy, off, more, ws, accumulate=True)
    close(more, 2 * dw.double(), odt, 2.0 ** -22 * (n + 1) * dw.double().abs().amax())
    assert B.moe_read_status(ws) == 0
