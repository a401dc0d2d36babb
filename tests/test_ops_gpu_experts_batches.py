"""The example's experts with batches of fewer rows than they were made for: the bits of experts made for each."""
import importlib.util
import os

import pytest
import torch

from ops_util import gen, randn

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ffn(cuda_lib):
    spec = importlib.util.spec_from_file_location("expert_ffn", os.path.join(ROOT, "examples", "expert_ffn.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("keep_rows", [True, False])
@pytest.mark.parametrize("d,f", [(1024, 264), (131, 67)])
def test_batches_of_fewer_rows(ffn, d, f, keep_rows):
    E, k, most = 4, 2, 300
    g = gen(d)
    W1 = randn(g, E, d, 2 * f, dtype=torch.bfloat16, std=d ** -0.5)
    W2 = randn(g, E, f, d, dtype=torch.bfloat16, std=f ** -0.5)
    norm_w, norm_b = randn(g, d, dtype=torch.bfloat16, mean=1.0), randn(g, d, dtype=torch.bfloat16)
    m = ffn.SwiGLUExperts(W1, W2, most * k, keep_rows)
    for T in (most, 3, 1, 170, 40):
        x, dout = randn(g, T, d, dtype=torch.bfloat16), randn(g, T, d, dtype=torch.bfloat16)
        ids = torch.rand(T, E, generator=g, device="cuda").topk(k).indices.to(torch.int32).reshape(-1)
        weights = torch.softmax(randn(g, T, k), 1)
        alone = ffn.SwiGLUExperts(W1, W2, T * k, keep_rows)
        got = []
        for e in (m, alone):
            e.reset()
            out, grads = ffn.train_step(x, norm_w, norm_b, ids, weights, E, e.forward, e.backward, dout)
            got.append([out, *(grads[n] for n in sorted(grads)), e.dW1.clone(), e.dW2.clone()])
            assert e.status() == 0
        assert all(torch.equal(a, b) for a, b in zip(*got)), T
