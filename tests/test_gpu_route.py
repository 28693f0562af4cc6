"""Routing against plain numpy in 64 bits: picks are equal; a weight is an exponential (2 ulp of its value and half a
step of its argument, which is at most some hundred here) over a sum of at most 1024 of them, in fp32:
(2 + 2 + 40 + |l| ) 2^-23 of it is allowed for, the gradients twice that of the terms' sizes."""
import numpy as np
import pytest

from gpu_harness import Guarded

pytestmark = pytest.mark.gpu

U = 2.0 ** -23


def _plain(logits, k, again):
    n, e = logits.shape
    expert = np.full((n, k), -1, np.int64)
    weights = np.zeros((n, k))
    p = np.zeros((n, e))
    for i in range(n):
        order = np.argsort(-logits[i], kind="stable")[:k]
        order = order[logits[i][order] > -np.inf]
        expert[i, :len(order)] = order
        if len(order) == 0:
            continue
        each = np.exp(logits[i] - logits[i].max())
        p[i] = each / each.sum()
        w = p[i][order]
        weights[i, :len(order)] = w / w.sum() if again else w
    return expert, weights, p


def _plain_grad(dw, expert, weights, p, again):
    d = np.zeros_like(p)
    for i in range(len(p)):
        live = expert[i] >= 0
        g, w = np.where(live, dw[i], 0.0), weights[i]
        s = (w * g).sum()
        if not again:
            d[i] = -p[i] * s
        for j in np.flatnonzero(live):
            d[i, expert[i, j]] = w[j] * (g[j] - s)
    return d


@pytest.mark.parametrize("again", [1, 0])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("n,e,k", [(1, 1, 1), (8, 64, 4), (300, 37, 3), (5, 1024, 32), (33, 1000, 8), (70, 256, 8),
                                   (65, 5, 5), (9, 32, 32), (2000, 8, 2), (40, 100, 7), (12, 513, 1), (7, 520, 9)])
def test_routing(cuda_lib, n, e, k, kind, again):
    import torch
    so = cuda_lib
    rng = np.random.default_rng(n * e + k)
    t = {"f32": torch.float32, "bf16": torch.bfloat16}[kind]
    x = rng.standard_normal((n, e)) * 3
    x[rng.random((n, e)) < 0.2] = -np.inf
    x[rng.random((n, e)) < 0.1] = 1.5                          # equals
    x[rng.random((n, e)) < 0.05] = 0.0
    x[rng.random((n, e)) < 0.05] = -0.0
    x[rng.random(n) < 0.1] = -np.inf
    G = Guarded(seed=e)
    logits, dlogits = G.empty((n, e), t), G.empty((n, e), t)
    logits.copy_(torch.from_numpy(x))
    expert, weights = G.array(np.full((n, k), 77, np.int64)), G.array(np.full((n, k), 7.0, np.float32))
    dw = rng.standard_normal((n, k)).astype(np.float32)
    err = G.error_word()
    so.check(so.sparse_expert_route(logits, n, e, k, again, expert, weights, err))
    ref, wref, p = _plain(logits.double().cpu().numpy(), k, again)
    dw[ref < 0] = np.nan                                       # not looked at
    so.check(so.sparse_expert_route_grad(G.array(dw), logits, n, e, k, again, expert, weights, dlogits, err))
    G.check("route")
    assert int(err.item()) == 0
    assert np.array_equal(expert.cpu().numpy(), ref)
    assert (np.abs(weights.double().cpu().numpy() - wref) <= 60 * U * wref).all()
    dw = np.where(ref < 0, 0.0, dw).astype(np.float64)
    d = _plain_grad(dw, ref, wref, p, again)
    size = np.abs(_plain_grad(np.abs(dw), ref, wref, p, again)) + 2 * p * np.abs(wref * dw).sum(1, keepdims=True)
    b = 2.0 ** -8 if kind == "bf16" else 0.0
    assert (np.abs(dlogits.double().cpu().numpy() - d) <= 120 * U * (size + np.abs(wref * dw).sum(1, keepdims=True)) + b * np.abs(d)).all()
