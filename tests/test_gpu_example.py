"""The example model learns: every operator and both optimizers at work in one training step."""
import importlib.util
import os

import pytest

from conftest import ROOT

pytestmark = pytest.mark.gpu


def _example():
    spec = importlib.util.spec_from_file_location("table_and_experts", os.path.join(ROOT, "examples", "table_and_experts.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_the_example_learns(cuda_lib):
    losses = _example().main(60)
    # at the start the loss is about 2 (a unit normal row against a unit normal target)
    assert 1.5 < losses[0] < 4.0
    assert sum(losses[-5:]) / 5 < 0.7 * losses[0]


def test_its_gradients_are_those_of_autograd(cuda_lib):
    """One step's gradients of the table and of the experts' matrices against torch's own, in 64 bits."""
    import torch
    ex = _example()
    model = ex.Model(seed=3)
    tokens = ex.lookups(0)
    table, up, down = (t.detach().double().clone().requires_grad_() for t in (model.table, model.up, model.down))
    y = torch.nn.functional.layer_norm(table[tokens], (ex.WIDTH,), model.gamma.double(), model.beta.double(), ex.EPS)
    score, picked = (y @ model.router.double()).topk(ex.PICKED, dim=1)
    weights = torch.softmax(score, 1)
    out = y
    for j in range(ex.PICKED):
        for e in range(ex.EXPERTS):
            rows = (picked[:, j] == e).nonzero()[:, 0]
            mixed = torch.relu(y[rows] @ up[e]) @ down[e] * weights[rows, j, None]
            out = out.index_add(0, rows, mixed)
    off = out - model.target.double()[tokens]
    (off * off).mean().backward()

    captured = {}
    so = ex.so

    class Spy:
        def __getattr__(self, name):
            return getattr(so, name)

        def sparse_muon_step(self, w, buf, g, *args):
            captured[tuple(g.shape)] = g.clone()
            return so.sparse_muon_step(w, buf, g, *args)

    ex.so = Spy()
    model.step(tokens)
    torch.cuda.synchronize()
    assert int(model.err.item()) == 0
    got = torch.zeros_like(table).index_add(0, tokens, model.dx.double())
    # fp32 all the way, sums of at most a few thousand terms: 1e-4 of the gradient's norm
    for mine, ref in ((got, table.grad), (captured[tuple(up.shape)], up.grad), (captured[tuple(down.shape)], down.grad)):
        assert float((mine.double() - ref).norm()) <= 1e-4 * float(ref.norm())
