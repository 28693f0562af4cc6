"""Argument checks of the operators around the table step, on the host (no GPU): everything here is
refused, or is a size query, before anything would be enqueued; the pointers are never dereferenced."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def so():
    from lazy_optimizers_embedding_gb300 import build
    build.build()
    from lazy_optimizers_embedding_gb300 import binding
    return binding


P = ctypes.c_void_p(256)
WS = 1 << 40


def test_layer_norm_refusals(so):
    f = so.LIB.sparse_layer_norm

    def code(x=P, xt=0, r=8, c=16, idx=None, n=8, eps=1e-5, y=P, yt=0, err=P):
        return f(x, xt, r, c, idx, n, P, P, eps, y, yt, P, P, err, None)

    bad = [dict(xt=2), dict(yt=-1), dict(xt=1, yt=0), dict(r=-1), dict(c=0), dict(c=1 << 31), dict(n=-1), dict(n=9),
           dict(eps=-1.0), dict(eps=float("inf")), dict(eps=float("nan")), dict(x=None), dict(y=None), dict(err=None),
           dict(r=1 << 62, idx=P)]
    for b in bad:
        assert code(**b) == so.ERR_INVALID_ARG, b
    assert code(n=0) == so.OK and code(n=0, x=None, y=None) == so.OK


def test_layer_norm_grad_refusals(so):
    f = so.LIB.sparse_layer_norm_grad
    need = so.sparse_layer_norm_workspace_size(8, 16)
    assert need >= 2 * 16 * 4

    def code(dy=P, x=P, mean=P, rstd=P, dx=P, dgamma=P, dbeta=P, ws=P, size=need, err=P, n=8):
        return f(dy, 0, x, 0, 8, 16, None, n, P, mean, rstd, dx, dgamma, dbeta, ws, size, err, None)

    for name in ("dy", "x", "mean", "rstd", "dx", "err"):
        assert code(**{name: None}) == so.ERR_INVALID_ARG, name
    for b in (dict(ws=None), dict(size=need - 1), dict(ws=ctypes.c_void_p(255))):
        assert code(**b) == so.ERR_WORKSPACE, b


def test_workspaces_grow_with_what_they_hold(so):
    assert so.sparse_layer_norm_workspace_size(0, 8) >= 0
    assert so.sparse_layer_norm_workspace_size(1 << 20, 128) <= 1024 * 2 * 128 * 4
    # a few thousand slots need none, so only an array with an address; millions need a count for every
    # expert and tile
    assert so.sparse_expert_workspace_size(100, 2, 64) == 256
    assert 0 < so.sparse_expert_workspace_size(1 << 20, 8, 64) <= 64 * 4 * 513
    one, three = (so.sparse_muon_workspace_size(2, 300, 500, p) for p in (1, 3))
    assert 0 < one < three
    # X twice in two parts, A and B in one or two
    assert three <= 2 * (4 * 300 * 512 + 4 * 300 * 320) * 2 + 65536
    assert so.sparse_muon_workspace_size(0, 300, 500, 3) == 0


def test_expert_refusals(so):
    L = so.LIB

    def sort(expert=P, n=8, k=2, e=4, offsets=P, pos=P, ws=P, size=WS, err=P):
        return L.sparse_expert_sort(expert, n, k, e, offsets, None, pos, ws, size, err, None)

    for b in (dict(n=-1), dict(k=0), dict(n=1 << 31), dict(e=0), dict(e=1025), dict(expert=None), dict(offsets=None),
              dict(pos=None), dict(err=None)):
        assert sort(**b) == so.ERR_INVALID_ARG, b
    assert sort(ws=None) == so.ERR_WORKSPACE and sort(ws=ctypes.c_void_p(3)) == so.ERR_WORKSPACE
    assert sort(n=1 << 20, size=16) == so.ERR_WORKSPACE

    def combine(ys=P, t=0, n=8, k=2, c=16, pos=P, y=P, err=P):
        return L.sparse_expert_combine(ys, t, n, k, c, pos, None, y, err, None)

    for b in (dict(ys=None), dict(t=5), dict(c=0), dict(c=(1 << 30) + 1), dict(pos=None), dict(y=None), dict(err=None)):
        assert combine(**b) == so.ERR_INVALID_ARG, b
    assert combine(n=0) == so.OK
    assert L.sparse_expert_dispatch(P, 0, 8, 2, 16, P, None, 4, P, P, None) == so.ERR_INVALID_ARG
    assert L.sparse_expert_combine_grad(P, P, 0, 8, 2, 16, P, P, 1025, None, P, None, P, None) == so.ERR_INVALID_ARG


def test_newton_schulz_refusals(so):
    good = dict(a=3.4445, b=-4.7750, c=2.0315, eps=1e-7, steps=5, products=3)

    def code(u=P, t=0, batch=1, r=8, cols=8, out=P, ws=P, size=WS, err=P, **cfg):
        ns = so.NsConfig(**{**good, **cfg})
        return so.LIB.sparse_orthogonalize(u, t, batch, r, cols, ns, out, 0, ws, size, err, None)

    # coefficients whose X, A, B or a I + B leave the range that f16 operands hold
    for b in (dict(a=4.5, b=0.0, c=0.0, steps=1), dict(a=1.0, b=-4.0, c=0.0, steps=1), dict(a=3.95, b=-4.0, c=1.0, steps=1),
              dict(steps=0), dict(steps=65), dict(products=2), dict(eps=-1e-9), dict(u=None), dict(out=None), dict(t=3),
              dict(r=0), dict(cols=(1 << 20) + 1), dict(batch=1 << 20, r=1 << 10, cols=1 << 10), dict(err=None)):
        assert code(**b) == so.ERR_INVALID_ARG, b
    assert code(ws=None) == so.ERR_WORKSPACE and code(size=100) == so.ERR_WORKSPACE
    assert code(batch=0, u=None, out=None, ws=None) == so.OK


def test_muon_step_refusals(so):
    ns = so.NsConfig(a=3.4445, b=-4.7750, c=2.0315, eps=1e-7, steps=5, products=1)
    good = dict(lr=0.02, momentum=0.95, weight_decay=0.1, scale=1.0, nesterov=1, ns=ns)

    def code(w=P, buf=P, g=P, t=1, ws=P, size=WS, err=P, **cfg):
        return so.LIB.sparse_muon_step(w, buf, g, t, 1, 8, 8, so.MuonConfig(**{**good, **cfg}), ws, size, err, None)

    nan = float("nan")
    for b in (dict(w=None), dict(buf=None), dict(g=None), dict(t=2), dict(err=None), dict(lr=nan), dict(momentum=-0.5),
              dict(weight_decay=-0.1), dict(scale=nan)):
        assert code(**b) == so.ERR_INVALID_ARG, b
    assert code(ws=None) == so.ERR_WORKSPACE
