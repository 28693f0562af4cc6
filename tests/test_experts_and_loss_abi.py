"""Argument checks of routing, the experts' products and the loss over a table's rows, on the host (no GPU): everything
here is refused, or is a size query, before anything would be enqueued; the pointers are never dereferenced."""
import ctypes

import pytest

P = ctypes.c_void_p(256)
WS = 1 << 45


@pytest.fixture(scope="module")
def so():
    from lazy_optimizers_embedding_gb300 import build
    build.build()
    from lazy_optimizers_embedding_gb300 import binding
    return binding


def test_route_refusals(so):
    def code(logits=P, t=0, n=8, e=16, k=4, expert=P, weights=P, err=P):
        return so.LIB.sparse_expert_route(logits, t, n, e, k, 1, expert, weights, err, None)

    for b in (dict(logits=None), dict(t=2), dict(t=-1), dict(n=-1), dict(e=0), dict(e=1025), dict(k=0), dict(k=17), dict(e=64, k=33),
              dict(expert=None), dict(weights=None), dict(err=None), dict(n=1 << 62)):
        assert code(**b) == so.ERR_INVALID_ARG, b
    assert code(n=0) == so.OK and code(n=0, logits=None, expert=None, weights=None) == so.OK

    def grad(dw=P, logits=P, t=0, n=8, e=16, k=4, again=1, expert=P, weights=P, out=P, err=P):
        return so.LIB.sparse_expert_route_grad(dw, logits, t, n, e, k, again, expert, weights, out, err, None)

    for b in (dict(dw=None), dict(logits=None, again=0), dict(expert=None), dict(weights=None), dict(out=None), dict(err=None), dict(k=0),
              dict(t=7), dict(e=1025)):
        assert grad(**b) == so.ERR_INVALID_ARG, b
    assert grad(n=0, logits=None) == so.OK


def test_matmul_refusals(so):
    def code(x=P, w=P, t=0, n=8, a=16, b=24, off=P, e=4, y=P, ws=P, size=WS, err=P):
        return so.LIB.sparse_expert_matmul(x, w, t, n, a, b, 0, off, e, y, ws, size, err, None)

    for b in (dict(x=None), dict(w=None), dict(t=2), dict(n=-1), dict(n=1 << 31), dict(a=0), dict(b=0), dict(a=(1 << 20) + 1),
              dict(b=(1 << 20) + 1), dict(off=None), dict(e=0), dict(e=1025), dict(y=None), dict(err=None),
              dict(n=1 << 30, a=1 << 10), dict(e=1024, a=1 << 14, b=1 << 14)):
        assert code(**b) == so.ERR_INVALID_ARG, b
    assert code(ws=None) == so.ERR_WORKSPACE and code(ws=ctypes.c_void_p(128)) == so.ERR_WORKSPACE
    assert code(size=255) == so.ERR_WORKSPACE
    assert code(n=0, x=None, w=None, off=None, y=None, ws=None) == so.OK

    def grad(x=P, dy=P, t=1, n=8, a=16, b=24, off=P, e=4, dw=P, dt=0, ws=P, size=WS, err=P):
        return so.LIB.sparse_expert_matmul_grad(x, dy, t, n, a, b, off, e, dw, dt, ws, size, err, None)

    for b in (dict(x=None), dict(dy=None), dict(t=3), dict(dt=2), dict(t=0, dt=1), dict(off=None), dict(dw=None), dict(err=None), dict(e=0),
              dict(a=-5), dict(n=0, dw=None)):
        assert grad(**b) == so.ERR_INVALID_ARG, b
    assert grad(ws=None) == so.ERR_WORKSPACE


def test_matmul_workspaces(so):
    import torch
    bf, f = torch.bfloat16, torch.float32
    size = so.sparse_expert_matmul_workspace_size
    # bf16 rows of whole 16 bytes are read where they lie; others are copied, fp32 is split in three
    assert size(bf, 100_000, 1024, 2048, 64) == 256
    rows, matrices = 100_000 * 2048, 64 * 1024 * 2048
    assert 2 * (rows + matrices) <= size(bf, 100_000, 1024, 2048, 64, False) <= 2 * (rows * 1.6 + matrices) + (1 << 20)
    assert 6 * (rows + matrices) <= size(f, 100_000, 1024, 2048, 64) <= 6 * (rows * 1.6 + matrices) + (1 << 20)
    assert size(bf, 100_000, 1023, 2047, 64) > 2 * (rows + matrices) * 0.99
    assert size(f, 0, 8, 8, 3) == 256 and size(f, -1, 8, 8, 3) == 0 and size(f, 8, 8, 8, 1025) == 0


def test_loss_refusals(so):
    def code(x=P, w=P, t=0, n=8, c=16, v=100, target=P, loss=P, lse=P, ws=P, size=WS, err=P):
        return so.LIB.sparse_vocab_loss(x, w, t, n, c, v, target, loss, lse, ws, size, err, None)

    for b in (dict(x=None), dict(w=None), dict(t=2), dict(n=-1), dict(n=(1 << 30) + 1), dict(c=0), dict(c=(1 << 20) + 1), dict(v=0),
              dict(v=(1 << 30) + 1), dict(target=None), dict(loss=None), dict(lse=None), dict(err=None), dict(v=1 << 30, c=1 << 10),
              dict(n=1 << 25, v=1 << 25, c=1)):
        assert code(**b) == so.ERR_INVALID_ARG, b
    assert code(ws=None) == so.ERR_WORKSPACE and code(size=200) == so.ERR_WORKSPACE and code(ws=ctypes.c_void_p(64)) == so.ERR_WORKSPACE
    assert code(n=0, x=None, w=None, target=None, loss=None, lse=None, ws=None) == so.OK

    def grad(dloss=None, x=P, w=P, t=1, n=8, c=16, v=100, target=P, lse=P, dx=P, dw=P, ws=P, size=WS, err=P):
        return so.LIB.sparse_vocab_loss_grad(dloss, x, w, t, n, c, v, target, lse, dx, dw, ws, size, err, None)

    for b in (dict(x=None), dict(w=None), dict(t=9), dict(target=None), dict(lse=None), dict(err=None), dict(c=0)):
        assert grad(**b) == so.ERR_INVALID_ARG, b
    assert grad(ws=None) == so.ERR_WORKSPACE
    assert grad(dx=None, dw=None, ws=None) == so.OK and grad(n=0, dw=None) == so.OK


def test_loss_workspaces(so):
    """The scores are never kept: what a call needs grows with a piece of them at most."""
    import torch
    bf, f = torch.bfloat16, torch.float32
    size = so.sparse_vocab_loss_workspace_size
    assert size(bf, 8192, 2048, 100_000, False) < 40 << 20
    whole = 8192 * 100_000 * 2
    assert size(bf, 8192, 2048, 100_000, True) < (256 << 20) + 8192 * 2048 * 4 + (2 << 20) < whole / 4
    assert size(f, 2048, 64, 1_000_000, True) < 6 * 1_000_000 * 64 + (160 << 20)
    assert size(bf, 16, 64, 5000, False) <= size(bf, 16, 64, 5000, True)
    assert size(f, 0, 8, 8, True) == 256 and size(f, 8, 8, 0, True) == 0
    with pytest.raises(KeyError):
        size(torch.float16, 8, 8, 8, True)
