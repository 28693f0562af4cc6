"""The compiled module behind the binding's calls of the operators around the table step: it takes what
is of the common kind and leaves everything else (None) to the binding, which converts or refuses it."""
import ctypes

import numpy as np
import pytest


@pytest.fixture(scope="module")
def so():
    from lazy_optimizers_embedding_gb300 import binding
    return binding


def test_what_is_not_of_the_common_kind_is_left(so):
    import torch
    f = torch.zeros(4, 8)
    m = torch.zeros(4)
    e = torch.zeros(1, dtype=torch.int32)
    good = [f, 4, 8, None, 4, None, None, 1e-5, f, m, m, e, None]
    for call in ([], good, good[:-1], [3, *good[1:]], [None, "4", *good[2:]], [None, 1 << 70, *good[2:]]):
        assert so._pycall.layer_norm(*call) is None         # tensors of the host among them
    assert so._pycall.orthogonalize(None, 1, 2, 2, 5, None, None, None, None) is None
    assert so._pycall.muon_step(None, None, None, 1, 2, 2, so.NsConfig(), None, None, None) is None


def test_the_binding_refuses_what_is_left(so):
    import torch
    f, m, e = torch.zeros(4, 8), torch.zeros(4), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        so.sparse_layer_norm(f, 4, 8, None, 4, None, None, 1e-5, f, m, m, e)
    with pytest.raises(TypeError):
        so.sparse_layer_norm("x", 4, 8, None, 4, None, None, 1e-5, f, m, m, e)


@pytest.mark.gpu
def test_both_ways_give_the_same(cuda_lib):
    """With a stream given the binding's own path runs."""
    import torch
    so = cuda_lib
    dev = "cuda"
    n, c, k, experts = 50, 96, 2, 5
    g = torch.Generator(device=dev).manual_seed(1)
    r = lambda *s: torch.randn(*s, device=dev, generator=g)  # noqa: E731
    x, dy, gamma, beta, table = r(n, c), r(n, c), r(c), r(c), r(200, c)
    idx = torch.randint(0, 200, (n,), device=dev, generator=g)
    expert = torch.randint(-1, experts, (n, k), device=dev, generator=g)
    w, ys, u = r(n, k), r(n * k, c), r(2, 40, 70)
    cfg = so.NsConfig(a=3.4445, b=-4.7750, c=2.0315, eps=1e-7, steps=5, products=3)
    step = so.MuonConfig(lr=0.02, momentum=0.95, weight_decay=0.1, scale=1.0, nesterov=1, ns=cfg)

    def all_calls(stream):
        e = so.error_word()
        y, dx, xs, dys = torch.zeros(n, c, device=dev), torch.zeros(n, c, device=dev), torch.zeros(n * k, c, device=dev), torch.zeros(n * k, c, device=dev)
        out, mean, rstd, dg, db = torch.zeros_like(u), torch.zeros(n, device=dev), torch.zeros(n, device=dev), torch.zeros(c, device=dev), torch.zeros(c, device=dev)
        comb, dw = torch.zeros(n, c, device=dev), torch.zeros(n, k, device=dev)
        off, src, pos = torch.zeros(experts + 1, dtype=torch.int64, device=dev), torch.zeros(n * k, dtype=torch.int32, device=dev), torch.zeros(n, k, dtype=torch.int32, device=dev)
        wt, buf = x.clone().view(1, n, c), torch.zeros(1, n, c, device=dev)
        size = max(so.sparse_layer_norm_workspace_size(n, c), so.sparse_expert_workspace_size(n, k, experts),
                   so.sparse_muon_workspace_size(2, 40, 70, 3), so.sparse_muon_workspace_size(1, n, c, 3))
        ws = torch.zeros(size, dtype=torch.uint8, device=dev)
        codes = [so.sparse_layer_norm(table, 200, c, idx, n, gamma, beta, 1e-5, y, mean, rstd, e, stream),
                 so.sparse_layer_norm_grad(dy, table, 200, c, idx, n, gamma, mean, rstd, dx, dg, db, ws, e, stream),
                 so.sparse_expert_sort(expert, n, k, experts, off, src, pos, ws, e, stream),
                 so.sparse_expert_dispatch(x, n, k, c, pos, off, experts, xs, e, stream),
                 so.sparse_expert_combine(ys, n, k, c, pos, w, comb, e, stream),
                 so.sparse_expert_combine_grad(dy, ys, n, k, c, pos, off, experts, w, dys, dw, e, stream),
                 so.sparse_orthogonalize(u, 2, 40, 70, cfg, out, ws, e, stream),
                 so.sparse_muon_step(wt, buf, dy, 1, n, c, step, ws, e, stream)]
        assert codes == [so.OK] * 8
        torch.cuda.synchronize()
        assert int(e.item()) == 0
        return [t.cpu().numpy() for t in (y, mean, rstd, dx, dg, db, off, src, pos, xs, comb, dys, dw, out, wt, buf)]

    for a, b in zip(all_calls(None), all_calls(torch.cuda.current_stream())):
        assert np.abs(b).sum() > 0 and np.array_equal(a, b)


@pytest.mark.gpu
def test_refusals_and_conversions(cuda_lib):
    import torch
    so = cuda_lib
    x, y, m, e = torch.randn(4, 8, device="cuda"), torch.zeros(4, 8, device="cuda"), torch.zeros(4, device="cuda"), so.error_word()

    def norm(x=x, y=y, n=4, m=m, eps=1e-5, e=e):
        return so.sparse_layer_norm(x, 4, 8, None, n, None, None, eps, y, m, m, e)

    assert norm() == so.OK and norm(eps=0) == so.OK and norm(n=np.int64(4)) == so.OK
    assert so._pycall.layer_norm(x, 4, 8, None, 4, None, None, 1e-5, y, m, m, e, None) == so.OK
    assert norm(m=None) == so.OK and norm(e=None) == so.ERR_INVALID_ARG and norm(n=-1) == so.ERR_INVALID_ARG
    assert norm(m=m.data_ptr()) == so.OK                     # a pointer as an integer
    for bad, error in ((dict(x=x.double()), TypeError), (dict(x=x.t()), ValueError), (dict(y=y.cpu()), ValueError),
                       (dict(m=m.bfloat16()), TypeError), (dict(e=e.long()), TypeError), (dict(x="x"), TypeError)):
        with pytest.raises(error):
            norm(**bad)
    with pytest.raises((TypeError, ctypes.ArgumentError)):
        so.sparse_orthogonalize(x.view(1, 4, 8), 1, 4, 8, so.SgdConfig(), y, torch.zeros(1 << 20, dtype=torch.uint8, device="cuda"), e)
    with torch.cuda.stream(torch.cuda.Stream()):             # the stream that is current at the call
        assert norm() == so.OK
        torch.cuda.current_stream().synchronize()
    assert int(e.item()) == 0 and torch.isfinite(y).all()
