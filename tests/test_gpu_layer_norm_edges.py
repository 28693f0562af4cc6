"""Layer norm where each of its kernels can go wrong: looked-up rows that are not there, values that are
not finite, means far above the spread, widths on both sides of where another kernel takes over.

Bounds as in the tests of the ordinary cases: u = 2^-24, a row sum's error is below K u sum|terms|
with K = c / 512 + 64, a column sum adds at most 512 terms in a row."""
import numpy as np
import pytest

from test_gpu_layer_norm import U, Case, _np

pytestmark = pytest.mark.gpu

# rows, columns, types: of registers, of the ring forward (packed, pairs, single values), of the ring
# backward too, of wide rows
KERNELS = [(33, 512, "f32", "f32"), (33, 1000, "bf16", "bf16"), (33, 2048, "bf16", "bf16"), (33, 2050, "f32", "bf16"),
           (33, 1111, "f32", "f32"), (33, 1111, "bf16", "bf16"), (33, 1111, "f32", "bf16"), (2100, 8192, "f32", "f32"),
           (2100, 8192, "bf16", "bf16"), (6600, 2560, "f32", "bf16"), (33, 9000, "bf16", "bf16")]


@pytest.mark.parametrize("n,c,xt,yt", KERNELS)
def test_rows_that_are_not_there(cuda_lib, n, c, xt, yt):
    import torch
    so = cuda_lib
    rng = np.random.default_rng(n + c)
    idx = rng.integers(0, 40, n)
    k = Case(torch, so, n, c, xt, yt, idx=idx, rows=40)
    k.run()
    assert int(k.err.item()) == 0
    want = [t.clone() for t in (k.y, k.dx, k.mean, k.rstd)]
    bad = [0, n // 2, n // 2 + 1, n - 1]
    idx[bad] = [40, -1, 1 << 40, -(1 << 62)]
    k.idx.copy_(torch.from_numpy(idx))
    for t in (k.y, k.dx, k.mean, k.rstd):
        t.fill_(7.0)
    so.check(so.sparse_layer_norm(k.x, 40, c, k.idx, n, k.gamma, k.beta, 1e-5, k.y, k.mean, k.rstd, k.err))
    assert int(k.err.item()) == so.ERR_INDEX_OUT_OF_RANGE
    k.err.zero_()
    so.check(so.sparse_layer_norm_grad(k.dy, k.x, 40, c, k.idx, n, k.gamma, k.mean, k.rstd, k.dx, k.dgamma, k.dbeta,
                                       k.ws, k.err))
    assert int(k.err.item()) == so.ERR_INDEX_OUT_OF_RANGE
    k.G.check("layer norm")
    for got, ref in zip((k.y, k.dx, k.mean, k.rstd), want):
        assert (got[bad] == 7.0).all()
        got[bad] = ref[bad]
        assert torch.equal(got, ref)


@pytest.mark.parametrize("n,c,xt,yt", KERNELS)
def test_nan_and_infinity_stay_in_their_rows(cuda_lib, n, c, xt, yt):
    import torch
    k = Case(torch, cuda_lib, n, c, xt, yt)
    rows = {1: (0, float("nan")), n // 2: (c - 1, float("inf")), n - 2: (c // 2, -float("inf"))}
    for i, (j, v) in rows.items():
        k.x[i, j] = v
    k.run()
    bad = list(rows)
    keep = np.array([i not in rows for i in range(n)])
    assert torch.isnan(k.y[bad]).all() and torch.isnan(k.dx[bad]).all()
    assert np.isfinite(_np(k.y)[keep]).all() and np.isfinite(_np(k.dx)[keep]).all()
    k = Case(torch, cuda_lib, n, c, xt, yt)
    k.dy[1, c - 1] = float("nan")
    k.run()
    assert torch.isnan(k.dx[1]).all() and torch.isnan(k.dbeta[c - 1]) and torch.isnan(k.dgamma[c - 1])
    k.dx[1] = 0.0
    assert torch.isfinite(k.dx).all() and torch.isfinite(k.dgamma[:c - 1]).all() and torch.isfinite(k.dbeta[:c - 1]).all()


@pytest.mark.parametrize("n,c,yt", [(40, 64, "f32"), (40, 200, "bf16"), (40, 1024, "f32"), (40, 3000, "f32"), (2100, 8192, "f32"),
                                    (6600, 2560, "bf16"), (40, 333, "f32"), (40, 1111, "f32"), (40, 1111, "bf16"), (40, 2050, "f32"),
                                    (40, 9000, "f32")])
def test_a_mean_far_above_the_spread(cuda_lib, n, c, yt):
    """x - mean is exact here, so xhat is off by the roundings of the difference times rstd alone, 3 u of
    itself, and not by a rounding of mean times rstd."""
    import torch
    so = cuda_lib
    k = Case(torch, so, n, c, "f32", yt)
    rng = np.random.default_rng(c)
    d = rng.integers(-8, 9, (n, c)).astype(np.float64)
    mean = 2.0 ** 20 + rng.integers(-1000, 1000, (n, 1))
    rstd = np.float32(1.0 / np.sqrt((d * d).mean(1, keepdims=True))).astype(np.float64)
    k.x.copy_(torch.from_numpy((mean + d).astype(np.float32)))
    k.mean.copy_(torch.from_numpy(mean[:, 0].astype(np.float32)))
    k.rstd.copy_(torch.from_numpy(rstd[:, 0].astype(np.float32)))
    so.check(so.sparse_layer_norm_grad(k.dy, k.x, n, c, None, n, k.gamma, k.mean, k.rstd, k.dx, k.dgamma, k.dbeta,
                                       k.ws, k.err))
    k.G.check("layer norm")
    dy, gamma, xhat = _np(k.dy), _np(k.gamma), d * rstd
    h = dy * gamma
    a, b = h.mean(1, keepdims=True), (h * xhat).mean(1, keepdims=True)
    K = c / 512 + 64
    size = np.abs(h) + np.abs(h).mean(1, keepdims=True) + np.abs(xhat) * np.abs(h * xhat).mean(1, keepdims=True)
    assert (np.abs(_np(k.dx) - rstd * (h - a - xhat * b)) <= 2 * K * U * rstd * size).all()
    assert (np.abs(_np(k.dgamma) - (dy * xhat).sum(0)) <= (512 + 4) * U * np.abs(dy * xhat).sum(0)).all()
    assert (np.abs(_np(k.dbeta) - dy.sum(0)) <= 512 * U * np.abs(dy).sum(0)).all()


# columns on both sides of where another kernel takes over: (fp32 or bf16 x), (single values, pairs, packed)
TAKEN = [(255, "f32", 9, "", ""), (256, "f32", 9, "", ""), (257, "f32", 9, "ring", "ring"), (254, "f32", 9, "", ""),
         (258, "f32", 9, "ring", "ring"), (511, "bf16", 9, "", ""), (513, "bf16", 9, "ring", "ring"), (510, "bf16", 9, "", ""),
         (514, "bf16", 9, "ring", "ring"), (1024, "f32", 9, "", ""), (1028, "f32", 9, "ring", ""), (1024, "bf16", 9, "", ""),
         (1032, "bf16", 9, "ring", ""), (8192, "bf16", 2047, "ring", ""), (8192, "bf16", 2048, "ring", "ring"),
         (4096, "f32", 4096, "ring", ""), (4100, "f32", 4096, "ring", "ring"), (8191, "f32", 9, "ring", "ring"),
         (8192, "f32", 9, "ring", ""), (8193, "f32", 9, "wide", "wide"), (8196, "f32", 9, "wide", "wide"),
         (8200, "bf16", 9, "wide", "wide")]


@pytest.mark.parametrize("c,kind,n,forward,back", TAKEN)
def test_which_kernel_takes_a_row(cuda_lib, c, kind, n, forward, back):
    import torch
    so = cuda_lib
    k = Case(torch, so, n, c, kind, kind)
    so.sparse_profile_enable()
    so.sparse_profile_reset()
    try:
        k.run()
        names = set(so.sparse_profile_read())
    finally:
        so.sparse_profile_enable(False)
    name = lambda base, which: base + ("_" + which if which else "")  # noqa: E731
    assert names == {name("layer_norm", forward), name("layer_norm_grad", back), "layer_norm_grad_join"}
    k.compare()


@pytest.mark.parametrize("c", [64, 1111, 2048, 9000])
def test_rows_of_zeros_with_any_eps_above_zero(cuda_lib, c):
    """x - mean is 0, so y is beta, also where eps is below what fp32 holds or past it."""
    import torch
    for eps in (1e-5, 1e-38, 1e-44, 1e-60, 1e60):
        k = Case(torch, cuda_lib, 5, c, "f32", "f32")
        k.x.zero_()
        so = cuda_lib
        so.check(so.sparse_layer_norm(k.x, 5, c, None, 5, k.gamma, k.beta, eps, k.y, k.mean, k.rstd, k.err))
        k.G.check("layer norm")
        assert (k.y == k.beta).all() and (k.mean == 0).all() and torch.isfinite(k.rstd).all(), eps
