"""Layer norm and its backward pass against the formulas in 64 bits.

Error bounds, per element, with u = 2^-24 (half an ulp of 1 in fp32).  A lane adds up to 16 values,
or c/512 in a wide row, then come 5 shuffle levels and up to 16 warps: a row sum's error is below
K u sum|terms| with K = c/512 + 64.  So |d mu| <= K u mean|x|; xhat = (x - mu) rstd is off by
E = K u (mean|x| rstd + |xhat|), rstd relatively by K u.  y adds the rounding of gamma, beta and the sum.
dx = rstd (h - mean h - xhat mean(h xhat)) inherits E in both places of xhat.  A column sum adds at
most D = 512 terms in a row for the sizes here (rows of a group, groups of a block, blocks / 8).
A bf16 output is rounded once more: 2^-8 of its value.
"""
import numpy as np
import pytest

from gpu_harness import Guarded

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF = 2.0 ** -8
TYPES = [("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16")]
SHAPES = [(1, 1), (3, 1), (1, 2), (5, 7), (2, 8), (7, 31), (33, 64), (100, 129), (17, 512), (9, 1000), (4, 2048),
          (3, 8192), (2, 8193), (3, 20001), (5000, 24), (700, 4096), (2000, 300), (8300, 1400), (301, 3333)]


def _dt(torch, name):
    return {"f32": torch.float32, "bf16": torch.bfloat16}[name]


def _formula(x, gamma, beta, eps):
    c = x.shape[1]
    mu = x.sum(1, keepdims=True) / c
    d = x - mu
    rstd = 1.0 / np.sqrt((d * d).sum(1, keepdims=True) / c + eps)
    xhat = d * rstd
    return xhat * gamma + beta, mu, rstd, xhat


def _grads(dy, xhat, rstd, gamma):
    h = dy * gamma
    a, b = h.mean(1, keepdims=True), (h * xhat).mean(1, keepdims=True)
    return rstd * (h - a - xhat * b), (dy * xhat).sum(0), dy.sum(0)


def _np(t):
    return t.detach().double().cpu().numpy()


class Case:
    """Inputs in guarded device memory, with the same values in 64 bits."""

    def __init__(self, torch, so, n, c, xt, yt, seed=0, idx=None, rows=None, shift=0, gamma=True, mean=0.5, std=1.0):
        rng = np.random.default_rng(seed + 7 * n + c)
        self.torch, self.so, self.n, self.c = torch, so, n, c
        self.G = Guarded(seed=n + c)
        self.r = rows or n
        self.x = self.typed(rng.standard_normal((self.r, c)) * std + mean, xt, shift)
        self.dy = self.typed(rng.standard_normal((n, c)), yt, shift)
        self.gamma = self.typed(1 + 0.3 * rng.standard_normal(c), "f32") if gamma else None
        self.beta = self.typed(0.3 * rng.standard_normal(c), "f32") if gamma else None
        self.idx = None if idx is None else self.G.array(np.asarray(idx, np.int64))
        self.y, self.dx = self.blank((n, c), yt, shift), self.blank((n, c), xt, shift)
        self.mean, self.rstd = self.G.zeros(n), self.G.zeros(n)
        self.dgamma, self.dbeta = self.G.zeros(c), self.G.zeros(c)
        self.ws = self.G.empty(max(so.sparse_layer_norm_workspace_size(n, c), 256), torch.uint8)
        self.err = self.G.error_word()

    def blank(self, shape, kind, shift=0):
        flat = self.G.zeros(int(np.prod(shape)) + shift, _dt(self.torch, kind))
        return flat[shift:].view(shape)

    def typed(self, a, kind, shift=0):
        t = self.blank(a.shape, kind, shift)
        t.copy_(self.torch.from_numpy(np.ascontiguousarray(a, np.float32)))
        return t

    def run(self, eps=1e-5, want=True, stream=None):
        so = self.so
        so.check(so.sparse_layer_norm(self.x, self.r, self.c, self.idx, self.n, self.gamma, self.beta, eps, self.y,
                                      self.mean, self.rstd, self.err, stream), "layer_norm")
        so.check(so.sparse_layer_norm_grad(self.dy, self.x, self.r, self.c, self.idx, self.n, self.gamma, self.mean,
                                           self.rstd, self.dx, self.dgamma if want else None,
                                           self.dbeta if want else None, self.ws if want else None, self.err, stream),
                 "layer_norm_grad")
        self.G.check("layer norm")

    def compare(self, eps=1e-5, keep=None):
        c = self.c
        x, dy = _np(self.x), _np(self.dy)
        if self.idx is not None:
            x = x[self.idx.cpu().numpy()]
        rows = np.ones(self.n, bool) if keep is None else keep
        x, dy = x[rows], dy[rows]
        gamma = _np(self.gamma) if self.gamma is not None else np.ones(c)
        beta = _np(self.beta) if self.beta is not None else np.zeros(c)
        y, mu, rstd, xhat = _formula(x, gamma, beta, eps)
        dx, dg, db = _grads(dy, xhat, rstd, gamma)
        K, D = c / 512 + 64, 512
        ax = np.abs(x).mean(1, keepdims=True)
        E = K * U * (ax * rstd + np.abs(xhat))
        by = BF if self.y.dtype == self.torch.bfloat16 else 0.0
        bx = BF if self.dx.dtype == self.torch.bfloat16 else 0.0

        def near(what, got, ref, tol):
            bad = ~(np.abs(got - ref) <= tol + 1e-30)
            assert not bad.any(), (what, int(bad.sum()), got[bad][:3], ref[bad][:3], np.broadcast_to(tol, ref.shape)[bad][:3])

        near("mean", _np(self.mean)[rows], mu[:, 0], K * U * ax[:, 0])
        near("rstd", _np(self.rstd)[rows], rstd[:, 0], K * U * rstd[:, 0] * (1 + (ax * rstd)[:, 0] ** 2 * K * U))
        near("y", _np(self.y)[rows], y, np.abs(gamma) * E + 4 * U * (np.abs(y) + np.abs(beta)) + by * np.abs(y))
        h = dy * gamma
        ah, ahx = np.abs(h).mean(1, keepdims=True), np.abs(h * xhat).mean(1, keepdims=True)
        tol = 2 * K * U * rstd * (1 + ax * rstd) * (np.abs(h) + ah + (np.abs(xhat) + 1) * (ahx + ah))
        near("dx", _np(self.dx)[rows], dx, tol + bx * np.abs(dx))
        near("dgamma", _np(self.dgamma), dg, D * U * np.abs(dy * xhat).sum(0) + (np.abs(dy) * E).sum(0))
        near("dbeta", _np(self.dbeta), db, D * U * np.abs(dy).sum(0))


@pytest.mark.parametrize("xt,yt", TYPES)
@pytest.mark.parametrize("n,c", SHAPES)
def test_layer_norm_and_gradients(cuda_lib, n, c, xt, yt):
    import torch
    k = Case(torch, cuda_lib, n, c, xt, yt)
    k.run()
    assert int(k.err.item()) == 0
    k.compare()


@pytest.mark.parametrize("xt,yt", TYPES)
@pytest.mark.parametrize("shift", [1, 3])
@pytest.mark.parametrize("c", [256, 1111, 2048])
def test_arrays_of_any_alignment(cuda_lib, c, shift, xt, yt):
    import torch
    k = Case(torch, cuda_lib, 50, c, xt, yt, shift=shift)
    k.run()
    k.compare()


@pytest.mark.parametrize("c", [24, 128, 515, 9000])
def test_looked_up_rows_are_the_tables(cuda_lib, c):
    import torch
    rng = np.random.default_rng(c)
    idx = rng.integers(0, 40, 300)
    idx[:20] = 39                       # repeats
    k = Case(torch, cuda_lib, 300, c, "f32", "f32", idx=idx, rows=40)
    k.run()
    assert int(k.err.item()) == 0
    k.compare()


def test_a_bad_lookup_is_reported_and_its_row_left(cuda_lib):
    import torch
    for c in (64, 9000):
        idx = np.array([0, 5, 40, 3, -1, 2])
        k = Case(torch, cuda_lib, 6, c, "f32", "f32", idx=np.clip(idx, 0, 39), rows=40)
        k.idx.copy_(torch.from_numpy(idx))
        k.y.fill_(7.0)
        k.dx.fill_(7.0)
        k.run()
        assert int(k.err.item()) == cuda_lib.ERR_INDEX_OUT_OF_RANGE
        y, dx = _np(k.y), _np(k.dx)
        assert (y[[2, 4]] == 7.0).all() and (dx[[2, 4]] == 7.0).all()
        x = _np(k.x)
        ref = _formula(x[[0, 5, 3, 2]], _np(k.gamma), _np(k.beta), 1e-5)[0]
        assert np.abs(y[[0, 1, 3, 5]] - ref).max() < 1e-4


def test_without_scale_shift_or_their_gradients(cuda_lib):
    import torch
    k = Case(torch, cuda_lib, 37, 96, "bf16", "bf16", gamma=False)
    k.run()
    k.compare()
    k.dgamma.fill_(3.0)
    k.run(want=False)
    assert (k.dgamma == 3.0).all()


def test_rows_without_spread_large_means_and_far_scales(cuda_lib):
    import torch
    for mean, std, eps in ((0.1, 0.0, 1e-5), (100.0, 1.0, 1e-5), (0.0, 1e-12, 1e-5), (0.0, 1e12, 0.0), (3.0, 0.5, 0.0)):
        k = Case(torch, cuda_lib, 12, 200, "f32", "f32", mean=mean, std=std)
        k.run(eps=eps)
        k.compare(eps=eps)


def test_nan_and_infinity_stay_in_their_rows(cuda_lib):
    import torch
    for c in (130, 1000, 9000):
        k = Case(torch, cuda_lib, 9, c, "f32", "f32")
        k.x[2, 5] = float("nan")
        k.x[6, c - 1] = float("inf")
        k.run()
        keep = np.array([i not in (2, 6) for i in range(9)])
        assert np.isnan(_np(k.y)[[2, 6]]).all() and np.isnan(_np(k.dx)[[2, 6]]).all()
        assert np.isfinite(_np(k.y)[keep]).all() and np.isfinite(_np(k.dx)[keep]).all()


def test_no_rows(cuda_lib):
    import torch
    k = Case(torch, cuda_lib, 0, 64, "f32", "f32", rows=1)
    k.dgamma.fill_(3.0)
    k.run()
    assert (k.dgamma == 0.0).all() and (k.dbeta == 0.0).all()


def test_equal_inputs_give_equal_bits_on_any_stream(cuda_lib):
    import torch
    k = Case(torch, cuda_lib, 3000, 384, "bf16", "bf16")
    k.run()
    first = [t.clone() for t in (k.y, k.dx, k.dgamma, k.dbeta, k.mean, k.rstd)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for t in (k.y, k.dx, k.dgamma, k.dbeta, k.mean, k.rstd):
        t.zero_()
    torch.cuda.synchronize()
    k.run(stream=s)
    for a, b in zip(first, (k.y, k.dx, k.dgamma, k.dbeta, k.mean, k.rstd)):
        assert torch.equal(a, b)


def test_elements_past_32_bits(cuda_lib):
    """2.3e9 elements: rows at both ends against the formula, and dbeta, whose sum of equal dy is known."""
    import torch
    so = cuda_lib
    n, c = 1_150_000, 2000
    x = torch.empty(n, c, dtype=torch.bfloat16, device="cuda").normal_()
    dy = torch.full((n, c), 0.5, dtype=torch.bfloat16, device="cuda")
    y, dx = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    dgamma, dbeta = torch.empty(c, device="cuda"), torch.empty(c, device="cuda")
    ws = torch.empty(so.sparse_layer_norm_workspace_size(n, c), dtype=torch.uint8, device="cuda")
    err = so.error_word()
    so.check(so.sparse_layer_norm(x, n, c, None, n, None, None, 1e-5, y, mean, rstd, err))
    so.check(so.sparse_layer_norm_grad(dy, x, n, c, None, n, None, mean, rstd, dx, dgamma, dbeta, ws, err))
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    for rows in (slice(0, 3), slice(n - 3, n)):
        ref = _formula(_np(x[rows]), 1.0, 0.0, 1e-5)[0]
        assert np.abs(_np(y[rows]) - ref).max() <= BF * np.abs(ref).max()
        assert np.abs(_np(dx[rows])).max() <= 1e-4          # equal dy: h - mean(h) and mean(h xhat) are 0
    # 575000 is a sum of halves: exact until 2^23 of them, then partial sums of up to 2^23 / 2
    assert np.abs(_np(dbeta) - 0.5 * n).max() <= 512 * U * 0.5 * n


def test_gradients_against_differences_of_the_formula(cuda_lib):
    import torch
    k = Case(torch, cuda_lib, 6, 40, "f32", "f32")
    k.run()
    rng = np.random.default_rng(5)
    x, dy, gamma, beta = _np(k.x), _np(k.dy), _np(k.gamma), _np(k.beta)
    ex, eg, eb = rng.standard_normal(x.shape), rng.standard_normal(40), rng.standard_normal(40)
    h = 1e-4

    def loss(s):
        return (dy * _formula(x + s * ex, gamma + s * eg, beta + s * eb, 1e-5)[0]).sum()

    slope = (loss(h) - loss(-h)) / (2 * h)
    got = (_np(k.dx) * ex).sum() + (_np(k.dgamma) * eg).sum() + (_np(k.dbeta) * eb).sum()
    # h^2 truncation (third derivatives of order 1 on 240 elements) and the fp32 bounds above
    size = np.abs(_np(k.dx) * ex).sum() + np.abs(_np(k.dgamma) * eg).sum() + np.abs(_np(k.dbeta) * eb).sum()
    assert abs(got - slope) <= 1e-5 * size


def test_refusals(cuda_lib):
    import torch
    so = cuda_lib
    k = Case(torch, so, 8, 32, "f32", "f32")
    ok = [k.x, 8, 32, None, 8, k.gamma, k.beta, 1e-5, k.y, k.mean, k.rstd, k.err]

    def code(at, value):
        a = list(ok)
        a[at] = value
        return so.sparse_layer_norm(*a)

    assert so.sparse_layer_norm(*ok) == so.OK
    for at, value in ((1, -1), (1, 7), (2, 0), (2, 1 << 31), (4, -1), (7, -1.0), (7, float("nan")),
                      (7, float("inf")), (11, None)):
        assert code(at, value) == so.ERR_INVALID_ARG, (at, value)
    with pytest.raises(TypeError):
        code(0, k.x.double())
    with pytest.raises(ValueError):
        code(0, k.x.t())
    # bf16 rows have bf16 outputs
    assert so.sparse_layer_norm(k.x.bfloat16(), 8, 32, None, 8, None, None, 1e-5, k.y, None, None,
                                k.err) == so.ERR_INVALID_ARG
    g = [k.dy, k.x, 8, 32, None, 8, k.gamma, k.mean, k.rstd, k.dx, k.dgamma, k.dbeta]
    assert so.sparse_layer_norm_grad(*g, k.ws, k.err) == so.OK
    assert so.sparse_layer_norm_grad(*g, None, k.err) == so.ERR_WORKSPACE
    assert so.sparse_layer_norm_grad(*g, k.ws[:8], k.err) == so.ERR_WORKSPACE
    assert so.sparse_layer_norm_grad(*g, k.ws[1:], k.err) == so.ERR_WORKSPACE
    for at in (7, 8):
        assert so.sparse_layer_norm_grad(*[None if i == at else v for i, v in enumerate(g)], k.ws,
                                         k.err) == so.ERR_INVALID_ARG
    torch.cuda.synchronize()
    assert int(k.err.item()) == 0
    assert so.sparse_layer_norm_workspace_size(-1, 4) == 0 and so.sparse_layer_norm_workspace_size(4, 0) == 0


@pytest.mark.parametrize("xt,yt", TYPES)
@pytest.mark.parametrize("c", [1489, 1501, 1519, 1527, 3001, 3041])
def test_rows_whose_ring_is_about_48_kb(cuda_lib, c, xt, yt):
    """Dynamic and static shared memory together pass what a launch has without asking."""
    import torch
    k = Case(torch, cuda_lib, 9, c, xt, yt)
    k.run()
    assert int(k.err.item()) == 0
    k.compare()


@pytest.mark.parametrize("xt,yt", TYPES)
@pytest.mark.parametrize("n,c,shift", [(2, 60000, 0), (3, 60001, 0), (700, 9000, 0), (613, 8200, 1), (20, 16384, 0)])
def test_rows_wider_than_the_groups(cuda_lib, n, c, shift, xt, yt):
    """Rows held in shared memory, two at a time and one, and rows that shared memory does not hold."""
    import torch
    idx = np.random.default_rng(n).integers(0, n + 3, n)
    idx[n // 2] = n + 3                 # bad: the odd row of a pair or the even one of another
    k = Case(torch, cuda_lib, n, c, xt, yt, idx=np.minimum(idx, n + 2), rows=n + 3, shift=shift)
    k.run()
    assert int(k.err.item()) == 0
    k.compare()
    want = [t.clone() for t in (k.y, k.dx, k.mean, k.rstd)]
    for t in (k.y, k.dx, k.mean, k.rstd):
        t.zero_()
    k.idx[n // 2] = n + 3
    so = cuda_lib
    assert so.sparse_layer_norm(k.x, k.r, c, k.idx, n, k.gamma, k.beta, 1e-5, k.y, k.mean, k.rstd, k.err) == so.OK
    assert so.sparse_layer_norm_grad(k.dy, k.x, k.r, c, k.idx, n, k.gamma, want[2], want[3], k.dx, None, None, None,
                                     k.err) == so.OK
    k.G.check("layer norm")
    assert int(k.err.item()) == so.ERR_INDEX_OUT_OF_RANGE
    for got, ref in zip((k.y, k.dx, k.mean, k.rstd), want):
        assert not got[n // 2].any()
        got[n // 2] = ref[n // 2]
        assert torch.equal(got, ref)


@pytest.mark.parametrize("xt,yt", TYPES)
@pytest.mark.parametrize("n,c,shift", [(40, 22, 0), (300, 94, 0), (33, 236, 0), (40, 602, 0), (700, 1110, 0),
                                       (20, 4098, 0), (9, 9002, 0), (50, 64, 2), (50, 256, 2), (50, 2048, 2),
                                       (9, 8200, 2)])
def test_rows_of_pairs(cuda_lib, n, c, shift, xt, yt):
    """Rows of an even number of values, or arrays aligned to two of them: accesses of two."""
    import torch
    k = Case(torch, cuda_lib, n, c, xt, yt, shift=shift)
    k.run()
    assert int(k.err.item()) == 0
    k.compare()


@pytest.mark.parametrize("xt,yt", TYPES)
@pytest.mark.parametrize("n,c", [(16700, 1048), (6600, 2560), (4100, 4104), (3300, 5120)])
def test_many_long_rows(cuda_lib, n, c, xt, yt):
    """Enough long rows for the ring backward, groups of 72 to 320 lanes."""
    import torch
    k = Case(torch, cuda_lib, n, c, xt, yt)
    k.run()
    assert int(k.err.item()) == 0
    k.compare()
