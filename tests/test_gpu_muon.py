"""Newton-Schulz orthogonalisation and the Muon step against the formulas in 64 bits.

Results are compared in the Frobenius norm.  A 64-bit simulation of the kernels' f16 splits and
roundings over flat, decaying and low-rank spectra (64 x 128 to 1024 x 1024) is off by at most 2.0e-3 of
the norm with one product and 6.5e-6 with three; the bounds are 2.5 times the first and three times the
second, which also holds the fp32 accumulation.  Rounding to bf16 adds at most 2^-9 of the norm.
Weights: (1 - lr wd) w - lr s O adds the bound of O times lr s, and 2 roundings of fp32.
"""
import numpy as np
import pytest

from gpu_harness import Guarded

pytestmark = pytest.mark.gpu

NS = (3.4445, -4.7750, 2.0315)
TOL = {1: 5e-3, 3: 2e-5}
SHAPES = [(1, 1, 1), (1, 1, 5), (2, 5, 1), (3, 7, 7), (1, 16, 16), (2, 64, 128), (1, 128, 64), (1, 129, 200),
          (3, 200, 129), (1, 100, 1000), (2, 1000, 100), (1, 257, 511), (2, 384, 640), (1, 24, 5000), (1, 900, 1030),
          (40, 33, 65), (1, 100, 600), (2, 50, 1500), (1, 2048, 120), (20, 128, 1030), (1, 1100, 1300), (400, 20, 24)]


def _np(t):
    return t.detach().double().cpu().numpy()


def _formula(u, steps=5, eps=1e-7, coef=NS):
    a, b, c = coef
    tall = u.shape[1] > u.shape[2]
    x = np.swapaxes(u, 1, 2) if tall else u
    x = x / (np.sqrt((x * x).sum((1, 2), keepdims=True)) + eps)
    for _ in range(steps):
        g = x @ np.swapaxes(x, 1, 2)
        x = a * x + (b * g + c * (g @ g)) @ x
    return np.swapaxes(x, 1, 2) if tall else x


def _spectrum(rng, batch, r, c, kind):
    g = rng.standard_normal((batch, r, c))
    if kind == "low rank":
        k = max(1, min(r, c) // 16)
        g = rng.standard_normal((batch, r, k)) @ rng.standard_normal((batch, k, c)) + 0.05 * g
    if kind == "decaying":
        u, s, v = np.linalg.svd(g, full_matrices=False)
        g = (u * np.exp(-np.linspace(0, 9, s.shape[1]))) @ v
    return g


def _off(got, ref):
    """The largest relative Frobenius error of a batch."""
    d = np.sqrt(((got - ref) ** 2).sum((1, 2)))
    return float((d / np.maximum(np.sqrt((ref ** 2).sum((1, 2))), 1e-30)).max())


class Case:
    def __init__(self, torch, so, u, products, in_type="f32", out_type="f32", shift=0, steps=5, eps=1e-7, coef=NS):
        dt = {"f32": torch.float32, "bf16": torch.bfloat16}
        self.torch, self.so = torch, so
        self.b, self.r, self.c = u.shape
        self.G = Guarded(seed=self.r)
        self.u = self.G.zeros(u.size + shift, dt[in_type])[shift:].view(u.shape)
        self.u.copy_(torch.from_numpy(np.ascontiguousarray(u, np.float32)))
        self.out = self.G.zeros(u.size + shift, dt[out_type])[shift:].view(u.shape)
        self.ws = self.G.empty(so.sparse_muon_workspace_size(self.b, self.r, self.c, products), torch.uint8)
        self.ws.fill_(255)           # NaN wherever a kernel would read what none wrote
        self.err = self.G.error_word()
        self.cfg = so.NsConfig(a=coef[0], b=coef[1], c=coef[2], eps=eps, steps=steps, products=products)

    def run(self, stream=None):
        self.so.check(self.so.sparse_orthogonalize(self.u, self.b, self.r, self.c, self.cfg, self.out, self.ws,
                                                   self.err, stream), "orthogonalize")
        self.G.check("orthogonalize")
        return _np(self.out)


@pytest.mark.parametrize("products,in_type,out_type", [(3, "f32", "f32"), (1, "bf16", "bf16"), (1, "f32", "bf16"),
                                                       (3, "bf16", "f32")])
@pytest.mark.parametrize("batch,r,c", SHAPES)
def test_orthogonalize(cuda_lib, batch, r, c, products, in_type, out_type):
    import torch
    u = np.random.default_rng(r * 7 + c).standard_normal((batch, r, c))
    k = Case(torch, cuda_lib, u, products, in_type, out_type)
    got = k.run()
    assert int(k.err.item()) == 0
    assert _off(got, _formula(_np(k.u))) <= TOL[products] + (2.0 ** -9 if out_type == "bf16" else 0.0)


@pytest.mark.parametrize("products", [1, 3])
@pytest.mark.parametrize("kind", ["low rank", "decaying"])
@pytest.mark.parametrize("r,c", [(64, 128), (320, 200), (512, 512)])
def test_spectra(cuda_lib, r, c, kind, products):
    import torch
    k = Case(torch, cuda_lib, _spectrum(np.random.default_rng(r), 1, r, c, kind), products)
    assert _off(k.run(), _formula(_np(k.u))) <= TOL[products]


@pytest.mark.parametrize("products", [1, 3])
def test_steps_coefficients_and_scales(cuda_lib, products):
    import torch
    u = np.random.default_rng(3).standard_normal((2, 70, 150))
    for steps, coef, scale in ((1, NS, 1.0), (2, NS, 1.0), (9, (1.5, -0.5, 0.0), 1.0), (12, (1.875, -1.25, 0.375), 1.0),
                               (5, NS, 1e-12), (5, NS, 1e12)):
        k = Case(torch, cuda_lib, u * scale, products, steps=steps, coef=coef, eps=0.0)
        assert _off(k.run(), _formula(_np(k.u), steps, 0.0, coef)) <= TOL[products], (steps, coef, scale)


@pytest.mark.parametrize("shift", [1, 3])
@pytest.mark.parametrize("r,c", [(40, 96), (96, 40)])
def test_arrays_of_any_alignment(cuda_lib, r, c, shift):
    import torch
    u = np.random.default_rng(4).standard_normal((2, r, c))
    for products, t in ((3, "f32"), (1, "bf16")):
        k = Case(torch, cuda_lib, u, products, t, t, shift=shift)
        assert _off(k.run(), _formula(_np(k.u))) <= TOL[products] + 2.0 ** -9


def test_nothing_in_nothing_out(cuda_lib):
    import torch
    u = np.random.default_rng(5).standard_normal((3, 20, 30))
    u[1] = 0.0
    k = Case(torch, cuda_lib, u, 3)
    got = k.run()
    assert (got[1] == 0).all() and _off(got[[0, 2]], _formula(_np(k.u))[[0, 2]]) <= TOL[3]
    k = Case(torch, cuda_lib, np.zeros((0, 20, 30)), 3)
    assert cuda_lib.sparse_orthogonalize(k.u, 0, 20, 30, k.cfg, k.out, None, k.err) == cuda_lib.OK


def test_a_value_that_is_not_finite_is_reported(cuda_lib):
    import torch
    for bad in (float("nan"), float("inf"), -float("inf")):
        u = np.random.default_rng(6).standard_normal((2, 20, 30))
        k = Case(torch, cuda_lib, u, 1)
        k.u[1, 3, 4] = bad
        k.run()
        assert int(k.err.item()) == cuda_lib.ERR_NON_FINITE


def test_equal_inputs_give_equal_bits_alone_in_a_batch_and_on_any_stream(cuda_lib):
    import torch
    u = np.random.default_rng(7).standard_normal((5, 150, 260))
    for products in (1, 3):
        k = Case(torch, cuda_lib, u, products)
        first = k.run()
        k.out.zero_()
        torch.cuda.synchronize()
        assert np.array_equal(first, k.run(stream=torch.cuda.Stream()))
        assert np.array_equal(first[2:3], Case(torch, cuda_lib, u[2:3], products).run())


def test_a_captured_call_gives_the_same_bits(cuda_lib):
    import torch
    for shape, products in (((1, 60, 90), 3), ((2, 300, 400), 1)):
        k = Case(torch, cuda_lib, np.random.default_rng(8).standard_normal(shape), products)
        first = k.run()
        s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            k.so.check(k.so.sparse_orthogonalize(k.u, k.b, k.r, k.c, k.cfg, k.out, k.ws, k.err, s))
        k.out.zero_()
        g.replay()
        k.G.check("replay")
        assert np.array_equal(first, _np(k.out))


class Step:
    def __init__(self, torch, so, batch, r, c, g_type="f32", nesterov=1, products=3, seed=0):
        rng = np.random.default_rng(seed)
        self.torch, self.so, self.shape = torch, so, (batch, r, c)
        self.G = G = Guarded(seed=r)
        self.w = G.array((0.1 * rng.standard_normal(self.shape)).astype(np.float32))
        self.buf = G.array(rng.standard_normal(self.shape).astype(np.float32))
        self.g = G.zeros(self.shape, {"f32": torch.float32, "bf16": torch.bfloat16}[g_type])
        self.rng = rng
        self.ws = G.empty(so.sparse_muon_workspace_size(batch, r, c, products), torch.uint8)
        self.err = G.error_word()
        self.cfg = so.MuonConfig(lr=0.02, momentum=0.95, weight_decay=0.1, scale=1.5, nesterov=nesterov,
                                 ns=so.NsConfig(a=NS[0], b=NS[1], c=NS[2], eps=1e-7, steps=5, products=products))

    def gradient(self):
        self.g.copy_(self.torch.from_numpy(self.rng.standard_normal(self.shape).astype(np.float32)))

    def run(self):
        self.so.check(self.so.sparse_muon_step(self.w, self.buf, self.g, *self.shape, self.cfg, self.ws, self.err))
        self.G.check("muon step")


@pytest.mark.parametrize("products", [1, 3])
@pytest.mark.parametrize("nesterov", [0, 1])
@pytest.mark.parametrize("batch,r,c,g_type", [(1, 40, 100, "f32"), (3, 130, 70, "bf16"), (1, 1, 9, "f32"),
                                              (2, 200, 200, "bf16")])
def test_muon_steps(cuda_lib, batch, r, c, g_type, nesterov, products):
    import torch
    k = Step(torch, cuda_lib, batch, r, c, g_type, nesterov, products)
    w, buf = _np(k.w), _np(k.buf)
    allowed = np.zeros_like(buf)
    for t in range(3):
        k.gradient()
        k.run()
        g = _np(k.g)
        # a step adds the rounding of the momentum (2^-24 of the old buffer's share) and of the sum
        allowed = 0.95 * allowed + 2.0 ** -23 * (np.abs(0.95 * buf) + np.abs(g))
        buf = 0.95 * buf + g
        assert (np.abs(_np(k.buf) - buf) <= allowed).all()
        # the step's own O, from the buffer it wrote
        o = _formula(g + 0.95 * _np(k.buf) if nesterov else _np(k.buf))
        before, w = w, (1 - 0.02 * 0.1) * w - 0.03 * o
        norm = np.sqrt((o * o).sum((1, 2)))
        err = np.sqrt(((_np(k.w) - w) ** 2).sum((1, 2)))
        size = np.sqrt((before ** 2).sum((1, 2))) + 0.03 * norm
        assert (err <= 0.03 * TOL[products] * norm + 2.0 ** -22 * size).all()
        w = _np(k.w)
    assert int(k.err.item()) == 0


def test_a_bad_gradient_or_a_set_error_word_changes_nothing(cuda_lib):
    import torch
    for case in ("nan", "set"):
        k = Step(torch, cuda_lib, 4, 50, 30)
        k.gradient()
        if case == "nan":
            k.g[3, 49, 29] = float("nan")
        else:
            k.err.fill_(cuda_lib.ERR_STEP_ORDER)
        w, buf = k.w.clone(), k.buf.clone()
        k.run()
        assert torch.equal(w, k.w) and torch.equal(buf, k.buf)
        assert int(k.err.item()) == (cuda_lib.ERR_NON_FINITE if case == "nan" else cuda_lib.ERR_STEP_ORDER)


def test_refusals(cuda_lib):
    import torch
    so = cuda_lib
    k = Case(torch, so, np.ones((1, 8, 8)), 3)

    def code(ws=k.ws, u=k.u, out=k.out, err=k.err, batch=1, r=8, c=8, **cfg):
        v = {**dict(a=NS[0], b=NS[1], c=NS[2], eps=1e-7, steps=5, products=3), **cfg}
        return so.sparse_orthogonalize(u, batch, r, c, so.NsConfig(**v), out, ws, err)

    assert code() == so.OK
    nan = float("nan")
    for bad in (dict(a=nan), dict(eps=-1.0), dict(eps=nan), dict(steps=0), dict(steps=65), dict(products=2),
                dict(a=8.0), dict(b=20.0), dict(r=0), dict(c=-1), dict(batch=-1), dict(r=1 << 21), dict(err=None)):
        assert code(**bad) == so.ERR_INVALID_ARG, bad
    assert code(ws=None) == so.ERR_WORKSPACE and code(ws=k.ws[:-1]) == so.ERR_WORKSPACE
    assert code(ws=k.ws[1:]) == so.ERR_WORKSPACE
    with pytest.raises(TypeError):
        code(u=k.u.double())
    s = Step(torch, so, 1, 8, 8)
    for name, value in (("lr", nan), ("momentum", -0.1), ("weight_decay", -1.0), ("scale", float("inf"))):
        cfg = so.MuonConfig.from_buffer_copy(s.cfg)
        setattr(cfg, name, value)
        assert so.sparse_muon_step(s.w, s.buf, s.g, 1, 8, 8, cfg, s.ws, s.err) == so.ERR_INVALID_ARG
    with pytest.raises(TypeError):
        so.sparse_muon_step(s.w.bfloat16(), s.buf, s.g, 1, 8, 8, s.cfg, s.ws, s.err)
    assert so.sparse_muon_workspace_size(1, 8, 8, 2) == 0 and so.sparse_muon_workspace_size(1, 0, 8, 1) == 0
    torch.cuda.synchronize()
    assert int(k.err.item()) == 0 and int(s.err.item()) == 0


FEW = [(1, 3664, 32), (1, 30, 8192), (1, 17, 831), (3, 831, 50), (59, 44, 860), (160, 32, 512), (2, 64, 4096),
       (1, 4090, 64), (5, 8190, 3), (40, 16, 2050)]


@pytest.mark.parametrize("kind", ["flat", "low rank", "decaying"])
@pytest.mark.parametrize("batch,r,c", FEW)
def test_few_long_rows(cuda_lib, batch, r, c, kind):
    """Rows whose columns lie in parts below one another, in one block and in clusters."""
    import torch
    u = _spectrum(np.random.default_rng(r + c), batch, r, c, kind)
    k = Case(torch, cuda_lib, u, 3)
    got = k.run()
    assert int(k.err.item()) == 0
    assert _off(got, _formula(_np(k.u))) <= TOL[3]
    k.out.zero_()
    assert np.array_equal(got, k.run())
    k = Case(torch, cuda_lib, u[:1], 1, "bf16", "bf16", shift=1)
    assert _off(k.run(), _formula(_np(k.u))) <= TOL[3] + 2.0 ** -9


@pytest.mark.parametrize("batch,r,c,g_type", [(70, 24, 700, "f32"), (3, 1001, 40, "bf16"), (1, 60, 4000, "bf16")])
def test_muon_steps_of_few_long_rows(cuda_lib, batch, r, c, g_type):
    test_muon_steps(cuda_lib, batch, r, c, g_type, 1, 3)
