"""Newton-Schulz and the Muon step where they can go wrong: matrices without a norm or with a tiny one,
values that are not finite and set error words on the path of matrices that no cluster holds, blocks that
work on several tiles, long sums, arrays past 2^31 elements.

Bounds, in the Frobenius norm relative to the result's.  A 64-bit simulation of the kernels' splits
and roundings is off by at most 2.6e-3 with one product and 3.6e-5 with three over flat, decaying,
low-rank and rank-one spectra, the largest of both for rank one (fp32 products: 1e-4); over the flat
ones used here, 1.5e-3 and 5e-7.  Asserted: 5e-3 and 2e-5, as fp32 accumulation adds to both.  The unit
rounds every one of K / 16 sums towards zero, by at most 2^-23 of it: with one product A is smaller by
up to K 2^-27 of itself.  The result moves by at most twice that (x (a + b x^2 + c x^4) by
|b x^3 + 2 c x^5| <= 1.3 for x up to 1.13, and later steps do not enlarge it about their fixed points).
Rounding to bf16 adds 2^-9."""
import pytest

from gpu_harness import Guarded

pytestmark = pytest.mark.gpu

NS = (3.4445, -4.7750, 2.0315)
TOL = {1: 5e-3, 3: 2e-5}
DTYPES = {"f32": "float32", "bf16": "bfloat16"}


def _formula(torch, u, eps=1e-7, steps=5):
    """In 64 bits, on the device, by plain products."""
    a, b, c = NS
    u = u.double()
    tall = u.shape[1] > u.shape[2]
    x = u.transpose(1, 2) if tall else u
    norm = (x * x).sum((1, 2), keepdim=True).sqrt() + eps
    x = torch.where(norm > 0, x / norm, torch.zeros_like(x))
    for _ in range(steps):
        g = x @ x.transpose(1, 2)
        x = a * x + (b * g + c * (g @ g)) @ x
    return x.transpose(1, 2) if tall else x


def _off(got, ref):
    d = (got.double() - ref).square().sum((1, 2)).sqrt()
    return float((d / ref.square().sum((1, 2)).sqrt().clamp_min(1e-30)).max())


class Case:
    def __init__(self, torch, so, u, products, out_type="f32", eps=1e-7, shift=0, guarded=True):
        self.torch, self.so, self.shape = torch, so, tuple(u.shape)
        self.u = u
        self.G = G = Guarded(seed=u.shape[1])
        dt = getattr(torch, DTYPES[out_type])
        self.out = G.zeros(u.numel() + shift, dt)[shift:].view(u.shape) if guarded else torch.zeros(u.shape, dtype=dt, device="cuda")
        size = so.sparse_muon_workspace_size(*self.shape, products)
        self.ws = G.empty(size, torch.uint8) if guarded else torch.empty(size, dtype=torch.uint8, device="cuda")
        self.ws.fill_(255)
        self.err = G.error_word()
        self.cfg = so.NsConfig(a=NS[0], b=NS[1], c=NS[2], eps=eps, steps=5, products=products)

    def run(self):
        self.so.check(self.so.sparse_orthogonalize(self.u, *self.shape, self.cfg, self.out, self.ws, self.err))
        self.G.check("orthogonalize")
        return self.out


class Step:
    def __init__(self, torch, so, shape, g_type="f32", products=3, eps=1e-7, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.torch, self.so, self.shape = torch, so, shape
        self.G = G = Guarded(seed=shape[1])
        rand = lambda: torch.randn(*shape, device="cuda", generator=gen)  # noqa: E731
        self.w, self.buf = G.zeros(shape), G.zeros(shape)
        self.w.copy_(0.1 * rand())
        self.buf.copy_(rand())
        self.g = G.zeros(shape, getattr(torch, DTYPES[g_type]))
        self.g.copy_(rand())
        self.ws = G.empty(so.sparse_muon_workspace_size(*shape, products), torch.uint8)
        self.err = G.error_word()
        self.cfg = so.MuonConfig(lr=0.02, momentum=0.95, weight_decay=0.1, scale=1.5, nesterov=1,
                                 ns=so.NsConfig(a=NS[0], b=NS[1], c=NS[2], eps=eps, steps=5, products=products))

    def run(self, err=None, stream=None):
        self.so.check(self.so.sparse_muon_step(self.w, self.buf, self.g, *self.shape, self.cfg, self.ws,
                                               self.err if err is None else err, stream))


def _randn(torch, shape, seed=0, dtype="f32"):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, device="cuda", generator=g).to(getattr(torch, DTYPES[dtype]))


# of a cluster; of the general path: wide, tall, wide with odd rows, tall with odd rows
PATHS = [(3, 20, 30), (3, 300, 400), (3, 400, 300), (3, 201, 333), (3, 333, 201)]


@pytest.mark.parametrize("products", [1, 3])
@pytest.mark.parametrize("eps", [0.0, 1e-38, 1e-60, 1e-7])
@pytest.mark.parametrize("shape", PATHS)
def test_a_matrix_of_zeros_gives_zeros(cuda_lib, shape, eps, products):
    import torch
    u = _randn(torch, shape)
    u[1] = 0.0
    k = Case(torch, cuda_lib, u, products, eps=eps)
    got = k.run()
    assert int(k.err.item()) == 0 and (got[1] == 0).all()
    assert _off(got, _formula(torch, u, eps)) <= TOL[products]


@pytest.mark.parametrize("products", [1, 3])
@pytest.mark.parametrize("shape", PATHS)
def test_a_norm_whose_square_fp32_cannot_hold(cuda_lib, shape, products):
    """Down to values below the normal range; norms on both sides of 2^-40, where the sums change over."""
    import torch
    for scale, eps in ((1e-24, 0.0), (1e-24, 1e-30), (1e-24, 1e-23), (1e-30, 1e-40), (1e-36, 0.0), (1e-20, 0.0), (3e-15, 0.0),
                       (1e-14, 1e-14), (1e-12, 0.0)):
        u = _randn(torch, shape) * scale
        k = Case(torch, cuda_lib, u, products, eps=eps)
        got = k.run()
        assert int(k.err.item()) == 0
        assert _off(got, _formula(torch, u, eps)) <= TOL[products], (scale, eps)


@pytest.mark.parametrize("products", [1, 3])
@pytest.mark.parametrize("shape", PATHS)
def test_a_step_without_gradient_only_decays(cuda_lib, shape, products):
    import torch
    k = Step(torch, cuda_lib, shape, products=products, eps=0.0)
    k.g.zero_()
    k.buf[1] = 0.0
    k.g[2].copy_(_randn(torch, shape)[2] * 1e-24)
    k.buf[2] = 0.0
    w = k.w.double()
    k.run()
    k.G.check("muon step")
    assert int(k.err.item()) == 0 and (k.buf[1] == 0).all()
    keep = 1 - 0.02 * 0.1
    assert float((k.w[1].double() - keep * w[1]).abs().max()) <= 2.0 ** -23 * float(w[1].abs().max())
    o = _formula(torch, k.g.double() + 0.95 * k.buf.double(), 0.0)[2]
    off = (k.w[2].double() - (keep * w[2] - 0.03 * o)).norm()
    assert float(off) <= 0.03 * TOL[products] * float(o.norm()) + 2.0 ** -22 * float(w[2].norm() + 0.03 * o.norm())


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("products", [1, 3])
@pytest.mark.parametrize("shape", PATHS)
def test_a_bad_value_or_a_set_word_leaves_the_weights(cuda_lib, shape, products, bad):
    import torch
    so = cuda_lib
    k = Case(torch, so, _randn(torch, shape), products)
    k.u[2, -1, -1] = bad
    k.run()
    assert int(k.err.item()) == so.ERR_NON_FINITE
    for g_type in ("f32", "bf16"):
        for what in ("value", "word"):
            k = Step(torch, so, shape, g_type, products)
            w, buf = k.w.clone(), k.buf.clone()
            if what == "value":
                k.g[0, 1, 2] = bad
            else:
                k.err.fill_(so.ERR_STEP_ORDER)
            k.run()
            k.G.check("muon step")
            assert torch.equal(w, k.w) and torch.equal(buf, k.buf)
            assert int(k.err.item()) == (so.ERR_NON_FINITE if what == "value" else so.ERR_STEP_ORDER)


@pytest.mark.parametrize("shape,products", [((2000, 64, 128), 3), ((1, 1500, 1500), 3), ((6, 1000, 1100), 1), ((1, 1600, 700), 1)])
def test_a_word_set_while_a_step_runs_stops_all_of_it_or_nothing(cuda_lib, shape, products):
    """Another stream copies an error into the word at some moment: the step is whole or has not been."""
    import torch
    so = cuda_lib
    k = Step(torch, so, shape, products=products)
    w0, buf0 = k.w.clone(), k.buf.clone()
    k.run()
    torch.cuda.synchronize()
    t0, t1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    k.w.copy_(w0), k.buf.copy_(buf0)
    t0.record()
    k.run()
    t1.record()
    torch.cuda.synchronize()
    w1, buf1 = k.w.clone(), k.buf.clone()
    cycles = int(t0.elapsed_time(t1) * 1.9e6 * 1.2)
    word = torch.full((1,), so.ERR_STEP_ORDER, dtype=torch.int32).pin_memory()
    main, other = torch.cuda.Stream(), torch.cuda.Stream()
    seen = set()
    for i in range(60):
        k.w.copy_(w0), k.buf.copy_(buf0), k.err.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(other):
            torch.cuda._sleep(max(1, cycles * i // 60))
            k.err.copy_(word, non_blocking=True)
        k.run(stream=main)
        torch.cuda.synchronize()
        whole = torch.equal(k.w, w1) and torch.equal(k.buf, buf1)
        assert whole or (torch.equal(k.w, w0) and torch.equal(k.buf, buf0)), i
        seen.add(whole)
    k.G.check("muon step")
    assert True in seen


def _shape(kind, m, n, k, batch, sms):
    """Blocks to a tile, parts of its inner dimension, columns; tiles; blocks or pairs that share them: the
    cheapest by the kernels' rule, for one product."""
    sym = kind != "update"
    best = None
    chunks = -(-k // 64)
    for pair, split, bn in ((2, 1, 256), (2, 1, 128), (1, 1, 128), (1, 1, 64), (1, 2, 128), (1, 4, 128)):
        units, tm = sms // (pair * split), 128 * pair
        tiles = batch * (sum((i * tm + tm - 1) // bn + 1 for i in range(-(-m // tm))) if sym else -(-m // tm) * -(-n // bn))
        if split > 1 and (tiles > units or chunks < 2 * split):
            continue
        stage = 8192 * (2 + bn // pair // 64)
        cost = -(-tiles // units) * -(-chunks // split) * max(2 * bn, stage // 80) + (6000 if split > 1 else 0)
        if best is None or cost < best[0]:
            best = cost, (pair, split, bn), tiles, units
    return best[1:]


# one product: tiles of 256 columns and of 128, by pairs and alone, three epilogue groups (inner
# dimension below 1024) and two, several tiles a block, remainders in rows and columns, tall ones
TILES = [(16, 760, 2040), (1, 3001, 4090), (1, 4090, 4100), (1, 4100, 3001), (20, 1000, 1001), (6, 1000, 1100), (1, 1500, 2300),
         (2, 3000, 1400), (8, 520, 1500), (40, 300, 1100), (12, 700, 500), (2, 200, 20000), (30, 129, 4000)]


def test_the_shapes_reach_every_kind_of_tile(cuda_lib):
    import torch
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    reached = set()
    for batch, r, c in TILES:
        m, n = min(r, c), max(r, c)
        for kind, cols, inner in (("gram", m, n), ("poly", m, m), ("update", n, m)):
            shape, tiles, units = _shape(kind, m, cols, inner, batch, sms)
            reached.add((kind, shape, inner < 1024 and shape[0] == 2, tiles > units))
    assert {("gram", (2, 1, 256), False, True), ("gram", (1, 1, 128), False, True), ("gram", (2, 1, 128), False, True),
            ("poly", (2, 1, 256), False, True), ("poly", (2, 1, 256), True, True), ("poly", (2, 1, 128), True, True),
            ("update", (2, 1, 256), False, True), ("update", (2, 1, 256), True, True),
            ("update", (2, 1, 128), True, True)} <= reached


@pytest.mark.parametrize("in_type,out_type", [("bf16", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("shape", TILES)
def test_blocks_with_several_tiles(cuda_lib, shape, in_type, out_type):
    import torch
    u = _randn(torch, shape, dtype=in_type)
    k = Case(torch, cuda_lib, u, 1, out_type)
    got = k.run().clone()
    assert int(k.err.item()) == 0
    assert _off(got, _formula(torch, u)) <= TOL[1] + (2.0 ** -9 if out_type == "bf16" else 0.0)
    k.out.zero_()
    assert torch.equal(got, k.run())


@pytest.mark.parametrize("shape", [(16, 760, 2040), (1, 4100, 3001), (20, 1000, 1001)])
@pytest.mark.parametrize("g_type,products", [("bf16", 1), ("f32", 3)])
def test_steps_of_blocks_with_several_tiles(cuda_lib, shape, g_type, products):
    import torch
    k = Step(torch, cuda_lib, shape, g_type, products)
    w, buf = k.w.double(), k.buf.double()
    k.run()
    k.G.check("muon step")
    assert int(k.err.item()) == 0
    g = k.g.double()
    new = 0.95 * buf + g
    assert ((k.buf.double() - new).abs() <= 2.0 ** -23 * (0.95 * buf.abs() + g.abs())).all()
    o = _formula(torch, g + 0.95 * k.buf.double())
    norm = lambda t: t.square().sum((1, 2)).sqrt()  # noqa: E731
    off = norm(k.w.double() - ((1 - 0.02 * 0.1) * w - 0.03 * o))
    assert (off <= 0.03 * TOL[products] * norm(o) + 2.0 ** -22 * (norm(w) + 0.03 * norm(o))).all()


@pytest.mark.parametrize("shape", [(1, 200, 131072), (1, 1 << 18, 130), (1, 140, 1 << 20)])
def test_one_product_over_long_rows(cuda_lib, shape):
    """The drift of sums that are rounded towards zero, K 2^-27 of A and at most twice that of the result."""
    import torch
    u = _randn(torch, shape)
    k = Case(torch, cuda_lib, u, 1)
    got = k.run()
    assert int(k.err.item()) == 0
    assert _off(got, _formula(torch, u)) <= TOL[1] + 2 * max(shape) * 2.0 ** -27


@pytest.mark.parametrize("shift", [1, 2])
@pytest.mark.parametrize("shape", [(2, 300, 402), (2, 402, 300), (2, 302, 400), (2, 130, 1001)])
def test_arrays_of_any_alignment_past_a_cluster(cuda_lib, shape, shift):
    import torch
    for products, t in ((1, "bf16"), (3, "f32")):
        base = _randn(torch, (shape[0] * shape[1] * shape[2] + shift,), dtype=t)
        u = base[shift:].view(shape)
        k = Case(torch, cuda_lib, u, products, t, shift=shift)
        got = k.run()
        assert _off(got, _formula(torch, u)) <= TOL[products] + (2.0 ** -9 if t == "bf16" else 0.0)


@pytest.mark.parametrize("shape,products", [((33000, 256, 256), 1), ((265000, 64, 128), 3)])
def test_elements_past_2_31(cuda_lib, shape, products):
    import torch
    free, _ = torch.cuda.mem_get_info()
    if free < 100 << 30:
        pytest.skip("needs 100 GB")
    u = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    assert u.numel() > 1 << 31
    for i in range(0, shape[0], 8192):
        u[i:i + 8192] = _randn(torch, u[i:i + 8192].shape, seed=i, dtype="bf16")
    k = Case(torch, cuda_lib, u, products, "bf16", guarded=False)
    got = k.run()
    assert int(k.err.item()) == 0
    last = shape[0]
    for i in (0, last // 2, last - 3):
        assert _off(got[i:i + 3], _formula(torch, u[i:i + 3])) <= TOL[products] + 2.0 ** -9
    del k, got, u
    torch.cuda.empty_cache()
