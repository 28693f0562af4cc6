"""The products of every expert's rows with its matrix, and their gradients, against plain numpy in 64 bits.

Bounds, with S = sum|x w| of an element.  The tensor unit adds 16 exact products of bf16 values and the running
sum at a time and cuts each off at 2^-24 of the largest at most: 17 2^-24 of S a step, K / 16 steps in a
run.  Runs are emptied into fp32 sums every 512 values (32 steps) where the result is fp32: a rounding of
2^-24 for each.  fp32 values are three bf16 parts, off by 2^-27 each, and products below 2^-25 are left
out; five products go to a second accumulator, below 2^-7 of the first.  So
  fp32 (and bf16 rows, fp32 result):  (34 17 + K / 512 + 8) 2^-24 S
  bf16 result:                        (17 K / 16) 2^-24 S + 2^-8 |y|
The first is far from what random signs leave, so the whole is held to 2^-19 of its norm as well: 32 steps
that lose 2^-24 of the running sum each are 2^-19, half of that where the sum grows evenly.
"""
import numpy as np
import pytest

from gpu_harness import Guarded

pytestmark = pytest.mark.gpu

E24, BF = 2.0 ** -24, 2.0 ** -8
COUNTS = [[0, 1, 5, 0, 33, 64, 65, 300], [1], [0], [0, 0, 0, 7], [256, 257, 255, 31, 32], [1000, 0, 129], [2] * 70]
SHAPES = [(1, 1), (8, 16), (64, 64), (515, 771), (128, 2048), (2048, 40), (40, 2056), (1032, 136), (7, 300)]


def _np(t):
    return t.detach().double().cpu().numpy()


class Case:
    def __init__(self, torch, so, counts, a, b, kind, dw="f32", tail=3, shift=0, seed=0, one_sign=False):
        rng = np.random.default_rng(seed)
        self.torch, self.so, self.a, self.b, self.experts = torch, so, a, b, len(counts)
        self.n = n = sum(counts) + tail
        self.bounds = np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)
        self.G = Guarded(seed=a + b)
        self.type = {"f32": torch.float32, "bf16": torch.bfloat16}[kind]
        self.shift = shift
        draw = (lambda *s: rng.random(s)) if one_sign else (lambda *s: rng.standard_normal(s))
        self.x, self.dy = self.typed(draw(n, a)), self.typed(draw(n, b))
        self.w = self.typed(draw(len(counts), a, b))
        self.y, self.dx = self.blank((n, b)), self.blank((n, a))
        self.dw = self.blank((len(counts), a, b), {"f32": torch.float32, "bf16": torch.bfloat16}[dw])
        for t in (self.y, self.dx, self.dw):
            t.fill_(9.0)
        live = self.bounds[-1]
        self.x[live:] = float("nan")     # nobody looks at these
        self.dy[live:] = float("nan")
        self.offsets = self.G.array(self.bounds)
        self.err = self.G.error_word()
        size = so.sparse_expert_matmul_workspace_size(self.type, n, a, b, len(counts), shift == 0)
        self.ws = self.G.empty(size, torch.uint8)
        self.ws.fill_(0xff)              # NaN to whoever reads what was not written

    def blank(self, shape, dtype=None):
        return self.G.zeros(int(np.prod(shape)) + self.shift, dtype or self.type)[self.shift:].view(shape)

    def typed(self, v):
        t = self.blank(v.shape)
        t.copy_(self.torch.from_numpy(np.ascontiguousarray(v, np.float32)))
        return t

    def run(self, stream=None):
        so, n, a, b, e = self.so, self.n, self.a, self.b, self.experts
        so.check(so.sparse_expert_matmul(self.x, self.w, n, a, b, 0, self.offsets, e, self.y, self.ws, self.err, stream))
        so.check(so.sparse_expert_matmul(self.dy, self.w, n, a, b, 1, self.offsets, e, self.dx, self.ws, self.err, stream))
        so.check(so.sparse_expert_matmul_grad(self.x, self.dy, n, a, b, self.offsets, e, self.dw, self.ws, self.err, stream))

    def check(self):
        self.G.check("expert matmul")
        assert int(self.err.item()) == 0

    def compare(self):
        x, dy, w = _np(self.x), _np(self.dy), _np(self.w)
        y, dx, dw = _np(self.y), _np(self.dx), _np(self.dw)
        live = self.bounds[-1]
        assert (y[live:] == 0).all() and (dx[live:] == 0).all()
        for e in range(self.experts):
            rows = slice(self.bounds[e], self.bounds[e + 1])
            self.near(y[rows], x[rows] @ w[e], np.abs(x[rows]) @ np.abs(w[e]), self.a, self.y.dtype)
            self.near(dx[rows], dy[rows] @ w[e].T, np.abs(dy[rows]) @ np.abs(w[e]).T, self.b, self.dx.dtype)
            self.near(dw[e], x[rows].T @ dy[rows], np.abs(x[rows]).T @ np.abs(dy[rows]), rows.stop - rows.start, self.dw.dtype)

    def near(self, got, ref, size, k, dtype):
        assert np.isfinite(got).all()
        if dtype == self.torch.float32:
            bound = (34 * 17 + k / 512 + 8) * E24 * size
            assert np.linalg.norm(got - ref) <= 2.0 ** -19 * np.linalg.norm(ref)
        else:
            bound = (17 * (k / 16 + 1)) * E24 * size + BF * np.abs(ref)
        assert (np.abs(got - ref) <= bound).all()


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("a,b", SHAPES)
@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: "-".join(map(str, c[:8])))
def test_products_and_gradients(cuda_lib, counts, a, b, kind):
    import torch
    t = Case(torch, cuda_lib, counts, a, b, kind)
    t.run()
    t.check()
    t.compare()


@pytest.mark.parametrize("a,b", [(64, 96), (333, 70), (512, 264)])
def test_bf16_matrix_gradients(cuda_lib, a, b):
    import torch
    t = Case(torch, cuda_lib, [5, 0, 700, 64], a, b, "bf16", dw="bf16")
    t.run()
    t.check()
    t.compare()


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_any_alignment(cuda_lib, kind):
    import torch
    t = Case(torch, cuda_lib, [5, 0, 200, 64], 72, 136, kind, shift=1)
    t.run()
    t.check()
    t.compare()


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("counts,a,b", [([4000, 3000], 64, 64), ([700], 8200, 24), ([9000], 16, 16), ([40], 20000, 8)])
def test_long_sums_of_one_sign(cuda_lib, counts, a, b, kind):
    """Every cut-off goes the same way; the inner dimension is split over blocks where there are few tiles."""
    import torch
    t = Case(torch, cuda_lib, counts, a, b, kind, one_sign=True)
    t.run()
    t.check()
    t.compare()
