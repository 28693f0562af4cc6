"""Tokens sorted by expert and back, against plain numpy.

The sort is whole numbers and dispatch copies: equal.  Combine adds k products in slot order in
fp32: its error is below (k + 1) u sum|w ys|, u = 2^-24.  A slot's dot product adds at most
8 ceil(c / 1024) values in a lane, then 5 shuffle levels and 8 warps: (8 ceil(c/1024) + 32) u sum|dy ys|.
A bf16 output is rounded once more: 2^-8 of its value.
"""
import numpy as np
import pytest

from gpu_harness import Guarded

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF = 2.0 ** -8
# n, k, experts, c, share of slots that go nowhere
CASES = [(1, 1, 1, 1, 0.0), (8, 4, 64, 2048, 0.0), (3, 2, 5, 7, 0.3), (1000, 8, 128, 33, 0.0), (4096, 1, 9, 40, 0.1),
         (4097, 1, 300, 16, 0.1), (1025, 4, 1024, 24, 0.2), (70000, 8, 256, 8, 0.01), (600, 3, 17, 5000, 0.5),
         (5, 13, 20, 96, 0.2), (300, 2, 4, 1111, 0.0)]


def _dt(torch, name):
    return {"f32": torch.float32, "bf16": torch.bfloat16}[name]


def _np(t):
    return t.detach().double().cpu().numpy()


def _sorted(expert, experts):
    flat = expert.reshape(-1)
    order = np.argsort(np.where(flat < 0, experts, flat), kind="stable")
    live = int((flat >= 0).sum())
    pos = np.full(flat.size, -1, np.int32)
    pos[order[:live]] = np.arange(live)
    src = np.full(flat.size, -1, np.int32)
    src[:live] = order[:live]
    counts = np.bincount(flat[flat >= 0], minlength=experts)
    return np.concatenate([[0], np.cumsum(counts)]), src, pos


class Case:
    def __init__(self, torch, so, expert, experts, c, kind, seed=0, shift=0):
        n, k = expert.shape
        rng = np.random.default_rng(seed)
        self.torch, self.so, self.n, self.k, self.experts, self.c = torch, so, n, k, experts, c
        self.G = G = Guarded(seed=n + c)
        self.shift = shift
        self.expert = G.array(expert.astype(np.int64))
        self.offsets, self.src = G.empty(experts + 1, torch.int64), G.empty(n * k, torch.int32)
        self.pos = G.empty((n, k), torch.int32)
        self.ws = G.empty(max(so.sparse_expert_workspace_size(n, k, experts), 256), torch.uint8)
        self.err = G.error_word()
        self.x, self.dy = self.typed(rng.standard_normal((n, c)), kind), self.typed(rng.standard_normal((n, c)), kind)
        self.ys = self.typed(rng.standard_normal((n * k, c)), kind)
        self.w = self.typed(rng.random((n, k)), "f32", 0)
        self.xs, self.dys = self.blank((n * k, c), kind), self.blank((n * k, c), kind)
        self.y, self.dx = self.blank((n, c), kind), self.blank((n, c), kind)
        self.dw = self.blank((n, k), "f32", 0)
        for t in (self.xs, self.dys, self.y, self.dx, self.dw):
            t.fill_(9.0)

    def blank(self, shape, kind, shift=None):
        shift = self.shift if shift is None else shift
        return self.G.zeros(int(np.prod(shape)) + shift, _dt(self.torch, kind))[shift:].view(shape)

    def typed(self, a, kind, shift=None):
        t = self.blank(a.shape, kind, shift)
        t.copy_(self.torch.from_numpy(np.ascontiguousarray(a, np.float32)))
        return t

    def run(self, weights=True, stream=None):
        so, n, k, e, c = self.so, self.n, self.k, self.experts, self.c
        w = self.w if weights else None
        so.check(so.sparse_expert_sort(self.expert, n, k, e, self.offsets, self.src, self.pos, self.ws, self.err, stream))
        so.check(so.sparse_expert_dispatch(self.x, n, k, c, self.pos, self.offsets, e, self.xs, self.err, stream))
        so.check(so.sparse_expert_combine(self.ys, n, k, c, self.pos, w, self.y, self.err, stream))
        so.check(so.sparse_expert_combine_grad(self.dy, self.ys, n, k, c, self.pos, self.offsets, e, w, self.dys,
                                               self.dw, self.err, stream))
        so.check(so.sparse_expert_combine(self.xs, n, k, c, self.pos, None, self.dx, self.err, stream))
        self.G.check("expert")

    def compare(self, weights=True):
        n, k, c = self.n, self.k, self.c
        offsets, src, pos = _sorted(self.expert.cpu().numpy(), self.experts)
        assert np.array_equal(self.offsets.cpu().numpy(), offsets)
        assert np.array_equal(self.src.cpu().numpy(), src)
        assert np.array_equal(self.pos.cpu().numpy().reshape(-1), pos)
        live = int(offsets[-1])
        x, dy, ys = _np(self.x), _np(self.dy), _np(self.ys)
        slots = src[:live]
        xs = np.zeros((n * k, c))
        xs[:live] = x[slots // k]
        assert np.array_equal(_np(self.xs), xs)
        w = _np(self.w).reshape(-1)[slots] if weights else np.ones(live)
        y, ay = np.zeros((n, c)), np.zeros((n, c))
        np.add.at(y, slots // k, ys[:live] * w[:, None])
        np.add.at(ay, slots // k, np.abs(ys[:live] * w[:, None]))
        b = BF if self.y.dtype == self.torch.bfloat16 else 0.0
        assert (np.abs(_np(self.y) - y) <= (k + 1) * U * ay + b * np.abs(y)).all()
        dys = np.zeros((n * k, c))
        dys[:live] = dy[slots // k] * w[:, None]
        assert (np.abs(_np(self.dys) - dys) <= (b + U) * np.abs(dys)).all()
        dw, aw = np.zeros(n * k), np.zeros(n * k)
        dw[slots] = (dy[slots // k] * ys[:live]).sum(1)
        aw[slots] = np.abs(dy[slots // k] * ys[:live]).sum(1)
        assert (np.abs(_np(self.dw).reshape(-1) - dw) <= (8 * -(-c // 1024) + 32) * U * aw).all()
        # dispatch's gradient of xs itself: x times the slots that it was copied to
        dx = x * (pos.reshape(n, k) >= 0).sum(1)[:, None]
        assert (np.abs(_np(self.dx) - dx) <= ((k + 1) * U + b) * np.abs(dx)).all()


def _experts(rng, n, k, experts, gone):
    e = rng.integers(0, experts, (n, k))
    e[rng.random((n, k)) < gone] = -1
    return e


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("n,k,experts,c,gone", CASES)
def test_there_and_back(cuda_lib, n, k, experts, c, gone, kind):
    import torch
    case = Case(torch, cuda_lib, _experts(np.random.default_rng(n + c), n, k, experts, gone), experts, c, kind)
    case.run()
    assert int(case.err.item()) == 0
    case.compare()


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("shift", [1, 3])
def test_arrays_of_any_alignment_without_weights(cuda_lib, shift, kind):
    import torch
    case = Case(torch, cuda_lib, _experts(np.random.default_rng(1), 77, 3, 6, 0.2), 6, 64, kind, shift=shift)
    case.run(weights=False)
    case.compare(weights=False)


@pytest.mark.parametrize("n,k", [(50, 3), (3000, 4)])
def test_one_expert_has_all_or_none(cuda_lib, n, k):
    import torch
    for e in (np.full((n, k), 7), np.full((n, k), -1)):
        case = Case(torch, cuda_lib, e, 8, 48, "bf16")
        case.run()
        assert int(case.err.item()) == 0
        case.compare()


def test_nothing_is_read_where_no_slot_is(cuda_lib):
    import torch
    e = np.array([[0, -1], [-1, -1], [1, 0]])
    case = Case(torch, cuda_lib, e, 2, 20, "f32")
    case.ys[3:] = float("nan")          # rows past the last sorted place
    case.w[1] = float("nan")            # weights of slots that go nowhere
    case.run()
    assert np.isfinite(_np(case.y)).all() and np.isfinite(_np(case.dys)).all() and np.isfinite(_np(case.dw)).all()
    assert (_np(case.y)[1] == 0).all() and (_np(case.dw)[1] == 0).all()


@pytest.mark.parametrize("n", [40, 5000])
def test_a_bad_expert_is_reported(cuda_lib, n):
    import torch
    for bad in (6, -2, 1 << 40):
        e = _experts(np.random.default_rng(2), n, 2, 6, 0.1)
        e[n // 2, 1] = bad
        case = Case(torch, cuda_lib, e, 6, 16, "f32")
        case.run()
        assert int(case.err.item()) == cuda_lib.ERR_INDEX_OUT_OF_RANGE


def test_a_bad_place_is_reported_and_not_followed(cuda_lib):
    import torch
    so = cuda_lib
    case = Case(torch, so, np.zeros((6, 2), np.int64), 1, 16, "f32")
    case.run()
    case.pos[3, 1] = 12
    case.pos[4, 0] = -5
    so.check(so.sparse_expert_combine(case.ys, 6, 2, 16, case.pos, None, case.y, case.err))
    so.check(so.sparse_expert_dispatch(case.x, 6, 2, 16, case.pos, case.offsets, 1, case.xs, case.err))
    case.G.check("bad place")
    assert int(case.err.item()) == so.ERR_INDEX_OUT_OF_RANGE


def test_elements_past_32_bits(cuda_lib):
    """2.4e9 sorted elements: rows of the first and the last expert."""
    import torch
    so = cuda_lib
    n, k, e, c = 300_000, 2, 3, 4000
    expert = torch.zeros(n, k, dtype=torch.int64, device="cuda")
    expert[:, 1] = 2
    x = torch.empty(n, c, dtype=torch.bfloat16, device="cuda").normal_()
    xs = torch.empty(n * k, c, dtype=torch.bfloat16, device="cuda")
    dxs, y = torch.empty_like(xs), torch.empty_like(x)
    offsets = torch.empty(e + 1, dtype=torch.int64, device="cuda")
    pos = torch.empty(n, k, dtype=torch.int32, device="cuda")
    w = torch.full((n, k), 0.5, device="cuda")
    ws = torch.empty(max(so.sparse_expert_workspace_size(n, k, e), 256), dtype=torch.uint8, device="cuda")
    err = so.error_word()
    so.check(so.sparse_expert_sort(expert, n, k, e, offsets, None, pos, ws, err))
    so.check(so.sparse_expert_dispatch(x, n, k, c, pos, offsets, e, xs, err))
    so.check(so.sparse_expert_combine(xs, n, k, c, pos, w, y, err))
    so.check(so.sparse_expert_combine_grad(x, xs, n, k, c, pos, offsets, e, w, dxs, None, err))
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and offsets.tolist() == [0, n, n, 2 * n]
    assert torch.equal(pos[:, 1], torch.arange(n, 2 * n, dtype=torch.int32, device="cuda"))
    for at in (slice(0, 5), slice(n - 5, n)):
        assert torch.equal(xs[at], x[at]) and torch.equal(xs[n:][at], x[at])
        assert torch.equal(y[at], x[at]) and torch.equal(dxs[n:][at], x[at] * 0.5)


def test_weights_gradient_against_differences(cuda_lib):
    """L = sum(dy * combine(ys, w)) is linear in w and in ys: the slope is exact up to rounding."""
    import torch
    e = _experts(np.random.default_rng(3), 30, 4, 5, 0.2)
    case = Case(torch, cuda_lib, e, 5, 64, "f32")
    case.run()
    rng = np.random.default_rng(4)
    ew, ey = rng.standard_normal((30, 4)), rng.standard_normal((120, 64))
    _, src, pos = _sorted(e, 5)
    ys, w, dy = _np(case.ys), _np(case.w), _np(case.dy)
    live = (pos >= 0).reshape(30, 4)

    def loss(s):
        rows = (ys + s * ey)[np.maximum(pos, 0)].reshape(30, 4, 64)
        return (dy[:, None] * rows * ((w + s * ew) * live)[:, :, None]).sum()

    slope = (loss(0.5) - loss(-0.5))         # the s^2 term cancels
    got = (_np(case.dw) * ew).sum() + (_np(case.dys) * ey).sum()
    size = np.abs(_np(case.dw) * ew).sum() + np.abs(_np(case.dys) * ey).sum()
    assert abs(got - slope) <= 64 * U * size


def test_equal_inputs_give_equal_bits_on_any_stream(cuda_lib):
    import torch
    case = Case(torch, cuda_lib, _experts(np.random.default_rng(6), 9000, 4, 60, 0.1), 60, 72, "bf16")
    case.run()
    outs = (case.pos, case.src, case.offsets, case.xs, case.y, case.dys, case.dw, case.dx)
    first = [t.clone() for t in outs]
    for t in outs:
        t.zero_()
    torch.cuda.synchronize()
    case.run(stream=torch.cuda.Stream())
    for a, b in zip(first, outs):
        assert torch.equal(a, b)


def test_refusals_and_no_tokens(cuda_lib):
    import torch
    so = cuda_lib
    case = Case(torch, so, np.zeros((4, 2), np.int64), 3, 16, "f32")
    ok = [case.expert, 4, 2, 3, case.offsets, case.src, case.pos, case.ws, case.err]

    def code(at, value):
        a = list(ok)
        a[at] = value
        return so.sparse_expert_sort(*a)

    assert so.sparse_expert_sort(*ok) == so.OK
    for at, value in ((1, -1), (1, 1 << 31), (2, 0), (3, 0), (3, 1025), (4, None), (6, None), (8, None)):
        assert code(at, value) == so.ERR_INVALID_ARG, (at, value)
    assert code(7, None) == so.ERR_WORKSPACE
    with pytest.raises(TypeError):
        code(0, case.expert.int())
    with pytest.raises(TypeError):
        so.sparse_expert_combine(case.ys, 4, 2, 16, case.pos, None, case.y.bfloat16(), case.err)
    assert so.sparse_expert_combine(case.ys, 4, 2, 0, case.pos, None, case.y, case.err) == so.ERR_INVALID_ARG
    assert so.sparse_expert_combine(case.ys, 4, 2, 16, None, None, case.y, case.err) == so.ERR_INVALID_ARG
    assert so.sparse_expert_dispatch(case.x, 4, 2, 16, case.pos, None, 3, case.xs, case.err) == so.ERR_INVALID_ARG
    assert so.sparse_expert_combine_grad(case.dy, case.ys, 4, 2, 16, case.pos, case.offsets, 0, None, case.dys, None,
                                         case.err) == so.ERR_INVALID_ARG
    assert so.sparse_expert_workspace_size(4, 2, 0) == 0 and so.sparse_expert_workspace_size(1 << 31, 2, 3) == 0
    case.offsets.fill_(5)
    assert so.sparse_expert_sort(None, 0, 2, 3, case.offsets, None, None, None, case.err) == so.OK
    assert so.sparse_expert_combine(case.ys, 0, 2, 16, None, None, case.y, case.err) == so.OK
    torch.cuda.synchronize()
    assert (case.offsets == 0).all() and int(case.err.item()) == 0


@pytest.mark.parametrize("n,experts", [(1000, 721), (1000, 722), (1500, 371), (1500, 372), (4096, 188), (4096, 189)])
def test_sorts_whose_counts_are_about_48_kb(cuda_lib, n, experts):
    """Dynamic and static shared memory together pass what a launch has without asking."""
    import torch
    case = Case(torch, cuda_lib, np.random.default_rng(n + experts).integers(-1, experts, (n, 1)), experts, 8, "f32")
    case.run()
    assert int(case.err.item()) == 0
    case.compare()
    assert cuda_lib.sparse_expert_workspace_size(n, 1, experts) > 0   # an array of this size has an address


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("c,shift", [(2, 0), (6, 0), (30, 0), (262, 0), (1030, 0), (64, 2), (1024, 2)])
def test_rows_of_pairs(cuda_lib, c, shift, kind):
    """Rows of an even number of values, or arrays aligned to two of them: accesses of two."""
    import torch
    case = Case(torch, cuda_lib, np.random.default_rng(c).integers(-1, 7, (210, 3)), 7, c, kind, shift=shift)
    case.run()
    assert int(case.err.item()) == 0
    case.compare()
