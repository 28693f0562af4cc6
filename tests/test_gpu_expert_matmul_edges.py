"""The experts' products where they can go wrong: tiles by pairs of blocks, rows that are not finite, offsets that
are none, arrays past 2^31 elements, values at the ends of fp32, other streams, captured graphs, equal bits.
Bounds as in test_gpu_expert_matmul, against products in 64 bits on the GPU."""
import numpy as np
import pytest

from gpu_harness import Guarded

pytestmark = pytest.mark.gpu

E24, BF = 2.0 ** -24, 2.0 ** -8


def _near(torch, got, x, y, dtype, where=""):
    """got against x @ y in 64 bits."""
    x, y = x.double(), y.double()
    ref, size, k = x @ y, x.abs() @ y.abs(), x.shape[1]
    off = (got.double() - ref).abs()
    if dtype == torch.float32:
        bound = (34 * 17 + k / 512 + 8) * E24 * size
        assert float((got.double() - ref).norm()) <= 2.0 ** -19 * float(ref.norm()), where
    else:
        bound = 17 * (k / 16 + 1) * E24 * size + BF * ref.abs()
    assert bool((off <= bound).all()), where


def _call(torch, so, x, w, dy, offsets, ws=None, dw_type=None, err=None, stream=None):
    n, (e, a, b) = x.shape[0], w.shape
    ws = ws if ws is not None else torch.empty(so.sparse_expert_matmul_workspace_size(x.dtype, n, a, b, e), dtype=torch.uint8, device="cuda")
    err = err if err is not None else so.error_word()
    y, dx = torch.full((n, b), 7.0, dtype=x.dtype, device="cuda"), torch.full((n, a), 7.0, dtype=x.dtype, device="cuda")
    dw = torch.full((e, a, b), 7.0, dtype=dw_type or x.dtype, device="cuda")
    so.check(so.sparse_expert_matmul(x, w, n, a, b, 0, offsets, e, y, ws, err, stream))
    so.check(so.sparse_expert_matmul(dy, w, n, a, b, 1, offsets, e, dx, ws, err, stream))
    so.check(so.sparse_expert_matmul_grad(x, dy, n, a, b, offsets, e, dw, ws, err, stream))
    return y, dx, dw, err


def _case(torch, counts, a, b, kind, seed=0, tail=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = {"f32": torch.float32, "bf16": torch.bfloat16}[kind]
    r = lambda *s: torch.randn(*s, device="cuda", generator=g).to(t)  # noqa: E731
    bounds = [0] + np.cumsum(counts).tolist()
    n = bounds[-1] + tail
    return r(n, a), r(len(counts), a, b), r(n, b), torch.tensor(bounds, device="cuda"), bounds


@pytest.mark.parametrize("kind,dw", [("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("counts,a,b", [([300, 0, 1, 257, 64, 63, 65, 511] * 5, 520, 1032), ([5000], 264, 8200), ([70] * 300, 256, 512),
                                        ([2000, 3000, 1], 2048, 1024)], ids=["ragged", "one", "many", "wide"])
def test_tiles_by_pairs(cuda_lib, counts, a, b, kind, dw):
    import torch
    x, w, dy, offsets, bounds = _case(torch, counts, a, b, kind, tail=5)
    x[bounds[-1]:] = float("inf")
    dy[bounds[-1]:] = float("nan")
    t = {"f32": torch.float32, "bf16": torch.bfloat16}[dw]
    y, dx, dw, err = _call(torch, cuda_lib, x, w, dy, offsets, dw_type=t)
    assert int(err.item()) == 0
    assert not y[bounds[-1]:].any() and not dx[bounds[-1]:].any()
    for e in range(len(counts)):
        s = slice(bounds[e], bounds[e + 1])
        _near(torch, y[s], x[s], w[e], y.dtype, f"y {e}")
        _near(torch, dx[s], dy[s], w[e].T, y.dtype, f"dx {e}")
        _near(torch, dw[e], x[s].T, dy[s], dw.dtype, f"dw {e}")
    again = _call(torch, cuda_lib, x, w, dy, offsets, dw_type=t)
    assert all(torch.equal(p, q) for p, q in zip((y, dx, dw), again[:3]))


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_what_is_not_finite_stays_where_it_belongs(cuda_lib, kind):
    import torch
    counts = [70, 64, 0, 130, 5]
    x, w, dy, offsets, b = _case(torch, counts, 96, 160, kind)
    x[75, 3], dy[140, 9], w[4, 7, 11] = float("nan"), float("inf"), float("nan")
    y, dx, dw, err = _call(torch, cuda_lib, x, w, dy, offsets)
    assert int(err.item()) == 0
    bad = ~torch.isfinite(y)
    assert bad[75].all() and bad[b[4]:, 11].all()
    bad[75] = False
    bad[b[4]:, 11] = False
    assert not bad.any()
    bad = ~torch.isfinite(dx)
    assert bad[140].all() and bad[b[4]:, 7].all()
    bad[140] = False
    bad[b[4]:, 7] = False
    assert not bad.any()
    bad = ~torch.isfinite(dw)
    assert bad[1, 3].all() and bad[3, :, 9].all()
    bad[1, 3] = False
    bad[3, :, 9] = False
    assert not bad.any()


def test_values_at_the_ends_of_fp32(cuda_lib):
    """Every value is three bf16 parts whatever its size: products of rows of very large and very small values, the bound
    element by element; values above bf16's largest are cut off and not infinite."""
    import torch
    x, w, dy, offsets, b = _case(torch, [100, 33], 200, 72, "f32")
    x *= torch.logspace(-18, 18, 200, device="cuda")
    w *= torch.logspace(15, -15, 200, device="cuda")[None, :, None]
    y = _call(torch, cuda_lib, x, w, dy, offsets)[0]
    for e in range(2):
        s = slice(b[e], b[e + 1])
        ref, size = x[s].double() @ w[e].double(), x[s].double().abs() @ w[e].double().abs()
        assert bool(((y[s].double() - ref).abs() <= (34 * 17 + 9) * E24 * size).all())
    x.zero_()
    w.zero_()
    x[0, 0], w[0, 0, 0], w[0, 0, 1] = 3.402e38, 1.0, 0.5
    y = _call(torch, cuda_lib, x, w, dy, offsets)[0]
    assert abs(float(y[0, 0]) / 3.402e38 - 1) < 1e-6 and abs(float(y[0, 1]) / 1.701e38 - 1) < 1e-6


@pytest.mark.parametrize("bad", [[0, 5, 3, 9], [0, -1, 3, 9], [0, 3, 5, 11], [1, 3, 5, 9], [0, 3, 5, 1 << 40]])
def test_offsets_that_are_none(cuda_lib, bad):
    import torch
    so = cuda_lib
    x, w, dy, _, _ = _case(torch, [3, 3, 4], 16, 24, "bf16")
    err = _call(torch, so, x, w, dy, torch.tensor(bad, device="cuda"))[3]
    assert int(err.item()) == so.ERR_INDEX_OUT_OF_RANGE


def test_no_rows(cuda_lib):
    import torch
    so = cuda_lib
    err, dw = so.error_word(), torch.full((3, 8, 16), 5.0, device="cuda")
    off = torch.zeros(4, dtype=torch.int64, device="cuda")
    x = torch.empty(0, 8, device="cuda")
    assert so.sparse_expert_matmul(x, dw, 0, 8, 16, 0, off, 3, torch.empty(0, 16, device="cuda"), None, err) == so.OK
    assert so.sparse_expert_matmul_grad(x, torch.empty(0, 16, device="cuda"), 0, 8, 16, off, 3, dw, None, err) == so.OK
    assert not dw.any()


@pytest.mark.parametrize("a,b", [(4096, 8), (8, 4096)])
def test_elements_past_32_bits(cuda_lib, a, b):
    import torch
    so = cuda_lib
    n = 530_000                                               # 2.17e9 values on one side
    x, dy = torch.zeros(n, a, dtype=torch.bfloat16, device="cuda"), torch.zeros(n, b, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    x[-300:].normal_(generator=g)
    dy[-300:].normal_(generator=g)
    w = torch.randn(2, a, b, device="cuda", generator=g).bfloat16()
    offsets = torch.tensor([0, n - 200, n], device="cuda")
    y, dx, dw, err = _call(torch, so, x, w, dy, offsets)
    assert int(err.item()) == 0
    for e, s in ((0, slice(n - 300, n - 200)), (1, slice(n - 200, n))):
        _near(torch, y[s], x[s], w[e], torch.bfloat16)
        _near(torch, dx[s], dy[s], w[e].T, torch.bfloat16)
        _near(torch, dw[e], x[s].T, dy[s], torch.bfloat16)
    assert not y[:n - 300].any() and not dx[:n - 300].any()


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_streams_and_graphs(cuda_lib, kind):
    """On another stream, captured, and two captured graphs with one workspace replayed in turn."""
    import torch
    so = cuda_lib
    x, w, dy, offsets, b = _case(torch, [300, 0, 17, 64], 264, 200, kind)
    first = _call(torch, so, x, w, dy, offsets)[:3]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = _call(torch, so, x, w, dy, offsets)[:3]
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(first, other))
    ws = torch.empty(so.sparse_expert_matmul_workspace_size(x.dtype, x.shape[0], 264, 200, 4), dtype=torch.uint8, device="cuda")
    err, graphs, outs = so.error_word(), [], []
    for _ in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(_call(torch, so, x, w, dy, offsets, ws=ws, err=err)[:3])
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    for o in outs:
        assert all(torch.equal(p, q) for p, q in zip(first, o))
    x.mul_(2.0)                                               # other inputs in the same place
    graphs[0].replay()
    assert torch.equal(outs[0][0].double(), 2 * first[0].double())


def test_workspace_refusals(cuda_lib):
    import torch
    so = cuda_lib
    x, w, dy, offsets, _ = _case(torch, [30, 40], 20, 24, "f32")
    size = so.sparse_expert_matmul_workspace_size(torch.float32, 70, 20, 24, 2)
    y, err = torch.empty(70, 24, device="cuda"), so.error_word()
    # the size is that of the three calls' largest: one call may need less, but none as little as this
    for ws in (None, torch.empty(255, dtype=torch.uint8, device="cuda"), torch.empty(size + 256, dtype=torch.uint8, device="cuda")[8:]):
        assert so.sparse_expert_matmul(x, w, 70, 20, 24, 0, offsets, 2, y, ws, err) == so.ERR_WORKSPACE
    G = Guarded()
    y = G.zeros((70, 24))
    ws = G.empty(size, torch.uint8)
    assert so.sparse_expert_matmul(x, w, 70, 20, 24, 0, offsets, 2, y, ws, err) == so.OK
    G.check("the least workspace")
