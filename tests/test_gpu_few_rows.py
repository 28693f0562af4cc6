"""Few fp32 rows against matrices that would have to be packed: read where they lie.  Sums are plain fp32 ones here: a lane adds up k / 8 or k / 8 products in order, some tens of partial sums come after, so an element is off by at most
(k / 8 + 60) 2^-24 of the sum of its terms' sizes.  (More rows, and bf16: as in test_gpu_expert_matmul.)"""
import numpy as np
import pytest

from test_gpu_expert_matmul import Case as Products
from test_gpu_vocab_loss import Case as Loss

pytestmark = pytest.mark.gpu

E24, BF = 2.0 ** -24, 2.0 ** -8


def _np(t):
    return t.detach().double().cpu().numpy()


# both sides of the row count from which the tensor unit takes over; everything in one expert, or nothing in most
@pytest.mark.parametrize("kind,dw", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("a,b", [(1, 1), (3, 5), (64, 128), (515, 771), (1029, 33), (36, 4100), (4100, 36)])
@pytest.mark.parametrize("counts", [[1], [0, 3, 0], [16], [17], [61], [62], [1] * 30 + [0] * 70 + [2] * 10, [0, 40, 1, 0, 7]],
                         ids=lambda c: "-".join(map(str, c[:4])))
def test_products(cuda_lib, counts, a, b, kind, dw):
    import torch
    t = Products(torch, cuda_lib, counts, a, b, kind, dw=dw)       # 3 rows more that belong to none
    t.run()
    t.check()
    x, dy, w = _np(t.x), _np(t.dy), _np(t.w)
    live = t.bounds[-1]
    assert not _np(t.y)[live:].any() and not _np(t.dx)[live:].any()
    for e in range(len(counts)):
        s = slice(t.bounds[e], t.bounds[e + 1])
        for got, p, q, k, out in ((t.y[s], x[s], w[e], a, t.y), (t.dx[s], dy[s], w[e].T, b, t.dx), (t.dw[e], x[s].T, dy[s], counts[e], t.dw)):
            ref, size = p @ q, np.abs(p) @ np.abs(q)
            few = kind == "f32" and t.n <= 64 and t.n <= 16 * len(counts)
            bound = (k / 8 + 60 if few else 17 * (k / 16 + 1) if out.dtype == torch.bfloat16 else 34 * 17 + k / 512 + 8) * E24 * size
            assert (np.abs(_np(got) - ref) <= bound + (BF * np.abs(ref) if out.dtype == torch.bfloat16 else 0.0)).all()


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("n", [1, 5, 16, 17, 32, 33])
@pytest.mark.parametrize("c,v", [(1, 3), (7, 127), (64, 5000), (515, 1000), (1028, 129), (2050, 300)])
def test_loss(cuda_lib, n, c, v, shift):
    import torch
    t = Loss(torch, cuda_lib, n, c, v, "f32", shift=shift)
    t.run()
    t.check()
    t.compare()


def test_equal_bits_and_bad_offsets(cuda_lib):
    import torch
    so = cuda_lib
    t = Products(torch, so, [5, 0, 9], 100, 300, "f32")
    t.run()
    first = [p.clone() for p in (t.y, t.dx, t.dw)]
    for p in (t.y, t.dx, t.dw):
        p.fill_(3.0)
    t.run()
    t.check()
    assert all(torch.equal(p, q) for p, q in zip(first, (t.y, t.dx, t.dw)))
    for bad in ([0, 5, 3, 14], [0, -1, 5, 14], [1, 5, 5, 14], [0, 5, 5, 1 << 33]):
        t.offsets.copy_(torch.tensor(bad, device="cuda"))
        for call in (lambda: so.sparse_expert_matmul(t.x, t.w, t.n, 100, 300, 0, t.offsets, 3, t.y, t.ws, t.err),
                     lambda: so.sparse_expert_matmul(t.dy, t.w, t.n, 100, 300, 1, t.offsets, 3, t.dx, t.ws, t.err),
                     lambda: so.sparse_expert_matmul_grad(t.x, t.dy, t.n, 100, 300, t.offsets, 3, t.dw, t.ws, t.err)):
            t.err.zero_()
            assert call() == so.OK
            t.G.check("bad offsets")
            assert int(t.err.item()) == so.ERR_INDEX_OUT_OF_RANGE


def test_targets_that_are_no_rows(cuda_lib):
    import torch
    so = cuda_lib
    t = Loss(torch, so, 9, 20, 50, "f32")
    t.run()
    for bad in (-2, 50, 1 << 35):
        t.target[4] = bad
        for part in (0, 1):
            t.err.zero_()
            if part == 0:
                so.check(so.sparse_vocab_loss(t.x, t.w, 9, 20, 50, t.target, t.loss, t.lse, t.ws, t.err))
            else:
                so.check(so.sparse_vocab_loss_grad(t.dloss, t.x, t.w, 9, 20, 50, t.target, t.lse, t.dx, t.dw, t.ws, t.err))
            t.G.check("bad target")
            assert int(t.err.item()) == so.ERR_INDEX_OUT_OF_RANGE


# both sides of every count of tokens that changes the kernels of the loss or of its gradient
@pytest.mark.parametrize("n", [2, 3, 4, 8, 9, 12])
@pytest.mark.parametrize("c,v", [(1, 1), (33, 4097), (64, 70001), (515, 20000), (1100, 640), (4100, 257)])
def test_few_tokens_there_and_back(cuda_lib, n, c, v):
    import torch
    for shift in (0, 1):
        t = Loss(torch, cuda_lib, n, c, v, "f32", shift=shift)
        t.run()
        t.check()
        if v > 1:
            t.compare()
            continue
        # A table of one row: every result is 0, and no share of its norm a bound.  The gradient's score may be added up in another order
        # than lse's, so p = exp(z - lse) is off by the errors of both, twice the first term, and by the exponential's own, the second.
        x, w, lse, d = _np(t.x), _np(t.w), _np(t.lse), _np(t.dloss)
        near = 2 * 560 * E24 * np.abs(x @ w.T) + (16 + np.abs(lse[:, None])) * 4 * E24
        far = d[:, None] * near
        assert (np.abs(_np(t.dx)) <= far @ np.abs(w)).all() and (np.abs(_np(t.dw)) <= far.T @ np.abs(x)).all()
        assert (np.abs(_np(t.loss)) <= near[:, 0]).all()      # lse less the score, off by as much


@pytest.mark.parametrize("n", [1, 3, 7])
@pytest.mark.parametrize("c,v", [(40, 905), (515, 3001)])
def test_few_tokens_results_one_by_one_masked_and_captured(cuda_lib, n, c, v):
    """dx and dw alone are those of both together; a token that does not count leaves nothing, whatever its row holds; two graphs share a
    workspace; equal inputs give equal bits."""
    import torch
    so = cuda_lib
    g = torch.Generator(device="cuda").manual_seed(n)
    x, w = torch.randn(n, c, device="cuda", generator=g), torch.randn(v, c, device="cuda", generator=g) * c ** -0.5
    target, dloss = torch.randint(0, v, (n,), device="cuda", generator=g), torch.rand(n, device="cuda", generator=g) + 0.5
    target[n // 2] = -1
    x[n // 2], dloss[n // 2] = 0.0, float("nan")
    ws = torch.empty(so.sparse_vocab_loss_workspace_size(x.dtype, n, c, v, True), dtype=torch.uint8, device="cuda")
    err = so.error_word()

    def run(x, dx, dw):
        loss, lse = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
        so.check(so.sparse_vocab_loss(x, w, n, c, v, target, loss, lse, ws, err))
        so.check(so.sparse_vocab_loss_grad(dloss, x, w, n, c, v, target, lse, dx, dw, ws, err))

    dx, dw = torch.empty_like(x), torch.empty_like(w)
    run(x, dx, dw)
    z = x.double() @ w.double().T
    p = torch.exp(z - torch.logsumexp(z, 1, keepdim=True))
    live = target >= 0
    p[torch.arange(n, device="cuda")[live], target[live]] -= 1.0
    p = torch.where(live[:, None], p * dloss.double()[:, None], 0.0)
    # slopes: 2^-19 of their scores' exponentials at the most; sums of v and of n terms
    for got, ref, terms in ((dx, p @ w.double(), p.abs() @ w.double().abs()), (dw, p.T @ x.double(), p.abs().T @ x.double().abs())):
        assert bool(((got.double() - ref).abs() <= (v / 8 + 60) * E24 * terms + 2.0 ** -19 * terms).all())
    dirty = x.clone()
    dirty[n // 2] = float("nan")
    one, two = torch.full_like(dx, 3.0), torch.full_like(dw, 3.0)
    run(dirty, one, None)
    run(dirty, None, two)
    assert torch.equal(one, dx) and torch.equal(two, dw) and not one[n // 2].any()
    graphs, outs = [], []
    for _ in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        outs.append((torch.empty_like(dx), torch.empty_like(dw)))
        with torch.cuda.graph(graphs[-1]):
            run(dirty, *outs[-1])
    for _ in range(3):
        for q in graphs:
            q.replay()
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    assert all(torch.equal(a, b) for o in outs for a, b in zip(o, (dx, dw)))
