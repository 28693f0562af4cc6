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
