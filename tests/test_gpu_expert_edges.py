"""The dot products of combine's gradient where their sums are longest and of one sign, so that every
rounding goes the same way: a warp has a token, a lane adds up to c / 32 + 8 products in fp32 one after the
other, then come 5 shuffle levels, so a product is off by at most (c / 32 + 13) u sum|dy ys|, u = 2^-24."""
import numpy as np
import pytest

from test_gpu_expert import U, Case, _np

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("n,k,c", [(40, 3, 5000), (7, 2, 20001), (9, 9, 4098), (300, 1, 3), (2, 4, 65536)])
def test_long_dot_products_of_one_sign(cuda_lib, n, k, c, kind):
    import torch
    rng = np.random.default_rng(c)
    t = Case(torch, cuda_lib, rng.integers(-1, 6, (n, k)), 6, c, kind)
    t.dy.copy_(torch.from_numpy(rng.random((n, c)).astype(np.float32)))
    t.ys.copy_(torch.from_numpy(rng.random((n * k, c)).astype(np.float32)))
    t.run()
    t.G.check("experts")
    assert int(t.err.item()) == 0
    pos, dy, ys, dw = t.pos.cpu().numpy(), _np(t.dy), _np(t.ys), _np(t.dw)
    for i in range(n):
        for j in range(k):
            if pos[i, j] < 0:
                assert dw[i, j] == 0.0
                continue
            ref = (dy[i] * ys[pos[i, j]]).sum()
            assert abs(dw[i, j] - ref) <= (c / 32 + 13) * U * ref
