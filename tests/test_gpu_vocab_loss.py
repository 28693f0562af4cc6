"""Softmax cross entropy over a table's rows and its gradient, against plain numpy in 64 bits.

A score is a dot product as in the experts' products (test_gpu_expert_matmul): off by d = 560 2^-24 S, S = max
over rows of sum|x w|, at the most, and by 2^-20 of its norm as a rule.  lse is off by no more than its scores,
and by the exponentials and sums in fp32: (16 + |lse|) 2^-22.  loss by both.  A slope p - [t] is off by p times that;
with bf16 it is rounded to 2^-8 of its value, and the products' results once more.
"""
import numpy as np
import pytest

from gpu_harness import Guarded

pytestmark = pytest.mark.gpu

E24, BF = 2.0 ** -24, 2.0 ** -8
SIZES = [(1, 8, 5), (3, 64, 1000), (256, 128, 5000), (130, 515, 777), (1000, 72, 300), (16, 2048, 2000), (300, 33, 4100),
         (2, 1, 1), (129, 64, 20000), (700, 136, 3000), (513, 100, 40001), (1, 128, 70000), (2100, 64, 129)]


def _np(t):
    return t.detach().double().cpu().numpy()


class Case:
    def __init__(self, torch, so, n, c, v, kind, seed=0, shift=0, std=1.0):
        rng = np.random.default_rng(seed + n)
        self.torch, self.so, self.n, self.c, self.v = torch, so, n, c, v
        self.type = {"f32": torch.float32, "bf16": torch.bfloat16}[kind]
        self.G, self.shift = Guarded(seed=n + c), shift
        self.x, self.w = self.typed(rng.standard_normal((n, c))), self.typed(rng.standard_normal((v, c)) * std * 1.5 / np.sqrt(c))
        target = rng.integers(0, v, n)
        target[rng.random(n) < 0.2] = -1
        if n > 3:
            target[0], target[1], target[2] = 0, v - 1, v - 1
        self.target = self.G.array(target.astype(np.int64))
        self.dloss = self.G.array(rng.random(n).astype(np.float32) / n)
        self.loss, self.lse = self.G.array(np.full(n, 7.0, np.float32)), self.G.array(np.full(n, 7.0, np.float32))
        self.dx, self.dw = self.blank((n, c)), self.blank((v, c))
        self.dx.fill_(9.0)
        self.dw.fill_(9.0)
        self.err = self.G.error_word()
        self.ws = self.G.empty(so.sparse_vocab_loss_workspace_size(self.type, n, c, v, True, shift == 0), torch.uint8)
        self.ws.fill_(0xff)

    def blank(self, shape):
        return self.G.zeros(int(np.prod(shape)) + self.shift, self.type)[self.shift:].view(shape)

    def typed(self, a):
        t = self.blank(a.shape)
        t.copy_(self.torch.from_numpy(np.ascontiguousarray(a, np.float32)))
        return t

    def run(self, dloss=True, stream=None):
        so, n, c, v = self.so, self.n, self.c, self.v
        so.check(so.sparse_vocab_loss(self.x, self.w, n, c, v, self.target, self.loss, self.lse, self.ws, self.err, stream))
        so.check(so.sparse_vocab_loss_grad(self.dloss if dloss else None, self.x, self.w, n, c, v, self.target, self.lse,
                                           self.dx, self.dw, self.ws, self.err, stream))

    def check(self):
        self.G.check("vocab loss")
        assert int(self.err.item()) == 0

    def compare(self, dloss=True):
        x, w, t = _np(self.x), _np(self.w), self.target.cpu().numpy()
        live = t >= 0
        z = x @ w.T
        top = z.max(1)
        lse = top + np.log(np.exp(z - top[:, None]).sum(1))
        rows = np.arange(self.n)
        hit = z[rows, np.maximum(t, 0)]
        near = 560 * E24 * (np.abs(x) @ np.abs(w).T).max(1) + (16 + np.abs(lse)) * 4 * E24
        assert (np.abs(_np(self.lse) - lse) <= near).all()
        loss = np.where(live, lse - hit, 0.0)
        assert (np.abs(_np(self.loss) - loss) <= 2 * near * live).all()
        # all together, as the drift of random signs leaves it
        assert np.linalg.norm(_np(self.lse) - lse) <= 2.0 ** -19 * (np.linalg.norm(lse) + np.linalg.norm(top))
        d = (_np(self.dloss) if dloss else np.ones(self.n)) * live
        g = np.exp(z - lse[:, None])
        p = g.copy()
        g[rows, np.maximum(t, 0)] -= 1.0
        g *= d[:, None]
        if self.type == self.torch.float32:
            off = 2 * near[:, None] * p * d[:, None] + 2.0 ** -22 * np.abs(g)
            for got, ref, size, far in ((self.dx, g @ w, np.abs(g) @ np.abs(w), off @ np.abs(w)),
                                        (self.dw, g.T @ x, np.abs(g).T @ np.abs(x), off.T @ np.abs(x))):
                got = _np(got)
                assert (np.abs(got - ref) <= far + (34 * 17 + 700) * E24 * size).all()
                assert np.linalg.norm(got - ref) <= 2.0 ** -18 * np.linalg.norm(ref)
        else:
            off = 2 * near[:, None] * p * d[:, None] + BF * np.abs(g)
            for got, ref, size, far, k in ((self.dx, g @ w, np.abs(g) @ np.abs(w), off @ np.abs(w), self.v),
                                           (self.dw, g.T @ x, np.abs(g).T @ np.abs(x), off.T @ np.abs(x), self.n)):
                got = _np(got)
                assert (np.abs(got - ref) <= far + 17 * (k / 16 + 1) * E24 * size + BF * np.abs(ref) * 1.01).all()
                assert np.linalg.norm(got - ref) <= BF * np.linalg.norm(ref)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("n,c,v", SIZES)
def test_loss_and_gradient(cuda_lib, n, c, v, kind):
    import torch
    t = Case(torch, cuda_lib, n, c, v, kind)
    t.run()
    t.check()
    t.compare()
