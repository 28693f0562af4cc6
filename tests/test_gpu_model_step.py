"""A run of the operators as a training step has them: rows of a table looked up and normed, routed, sorted, dispatched,
through the experts' products, combined, and scored against the table itself, with every gradient back to the table,
against autograd in 64 bits; and the compiled calls against ctypes'."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

ROWS, C, H, E, K, N, EPS = 3000, 72, 136, 7, 2, 500, 1e-5


class Step:
    def __init__(self, torch, so, kind, seed=0):
        self.torch, self.so = torch, so
        self.t = t = {"f32": torch.float32, "bf16": torch.bfloat16}[kind]
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *s, std=1.0, dtype=torch.float32: (torch.randn(*s, device="cuda", generator=g) * std).to(dtype)  # noqa: E731
        self.table, self.out = r(ROWS, C), r(ROWS, C, std=1.5 * C ** -0.5, dtype=t)
        self.gamma, self.beta, self.router = r(C, std=0.1) + 1, r(C, std=0.1), r(C, E, std=0.3)
        self.up, self.down = r(E, C, H, std=C ** -0.5, dtype=t), r(E, H, C, std=H ** -0.5, dtype=t)
        self.tokens = torch.randint(0, ROWS, (N,), device="cuda", generator=g)
        self.next = torch.randint(0, ROWS, (N,), device="cuda", generator=g)
        self.next[::11] = -1
        live = (self.next >= 0).float()
        self.dloss = live / live.sum()
        new = lambda *s, dtype=torch.float32: torch.empty(s, dtype=dtype, device="cuda")  # noqa: E731
        s = N * K
        self.y, self.mean, self.rstd = new(N, C, dtype=t), new(N), new(N)
        self.expert, self.weights, self.dweights = new(N, K, dtype=torch.int64), new(N, K), new(N, K)
        self.offsets, self.pos = new(E + 1, dtype=torch.int64), new(N, K, dtype=torch.int32)
        self.xs, self.hidden, self.ys = new(s, C, dtype=t), new(s, H, dtype=t), new(s, C, dtype=t)
        self.mixed, self.loss, self.lse = new(N, C, dtype=t), new(N), new(N)
        self.dz, self.dout, self.dys, self.dh = new(N, C, dtype=t), new(ROWS, C, dtype=t), new(s, C, dtype=t), new(s, H, dtype=t)
        self.dxs, self.dmixed = new(s, C, dtype=t), new(N, C, dtype=t)
        self.dup, self.ddown, self.dlogits = new(E, C, H), new(E, H, C), new(N, E)
        self.dx, self.dgamma, self.dbeta = new(N, C), new(C), new(C)
        self.err = so.error_word()
        self.ws = new(max(so.sparse_expert_workspace_size(N, K, E), so.sparse_expert_matmul_workspace_size(t, s, C, H, E),
                          so.sparse_expert_matmul_workspace_size(t, s, H, C, E), so.sparse_vocab_loss_workspace_size(t, N, C, ROWS, True),
                          so.sparse_layer_norm_workspace_size(N, C)), dtype=torch.uint8)

    def run(self, stream=None):
        """stream given: the binding's own path, by ctypes."""
        so, torch, s = self.so, self.torch, N * K
        ok = lambda code: so.check(code)  # noqa: E731
        ws, err, off = self.ws, self.err, self.offsets
        ok(so.sparse_layer_norm(self.table, ROWS, C, self.tokens, N, self.gamma, self.beta, EPS, self.y, self.mean, self.rstd, err, stream))
        ok(so.sparse_expert_route(self.y.float() @ self.router, N, E, K, 1, self.expert, self.weights, err, stream))
        ok(so.sparse_expert_sort(self.expert, N, K, E, off, None, self.pos, ws, err, stream))
        ok(so.sparse_expert_dispatch(self.y, N, K, C, self.pos, off, E, self.xs, err, stream))
        ok(so.sparse_expert_matmul(self.xs, self.up, s, C, H, 0, off, E, self.hidden, ws, err, stream))
        active = torch.relu(self.hidden)
        ok(so.sparse_expert_matmul(active, self.down, s, H, C, 0, off, E, self.ys, ws, err, stream))
        ok(so.sparse_expert_combine(self.ys, N, K, C, self.pos, self.weights, self.mixed, err, stream))
        z = self.y + self.mixed
        ok(so.sparse_vocab_loss(z, self.out, N, C, ROWS, self.next, self.loss, self.lse, ws, err, stream))
        ok(so.sparse_vocab_loss_grad(self.dloss, z, self.out, N, C, ROWS, self.next, self.lse, self.dz, self.dout, ws, err, stream))
        ok(so.sparse_expert_combine_grad(self.dz, self.ys, N, K, C, self.pos, off, E, self.weights, self.dys, self.dweights, err, stream))
        ok(so.sparse_expert_matmul(self.dys, self.down, s, H, C, 1, off, E, self.dh, ws, err, stream))
        ok(so.sparse_expert_matmul_grad(active, self.dys, s, H, C, off, E, self.ddown, ws, err, stream))
        dh = self.dh * (self.hidden > 0)
        ok(so.sparse_expert_matmul(dh, self.up, s, C, H, 1, off, E, self.dxs, ws, err, stream))
        ok(so.sparse_expert_matmul_grad(self.xs, dh, s, C, H, off, E, self.dup, ws, err, stream))
        ok(so.sparse_expert_combine(self.dxs, N, K, C, self.pos, None, self.dmixed, err, stream))
        ok(so.sparse_expert_route_grad(self.dweights, None, N, E, K, 1, self.expert, self.weights, self.dlogits, err, stream))
        dy = (self.dz.float() + self.dmixed.float() + self.dlogits @ self.router.t()).to(self.t)
        ok(so.sparse_layer_norm_grad(dy, self.table, ROWS, C, self.tokens, N, self.gamma, self.mean, self.rstd, self.dx, self.dgamma,
                                     self.dbeta, ws, err, stream))
        return {n: getattr(self, n) for n in ("loss", "weights", "dx", "dgamma", "dbeta", "dup", "ddown", "dout", "dlogits")}


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_a_step_of_all_of_them(cuda_lib, kind):
    import torch
    m = Step(torch, cuda_lib, kind)
    got = m.run()
    torch.cuda.synchronize()
    assert int(m.err.item()) == 0
    leaf = lambda t: t.detach().double().clone().requires_grad_()  # noqa: E731
    table, out, up, down, router, gamma, beta = map(leaf, (m.table, m.out, m.up, m.down, m.router, m.gamma, m.beta))
    y = torch.nn.functional.layer_norm(table[m.tokens], (C,), gamma, beta, EPS)
    logits = y @ router
    picked = m.expert                                        # the picks themselves are whole numbers, compared elsewhere
    w = torch.softmax(logits.gather(1, picked), 1)
    z = y
    for j in range(K):
        for e in range(E):
            rows = (picked[:, j] == e).nonzero()[:, 0]
            # which units are active is a truth value as the picks are: a unit next to 0 counts as a whole on either side of
            # it, and with bf16 one in some hundred changes sides (a 2^-8 of its spread away), 5 % of a gradient's norm
            on = m.hidden[m.pos[rows, j].long()] > 0
            z = z.index_add(0, rows, (y[rows] @ up[e]) * on @ down[e] * w[rows, j, None])
    live = m.next >= 0
    loss = torch.where(live, torch.nn.functional.cross_entropy(z @ out.T, m.next.clamp(min=0), reduction="none"), 0.0)
    (loss * m.dloss.double()).sum().backward()
    dx = torch.zeros_like(table).index_add(0, m.tokens, got["dx"].double())
    # fp32: sums of some hundred terms through eight operators, 2^-16.  bf16: some ten roundings of 2^-8 on the way, of random sign
    bound = 2.0 ** -16 if kind == "f32" else 10 ** 0.5 * 2.0 ** -8 * 2
    for name, mine, ref in (("loss", got["loss"], loss.detach()), ("table", dx, table.grad), ("out", got["dout"], out.grad), ("up", got["dup"], up.grad),
                            ("down", got["ddown"], down.grad), ("gamma", got["dgamma"], gamma.grad), ("beta", got["dbeta"], beta.grad)):
        assert float((mine.double() - ref).norm()) <= bound * float(ref.norm()), name


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_a_step_captured_and_by_ctypes(cuda_lib, kind):
    import torch
    m = Step(torch, cuda_lib, kind, seed=1)
    first = {n: t.clone() for n, t in m.run().items()}
    by_ctypes = {n: t.clone() for n, t in m.run(torch.cuda.current_stream()).items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = m.run()
    for t in outs.values():
        t.fill_(7.0)
    graph.replay()
    torch.cuda.synchronize()
    assert int(m.err.item()) == 0
    for n, t in first.items():
        assert torch.equal(t, by_ctypes[n]) and torch.equal(t, outs[n]), n


def test_two_threads(cuda_lib):
    """Two host threads with a stream and a workspace each."""
    import threading

    import torch
    steps = [Step(torch, cuda_lib, k, seed=3) for k in ("f32", "bf16")]
    first = [{n: t.clone() for n, t in m.run().items()} for m in steps]
    torch.cuda.synchronize()
    failed = []

    def work(m, ref):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(10):
                    got = m.run()
                    torch.cuda.current_stream().synchronize()
                    for n, t in ref.items():
                        assert torch.equal(t, got[n]), n
        except BaseException as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work, args=a) for a in zip(steps, first)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("again", [0, 1])
def test_route_where_it_can_go_wrong(cuda_lib, kind, again):
    """The type's lowest value is a score (a mask that leaves something), -inf is none; rows of equals, of more than a warp's
    candidates; NaN and +inf."""
    import torch
    so = cuda_lib
    t = {"f32": torch.float32, "bf16": torch.bfloat16}[kind]
    for e, k in ((40, 4), (256, 8), (1000, 32)):
        x = torch.randn(64, e, device="cuda").to(t)
        low = torch.finfo(t).min
        x[0], x[1], x[2], x[3] = 0.0, low, -float("inf"), 2.5
        x[1, 3] = 0.5
        x[4, 1:] = -float("inf")
        x[5, : e - 2] = 1.0
        x[6, ::2] = 3.0
        x[7, :k - 1], x[7, k - 1:] = low, -float("inf")
        err, expert, weights = so.error_word(), torch.empty(64, k, dtype=torch.int64, device="cuda"), torch.empty(64, k, device="cuda")
        so.check(so.sparse_expert_route(x, 64, e, k, again, expert, weights, err))
        assert int(err.item()) == 0
        f = x.double()
        value, order = torch.sort(f, dim=1, descending=True, stable=True)
        gone = value[:, :k] == -float("inf")
        assert torch.equal(expert, torch.where(gone, -1, order[:, :k]))
        top = torch.where(gone[:, :1], 0.0, value[:, :1])
        each = torch.exp(value[:, :k] - top)
        total = each.sum(1, keepdim=True) if again else torch.exp(f - top).sum(1, keepdim=True)
        ref = torch.where(gone, 0.0, each / torch.where(total > 0, total, 1.0))
        assert bool(((weights.double() - ref).abs() <= 60 * 2.0 ** -23 * ref).all())
        grad, dw = torch.full_like(x, 9.0), torch.randn(64, k, device="cuda")
        so.check(so.sparse_expert_route_grad(dw, x, 64, e, k, again, expert, weights, grad, err))
        assert int(err.item()) == 0 and torch.isfinite(grad).all() and not grad[2].any()
        for bad in (float("nan"), float("inf")):
            y = x.clone()
            y[9, e - 1] = bad
            err = so.error_word()
            so.check(so.sparse_expert_route(y, 64, e, k, again, expert, weights, err))
            assert int(err.item()) == so.ERR_NON_FINITE
        err = so.error_word()
        wrong = torch.where(expert >= 0, e, expert)
        so.check(so.sparse_expert_route_grad(dw, x, 64, e, k, again, wrong, weights, grad, err))
        assert int(err.item()) == so.ERR_INDEX_OUT_OF_RANGE


def test_routes_gradient_by_differences(cuda_lib):
    import torch
    so = cuda_lib
    g = torch.Generator(device="cuda").manual_seed(4)
    x, dw = torch.randn(200, 24, device="cuda", generator=g), torch.randn(200, 3, device="cuda", generator=g)
    for again in (0, 1):
        def weights(y):
            ex, w = torch.empty(200, 3, dtype=torch.int64, device="cuda"), torch.empty(200, 3, device="cuda")
            so.check(so.sparse_expert_route(y, 200, 24, 3, again, ex, w, so.error_word()))
            return ex, w
        expert, w = weights(x)
        grad = torch.empty_like(x)
        so.check(so.sparse_expert_route_grad(dw, x, 200, 24, 3, again, expert, w, grad, so.error_word()))
        d = torch.randn(200, 24, device="cuda", generator=g)
        h = 2.0 ** -8
        (eu, up), (ed, down) = weights(x + h * d), weights(x - h * d)
        same = (eu == expert).all(1) & (ed == expert).all(1)     # where no pick changes
        assert int(same.sum()) > 100
        slope = ((up.double() - down.double()) / (2 * h) * dw.double()).sum(1)
        mine = (grad.double() * d.double()).sum(1)
        # third derivatives of weights: below 3 |d|^3 |dw|, |d| up to 4; weights are off by 2^-22, over h
        assert float((slope - mine)[same].abs().max()) <= h * h / 6 * 3 * 64 * 8 + 3 * 4 * 2.0 ** -22 / h
