"""The loss over a table's rows where it can go wrong: pieces of the table, tokens that do not count, targets that are
no rows, scores far apart, tables past 2^31 elements, results that are not wanted, streams, graphs, equal bits."""
import pytest

from test_gpu_vocab_loss import BF, E24, Case

pytestmark = pytest.mark.gpu


def _reference(torch, x, w, target, dloss):
    x, w = x.double(), w.double()
    z = x @ w.T
    lse = torch.logsumexp(z, 1)
    live, rows, hit = target >= 0, torch.arange(len(x), device="cuda"), target.clamp(min=0)
    loss = torch.where(live, lse - z[rows, hit], 0.0)
    g = torch.exp(z - lse[:, None])
    g[rows, hit] -= 1.0
    g *= torch.where(live, dloss.double(), 0.0)[:, None]
    return loss, lse, g @ w, g.T @ x


def _run(torch, so, x, w, target, dloss, ws=None, err=None):
    n, (v, c) = x.shape[0], w.shape
    loss, lse, dx, dw = torch.empty(n, device="cuda"), torch.empty(n, device="cuda"), torch.empty_like(x), torch.empty_like(w)
    ws = ws if ws is not None else torch.empty(so.sparse_vocab_loss_workspace_size(x.dtype, n, c, v, True), dtype=torch.uint8, device="cuda")
    err = err if err is not None else so.error_word()
    so.check(so.sparse_vocab_loss(x, w, n, c, v, target, loss, lse, ws, err))
    so.check(so.sparse_vocab_loss_grad(dloss, x, w, n, c, v, target, lse, dx, dw, ws, err))
    return loss, lse, dx, dw, err


def _case(torch, n, c, v, kind, seed=0, std=1.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = {"f32": torch.float32, "bf16": torch.bfloat16}[kind]
    x = torch.randn(n, c, device="cuda", generator=g).to(t)
    w = (torch.randn(v, c, device="cuda", generator=g) * std * c ** -0.5).to(t)
    target = torch.randint(0, v, (n,), device="cuda", generator=g)
    target[torch.rand(n, device="cuda", generator=g) < 0.1] = -1
    return x, w, target, torch.rand(n, device="cuda", generator=g) + 0.5


# pieces: 2 and 3 of them with these sizes; both sides of the narrow rows' end; tiles by pairs and by one block
@pytest.mark.parametrize("n,c,v,kind", [(9000, 136, 30000, "bf16"), (3000, 136, 30000, "f32"), (2000, 128, 30000, "f32"),
                                        (2000, 128, 30000, "bf16"), (100, 264, 50000, "f32"), (128, 1032, 9999, "bf16"), (5000, 64, 400, "bf16"),
                                        (4000, 520, 300, "f32")])
def test_large_sizes(cuda_lib, n, c, v, kind):
    """Norms: scores are off by 2^-20 or so each (a run of 32 sums), slopes and results with bf16 by 2^-8 at most."""
    import torch
    x, w, target, dloss = _case(torch, n, c, v, kind)
    got = _run(torch, cuda_lib, x, w, target, dloss)
    assert int(got[4].item()) == 0
    ref = _reference(torch, x, w, target, dloss)
    for i, (p, q) in enumerate(zip(got[:4], ref)):
        bound = 2.0 ** -19 if i < 2 else 2.0 ** -18 if kind == "f32" else BF
        assert float((p.double() - q).norm()) <= bound * float(q.norm()), i
    again = _run(torch, cuda_lib, x, w, target, dloss)
    assert all(torch.equal(p, q) for p, q in zip(got[:4], again[:4]))


def test_one_dloss_for_all_loses_no_more_than_the_results_rounding(cuda_lib):
    """Under a mean the largest slopes are all dloss less a probability: rounded as such they would be off alike."""
    import torch
    for c in (64, 256):
        x, w, target, _ = _case(torch, 1500, c, 20000, "bf16")
        target.clamp_(min=0)
        for d in (1.0526e-4, 1.9e-4, -0.33):                  # significands next to 1 and 2
            dloss = torch.full((1500,), d, device="cuda")
            dx, dw = _run(torch, cuda_lib, x, w, target, dloss)[2:4]
            ref = _reference(torch, x, w, target, dloss)
            # a result's rounding: 2^-8 / sqrt(3) of its norm at the most, the slopes' own half of that at most
            for p, q in ((dx, ref[2]), (dw, ref[3])):
                assert float((p.double() - q).norm()) <= 1.25 * BF / 3 ** 0.5 * float(q.norm())


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("c", [40, 200])
def test_tokens_that_do_not_count(cuda_lib, c, kind):
    import torch
    so = cuda_lib
    x, w, target, dloss = _case(torch, 300, c, 700, kind)
    dloss[target < 0] = float("nan")                          # not looked at
    loss, lse, dx, dw, err = _run(torch, so, x, w, target, dloss)
    assert int(err.item()) == 0 and torch.isfinite(dw).all()
    assert not loss[target < 0].any() and not dx[target < 0].any() and (dx[target >= 0] != 0).any(1).all()
    target.fill_(-1)
    loss, lse, dx, dw, err = _run(torch, so, x, w, target, dloss)
    assert int(err.item()) == 0
    assert not loss.any() and not dx.any() and not dw.any() and torch.isfinite(lse).all()


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("c", [40, 200])
@pytest.mark.parametrize("bad", [-2, 700, 1 << 40, -(1 << 40)])
def test_targets_that_are_no_rows(cuda_lib, c, kind, bad):
    import torch
    so = cuda_lib
    x, w, target, dloss = _case(torch, 300, c, 700, kind)
    n, v = 300, 700
    loss, lse, ws = torch.empty(n, device="cuda"), torch.zeros(n, device="cuda"), torch.empty(
        so.sparse_vocab_loss_workspace_size(x.dtype, n, c, v, True), dtype=torch.uint8, device="cuda")
    target[123] = bad
    err = so.error_word()
    so.check(so.sparse_vocab_loss(x, w, n, c, v, target, loss, lse, ws, err))
    assert int(err.item()) == so.ERR_INDEX_OUT_OF_RANGE
    err.zero_()
    so.check(so.sparse_vocab_loss_grad(dloss, x, w, n, c, v, target, lse, torch.empty_like(x), torch.empty_like(w), ws, err))
    assert int(err.item()) == so.ERR_INDEX_OUT_OF_RANGE


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("c", [64, 136])
def test_scores_far_apart(cuda_lib, c, kind):
    """Scores of hundreds of either sign, of one token all far below zero (the rows behind the table's last must not count)."""
    import torch
    x, w, target, dloss = _case(torch, 200, c, 1003, kind, std=40.0)
    w[:, 0] = 30.0
    x[7] = 0.0
    x[7, 0] = -8.0                                            # every score of token 7 is about -240
    target.clamp_(min=0)
    got = _run(torch, cuda_lib, x, w, target, dloss)
    ref = _reference(torch, x, w, target, dloss)
    assert int(got[4].item()) == 0
    # scores of some hundreds: 2^-20 of them is 3e-4 in an exponent
    size = (x.double().abs() @ w.double().abs().T).amax(1)
    near = 64 * E24 * size + 1e-5
    assert bool(((got[1].double() - ref[1]).abs() <= near).all()) and bool(((got[0].double() - ref[0]).abs() <= 2 * near).all())
    slack = float(near.max()) + (BF if kind == "bf16" else 1e-5)
    assert all(float((p.double() - q).norm()) <= 2 * slack * float(q.norm()) for p, q in zip(got[2:4], ref[2:4]))
    assert all(torch.isfinite(p).all() for p in got[:4])


def test_what_is_not_wanted(cuda_lib):
    import torch
    so = cuda_lib
    for c in (48, 160):
        x, w, target, dloss = _case(torch, 90, c, 500, "f32")
        _, lse, dx, dw, err = _run(torch, so, x, w, target, dloss)
        ws = torch.empty(so.sparse_vocab_loss_workspace_size(x.dtype, 90, c, 500, True), dtype=torch.uint8, device="cuda")
        one, two = torch.empty_like(x), torch.empty_like(w)
        so.check(so.sparse_vocab_loss_grad(dloss, x, w, 90, c, 500, target, lse, one, None, ws, err))
        so.check(so.sparse_vocab_loss_grad(dloss, x, w, 90, c, 500, target, lse, None, two, ws, err))
        so.check(so.sparse_vocab_loss_grad(dloss, x, w, 90, c, 500, target, lse, None, None, None, err))
        assert torch.equal(one, dx) and torch.equal(two, dw)
        ones = _run(torch, so, x, w, target, None)
        full = _run(torch, so, x, w, target, torch.ones(90, device="cuda"))
        assert all(torch.equal(p, q) for p, q in zip(ones[:4], full[:4]))
    assert so.sparse_vocab_loss(x[:0], w, 0, c, 500, target[:0], lse[:0], lse[:0], None, err) == so.OK
    dw.fill_(3.0)
    assert so.sparse_vocab_loss_grad(None, x[:0], w, 0, c, 500, target[:0], lse[:0], x[:0], dw, None, err) == so.OK
    assert not dw.any()


@pytest.mark.parametrize("c", [64, 2056])
def test_tables_past_32_bits(cuda_lib, c):
    import torch
    so = cuda_lib
    v, n = (1 << 31) // c + 5000, 5
    w = torch.empty(v, c, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(2)
    for at in range(0, v, 1 << 20):
        w[at:at + (1 << 20)].normal_(0.0, c ** -0.5, generator=g)
    x = torch.randn(n, c, device="cuda", generator=g).bfloat16()
    target = torch.tensor([v - 1, v - 2, 0, -1, v - 4000], device="cuda")
    dloss = torch.ones(n, device="cuda")
    loss, lse, dx, dw, err = _run(torch, so, x, w, target, dloss)
    assert int(err.item()) == 0
    z = torch.cat([x.double() @ w[at:at + (1 << 18)].double().T for at in range(0, v, 1 << 18)], 1)
    ref = torch.logsumexp(z, 1)
    assert float((lse.double() - ref).abs().max()) <= 1e-5
    hit = z[torch.arange(n, device="cuda"), target.clamp(min=0)]
    assert float((loss.double() - torch.where(target >= 0, ref - hit, 0.0)).abs().max()) <= 2e-5
    p = torch.exp(z - ref[:, None])
    p[torch.arange(n, device="cuda"), target.clamp(min=0)] -= 1.0
    p[3] = 0.0
    for s in (slice(v - 4200, v), slice(0, 300)):
        r = p[:, s].T @ x.double()
        assert float((dw[s].double() - r).norm()) <= BF * float(r.norm())


@pytest.mark.parametrize("c", [64, 200])
def test_streams_and_graphs(cuda_lib, c):
    import torch
    so = cuda_lib
    x, w, target, dloss = _case(torch, 400, c, 3000, "bf16")
    first = _run(torch, so, x, w, target, dloss)[:4]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = _run(torch, so, x, w, target, dloss)[:4]
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(first, other))
    ws = torch.empty(so.sparse_vocab_loss_workspace_size(x.dtype, 400, c, 3000, True), dtype=torch.uint8, device="cuda")
    err, graphs, outs = so.error_word(), [], []
    for _ in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(_run(torch, so, x, w, target, dloss, ws=ws, err=err)[:4])
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    for o in outs:
        assert all(torch.equal(p, q) for p, q in zip(first, o))


def test_any_alignment(cuda_lib):
    import torch
    for kind in ("bf16", "f32"):
        for c in (64, 72, 136):
            t = Case(torch, cuda_lib, 200, c, 900, kind, shift=1)
            t.run()
            t.check()
            t.compare()


def test_gradient_by_differences(cuda_lib):
    """dx of the loss's sum against differences of the loss itself: central ones of fp32 losses, 2^-23 of about 7 over 2 h."""
    import torch
    so = cuda_lib
    x, w, target, _ = _case(torch, 40, 96, 800, "f32")
    target.clamp_(min=0)
    dx = _run(torch, so, x, w, target, None)[2]
    g = torch.Generator(device="cuda").manual_seed(9)
    d = torch.randn(40, 96, device="cuda", generator=g)
    h = 2.0 ** -6
    up, down = (_run(torch, so, (x + s * h * d), w, target, None)[0] for s in (1, -1))
    slope, mine = (up.double() - down.double()) / (2 * h), (dx.double() * d.double()).sum(1)
    # a third derivative of a few units times h^2 / 6, and the losses' own errors (2^-19 of 7 each) over h
    assert float((slope - mine).abs().max()) <= 2.0 ** -12 * 20 / 6 + 7 * 2.0 ** -19 / h


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("c", [40, 64, 128, 131, 200, 264])
def test_rows_of_tokens_that_do_not_count_are_not_looked_at(cuda_lib, c, kind):
    """A padded batch's rows hold anything: results are those of zeros there, bit for bit, whatever else they were."""
    import torch
    so = cuda_lib
    x, w, target, dloss = _case(torch, 333, c, 905, kind)
    target[300:] = -1                                         # a batch's padding
    none = target < 0
    for size in (333, 1):                                     # and a single token
        for d in (dloss, None):
            d = d if d is None else d[-size:].contiguous()
            clean, t = x[-size:].clone(), target[-size:].contiguous()
            clean[none[-size:]] = 0.0
            want = _run(torch, so, clean, w, t, d)
            for what in (float("nan"), float("inf"), -float("inf")):
                dirty = clean.clone()
                dirty[none[-size:]] = what
                got = _run(torch, so, dirty, w, t, d)
                assert int(got[4].item()) == 0
                assert all(torch.equal(p, q) for p, q in zip((got[0], got[2], got[3]), (want[0], want[2], want[3])))
                assert torch.equal(got[1][t >= 0], want[1][t >= 0])
