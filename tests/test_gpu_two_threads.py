"""Calls of two host threads on one device, whose kernels want different amounts of shared memory: what a
thread asks for must not take from the other's launch.  Both routes of the binding let go of the
interpreter during a call, so the threads' calls do overlap."""
import threading

import pytest

pytestmark = pytest.mark.gpu

CALLS = 3000


def _overlapping(torch, calls):
    """Every call CALLS times by a thread and stream of its own; the codes other than 0."""
    bad, start = [], threading.Barrier(len(calls))

    def loop(call):
        with torch.cuda.stream(torch.cuda.Stream()):
            start.wait()
            for i in range(CALLS):
                code = call()
                if code != 0:
                    bad.append((i, code))
                    break
                if i % 256 == 255:
                    torch.cuda.current_stream().synchronize()
            torch.cuda.current_stream().synchronize()

    threads = [threading.Thread(target=loop, args=(c,)) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    return bad


def _norm(torch, so, n, c, x_type, back):
    x = torch.randn(n, c, device="cuda").to(x_type)
    y, dx, dy = torch.empty_like(x), torch.empty_like(x), torch.randn(n, c, device="cuda").to(x_type)
    mean, rstd, gamma = torch.zeros(n, device="cuda"), torch.ones(n, device="cuda"), torch.ones(c, device="cuda")
    err = so.error_word()
    torch.cuda.synchronize()
    if back:
        return lambda: so.sparse_layer_norm_grad(dy, x, n, c, None, n, gamma, mean, rstd, dx, None, None, None, err)
    return lambda: so.sparse_layer_norm(x, n, c, None, n, gamma, gamma, 1e-5, y, mean, rstd, err)


def _sort(torch, so, n, k, experts):
    expert = torch.randint(0, experts, (n, k), device="cuda")
    off, pos = torch.empty(experts + 1, dtype=torch.int64, device="cuda"), torch.empty(n, k, dtype=torch.int32, device="cuda")
    ws = torch.empty(so.sparse_expert_workspace_size(n, k, experts), dtype=torch.uint8, device="cuda")
    err = so.error_word()
    torch.cuda.synchronize()
    return lambda: so.sparse_expert_sort(expert, n, k, experts, off, None, pos, ws, err)


# rows that pass through the ring (1025 to 8192 columns) and wider ones held whole, both ways
@pytest.mark.parametrize("c,back", [((4096, 8192), False), ((16384, 40000), False), ((16384, 40000), True),
                                    ((1111, 3333), True)])
def test_layer_norm(cuda_lib, c, back):
    import torch
    kind = torch.float32 if c[0] == 1111 else torch.bfloat16
    assert _overlapping(torch, [_norm(torch, cuda_lib, 16, cols, kind, back) for cols in c]) == []


def test_expert_sort(cuda_lib):
    import torch
    assert _overlapping(torch, [_sort(torch, cuda_lib, 2048, 2, e) for e in (128, 512, 1024)]) == []
