"""A small model around an embedding table, trained with the library's operators.

Tokens look rows of a table up; a layer norm of the rows feeds a router and the two experts it picks
for each token; the experts' weighted outputs are added to the normalised row, and the model learns to
give every token its own target vector.  One step is

  forward   sparse_layer_norm (lookup and norm in one pass), sparse_expert_route, sparse_expert_sort,
            sparse_expert_dispatch, sparse_expert_matmul twice with the activation between, sparse_expert_combine
  backward  sparse_expert_combine_grad, sparse_expert_matmul the other way round and sparse_expert_matmul_grad,
            sparse_expert_combine (dispatch's gradient), sparse_expert_route_grad, sparse_layer_norm_grad, whose
            dx rows are the table's gradient as they are
  update    sparse_adam_table_step for the table (raw lookups, duplicates summed), sparse_muon_step for
            the experts' matrices, plain gradient descent for the few other weights

    python examples/table_and_experts.py [steps]
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from lazy_optimizers_embedding_gb300 import binding as so  # noqa: E402

ROWS, WIDTH, HIDDEN, EXPERTS, PICKED, TOKENS = 5000, 128, 256, 8, 2, 4096
EPS = 1e-5


class Model:
    def __init__(self, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)

        def normal(*shape, std):
            return torch.empty(shape, device=device).normal_(0.0, std, generator=g)

        self.table, self.target = normal(ROWS, WIDTH, std=0.02), normal(ROWS, WIDTH, std=1.0)
        self.m, self.v = torch.zeros_like(self.table), torch.zeros_like(self.table)
        self.last = torch.zeros(ROWS, dtype=torch.int64, device=device)
        self.gamma, self.beta = torch.ones(WIDTH, device=device), torch.zeros(WIDTH, device=device)
        self.router = normal(WIDTH, EXPERTS, std=0.1)
        self.up, self.down = normal(EXPERTS, WIDTH, HIDDEN, std=WIDTH ** -0.5), normal(EXPERTS, HIDDEN, WIDTH, std=HIDDEN ** -0.5)
        self.up_buf, self.down_buf = torch.zeros_like(self.up), torch.zeros_like(self.down)
        self.err, self.t = so.error_word(device), 0

        # the step's buffers and workspaces
        n, c, s = TOKENS, WIDTH, TOKENS * PICKED
        new = lambda *shape, dtype=torch.float32: torch.empty(shape, dtype=dtype, device=device)  # noqa: E731
        self.y, self.mean, self.rstd, self.mixed = new(n, c), new(n), new(n), new(n, c)
        self.offsets, self.pos = new(EXPERTS + 1, dtype=torch.int64), new(n, PICKED, dtype=torch.int32)
        self.xs, self.dys, self.dweights, self.dx_experts = new(s, c), new(s, c), new(n, PICKED), new(n, c)
        self.picked, self.weights, self.dlogits = new(n, PICKED, dtype=torch.int64), new(n, PICKED), new(n, EXPERTS)
        self.hidden, self.ys, self.dactive, self.dxs = new(s, HIDDEN), new(s, c), new(s, HIDDEN), new(s, c)
        self.dup, self.ddown = torch.empty_like(self.up), torch.empty_like(self.down)
        self.dx, self.dgamma, self.dbeta = new(n, c), new(c), new(c)
        ns = so.NsConfig(a=3.4445, b=-4.7750, c=2.0315, eps=1e-7, steps=5, products=1)
        self.muon = so.MuonConfig(lr=0.02, momentum=0.95, weight_decay=0.0, scale=1.0, nesterov=1, ns=ns)
        self.adam = so.AdamConfig(lr=5e-3, beta1=0.9, beta2=0.99, eps=1e-8)
        self.ws = torch.empty(max(so.sparse_layer_norm_workspace_size(n, c),
                                  so.sparse_expert_workspace_size(n, PICKED, EXPERTS),
                                  so.sparse_expert_matmul_workspace_size(torch.float32, s, WIDTH, HIDDEN, EXPERTS),
                                  so.sparse_expert_matmul_workspace_size(torch.float32, s, HIDDEN, WIDTH, EXPERTS),
                                  so.sparse_muon_workspace_size(EXPERTS, WIDTH, HIDDEN, 1),
                                  so.sparse_workspace_size(n, c, ROWS)), dtype=torch.uint8, device=device)

    def step(self, tokens):
        n, c, h, k, e = TOKENS, WIDTH, HIDDEN, PICKED, EXPERTS
        # forward
        so.check(so.sparse_layer_norm(self.table, ROWS, c, tokens, n, self.gamma, self.beta, EPS, self.y, self.mean,
                                      self.rstd, self.err))
        so.check(so.sparse_expert_route(self.y @ self.router, n, e, k, 1, self.picked, self.weights, self.err))
        so.check(so.sparse_expert_sort(self.picked, n, k, e, self.offsets, None, self.pos, self.ws, self.err))
        so.check(so.sparse_expert_dispatch(self.y, n, k, c, self.pos, self.offsets, e, self.xs, self.err))
        so.check(so.sparse_expert_matmul(self.xs, self.up, n * k, c, h, 0, self.offsets, e, self.hidden, self.ws, self.err))
        active = torch.relu(self.hidden)
        so.check(so.sparse_expert_matmul(active, self.down, n * k, h, c, 0, self.offsets, e, self.ys, self.ws, self.err))
        so.check(so.sparse_expert_combine(self.ys, n, k, c, self.pos, self.weights, self.mixed, self.err))
        off = self.y + self.mixed - self.target[tokens]
        loss = (off * off).mean()

        # backward
        dout = off * (2.0 / off.numel())
        so.check(so.sparse_expert_combine_grad(dout, self.ys, n, k, c, self.pos, self.offsets, e, self.weights, self.dys,
                                               self.dweights, self.err))
        so.check(so.sparse_expert_matmul(self.dys, self.down, n * k, h, c, 1, self.offsets, e, self.dactive, self.ws, self.err))
        so.check(so.sparse_expert_matmul_grad(active, self.dys, n * k, h, c, self.offsets, e, self.ddown, self.ws, self.err))
        dhidden = self.dactive * (self.hidden > 0)
        so.check(so.sparse_expert_matmul(dhidden, self.up, n * k, c, h, 1, self.offsets, e, self.dxs, self.ws, self.err))
        so.check(so.sparse_expert_matmul_grad(self.xs, dhidden, n * k, c, h, self.offsets, e, self.dup, self.ws, self.err))
        so.check(so.sparse_expert_combine(self.dxs, n, k, c, self.pos, None, self.dx_experts, self.err))
        so.check(so.sparse_expert_route_grad(self.dweights, None, n, e, k, 1, self.picked, self.weights, self.dlogits, self.err))
        dy = dout + self.dx_experts + self.dlogits @ self.router.t()
        so.check(so.sparse_layer_norm_grad(dy, self.table, ROWS, c, tokens, n, self.gamma, self.mean, self.rstd, self.dx,
                                           self.dgamma, self.dbeta, self.ws, self.err))

        # update
        self.t += 1
        so.check(so.sparse_adam_table_step(self.table, self.m, self.v, self.last, so.LAST_STEP_PER_ROW, ROWS, c,
                                           so.row_coo(tokens, self.dx, False), self.t, self.adam, so.DORMANCY_DECAY,
                                           self.ws, self.err))
        so.check(so.sparse_muon_step(self.up, self.up_buf, self.dup, e, c, h, self.muon, self.ws, self.err))
        so.check(so.sparse_muon_step(self.down, self.down_buf, self.ddown, e, h, c, self.muon, self.ws, self.err))
        self.router -= 0.5 * (self.y.t() @ self.dlogits)
        self.gamma -= 0.5 * self.dgamma
        self.beta -= 0.5 * self.dbeta
        return loss


def lookups(step, device="cuda"):
    """A step's tokens: many of a few rows, few of many."""
    g = torch.Generator(device=device).manual_seed(1000 + step)
    u = torch.rand(TOKENS, generator=g, device=device)
    return (ROWS * u * u * u).long().clamp_(max=ROWS - 1)


def main(steps=100):
    model = Model()
    losses = []
    for step in range(steps):
        losses.append(model.step(lookups(step)))
        if step % 20 == 0 or step + 1 == steps:
            print(f"step {step:4d}  loss {float(losses[-1]):.4f}", flush=True)
    code = int(model.err.item())
    if code:
        raise SystemExit(f"the library reported: {so.status_string(code)}")
    return [float(x) for x in losses]


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 100)
