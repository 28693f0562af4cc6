"""What the dense operators around the embedding step are measured on.

Three operators that a model with a sparse embedding table trains and serves with, next to the
lazy table step itself:

  norm    layer norm of looked-up table rows or of dense rows, and its backward pass with the
          reduction of the scale's and shift's gradients over all rows
  expert  tokens sorted by expert and back: the stable sort by expert, the rows spread to their
          sorted places, the experts' outputs weighted and summed per token, and the gradients
  muon    an update orthogonalised by Newton-Schulz products, alone or inside the Muon step of
          the matrices (momentum, weight decay and update)

Every case has "op" with one of the three names.  `run` computes the plain form in 32 bits with
torch, or calls the library's entry points where `own` is true.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
LN_EPS = 1e-5
NS = (3.4445, -4.7750, 2.0315)     # the quintic X <- a X + (b A + c A^2) X with A = X X^T
NS_EPS = 1e-7
NS_STEPS = 5
LR, MOMENTUM, DECAY = 0.02, 0.95, 0.01


def listed():
    return [
        # one decoding step of a handful of sequences: latency alone
        {"name": "norm decode", "op": "norm", "n": 4, "c": 2048, "rows": 0, "x": "bf16", "y": "bf16", "grad": False},
        # odd width, fp32, rows that start at any 4-byte boundary
        {"name": "norm odd", "op": "norm", "n": 5003, "c": 1111, "rows": 0, "x": "f32", "y": "f32", "grad": True},
        # the embedding norm of a training step on the 10M x 128 table: Zipf lookups, backward rows for the table step
        {"name": "norm table", "op": "norm", "n": 262144, "c": 128, "rows": 10_000_000, "x": "f32", "y": "f32",
         "grad": True},
        # a block's norm in training, bf16 activations
        {"name": "norm train", "op": "norm", "n": 16384, "c": 4096, "rows": 0, "x": "bf16", "y": "bf16", "grad": True},
        # one decoding step: 8 tokens, 4 experts each
        {"name": "expert decode", "op": "expert", "n": 8, "k": 4, "experts": 64, "c": 2048, "type": "bf16",
         "padded": 0.0, "grad": False},
        # ragged everything, a fifth of the tokens padding that goes to no expert
        {"name": "expert odd", "op": "expert", "n": 3001, "k": 3, "experts": 37, "c": 515, "type": "f32",
         "padded": 0.2, "grad": True},
        # a prompt through wide experts, forward only
        {"name": "expert prompt", "op": "expert", "n": 32768, "k": 2, "experts": 16, "c": 4096, "type": "bf16",
         "padded": 0.05, "grad": False},
        # a training step of many small experts
        {"name": "expert train", "op": "expert", "n": 16384, "k": 8, "experts": 128, "c": 2048, "type": "bf16",
         "padded": 0.0, "grad": True},
        # a small head: launches and latency
        {"name": "muon small", "op": "muon", "step": True, "batch": 1, "r": 64, "c": 128, "type": "f32"},
        # a tall fp32 matrix of odd sizes, the whole step
        {"name": "muon tall", "op": "muon", "step": True, "batch": 1, "r": 2501, "c": 1003, "type": "f32"},
        # every expert's matrix of one layer, bf16 in and out
        {"name": "muon experts", "op": "muon", "step": False, "batch": 16, "r": 768, "c": 2048, "type": "bf16"},
        # a large square projection
        {"name": "muon large", "op": "muon", "step": False, "batch": 1, "r": 4096, "c": 4096, "type": "bf16"},
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm", "expert", "muon"))
    if op == "norm":
        c = _log(rng, 16, 8192)
        if rng.random() < 0.6:
            c = max(8, c // 8 * 8)
        n = _log(rng, 1, max(1, min(262144, 16384 * 4096 // c)))
        x, y = rng.choice((("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16")))
        rows = _log(rng, 1000, 400_000_000 // c) if x == "f32" and rng.random() < 0.5 else 0
        return {"op": "norm", "n": n, "c": c, "rows": rows, "x": x, "y": y, "grad": rng.random() < 0.7}
    if op == "expert":
        k = rng.choice((1, 2, 3, 4, 6, 8))
        experts = _log(rng, max(2, k), 256)
        c = _log(rng, 64, 4096)
        if rng.random() < 0.6:
            c = c // 8 * 8
        n = _log(rng, 1, max(1, min(32768, 16384 * 8 * 2048 // (k * c))))
        return {"op": "expert", "n": n, "k": k, "experts": experts, "c": c, "type": rng.choice(("f32", "bf16")),
                "padded": rng.choice((0.0, 0.0, 0.1, 0.5)), "grad": rng.random() < 0.6}
    r, c = _log(rng, 16, 4096), _log(rng, 16, 4096)
    if rng.random() < 0.5:
        r, c = max(16, r // 16 * 16), max(16, c // 16 * 16)
    m = min(r, c)
    batch = _log(rng, 1, max(1, min(64, 4096 ** 3 // (m * r * c))))
    kind = rng.choice(("f32", "bf16"))
    return {"op": "muon", "step": kind == "f32" and rng.random() < 0.6, "batch": batch, "r": r, "c": c, "type": kind}


# ------------------------------------------------------------------------------------ inputs
def _zipf(gen, n, rows, s=1.05):
    """n lookups of a table of `rows` rows, Zipf(s): rank k is row k - 1."""
    cdf = torch.arange(1, rows + 1, dtype=torch.float64, device="cuda").pow_(-s).cumsum_(0)
    u = torch.rand(n, generator=gen, dtype=torch.float64, device="cuda") * cdf[-1]
    return torch.searchsorted(cdf, u, right=True).clamp_(max=rows - 1)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, dtype=torch.float32, std=1.0, mean=0.0):
        t = torch.empty(shape, dtype=torch.float32, device="cuda").normal_(mean, std, generator=gen)
        return t.to(dtype)

    def blank(*shape, dtype=torch.float32):
        return torch.empty(shape, dtype=dtype, device="cuda")

    s = {"case": dict(case), "err": torch.zeros(1, dtype=torch.int32, device="cuda")}
    if case["op"] == "norm":
        n, c, rows = case["n"], case["c"], case["rows"]
        xt, yt = DTYPES[case["x"]], DTYPES[case["y"]]
        if rows:   # a table's rows, small values as the table starts
            s["x"], s["idx"] = normal(rows, c, dtype=xt, std=0.01, mean=0.002), _zipf(gen, n, rows)
        else:
            s["x"], s["idx"] = normal(n, c, dtype=xt, mean=0.3), None
        s["gamma"], s["beta"] = normal(c, std=0.1, mean=1.0), normal(c, std=0.1)
        s["y"], s["mean"], s["rstd"] = blank(n, c, dtype=yt), blank(n), blank(n)
        if case["grad"]:
            s["dy"] = normal(n, c, dtype=yt)
            s["dx"], s["dgamma"], s["dbeta"] = blank(n, c, dtype=xt), blank(c), blank(c)
    elif case["op"] == "expert":
        n, k, e, c, t = case["n"], case["k"], case["experts"], case["c"], DTYPES[case["type"]]
        score = normal(n, e) + normal(e)                      # some experts are liked more than others
        top = score.topk(k, dim=1)
        s["expert"] = top.indices.contiguous()
        s["weights"] = torch.softmax(top.values, 1).contiguous()
        if case["padded"]:
            gone = torch.rand(n, generator=gen, device="cuda") < case["padded"]
            s["expert"][gone] = -1
        s["x"], s["ys"] = normal(n, c, dtype=t), normal(n * k, c, dtype=t)
        s["offsets"] = blank(e + 1, dtype=torch.int64)
        s["src"], s["pos"] = blank(n * k, dtype=torch.int32), blank(n, k, dtype=torch.int32)
        s["xs"], s["y"] = blank(n * k, c, dtype=t), blank(n, c, dtype=t)
        if case["grad"]:
            s["dy"], s["dxs"] = normal(n, c, dtype=t), normal(n * k, c, dtype=t)
            s["dys"], s["dweights"], s["dx"] = blank(n * k, c, dtype=t), blank(n, k), blank(n, c, dtype=t)
    else:
        b, r, c, t = case["batch"], case["r"], case["c"], DTYPES[case["type"]]
        # a gradient's spectrum: a few strong directions over a floor of noise
        low = min(16, r, c)
        g = torch.matmul(normal(b, r, low), normal(b, low, c)) / math.sqrt(low) + 0.5 * normal(b, r, c)
        if case["step"]:
            s["g"], s["buf"], s["w"] = g.to(t), normal(b, r, c), normal(b, r, c, std=0.02)
        else:
            s["u"], s["out"] = g.to(t), blank(b, r, c, dtype=t)
    return s


# ------------------------------------------------------------------------------------ plain forms
def _plain_norm(s):
    case = s["case"]
    c, yt, xt = case["c"], s["y"].dtype, s["x"].dtype
    x = (s["x"] if s["idx"] is None else s["x"][s["idx"]]).float()
    mean = x.sum(1) / c
    d = x - mean[:, None]
    rstd = 1.0 / torch.sqrt((d * d).sum(1) / c + LN_EPS)
    xhat = d * rstd[:, None]
    out = {"y": (xhat * s["gamma"] + s["beta"]).to(yt), "mean": mean, "rstd": rstd}
    if case["grad"]:
        dy = s["dy"].float()
        h = dy * s["gamma"]
        a, b = h.sum(1) / c, (h * xhat).sum(1) / c
        out["dx"] = (rstd[:, None] * (h - a[:, None] - xhat * b[:, None])).to(xt)
        out["dgamma"], out["dbeta"] = (dy * xhat).sum(0), dy.sum(0)
    return out


def _plain_expert(s):
    case = s["case"]
    n, k, e, c = case["n"], case["k"], case["experts"], case["c"]
    t = s["x"].dtype
    flat = s["expert"].reshape(-1)
    routed = flat >= 0
    key, order = torch.sort(torch.where(routed, flat, e), stable=True)
    offsets = torch.searchsorted(key, torch.arange(e + 1, device=key.device))
    kept = key < e
    src = torch.where(kept, order, -1).to(torch.int32)
    pos = torch.empty_like(order)
    pos[order] = torch.arange(n * k, device=key.device)
    place = pos.reshape(n, k)
    live = routed.reshape(n, k)
    out = {"offsets": offsets, "src": src, "pos": torch.where(live, place, -1).to(torch.int32)}
    out["xs"] = torch.where(kept[:, None], s["x"][order // k], 0)
    w = torch.where(live, s["weights"], 0.0)
    picked = torch.where(live[:, :, None], s["ys"][place].float(), 0.0)
    out["y"] = (picked * w[:, :, None]).sum(1).to(t)
    if case["grad"]:
        dy = s["dy"].float()
        each = (dy[:, None, :] * s["weights"][:, :, None]).to(t).reshape(n * k, c)
        out["dys"] = torch.where(kept[:, None], each[order], 0)
        out["dweights"] = (picked * dy[:, None, :]).sum(2)
        out["dx"] = torch.where(live[:, :, None], s["dxs"][place].float(), 0.0).sum(1).to(t)
    return out


def _newton_schulz(u):
    a, b, c = NS
    x = u.mT if u.shape[1] > u.shape[2] else u
    x = x / (torch.sqrt((x * x).sum((1, 2), keepdim=True)) + NS_EPS)
    for _ in range(NS_STEPS):
        g = torch.matmul(x, x.mT)
        x = a * x + torch.matmul(b * g + c * torch.matmul(g, g), x)
    return x.mT if u.shape[1] > u.shape[2] else x


def _step_scale(case):
    return math.sqrt(max(1.0, case["r"] / case["c"]))


def _plain_muon(s):
    case = s["case"]
    if not case["step"]:
        return {"out": _newton_schulz(s["u"].float()).to(s["out"].dtype)}
    g = s["g"].float()
    s["buf"].mul_(MOMENTUM).add_(g)
    o = _newton_schulz(g + MOMENTUM * s["buf"])
    s["w"].mul_(1.0 - LR * DECAY).sub_((LR * _step_scale(case)) * o)
    return {"w": s["w"], "buf": s["buf"]}


# ------------------------------------------------------------------------------------ the library's calls
def _plan(s):
    """The workspace and configuration that a program keeps beside its tensors."""
    from lazy_optimizers_embedding_gb300 import binding as so
    case = s["case"]
    s["so"] = so
    size = 0
    if case["op"] == "norm":
        size = so.sparse_layer_norm_workspace_size(case["n"], case["c"])
    elif case["op"] == "expert":
        size = so.sparse_expert_workspace_size(case["n"], case["k"], case["experts"])
    else:
        products = 3 if case["type"] == "f32" else 1
        ns = so.NsConfig(a=NS[0], b=NS[1], c=NS[2], eps=NS_EPS, steps=NS_STEPS, products=products)
        s["cfg"] = ns
        if case["step"]:
            s["cfg"] = so.MuonConfig(lr=LR, momentum=MOMENTUM, weight_decay=DECAY, scale=_step_scale(case), nesterov=1,
                                     ns=ns)
        size = so.sparse_muon_workspace_size(case["batch"], case["r"], case["c"], products)
    s["ws"] = torch.empty(max(size, 256), dtype=torch.uint8, device="cuda")
    return so


def _own_norm(so, s):
    case = s["case"]
    n, c, rows = case["n"], case["c"], case["rows"] or case["n"]
    so.check(so.sparse_layer_norm(s["x"], rows, c, s["idx"], n, s["gamma"], s["beta"], LN_EPS, s["y"], s["mean"],
                                  s["rstd"], s["err"]))
    out = {"y": s["y"], "mean": s["mean"], "rstd": s["rstd"]}
    if case["grad"]:
        so.check(so.sparse_layer_norm_grad(s["dy"], s["x"], rows, c, s["idx"], n, s["gamma"], s["mean"], s["rstd"],
                                           s["dx"], s["dgamma"], s["dbeta"], s["ws"], s["err"]))
        out.update(dx=s["dx"], dgamma=s["dgamma"], dbeta=s["dbeta"])
    return out


def _own_expert(so, s):
    case = s["case"]
    n, k, e, c = case["n"], case["k"], case["experts"], case["c"]
    so.check(so.sparse_expert_sort(s["expert"], n, k, e, s["offsets"], s["src"], s["pos"], s["ws"], s["err"]))
    so.check(so.sparse_expert_dispatch(s["x"], n, k, c, s["pos"], s["offsets"], e, s["xs"], s["err"]))
    so.check(so.sparse_expert_combine(s["ys"], n, k, c, s["pos"], s["weights"], s["y"], s["err"]))
    out = {name: s[name] for name in ("offsets", "src", "pos", "xs", "y")}
    if case["grad"]:
        so.check(so.sparse_expert_combine_grad(s["dy"], s["ys"], n, k, c, s["pos"], s["offsets"], e, s["weights"],
                                               s["dys"], s["dweights"], s["err"]))
        so.check(so.sparse_expert_combine(s["dxs"], n, k, c, s["pos"], None, s["dx"], s["err"]))
        out.update(dys=s["dys"], dweights=s["dweights"], dx=s["dx"])
    return out


def _own_muon(so, s):
    case = s["case"]
    b, r, c = case["batch"], case["r"], case["c"]
    if not case["step"]:
        so.check(so.sparse_orthogonalize(s["u"], b, r, c, s["cfg"], s["out"], s["ws"], s["err"]))
        return {"out": s["out"]}
    so.check(so.sparse_muon_step(s["w"], s["buf"], s["g"], b, r, c, s["cfg"], s["ws"], s["err"]))
    return {"w": s["w"], "buf": s["buf"]}


def run(state):
    op = state["case"]["op"]
    if own:
        so = state.get("so") or _plan(state)
        return {"norm": _own_norm, "expert": _own_expert, "muon": _own_muon}[op](so, state)
    return {"norm": _plain_norm, "expert": _plain_expert, "muon": _plain_muon}[op](state)


# ------------------------------------------------------------------------------------ what a pass cannot do without
def _size(name):
    return 2 if name == "bf16" else 4


def work(case):
    if case["op"] == "norm":
        n, c, xs, ys = case["n"], case["c"], _size(case["x"]), _size(case["y"])
        rows = n
        if case["rows"]:     # each table row that is looked up at all, read once
            rows = min(n, case["rows"]) if case["rows"] < n else _distinct(n, case["rows"])
        moved = rows * c * xs + (8 * n if case["rows"] else 0) + 8 * c + n * c * ys + 8 * n
        flops = 8 * n * c
        if case["grad"]:
            moved += n * c * (ys + xs) + 8 * c
            flops += 14 * n * c
        return {"bytes": moved, "flops": flops}
    if case["op"] == "expert":
        n, k, e, c, size = case["n"], case["k"], case["experts"], case["c"], _size(case["type"])
        live = int(n * k * (1.0 - case["padded"]))
        moved = 8 * n * k + 8 * (e + 1) + 8 * n * k + 4 * n * k          # ids, offsets, src and pos, weights
        moved += size * c * (n + n * k) + size * c * (live + n)         # spread rows; weighted sum
        flops = 2 * live * c
        if case["grad"]:
            moved += size * c * (n + n * k) + 4 * n * k + size * c * (live + n)   # the sum's rows were read above
            flops += 4 * live * c
        return {"bytes": moved, "flops": flops}
    b, r, c, size = case["batch"], case["r"], case["c"], _size(case["type"])
    m, n = min(r, c), max(r, c)
    # a symmetric product needs one of its halves: A and A^2; then B X
    flops = b * NS_STEPS * (m * m * n + m * m * m + 2 * m * m * n)
    return {"bytes": b * r * c * (size + 16 if case["step"] else 2 * size), "flops": flops}


def _distinct(n, rows, s=1.05):
    """The expected number of different rows among n Zipf(s) lookups of `rows`."""
    k = torch.arange(1, rows + 1, dtype=torch.float64).pow_(-s)
    return int((-torch.expm1(n * torch.log1p(-(k / k.sum()).clamp_(max=1 - 1e-12)))).sum())


# ------------------------------------------------------------------------------------ 64 bits
def _exact_norm(case, s):
    with torch.enable_grad():
        rows = s["x"] if s["idx"] is None else s["x"].index_select(0, s["idx"])
        x = rows.double().requires_grad_(case["grad"])
        gamma = s["gamma"].double().requires_grad_(case["grad"])
        beta = s["beta"].double().requires_grad_(case["grad"])
        y = torch.nn.functional.layer_norm(x, (case["c"],), gamma, beta, LN_EPS)
        var, mean = torch.var_mean(x.detach(), 1, correction=0)
        out = {"y": y.detach(), "mean": mean, "rstd": (var + LN_EPS).rsqrt()}
        if case["grad"]:
            out["dx"], out["dgamma"], out["dbeta"] = torch.autograd.grad(y, (x, gamma, beta), s["dy"].double())
    return out


def _exact_expert(case, s):
    n, k, c = case["n"], case["k"], case["c"]
    dev = s["x"].device
    flat = s["expert"].reshape(-1)
    slots = torch.argsort(flat, stable=True)
    slots = slots[int((flat < 0).sum()):]                  # padding sorts first
    token, count = slots // k, slots.numel()

    def spread(rows):                                      # sorted rows, then nothing
        return torch.cat([rows, rows.new_zeros(n * k - count, c)])

    w = s["weights"].reshape(-1)[slots].double()
    ys = s["ys"][:count].double()
    out = {"offsets": None, "src": None, "pos": None, "xs": spread(s["x"][token].double()),
           "y": torch.zeros(n, c, dtype=torch.float64, device=dev).index_add_(0, token, ys * w[:, None])}
    if case["grad"]:
        dy = s["dy"].double()[token]
        out["dys"] = spread(dy * w[:, None])
        dw = torch.zeros(n * k, dtype=torch.float64, device=dev)
        dw[slots] = torch.einsum("ij,ij->i", dy, ys)
        out["dweights"] = dw.reshape(n, k)
        out["dx"] = torch.zeros(n, c, dtype=torch.float64, device=dev).index_add_(0, token, s["dxs"][:count].double())
    return out


def _exact_muon(case, s):
    a, b, c = NS
    if case["step"]:
        buf = MOMENTUM * s["buf"].double() + s["g"].double()
        u = s["g"].double() + MOMENTUM * buf
    else:
        u = s["u"].double()
    tall = case["r"] > case["c"]
    u = u / (torch.linalg.vector_norm(u, dim=(1, 2), keepdim=True) + NS_EPS)
    # every factor is a polynomial in the first Gram matrix: they commute, so the Gram matrices
    # of later steps and the product of all factors need no further product with the update
    gram = u.mT @ u if tall else u @ u.mT
    eye = torch.eye(gram.shape[1], dtype=torch.float64, device=gram.device)
    whole = eye
    for _ in range(NS_STEPS):
        p = a * eye + gram @ (b * eye + c * gram)
        whole, gram = whole @ p, gram @ (p @ p)
    o = u @ whole if tall else whole @ u
    if not case["step"]:
        return {"out": o}
    return {"w": (1.0 - LR * DECAY) * s["w"].double() - LR * _step_scale(case) * o, "buf": buf}


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "expert": _exact_expert, "muon": _exact_muon}[case["op"]](case, s)
