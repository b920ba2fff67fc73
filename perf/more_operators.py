"""What a training step of the MoE layer needs beside the experts' gradients
and AdamW, as measurable cases.

Four operators:

  balance_loss      the load-balancing loss over the tokens that count (a
                    padded batch has a mask), with the per-expert counts and
                    probability sums that its gradient needs
  router_backward   the gradient of the router: of the renormalised top-k
                    weights and of the balance loss through the softmax, and
                    of the gate's product: the gate matrix' gradient and x's
  orthogonalize     matrices made nearly orthogonal by Newton-Schulz products
  muon_step         the Muon step over many matrices: momentum, the
                    orthogonalised update, weight decay, the bf16 copy

``run`` computes a case with plain torch operations in 32 bits, rounded once
at the end, or, where ``own`` is true, through the framework's entry points.
"""
import math
import random

import torch

own = False

# the quintic iteration X <- (a + b XX' + c (XX')^2) X
NS = (3.4445, -4.7750, 2.0315)
ITERATIONS = 5


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the fp32 layer of the framework's own tests: a call's latency
        {"name": "balance_tiny", "op": "balance_loss", "T": 64, "E": 8, "K": 2, "skew": 0.0, "length": 0, "tau": 1.0},
        # the benchmark's prefill batch, 4 sequences of up to 2048 tokens, padded
        {"name": "balance_prefill_padded", "op": "balance_loss", "T": 8192, "E": 32, "K": 2, "skew": 0.0,
         "length": 2048, "tau": 1.0},
        # the most experts and choices that a layer has, a long batch with uneven experts
        {"name": "balance_many_experts", "op": "balance_loss", "T": 131072, "E": 256, "K": 8, "skew": 0.7,
         "length": 0, "tau": 1.0},
        # the fp32 layer of the framework's own tests, with a gate bias
        {"name": "router_bwd_tiny_f32", "op": "router_backward", "T": 64, "H": 256, "E": 8, "K": 2, "skew": 0.0,
         "length": 0, "tau": 1.0, "bias": True, "dlogits": True, "dtype": "f32"},
        # odd sizes throughout, padded sequences, a softer router
        {"name": "router_bwd_odd", "op": "router_backward", "T": 777, "H": 1000, "E": 12, "K": 3, "skew": 0.6,
         "length": 111, "tau": 2.0, "bias": True, "dlogits": True, "dtype": "bf16"},
        # the benchmark's prefill layer
        {"name": "router_bwd_prefill", "op": "router_backward", "T": 8192, "H": 3584, "E": 32, "K": 2, "skew": 0.0,
         "length": 0, "tau": 1.0, "bias": False, "dlogits": False, "dtype": "bf16"},
        # the long wide layer of many narrow experts, padded sequences of up to 4096 tokens
        {"name": "router_bwd_wide_padded", "op": "router_backward", "T": 32768, "H": 4096, "E": 64, "K": 2,
         "skew": 0.5, "length": 4096, "tau": 1.0, "bias": False, "dlogits": False, "dtype": "bf16"},
        # one small matrix: the call's latency
        {"name": "orthogonalize_short", "op": "orthogonalize", "batch": 1, "rows": 64, "cols": 96, "dtype": "f32"},
        # odd tall matrices, no dimension a multiple of a tile
        {"name": "orthogonalize_odd", "op": "orthogonalize", "batch": 3, "rows": 1416, "cols": 1001, "dtype": "bf16"},
        # the experts of the framework's small training example
        {"name": "muon_small_experts", "op": "muon_step", "layout": "experts", "H": 256, "E": 8, "F": 512, "G": 1,
         "grad": "f32"},
        # eight experts of the benchmark's prefill layer
        {"name": "muon_experts", "op": "muon_step", "layout": "experts", "H": 3584, "E": 8, "F": 2560, "G": 1,
         "grad": "bf16"},
        # narrow SwiGLU experts of the wide layer: gate and up projection are matrices of their own
        {"name": "muon_wide_swiglu", "op": "muon_step", "layout": "experts", "H": 4096, "E": 16, "F": 1408, "G": 2,
         "grad": "bf16"},
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    def dim(lo, hi):
        return max(8, spread(lo, hi) // 8 * 8)

    op = rng.choice(["balance_loss", "router_backward", "orthogonalize", "muon_step"])
    if op == "orthogonalize":
        # any sizes at all, the batch as far as the largest listed case's work
        case = {"op": op, "batch": 1, "rows": spread(1, 4096), "cols": spread(1, 4096),
                "dtype": rng.choice(["f32", "bf16"])}
        case["batch"] = max(1, min(spread(1, 16), int(2e12 / work(case)["flops"])))
        return case
    if op == "muon_step":
        grad = rng.choice(["bf16", "f32"])
        if rng.random() < 0.5:
            return {"op": op, "layout": "mixed", "tensors": spread(1, 24), "largest": spread(64, 2048), "grad": grad}
        case = {"op": op, "layout": "experts", "H": dim(64, 4096), "E": 1, "F": dim(64, 2816), "G": rng.randint(1, 2),
                "grad": grad}
        case["E"] = max(1, min(spread(1, 16), int(4e12 / work(case)["flops"])))
        return case
    E = spread(2, 256)
    K = rng.randint(1, min(E, 8))
    case = {"op": op, "T": spread(1, 65536), "E": E, "K": K, "skew": rng.choice([0.0, 0.0, 0.5, 1.0]),
            "length": 0, "tau": rng.choice([1.0, 1.0, 0.5, 2.0])}
    if op == "router_backward":
        f32 = rng.random() < 0.25
        case.update(H=dim(64, 4096), bias=rng.random() < 0.5, dlogits=rng.random() < 0.5,
                    dtype="f32" if f32 else "bf16")
        # fp32 layers are the checking ones: small
        if f32:
            case.update(T=spread(1, 1000), H=dim(64, 1024))
        top = work(next(c for c in listed() if c["name"] == "router_bwd_wide_padded"))
        while any(work(case)[k] > top[k] for k in top):
            case["T"] = case["T"] * 3 // 4
    if rng.random() < 0.5:
        case["length"] = spread(1, max(1, case["T"]))
    return case


def shapes(case):
    """(matrices, rows, columns) of each tensor of an optimiser case."""
    if case["layout"] == "experts":
        return [(case["E"] * case["G"], case["F"], case["H"]), (case["E"], case["H"], case["F"])]
    r = random.Random(case["tensors"] * 7919 + case["largest"])
    return [(r.choice((1, 1, 2)), max(1, int(case["largest"] ** r.random())), max(1, int(case["largest"] ** r.random())))
            for _ in range(case["tensors"])]


def newton_schulz_flops(batch, rows, cols):
    """X X' and its square are symmetric: half of each is enough."""
    s, n = min(rows, cols), max(rows, cols)
    return ITERATIONS * batch * (3.0 * s * s * n + 1.0 * s * s * s)


def work(case):
    op = case["op"]
    if op == "orthogonalize":
        n = case["batch"] * case["rows"] * case["cols"]
        return {"bytes": n * (2 + (4 if case["dtype"] == "f32" else 2)),
                "flops": newton_schulz_flops(case["batch"], case["rows"], case["cols"])}
    if op == "muon_step":
        n = sum(b * r * c for b, r, c in shapes(case))
        return {"bytes": n * (8 + 8 + 2 + (2 if case["grad"] == "bf16" else 4)),
                "flops": sum(newton_schulz_flops(*s) for s in shapes(case)) + 10.0 * n}
    T, E, K = case["T"], case["E"], case["K"]
    mask = T if case["length"] else 0
    if op == "balance_loss":
        return {"bytes": T * E * 4 + T * K * 4 + mask + E * 8, "flops": 5.0 * T * E}
    H, es = case["H"], 4 if case["dtype"] == "f32" else 2
    return {"bytes": 2 * T * H * es + T * E * (8 if case["dlogits"] else 4) + T * K * 8 + mask + E * H * (es + 4),
            "flops": 4.0 * T * E * H + 10.0 * T * E}


# ------------------------------------------------------------------ inputs

def dtype_of(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, shape, scale, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype).mul_(scale)


def update_like(g, batch, rows, cols, scale):
    """A gradient as a layer's matrix has it: a few directions that many
    tokens share over the noise of the rest."""
    noise = normal(g, (batch, rows, cols), scale)
    rank = min(4, rows, cols)
    left, right = normal(g, (batch, rows, rank), 1.0), normal(g, (batch, rank, cols), scale)
    return noise + left @ right


def routing(case, g):
    """Scores skewed towards low experts, each token's K best, and for padded
    sequences of ``length`` tokens the mask of the real ones."""
    T, E, K = case["T"], case["E"], case["K"]
    prior = -case["skew"] * torch.log(torch.arange(1, E + 1, device="cuda", dtype=torch.float32))
    s = {"case": case, "logits": normal(g, (T, E), 1.0) + prior, "mask": None}
    s["ids"] = s["logits"].topk(K, dim=1).indices.to(torch.int32).contiguous()
    if case["length"]:
        rows = -(-T // case["length"])
        real = torch.randint(1, case["length"] + 1, (rows, 1), generator=g, device="cuda")
        real[0] = case["length"]
        s["mask"] = (torch.arange(case["length"], device="cuda") < real).view(-1)[:T].contiguous()
        s["logits"][~s["mask"]] = math.nan     # nothing meaningful in the padding
    return s


def prepare(case, seed):
    g = generator(seed)
    if case["op"] == "orthogonalize":
        x = update_like(g, case["batch"], case["rows"], case["cols"], 1e-3)
        return {"case": case, "x": x.to(dtype_of(case["dtype"]))}
    if case["op"] == "muon_step":
        s = {"case": case, "p": [], "p16": [], "g": [], "m": [], "lr": 3e-4, "wd": 0.1, "mu": 0.95,
             "grad_scale": torch.full((1,), 0.75, device="cuda")}
        for b, r, c in shapes(case):
            p = normal(g, (b, r, c), 0.02)
            s["p"].append(p)
            s["p16"].append(p.to(torch.bfloat16))
            s["g"].append(update_like(g, b, r, c, 1e-3).to(dtype_of(case["grad"])))
            s["m"].append(update_like(g, b, r, c, 3e-3))
        return s
    s = routing(case, g)
    if case["op"] == "balance_loss":
        return s
    T, H, E, K, dt = case["T"], case["H"], case["E"], case["K"], dtype_of(case["dtype"])
    s["x"] = normal(g, (T, H), 1.0, dt)
    bound = math.sqrt(6.0 / (H + E))
    s["Wg"] = torch.empty((E, H), device="cuda", dtype=dt).uniform_(-bound, bound, generator=g)
    s["dw"] = normal(g, (T, K), 1.0 / T)
    s["dloss"] = torch.full((1,), 0.5, device="cuda")
    if s["mask"] is not None:
        s["x"][~s["mask"]] = math.nan
        s["dw"][~s["mask"]] = math.nan
    # the counts that the loss' call left
    real = s["ids"].long() if s["mask"] is None else s["ids"].long()[s["mask"]]
    s["count"] = torch.bincount(real.view(-1), minlength=E).to(torch.int32)
    s["tokens"] = torch.full((1,), real.shape[0], dtype=torch.int32, device="cuda")
    return s


# ------------------------------------------------------------------ plain forms

def softmax(l):
    e = torch.exp(l - l.amax(dim=-1, keepdim=True))
    return e / e.sum(dim=-1, keepdim=True)


def masked(s, rows, value):
    return rows if s["mask"] is None else torch.where(s["mask"][:, None], rows, value)


def plain_balance_loss(s):
    case = s["case"]
    T, E, K = case["T"], case["E"], case["K"]
    p = masked(s, softmax(masked(s, s["logits"], 0.0) / case["tau"]), 0.0)
    psum = p.sum(0, dtype=torch.float64).float()
    slot = masked(s, s["ids"], E).long().view(-1)      # the padding's slots go behind the last expert
    count = torch.zeros(E + 1, dtype=torch.int32, device="cuda").index_add_(0, slot, torch.ones_like(slot, dtype=torch.int32))
    count = count[:E]
    tokens = torch.full((1,), T, dtype=torch.int32, device="cuda") if s["mask"] is None else \
        s["mask"].sum().to(torch.int32).view(1)
    n = tokens.double().clamp(min=1)
    loss = (E * (count.double() / (n * K) * (psum.double() / n)).sum(0, keepdim=True)).float()
    return {"psum": psum, "count": count, "tokens": tokens, "loss": loss}


def plain_router_backward(s):
    case, dt = s["case"], dtype_of(s["case"]["dtype"])
    E, K = case["E"], case["K"]
    l, ids = masked(s, s["logits"], 0.0) / case["tau"], s["ids"].long()
    p, w, dw = softmax(l), softmax(l.gather(1, ids)), masked(s, s["dw"], 0.0)
    n = s["tokens"].double()
    c = (s["dloss"].double() * E * s["count"].double() / (n * n * K)).float()
    dl = p * (c - (p * c).sum(1, keepdim=True))
    dl = dl.scatter_add(1, ids, w * (dw - (w * dw).sum(1, keepdim=True)))
    dl = masked(s, dl / case["tau"], 0.0)
    x = masked(s, s["x"].float(), 0.0)
    out = {"dWg": dl.mT @ x, "dx": (dl @ s["Wg"].float()).to(dt)}
    if case["bias"]:
        out["dbias"] = dl.sum(0)
    if case["dlogits"]:
        out["dlogits"] = dl
    return out


def newton_schulz(u):
    a, b, c = NS
    x = u / torch.sqrt((u * u).sum(dim=(1, 2), keepdim=True))
    tall = u.shape[1] > u.shape[2]
    x = x.mT if tall else x
    for _ in range(ITERATIONS):
        A = torch.bmm(x, x.mT)
        x = a * x + torch.bmm(b * A + c * torch.bmm(A, A), x)
    return x.mT if tall else x


def plain_orthogonalize(s):
    return {"out": newton_schulz(s["x"].float()).to(torch.bfloat16).contiguous()}


def plain_muon_step(s):
    for i, (p, g, m) in enumerate(zip(s["p"], s["g"], s["m"])):
        g = g.float() * s["grad_scale"]
        s["m"][i] = m = m * s["mu"] + g
        step = s["lr"] * 0.2 * math.sqrt(max(p.shape[1:]))
        s["p"][i] = p * (1.0 - s["lr"] * s["wd"]) - step * newton_schulz(g + s["mu"] * m)
        s["p16"][i] = s["p"][i].to(torch.bfloat16)
    return {k: list(s[k]) for k in ("p", "p16", "m")}


# ------------------------------------------------------------------ the framework's calls

def plan_of(s):
    """The description, workspace and result buffers that a program keeps."""
    import sparse_mixture_experts_topk_gb300 as moe
    case, plan = s["case"], {"moe": moe}

    def buf(*shape, dtype=torch.float32):
        return torch.empty(shape, dtype=dtype, device="cuda")

    if case["op"] == "orthogonalize":
        plan["out"] = {"out": torch.empty_like(s["x"], dtype=torch.bfloat16)}
        plan["ws"] = moe.orthogonalize_workspace(case["batch"], case["rows"], case["cols"])
        return plan
    if case["op"] == "muon_step":
        plan["tensors"] = moe.muon_tensors(
            [{"p": p, "p16": p16, "g": g, "m": m, "weight_decay": s["wd"], "scale": 0.2 * math.sqrt(max(p.shape[1:]))}
             for p, p16, g, m in zip(s["p"], s["p16"], s["g"], s["m"])])
        plan["params"] = moe.make_muon(lr=s["lr"], momentum=s["mu"], nesterov=True, iterations=ITERATIONS)
        plan["ws"] = moe.muon_workspace(plan["tensors"])
        return plan
    T, E, K, H = case["T"], case["E"], case["K"], case.get("H", 8)
    plan["desc"] = moe.make_desc(T, H, E, K, 8, dtype=moe.MOE_BF16 if case.get("dtype") == "bf16" else moe.MOE_F32,
                                 temperature=case["tau"])
    plan["ws"] = moe.router_backward_workspace(plan["desc"])
    if case["op"] == "balance_loss":
        plan["out"] = {"psum": buf(E), "count": buf(E, dtype=torch.int32), "tokens": buf(1, dtype=torch.int32),
                       "loss": buf(1)}
    else:
        plan["out"] = {"dWg": buf(E, H), "dx": torch.empty_like(s["x"])}
        if case["bias"]:
            plan["out"]["dbias"] = buf(E)
        if case["dlogits"]:
            plan["out"]["dlogits"] = buf(T, E)
    return plan


def own_run(s):
    if "plan" not in s:
        s["plan"] = plan_of(s)
    q, op = s["plan"], s["case"]["op"]
    moe, o = q["moe"], q.get("out")
    if op == "balance_loss":
        moe.moe_balance_loss(q["desc"], s["logits"], s["ids"], s["mask"], o["psum"], o["count"], o["tokens"], o["loss"],
                             q["ws"])
    elif op == "router_backward":
        moe.moe_router_backward(q["desc"], s["x"], s["Wg"], s["logits"], s["ids"], s["dw"], s["dloss"], s["count"],
                                s["tokens"], s["mask"], o.get("dlogits"), o["dWg"], o.get("dbias"), o["dx"], q["ws"])
    elif op == "orthogonalize":
        moe.moe_orthogonalize(s["x"], o["out"], ITERATIONS, q["ws"])
    else:
        moe.moe_muon_step(q["tensors"], q["params"], s["grad_scale"], None, q["ws"])
        return {k: list(s[k]) for k in ("p", "p16", "m")}
    return o


def run(state):
    if own:
        return own_run(state)
    return {"balance_loss": plain_balance_loss, "router_backward": plain_router_backward,
            "orthogonalize": plain_orthogonalize, "muon_step": plain_muon_step}[state["case"]["op"]](state)


# ------------------------------------------------------------------ the definition in 64 bits

def exact_orthogonal(u):
    """The iteration on the smaller side's Gram matrix: the polynomial's
    factors are gathered, then applied to the matrix once."""
    a, b, c = NS
    u = u.double()
    s, tall = min(u.shape), u.shape[0] > u.shape[1]
    u = u / torch.linalg.matrix_norm(u)
    gram = u.T @ u if tall else u @ u.T
    one = torch.eye(s, dtype=torch.float64, device="cuda")
    total = one
    for _ in range(ITERATIONS):
        step = a * one + b * gram + c * (gram @ gram)
        total, gram = step @ total, step @ gram @ step
    return u @ total if tall else total @ u


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "orthogonalize":
        return {"out": torch.stack([exact_orthogonal(u) for u in s["x"]])}
    if op == "muon_step":
        out = {"p": [], "p16": [], "m": []}
        for p, g, m in zip(s["p"], s["g"], s["m"]):
            g = s["grad_scale"].double() * g.double()
            m = g + s["mu"] * m.double()
            O = torch.stack([exact_orthogonal(u) for u in s["mu"] * m + g])
            p = p.double() - s["lr"] * (s["wd"] * p.double() + 0.2 * max(p.shape[1:]) ** 0.5 * O)
            out["p"].append(p)
            out["p16"].append(p)
            out["m"].append(m)
        return out
    T, E, K, tau = case["T"], case["E"], case["K"], case["tau"]
    real = torch.arange(T, device="cuda") if s["mask"] is None else torch.nonzero(s["mask"]).view(-1)
    z = s["logits"][real].double() / tau
    p = torch.exp(z - torch.logsumexp(z, dim=1, keepdim=True))
    if op == "balance_loss":
        count = torch.bincount(s["ids"][real].long().view(-1), minlength=E)
        n = len(real)
        loss = torch.dot(count.double(), p.sum(0)).view(1) * (E / (n * K) / n)
        return {"psum": p.sum(0), "count": None, "tokens": None, "loss": loss}
    n = float(s["tokens"])
    c = s["dloss"].double() * s["count"].double() * (E / (n * K) / n)
    rows = p * (c - torch.mv(p, c)[:, None])
    chosen = s["ids"][real].long()
    pk = p.gather(1, chosen)
    w = pk / pk.sum(1, keepdim=True)
    dw = s["dw"][real].double()
    # the quotient's gradient, then the softmax': dp_j = (dw_j - <w, dw>) / sum, dl = p (dp - <p, dp>), <p, dp> = 0
    rows.scatter_add_(1, chosen, w * (dw - torch.einsum("tk,tk->t", w, dw)[:, None]))
    dl = torch.zeros((T, E), dtype=torch.float64, device="cuda")
    dl[real] = rows / tau
    out = {"dWg": torch.einsum("te,th->eh", dl[real], s["x"][real].double()), "dx": dl @ s["Wg"].double()}
    if case["bias"]:
        out["dbias"] = dl.sum(0)
    if case["dlogits"]:
        out["dlogits"] = dl
    return out
