"""The operators that train the MoE layer, as measurable cases.

Four operators, which one training step of the layer runs in this order:

  combine_backward    the gradient of the weighted combine: dout -> each kept
                      slot's row (times its routing weight), and the weights'
                      own gradient
  ffn_backward        the gradient of the experts' two products, GELU or
                      SwiGLU experts, with the weights' and biases' gradients
  dispatch_backward   the gradient of sorting the tokens by expert: each
                      token's slots' rows summed, plus what another path of
                      the same x has already
  adamw               the AdamW step over many tensors at once, moments in 32
                      or in 8 bits

``run`` computes a case with plain torch operations in 32 bits, rounded once
at the end, or, where ``own`` is true, through the framework's entry points.
"""
import math
import random

import torch

own = False

BLOCK = 256          # elements that share a scale in the 8-bit moments
TINY = 2.0 ** -100   # a block whose largest value is below this is held as zeros


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the fp32 layer of the framework's own tests: a call's latency
        {"name": "combine_bwd_tiny_f32", "op": "combine_backward", "T": 64, "H": 256, "E": 8, "K": 2, "cap": 0,
         "skew": 0.0, "dtype": "f32"},
        # the benchmark's prefill layer: batch 4 of 2048 tokens
        {"name": "combine_bwd_prefill", "op": "combine_backward", "T": 8192, "H": 3584, "E": 32, "K": 2, "cap": 0,
         "skew": 0.0, "dtype": "bf16"},
        # top-4 with Zipf-skewed experts and a capacity: half of the slots are dropped
        {"name": "combine_bwd_zipf_cap", "op": "combine_backward", "T": 16384, "H": 3584, "E": 32, "K": 4,
         "cap": 2048, "skew": 1.2, "dtype": "bf16"},
        # a short ragged batch
        {"name": "dispatch_bwd_short", "op": "dispatch_backward", "T": 37, "H": 3584, "E": 32, "K": 2, "cap": 0,
         "skew": 0.0, "add": False, "dtype": "bf16"},
        # the long wide layer of many narrow experts, added to the residual path's gradient
        {"name": "dispatch_bwd_wide", "op": "dispatch_backward", "T": 32768, "H": 4096, "E": 64, "K": 2, "cap": 0,
         "skew": 0.0, "add": True, "dtype": "bf16"},
        # the fp32 layer of the framework's own tests
        {"name": "ffn_bwd_tiny_f32", "op": "ffn_backward", "T": 64, "H": 256, "E": 8, "K": 2, "F": 512, "cap": 0,
         "skew": 0.0, "act": "gelu", "bias": True, "dtype": "f32"},
        # odd sizes throughout: no dimension a multiple of a tile, experts with few rows, biases
        {"name": "ffn_bwd_odd", "op": "ffn_backward", "T": 777, "H": 1000, "E": 12, "K": 3, "F": 1416, "cap": 0,
         "skew": 0.6, "act": "gelu", "bias": True, "dtype": "bf16"},
        # the benchmark's prefill layer
        {"name": "ffn_bwd_prefill", "op": "ffn_backward", "T": 8192, "H": 3584, "E": 32, "K": 2, "F": 2560, "cap": 0,
         "skew": 0.0, "act": "gelu", "bias": False, "dtype": "bf16"},
        # the same with SwiGLU experts
        {"name": "ffn_bwd_prefill_swiglu", "op": "ffn_backward", "T": 8192, "H": 3584, "E": 32, "K": 2, "F": 2560,
         "cap": 0, "skew": 0.0, "act": "swiglu", "bias": False, "dtype": "bf16"},
        # gates, norms and biases: many short tensors, where the call's latency counts
        {"name": "adamw_short_tensors", "op": "adamw", "layout": "mixed", "tensors": 96, "largest": 20000,
         "bits": 32, "grad": "f32"},
        # one layer of eight experts, a tensor for each expert's matrix
        {"name": "adamw_experts", "op": "adamw", "layout": "experts", "H": 3584, "E": 8, "F": 2560, "bits": 32,
         "grad": "bf16"},
        # the benchmark's layer of 32 experts with its moments in 8 bits
        {"name": "adamw_experts_8bit", "op": "adamw", "layout": "experts", "H": 3584, "E": 32, "F": 2560, "bits": 8,
         "grad": "bf16"},
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    def dim(lo, hi):
        return max(8, spread(lo, hi) // 8 * 8)

    op = rng.choice(["combine_backward", "dispatch_backward", "ffn_backward", "adamw"])
    if op == "adamw":
        bits, grad = rng.choice([8, 32]), rng.choice(["bf16", "f32"])
        if rng.random() < 0.5:
            return {"op": op, "layout": "mixed", "tensors": spread(1, 400), "largest": spread(1000, 4000000),
                    "bits": bits, "grad": grad}
        return {"op": op, "layout": "experts", "H": dim(256, 4096), "E": rng.randint(2, 16), "F": dim(256, 2816),
                "bits": bits, "grad": grad}
    E = spread(2, 64)
    K = rng.randint(1, min(E, 4))
    f32 = rng.random() < 0.25
    case = {"op": op, "T": spread(1, 16384), "H": dim(128, 4096), "E": E, "K": K,
            "skew": rng.choice([0.0, 0.0, 0.5, 1.0]), "dtype": "f32" if f32 else "bf16"}
    case["cap"] = -(-case["T"] // E) * K if rng.random() < 0.4 else 0
    if op == "dispatch_backward":
        case["add"] = rng.random() < 0.5
    if op == "ffn_backward":
        # fp32 layers are the checking ones: small
        if f32:
            case.update(T=spread(1, 300), H=dim(64, 384), F=dim(64, 640))
            case["cap"] = -(-case["T"] // E) * K if case["cap"] else 0
        else:
            case["F"] = dim(128, 2816)
            if not case["cap"]:
                case["skew"] = min(case["skew"], 0.5)
        case["act"] = rng.choice(["gelu", "gelu", "swiglu"])
        case["bias"] = rng.random() < 0.5
        # no more weights and no more products than the largest listed case
        top = work(next(c for c in listed() if c["name"] == "ffn_bwd_prefill_swiglu"))
        while work(case)["bytes"] > top["bytes"] and case["E"] > case["K"]:
            case["E"] -= 1
        while work(case)["flops"] > top["flops"] or work(case)["bytes"] > top["bytes"]:
            case["T"] = case["T"] * 3 // 4
        case["cap"] = -(-case["T"] // case["E"]) * case["K"] if case["cap"] else 0
    return case


def kept_rows(case):
    """The slots that the capacity keeps; with one, by each expert's share of a
    sample of tokens (the rows of a run follow its seed)."""
    T, E, K, cap = case["T"], case["E"], case["K"], case["cap"]
    if not cap:
        return T * K
    prior = -case["skew"] * torch.log(torch.arange(1, E + 1, dtype=torch.float32))
    scores = torch.randn((4096, E), generator=torch.Generator().manual_seed(1)) + prior
    share = torch.bincount(scores.topk(K, dim=1).indices.view(-1), minlength=E) / 4096.0
    return int((share * T).clamp(max=cap).sum())


def work(case):
    if case["op"] == "adamw":
        n = sum(tensor_sizes(case))
        state = 16 if case["bits"] == 32 else 4 + 16.0 / BLOCK
        return {"bytes": n * (8 + 2 + (2 if case["grad"] == "bf16" else 4) + state), "flops": 16.0 * n}
    T, H, E, K = case["T"], case["H"], case["E"], case["K"]
    es = 4 if case["dtype"] == "f32" else 2
    rows = kept_rows(case)
    if case["op"] == "combine_backward":
        return {"bytes": (T * H + 2 * rows * H) * es + T * K * 12, "flops": 3.0 * rows * H}
    if case["op"] == "dispatch_backward":
        return {"bytes": (T * H * (2 if case["add"] else 1) + rows * H) * es + T * K * 4, "flops": 1.0 * rows * H}
    F, G = case["F"], 2 if case["act"] == "swiglu" else 1
    weights = E * H * F * (G + 1)
    bias = E * (2 * G * F + H) * 4 if case["bias"] else 0
    # the first product again, its gradient's two products, the second's two
    return {"bytes": (rows * (3 * H + F) + 2 * weights) * es + bias, "flops": 2.0 * rows * H * F * (3 * G + 2)}


# ------------------------------------------------------------------ inputs

def dtype_of(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, shape, scale, dtype):
    return (torch.randn(shape, generator=g, device="cuda", dtype=dtype)).mul_(scale)


def uniform(g, shape, bound, dtype):
    return torch.empty(shape, device="cuda", dtype=dtype).uniform_(-bound, bound, generator=g)


def routing(case, g):
    """A token's K experts by random scores (skewed towards low experts), the
    slots grouped by expert in slot order, at most `cap` of them kept."""
    T, E, K, cap = case["T"], case["E"], case["K"], case["cap"]
    prior = -case["skew"] * torch.log(torch.arange(1, E + 1, device="cuda", dtype=torch.float32))
    scores = torch.randn((T, E), generator=g, device="cuda") + prior
    top, ids = scores.topk(K, dim=1)
    w = torch.softmax(top, dim=1).contiguous()
    flat = ids.reshape(-1)
    order = flat.sort(stable=True).indices
    count = torch.bincount(flat, minlength=E)
    begin = count.cumsum(0) - count
    rank = torch.empty_like(flat)
    rank[order] = torch.arange(T * K, device="cuda") - begin[flat[order]]
    kept_of = count.clamp(max=cap) if cap else count
    offs = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
    offs[1:] = kept_of.cumsum(0)
    pos = torch.where(rank < kept_of[flat], offs[flat] + rank, -1)
    rows = int(offs[E])
    src = torch.empty(rows, dtype=torch.int64, device="cuda")
    kept = pos >= 0
    src[pos[kept]] = torch.arange(T * K, device="cuda")[kept]
    return {"w": w, "pos": pos.to(torch.int32), "offs": offs.to(torch.int32), "src": src, "rows": rows,
            "full": min(T * K, E * cap) if cap else T * K, "longest": max(1, int(kept_of.max()))}


def with_unused(rows, full, fill):
    """A permuted buffer as a program holds it: sized for the most rows that
    the capacity allows, nothing meaningful behind the last kept one."""
    b = torch.full((full, rows.shape[1]), fill, dtype=rows.dtype, device="cuda")
    b[:rows.shape[0]] = rows
    return b


def tensor_sizes(case):
    """Elements of each tensor of an optimiser case."""
    if case["layout"] == "experts":
        gate, matrix = case["E"] * case["H"], case["H"] * case["F"]
        return [gate] + [matrix] * (2 * case["E"]) + [case["F"]] * case["E"]
    r = random.Random(case["tensors"] * 7919 + case["largest"])
    return [max(1, int(case["largest"] ** r.random())) for _ in range(case["tensors"])]


def encode(x, magnitude):
    """8-bit floating point (4 exponent, 3 mantissa bits) with a scale for each
    block: the largest value maps to 448; a non-zero magnitude stays non-zero."""
    b = x.view(-1, BLOCK)
    top = b.abs().amax(dim=1, keepdim=True)
    big = top >= TINY
    inv = torch.where(big, 448.0 / top, 0.0)
    y = (b * inv).clamp_(-448.0, 448.0)
    if magnitude:
        y = torch.where((b > 0) & big, y.clamp(min=2.0 ** -9), y)
    scale = torch.where(big, top * (1.0 / 448.0), 0.0)
    return y.to(torch.float8_e4m3fn).view(-1), scale.view(-1)


def decode(code, scale):
    return (code.float().view(-1, BLOCK) * scale[:, None]).view(-1)


def prepare(case, seed):
    g = generator(seed)
    if case["op"] == "adamw":
        return prepare_adamw(case, g)
    T, H, E, K = case["T"], case["H"], case["E"], case["K"]
    dt = dtype_of(case)
    s = {"case": case, **routing(case, g)}
    rows = s["rows"]
    if case["op"] == "combine_backward":
        s["dout"] = normal(g, (T, H), 0.02, dt)
        s["y_perm"] = with_unused(normal(g, (rows, H), 1.0, dt), s["full"], math.nan)
    elif case["op"] == "dispatch_backward":
        s["dx_perm"] = with_unused(normal(g, (rows, H), 0.02, dt), s["full"], math.nan)
        s["dx_add"] = normal(g, (T, H), 0.02, dt) if case["add"] else None
    else:
        F, G = case["F"], 2 if case["act"] == "swiglu" else 1
        bound = math.sqrt(6.0 / (H + F))
        s["W1"], s["W2"] = uniform(g, (E, G * F, H), bound, dt), uniform(g, (E, H, F), bound, dt)
        s["b1"] = uniform(g, (E, G * F), 0.1, torch.float32) if case["bias"] else None
        s["x_perm"] = with_unused(normal(g, (T, H), 1.0, dt)[s["src"] // K], s["full"], math.nan)
        dy = normal(g, (T, H), 0.02, dt)[s["src"] // K] * s["w"].view(-1)[s["src"], None].to(dt)
        s["dy_perm"] = with_unused(dy, s["full"], math.nan)
        # the hidden rows as the forward pass left them
        s["h_perm"] = torch.full((s["full"], F), math.nan, device="cuda", dtype=dt)
        cut = s["offs"].tolist()
        for e in range(E):
            a = s["x_perm"][cut[e]:cut[e + 1]].float() @ s["W1"][e].float().mT
            a = a + s["b1"][e] if case["bias"] else a
            h = gelu(a) if G == 1 else a[:, :F] * torch.sigmoid(a[:, :F]) * a[:, F:]
            s["h_perm"][cut[e]:cut[e + 1]] = h.to(dt)
    return s


def prepare_adamw(case, g):
    """Every tensor has its place in one buffer of each kind, its start on a
    multiple of the block, zeros behind its end."""
    sizes = tensor_sizes(case)
    starts, n = [], 0
    for k in sizes:
        starts.append(n)
        n += -(-k // BLOCK) * BLOCK
    inside = torch.zeros(n, device="cuda")
    keep = torch.ones(n, device="cuda")
    lr, wd = 3e-4, 0.1
    for a, k in zip(starts, sizes):
        inside[a:a + k] = 1.0
        keep[a:a + k] = 1.0 - lr * wd if k > 20000 else 1.0     # short tensors do not decay
    p = normal(g, (n,), 0.02, torch.float32) * inside
    grad = normal(g, (n,), 1e-3, torch.float32) * inside
    m = normal(g, (n,), 3e-4, torch.float32) * inside
    v = (normal(g, (n,), 1e-3, torch.float32) * inside).square_().add_(1e-10 * inside)
    s = {"case": case, "sizes": sizes, "starts": starts, "keep": keep, "p": p, "p16": p.to(torch.bfloat16),
         "grad": grad.to(torch.bfloat16) if case["grad"] == "bf16" else grad,
         "grad_scale": torch.full((1,), 0.75, device="cuda"), "lr": lr, "wd": wd, "beta1": 0.9, "beta2": 0.95,
         "eps": 1e-8, "step": 100}
    if case["bits"] == 8:
        s["m"], s["m_scale"] = encode(m, False)
        s["v"], s["v_scale"] = encode(v.sqrt_(), True)
    else:
        s["m"], s["v"] = m, v
    return s


# ------------------------------------------------------------------ plain forms

def gelu(a):
    return 0.5 * a * (1.0 + torch.erf(a * math.sqrt(0.5)))


def gelu_slope(a):
    return 0.5 * (1.0 + torch.erf(a * math.sqrt(0.5))) + a * torch.exp(-0.5 * a * a) * (1.0 / math.sqrt(2 * math.pi))


def plain_combine_backward(s):
    T, K, dt = s["case"]["T"], s["case"]["K"], dtype_of(s["case"])
    dout, src, pos = s["dout"].float(), s["src"], s["pos"].view(T, K)
    dy = dout[src // K] * s["w"].view(-1)[src, None]
    y = s["y_perm"].float()[pos.clamp(min=0).long()]
    dw = torch.where(pos >= 0, (dout[:, None, :] * y).sum(-1), 0.0)
    return {"dy_perm": with_unused(dy.to(dt), s["full"], 0.0), "dw": dw}


def plain_dispatch_backward(s):
    T, K, dt = s["case"]["T"], s["case"]["K"], dtype_of(s["case"])
    pos = s["pos"].view(T, K)
    picked = s["dx_perm"].float()[pos.clamp(min=0).long()]
    dx = torch.where((pos >= 0)[..., None], picked, 0.0).sum(1)
    if s["dx_add"] is not None:
        dx = dx + s["dx_add"].float()
    return {"dx": dx.to(dt)}


def plain_ffn_backward(s):
    """The experts' rows padded to the longest expert, then batched products."""
    case, dt = s["case"], dtype_of(s["case"])
    F, M = case["F"], s["longest"]
    offs = s["offs"].long()
    at = offs[:-1, None] + torch.arange(M, device="cuda")
    real = (at < offs[1:, None])[..., None]
    at = at.clamp(max=s["rows"] - 1)
    x = torch.where(real, s["x_perm"].float()[at], 0.0)
    dy = torch.where(real, s["dy_perm"].float()[at], 0.0)
    h = torch.where(real, s["h_perm"].float()[at], 0.0)
    W1, W2 = s["W1"].float(), s["W2"].float()
    a = torch.bmm(x, W1.mT)
    if s["b1"] is not None:
        a = a + s["b1"][:, None, :]
    dh = torch.bmm(dy, W2)
    if case["act"] == "swiglu":
        gate, up = a[..., :F], a[..., F:]
        sig = torch.sigmoid(gate)
        da = torch.cat([dh * up * sig * (1.0 + gate * (1.0 - sig)), dh * gate * sig], dim=-1)
    else:
        da = dh * gelu_slope(a)
    r = torch.arange(s["rows"], device="cuda")
    e = torch.searchsorted(offs[1:].contiguous(), r, right=True)
    dx = torch.bmm(da, W1)[e, r - offs[e]]
    out = {"dx_perm": with_unused(dx.to(dt), s["full"], 0.0), "dW1": torch.bmm(da.mT, x).to(dt),
           "dW2": torch.bmm(dy.mT, h).to(dt)}
    if case["bias"]:
        out["db1"], out["db2"] = da.sum(1), dy.sum(1)
    return out


def plain_adamw(s):
    case = s["case"]
    b1, b2, step = s["beta1"], s["beta2"], s["step"]
    g = s["grad"].float() * s["grad_scale"]
    if case["bits"] == 8:
        m, r = decode(s["m"], s["m_scale"]), decode(s["v"], s["v_scale"])
        v = r * r
    else:
        m, v = s["m"], s["v"]
    m = m * b1 + g * (1.0 - b1)
    v = v * b2 + (g * g) * (1.0 - b2)
    r = v.sqrt()
    denom = r * (1.0 / math.sqrt(1.0 - b2 ** step)) + s["eps"]
    s["p"] = s["p"] * s["keep"] - (m / denom) * (s["lr"] / (1.0 - b1 ** step))
    s["p16"] = s["p"].to(torch.bfloat16)
    if case["bits"] == 8:
        s["m"], s["m_scale"] = encode(m, False)
        s["v"], s["v_scale"] = encode(r, True)
    else:
        s["m"], s["v"] = m, v
    return adamw_outputs(s)


def adamw_outputs(s):
    return {k: s[k] for k in ("p", "p16", "m", "v", "m_scale", "v_scale") if k in s}


# ------------------------------------------------------------------ the framework's calls

def layer_plan(s):
    """The description, workspace and result buffers that a program keeps."""
    import sparse_mixture_experts_topk_gb300 as moe
    case = s["case"]
    T, H, E, K, dt = case["T"], case["H"], case["E"], case["K"], dtype_of(case)
    F = case.get("F", 8)
    flags = moe.MOE_FLAG_SWIGLU if case.get("act") == "swiglu" else 0
    d = moe.make_desc(T, H, E, K, F, case["cap"], moe.MOE_F32 if case["dtype"] == "f32" else moe.MOE_BF16, flags)

    def buf(shape, dtype=dt):
        return torch.empty(shape, dtype=dtype, device="cuda")

    plan = {"moe": moe, "desc": d}
    rows = torch.zeros((s["full"], H), dtype=dt, device="cuda")     # those behind the last kept one stay as they are
    if case["op"] == "combine_backward":
        plan["out"] = {"dy_perm": rows, "dw": buf((T, K), torch.float32)}
    elif case["op"] == "dispatch_backward":
        plan["out"] = {"dx": buf((T, H))}
    else:
        plan["ws"] = moe.backward_workspace(d)
        plan["out"] = {"dx_perm": rows, "dW1": torch.empty_like(s["W1"]), "dW2": torch.empty_like(s["W2"])}
        if case["bias"]:
            plan["out"]["db1"], plan["out"]["db2"] = torch.empty_like(s["b1"]), buf((E, H), torch.float32)
    return plan


def adamw_plan(s):
    import sparse_mixture_experts_topk_gb300 as moe
    case, tensors = s["case"], []
    for a, k in zip(s["starts"], s["sizes"]):
        t = {"p": s["p"][a:a + k], "g": s["grad"][a:a + k], "m": s["m"][a:a + k], "v": s["v"][a:a + k],
             "p16": s["p16"][a:a + k], "weight_decay": s["wd"] if k > 20000 else 0.0}
        if case["bits"] == 8:
            blocks = slice(a // BLOCK, a // BLOCK + -(-k // BLOCK))
            t["m_scale"], t["v_scale"] = s["m_scale"][blocks], s["v_scale"][blocks]
        tensors.append(t)
    params = moe.make_adamw(lr=s["lr"], beta1=s["beta1"], beta2=s["beta2"], eps=s["eps"], step=s["step"])
    return {"moe": moe, "tensors": moe.adamw_tensors(tensors), "params": params}


def own_run(s):
    op = s["case"]["op"]
    if "plan" not in s:
        s["plan"] = adamw_plan(s) if op == "adamw" else layer_plan(s)
    q = s["plan"]
    moe = q["moe"]
    if op == "adamw":
        moe.moe_adamw_step(q["tensors"], q["params"], s["grad_scale"], None)
        return adamw_outputs(s)
    o = q["out"]
    if op == "combine_backward":
        moe.moe_combine_backward(q["desc"], s["dout"], s["y_perm"], s["pos"], s["w"], o["dy_perm"], o["dw"])
    elif op == "dispatch_backward":
        moe.moe_dispatch_backward(q["desc"], s["dx_perm"], s["pos"], s["dx_add"], o["dx"])
    else:
        moe.moe_expert_ffn_backward(q["desc"], s["x_perm"], s["h_perm"], s["dy_perm"], s["offs"], s["W1"], s["b1"],
                                    s["W2"], o["dx_perm"], o["dW1"], o.get("db1"), o["dW2"], o.get("db2"), q["ws"])
    return o


def run(state):
    if own:
        return own_run(state)
    return {"combine_backward": plain_combine_backward, "dispatch_backward": plain_dispatch_backward,
            "ffn_backward": plain_ffn_backward, "adamw": plain_adamw}[state["case"]["op"]](state)


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "adamw":
        return exact_adamw(s)
    T, K = case["T"], case["K"]
    pos = s["pos"].view(T, K).long()
    if case["op"] == "combine_backward":
        dout, w = s["dout"].double(), s["w"].double()
        dy = torch.zeros((s["full"], case["H"]), dtype=torch.float64, device="cuda")
        dw = torch.zeros((T, K), dtype=torch.float64, device="cuda")
        for j in range(K):
            t = torch.nonzero(pos[:, j] >= 0).view(-1)
            r = pos[t, j]
            dy[r] = dout[t] * w[t, j, None]
            dw[t, j] = torch.einsum("th,th->t", dout[t], s["y_perm"][r].double())
        return {"dy_perm": dy, "dw": dw}
    if case["op"] == "dispatch_backward":
        dx = s["dx_add"].double() if case["add"] else torch.zeros((T, case["H"]), dtype=torch.float64, device="cuda")
        dx = dx.index_add(0, s["src"] // K, s["dx_perm"][:s["rows"]].double())
        return {"dx": dx}
    F, cut = case["F"], s["offs"].tolist()
    out = {"dx_perm": torch.zeros_like(s["x_perm"], dtype=torch.float64),
           "dW1": torch.empty_like(s["W1"], dtype=torch.float64),
           "dW2": torch.empty_like(s["W2"], dtype=torch.float64)}
    if case["bias"]:
        out["db1"] = torch.empty_like(s["b1"], dtype=torch.float64)
        out["db2"] = torch.empty((case["E"], case["H"]), dtype=torch.float64, device="cuda")
    for e in range(case["E"]):
        rows = slice(cut[e], cut[e + 1])
        x, h, dy = (s[k][rows].double() for k in ("x_perm", "h_perm", "dy_perm"))
        W1, W2 = s["W1"][e].double(), s["W2"][e].double()
        a = x @ W1.T + (s["b1"][e].double() if case["bias"] else 0.0)
        dh = dy @ W2
        if case["act"] == "swiglu":
            z, u = a[:, :F], a[:, F:]
            q = 1.0 / (1.0 + torch.exp(-z))
            da = torch.cat([dh * u * (q + z * q * (1.0 - q)), dh * (z * q)], dim=1)
        else:
            da = dh * (torch.special.ndtr(a) + a * torch.exp(-a * a / 2) / math.sqrt(2 * math.pi))
        out["dx_perm"][rows] = da @ W1
        out["dW1"][e], out["dW2"][e] = da.T @ x, dy.T @ h
        if case["bias"]:
            out["db1"][e], out["db2"][e] = da.sum(0), dy.sum(0)
    return out


def exact_adamw(s):
    b1, b2, t, eight = s["beta1"], s["beta2"], s["step"], s["case"]["bits"] == 8
    g = s["grad"].double() * s["grad_scale"].double()
    m0, v0 = s["m"].double(), s["v"].double()
    if eight:
        m0 = m0 * s["m_scale"].double().repeat_interleave(BLOCK)
        v0 = (v0 * s["v_scale"].double().repeat_interleave(BLOCK)).square()
    m = b1 * m0 + (1 - b1) * g
    v = b2 * v0 + (1 - b2) * g.square()
    hat = (m / (1 - b1 ** t)) / ((v / (1 - b2 ** t)).sqrt() + s["eps"])
    p = s["p"].double() * s["keep"].double() - s["lr"] * hat
    out = {"p": p, "p16": p}
    if not eight:
        return {**out, "m": m, "v": v}
    # the codes' roundings are not computed numbers of 64 bits; their scales are
    r = v.sqrt()
    return {**out, "m": None, "v": None, "m_scale": m.view(-1, BLOCK).abs().amax(1) / 448,
            "v_scale": r.view(-1, BLOCK).amax(1) / 448}
