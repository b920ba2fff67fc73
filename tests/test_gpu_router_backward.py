"""The balance loss and the router's gradient against a plain implementation
in 64 bits: every lane layout of the experts, one token, padded batches whose
padding holds NaN, temperatures, ids without an expert, each result alone."""
import numpy as np
import pytest

import sparse_mixture_experts_topk_gb300 as moe

pytestmark = pytest.mark.gpu

U32, U16 = 2.0 ** -24, 2.0 ** -8      # half a step of fp32 and of bf16, relative


def t_():
    import torch
    return torch


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sparse_mixture_experts_topk_gb300 import build
    build.build()


def case(T, H, E, K, dtype="bf16", mask=False, tau=1.0, missing=False, seed=0, poison=True):
    """Inputs as numpy fp64 of the values that the call reads, and their tensors."""
    r = np.random.default_rng([seed, T, H, E, K])
    t = t_()
    td = t.bfloat16 if dtype == "bf16" else t.float32

    def dev(a, dt):
        return t.from_numpy(np.asarray(a)).to("cuda").to(dt).contiguous()

    c = {"T": T, "H": H, "E": E, "K": K, "dtype": dtype, "tau": tau}
    logits = r.standard_normal((T, E)).astype(np.float32) * 2
    ids = np.argsort(-logits, axis=1, kind="stable")[:, :K].astype(np.int32) if T else np.zeros((0, K), np.int32)
    if missing:
        ids[r.random((T, K)) < 0.3] = -1
    x, Wg = dev(r.standard_normal((T, H)), td), dev(r.standard_normal((E, H)) * 0.1, td)
    dw = r.standard_normal((T, K)).astype(np.float32)
    m = r.random(T) < 0.6 if mask else np.ones(T, bool)
    c["mask"] = m
    c["t"] = {"logits": dev(logits, t.float32), "ids": dev(ids, t.int32), "x": x, "Wg": Wg, "dw": dev(dw, t.float32),
              "dloss": t.full((1,), 0.7, device="cuda"), "mask": dev(m, t.bool) if mask else None}
    c["n"] = {"logits": logits.astype(np.float64), "ids": ids, "x": x.double().cpu().numpy(),
              "Wg": Wg.double().cpu().numpy(), "dw": dw.astype(np.float64), "dloss": float(np.float32(0.7))}
    if mask and poison:
        for k, v in (("logits", np.nan), ("x", np.inf), ("dw", np.nan)):
            c["t"][k][c["t"]["mask"].logical_not()] = v
        c["t"]["ids"][c["t"]["mask"].logical_not()] = 12345
    count = np.bincount(ids[m].ravel() + 1, minlength=E + 1)[1:]
    c["count"], c["tokens"] = count, int(m.sum())
    c["t"]["count"], c["t"]["tokens"] = dev(count, t.int32), dev([c["tokens"]], t.int32)
    c["desc"] = moe.make_desc(T, H, E, K, 8, dtype=moe.MOE_BF16 if dtype == "bf16" else moe.MOE_F32, temperature=tau)
    return c


def oracle(c, with_dw=True, with_loss=True):
    n, T, E, K, tau = c["n"], c["T"], c["E"], c["K"], c["tau"]
    z = n["logits"] / np.float64(tau)
    p = np.exp(z - z.max(1, keepdims=True)) if T else z
    p = p / p.sum(1, keepdims=True)
    m = c["mask"][:, None]
    tokens = c["tokens"]
    psum = np.where(m, p, 0).sum(0)
    loss = E * (c["count"] * psum).sum() / (tokens * K * tokens) if tokens else 0.0
    dl, size = np.zeros((T, E)), np.zeros((T, E))    # size: the magnitudes that the rounding errors go with
    if with_loss and tokens:
        cc = n["dloss"] * E * c["count"] / (float(tokens) ** 2 * K)
        dot = (p * cc).sum(1, keepdims=True)
        dl += p * (cc - dot)
        size += p * (cc + dot)
    if with_dw:
        for t in range(T):
            has = np.nonzero(n["ids"][t] >= 0)[0]
            e = n["ids"][t][has]
            w = p[t, e] / p[t, e].sum() if len(e) else p[t, e]
            g = n["dw"][t][has]
            np.add.at(dl[t], e, w * (g - (w * g).sum()))
            np.add.at(size[t], e, w * (abs(g) + (w * abs(g)).sum()))
    dl, size = np.where(m, dl, 0) / tau, np.where(m, size, 0) / tau
    x = np.where(m, n["x"], 0)
    return {"psum": psum, "loss": loss, "dlogits": dl, "size": size, "dWg": dl.T @ x, "dWg_size": size.T @ abs(x),
            "dbias": dl.sum(0), "dbias_size": size.sum(0), "dx": dl @ n["Wg"], "dx_size": size @ abs(n["Wg"])}


def run_backward(c, want=("dlogits", "dWg", "dbias", "dx"), flags=0, dw=True, dloss=True, ws=None):
    t, q = t_(), c["t"]
    T, H, E = c["T"], c["H"], c["E"]
    d = moe.make_desc(T, H, E, c["K"], 8, dtype=c["desc"].dtype, flags=flags, temperature=c["tau"])
    ws = moe.router_backward_workspace(d) if ws is None else ws
    out = {"dlogits": t.full((T, E), 7.0, device="cuda"), "dWg": t.full((E, H), 7.0, device="cuda"),
           "dbias": t.full((E,), 7.0, device="cuda"), "dx": t.full((T, H), 7.0, device="cuda").to(q["x"].dtype)}
    out = {k: out[k] if k in want else None for k in out}
    moe.moe_router_backward(d, q["x"] if "dWg" in want else None, q["Wg"] if "dx" in want else None, q["logits"],
                            q["ids"], q["dw"] if dw else None, q["dloss"] if dloss else None,
                            q["count"] if dloss else None, q["tokens"] if dloss else None, q["mask"], out["dlogits"],
                            out["dWg"], out["dbias"], out["dx"], ws)
    t.cuda.synchronize()
    assert moe.moe_get_device_error(ws) == 0
    return out


def check_backward(c, out, ref):
    """The scores over tau are off by half a step of their size twice (times tau^-1, less the largest), so
    p by 4 zmax half steps; the exponential, the sums over at most 256 experts (8 a lane, 5 shuffles) and the
    products add fewer than 64.  A sum over T tokens adds a half step of its terms' sum for each (tensor cores
    round towards zero: a whole one)."""
    f64 = {k: v.double().cpu().numpy() for k, v in out.items() if v is not None}
    zmax = abs(c["n"]["logits"]).max(initial=0) / c["tau"]
    u = (64 + 4 * zmax) * U32
    T, E = c["T"], c["E"]
    for k, v in f64.items():
        assert np.isfinite(v).all(), k
    if "dlogits" in f64:
        assert (abs(f64["dlogits"] - ref["dlogits"]) <= u * ref["size"] + 1e-37).all()
    if "dbias" in f64:
        assert (abs(f64["dbias"] - ref["dbias"]) <= (u + T * U32) * ref["dbias_size"] + 1e-37).all()
    if "dWg" in f64:
        assert (abs(f64["dWg"] - ref["dWg"]) <= (u + 2 * T * U32) * ref["dWg_size"] + 1e-37).all()
    if "dx" in f64:
        if c["dtype"] == "bf16":   # dlogits in two bf16 parts: 2^-16; the result rounded once
            tol = (u + 2 * E * U32 + 2.0 ** -16) * ref["dx_size"] * (1 + U16) + U16 * abs(ref["dx"])
        else:
            tol = (u + E * U32) * ref["dx_size"]
        assert (abs(f64["dx"] - ref["dx"]) <= tol + 1e-37).all()


SHAPES = [(1, 64, 8, 2), (3, 8, 2, 1), (64, 256, 8, 2), (130, 136, 5, 3), (257, 1000, 12, 3), (300, 264, 33, 4),
          (129, 520, 64, 8), (200, 128, 100, 2), (131, 72, 130, 8), (77, 3584, 256, 8), (1025, 320, 32, 2)]


@pytest.mark.parametrize("mask", [False, True])
@pytest.mark.parametrize("tau", [1.0, 0.5])
@pytest.mark.parametrize("T,H,E,K", SHAPES + [(70000, 8, 32, 2)])
def test_balance_loss(T, H, E, K, tau, mask):
    c = case(T, H, E, K, mask=mask, tau=tau, missing=T % 2 == 0, seed=1)
    t, q, ref = t_(), c["t"], oracle(c, False, False)
    ws = moe.router_backward_workspace(c["desc"])
    psum, loss = t.full((E,), 7.0, device="cuda"), t.full((1,), 7.0, device="cuda")
    count, tokens = t.full((E,), 7, dtype=t.int32, device="cuda"), t.full((1,), 7, dtype=t.int32, device="cuda")
    for _ in range(2):    # the workspace is left as it has to be found
        moe.moe_balance_loss(c["desc"], q["logits"], q["ids"], q["mask"], psum, count, tokens, loss, ws)
    t.cuda.synchronize()
    assert moe.moe_get_device_error(ws) == 0
    assert (count.cpu().numpy() == c["count"]).all() and tokens.item() == c["tokens"]
    # probabilities as in check_backward; fp32 sums of at most 2^13 tokens, each at most a half step of the sum
    zmax = abs(c["n"]["logits"]).max() / tau
    u = (64 + 4 * zmax + min(T, 8192)) * U32
    assert (abs(psum.double().cpu().numpy() - ref["psum"]) <= u * ref["psum"] + 1e-37).all()
    assert abs(loss.item() - ref["loss"]) <= (u + 4 * U32) * ref["loss"]


def test_balance_loss_is_the_aux_loss_and_results_may_be_left_out():
    c = case(500, 64, 16, 2, seed=2)
    t, q = t_(), c["t"]
    ws = moe.router_backward_workspace(c["desc"])
    psum, loss, aux = (t.empty(n, device="cuda") for n in (16, 1, 1))
    count, tokens = t.empty(16, dtype=t.int32, device="cuda"), t.empty(1, dtype=t.int32, device="cuda")
    moe.moe_balance_loss(c["desc"], q["logits"], q["ids"], None, psum, count, tokens, loss, ws)
    moe.moe_aux_loss(c["desc"], psum, count, aux)
    assert abs(loss.item() - aux.item()) <= 32 * U32 * loss.item()
    for k in ("psum", "count", "tokens", "loss"):
        full = {"psum": psum, "count": count, "tokens": tokens, "loss": loss}
        alone = {n: t.zeros_like(v) if n == k else None for n, v in full.items()}
        moe.moe_balance_loss(c["desc"], q["logits"], q["ids"], None, alone["psum"], alone["count"], alone["tokens"],
                             alone["loss"], ws)
        assert (alone[k] == full[k]).all(), k


@pytest.mark.parametrize("T", [0, 40])
def test_no_token_counts(T):
    """No token at all, or a mask that leaves none: zeros, no NaN."""
    c = case(T, 64, 8, 2, seed=3)
    t, q = t_(), c["t"]
    ws = moe.router_backward_workspace(c["desc"])
    mask = t.zeros(T, dtype=t.uint8, device="cuda")
    q["logits"].fill_(float("nan"))
    q["x"].fill_(float("nan"))
    psum, loss = t.full((8,), 7.0, device="cuda"), t.full((1,), 7.0, device="cuda")
    count, tokens = t.full((8,), 7, dtype=t.int32, device="cuda"), t.full((1,), 7, dtype=t.int32, device="cuda")
    moe.moe_balance_loss(c["desc"], q["logits"], q["ids"], mask, psum, count, tokens, loss, ws)
    for v in (psum, loss, count, tokens):
        assert (v == 0).all()
    for flags in (0, moe.MOE_FLAG_SIMT_ROUTER):
        q.update(mask=mask, count=count, tokens=tokens)
        out = run_backward(c, flags=flags)
        for k, v in out.items():
            assert (v == 0).all(), k


@pytest.mark.parametrize("mask", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "bf16_simt", "f32"])
@pytest.mark.parametrize("T,H,E,K", SHAPES)
def test_router_gradient(T, H, E, K, kind, mask):
    c = case(T, H, E, K, kind[:4].rstrip("_"), mask=mask, tau=0.5 if T % 2 else 1.0, seed=4)
    out = run_backward(c, flags=moe.MOE_FLAG_SIMT_ROUTER if kind == "bf16_simt" else 0)
    check_backward(c, out, oracle(c))


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_router_gradient_without_the_loss_or_the_weights_and_with_missing_experts(kind):
    c = case(333, 264, 24, 4, kind, mask=True, missing=True, tau=2.0, seed=5)
    for dw, dloss in ((True, False), (False, True), (True, True), (False, False)):
        check_backward(c, run_backward(c, dw=dw, dloss=dloss), oracle(c, dw, dloss))


@pytest.mark.parametrize("kind", ["bf16", "bf16_simt", "f32"])
def test_router_gradient_is_deterministic_and_each_result_alone_is_the_same(kind):
    c = case(700, 392, 40, 3, kind[:4].rstrip("_"), mask=True, seed=6)
    flags = moe.MOE_FLAG_SIMT_ROUTER if kind == "bf16_simt" else 0
    first = run_backward(c, flags=flags)
    ws = moe.router_backward_workspace(moe.make_desc(700, 392, 40, 3, 8, dtype=c["desc"].dtype, flags=flags))
    for _ in range(2):
        again = run_backward(c, flags=flags, ws=ws)
        for k in first:
            assert (first[k] == again[k]).all(), k
    for k in first:
        assert (run_backward(c, want=(k,), flags=flags)[k] == first[k]).all(), k


def test_an_id_outside_the_experts_is_recorded_and_counts_for_none():
    c = case(50, 64, 8, 2, "f32", seed=7)
    t, q = t_(), c["t"]
    q["ids"][3, 1] = 8
    q["ids"][4, 0] = -2
    c["n"]["ids"][3, 1] = c["n"]["ids"][4, 0] = -1
    c["count"] = np.bincount(c["n"]["ids"].ravel() + 1, minlength=9)[1:]
    q["count"] = t.from_numpy(c["count"]).to(t.int32).cuda()
    ws = moe.router_backward_workspace(c["desc"])
    count = t.empty(8, dtype=t.int32, device="cuda")
    moe.moe_balance_loss(c["desc"], q["logits"], q["ids"], None, None, count, None, None, ws)
    assert moe.moe_get_device_error(ws) == moe.MOE_ERR_DEVICE
    assert (count.cpu().numpy() == c["count"]).all()
    dl = t.empty((50, 8), device="cuda")
    moe.moe_router_backward(c["desc"], None, None, q["logits"], q["ids"], q["dw"], q["dloss"], q["count"], q["tokens"],
                            None, dl, None, None, None, ws)
    assert moe.moe_get_device_error(ws) == moe.MOE_ERR_DEVICE
    check_backward(c, {"dlogits": dl}, oracle(c))


def test_router_gradient_against_differences():
    """The loss <dw, w(l)> + dloss * balance(l) (counts held) along random directions of the scores: central
    differences of the 64-bit forward formulas with a step of 1e-4 are within 1e-7 of its derivative."""
    c = case(40, 16, 12, 3, "f32", tau=0.7, seed=8)
    n, r = c["n"], np.random.default_rng(9)

    def value(l):
        z = l / np.float64(np.float32(0.7))
        p = np.exp(z - z.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
        pk = np.take_along_axis(p, n["ids"].astype(np.int64), 1)
        w = pk / pk.sum(1, keepdims=True)
        return (n["dw"] * w).sum() + n["dloss"] * 12 * (c["count"] * p.sum(0)).sum() / (40 * 3 * 40)

    got = run_backward(c, want=("dlogits",))["dlogits"].double().cpu().numpy()
    for _ in range(4):
        d = r.standard_normal((40, 12))
        quotient = (value(n["logits"] + 1e-4 * d) - value(n["logits"] - 1e-4 * d)) / 2e-4
        assert abs(quotient - (got * d).sum()) <= 1e-5 * np.abs(got * d).sum()


@pytest.mark.parametrize("off", [0, 1, 3])
@pytest.mark.parametrize("T,E,K", [(2, 2, 1), (96, 12, 3), (4096, 16, 2), (65536, 128, 4)])
def test_balance_gradient_of_nearly_equal_counts(T, E, K, off):
    """As small as the counts' differences, and as exact: with p off by u as in check_backward, c - <p, c> (2 max|c - mean|
    at most) brings 2 u p max|c - mean|, and the error of <p, c> and the roundings of c and the product under 2 u more;
    nothing where all counts are equal."""
    r = np.random.default_rng([T, E, off])
    t = t_()
    z = r.standard_normal((T, E)).astype(np.float32)
    count = np.full(E, T * K // E)
    count[0] += off
    count[-1] -= off
    if count.min() < 0:
        pytest.skip("fewer choices than that")
    f32, i32 = dict(device="cuda", dtype=t.float32), dict(device="cuda", dtype=t.int32)
    d = moe.make_desc(T, 64, E, K, 8)
    out = t.full((T, E), 7.0, **f32)
    ws = moe.router_backward_workspace(d)
    moe.moe_router_backward(d, None, None, t.tensor(z, **f32), t.zeros(T, K, **i32), None, t.full((1,), 0.7, **f32),
                            t.tensor(count, **i32), t.tensor([T], **i32), None, out, None, None, None, ws)
    p = np.exp(z.astype(np.float64) - z.max(axis=1, keepdims=True))
    p /= p.sum(axis=1, keepdims=True)
    c = float(np.float32(0.7)) / T * E * (count - count.mean()) / (T * K)
    want = p * (c - p @ c[:, None])
    assert (abs(out.double().cpu().numpy() - want) <= 4 * (64 + 4 * abs(z).max()) * U32 * p * abs(c).max()).all()


def test_scores_of_minus_infinity():
    """Experts switched off by a score of -infinity have no probability and no gradient."""
    c = case(60, 64, 16, 2, "bf16", seed=10)
    off = np.zeros((60, 16), bool)
    off[:, 5] = True
    off[7, :14] = True
    c["n"]["logits"][off] = -1e300
    c["t"]["logits"][t_().from_numpy(off).cuda()] = -float("inf")
    ids = np.argsort(-c["n"]["logits"], axis=1, kind="stable")[:, :2].astype(np.int32)
    c["n"]["ids"], c["t"]["ids"] = ids, t_().from_numpy(ids).cuda()
    c["count"] = np.bincount(ids.ravel(), minlength=16)
    c["t"]["count"] = t_().from_numpy(c["count"]).to(t_().int32).cuda()
    out, ref = run_backward(c), oracle(c)
    assert (out["dlogits"].cpu().numpy()[off] == 0).all()
    c["n"]["logits"] = np.where(off, 0, c["n"]["logits"])      # for the bound alone
    check_backward(c, out, ref)


@pytest.mark.parametrize("E,want", [(12, ("dWg", "dx", "dbias")), (100, ("dx",)), (200, ("dWg",))])
def test_expired_wait_reports_timeout_and_context_survives(E, want):
    """The first panels' barrier waits for an arrival that nobody makes: every role gives up, what is in flight
    lands, tensor memory is freed and the error word says so.  The next call, in the same workspace, is right."""
    t = t_()
    c = case(1500, 520, E, 2, mask=True, seed=11)
    ws = moe.router_backward_workspace(c["desc"])
    start, end = (t.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    d = moe.make_desc(1500, 520, E, 2, 8, flags=moe.MOE_FLAG_TEST_WAIT_TIMEOUT)
    q = c["t"]
    out = dict(dWg=t.empty(E, 520, device="cuda"), dx=t.empty_like(q["x"]), dbias=t.empty(E, device="cuda"))
    out = {k: v if k in want else None for k, v in out.items()}
    moe.moe_router_backward(d, q["x"], q["Wg"], q["logits"], q["ids"], q["dw"], q["dloss"], q["count"], q["tokens"],
                            q["mask"], None, out["dWg"], out["dbias"], out["dx"], ws)
    end.record()
    t.cuda.synchronize()
    assert moe.moe_get_device_error(ws) == moe.MOE_ERR_TIMEOUT
    assert start.elapsed_time(end) < 30e3
    check_backward(c, run_backward(c, ws=ws), oracle(c))      # the read cleared the error word
