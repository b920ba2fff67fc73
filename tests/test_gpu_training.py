"""The training calls on the GPU against the float64 oracle.

Tolerances, element by element.  u = 2^-24 and b = 2^-8 are the largest
relative errors of one rounding to fp32 and to bf16.  An fp32 sum of n products
a_i b_i makes n roundings, each at most u times a partial sum, and a partial
sum is at most |a| |b| (Cauchy-Schwarz); roundings to nearest are taken as
independent and centred, so by Hoeffding's inequality their total is beyond
7 sqrt(n) u |a| |b| with a chance below 1e-10.  Errors carried on from an
earlier step add to that with the slope of what follows."""
import numpy as np
import pytest

import sparse_mixture_experts_topk_gb300 as moe
from sparse_mixture_experts_topk_gb300 import workloads as W
from oracle import moe_oracle as O
from oracle import train_oracle as G

from harness import to_dev, to_np, as_f64

pytestmark = pytest.mark.gpu

U, B = 2.0 ** -24, 2.0 ** -8
NAN_BF16, INF_BF16 = 0x7FC0, 0x7F80


@pytest.fixture(scope="module", autouse=True)
def _built():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_mixture_experts_topk_gb300 import build
    build.build()
    moe.lib()


def t_():
    import torch
    return torch


def pack(a, dtype):
    return W.f32_to_bf16_bits(a.astype(np.float32)) if dtype == "bf16" else a.astype(np.float32)


def wide(a, dtype):
    return O.widen(a, "bf16") if dtype == "bf16" else a.astype(np.float64)


def round_tol(ref, dtype):
    """The final rounding, and fp32's smallest numbers."""
    return np.abs(ref) * (B if dtype == "bf16" else U) * 1.01 + 1e-38


def within(got, ref, tol, what):
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.nanmax(np.abs(got - ref)):.3g}"


def tensor(shape, dtype, fill=None):
    t = t_()
    dt = t.bfloat16 if dtype == "bf16" else t.float32
    return t.full(shape, float("nan") if fill is None else fill, dtype=dt, device="cuda")


def route(T, E, K, cap, seed):
    rng = np.random.default_rng(seed)
    ids = np.stack([rng.permutation(E)[:K] for _ in range(T)]).reshape(T, K)
    return O.dispatch(ids, E, cap), rng


# ---------------------------------------------------------------- token exchange

# one token; rows of one vector, of just over the one-warp rows, odd numbers of vectors; every slot
# array size (K = 1, 2, 3, 4, 5, 8); capacities that drop slots and leave tokens without any
EXCHANGE = [(1, 8, 4, 2, 0), (1, 3584, 32, 2, 0), (5, 8, 2, 1, 1), (37, 520, 5, 3, 0), (64, 256, 8, 2, 0),
            (130, 528, 12, 4, 20), (77, 1000, 9, 5, 13), (33, 136, 16, 8, 4), (300, 512, 3, 2, 10),
            (1000, 64, 64, 1, 3), (3, 4104, 8, 8, 1)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,E,K,cap", EXCHANGE)
def test_exchange_gradients(T, H, E, K, cap, dtype):
    t = t_()
    d, rng = route(T, E, K, cap, T * 1000 + H)
    desc = moe.make_desc(T, H, E, K, 8, cap, moe.MOE_BF16 if dtype == "bf16" else moe.MOE_F32)
    R, kept = moe.moe_max_rows(desc), int(d["offs"][E])
    dout, add = (pack(rng.standard_normal((T, H)), dtype) for _ in range(2))
    rows = np.full((R, H), np.nan)
    rows[:kept] = rng.standard_normal((kept, H))
    rows = pack(rows, dtype) if dtype == "f32" else np.where(np.isnan(rows), np.uint16(NAN_BF16),
                                                             pack(np.nan_to_num(rows), dtype))
    w = rng.uniform(0.05, 1, (T, K)).astype(np.float32)
    pos = to_dev(d["pos"].astype(np.int32), "i32")
    D = [to_dev(v, dtype) for v in (dout, rows, add)]
    wd = to_dev(w, "f32")

    # combine: dy is one product, rounded; dw a sum of H products
    y64, dout64 = wide(rows, dtype)[:kept], wide(dout, dtype)
    dy, dw = G.combine_backward(dout64, y64, d["pos"], w.astype(np.float64))
    dyg, dwg = tensor((R, H), dtype), tensor((T, K), "f32")
    moe.moe_combine_backward(desc, D[0], D[1], pos, wd, dyg, dwg)
    got = as_f64(dyg)
    within(got[:kept], dy, round_tol(dy, dtype) + np.abs(dy) * U, "dy")
    assert np.isnan(got[kept:]).all()                                # rows without a slot are left alone
    norm = np.zeros((T, K))
    for s in np.nonzero(d["pos"] >= 0)[0]:
        norm.flat[s] = np.linalg.norm(dout64[s // K]) * np.linalg.norm(y64[d["pos"][s]])
    within(as_f64(dwg), dw, 7 * np.sqrt(H) * U * norm + 1e-38, "dw")
    assert (as_f64(dwg).reshape(-1)[d["pos"] < 0] == 0).all()
    # each result alone gives the same bits
    one, two = tensor((R, H), dtype), tensor((T, K), "f32")
    moe.moe_combine_backward(desc, D[0], None, pos, wd, one, None)
    moe.moe_combine_backward(desc, D[0], D[1], pos, wd, None, two)
    assert (to_np(one)[:kept] == to_np(dyg)[:kept]).all() and (to_np(two) == to_np(dwg)).all()

    # dispatch, with and without an addend, and onto the addend itself
    for use in (False, True):
        dx = G.dispatch_backward(y64, d["pos"], T, K, wide(add, dtype) if use else None)
        size = G.dispatch_backward(np.abs(y64), d["pos"], T, K, np.abs(wide(add, dtype)) if use else None)
        out = tensor((T, H), dtype)
        moe.moe_dispatch_backward(desc, D[1], pos, D[2] if use else None, out)
        within(as_f64(out), dx, round_tol(dx, dtype) + (K + 1) * U * size, "dx")
    same = D[2].clone()
    moe.moe_dispatch_backward(desc, D[1], pos, same, same)
    assert (to_np(same) == to_np(out)).all()


def test_exchange_follows_its_stream_and_captures():
    """On another stream than the current one, and replayed from a CUDA graph
    with new contents in the same buffers."""
    t = t_()
    d, rng = route(50, 6, 2, 0, 4)
    desc = moe.make_desc(50, 256, 6, 2, 8)
    y, dout = (to_dev(pack(rng.standard_normal((n, 256)), "bf16"), "bf16") for n in (100, 50))
    pos, w = to_dev(d["pos"].astype(np.int32), "i32"), to_dev(rng.uniform(size=(50, 2)).astype(np.float32), "f32")
    want, want_dw, want_dx = tensor((100, 256), "bf16"), tensor((50, 2), "f32"), tensor((50, 256), "bf16")
    moe.moe_combine_backward(desc, dout, y, pos, w, want, want_dw)
    moe.moe_dispatch_backward(desc, want, pos, None, want_dx)
    t.cuda.synchronize()
    dy, dw, dx = tensor((100, 256), "bf16"), tensor((50, 2), "f32"), tensor((50, 256), "bf16")
    t.cuda.synchronize()
    s = t.cuda.Stream()
    moe.moe_combine_backward(desc, dout, y, pos, w, dy, dw, stream=s)
    moe.moe_dispatch_backward(desc, dy, pos, None, dx, stream=s)
    s.synchronize()
    assert t.equal(dy, want) and t.equal(dw, want_dw) and t.equal(dx, want_dx)
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g):
        moe.moe_combine_backward(desc, dout, y, pos, w, dy, dw)
        moe.moe_dispatch_backward(desc, dy, pos, None, dx)
    dout.mul_(2)
    g.replay()
    t.cuda.synchronize()
    assert t.equal(dy, want * 2) and t.equal(dw, want_dw * 2) and t.equal(dx, want_dx * 2)


# ---------------------------------------------------------------- expert FFN

def ffn_case(counts, H, F, act, bias, dtype, seed, extra=3):
    """Rows for experts of the given counts, `extra` meaningless ones behind."""
    rng = np.random.default_rng(seed)
    E, g, n = len(counts), 2 if act == "swiglu" else 1, sum(counts)
    bound = np.sqrt(6.0 / (H + F))
    c = dict(counts=counts, E=E, H=H, F=F, g=g, act=act, dtype=dtype, n=n, R=n + extra)
    c["offs"] = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    c["W1"] = pack(rng.uniform(-bound, bound, (E, g * F, H)), dtype)
    c["W2"] = pack(rng.uniform(-bound, bound, (E, H, F)), dtype)
    c["b1"] = rng.uniform(-0.3, 0.3, (E, g * F)).astype(np.float32) if bias else None
    c["x"], c["dy"] = pack(rng.standard_normal((n, H)), dtype), pack(rng.standard_normal((n, H)), dtype)
    h = np.zeros((n, F))
    for e in range(E):
        r = slice(c["offs"][e], c["offs"][e + 1])
        a = wide(c["x"][r], dtype) @ wide(c["W1"][e], dtype).T + (c["b1"][e] if bias else 0)
        h[r] = O.silu(a[:, :F]) * a[:, F:] if g == 2 else O.gelu(a)
    c["h"] = pack(h, dtype)
    return c


def with_tail(a, R, dtype):
    """The permuted buffer of R rows: NaN behind the last kept one."""
    full = np.full((R, a.shape[1]), NAN_BF16 if dtype == "bf16" else np.nan, dtype=a.dtype)
    full[:len(a)] = a
    return to_dev(full, dtype)


def run_ffn(c, flags=0, want=("dx", "dW1", "db1", "dW2", "db2"), ws=None):
    E, H, F, R, dtype = c["E"], c["H"], c["F"], c["R"], c["dtype"]
    if c["act"] == "swiglu":
        flags |= moe.MOE_FLAG_SWIGLU
    desc = moe.make_desc(R, H, E, 1, F, 0, moe.MOE_BF16 if dtype == "bf16" else moe.MOE_F32, flags)
    ws = moe.backward_workspace(desc) if ws is None else ws
    ws[256:].view(t_().uint8).fill_(0xFF)      # NaN in every format: nothing is read before it is written
    o = dict(dx=tensor((R, H), dtype, -7.0), dW1=tensor((E, c["g"] * F, H), dtype), dW2=tensor((E, H, F), dtype),
             db1=tensor((E, c["g"] * F), "f32"), db2=tensor((E, H), "f32"))
    q = {k: o[k] if k in want else None for k in o}
    moe.moe_expert_ffn_backward(desc, with_tail(c["x"], R, dtype), with_tail(c["h"], R, dtype),
                                with_tail(c["dy"], R, dtype), to_dev(c["offs"], "i32"), to_dev(c["W1"], dtype),
                                to_dev(c["b1"], "f32"), to_dev(c["W2"], dtype), q["dx"], q["dW1"], q["db1"], q["dW2"],
                                q["db2"], ws)
    t_().cuda.synchronize()
    assert moe.moe_get_device_error(ws) == 0
    return o


def dot_tol(A, Bm):
    """Bound of the fp32 roundings of A @ Bm."""
    return 7 * np.sqrt(max(1, A.shape[1])) * U * np.outer(np.linalg.norm(A, axis=1), np.linalg.norm(Bm, axis=0))


def sum_tol(A, b2):
    """7 sqrt(sum of squares) of independent errors at most b2[i] times |A|'s entries."""
    return 7 * np.sqrt(np.square(A) @ np.square(b2))


def check_ffn(c, o, which=("dx", "dW1", "db1", "dW2", "db2")):
    dtype, F = c["dtype"], c["F"]
    fin = B if dtype == "bf16" else U       # da as an operand
    for e in range(c["E"]):
        r = slice(c["offs"][e], c["offs"][e + 1])
        x, h, dy = (wide(c[k][r], dtype) for k in ("x", "h", "dy"))
        W1, W2 = wide(c["W1"][e], dtype), wide(c["W2"][e], dtype)
        b1 = None if c["b1"] is None else c["b1"][e].astype(np.float64)
        ref = G.expert_ffn_backward(x, h, dy, W1, W2, b1, c["act"])
        ta, th = dot_tol(x, W1.T) + np.abs(ref["a"]) * U, dot_tol(dy, W2)
        # the slopes' own evaluation: a few fp32 roundings of terms of order 1 + |a|
        few = 16 * U
        if c["act"] == "swiglu":
            z, u, dh = ref["a"][:, :F], ref["a"][:, F:], ref["dh"]
            s1, s0 = np.abs(G.silu_slope(z)), np.abs(z * G.sigmoid(z))
            # |SiLU'| <= 1.1, |SiLU''| <= 1/2
            tda = np.concatenate([np.abs(u) * s1 * th + np.abs(dh) * (1.1 * ta[:, F:] + 0.5 * np.abs(u) * ta[:, :F]
                                                                      + few * (1 + np.abs(z)) * np.abs(u)),
                                  s0 * th + np.abs(dh) * (1.1 * ta[:, :F] + few * (1 + np.abs(z)))], axis=1)
        else:
            # |GELU''| <= 2 phi(0) < 0.8
            tda = np.abs(G.gelu_slope(ref["a"])) * th + np.abs(ref["dh"]) * (0.8 * ta + few * (1 + np.abs(ref["a"])))
        da, near = ref["da"], fin * np.abs(ref["da"])
        tol = dict(dx=dot_tol(da, W1) + tda @ np.abs(W1) + sum_tol(near, W1),
                   dW1=dot_tol(da.T, x) + tda.T @ np.abs(x) + sum_tol(near.T, x),
                   db1=tda.sum(0) + 7 * np.sqrt(len(x)) * U * np.abs(da).sum(0),
                   dW2=dot_tol(dy.T, h), db2=7 * np.sqrt(len(x)) * U * np.abs(dy).sum(0))
        got = dict(dx=as_f64(o["dx"])[r], **{k: as_f64(o[k])[e] for k in ("dW1", "db1", "dW2", "db2")})
        for k in which:
            within(got[k], ref[k], tol[k] + round_tol(ref[k], "f32" if k[:2] == "db" else dtype), f"expert {e} {k}")
    if "dx" in which:
        assert (as_f64(o["dx"])[c["n"]:] == -7.0).all()     # rows from offs[E] on are left alone


FFN = [
    # one row; experts without rows at both ends and in the middle
    ([1], 8, 8), ([0, 1, 0], 64, 32), ([0, 0, 5, 0, 2], 40, 24),
    # every side of a 16-row step, a 64-row block and a 128- and 256-row tile
    ([15, 16, 17, 63, 64, 65], 128, 192), ([127, 128, 129, 0, 255, 256, 257], 256, 136),
    # sizes that are no multiple of a tile, rows of several tiles
    ([300, 7, 513], 520, 264), ([33, 48, 49], 1000, 328), ([31, 96, 160], 72, 648),
    # more tiles than SM pairs: every pair works through several, of experts of all lengths
    ([20, 300, 0, 64, 5, 257] * 7, 520, 528),
]


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("act", ["gelu", "swiglu"])
@pytest.mark.parametrize("kind", ["bf16", "bf16_simt", "f32"])
@pytest.mark.parametrize("counts,H,F", FFN)
def test_ffn_gradient(counts, H, F, kind, act, bias):
    c = ffn_case(counts, H, F, act, bias, kind[:4].rstrip("_"), 11 + H)
    check_ffn(c, run_ffn(c, moe.MOE_FLAG_SIMT_FFN if kind == "bf16_simt" else 0))


@pytest.mark.parametrize("act", ["gelu", "swiglu"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_ffn_gradient_is_deterministic_and_each_result_alone_is_the_same(act, dtype):
    c = ffn_case([70, 0, 260, 129], 264, 328, act, True, dtype, 5)
    first = run_ffn(c)
    again = run_ffn(c)
    for k in first:
        assert (to_np(first[k])[:c["n"]] == to_np(again[k])[:c["n"]]).all(), k
        alone = run_ffn(c, want=(k,))
        assert (to_np(first[k])[:c["n"]] == to_np(alone[k])[:c["n"]]).all(), k


@pytest.mark.parametrize("poison", [NAN_BF16, INF_BF16])
def test_ffn_gradient_keeps_an_experts_nan_to_itself(poison):
    """NaN or infinity in one expert's rows: the other experts' results are
    the bits they were, whatever shares a tile or a block of rows with them."""
    c = ffn_case([20, 33, 70, 5], 136, 200, "gelu", True, "bf16", 6)
    clean = run_ffn(c)
    r = slice(c["offs"][1], c["offs"][2])
    for k in ("x", "h", "dy"):
        c[k][r] = poison
    dirty = run_ffn(c)
    for e in (0, 2, 3):
        rows = slice(c["offs"][e], c["offs"][e + 1])
        assert (to_np(clean["dx"])[rows] == to_np(dirty["dx"])[rows]).all()
        for k in ("dW1", "db1", "dW2", "db2"):
            assert (to_np(clean[k])[e] == to_np(dirty[k])[e]).all(), (e, k)
    assert not np.isfinite(as_f64(dirty["dW2"])[1]).any()


@pytest.mark.parametrize("flags", [0, moe.MOE_FLAG_SIMT_FFN])
def test_ffn_gradient_without_rows(flags):
    """No token at all, and tokens whose slots were all dropped: weight
    gradients are zeros, nothing else is touched."""
    t = t_()
    for T in (0, 6):
        desc = moe.make_desc(T, 64, 4, 2, 32, flags=flags)
        ws = moe.backward_workspace(desc)
        offs = t.zeros(5, dtype=t.int32, device="cuda")
        W1, W2 = tensor((4, 32, 64), "bf16", 1.0), tensor((4, 64, 32), "bf16", 1.0)
        rows = tensor((max(1, moe.moe_max_rows(desc)), 64), "bf16")
        h = tensor((rows.shape[0], 32), "bf16")
        dx, dW1, dW2 = tensor(rows.shape, "bf16", 3.0), tensor(W1.shape, "bf16"), tensor(W2.shape, "bf16")
        db1, db2 = tensor((4, 32), "f32"), tensor((4, 64), "f32")
        moe.moe_expert_ffn_backward(desc, rows, h, rows, offs, W1, None, W2, dx, dW1, db1, dW2, db2, ws)
        t.cuda.synchronize()
        assert moe.moe_get_device_error(ws) == 0
        for g in (dW1, dW2, db1, db2):
            assert (g == 0).all()
        assert (dx == 3.0).all()


def test_ffn_gradient_against_differences_of_the_forward_call():
    """fp32: the loss <dy, moe_expert_ffn(x)> along a random direction of each
    input.  The forward call's fp32 rounding is about 1e-6 of the loss's terms
    (norm |dy| |y|); with a step of 2^-6 along a unit direction the quotient's
    rounding is below 2e-4 |dy| |y| and its curvature term below 2^-12 times
    the third derivative, which for these O(1) activations is below 1e-2 of
    the same product."""
    t = t_()
    c = ffn_case([9, 0, 20], 64, 96, "gelu", True, "f32", 21, extra=0)
    desc = moe.make_desc(c["R"], c["H"], 3, 1, c["F"], 0, moe.MOE_F32)
    fws = moe.workspace(desc)
    v = {k: to_dev(c[k], "f32") for k in ("x", "W1", "b1", "W2", "dy")}
    offs = to_dev(c["offs"], "i32")
    h, y = tensor((c["R"], c["F"]), "f32"), tensor((c["R"], c["H"]), "f32")

    def loss(**over):
        q = {**v, **over}
        moe.moe_expert_ffn(desc, q["x"], offs, q["W1"], q["b1"], q["W2"], None, h, y, fws)
        return float((q["dy"].double() * y.double()).sum())

    loss()
    c["h"] = to_np(h).copy()
    o = run_ffn(c)
    scale = float(v["dy"].double().norm() * y.double().norm())
    rng = np.random.default_rng(2)
    for name, grad in (("x", "dx"), ("W1", "dW1"), ("b1", "db1"), ("W2", "dW2")):
        way = rng.standard_normal(c[name].shape)
        way = to_dev((way / np.linalg.norm(way)).astype(np.float32), "f32")
        step = 2.0 ** -6
        got = (loss(**{name: v[name] + step * way}) - loss(**{name: v[name] - step * way})) / (2 * step)
        want = float((o[grad].double() * way.double()).sum())
        assert abs(got - want) <= 5e-4 * scale, (name, got, want)


# ---------------------------------------------------------------- AdamW

f32 = np.float32


def state(n, bits, rng):
    m = (rng.standard_normal(n) * 3e-4).astype(f32)
    v = np.square(rng.standard_normal(n) * 1e-3).astype(f32)
    if bits == 32:
        return m, v, None, None
    (m, ms), (v, vs) = encode(m, False), encode(np.sqrt(v), True)
    return m, v, ms, vs


def blocks_of(x):
    pad = np.zeros(-(-len(x) // 256) * 256, dtype=x.dtype)
    pad[:len(x)] = x
    return pad.reshape(-1, 256)


def encode(x, keep_non_zero):
    """The 8-bit moments as the header describes them, every fp32 operation rounded by itself."""
    b = blocks_of(x)
    top = np.abs(b).max(1)
    big = top >= f32(2.0 ** -100)
    with np.errstate(divide="ignore", over="ignore", invalid="ignore"):
        inv = np.where(big, (f32(1) / top) * f32(448), f32(0)).astype(f32)
        y = (b * inv[:, None]).astype(f32)
    y = np.where(big[:, None], y, f32(0))
    if keep_non_zero:
        y = np.where((b > 0) & big[:, None], np.maximum(y, f32(2.0 ** -9)), y)
    scale = np.where(big, top * f32(1.0 / 448.0), f32(0)).astype(f32)
    return G.encode_e4m3(y).reshape(-1)[:len(x)], scale


def decode(code, scale):
    return (blocks_of(G.decode_e4m3(code).astype(f32)) * scale[:, None]).reshape(-1)[:len(code)]


def step32(p, g, m, v, gs, hp, wd):
    """The step in fp32, operation by operation."""
    b1, b2 = f32(hp["beta1"]), f32(hp["beta2"])
    g = (g * f32(gs)).astype(f32)
    m = m * b1 + g * f32(1 - hp["beta1"])
    v = v * b2 + (g * g) * f32(1 - hp["beta2"])
    return m.astype(f32), v.astype(f32), np.sqrt(v.astype(f32))


ADAMW = [[1], [255], [256], [257], [3, 1, 4096, 255, 513, 0, 70000], [5] * 41, [17] * 399 + [1000] * 5]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("grad", ["bf16", "f32"])
@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("sizes", ADAMW, ids=lambda s: f"{len(s)}x{max(s)}")
def test_adamw(sizes, shift, grad, bits):
    """shift = 1: every tensor starts one element past an aligned address."""
    t = t_()
    rng = np.random.default_rng(sum(sizes) + shift)
    hp = dict(lr=2e-3, beta1=0.9, beta2=0.95, eps=1e-8, step=7)
    gs, want, tensors, dev = 0.375, [], [], []

    def place(a, dt):
        buf = t.zeros(len(a) + 8 + shift, dtype=dt, device="cuda")
        s = buf[shift:shift + len(a)]
        if dt == t.float8_e4m3fn:
            s.view(t.uint8).copy_(t.from_numpy(a))
        elif dt == t.bfloat16:
            s.copy_(t.from_numpy(a.view(np.int16)).view(t.bfloat16))
        else:
            s.copy_(t.from_numpy(a))
        return s, buf

    for i, n in enumerate(sizes):
        p = rng.standard_normal(n).astype(f32)
        g = (rng.standard_normal(n) * 1e-2).astype(f32)
        g[: n // 3] = 0
        gp = pack(g, grad)
        g = wide(gp, grad).astype(f32)
        m, v, ms, vs = state(n, bits, rng)
        wd = 0.1 * (i % 3)
        m0, v0 = (m, v) if bits == 32 else (decode(m, ms), np.square(decode(v, vs)))
        m1, v1, r1 = step32(p, g, m0, v0, gs, hp, wd)
        p64, m64, v64 = G.adamw(*(a.astype(np.float64) for a in (p, g * f32(gs), m0, v0)), weight_decay=wd, **hp)
        want.append(dict(p=p64, upd=np.abs(p64 - p.astype(np.float64)), m=m1, v=v1, r=r1, m64=m64, v64=v64, m0=m0, g=g * f32(gs), p0=p))
        st = t.float32 if bits == 32 else t.float8_e4m3fn
        f = dict(p=place(p, t.float32), g=place(gp, t.float32 if grad == "f32" else t.bfloat16), m=place(m, st),
                 v=place(v, st), p16=place(np.zeros(n, np.uint16), t.bfloat16))
        if bits == 8:
            f["m_scale"], f["v_scale"] = place(ms, t.float32), place(vs, t.float32)
        dev.append(f)
        tensors.append({**{k: a[0] for k, a in f.items()}, "weight_decay": wd})
    plan = moe.adamw_tensors(tensors)
    scale = t.tensor([gs], device="cuda")
    skip = t.ones(1, dtype=t.int32, device="cuda")
    before = [{k: to_np(a[1].view(t.uint8)).copy() for k, a in f.items()} for f in dev]
    moe.moe_adamw_step(plan, moe.make_adamw(**hp), scale, skip)
    for f, b in zip(dev, before):     # a skipped step changes nothing
        for k, a in f.items():
            assert (to_np(a[1].view(t.uint8)) == b[k]).all(), k
    skip.zero_()
    moe.moe_adamw_step(plan, moe.make_adamw(**hp), scale, skip)
    t.cuda.synchronize()
    for f, b, q, n in zip(dev, before, want, sizes):
        got = {k: a[0] for k, a in f.items()}
        p = to_np(got["p"]).astype(np.float64)
        # m: two products and a sum; the quotient carries m's error and a few roundings more
        c1 = 1 - hp["beta1"] ** hp["step"]
        em = 3 * U * (0.9 * np.abs(q["m0"]) + 0.1 * np.abs(q["g"])).astype(np.float64)
        denom = np.sqrt(q["v64"] / (1 - hp["beta2"] ** hp["step"])) + hp["eps"]
        hat = np.abs(q["m64"]) / c1 / denom
        within(p, q["p"], 3 * U * np.abs(q["p0"]) + hp["lr"] * (em / c1 / denom + 16 * U * hat) + 1e-38, "p")
        assert (to_np(got["p16"]) == W.f32_to_bf16_bits(to_np(got["p"]))).all()
        if bits == 32:
            assert (to_np(got["m"]) == q["m"]).all() and (to_np(got["v"]) == q["v"]).all()
        else:
            for k, x, keep in (("m", q["m"], False), ("v", q["r"], True)):
                code, sc = encode(x, keep)
                assert (to_np(got[k].view(t.uint8)) == code).all(), k
                assert (to_np(got[k + "_scale"]) == sc).all(), k
            assert (G.decode_e4m3(to_np(got["v"].view(t.uint8)))[q["r"] > 0] > 0).all()
        for k, a in f.items():            # nothing around a tensor is written
            size = a[0].element_size()
            raw = to_np(a[1].view(t.uint8))
            lo, hi = shift * size, (shift + a[0].numel()) * size
            assert (raw[:lo] == b[k][:lo]).all() and (raw[hi:] == b[k][hi:]).all(), k


def one_tensor(n, bits, g):
    t = t_()
    z = t.zeros(n, device="cuda")
    d = dict(p=z.clone(), g=g)
    if bits == 8:
        nb = -(-n // 256)
        d.update(m=t.zeros(n, dtype=t.float8_e4m3fn, device="cuda"), v=t.zeros(n, dtype=t.float8_e4m3fn, device="cuda"),
                 m_scale=t.zeros(nb, device="cuda"), v_scale=t.zeros(nb, device="cuda"))
    else:
        d.update(m=z.clone(), v=z.clone())
    return d


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_non_finite_gradients(bits):
    """A NaN or an infinity spoils its element (32 bits) or its block (8 bits)
    and no other; the next step reads it back as NaN."""
    t = t_()
    g = t.full((1024,), 1e-3, device="cuda")
    g[300], g[800] = float("nan"), float("inf")
    d = one_tensor(1024, bits, g)
    plan = moe.adamw_tensors([d])
    moe.moe_adamw_step(plan, moe.make_adamw(1e-3, step=1))
    g.fill_(1e-3)
    moe.moe_adamw_step(plan, moe.make_adamw(1e-3, step=2))
    p = to_np(d["p"])
    bad = np.zeros(1024, bool)
    if bits == 8:
        bad[256:512] = bad[768:1024] = True
    else:
        bad[300] = bad[800] = True
    assert np.isfinite(p[~bad]).all() and (p[~bad] < 0).all()
    assert np.isnan(p[bad]).all()


@pytest.mark.parametrize("value", [0.0, 1e-42, 1e-25, 1e-8, 1e18])
def test_adamw_8bit_from_zero_at_any_size_of_gradient(value):
    """From zeroed moments the first update is lr times the sign, at any size
    of the gradient that the moments can hold; a block of zeros stays zeros."""
    t = t_()
    g = t.full((700,), value, device="cuda")
    g[::2] *= -1
    d = one_tensor(700, 8, g)
    moe.moe_adamw_step(moe.adamw_tensors([d]), moe.make_adamw(1e-3, eps=0.0 if value >= 1e-15 else 1e-8))
    p = to_np(d["p"])
    if value >= 1e-15:
        assert np.allclose(np.abs(p), 1e-3, rtol=1e-5) and (np.sign(p) == -np.sign(to_np(g))).all()
    else:
        assert np.isfinite(p).all() and (np.abs(p) <= 1e-3).all()
    assert np.isfinite(to_np(d["m_scale"])).all() and np.isfinite(to_np(d["v_scale"])).all()
    if value == 0.0:
        assert (p == 0).all() and (to_np(d["m"].view(t.uint8)) == 0).all() and (to_np(d["v_scale"]) == 0).all()


def test_adamw_learns_with_8_bit_moments():
    """A quadratic with noisy gradients: the 8-bit moments end within a tenth
    of the distance that the start had, as the 32-bit ones do."""
    t = t_()
    gen = t.Generator(device="cuda").manual_seed(0)
    goal = t.randn(4096, generator=gen, device="cuda")
    left = {}
    for bits in (32, 8):
        g = t.zeros(4096, device="cuda")
        d = one_tensor(4096, bits, g)
        plan = moe.adamw_tensors([d])
        for step in range(1, 401):
            g.copy_(d["p"] - goal + 0.1 * t.randn(4096, generator=gen, device="cuda"))
            moe.moe_adamw_step(plan, moe.make_adamw(1e-2, beta2=0.95, step=step))
        left[bits] = float((d["p"] - goal).norm() / goal.norm())
    assert left[32] < 0.1 and left[8] < 0.1, left
