"""Newton-Schulz orthogonalisation and the Muon step against a plain
implementation in 64 bits."""
import numpy as np
import pytest

import sparse_mixture_experts_topk_gb300 as moe

pytestmark = pytest.mark.gpu

NS = (3.4445, -4.7750, 2.0315)
U32, U16 = 2.0 ** -24, 2.0 ** -8      # half a step of fp32 and of bf16, relative


def t_():
    import torch
    return torch


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sparse_mixture_experts_topk_gb300 import build
    build.build()


def newton_schulz(u, iterations, held=lambda v: v):
    """The iteration in 64 bits; ``held`` rounds what the kernels hold."""
    a, b, c = NS
    u = np.asarray(u, np.float64)
    norm = np.linalg.norm(u)
    if norm == 0:
        return np.zeros_like(u)
    x = held((u.T if u.shape[0] > u.shape[1] else u) / norm)
    for _ in range(iterations):
        A = held(x @ x.T)
        x = held(held(a * np.eye(len(x)) + b * A + c * (A @ A)) @ x)
    return x.T if u.shape[0] > u.shape[1] else x


def fp16(v):
    return (v * 4096.0).astype(np.float16).astype(np.float64) / 4096.0


def check(got, u, iterations, out_step):
    """Within twice the distance that the same iteration with every held value rounded to fp16 has (the kernels'
    sums are in fp32, 2^-24 a term, and short products of products may be rounded once more), and the result's own
    rounding; a matrix of one element has no averaging, hence the floor of 16 fp16 half steps."""
    want = newton_schulz(u, iterations)
    norm = np.linalg.norm(want)
    model = np.linalg.norm(newton_schulz(u, iterations, fp16) - want)
    assert np.linalg.norm(got - want) <= 2 * model + (out_step + 16 * 2.0 ** -12) * norm


def update_like(r, *shape):
    u = r.standard_normal(shape)
    k = min(4, *shape[-2:])
    return (u + r.standard_normal(shape[:-1] + (k,)) @ r.standard_normal(shape[:-2] + (k, shape[-1]))) * 1e-3


def dev(a, dtype="f32"):
    t = t_()
    return t.from_numpy(np.ascontiguousarray(a)).to("cuda").to(t.bfloat16 if dtype == "bf16" else t.float32)


def run(x, out_dtype, iterations=5):
    t = t_()
    b = int(np.prod(x.shape[:-2], dtype=np.int64))
    ws = moe.orthogonalize_workspace(b, x.shape[-2], x.shape[-1])
    out = t.full(x.shape, 7.0, device="cuda").to(t.bfloat16 if out_dtype == "bf16" else t.float32)
    moe.moe_orthogonalize(x, out, iterations, ws)
    t.cuda.synchronize()
    assert moe.moe_get_device_error(ws) == 0
    return out


SHAPES = [(1, 1, 1), (2, 1, 7), (1, 5, 1), (3, 2, 2), (1, 64, 96), (2, 96, 64), (1, 17, 1000), (2, 257, 300),
          (1, 255, 256), (1, 1001, 130), (2, 520, 520), (1, 384, 1537), (1, 640, 768), (5, 129, 511),
          # on chip, by one, two, four and eight CTAs, and just past that
          (3, 128, 512), (2, 128, 513), (1, 600, 100), (2, 100, 2000), (1, 3000, 33), (2, 128, 4096), (1, 4096, 127),
          (1, 3, 4090), (1, 129, 512), (1, 128, 4100)]


@pytest.mark.parametrize("out_dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES)
def test_orthogonalize(shape, dtype, out_dtype):
    x = dev(update_like(np.random.default_rng(shape), *shape), dtype)
    out = run(x, out_dtype).double().cpu().numpy()
    for i in range(shape[0]):
        check(out[i], x[i].double().cpu().numpy(), 5, U16 if out_dtype == "bf16" else U32)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [(2, 1, 1), (3, 1, 6), (2, 9, 1), (2, 2, 2), (1, 13, 16), (2, 16, 16), (3, 16, 512),
                                   (2, 513, 16), (1, 7, 1001), (2, 1030, 3), (1, 1, 2049), (2, 16, 4096), (1, 4095, 15)])
def test_thin_matrices_are_iterated_in_fp32(shape, dtype):
    """Short sides of up to 16 hold fp32.  The model rounds X, A and B once; the kernel's sums round at each of up to
    30 partial sums (16 columns of a lane, 5 exchanges, 8 CTAs), which in a random walk is under 6 times as far.  A
    matrix of one element has no averaging: the three terms of a step, of 14 together, rounded a few times each, are
    64 half steps with what later steps make of them."""
    x = dev(update_like(np.random.default_rng(shape), *shape), dtype)
    out = run(x, "f32").double().cpu().numpy()
    for i in range(shape[0]):
        u = x[i].double().cpu().numpy()
        want = newton_schulz(u, 5)
        model = np.linalg.norm(newton_schulz(u, 5, lambda v: v.astype(np.float32).astype(np.float64)) - want)
        assert np.linalg.norm(out[i] - want) <= 6 * model + 64 * U32 * np.linalg.norm(want)


@pytest.mark.parametrize("iterations", [5, 4])
@pytest.mark.parametrize("shape", [(12, 1300, 1701), (12, 1900, 1304), (12, 1304, 1304)])
def test_batches_that_fill_the_gpu(shape, iterations):
    """Tiles of SM pairs, two iterations at a time for the longer matrices.  Two matrices in turn, so that two
    oracles do (in 64 bits on the GPU): equal matrices have equal bits wherever their tiles ran."""
    t = t_()
    a, b, c = NS
    x = dev(update_like(np.random.default_rng(shape), 2, *shape[1:])).repeat(shape[0] // 2, 1, 1)
    out = run(x, "f32", iterations)
    for i in range(2, shape[0]):
        assert (out[i] == out[i % 2]).all()

    def iterate(u, held):
        u = u.double()
        v = held((u.T if u.shape[0] > u.shape[1] else u) / u.norm())
        one = t.eye(len(v), dtype=t.float64, device="cuda")
        for _ in range(iterations):
            A = held(v @ v.T)
            v = held(held(a * one + b * A + c * (A @ A)) @ v)
        return v.T if u.shape[0] > u.shape[1] else v

    for i in range(2):
        want = iterate(x[i], lambda v: v)
        model = (iterate(x[i], lambda v: (v * 4096).half().double() / 4096) - want).norm()
        # as in check(); with two iterations at a time three more products are rounded
        assert (out[i].double() - want).norm() <= 2 * model + (U32 + 16 * 2.0 ** -12) * want.norm()


def on_gpu(u, iterations, held=lambda v: v):
    """newton_schulz for a batch, in 64 bits on the GPU; zeros for a zero matrix."""
    t = t_()
    a, b, c = NS
    flip = u.shape[-2] > u.shape[-1]
    v = u.double().mT if flip else u.double()
    norm = t.linalg.matrix_norm(v, keepdim=True)
    v = held(t.where(norm > 0, v / norm, 0.0))
    one = t.eye(v.shape[-2], dtype=t.float64, device="cuda")
    for _ in range(iterations):
        A = held(v @ v.mT)
        v = held(held(a * one + b * A + c * (A @ A)) @ v)
    return v.mT if flip else v


def check_batch(got, u, iterations, noise=0.0):
    """As check(), for each matrix."""
    t = t_()
    want = on_gpu(u, iterations)
    model = t.linalg.matrix_norm(on_gpu(u, iterations, lambda v: (v * 4096).half().double() / 4096) - want)
    off = t.linalg.matrix_norm(got.double() - want)
    assert (off <= 2 * model + (U32 + 16 * 2.0 ** -12) * t.linalg.matrix_norm(want) + noise).all()


def uneven(shape, dtype):
    """Matrices whose size a few of their elements tell, and others where they do not."""
    t = t_()
    n, rows, cols = shape
    gen = t.Generator(device="cuda").manual_seed(rows)
    x = t.randn(shape, device="cuda", generator=gen)
    for i in range(n):
        kind = i % 8
        if kind == 1:       # four strong directions
            x[i] += t.randn(rows, 4, device="cuda", generator=gen) @ t.randn(4, cols, device="cuda", generator=gen)
        elif kind == 2:
            x[i] = 0
        elif kind == 3:     # a single element
            v = x[i, rows // 2, cols // 3].item()
            x[i] = 0
            x[i, rows // 2, cols // 3] = v
        elif kind == 4:     # a few rows
            x[i, 3:] = 0
        elif kind == 5:     # columns of very different sizes
            x[i] *= t.exp(3 * t.randn(cols, device="cuda", generator=gen))
        elif kind == 6:
            x[i] *= 1e-25
        elif kind == 7:
            x[i] *= 1e25
    return x.to(t.bfloat16 if dtype == "bf16" else t.float32)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [(20, 601, 904), (24, 1000, 440), (10, 1024, 1024), (20, 601, 903)])
def test_batches_whose_norms_are_guessed(shape, dtype):
    x = uneven(shape, dtype)
    out = run(x, "f32")
    check_batch(out, x, 5)
    assert (run(x, "f32") == out).all()
    # off the 16-byte grid, and in place
    t = t_()
    y = t.empty(x.numel() + 1, dtype=x.dtype, device="cuda")[1:].view(shape)
    y.copy_(x)
    assert (run(y, "f32") == out).all()
    if dtype == "f32":
        ws = moe.orthogonalize_workspace(*shape)
        moe.moe_orthogonalize(y, y, 5, ws)
        assert (y == out).all()
    # each keeps to itself: NaN, and another's size
    y = x.clone()
    y[0, 3, 4] = float("nan")
    y[1] = y[2]
    again = run(y, "f32")
    assert again[0].isnan().all() and (again[1] == out[2]).all() and (again[2:] == out[2:]).all()


@pytest.mark.parametrize("iterations", [1, 2, 3, 4, 6])
@pytest.mark.parametrize("shape", [(200, 300), (300, 200), (264, 1100)])
def test_number_of_iterations(shape, iterations):
    x = dev(update_like(np.random.default_rng(iterations), *shape))
    check(run(x, "f32", iterations).double().cpu().numpy(), x.double().cpu().numpy(), iterations, U32)


def test_result_is_nearly_orthogonal():
    """Singular values of a Gaussian 200 x 800 are within (0.5, 1.5) / sqrt(200) of |u|: five iterations take them
    into the band that the quintic leaves, [0.68, 1.21]."""
    x = dev(np.random.default_rng(1).standard_normal((200, 800)))
    s = np.linalg.svd(run(x, "f32").double().cpu().numpy(), compute_uv=False)
    assert s.min() > 0.66 and s.max() < 1.22


def test_transposes_batches_and_repeats():
    """The same bits again, alone as in a batch, in place and off the 16-byte grid.  A transpose's norm is summed in
    another order, and a last bit of it moves roundings of X: the same result within the bound."""
    r = np.random.default_rng(2)
    x = dev(update_like(r, 7, 300, 200))
    out = run(x, "f32")
    assert (out == run(x, "f32")).all()
    flipped = run(x.mT.contiguous(), "f32").mT.double().cpu().numpy()
    for i in range(7):
        check(flipped[i], x[i].double().cpu().numpy(), 5, U32)
    for i in (0, 3, 6):
        assert (out[i] == run(x[i], "f32")).all()
    t = t_()
    flat = t.zeros(x.numel() + 1, device="cuda")
    y = flat[1:].view(x.shape)
    y.copy_(x)
    ws = moe.orthogonalize_workspace(7, 300, 200)
    moe.moe_orthogonalize(y, y, 5, ws)
    assert (y == out).all() and flat[0] == 0


@pytest.mark.parametrize("power", [-130, -70, -20, 20, 60, 120])
def test_scale_does_not_matter(power):
    """u and u 2^k have the same X but for values that vanish at the ends of fp32's range."""
    r = np.random.default_rng(3)
    u = update_like(r, 2, 60, 80) * 1e3
    x = dev(u)
    assert (run(x * 2.0 ** power, "f32") == run(x, "f32")).all() or power == -130
    if power == -130:     # subnormal inputs: bits are lost before the call
        y = x * 2.0 ** power
        got = run(y, "f32").double().cpu().numpy()
        for i in range(2):
            check(got[i], y[i].double().cpu().numpy() * 2.0 ** 130, 5, U32)


def test_a_zero_matrix_and_a_matrix_with_nan_keep_to_themselves():
    r = np.random.default_rng(4)
    x = dev(update_like(r, 5, 130, 270))
    clean = run(x, "f32")
    x[1] = 0
    x[2, 3, 4] = float("nan")
    x[3, 129, 269] = float("inf")
    out = run(x, "f32")
    assert (out[1] == 0).all()
    assert out[2].isnan().all() and out[3].isnan().all()
    assert (out[0] == clean[0]).all() and (out[4] == clean[4]).all()


@pytest.mark.parametrize("rows,cols", [(9, 40), (700, 16), (64, 96)])
def test_a_zero_matrix_and_a_matrix_with_nan_on_chip(rows, cols):
    r = np.random.default_rng(4)
    x = dev(update_like(r, 5, rows, cols))
    clean = run(x, "f32")
    x[1] = 0
    x[2, 3, 4] = float("nan")
    x[3, -1, -1] = float("inf")
    out = run(x, "f32")
    assert (out[1] == 0).all()
    assert out[2].isnan().all() and out[3].isnan().all()
    assert (out[0] == clean[0]).all() and (out[4] == clean[4]).all()


# ------------------------------------------------------------------ the step

def step_case(shapes, grad, seed, p16=True):
    r = np.random.default_rng(seed)
    t = t_()
    out = []
    for i, s in enumerate(shapes):
        p = dev(r.standard_normal(s) * 0.02)
        d = {"p": p, "g": dev(update_like(r, *s), grad), "m": dev(update_like(r, *s) * 3), "weight_decay": 0.1 * (i % 2)}
        if p16:
            d["p16"] = t.zeros(s, dtype=t.bfloat16, device="cuda")
        out.append(d)
    return out


def check_step(before, after, lr, mu, nesterov, iterations, factor):
    for b, a in zip(before, after):
        g = b["g"].astype(np.float64) * factor
        m = mu * b["m"] + g
        assert (abs(a["m"] - m) <= 4 * U32 * (abs(mu * b["m"]) + abs(g))).all()
        u = g + mu * m if nesterov else m
        size = b["p"].shape[-2:]
        scale = b.get("scale", 0.2 * np.sqrt(max(size)))
        keep = 1 - lr * b["weight_decay"]
        moved = (b["p"] * keep - a["p"]) / (lr * scale)
        noise = np.linalg.norm(b["p"]) * 4 * U32 / (lr * scale)      # p's own rounding, seen through the quotient
        for got, ui in zip(moved.reshape((-1,) + size), u.reshape((-1,) + size)):
            want = newton_schulz(ui, iterations)
            model = np.linalg.norm(newton_schulz(ui, iterations, fp16) - want)
            assert np.linalg.norm(got - want) <= 2 * model + 16 * 2.0 ** -12 * np.linalg.norm(want) + noise
        if "p16" in a:
            assert (a["p16"] == t_().from_numpy(a["p"]).float().to(t_().bfloat16).double().numpy()).all()


def numbers(tensors):
    return [{k: v.double().cpu().numpy() if hasattr(v, "cpu") else v for k, v in d.items()} for d in tensors]


@pytest.mark.parametrize("grad", ["f32", "bf16"])
@pytest.mark.parametrize("nesterov", [True, False])
def test_muon_step(grad, nesterov):
    """Tensors of several sizes, two of one size the other way round, batches, a single matrix, one element."""
    shapes = [(3, 96, 160), (2, 160, 96), (130, 257), (1, 1), (4, 8, 8), (2, 2, 24, 40)]
    tensors = step_case(shapes, grad, 5, p16=nesterov)
    t = t_()
    plan, params = moe.muon_tensors(tensors), moe.make_muon(0.02, 0.9, nesterov, 5)
    ws = moe.muon_workspace(plan)
    factor = t.full((1,), 0.5, device="cuda")
    for _ in range(2):
        before = numbers(tensors)
        moe.moe_muon_step(plan, params, factor, None, ws)
        check_step(before, numbers(tensors), 0.02, np.float64(np.float32(0.9)), nesterov, 5, 0.5)
    assert moe.moe_get_device_error(ws) == 0


@pytest.mark.parametrize("grad", ["f32", "bf16"])
@pytest.mark.parametrize("nesterov", [True, False])
def test_muon_step_of_batches_whose_norms_are_guessed(grad, nesterov):
    t = t_()
    mu, lr, f = float(np.float32(0.9)), 0.02, 0.5
    tensors = [{"p": t.randn(s, device="cuda") * 0.02, "g": uneven(s, grad), "m": uneven(s, "f32").flip(0).contiguous() * 0.1,
                "weight_decay": 0.1, "scale": 1.0} for s in [(16, 604, 900), (9, 900, 604)]]
    plan, params = moe.muon_tensors(tensors), moe.make_muon(lr, 0.9, nesterov, 5)
    ws = moe.muon_workspace(plan)
    before = [{k: v.clone() if hasattr(v, "clone") else v for k, v in d.items()} for d in tensors]
    moe.moe_muon_step(plan, params, t.full((1,), f, device="cuda"), None, ws)
    assert moe.moe_get_device_error(ws) == 0
    for b, a in zip(before, tensors):
        g, p = b["g"].double() * f, b["p"].double()
        m = mu * b["m"].double() + g
        assert ((a["m"].double() - m).abs() <= 4 * U32 * ((mu * b["m"].double()).abs() + g.abs())).all()
        u = g + mu * m if nesterov else m
        moved = (p * (1 - lr * 0.1) - a["p"].double()) / lr
        check_batch(moved, u, 5, t.linalg.matrix_norm(p) * 4 * U32 / lr)


def test_muon_step_skips_and_takes_no_tensor():
    tensors = step_case([(2, 40, 60)], "f32", 6)
    t = t_()
    plan, params = moe.muon_tensors(tensors), moe.make_muon(0.1)
    ws = moe.muon_workspace(plan)
    before = numbers(tensors)
    tensors[0]["g"][0, 1, 2] = float("nan")
    moe.moe_muon_step(plan, params, None, t.ones(1, dtype=t.int32, device="cuda"), ws)
    for b, a in zip(before, numbers(tensors)):
        for k in ("p", "m", "p16"):
            assert (a[k] == b[k]).all(), k
    moe.moe_muon_step(plan, params, None, t.zeros(1, dtype=t.int32, device="cuda"), ws)
    assert tensors[0]["p"][0].isnan().all() and not tensors[0]["p"][1].isnan().any()
    empty = moe.muon_tensors([])
    moe.moe_muon_step(empty, params, None, None, moe.muon_workspace(empty))


def test_more_tensors_than_a_launch_takes():
    tensors = step_case([(1 + i % 3, 24, 40) if i % 2 else (40, 24) for i in range(61)], "f32", 7)
    plan, params = moe.muon_tensors(tensors), moe.make_muon(0.02, 0.95, True, 3)
    ws = moe.muon_workspace(plan)
    before = numbers(tensors)
    moe.moe_muon_step(plan, params, None, None, ws)
    check_step(before, numbers(tensors), 0.02, np.float64(np.float32(0.95)), True, 3, 1.0)
