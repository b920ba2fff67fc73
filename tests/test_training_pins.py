"""Pins of the gradient oracle: against central differences of the forward
oracle, hand values, and exhaustive rounding."""
import numpy as np
import pytest

from oracle import moe_oracle as O
from oracle import train_oracle as G

STEP = 1e-5
# A central difference with step h of a function with third derivative D and
# rounding noise u |f| / h is off by D h^2 / 6 + 2^-52 |f| / h: with h = 1e-5
# and values of order 1 to 10 both terms are below 1e-9.
DIFF = 1e-7


def difference(f, x):
    """Gradient of the scalar f at the array x by central differences."""
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        keep = x[i]
        x[i] = keep + STEP
        up = f()
        x[i] = keep - STEP
        down = f()
        x[i] = keep
        g[i] = (up - down) / (2 * STEP)
    return g


@pytest.mark.parametrize("act", ["gelu", "swiglu"])
@pytest.mark.parametrize("bias", [False, True])
def test_expert_gradient_is_the_difference_quotient(act, bias):
    rng = np.random.default_rng(7)
    n, H, F = 3, 5, 4
    g = 2 if act == "swiglu" else 1
    x, W1, W2 = rng.normal(size=(n, H)), rng.normal(size=(g * F, H)), rng.normal(size=(H, F))
    b1, b2 = (rng.normal(size=g * F), rng.normal(size=H)) if bias else (None, None)
    dy = rng.normal(size=(n, H))

    def loss():
        return float((dy * O.expert_ffn(x, W1, W2, b1, b2, act=act)).sum())

    a = x @ W1.T + (0 if b1 is None else b1)
    h = O.silu(a[:, :F]) * a[:, F:] if act == "swiglu" else O.gelu(a)
    r = G.expert_ffn_backward(x, h, dy, W1, W2, b1, act)
    assert np.abs(r["dx"] - difference(loss, x)).max() < DIFF
    assert np.abs(r["dW1"] - difference(loss, W1)).max() < DIFF
    assert np.abs(r["dW2"] - difference(loss, W2)).max() < DIFF
    if bias:
        assert np.abs(r["db1"] - difference(loss, b1)).max() < DIFF
        assert np.abs(r["db2"] - difference(loss, b2)).max() < DIFF


def test_combine_and_dispatch_gradients_are_difference_quotients():
    rng = np.random.default_rng(8)
    T, K, E, H = 6, 2, 3, 4
    ids = np.stack([rng.permutation(E)[:K] for _ in range(T)])
    d = O.dispatch(ids, E, 3)
    assert d["dropped"] > 0
    R = int(d["offs"][E])
    y, w, dout = rng.normal(size=(R, H)), rng.uniform(size=(T, K)), rng.normal(size=(T, H))

    def loss():
        return float((dout * O.combine(y, d["pos"], w)).sum())

    dy, dw = G.combine_backward(dout, y, d["pos"], w)
    assert np.abs(dy - difference(loss, y)).max() < DIFF
    assert np.abs(dw - difference(loss, w)).max() < DIFF
    # the dispatch: x_perm[r] = x[src[r] // K]
    x, dxp = rng.normal(size=(T, H)), rng.normal(size=(R, H))
    dx = G.dispatch_backward(dxp, d["pos"], T, K)
    assert np.abs(dx - difference(lambda: float((dxp * x[d["src"] // K]).sum()), x)).max() < DIFF
    add = rng.normal(size=(T, H))
    assert np.allclose(G.dispatch_backward(dxp, d["pos"], T, K, add), dx + add, atol=1e-15)


def test_whole_layer_gradient_is_the_difference_quotient():
    """The three steps in a row are the gradient of the layer's output with
    the routing held fixed."""
    rng = np.random.default_rng(9)
    T, K, E, H, F = 4, 2, 3, 3, 2
    x, Wg = rng.normal(size=(T, H)), rng.normal(size=(E, H))
    W1, W2 = rng.normal(size=(E, F, H)), rng.normal(size=(E, H, F))
    ids, w, _ = O.route(O.gate_logits(x, Wg), K)
    d = O.dispatch(ids, E, 0)
    dout = rng.normal(size=(T, H))

    def loss():
        y = O.expert_outputs(x, d, W1, W2, ids=ids)
        return float((dout * O.combine(y, d["pos"], w)).sum())

    y = O.expert_outputs(x, d, W1, W2, ids=ids)
    dy, _ = G.combine_backward(dout, y, d["pos"], w)
    dxp = np.zeros_like(y)
    for e in range(E):
        r = slice(int(d["offs"][e]), int(d["offs"][e + 1]))
        xe = x[d["src"][r] // K]
        dxp[r] = G.expert_ffn_backward(xe, O.gelu(xe @ W1[e].T), dy[r], W1[e], W2[e])["dx"]
    assert np.abs(G.dispatch_backward(dxp, d["pos"], T, K) - difference(loss, x)).max() < DIFF


def test_adamw_by_hand():
    # first step from zero moments: the update is lr g / (|g| + eps) whatever |g|
    p, m, v = G.adamw(np.array([1.0, -2.0]), np.array([0.5, -3.0]), np.zeros(2), np.zeros(2), 0.1, 0.9, 0.99, 0.0, 1,
                      0.0)
    assert np.allclose(p, [0.9, -1.9]) and np.allclose(m, [0.05, -0.3]) and np.allclose(v, [0.0025, 0.09])
    # decay alone
    p, _, _ = G.adamw(np.array([2.0]), np.zeros(1), np.zeros(1), np.zeros(1), 0.1, 0.9, 0.99, 1e-8, 5, 0.5)
    assert np.allclose(p, [1.9])


def test_e4m3_rounds_every_midpoint_to_even():
    val = G.e4m3_values()
    assert val[126] == 448.0 and val[1] == 2.0 ** -9 and (np.diff(val) > 0).all()
    assert (G.encode_e4m3(val) == np.arange(127)).all() and (G.encode_e4m3(-val[1:]) == 128 + np.arange(1, 127)).all()
    mid = (val[1:] + val[:-1]) / 2
    code = G.encode_e4m3(mid)
    assert (code % 2 == 0).all()
    assert (G.encode_e4m3(np.nextafter(mid, 1e9)) == np.arange(1, 127)).all()
    assert (G.encode_e4m3(np.nextafter(mid, 0)) == np.arange(126)).all()
    assert G.encode_e4m3(np.array([1e9]))[0] == 126
    torch = pytest.importorskip("torch")
    x = np.random.default_rng(3).normal(size=20000).astype(np.float32) * 60
    want = torch.from_numpy(np.clip(x, -448, 448)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert (G.encode_e4m3(x.astype(np.float64)) == want).all()
