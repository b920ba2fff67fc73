"""The products of the router's gradient where a CTA walks over several tiles of
128 tokens: H = 4096 leaves four CTAs for a chunk of columns, so that 5000 tokens
are ten tiles each.  Rings wrap, accumulators are used again, sums go over
tiles; masks leave whole tiles without a token that counts."""
import pytest

import sparse_mixture_experts_topk_gb300 as moe

from test_gpu_router_backward import U16, t_

pytestmark = pytest.mark.gpu

Z32 = 2.0 ** -23      # a step of fp32: the tensor cores' sums round towards zero


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sparse_mixture_experts_topk_gb300 import build
    build.build()


def masks(T):
    """Random tokens, padded sequences, and single tiles at the ends and within."""
    t = t_()
    at = t.arange(T, device="cuda")
    gen = t.Generator(device="cuda").manual_seed(T)
    real = t.randint(1, 1100, (-(-T // 1100), 1), generator=gen, device="cuda")
    real[0] = 1
    return {"none": None, "random": t.rand(T, generator=gen, device="cuda") < 0.6,
            "sequences": (t.arange(1100, device="cuda") < real).view(-1)[:T].contiguous(),
            "first": at < 1, "last": at == T - 1, "within": (at >= 640) & (at < 700),
            "ends": (at < 100) | (at >= T - 3), "middle_out": (at < 256) | (at >= T // 2)}


def inputs(T, H, E, K, mask, seed=0):
    """x positive on the whole, so that sums grow; NaN in what the mask leaves out."""
    t = t_()
    g = t.Generator(device="cuda").manual_seed(seed * 1000 + E)

    def rand(*s):
        return t.randn(s, device="cuda", generator=g)

    q = {"logits": rand(T, E) * 2, "x": (rand(T, H) + 0.5).bfloat16(),
         "Wg": (rand(E, H) * 0.1).bfloat16(), "dw": rand(T, K)}
    q["ids"] = q["logits"].topk(K, dim=1).indices.int().contiguous()
    q["dloss"] = t.full((1,), 300.0, device="cuda")
    live = t.ones(T, dtype=t.bool, device="cuda") if mask is None else mask
    q["count"] = t.bincount(q["ids"][live].long().view(-1), minlength=E).int()
    q["tokens"] = live.sum().int().view(1)
    q["live"] = live
    for k in ("logits", "x", "dw"):
        q[k][~live] = float("nan")
    return q


def run(q, E, K, mask, want=("dlogits", "dWg", "dbias", "dx")):
    t = t_()
    T, H = q["x"].shape
    d = moe.make_desc(T, H, E, K, 8)
    ws = moe.router_backward_workspace(d)
    o = {"dlogits": t.full((T, E), 7.0, device="cuda"), "dWg": t.full((E, H), 7.0, device="cuda"),
         "dbias": t.full((E,), 7.0, device="cuda"), "dx": t.full((T, H), 7.0, device="cuda").bfloat16()}
    o = {k: v if k in want else None for k, v in o.items()}
    moe.moe_router_backward(d, q["x"], q["Wg"], q["logits"], q["ids"], q["dw"], q["dloss"], q["count"], q["tokens"], mask,
                            o["dlogits"], o["dWg"], o["dbias"], o["dx"], ws)
    t.cuda.synchronize()
    assert moe.moe_get_device_error(ws) == 0
    return o


def check_scores(q, o, E, K):
    """The scores' gradient against its formula in 64 bits; the bound is test_gpu_router_backward's."""
    t = t_()
    live = q["live"]
    z, ids, dw = q["logits"][live].double(), q["ids"][live].long(), q["dw"][live].double()
    p = t.softmax(z, 1)
    n = float(q["tokens"])
    c = q["dloss"].double() * E * q["count"].double() / (n * n * K)
    dot = (p @ c)[:, None]
    w = t.softmax(z.gather(1, ids), 1)
    want, size = p * (c - dot), p * (c + dot)
    want.scatter_add_(1, ids, w * (dw - (w * dw).sum(1, keepdim=True)))
    size.scatter_add_(1, ids, w * (dw.abs() + (w * dw.abs()).sum(1, keepdim=True)))
    got = o["dlogits"].double()
    assert (got[~live] == 0).all()
    assert ((got[live] - want).abs() <= (64 + 4 * z.abs().max()) * Z32 / 2 * size + 1e-37).all()


def check_products(q, o, E):
    """The products of the scores' gradient that the call returned, so that the sums alone are measured.
    dWg: a tile's tokens (four tiles' above 128 experts) are added up in the tensor cores, a step of the terms' sum
    for each, the parts of 2^-8 and 2^-16 of it included; tiles of a CTA and CTAs of a chunk are then added up in
    fp32, half a step each.  dx: see below, and its own rounding."""
    dl = o["dlogits"].double()
    x = q["x"].double()
    x[~q["live"]] = 0
    run_tiles = 1 if E <= 128 else 4
    want, size = dl.T @ x, dl.abs().T @ x.abs()
    assert ((o["dWg"].double() - want).abs() <= (run_tiles * 130 + 16) * Z32 * size + 1e-37).all()
    # rounding towards zero takes its share of the sums in one direction: a step for each of the MMAs that add up a
    # tile's high parts (8), and as many for what is smaller
    scale = (o["dWg"].double() * want).sum() / (want * want).sum()
    assert abs(scale.item() - 1) <= 16 * run_tiles * Z32
    bias = dl.sum(0)
    assert ((o["dbias"].double() - bias).abs() <= len(dl) * Z32 / 2 * dl.abs().sum(0) + 1e-37).all()
    W = q["Wg"].double()
    want, size = dl @ W, dl.abs() @ W.abs()
    got = o["dx"].double()
    assert (got[~q["live"]] == 0).all()
    # two bf16 parts leave out 2^-18 of each; an MMA adds 16 products to a sum, each of the 17 cut off by a step of the
    # sum of the magnitudes at most: the high parts take one for 16 experts, those before and behind them two more
    parts = 2.0 ** -18 + (17 * (-(-E // 16) + 2) + 1) * Z32
    assert ((got - want).abs() <= parts * size * (1 + U16) + U16 * want.abs() + 1e-37).all()


@pytest.mark.parametrize("kind", ["none", "random", "sequences", "first", "last", "within", "ends", "middle_out"])
@pytest.mark.parametrize("T,E,K", [(1300, 12, 3), (5000, 12, 2), (5000, 32, 2), (5000, 33, 4), (5000, 64, 2), (5000, 100, 2),
                                   (5000, 128, 8), (1300, 130, 2), (5000, 130, 4), (5000, 192, 2), (5000, 256, 8)])
def test_several_tiles_a_cta(T, E, K, kind):
    mask = masks(T)[kind]
    q = inputs(T, 4096, E, K, mask)
    o = run(q, E, K, mask)
    check_scores(q, o, E, K)
    check_products(q, o, E)
    again = run(q, E, K, mask)
    assert all((again[k] == o[k]).all() for k in o)
    for k in ("dWg", "dx"):
        assert (run(q, E, K, mask, (k,))[k] == o[k]).all()


@pytest.mark.parametrize("E", [12, 64, 200])
def test_sums_over_a_long_batch_are_not_biased(E):
    """32 tiles a CTA: sums that were not begun anew would be 1e-5 and more too small."""
    q = inputs(16384, 4096, E, 2, None, seed=1)
    o = run(q, E, 2, None)
    check_products(q, o, E)


@pytest.mark.parametrize("T,H,E", [(700, 5120, 12), (700, 7168, 64), (1500, 8, 130), (20000, 72, 256), (3000, 9728, 40)])
def test_other_widths(T, H, E):
    """One to 152 CTAs a chunk, the last chunk of a few columns."""
    mask = masks(T)["sequences"]
    q = inputs(T, H, E, 2, mask, seed=2)
    o = run(q, E, 2, mask)
    check_scores(q, o, E, 2)
    check_products(q, o, E)


@pytest.mark.parametrize("E", [5, 32, 64, 100, 256])
def test_dx_of_a_gate_whose_rows_are_nearly_alike(E):
    """A token's scores' gradients add up to zero, so that what Wg's rows share cancels in dx.  At the most, 128 with
    or without the last bit of bf16: dx' own rounding is 2^-9 of it at most, what two parts leave out 2^-18 / sqrt(3)
    of terms 256 times the size (half a bit's deviation) of those that dx adds up: 0.29 of 2^-9, and the sums' fp32 a
    fraction of that."""
    t = t_()
    q = inputs(1000, 264, E, 4, None, seed=3)
    gen = t.Generator(device="cuda").manual_seed(E)
    q["Wg"] = (128 + t.randint(0, 2, (E, 264), generator=gen, device="cuda")).bfloat16()
    o = run(q, E, 4, None)
    check_scores(q, o, E, 4)
    check_products(q, o, E)
    dl = o["dlogits"].double()
    # the call's own scores' gradients add up to zero but for their rounding, which is no product's: taken out
    want = dl @ (q["Wg"].double() - 128) + 128 * dl.sum(1, keepdim=True)
    off = (o["dx"].double() - want).square().mean().sqrt()
    assert off <= 1.5 * U16 / 2 * want.square().mean().sqrt()
