"""A call whose matrices of one size take several runs of the products: more
tensors than a launch takes, or more matrices than the workspace holds."""
import numpy as np
import pytest

import sparse_mixture_experts_topk_gb300 as moe

from test_gpu_orthogonalize import U32, check_batch, check_step, dev, numbers, run, step_case, t_, update_like

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sparse_mixture_experts_topk_gb300 import build
    build.build()


def clones(tensors):
    return [{k: v.clone() if hasattr(v, "clone") else v for k, v in d.items()} for d in tensors]


def repeats(tensors, results, iterations=5):
    """The same bits again, eagerly and replayed from a graph, from copies of the tensors."""
    t = t_()
    for captured in (False, True):
        again = clones(tensors)
        plan = moe.muon_tensors(again)
        ws, params = moe.muon_workspace(plan), moe.make_muon(0.02, iterations=iterations)
        t.cuda.synchronize()
        if captured:
            graph = t.cuda.CUDAGraph()
            with t.cuda.graph(graph):
                moe.moe_muon_step(plan, params, None, None, ws)
            graph.replay()
        else:
            moe.moe_muon_step(plan, params, None, None, ws)
        t.cuda.synchronize()
        assert moe.moe_get_device_error(ws) == 0
        for a, b in zip(again, results):
            assert all((a[k] == b[k]).all() for k in ("p", "m", "p16"))


def test_more_tensors_of_one_size_than_a_launch_takes():
    """Three runs of one size, each laid out anew in the workspace, another size in between, and small and thin
    matrices that start beside the last of them."""
    shapes = [s for i in range(30) for s in ([(1, 130, 200)] if i % 3 else [(2, 200, 130), (1, 150, 140)])]
    shapes += [(24, 40), (3, 100, 700), (9, 300), (2, 1500, 12)]
    tensors = step_case(shapes, "f32", 51)
    t = t_()
    plan, params = moe.muon_tensors(tensors), moe.make_muon(0.02)
    ws = moe.muon_workspace(plan)
    first, before = clones(tensors), numbers(tensors)
    moe.moe_muon_step(plan, params, None, None, ws)
    check_step(before, numbers(tensors), 0.02, np.float64(np.float32(0.95)), True, 5, 1.0)
    assert moe.moe_get_device_error(ws) == 0
    repeats(first, tensors)


def test_a_size_whose_first_run_guesses_its_norms():
    """24 tensors of 520 x 700 have 2^23 elements and more, the six behind them have not."""
    t = t_()
    gen = t.Generator(device="cuda").manual_seed(52)
    lr, mu = 0.02, float(np.float32(0.95))

    def rand(*s, scale=1.0):
        return t.randn(s, device="cuda", generator=gen) * scale

    tensors = []
    for i in range(30):
        s = (520, 700) if i % 2 else (700, 520)
        tensors.append({"p": rand(*s, scale=0.02), "p16": t.zeros(s, dtype=t.bfloat16, device="cuda"),
                        "g": rand(*s) + rand(s[0], 3) @ rand(3, s[1]), "m": rand(*s, scale=10.0 ** (i % 5 - 2)),
                        "weight_decay": 0.1, "scale": 1.0})
    tensors.append({"p": rand(60, 90), "p16": t.zeros((60, 90), dtype=t.bfloat16, device="cuda"), "g": rand(60, 90),
                    "m": rand(60, 90), "weight_decay": 0.1, "scale": 1.0})
    first = clones(tensors)
    plan, params = moe.muon_tensors(tensors), moe.make_muon(lr)
    ws = moe.muon_workspace(plan)
    moe.moe_muon_step(plan, params, None, None, ws)
    assert moe.moe_get_device_error(ws) == 0
    for b, a in zip(first, tensors):
        g, p = b["g"].double(), b["p"].double()
        m = mu * b["m"].double() + g
        assert ((a["m"].double() - m).abs() <= 4 * U32 * ((mu * b["m"].double()).abs() + g.abs())).all()
        moved = (p * (1 - lr * 0.1) - a["p"].double()) / lr
        check_batch(moved, g + mu * m, 5, t.linalg.matrix_norm(p) * 4 * U32 / lr)
        assert (a["p16"] == a["p"].to(t.bfloat16)).all()
    repeats(first, tensors)


def test_a_batch_larger_than_the_workspace_holds():
    """30000 matrices of 130 x 132: a part of 4 GiB and the rest.  Seven in turn, so that seven oracles do."""
    n = moe.moe_orthogonalize_workspace_size(30000, 130, 132)
    assert n == moe.moe_orthogonalize_workspace_size(60000, 130, 132)
    x = dev(update_like(np.random.default_rng(53), 7, 130, 132)).repeat(-(-30000 // 7), 1, 1)[:30000].contiguous()
    out = run(x, "f32")
    check_batch(out[:7], x[:7], 5)
    for i in range(7):
        assert (out[i::7] == out[i]).all()


@pytest.mark.parametrize("shape", [(2, 1, 5000), (3, 5000, 3), (2, 17, 7000), (1, 4100, 16), (1, 129, 129), (2, 32768, 2),
                                   (1, 60, 9000)])
def test_thin_matrices_longer_than_a_chip_takes(shape):
    x = dev(update_like(np.random.default_rng(shape), *shape))
    out = run(x, "f32")
    check_batch(out, x, 5)
    assert (run(x, "f32") == out).all()
