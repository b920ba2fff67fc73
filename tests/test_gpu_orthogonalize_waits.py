"""The bounded waits of the orthogonalisation: made to run out, the call ends,
reports a timeout and leaves every element of a result old or new."""
import time

import numpy as np
import pytest

import sparse_mixture_experts_topk_gb300 as moe

from test_gpu_orthogonalize import check, check_batch, check_step, dev, numbers, step_case, update_like, U32

pytestmark = pytest.mark.gpu

STALL = moe.MOE_ORTHOGONALIZE_TEST_WAIT_TIMEOUT


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sparse_mixture_experts_topk_gb300 import build
    build.build()


def ends(call, ws, limit):
    """The call reports a timeout within `limit` seconds."""
    import torch
    torch.cuda.synchronize()
    start = time.time()
    call()
    torch.cuda.synchronize()
    assert moe.moe_get_device_error(ws) == moe.MOE_ERR_TIMEOUT
    assert 1.0 < time.time() - start < limit


def expire(shape):
    """Nothing of out is written; the next call, in the same workspace, is right."""
    import torch
    x = dev(update_like(np.random.default_rng(shape), *shape))
    out = torch.full(shape, 7.0, device="cuda")
    ws = moe.orthogonalize_workspace(*shape)
    ends(lambda: moe.moe_orthogonalize(x, out, 5 | STALL, ws), ws, 30.0)
    assert (out == 7).all()
    moe.moe_orthogonalize(x, out, 5, ws)
    assert moe.moe_get_device_error(ws) == 0
    if x.numel() > 1 << 22:
        check_batch(out, x, 5)
        return
    for i in range(shape[0]):
        check(out[i].double().cpu().numpy(), x[i].double().cpu().numpy(), 5, U32)


@pytest.mark.parametrize("shape", [(3, 64, 96), (2, 100, 600), (2, 1100, 128), (1, 40, 4096)])
def test_expired_wait_on_chip(shape):
    expire(shape)


@pytest.mark.parametrize("shape", [(4, 300, 700), (1, 130, 200), (2, 700, 600), (12, 1300, 1701)])
def test_expired_wait_of_the_products(shape):
    """Tiles of 128 and of 256 columns, on as many pairs as there are tiles: a third of them stall at their first
    stage; of a third the leader's first producer gives up with a tile that only the others load, so that their
    copies' barriers were never armed; and of a third before a tile is known."""
    expire(shape)


def test_a_step_of_every_kind_of_matrix_whose_waits_expire():
    """Elements are old or new: the thin matrices have no such wait and get new ones, the others keep theirs."""
    import torch
    tensors = step_case([(3, 300, 400), (2, 600, 130), (4, 64, 96), (2, 1100, 40), (5, 300)], "bf16", 42)
    plan = moe.muon_tensors(tensors)
    ws = moe.muon_workspace(plan)
    before = numbers(tensors)
    ends(lambda: moe.moe_muon_step(plan, moe.make_muon(0.02, iterations=5 | STALL), None, None, ws), ws, 60.0)
    middle = numbers(tensors)
    mu = np.float64(np.float32(0.95))
    for b, a in zip(before[:4], middle):
        assert all((a[k] == b[k]).all() for k in ("p", "p16"))
    check_step(before[4:], middle[4:], 0.02, mu, True, 5, 1.0)
    moe.moe_muon_step(plan, moe.make_muon(0.02), None, None, ws)
    torch.cuda.synchronize()
    assert moe.moe_get_device_error(ws) == 0
    check_step(middle, numbers(tensors), 0.02, mu, True, 5, 1.0)


def test_a_step_whose_waits_expire_moves_m_alone():
    import torch
    tensors = step_case([(3, 64, 96), (2, 1100, 40)], "f32", 41)
    plan = moe.muon_tensors(tensors)
    ws = moe.muon_workspace(plan)
    before = numbers(tensors)
    ends(lambda: moe.moe_muon_step(plan, moe.make_muon(0.02, iterations=5 | STALL), None, None, ws), ws, 30.0)
    middle = numbers(tensors)
    mu = np.float64(np.float32(0.95))
    for b, a in zip(before, middle):
        assert all((a[k] == b[k]).all() for k in ("p", "p16"))
        m = mu * b["m"] + b["g"]
        assert (abs(a["m"] - m) <= 4 * U32 * (abs(mu * b["m"]) + abs(b["g"]))).all()
    moe.moe_muon_step(plan, moe.make_muon(0.02), None, None, ws)
    torch.cuda.synchronize()
    assert moe.moe_get_device_error(ws) == 0
    check_step(middle, numbers(tensors), 0.02, mu, True, 5, 1.0)
