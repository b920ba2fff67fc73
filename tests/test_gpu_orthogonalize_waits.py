"""The bounded waits of the orthogonalisation: made to run out, the call ends,
reports a timeout and leaves every element of a result old or new."""
import time

import numpy as np
import pytest

import sparse_mixture_experts_topk_gb300 as moe

from test_gpu_orthogonalize import check, check_step, dev, numbers, step_case, update_like, U32

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
    for i in range(shape[0]):
        check(out[i].double().cpu().numpy(), x[i].double().cpu().numpy(), 5, U32)


@pytest.mark.parametrize("shape", [(3, 64, 96), (2, 100, 600), (2, 1100, 128), (1, 40, 4096)])
def test_expired_wait_on_chip(shape):
    expire(shape)


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
