"""Matrices on chip whose cluster has CTAs with no column, or with few: their
stores to the others' shared memory come first."""
import numpy as np
import pytest

import sparse_mixture_experts_topk_gb300 as moe

from test_gpu_orthogonalize import check, check_step, dev, numbers, run, step_case, update_like, U32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sparse_mixture_experts_topk_gb300 import build
    build.build()


@pytest.mark.parametrize("shape", [(40, 40, 1025), (40, 1100, 33), (9, 128, 1536), (40, 17, 2049), (1, 2600, 120),
                                   (200, 12, 1100), (200, 2560, 3)])
def test_ctas_without_columns(shape):
    """Two matrices in turn, so that two oracles do; the others have their bits."""
    x = dev(update_like(np.random.default_rng(shape), min(2, shape[0]), *shape[1:]))
    x = x.repeat(-(-shape[0] // 2), 1, 1)[:shape[0]].contiguous()
    out = run(x, "f32")
    for _ in range(3):
        assert (run(x, "f32") == out).all()
    for i in range(2, shape[0]):
        assert (out[i] == out[i % 2]).all()
    for i in range(min(2, shape[0])):
        check(out[i].double().cpu().numpy(), x[i].double().cpu().numpy(), 5, U32)


def test_a_skipped_step_of_clusters():
    import torch
    tensors = step_case([(3, 64, 1100), (2000, 9), (2, 100, 600), (700, 300)], "f32", 31)
    plan, params = moe.muon_tensors(tensors), moe.make_muon(0.02)
    ws = moe.muon_workspace(plan)
    skip = torch.ones(1, dtype=torch.int32, device="cuda")
    before = numbers(tensors)
    for _ in range(3):
        moe.moe_muon_step(plan, params, None, skip, ws)
    for b, a in zip(before, numbers(tensors)):
        assert all((a[k] == b[k]).all() for k in ("p", "m", "p16"))
    skip.zero_()
    moe.moe_muon_step(plan, params, None, skip, ws)
    check_step(before, numbers(tensors), 0.02, np.float64(np.float32(0.95)), True, 5, 1.0)
    assert moe.moe_get_device_error(ws) == 0
