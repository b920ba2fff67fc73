"""The balance loss and the router's gradient where their work is shared out
unevenly: clusters with blocks that have no expert."""
import numpy as np
import pytest

import sparse_mixture_experts_topk_gb300 as moe

from test_gpu_router_backward import U32, case, oracle, t_

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sparse_mixture_experts_topk_gb300 import build
    build.build()


@pytest.mark.parametrize("mask", [False, True])
@pytest.mark.parametrize("E", [33, 65, 97, 129, 161])
def test_balance_loss_of_clusters_with_blocks_without_experts(E, mask):
    T, K = 5000, 3
    c = case(T, 8, E, K, mask=mask, seed=21)
    t, q, ref = t_(), c["t"], oracle(c, False, False)
    ws = moe.router_backward_workspace(c["desc"])
    for _ in range(20):
        psum, loss = t.full((E,), 7.0, device="cuda"), t.full((1,), 7.0, device="cuda")
        count, tokens = t.full((E,), 7, dtype=t.int32, device="cuda"), t.full((1,), 7, dtype=t.int32, device="cuda")
        moe.moe_balance_loss(c["desc"], q["logits"], q["ids"], q["mask"], psum, count, tokens, loss, ws)
        assert (count.cpu().numpy() == c["count"]).all() and tokens.item() == c["tokens"]
        # as in test_balance_loss
        u = (64 + 4 * abs(c["n"]["logits"]).max() + T) * U32
        assert (abs(psum.double().cpu().numpy() - ref["psum"]) <= u * ref["psum"] + 1e-37).all()
        assert abs(loss.item() - ref["loss"]) <= (u + 4 * U32) * ref["loss"]
    assert moe.moe_get_device_error(ws) == 0
