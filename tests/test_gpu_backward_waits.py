"""The bounded waits of the expert gradient's tensor-core kernels."""
import time

import numpy as np
import pytest

import sparse_mixture_experts_topk_gb300 as moe

from harness import to_dev
from test_gpu_training import check_ffn, ffn_case, run_ffn, with_tail

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_mixture_experts_topk_gb300 import build
    build.build()
    moe.lib()


def second_weight_gradient(counts):
    """dW2 alone of experts with these rows, H = F = 8: (seconds, dW2, what it has
    to be, error word).  The rows are zero but for a few, at both ends of an
    expert's rows too, so that the sums are exact."""
    import torch
    E, total = len(counts), int(np.sum(counts))
    offs = np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)
    desc = moe.make_desc(total, 8, E, 1, 8)
    ws = moe.backward_workspace(desc)
    dy = torch.zeros((total, 8), dtype=torch.bfloat16, device="cuda")
    want = np.zeros((E, 8, 8))
    rng = np.random.default_rng(total)
    for e in np.flatnonzero(counts):
        n = int(counts[e])
        for r in (0, 1, n // 3, n // 2, n - 2, n - 1):
            v = rng.integers(-4, 5, 8)
            dy[int(offs[e]) + r] = torch.from_numpy(v).to("cuda", torch.bfloat16)
            want[e] += np.outer(v, v)                    # at most 6 x 16 an entry: exact in bf16
    dW2 = torch.full((E, 8, 8), float("nan"), dtype=torch.bfloat16, device="cuda")
    W = torch.zeros(8, dtype=torch.bfloat16, device="cuda")
    at = torch.from_numpy(offs.astype(np.int32)).cuda()
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    moe.moe_expert_ffn_backward(desc, dy, dy, dy, at, W, None, W, None, None, None, dW2, None, ws)
    end.record()
    end.synchronize()
    return start.elapsed_time(end) / 1e3, dW2.double().cpu().numpy(), want, moe.moe_get_device_error(ws)


def long_tile(tiles, seconds):
    """`tiles` experts of one tile each, which one SM pair computes one after
    another, `seconds` each: tiles go round the pairs by number, and with H = F =
    8 an expert's dW2 is one tile.  The total has to be longer than a wait may take."""
    import torch
    pairs = min(torch.cuda.get_device_properties(0).multi_processor_count // 2, 80)
    busy = list(range(0, 256, pairs))[:tiles]
    assert len(busy) == tiles

    def counts(rows):
        c = np.zeros(256 if tiles > 1 else 1, np.int64)
        c[busy] = rows
        return c

    few = (4 << 20) + 5
    second_weight_gradient(counts(few))                  # the first call of a process, and the clocks
    took, got, want, error = second_weight_gradient(counts(few))
    assert error == 0 and (got == want).all()
    rows = int(few * seconds / (took / tiles)) | 1
    assert tiles * rows < 2 ** 31 - 256
    took, got, want, error = second_weight_gradient(counts(rows))
    torch.cuda.empty_cache()
    assert 2.3 < took < 6.0, took
    assert (got == want).all()
    assert error == 0


def test_a_launch_may_take_longer_than_one_wait():
    """A wait may take two seconds, a launch any number of them."""
    long_tile(4, 0.8)


def test_a_tile_may_take_longer_than_two_seconds():
    """The wait for an accumulator lasts as long as its tile's reduction."""
    long_tile(1, 2.8)


@pytest.mark.parametrize("act,want", [("gelu", ("dx", "dW1", "db1", "dW2", "db2")), ("swiglu", ("db1",))])
def test_expired_wait_reports_timeout_and_context_survives(act, want):
    """The barrier of each kernel's first stage waits for an arrival that nobody
    makes: every role gives up, what is in flight lands, tensor memory is freed
    and the error word says so.  The next call, in the same workspace, is right."""
    import torch
    c = ffn_case([300, 0, 20, 129], 520, 264, act, True, "bf16", 41)     # full, short and more stages than the ring
    flags = moe.MOE_FLAG_SWIGLU if act == "swiglu" else 0
    ws = moe.backward_workspace(moe.make_desc(c["R"], c["H"], c["E"], 1, c["F"], flags=flags))
    desc = moe.make_desc(c["R"], c["H"], c["E"], 1, c["F"], flags=flags | moe.MOE_FLAG_TEST_WAIT_TIMEOUT)
    x, h, dy = (with_tail(c[k], c["R"], "bf16") for k in ("x", "h", "dy"))
    W1, b1, W2 = to_dev(c["W1"], "bf16"), to_dev(c["b1"], "f32"), to_dev(c["W2"], "bf16")
    o = dict(dx=torch.empty_like(x), dW1=torch.empty_like(W1), db1=torch.empty_like(b1), dW2=torch.empty_like(W2),
             db2=torch.empty((c["E"], c["H"]), device="cuda"))
    start = time.time()
    moe.moe_expert_ffn_backward(desc, x, h, dy, to_dev(c["offs"], "i32"), W1, b1, W2,
                                *(o[k] if k in want else None for k in o), ws)
    torch.cuda.synchronize()
    took = time.time() - start
    assert moe.moe_get_device_error(ws) == moe.MOE_ERR_TIMEOUT
    assert took < 30.0
    check_ffn(c, run_ffn(c, ws=ws))                 # the read cleared the error word
