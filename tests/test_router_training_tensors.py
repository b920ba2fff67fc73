"""moe_balance_loss and moe_router_backward read tensors of a program's making:
another type than the call reads, too few values, values that do not lie one
after the other or that the GPU does not reach are refused before the call."""
import pytest

import sparse_mixture_experts_topk_gb300 as moe

torch = pytest.importorskip("torch")

A = 1 << 20          # an aligned address that is never read
T, H, E, K = 6, 64, 8, 2


class Ws(int):
    def numel(self):
        return 0         # whatever passes the checks of the tensors ends here


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sparse_mixture_experts_topk_gb300 import build
    build.build()


class Gpu:
    """What the binding asks a tensor, with the answers of one on a GPU: there is none to run on."""

    def __init__(self, t, contiguous=True, cuda=True, pinned=False):
        self.t, self.contiguous, self.is_cuda, self.pinned = t, contiguous, cuda, pinned

    dtype = property(lambda self: self.t.dtype)
    numel = property(lambda self: self.t.numel)
    element_size = property(lambda self: self.t.element_size)

    def is_contiguous(self):
        return self.contiguous

    def is_pinned(self):
        return self.pinned

    def data_ptr(self):
        return A


def shapes(dtype):
    f, i, d = torch.float32, torch.int32, dtype
    return {"x": (T * H, d), "Wg": (E * H, d), "logits": (T * E, f), "ids": (T * K, i), "mask": (T, torch.bool),
            "dw": (T * K, f), "dloss": (1, f), "count": (E, i), "tokens": (1, i), "psum": (E, f), "loss": (1, f),
            "dlogits": (T * E, f), "dWg": (E * H, f), "dgate_bias": (E, f), "dx": (T * H, d)}


CALLS = {"moe_balance_loss": ("logits", "ids", "mask", "psum", "count", "tokens", "loss"),
         "moe_router_backward": ("x", "Wg", "logits", "ids", "dw", "dloss", "count", "tokens", "mask", "dlogits", "dWg",
                                 "dgate_bias", "dx")}
READ = {"moe_balance_loss": CALLS["moe_balance_loss"][:3], "moe_router_backward": CALLS["moe_router_backward"][:9]}
CASES = [(f, name) for f, names in READ.items() for name in names]


def call(f, dtype=torch.bfloat16, **changed):
    d = moe.make_desc(T, H, E, K, 8, dtype=moe.MOE_BF16 if dtype == torch.bfloat16 else moe.MOE_F32)
    args = {n: Gpu(torch.zeros(s, dtype=dt)) for n, (s, dt) in shapes(dtype).items() if n in CALLS[f]}
    args.update(changed)
    with pytest.raises((ValueError, moe.MoeError)) as e:
        getattr(moe, f)(d, **args, ws=Ws(A), stream=0)
    return e.value


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("f,name", CASES)
def test_a_tensor_that_the_call_would_misread_is_refused(f, name, dtype):
    n, dt = shapes(dtype)[name]

    def refused(t):
        e = call(f, dtype, **{name: t})
        return isinstance(e, ValueError) and f in str(e) and name in str(e)

    others = [torch.int64, torch.float64, torch.float16]
    if name != "mask":
        others += [t for t in (torch.float32, torch.int32, torch.bfloat16, torch.bool) if t != dt]
    for other in others:
        assert refused(Gpu(torch.zeros(n, dtype=other))), other
    assert refused(Gpu(torch.zeros(n - 1, dtype=dt)))
    assert refused(Gpu(torch.zeros(n, dtype=dt), contiguous=False))
    assert refused(Gpu(torch.zeros(n, dtype=dt), cuda=False))
    assert refused(torch.zeros(n, dtype=dt))
    assert refused(torch.zeros(2 * n, dtype=dt)[::2])


@pytest.mark.parametrize("f,name", CASES)
def test_what_the_call_can_take_is_taken(f, name):
    """Longer buffers (but for the mask), values in pinned memory, addresses, and nothing: what stops the call is its
    workspace or what it cannot do without."""
    n, dt = shapes(torch.bfloat16)[name]
    taken = [Gpu(torch.zeros(n, dtype=dt)), Gpu(torch.zeros(n, dtype=dt), cuda=False, pinned=True), A, None]
    if name == "mask":
        taken += [Gpu(torch.zeros(n, dtype=torch.uint8))]
    else:
        taken += [Gpu(torch.zeros(n + 3, dtype=dt))]
    for t in taken:
        e = call(f, **{name: t})
        assert isinstance(e, moe.MoeError) and e.code == moe.MOE_ERR_WORKSPACE, (name, t)
