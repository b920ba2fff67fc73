"""What the AdamW step's Python side holds and refuses.  No step is launched:
CPU tensors that say they are on a GPU stand in for device tensors."""
import gc
import weakref

import pytest

import sparse_mixture_experts_topk_gb300 as moe

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sparse_mixture_experts_topk_gb300 import build
    build.build()


class OnDevice(torch.Tensor):
    is_cuda = True


def t(n, dtype=torch.float32):
    return torch.zeros(n, dtype=dtype).as_subclass(OnDevice)


@pytest.mark.parametrize("bits", [32, 8])
def test_a_description_keeps_its_tensors(bits):
    """The addresses are read once, so the tensors they belong to live as long
    as the description, whatever becomes of the caller's dicts."""
    st = torch.float32 if bits == 32 else torch.float8_e4m3fn
    d = dict(p=t(300), p16=t(300, torch.bfloat16), g=t(300), m=t(300, st), v=t(300, st))
    if bits == 8:
        d.update(m_scale=t(2), v_scale=t(2))
    alive = {k: weakref.ref(x) for k, x in d.items()}
    at = {k: x.data_ptr() for k, x in d.items()}
    plan = moe.adamw_tensors([d])
    for k in list(d):
        d[k] = None
    gc.collect()
    for k, ref in alive.items():
        assert ref() is not None and ref().data_ptr() == at[k], k
    a = plan.array[0]
    assert (a.p, a.p_bf16, a.grad, a.m, a.v) == tuple(at[k] for k in ("p", "p16", "g", "m", "v"))
    del plan, a
    gc.collect()
    assert all(ref() is None for ref in alive.values())     # and no longer


def test_the_steps_two_scalars_are_what_the_kernel_reads():
    """The kernel reads four bytes of each: a factor in fp32, a flag in int32,
    on the device.  (With no tensor in the description the call launches nothing.)"""
    plan, params = moe.adamw_tensors([]), moe.make_adamw(1e-3)
    scale, skip = t(1), t(1, torch.int32)
    for ok in ((None, None), (scale, None), (None, skip), (scale, skip), (scale[0], skip[0]), (1 << 20, 1 << 20)):
        moe.moe_adamw_step(plan, params, *ok, stream=0)
    for bad in (t(1, torch.bfloat16), t(1, torch.float64), t(1, torch.int32), t(2), t(0), torch.zeros(1)):
        with pytest.raises(ValueError, match="grad_scale"):
            moe.moe_adamw_step(plan, params, bad, skip, stream=0)
    for bad in (t(1, torch.bool), t(1, torch.int64), t(1, torch.uint8), t(1), t(2, torch.int32), t(0, torch.int32),
                torch.zeros(1, dtype=torch.int32)):
        with pytest.raises(ValueError, match="skip"):
            moe.moe_adamw_step(plan, params, scale, bad, stream=0)
