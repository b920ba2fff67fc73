"""What the AdamW step's Python side holds and refuses.  No step is launched:
CPU tensors that say they are on a GPU stand in for device tensors."""
import gc
import weakref

import pytest

import sparse_mixture_experts_topk_gb300 as moe

torch = pytest.importorskip("torch")


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
