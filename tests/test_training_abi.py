"""The training calls refuse bad arguments on the host, before any launch."""
import ctypes

import pytest

import sparse_mixture_experts_topk_gb300 as moe

A = 1 << 20          # an aligned address that is never read


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sparse_mixture_experts_topk_gb300 import build
    build.build()


def code(f, *args, **kw):
    with pytest.raises(moe.MoeError) as e:
        f(*args, **kw)
    return e.value.code


def desc(T=4, H=64, E=4, K=2, F=32, **kw):
    return moe.make_desc(T, H, E, K, F, **kw)


def test_combine_backward_refuses():
    f = moe.moe_combine_backward
    ok = dict(dout=A, y_perm=A, pos=A, w=A, dy_perm=A, dw=A)
    for name in ("dout", "pos", "w", "y_perm"):
        assert code(f, desc(), **{**ok, name: None}, stream=0) == moe.MOE_ERR_INVALID
    for name in ("dout", "y_perm", "dy_perm"):
        assert code(f, desc(), **{**ok, name: A + 8}, stream=0) == moe.MOE_ERR_INVALID
    assert code(f, desc(), **{**ok, "dy_perm": None, "dw": None}, stream=0) == moe.MOE_ERR_INVALID
    assert code(f, desc(H=60), **ok, stream=0) == moe.MOE_ERR_INVALID
    f(desc(T=0), None, None, None, None, None, None, stream=0)     # no token: nothing to do


def test_dispatch_backward_refuses():
    f = moe.moe_dispatch_backward
    ok = dict(dx_perm=A, pos=A, dx_add=A, dx=A)
    for name in ("dx_perm", "pos", "dx"):
        assert code(f, desc(), **{**ok, name: None}, stream=0) == moe.MOE_ERR_INVALID
    for name in ("dx_perm", "dx_add", "dx"):
        assert code(f, desc(), **{**ok, name: A + 4}, stream=0) == moe.MOE_ERR_INVALID
    assert code(f, desc(E=300), **ok, stream=0) == moe.MOE_ERR_INVALID
    f(desc(T=0), None, None, None, None, stream=0)


class Ws(int):
    """An address with a size, as a workspace tensor has."""

    def __new__(cls, at, n):
        w = int.__new__(cls, at)
        w.n = n
        return w

    def numel(self):
        return self.n


def test_expert_ffn_backward_refuses():
    f = moe.moe_expert_ffn_backward
    d = desc()
    n = moe.moe_backward_workspace_size(d)
    assert n >= 8 * 32 * 2
    names = ("x_perm", "h_perm", "dy_perm", "offs", "W1", "b1", "W2", "dx_perm", "dW1", "db1", "dW2", "db2")
    ok = dict.fromkeys(names, A)
    ws = Ws(A, n)
    for name in ("x_perm", "h_perm", "dy_perm", "offs", "W1", "W2"):
        assert code(f, d, **{**ok, name: None}, ws=ws, stream=0) == moe.MOE_ERR_INVALID, name
    for name in ("x_perm", "h_perm", "dy_perm", "W1", "W2", "dx_perm", "dW1", "dW2"):
        assert code(f, d, **{**ok, name: A + 2}, ws=ws, stream=0) == moe.MOE_ERR_INVALID, name
    none = dict.fromkeys(("dx_perm", "dW1", "db1", "dW2", "db2"))
    assert code(f, d, **{**ok, **none}, ws=ws, stream=0) == moe.MOE_ERR_INVALID
    for bad in (None, Ws(A, n - 1), Ws(A + 128, n)):
        assert code(f, d, **ok, ws=bad, stream=0) == moe.MOE_ERR_WORKSPACE
    assert code(f, desc(F=20), **ok, ws=ws, stream=0) == moe.MOE_ERR_INVALID
    assert code(moe.moe_backward_workspace_size, desc(F=20)) == moe.MOE_ERR_INVALID


def test_adamw_refuses():
    def call(count=1, gdt=moe.MOE_F32, bits=32, params=None, **kw):
        t = dict(p=A, p_bf16=None, grad=A, m=A, v=A, m_scale=None, v_scale=None, n=8, weight_decay=0.0, reserved=0)
        t.update(kw)
        arr = (moe.MoeAdamwTensor * 1)(moe.MoeAdamwTensor(**t))
        h = moe.make_adamw(1e-3) if params is None else params
        return moe.lib().moe_adamw_step(arr, count, gdt, bits, ctypes.byref(h), None, None, None)

    bad = moe.MOE_ERR_INVALID
    for name in ("p", "grad", "m", "v"):
        assert call(**{name: None}) == bad, name
        assert call(**{name: A + 1}) == bad, name
    assert call(p_bf16=A + 1) == bad and call(grad=A + 2) == bad
    assert call(m_scale=A) == bad and call(v_scale=A) == bad              # scales without 8-bit moments
    assert call(bits=8) == bad and call(bits=8, m_scale=A) == bad         # 8-bit moments without scales
    assert call(bits=8, m_scale=A, v_scale=A + 2) == bad
    assert call(bits=16) == bad and call(gdt=7) == bad
    assert call(n=-1) == bad and call(reserved=1) == bad and call(count=-1) == bad
    assert call(weight_decay=float("nan")) == bad and call(weight_decay=float("inf")) == bad
    assert call(n=(moe.MOE_ADAMW_BLOCK << 31) + 1) == moe.MOE_ERR_UNSUPPORTED
    for kw in (dict(lr=-1), dict(lr=float("nan")), dict(lr=float("inf")), dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.0),
               dict(beta2=float("nan")), dict(eps=-1e-8), dict(eps=float("inf")), dict(step=0)):
        assert call(params=moe.make_adamw(**{"lr": 1e-3, **kw})) == bad, kw
    assert call(n=0, p=None, grad=None, m=None, v=None) == moe.MOE_OK     # an empty tensor
    assert moe.lib().moe_adamw_step(None, 0, 0, 32, ctypes.byref(moe.make_adamw(1e-3)), None, None, None) == moe.MOE_OK
    assert moe.lib().moe_adamw_step(None, 1, 0, 32, ctypes.byref(moe.make_adamw(1e-3)), None, None, None) == bad
    assert moe.lib().moe_adamw_step((moe.MoeAdamwTensor * 1)(), 1, 0, 32, None, None, None, None) == bad


def test_adamw_tensors_refuses_what_does_not_fit():
    torch = pytest.importorskip("torch")

    def t(n, dtype=torch.float32):
        return torch.zeros(n, dtype=dtype)

    good = dict(p=t(8), g=t(8), m=t(8), v=t(8))
    for change in (dict(p=t(8, torch.bfloat16)), dict(g=t(8, torch.float16)), dict(m=t(8, torch.float8_e4m3fn)),
                   dict(g=t(7)), dict(m_scale=t(1)), dict(p16=t(8)), dict(lr=1.0),
                   dict(m=t(8, torch.float8_e4m3fn), v=t(8, torch.float8_e4m3fn)),
                   dict(m=t(8, torch.float8_e4m3fn), v=t(8, torch.float8_e4m3fn), m_scale=t(2), v_scale=t(1)),
                   {}):      # the last: tensors that are not on a GPU
        with pytest.raises(ValueError):
            moe.adamw_tensors([{**good, **change}])
    assert moe.adamw_tensors([]).count == 0


def test_struct_sizes_match_the_header():
    assert ctypes.sizeof(moe.MoeAdamwTensor) == 72 and ctypes.sizeof(moe.MoeAdamwParams) == 40
