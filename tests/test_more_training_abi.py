"""The balance loss, the router's gradient, the orthogonalisation and the Muon
step refuse bad arguments on the host, before any launch."""
import ctypes

import pytest

import sparse_mixture_experts_topk_gb300 as moe

A = 1 << 20          # an aligned address that is never read


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sparse_mixture_experts_topk_gb300 import build
    build.build()


class Ws(int):
    """An address with a size, as a workspace tensor has."""

    def __new__(cls, at, n):
        w = int.__new__(cls, at)
        w.n = n
        return w

    def numel(self):
        return self.n


def code(f, *args, **kw):
    with pytest.raises(moe.MoeError) as e:
        f(*args, **kw)
    return e.value.code


def desc(T=4, H=64, E=4, K=2, **kw):
    return moe.make_desc(T, H, E, K, 8, **kw)


def test_balance_loss_refuses():
    f, d = moe.moe_balance_loss, desc()
    ws = Ws(A, moe.moe_router_backward_workspace_size(d))
    ok = dict(logits=A, ids=A, mask=A, psum=A, count=A, tokens=A, loss=A, ws=ws, stream=0)
    for name in ("logits", "ids"):
        assert code(f, d, **{**ok, name: None}) == moe.MOE_ERR_INVALID
    assert code(f, d, **{**ok, "psum": None, "count": None, "tokens": None, "loss": None}) == moe.MOE_ERR_INVALID
    assert code(f, d, **{**ok, "logits": A + 4}) == moe.MOE_ERR_INVALID
    for name in ("ids", "psum", "count", "tokens", "loss"):
        assert code(f, d, **{**ok, name: A + 2}) == moe.MOE_ERR_INVALID
    for bad in (None, Ws(A + 16, 1 << 20), Ws(A, ws.n - 1)):
        assert code(f, d, **{**ok, "ws": bad}) == moe.MOE_ERR_WORKSPACE
    assert code(f, desc(E=257), **ok) == moe.MOE_ERR_INVALID


def test_router_backward_refuses():
    f, d = moe.moe_router_backward, desc()
    ws = Ws(A, moe.moe_router_backward_workspace_size(d))
    ok = dict(x=A, Wg=A, logits=A, ids=A, dw=A, dloss=A, count=A, tokens=A, mask=A, dlogits=A, dWg=A, dgate_bias=A,
              dx=A, ws=ws, stream=0)
    for name in ("x", "Wg", "logits", "ids", "count", "tokens"):
        assert code(f, d, **{**ok, name: None}) == moe.MOE_ERR_INVALID, name
    assert code(f, d, **{**ok, "dlogits": None, "dWg": None, "dgate_bias": None, "dx": None}) == moe.MOE_ERR_INVALID
    for name in ("x", "Wg", "logits", "dlogits", "dWg", "dx"):
        assert code(f, d, **{**ok, name: A + 8}) == moe.MOE_ERR_INVALID, name
    for name in ("ids", "dw", "dloss", "count", "tokens", "dgate_bias"):
        assert code(f, d, **{**ok, name: A + 2}) == moe.MOE_ERR_INVALID, name
    for bad in (None, Ws(A + 16, 1 << 30), Ws(A, ws.n - 1)):
        assert code(f, d, **{**ok, "ws": bad}) == moe.MOE_ERR_WORKSPACE
    assert code(f, desc(H=60), **ok) == moe.MOE_ERR_INVALID
    with pytest.raises(moe.MoeError):
        moe.moe_router_backward_workspace_size(desc(K=9, E=16))


def test_a_mask_is_a_byte_for_each_token():
    import torch
    d = desc(T=4)
    ws = Ws(A, moe.moe_router_backward_workspace_size(d))
    for bad in (torch.ones(4), torch.ones(4, dtype=torch.int32), torch.ones(5, dtype=torch.bool)):
        with pytest.raises(ValueError):
            moe.moe_balance_loss(d, A, A, bad, A, A, A, A, ws, 0)
        with pytest.raises(ValueError):
            moe.moe_router_backward(d, A, A, A, A, A, A, A, A, bad, A, A, A, A, ws, 0)


def test_orthogonalize_refuses():
    f = moe.lib().moe_orthogonalize
    n = moe.moe_orthogonalize_workspace_size(2, 30, 40)

    def call(x=A, xd=moe.MOE_F32, batch=2, rows=30, cols=40, it=5, out=A, od=moe.MOE_F32, ws=A, nbytes=n):
        return f(x, xd, batch, rows, cols, it, out, od, ws, nbytes, None)

    for kw in (dict(x=None), dict(out=None), dict(xd=2), dict(od=-1), dict(batch=-1), dict(rows=-1), dict(cols=-2),
               dict(it=0), dict(it=17), dict(x=A + 2), dict(out=A + 2), dict(xd=moe.MOE_BF16),
               dict(out=A + 1, od=moe.MOE_BF16)):
        assert call(**kw) == moe.MOE_ERR_INVALID, kw
    for kw in (dict(ws=None), dict(ws=A + 8), dict(nbytes=n - 1), dict(rows=300, cols=300, nbytes=n)):
        assert call(**kw) == moe.MOE_ERR_WORKSPACE, kw
    for kw in (dict(rows=32769), dict(cols=1 << 20), dict(batch=1 << 24)):
        assert call(**kw) == moe.MOE_ERR_UNSUPPORTED, kw
    for kw in (dict(batch=0), dict(rows=0), dict(cols=0)):
        assert call(x=None, out=None, ws=None, nbytes=0, **kw) == moe.MOE_OK
    assert code(moe.moe_orthogonalize_workspace_size, 1, 1, 32769) == moe.MOE_ERR_UNSUPPORTED


def matrices(**kw):
    t = dict(p=A, p_bf16=A, grad=A, m=A, batch=2, rows=30, cols=40, weight_decay=0.1, scale=1.0)
    t.update(kw)
    return (moe.MoeMuonTensor * 2)(moe.MoeMuonTensor(**t), moe.MoeMuonTensor(A, None, A, A, 1, 8, 8, 0.0, 1.0))


def test_muon_step_refuses():
    L = moe.lib()
    size = ctypes.c_size_t(0)
    assert L.moe_muon_workspace_size(matrices(), 2, ctypes.byref(size)) == moe.MOE_OK
    n = size.value

    def call(t=None, count=2, gd=moe.MOE_F32, params=None, scale=None, skip=None, ws=A, nbytes=n):
        params = moe.make_muon(0.1) if params is None else params
        return L.moe_muon_step(matrices() if t is None else t, count, gd, ctypes.byref(params), scale, skip, ws, nbytes,
                               None)

    nan, inf = float("nan"), float("inf")
    for kw in (dict(p=None), dict(grad=None), dict(m=None), dict(p=A + 2), dict(grad=A + 2), dict(m=A + 1),
               dict(p_bf16=A + 1), dict(batch=-1), dict(rows=-1), dict(weight_decay=nan), dict(scale=inf),
               dict(scale=nan)):
        assert call(t=matrices(**kw)) == moe.MOE_ERR_INVALID, kw
    for p in (moe.make_muon(nan), moe.make_muon(-1.0), moe.make_muon(inf), moe.make_muon(0.1, 1.0),
              moe.make_muon(0.1, -0.1), moe.make_muon(0.1, nan), moe.make_muon(0.1, iterations=0),
              moe.make_muon(0.1, iterations=17), moe.MoeMuonParams(0.1, 0.9, 2, 5)):
        assert call(params=p) == moe.MOE_ERR_INVALID
    assert call(gd=2) == moe.MOE_ERR_INVALID and call(count=-1) == moe.MOE_ERR_INVALID
    assert call(scale=A + 2) == moe.MOE_ERR_INVALID and call(skip=A + 1) == moe.MOE_ERR_INVALID
    assert L.moe_muon_step(None, 1, 0, ctypes.byref(moe.make_muon(0.1)), None, None, A, n, None) == moe.MOE_ERR_INVALID
    assert L.moe_muon_step(matrices(), 2, 0, None, None, None, A, n, None) == moe.MOE_ERR_INVALID
    for kw in (dict(ws=None), dict(ws=A + 8), dict(nbytes=n - 1)):
        assert call(**kw) == moe.MOE_ERR_WORKSPACE, kw
    assert call(t=matrices(rows=40000)) == moe.MOE_ERR_UNSUPPORTED
    assert call(count=0, ws=None, nbytes=0) == moe.MOE_OK
    none = (moe.MoeMuonTensor * 1)(moe.MoeMuonTensor(None, None, None, None, 0, 8, 8, 0.0, 1.0))
    assert call(t=none, count=1, ws=None, nbytes=0) == moe.MOE_OK


def test_muon_tensors_refuse():
    import torch
    p = torch.zeros(4, 8)
    ok = dict(p=p, g=p, m=p)
    for bad in ({**ok, "q": p}, {**ok, "p": p.view(-1)}, {**ok, "p": p.double()}, {**ok, "g": p.half()},
                {**ok, "m": p.bfloat16()}, {**ok, "p16": p}, {**ok, "g": torch.zeros(8, 4)}, ok):   # the last: on the CPU
        with pytest.raises(ValueError):
            moe.muon_tensors([bad])
    with pytest.raises(ValueError):
        moe.moe_orthogonalize(p, p, 5, None)          # on the CPU
    with pytest.raises(ValueError):
        moe.moe_orthogonalize(p.view(-1), p.view(-1), 5, None)


def test_workspace_sizes():
    """X twice and two short matrices, in fp16, rows padded to 16 bytes, in parts of at most 4 GiB."""
    one = moe.moe_orthogonalize_workspace_size(1, 1001, 300)
    assert one == moe.moe_orthogonalize_workspace_size(1, 300, 1001)
    assert one >= 256 + 2 * 300 * 1008 * 2 + 2 * 300 * 304 * 2
    assert moe.moe_orthogonalize_workspace_size(100000, 1000, 1000) <= (4 << 30) + (1 << 20)
    # one matrix of the largest size runs, whatever it takes
    assert moe.moe_orthogonalize_workspace_size(1, 32768, 32768) >= 4 * 32768 ** 2 * 2
