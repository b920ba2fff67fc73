"""The training calls of the router and the matrices together, as a program
runs them: on a stream of its own, captured and replayed, two at a time, after
a call that was skipped, and in the example."""
import numpy as np
import pytest

import sparse_mixture_experts_topk_gb300 as moe

pytestmark = pytest.mark.gpu


def t_():
    import torch
    return torch


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sparse_mixture_experts_topk_gb300 import build
    build.build()


class Step:
    """Router forward, balance loss, its gradient and a Muon step of the gate's
    and the experts' matrices, with buffers of its own."""

    def __init__(self, seed, T=300, H=264, E=12, K=2, F=200, dtype="bf16"):
        t = t_()
        g = t.Generator(device="cuda").manual_seed(seed)
        dt = t.bfloat16 if dtype == "bf16" else t.float32

        def rand(*shape, scale=1.0, to=t.float32):
            return (t.randn(shape, generator=g, device="cuda") * scale).to(to)

        f32, i32 = dict(device="cuda"), dict(dtype=t.int32, device="cuda")
        self.d = moe.make_desc(T, H, E, K, F, dtype=moe.MOE_BF16 if dtype == "bf16" else moe.MOE_F32)
        self.x, self.Wg, self.dw = rand(T, H, to=dt), rand(E, H, scale=0.1, to=dt), rand(T, K, scale=1.0 / T)
        self.mask = t.rand(T, generator=g, device="cuda") < 0.8
        self.ws, self.rws = moe.workspace(self.d), moe.router_backward_workspace(self.d)
        self.logits, self.w = t.zeros(T, E, **f32), t.zeros(T, K, **f32)
        self.ids = t.zeros(T, K, **i32)
        self.psum, self.count = t.zeros(E, **f32), t.zeros(E, **i32)
        self.tokens, self.loss = t.zeros(1, **i32), t.zeros(1, **f32)
        self.dloss = t.full((1,), 0.01, **f32)
        self.dWg, self.dbias, self.dx = t.zeros(E, H, **f32), t.zeros(E, **f32), t.zeros(T, H, dtype=dt, device="cuda")
        self.p = [rand(E, H, scale=0.02), rand(E, F, H, scale=0.02), rand(E, H, F, scale=0.02)]
        self.g = [self.dWg, rand(E, F, H), rand(E, H, F)]
        self.m = [t.zeros_like(p) for p in self.p]
        self.p16 = [t.zeros_like(p, dtype=t.bfloat16) for p in self.p]
        self.plan = moe.muon_tensors([{"p": p, "g": q, "m": m, "p16": c, "weight_decay": 0.1}
                                      for p, q, m, c in zip(self.p, self.g, self.m, self.p16)])
        self.mws = moe.muon_workspace(self.plan)
        self.params = moe.make_muon(0.01)

    def run(self, stream=None):
        d = self.d
        moe.moe_router_topk(d, self.x, self.Wg, None, self.logits, self.ids, self.w, None, self.ws, stream)
        moe.moe_balance_loss(d, self.logits, self.ids, self.mask, self.psum, self.count, self.tokens, self.loss,
                             self.rws, stream)
        moe.moe_router_backward(d, self.x, self.Wg, self.logits, self.ids, self.dw, self.dloss, self.count,
                                self.tokens, self.mask, None, self.dWg, self.dbias, self.dx, self.rws, stream)
        moe.moe_muon_step(self.plan, self.params, None, None, self.mws, stream)

    def results(self):
        t_().cuda.synchronize()
        assert moe.moe_get_device_error(self.rws) == 0 and moe.moe_get_device_error(self.mws) == 0
        return [v.clone() for v in [self.psum, self.count, self.tokens, self.loss, self.dWg, self.dbias, self.dx]
                + self.p + self.m + self.p16]


def same(a, b):
    return all((x == y).all() for x, y in zip(a, b))


def eager(seed, times=1, **kw):
    s = Step(seed, **kw)
    for _ in range(times):
        s.run()
    return s.results()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_captured_steps_replay_to_the_eager_bits(dtype):
    t = t_()
    want = eager(1, 3, dtype=dtype)
    s = Step(1, dtype=dtype)
    graph = t.cuda.CUDAGraph()
    t.cuda.synchronize()
    with t.cuda.graph(graph):
        s.run()
    for _ in range(3):
        graph.replay()
    assert same(s.results(), want)


def test_two_graphs_side_by_side():
    """Each with its own workspaces, replayed on two streams at once."""
    t = t_()
    want = [eager(2, 4), eager(3, 4, H=392, E=40)]
    steps = [Step(2), Step(3, H=392, E=40)]
    graphs, streams = [t.cuda.CUDAGraph() for _ in steps], [t.cuda.Stream() for _ in steps]
    t.cuda.synchronize()
    for s, g in zip(steps, graphs):
        with t.cuda.graph(g):
            s.run()
    t.cuda.synchronize()
    for _ in range(4):
        for g, st in zip(graphs, streams):
            with t.cuda.stream(st):
                g.replay()
    t.cuda.synchronize()
    for s, w in zip(steps, want):
        assert same(s.results(), w)


def test_a_stream_given_and_two_streams_at_once():
    t = t_()
    want = [eager(4), eager(5, T=1000)]
    steps, streams = [Step(4), Step(5, T=1000)], [t.cuda.Stream() for _ in range(2)]
    t.cuda.synchronize()
    for s, st in zip(steps, streams):
        s.run(st)
    t.cuda.synchronize()
    for s, w in zip(steps, want):
        assert same(s.results(), w)


def test_two_steps_that_fill_the_gpu_at_once():
    """Either call has tiles for more CTAs than the GPU holds, beside the other's: none may wait for a CTA that
    finds no room."""
    t = t_()

    def tensors(seed):
        g = t.Generator(device="cuda").manual_seed(seed)
        p = [t.randn(s, generator=g, device="cuda") * 0.02 for s in ((24, 520, 776), (24, 776, 520))]
        return [{"p": q, "g": t.randn(q.shape, generator=g, device="cuda"), "m": t.zeros_like(q)} for q in p]

    def results(ts):
        t.cuda.synchronize()
        return [v.clone() for d in ts for v in (d["p"], d["m"])]

    def plan(ts):
        p = moe.muon_tensors(ts)
        return p, moe.muon_workspace(p)

    params, want = moe.make_muon(0.01), []
    for seed in (1, 2):
        ts = tensors(seed)
        p, ws = plan(ts)
        for _ in range(10):
            moe.moe_muon_step(p, params, None, None, ws)
        want.append(results(ts))
    both = [tensors(1), tensors(2)]
    plans, streams = [plan(ts) for ts in both], [t.cuda.Stream() for _ in both]
    t.cuda.synchronize()
    for _ in range(10):
        for (p, ws), st in zip(plans, streams):
            moe.moe_muon_step(p, params, None, None, ws, st)
    for ts, w in zip(both, want):
        assert same(results(ts), w)
    assert all(moe.moe_get_device_error(ws) == 0 for _, ws in plans)


def test_captured_step_of_every_kind_of_matrix():
    """Two sizes of tensor-core batches, one with guessed norms, small matrices by one and by several CTAs and thin
    ones, which start beside those: replayed as in a loop of eager calls, alone and with another call behind it."""
    t = t_()

    def tensors():
        g = t.Generator(device="cuda").manual_seed(5)
        shapes = [(8, 200), (12, 1024, 800), (5, 64, 96), (2, 300, 500), (4096, 100), (3, 700, 16), (1, 1), (500, 300)]
        p = [t.randn(s, generator=g, device="cuda") * 0.02 for s in shapes]
        return [{"p": q, "g": t.randn(q.shape, generator=g, device="cuda"), "m": t.zeros_like(q)} for q in p]

    def results(ts):
        t.cuda.synchronize()
        return [v.clone() for d in ts for v in (d["p"], d["m"])]

    params = moe.make_muon(0.02)
    eager_ts = tensors()
    plan = moe.muon_tensors(eager_ts)
    ws = moe.muon_workspace(plan)
    for _ in range(6):
        moe.moe_muon_step(plan, params, None, None, ws)
    want = results(eager_ts)
    ts = tensors()
    plan2 = moe.muon_tensors(ts)
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        moe.moe_muon_step(plan2, params, None, None, ws)
        moe.moe_muon_step(plan2, params, None, None, ws)
    for _ in range(3):
        graph.replay()
    for got, w in zip(results(ts), want):
        assert (got == w).all()
    assert moe.moe_get_device_error(ws) == 0


def test_a_workspace_serves_calls_of_all_sizes_in_turn():
    """One workspace as large as the largest call's: what one call leaves in it does not reach the next."""
    big, small = Step(6, T=2000, H=520, E=64, F=320), Step(7, T=17, H=72, E=5, F=40)
    want = [eager(6, 2, T=2000, H=520, E=64, F=320), eager(7, 2, T=17, H=72, E=5, F=40)]
    small.rws, small.mws = big.rws, big.mws
    for _ in range(2):
        big.run()
        small.run()
    assert same(big.results(), want[0]) and same(small.results(), want[1])


def test_a_skipped_step_leaves_the_next_one_right():
    t = t_()
    want = eager(8)
    s = Step(8)
    moe.moe_muon_step(s.plan, s.params, None, t.ones(1, dtype=t.int32, device="cuda"), s.mws)
    s.run()
    assert same(s.results(), want)


def test_gradient_of_the_loss_ends_in_its_descent():
    """The scores moved a little against the balance loss' gradient alone lower the loss by |dl|^2 times the step,
    to first order (counts as they were)."""
    t = t_()
    s = Step(9, T=512, E=16)
    s.run()
    dl = t.empty_like(s.logits)
    moe.moe_router_backward(s.d, None, None, s.logits, s.ids, None, s.dloss, s.count, s.tokens, s.mask, dl, None, None,
                            None, s.rws)
    p = t.softmax(s.logits.double(), 1)[s.mask]
    q = t.softmax(s.logits.double() - 1e-3 * dl.double() / dl.double().norm(), 1)[s.mask]
    n = float(s.tokens)
    f = s.count.double() * 16 / (n * 2) / n * 0.01
    drop = ((p - q) @ f).sum().item()
    want = 1e-3 * dl.double().norm().item()
    # second order: |step|^2 / 2 times a curvature of at most max f
    assert abs(drop - want) <= 1e-6 * f.max().item() + 1e-4 * want


@pytest.mark.parametrize("optimiser", ["adamw", "muon"])
def test_example_runs(optimiser):
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "train_layer.py")
    spec = importlib.util.spec_from_file_location("train_layer", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    first, last = m.train(steps=3, T=64, H=64, E=4, K=2, F=96, optimiser=optimiser, balance=0.01, log=lambda *_: None)
    assert np.isfinite(first) and np.isfinite(last)
