"""What a GateTrainer keeps from call to call: its workspaces over changing batches, captures
and streams."""

import pytest
import torch

import routing_dispatch_expert_softmax_b200 as moe
from routing_dispatch_expert_softmax_b200 import workloads as wl

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    moe.load_library()
    yield
    torch.cuda.synchronize()


@pytest.fixture(scope="module")
def made():
    cfg = wl.TINY.with_T(300)
    t = wl.make_layer(cfg, DEV, 4)
    return cfg, t, moe.MoELayer(t["w_g"], t["bias"], t["w13"], t["w2"], cfg.k)


def offsets(T, S):
    return torch.linspace(0, T, S + 1, device=DEV).int()


def step(tr, x, dy, seqs=None):
    y = tr(x, seq_offsets=seqs)
    g = tr.backward(dy, dx=True, max_norm=1.0)
    return [t.clone() for t in (y, tr.loss, tr.counts, tr.tokens, tr.prob_mean, g.dw_g, g.dbias, g.dx, g.norm)
            if t is not None]


def same(a, b):
    return len(a) == len(b) and all(torch.equal(p, q) for p, q in zip(a, b))


def test_changing_batches_do_not_pile_up(made):
    cfg, t, layer = made
    tr = moe.GateTrainer(layer, z_coef=1e-3)
    dy = torch.randn(300, cfg.d, device=DEV).bfloat16()
    cases = [(T, S) for T in (300, 17, 299, 64, 201) for S in (1, 40, 7, 3, 12)]
    step(tr, t["x"], dy, offsets(300, 40))  # the largest of both
    held = None
    for T, S in cases:
        seqs = offsets(T, S) if S > 1 else None
        got = step(tr, t["x"][:T], dy[:T], seqs)
        want = step(moe.GateTrainer(layer, z_coef=1e-3), t["x"][:T], dy[:T], seqs)
        assert same(got, want), (T, S)
        assert tr.check() == moe.MOE_OK
        del got, want
        tr(t["x"][:1])  # the kept step's tensors are small
        tr.loss = None
        torch.cuda.synchronize()
        now = torch.cuda.memory_allocated()
        held = now if held is None else held
        assert now <= held + (1 << 16), (T, S, now - held)


def test_error_word_outlives_a_larger_workspace(made):
    cfg, t, layer = made
    tr = moe.GateTrainer(layer)
    bad = torch.tensor([0, 9], dtype=torch.int32, device=DEV)  # behind the last token
    tr(t["x"][:4], seq_offsets=bad)
    tr(t["x"])
    assert tr.check() == moe.MOE_ERR_DEVICE_CHECK
    assert tr.check() == moe.MOE_OK


def capture(tr, x, dy, seqs):
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = tr(x, seq_offsets=seqs)
        g = tr.backward(dy, dx=True, max_norm=1.0)
    return graph, [t for t in (y, tr.loss, tr.counts, tr.tokens, tr.prob_mean, g.dw_g, g.dbias, g.dx, g.norm)
                   if t is not None]


def test_first_call_under_capture(made):
    # the capture's own workspaces are set up by its replays, and eager calls have others
    cfg, t, layer = made
    x, dy = t["x"][:200].clone(), torch.randn(200, cfg.d, device=DEV).bfloat16()
    seqs = offsets(200, 5)  # as long as the graph, like x and dy
    want = step(moe.GateTrainer(layer), x, dy, seqs)
    tr = moe.GateTrainer(layer)
    graph, out = capture(tr, x, dy, seqs)
    assert same(step(tr, x, dy, seqs), want)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert same(out, want)
    assert same(step(tr, x, dy, seqs), want)
    del graph, out
    torch.cuda.empty_cache()
    assert same(step(tr, x, dy, seqs), want) and tr.check() == moe.MOE_OK


def test_two_captures_of_one_trainer_beside_each_other(made):
    cfg, t, layer = made
    xs = [t["x"].clone(), torch.randn(300, cfg.d, device=DEV).bfloat16()]
    dy, seqs = torch.randn(300, cfg.d, device=DEV).bfloat16(), offsets(300, 6)
    tr = moe.GateTrainer(layer, z_coef=1e-3)
    want = [step(tr, x, dy, seqs) for x in xs]
    made_graphs = [capture(tr, x, dy, seqs) for x in xs]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, (graph, _) in zip(streams, made_graphs):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for (_, out), w in zip(made_graphs, want):
        assert same(out, w)
    assert same(step(tr, xs[1], dy, seqs), want[1])


def test_clipping_several_layers_by_one_norm(made):
    cfg, t, layer = made
    dy = torch.randn(300, cfg.d, device=DEV).bfloat16()
    grads = []
    for seed in range(3):
        u = wl.make_layer(cfg, DEV, 10 + seed)
        tr = moe.GateTrainer(moe.MoELayer(u["w_g"], u["bias"], u["w13"], u["w2"], cfg.k))
        tr(u["x"])
        g = tr.backward(dy)
        grads += [v for v in (g.dw_g, g.dbias) if v is not None]
    whole = [g.clone() for g in grads]
    norm = torch.empty(1, device=DEV)
    moe.moe_clip_grads(grads, 0.25, norm)
    want = sum(float(g.double().square().sum()) for g in whole) ** 0.5
    assert want > 0.25 and abs(norm.item() - want) <= 1e-6 * want
    for g, w in zip(grads, whole):
        assert torch.allclose(g.double(), w.double() * (0.25 / (want + 1e-6)), rtol=1e-6, atol=0)
