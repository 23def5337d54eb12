"""One training step of the gate, all calls together, against the fp64 oracle.

The step's own logits, gates and expert outputs are inputs of the oracle (the
forward calls have their own tests); what is checked is the chain dy -> dw ->
dlogits -> dw_g, dbias, dx, and that the step's forward is the layer's.

Tolerances: each stage's relative bound on its magnitudes, added up.  dw is a
sum of d products (d u), the gate's part of dlogits multiplies it by gates and
subtracts (2 dw-sized terms, (k + 8) u), the balance part is bounded like a
softmax over E values ((4.44 D + 2 E + 40) u with D < 60), and the products sum
T or E terms; the tensor cores' sums count 2 u a term, three terms a token.
dx adds its operands' rounding to fp16 (2^-10 a product) and its own (2^-8)."""

import math

import numpy as np
import pytest
import torch

import routing_dispatch_expert_softmax_b200 as moe
from oracle import gate_train_oracle as go
from routing_dispatch_expert_softmax_b200 import workloads as wl

from parity_utils import U32, assert_layer_close, np64

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    moe.load_library()
    yield
    torch.cuda.synchronize()


def make(T, seed=0, fmt="bf16", **kw):
    cfg = wl.TINY.with_T(T) if not kw else wl.MoEConfig("step", T=T, **kw)
    t = wl.make_layer(cfg, DEV, seed)
    if fmt == "bf16":
        return cfg, t, moe.MoELayer(t["w_g"], t["bias"], t["w13"], t["w2"], cfg.k)
    q = wl.make_experts_fp8(cfg, DEV, seed)
    return cfg, t, moe.MoELayer(t["w_g"], t["bias"], q[0], q[2], cfg.k, w13_scale=q[1], w2_scale=q[3],
                                fp8_activations=fmt == "w8a8")


def check_step(trainer, x, dy, g, grads, mask=None, seqs=None):
    q = trainer._kept
    L, idx, w = np64(q["logits"]), q["idx"].cpu().numpy(), np64(q["w"])
    z, row = np64(q["z"]), q["row_of"].cpu().numpy()
    T, E = L.shape
    k, d = idx.shape[1], x.shape[1]
    a, b = trainer.balance_coef, trainer.z_coef
    loss, counts, tokens, mean = go.balance_loss(L, idx, a, b, mask, seqs)
    assert np.array_equal(trainer.counts.cpu().numpy(), counts)
    assert np.array_equal(trainer.tokens.cpu().numpy(), tokens)
    rel = (4.44 * 60 + 2 * E + 40) * U32
    assert np.allclose(np64(trainer.loss), loss, rtol=4 * rel, atol=0)
    dw, dz = go.combine_bwd(np64(dy), z, row, w)
    dl = go.gate_bwd(L, idx, w, dw, counts, a, b, g, mask, seqs)
    dWr, dbr, dxr = go.router_bwd(np64(x), np64(trainer.layer.w_g), dl)
    # dlogits' own bound: the gates' part, then the balance part
    mags = np.abs(np64(dy))[:, None, :] * np.abs(z[row.reshape(-1)]).reshape(T, k, d)
    dw_off = (d + 8) * U32 * mags.sum(2)
    size = np.abs(w) * (np.abs(dw) + (np.abs(w) * np.abs(dw)).sum(1, keepdims=True))
    off = w * (dw_off + (w * dw_off).sum(1, keepdims=True)) + (k + 8) * U32 * size
    dl_off = np.zeros_like(dl)
    np.put_along_axis(dl_off, idx.astype(np.int64), off, 1)
    aux = np.abs(go.gate_bwd(L, idx, w, None, counts, a, 0.0, g, mask, seqs))
    peak = np.abs(g) * a * E / max(1, k) * counts.max(initial=0) / max(1, tokens[:-2].max(initial=1)) ** 2
    zpart = np.abs(go.gate_bwd(L, idx, w, None, counts, 0.0, b, g, mask, seqs))
    dl_off += rel * (aux + zpart + 2 * peak) + 2 * U32 * np.abs(dl)
    n = 3 * T + 16
    ax, aW = np.abs(np64(x)), np.abs(np64(trainer.layer.w_g))
    bound = ax.T @ dl_off + 2 * n * U32 * (ax.T @ np.abs(dl))
    assert np.all(np.abs(np64(grads.dw_g) - dWr) <= 1.01 * bound + 1e-37)
    if grads.dbias is not None:
        bound = dl_off.sum(0) + (T + 4) * U32 * np.abs(dl).sum(0)
        assert np.all(np.abs(np64(grads.dbias) - dbr) <= 1.01 * bound + 1e-37)
    if grads.dx is not None:
        mag = np.abs(dl) @ aW.T
        low = 2.0 ** -39 * (np.abs(dl).max(1)[:, None] * aW.sum(1)[None] + np.abs(dl).sum(1)[:, None] * aW.max(1)[None])
        bound = dl_off @ aW.T + (2.0 ** -10 + 2.0 ** -20 + 2 * (E + 16) * U32) * mag + low
        assert np.all(np.abs(np64(grads.dx) - dxr) <= 1.01 * bound + 2.0 ** -8 * np.abs(dxr) + 1e-37)
    if grads.dz is not None:
        assert np.all(np.abs(np64(grads.dz) - dz) <= (2.0 ** -8 + 3 * U32) * np.abs(dz))


@pytest.mark.parametrize("T", [1, 5, 64, 300])
@pytest.mark.parametrize("fmt", ["bf16", "fp8", "w8a8"])
def test_step(T, fmt):
    cfg, t, layer = make(T, fmt=fmt)
    tr = moe.GateTrainer(layer, balance_coef=0.02, z_coef=1e-3)
    y = tr(t["x"])
    # the layer's own forward selects from the same logits; its expert kernels may differ
    assert_layer_close(y, np64(layer(t["x"])), "forward")
    dy = torch.randn(T, cfg.d, device=DEV).bfloat16()
    dloss = torch.full((1,), 1.5, device=DEV)
    grads = tr.backward(dy, dloss=dloss, dx=True, dz=True)
    assert tr.check() == moe.MOE_OK
    check_step(tr, t["x"], dy, 1.5, grads)


@pytest.mark.parametrize("kw", [dict(d=128, E=24, k=3, f=64, zipf_s=1.0), dict(d=192, E=130, k=8, f=64),
                                dict(d=64, E=1, k=1, f=64), dict(d=320, E=64, k=5, f=128, R=4)])
def test_step_with_sequences_and_mask(kw):
    T = 150
    cfg, t, layer = make(T, seed=3, **kw)
    mask = (torch.arange(T, device=DEV) % 7 != 2).to(torch.uint8)
    seqs = torch.tensor([0, 20, 20, 100, 140], dtype=torch.int32, device=DEV)
    tr = moe.GateTrainer(layer, balance_coef=0.05, z_coef=2e-3)
    tr(t["x"], token_mask=mask, seq_offsets=seqs)
    dy = torch.randn(T, cfg.d, device=DEV).bfloat16()
    grads = tr.backward(dy, dx=True)
    assert tr.check() == moe.MOE_OK
    check_step(tr, t["x"], dy, 1.0, grads, mask.cpu().numpy(), seqs.cpu().numpy())
    assert grads.dz is None and (grads.dbias is None) == (layer.bias is None)


def test_clipping_in_the_step():
    cfg, t, layer = make(64)
    tr = moe.GateTrainer(layer)
    tr(t["x"])
    dy = torch.randn(64, cfg.d, device=DEV).bfloat16()
    whole, cut = tr.backward(dy), tr.backward(dy, max_norm=0.5)
    parts = [whole.dw_g] + ([whole.dbias] if whole.dbias is not None else [])
    norm = math.sqrt(sum(float(p.double().square().sum()) for p in parts))
    assert norm > 0.5 and abs(cut.norm.item() - norm) <= 6 * U32 * norm
    ref = whole.dw_g.double() * (0.5 / (norm + 1e-6))
    assert bool(((cut.dw_g.double() - ref).abs() <= 9 * U32 * ref.abs()).all())


def test_step_captured_and_replayed_beside_an_eager_one():
    T = 96
    cfg, t, layer = make(T, seed=5)
    eager, tr = moe.GateTrainer(layer, z_coef=1e-3), moe.GateTrainer(layer, z_coef=1e-3)
    x, dy = t["x"].clone(), torch.randn(T, cfg.d, device=DEV).bfloat16()
    y0 = eager(x)
    g0 = eager.backward(dy, dx=True, max_norm=1.0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # first-use set-up outside the capture
        tr(x)
        tr.backward(dy, dx=True, max_norm=1.0)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = tr(x)
        g = tr.backward(dy, dx=True, max_norm=1.0)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, y0) and torch.equal(g.dw_g, g0.dw_g) and torch.equal(g.dx, g0.dx)
        assert torch.equal(tr.loss, eager.loss) and torch.equal(g.norm, g0.norm)
        eager(x)
        assert torch.equal(eager.backward(dy).dw_g.isfinite().all(), torch.tensor(True, device=DEV))
    # new inputs in the captured buffers
    x.copy_(torch.randn(T, cfg.d, device=DEV))
    graph.replay()
    y1 = eager(x)
    g1 = eager.backward(dy, dx=True, max_norm=1.0)
    torch.cuda.synchronize()
    assert torch.equal(y, y1) and torch.equal(g.dw_g, g1.dw_g)


def test_step_of_no_tokens():
    cfg, t, layer = make(4)
    tr = moe.GateTrainer(layer, z_coef=1e-3)
    y = tr(torch.empty(0, cfg.d, device=DEV).bfloat16())
    assert y.shape == (0, cfg.d) and tr.loss.tolist() == [0, 0, 0] and not tr.counts.any()
    g = tr.backward(torch.empty(0, cfg.d, device=DEV).bfloat16(), dx=True, dz=True, max_norm=1.0)
    assert not g.dw_g.any() and g.norm.item() == 0.0 and g.dx.shape == (0, cfg.d)
    assert tr.check() == moe.MOE_OK


def test_refusals():
    cfg, t, layer = make(16)
    tr = moe.GateTrainer(layer)
    with pytest.raises(RuntimeError, match="forward first"):
        tr.backward(t["x"])
    tr(t["x"])
    with pytest.raises(ValueError, match="shape"):
        tr.backward(t["x"][:8].contiguous())
    layer.rebalance(torch.ones(cfg.E, dtype=torch.int64), 8)
    with pytest.raises(NotImplementedError):
        tr(t["x"])
