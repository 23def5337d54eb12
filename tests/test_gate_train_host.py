"""CPU tests of the calls that train the gate: the oracle against differences
and worked values, workspace sizes, and the refusals of the C ABI and of the
Python binding.  Nothing here reaches a kernel."""

import ctypes
import math
import subprocess
import sys

import numpy as np
import pytest
import torch

import routing_dispatch_expert_softmax_b200 as moe
from oracle import gate_train_oracle as go
from routing_dispatch_expert_softmax_b200 import binding as B

SHAPE = dict(T=64, d=256, E=8, k=2, f=512, R=0)
P = 1 << 20          # an aligned address that no call may dereference
BAD = P + 1          # a misaligned one


@pytest.fixture(scope="module")
def lib():
    return B.load_library()


def ref(**kw):
    return ctypes.byref(B.MoEShape.of(**dict(SHAPE, **kw)))


# ------------------------------------------------------------------- oracle
def _batch(T, E, k, seed):
    r = np.random.default_rng(seed)
    L = r.normal(size=(T, E)) * 2
    idx = np.argsort(-L, axis=1, kind="stable")[:, :k]
    top = np.take_along_axis(L, idx, 1)
    w = np.exp(top - top[:, :1])
    return r, L, idx, w / w.sum(1, keepdims=True)


@pytest.mark.parametrize("seqs", [None, [0, 3, 3, 9], [2, 7, 11]])
@pytest.mark.parametrize("masked", [False, True])
def test_oracle_gradient_against_differences(seqs, masked):
    T, E, k = 12, 5, 2
    r, L, idx, w = _batch(T, E, k, 3)
    mask = (np.arange(T) % 4 != 1).astype(np.uint8) if masked else None
    dw = r.normal(size=(T, k))
    a, b, g = 0.3, 0.2, 1.7
    _, counts, _, _ = go.balance_loss(L, idx, a, b, mask, seqs)

    def value(M):
        top = np.take_along_axis(M, idx, 1)
        v = np.exp(top - top.max(1, keepdims=True))
        gates = v / v.sum(1, keepdims=True)
        return float((gates * dw).sum()) + g * go.balance_loss(M, idx, a, b, mask, seqs, counts)[0][0]

    got = go.gate_bwd(L, idx, w, dw, counts, a, b, g, mask, seqs)
    h = 1e-5
    for t in range(T):
        for e in range(E):
            up, dn = L.copy(), L.copy()
            up[t, e] += h
            dn[t, e] -= h
            # central difference: h^2/6 times a third derivative of order 10
            assert abs((value(up) - value(dn)) / (2 * h) - got[t, e]) < 1e-8


def test_oracle_balance_worked_values():
    # uniform probabilities: balance = coef * E * sum_e (c_e / (k N)) / E = coef
    L = np.zeros((6, 4))
    idx = np.array([[0, 1]] * 6)
    loss, c, n, mean = go.balance_loss(L, idx, 0.5, 2.0)
    assert c.tolist() == [[6, 6, 0, 0]] and n.tolist() == [6, 6, 1]
    assert np.allclose(mean, 0.25)
    assert math.isclose(loss[1], 0.5) and math.isclose(loss[2], 2 * math.log(4) ** 2)
    # every token sure of expert 0: the largest balance value, coef * E / k
    L[:, 0] = 200.0
    assert math.isclose(go.balance_loss(L, idx[:, :1], 0.5, 0.0)[0][1], 0.5 * 4)


def test_oracle_router_and_combine_against_products():
    r = np.random.default_rng(0)
    x, W, dl = r.normal(size=(5, 3)), r.normal(size=(3, 4)), r.normal(size=(5, 4))
    dW, db, dx = go.router_bwd(x, W, dl)
    h = 1e-6
    for i in range(3):
        for e in range(4):
            V = W.copy()
            V[i, e] += h
            assert abs((((x @ V) - (x @ W)) * dl).sum() / h - dW[i, e]) < 1e-6
    assert np.allclose(db, dl.sum(0)) and np.allclose(dx, dl @ W.T)
    dy, z, w = r.normal(size=(2, 3)), r.normal(size=(4, 3)), r.random((2, 2))
    row = np.array([[3, 0], [1, 2]])
    dw, dz = go.combine_bwd(dy, z, row, w)
    assert np.isclose(dw[0, 0], dy[0] @ z[3]) and np.allclose(dz[2], w[1, 1] * dy[1])


def test_oracle_clip():
    norm, out = go.clip_grads([np.array([3.0]), np.array([0.0, 4.0])], 1.0)
    assert norm == 5.0 and np.isclose(out[1][1], 4.0 / (5 + 1e-6))
    assert go.clip_grads([np.array([3.0])], 10.0)[1][0][0] == 3.0


# --------------------------------------------------------------- workspaces
def test_workspace_sizes(lib):
    size = lambda S=1, **kw: lib.moe_workspace_size_bwd(ref(**kw), S)  # noqa: E731
    assert size() > 0 and size(T=0) > 0
    assert size(0) == 0 and size(-1) == 0 and size(65536) == 0 and size(d=96) == 0
    assert lib.moe_workspace_size_bwd(None, 1) == 0
    assert size(65535) > size(1)
    assert size(T=1 << 20, E=1024, d=16384) > 0
    g = lib.moe_workspace_size_grads
    assert g(0) > 0 and g(65536) > g(1) > 0 and g(-1) == 0 and g(65537) == 0


# ----------------------------------------------------------------- refusals
def _vary(fn, good, bad):
    """Each argument of `bad` ({index: values}) in turn is refused."""
    for i, values in bad.items():
        for v in values:
            args = list(good)
            args[i] = v
            assert fn(*args) == moe.MOE_ERR_INVALID_ARG, (i, v)


def test_balance_loss_refuses(lib):
    good = [P, P, None, P, 4, ref(), 0.1, 0.1, P, P, P, None, P, None]
    _vary(lib.moe_balance_loss, good, {
        0: [None, BAD], 1: [None, BAD], 3: [BAD, None], 4: [0, -1, 65536],
        5: [None, ref(T=-1), ref(d=100), ref(k=9)], 6: [math.nan, math.inf], 7: [math.nan, -math.inf],
        8: [None, BAD], 9: [None, BAD], 10: [None, BAD], 11: [BAD], 12: [None, P + 64]})


def test_gate_bwd_refuses(lib):
    good = [P, P, P, P, None, None, 1, P, P, ref(), 0.1, 0.1, None, P, P, None]
    _vary(lib.moe_gate_bwd, good, {
        0: [None, BAD], 1: [None, BAD], 2: [None, BAD], 3: [BAD], 5: [BAD], 6: [0, 2, 65536],
        7: [BAD], 8: [None, BAD], 9: [None, ref(E=1025)], 10: [math.nan], 11: [math.inf],
        12: [BAD], 13: [None, BAD], 14: [None, P + 64]})
    neither = list(good)
    neither[3] = neither[7] = None
    assert lib.moe_gate_bwd(*neither) == moe.MOE_ERR_INVALID_ARG


def test_combine_bwd_refuses(lib):
    good = [P, P, P, P, ref(), P, P, None]
    _vary(lib.moe_combine_bwd, good, {0: [None, P + 8], 1: [None, P + 8], 2: [None, BAD],
                                      3: [None, BAD], 4: [None, ref(d=65)], 5: [BAD], 6: [P + 8]})
    assert lib.moe_combine_bwd(P, P, P, P, ref(), None, None, None) == moe.MOE_ERR_INVALID_ARG


def test_router_bwd_refuses(lib):
    good = [P, P, P, ref(), P, P, P, P, None]
    _vary(lib.moe_router_bwd, good, {0: [None, P + 8], 1: [None, BAD], 2: [None, BAD],
                                     3: [None, ref(T=(1 << 20) + 1)], 4: [BAD], 5: [BAD],
                                     6: [P + 8], 7: [None, P + 64]})
    assert (lib.moe_router_bwd(P, P, P, ref(), None, None, None, P, None)
            == moe.MOE_ERR_INVALID_ARG)


def _grads(*rows):
    arr = (B.MoEGrad * max(1, len(rows)))()
    for e, r in zip(arr, rows):
        e.data, e.out, e.n, e.dtype, e.out_dtype = r
    return arr


@pytest.mark.parametrize("row", [
    (None, P, 4, 0, 0), (P, None, 4, 0, 0), (P + 2, P, 4, 0, 0), (P + 1, P, 4, 1, 1),
    (P, P + 2, 4, 0, 0), (P, P + 1, 4, 1, 1), (P, P, -1, 0, 0), (P, P, (1 << 40) + 1, 0, 0),
    (P, P, 4, 2, 2), (P, P, 4, 0, 1), (P, P, 4, 1, 0),
])
def test_clip_refuses_entries(lib, row):
    ok = (P, P, 4, 0, 0)
    for g in (_grads(row), _grads(ok, row)):
        n = len(g)
        assert lib.moe_clip_grads(g, n, 1.0, P, P, None) == moe.MOE_ERR_INVALID_ARG
        assert lib.moe_grad_scale(g, n, P, 1.0, P, None) == moe.MOE_ERR_INVALID_ARG


def test_clip_refuses_arguments(lib):
    g = _grads((P, P, 4, 0, 0))
    _vary(lib.moe_clip_grads, [g, 1, 1.0, P, P, None],
          {0: [None], 1: [-1, 65537], 2: [-1.0, math.nan], 3: [BAD], 4: [None, P + 64]})
    _vary(lib.moe_grad_scale, [g, 1, P, 1.0, P, None],
          {0: [None], 1: [-1], 2: [None, P + 4], 3: [-1.0, math.nan], 4: [BAD]})
    _vary(lib.moe_grad_sumsq, [g, 1, P, P, None],
          {0: [None], 1: [-1], 2: [None, P + 4], 3: [None, P + 64]})
    # the sum looks at no out
    no_out = _grads((P, None, 4, 0, 0))
    assert lib.moe_grad_sumsq(no_out, 1, P, P + 64, None) == moe.MOE_ERR_INVALID_ARG


def test_valid_calls_need_a_gpu(lib):
    if torch.cuda.is_available():
        pytest.skip("a device is present")
    g = _grads((P, P, 4, 0, 0))
    for status in (
            lib.moe_balance_loss(P, P, None, None, 1, ref(), 0.1, 0.1, P, P, P, None, P, None),
            lib.moe_gate_bwd(P, P, P, P, None, None, 1, P, P, ref(), 0.1, 0.1, None, P, P, None),
            lib.moe_combine_bwd(P, P, P, P, ref(), P, P, None),
            lib.moe_router_bwd(P, P, P, ref(), P, P, P, P, None),
            lib.moe_clip_grads(g, 1, 1.0, P, P, None), lib.moe_grad_sumsq(g, 1, P, P, None),
            lib.moe_grad_scale(g, 1, P, math.inf, None, None)):
        assert status in (moe.MOE_ERR_CUDA, moe.MOE_ERR_UNSUPPORTED)


def test_empty_batch_calls(lib):
    # with no tokens these two have nothing to write and do not look further
    assert lib.moe_gate_bwd(None, None, None, None, None, None, 1, None, None, ref(T=0), 0.1, 0.1,
                            None, None, P, None) == moe.MOE_OK
    assert lib.moe_combine_bwd(None, None, None, None, ref(T=0), P, None, None) == moe.MOE_OK
    assert lib.moe_combine_bwd(None, None, None, None, ref(T=0), None, None, None) == moe.MOE_OK


def test_binding_refuses(lib):
    s = B.MoEShape.of(**SHAPE)
    cpu = torch.zeros(64, 8)
    ws = torch.zeros(1024, dtype=torch.uint8)
    i = torch.zeros(64, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA tensor"):
        moe.moe_balance_loss(cpu, i, cpu, cpu, cpu, s, ws)
    with pytest.raises(TypeError, match="logits is required"):
        moe.moe_balance_loss(None, i, cpu, cpu, cpu, s, ws)
    with pytest.raises(ValueError, match="seq_offsets"):
        moe.moe_balance_loss(cpu, i, cpu, cpu, cpu, s, ws, seq_offsets=torch.zeros(1))
    with pytest.raises(TypeError, match="dlogits is required"):
        moe.moe_gate_bwd(None, None, None, s, ws)
    with pytest.raises(ValueError, match="CUDA tensor"):
        moe.moe_combine_bwd(cpu, None, i, None, s, dw=cpu)
    with pytest.raises(TypeError, match="x is required"):
        moe.moe_router_bwd(None, None, cpu, s, ws, dw_g=cpu)
    with pytest.raises(ValueError, match="no gradients"):
        moe.GradList([])
    with pytest.raises(ValueError, match="as many outs"):
        moe.GradList([cpu], [cpu, cpu])
    with pytest.raises(TypeError, match="fp32 or bf16"):
        moe.moe_clip_grads([cpu.double()], 1.0)
    with pytest.raises(TypeError, match="out 0 must be"):
        moe.GradList([cpu], [cpu.bfloat16()])
    with pytest.raises(ValueError, match="elements"):
        moe.GradList([cpu], [cpu[:3]])
    with pytest.raises(ValueError, match="CUDA tensor"):
        moe.GradList([cpu])


def test_operand_checks(lib):
    class Seen(B._native.Operands):
        def _refuse(self, *a):
            raise KeyError(a)

    o = Seen("call")
    assert o.where == "call" and o.index is None
    t = torch.zeros(3, 4)
    assert o.ptr(None, torch.float32, (3, 4), "t", True) is None
    for a in ((None, torch.float32, (3, 4), "t"), (None, torch.float32, (3, 4), "t", False),
              (t, torch.float32, (3, 4), "t"),  # no CUDA tensor
              (t, torch.float32, ("x", 4), "t"), (t, "float32", None, "t"), (3, torch.float32, None, "t"),
              (torch.zeros(2, device="meta"), torch.float32, None, "t")):
        with pytest.raises(KeyError) as e:
            o.ptr(*a)
        assert e.value.args[0] == a[:4] and o.index is None
    o.index = 3
    assert o.index == 3
    with pytest.raises(TypeError):
        o.index = "cuda"
    with pytest.raises(ValueError):
        o.index = -1
    with pytest.raises(TypeError):
        o.ptr(t)
    with pytest.raises(TypeError):
        B._native.Operands("call", 1)

    class Silent(B._native.Operands):
        def _refuse(self, *a):
            pass

    with pytest.raises(RuntimeError, match="without a reason"):
        Silent("call").ptr(t, torch.float32, None, "t")


def test_addresses(lib):
    ts = [torch.zeros(i + 1) for i in range(5)]
    want = [t.data_ptr() for t in ts]
    got = np.frombuffer(B._native.addresses(ts, None), dtype=np.uint64).tolist()
    assert got == want
    got = np.frombuffer(B._native.addresses(ts[:2], ts[3:]), dtype=np.uint64).tolist()
    assert got == want[:2] + want[3:]
    assert B._native.addresses([], None) == b""
    for a in (((), None), ([3], None), ([], [None]), ([], 3)):
        with pytest.raises(TypeError):
            B._native.addresses(*a)
    # nothing is kept: references do not grow
    before = sys.getrefcount(ts[0])
    for _ in range(100):
        B._native.addresses(ts, ts)
    after = sys.getrefcount(ts[0])
    assert after == before


def test_extension_found_after_import(lib):
    # a process that imported the package before the extension was built finds it later
    code = ("import importlib, torch\n"
            "real = importlib.import_module\n"
            "def hide(name, *a):\n"
            "    if name.endswith('_operands'): raise ImportError(name)\n"
            "    return real(name, *a)\n"
            "importlib.import_module = hide\n"
            "import routing_dispatch_expert_softmax_b200 as moe\n"
            "from routing_dispatch_expert_softmax_b200 import binding as B\n"
            "assert B._native is None\n"
            "s = moe.MoEShape.of(1, 64, 1, 1, 64)\n"
            "for _ in range(2):\n"
            "    try: moe.moe_combine_bwd(None, None, None, None, s)\n"
            "    except RuntimeError as e: assert '_operands.so is not built' in str(e)\n"
            "    else: assert False\n"
            "importlib.import_module = real\n"
            "try: moe.moe_combine_bwd(None, None, None, None, s)\n"
            "except TypeError as e: assert 'dy is required' in str(e)\n"
            "else: assert False\n"
            "assert B._native is not None\n")
    p = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True)
    assert p.returncode == 0, p.stderr
