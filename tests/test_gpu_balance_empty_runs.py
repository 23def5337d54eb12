"""The balance loss over thousands of empty sequences in one place, between full ones."""

import math

import numpy as np
import pytest
import torch

import routing_dispatch_expert_softmax_b200 as moe
from oracle import gate_train_oracle as go

from parity_utils import U32, np64

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    moe.load_library()
    yield
    torch.cuda.synchronize()


def runs(T, S, at):
    """S + 1 offsets: sequences of some tokens around runs of empty ones at the places ``at``."""
    full = sorted({0, T, *at, *(a + 3 for a in at if a + 3 < T)})
    off = list(full)
    while len(off) < S + 1:
        off += at[: S + 1 - len(off)]
    return np.sort(np.array(off[:S + 1], dtype=np.int32))


def batch(T, E, k, off):
    r = np.random.default_rng(T + len(off))
    L = r.normal(size=(T, E)).astype(np.float32)
    idx = np.argsort(-L, axis=1, kind="stable")[:, :k].astype(np.int32)
    return L, idx, torch.as_tensor(off).to(DEV)


def call(L, idx, off, E, k):
    T, S = L.shape[0], len(off) - 1
    s = moe.MoEShape.of(T, 64, E, k, 64)
    ws = moe.workspace_balance(s, S)
    loss, mean = torch.full((3,), math.nan, device=DEV), torch.full((S, E), math.nan, device=DEV)
    counts = torch.full((S, E), -1, dtype=torch.int32, device=DEV)
    tokens = torch.full((S + 2,), -1, dtype=torch.int32, device=DEV)
    args = (torch.as_tensor(L).to(DEV), torch.as_tensor(idx).to(DEV), loss, counts, tokens, s, ws)
    step = lambda: moe.moe_balance_loss(*args, seq_offsets=off, prob_mean=mean)  # noqa: E731
    step()
    return step, ws, loss, counts, tokens, mean


@pytest.mark.parametrize("T,E,k,S,at", [(50, 8, 2, 300, [25]), (200, 8, 2, 5000, [1, 100, 199]), (700, 40, 3, 3000, [0, 350]),
                                        (64, 130, 4, 900, [31, 32, 33]), (3, 2, 1, 2000, [1, 2])])
def test_runs_of_empty_sequences(T, E, k, S, at):
    off = runs(T, S, at)
    L, idx, doff = batch(T, E, k, off)
    _, ws, loss, counts, tokens, mean = call(L, idx, doff, E, k)
    assert moe.moe_check(ws) == moe.MOE_OK
    ref, c, n, m = go.balance_loss(L, idx, 1e-2, 0.0, None, off)
    assert np.array_equal(counts.cpu().numpy(), c) and np.array_equal(tokens.cpu().numpy(), n)
    # a softmax over E values (D < 12) and sums of at most T rows, as in test_gpu_gate_train
    rel = (4.44 * 12 + 2 * E + T + 40) * U32
    assert np.all(np.abs(np64(mean) - m) <= rel * m + 1e-37)
    assert abs(loss[1].item() - ref[1]) <= 2 * rel * ref[1]


def test_offsets_that_do_not_ascend_still_end():
    for off in ([0, 5, 5, 3, 3, 40, 2, 50], [50, 0, 0, 0, 50], [7, 7, 7, 7], [0, 60, 0, 50], [-3, -3, 20, 20, 50]):
        L, idx, doff = batch(50, 8, 2, off)
        _, ws, *_ = call(L, idx, doff.int(), 8, 2)
        want = moe.MOE_OK if off == [7, 7, 7, 7] else moe.MOE_ERR_DEVICE_CHECK
        assert moe.moe_check(ws) == want


def test_a_run_costs_no_step_for_each_of_its_sequences():
    T, E, k, S = 8192, 16, 2, 65535
    L, idx, doff = batch(T, E, k, np.concatenate([[0], np.full(S - 1, T // 2 + 1), [T]]).astype(np.int32))
    even = torch.linspace(0, T, S + 1, device=DEV).int()
    best = []
    for off in (doff, even):
        step = call(L, idx, off, E, k)[0]
        t = []
        for _ in range(6):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            step()
            b.record()
            torch.cuda.synchronize()
            t.append(a.elapsed_time(b))
        best.append(min(t))
    assert best[0] < 4 * best[1], best  # one step each took 14 times as long
