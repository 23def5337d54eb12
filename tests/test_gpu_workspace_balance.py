"""The balance loss and the gate's gradient with the workspace that they ask for alone."""

import math

import pytest
import torch

import routing_dispatch_expert_softmax_b200 as moe

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.mark.parametrize("T,E,k,S", [(1, 1, 1, 1), (64, 8, 2, 1), (300, 130, 8, 1), (1000, 8, 2, 700), (20000, 256, 8, 1),
                                     (4096, 1024, 4, 16)])
def test_same_results_and_nothing_behind_it_is_touched(T, E, k, S):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    g = torch.Generator(device=DEV).manual_seed(T + E)
    L = torch.randn(T, E, generator=g, device=DEV)
    top, idx = torch.topk(L, k, dim=1)
    w, dw, idx = torch.softmax(top, 1), torch.randn(T, k, generator=g, device=DEV), idx.int()
    seqs = None if S == 1 else torch.sort(torch.randint(0, T + 1, (S + 1,), generator=g, device=DEV)).values.int()
    s = moe.MoEShape.of(T, 64, E, k, 64)
    need = moe.moe_workspace_size_balance(s, S)
    room = torch.full((need + 4096,), 0xff, dtype=torch.uint8, device=DEV)
    room[:64] = 0

    def step(ws):
        out = [torch.full((3,), math.nan, device=DEV), torch.full((S, E), -1, dtype=torch.int32, device=DEV),
               torch.full((S + 2,), -1, dtype=torch.int32, device=DEV), torch.full((S, E), math.nan, device=DEV),
               torch.full((T, E), math.nan, device=DEV)]
        moe.moe_balance_loss(L, idx, *out[:3], s, ws, z_coef=1e-3, seq_offsets=seqs, prob_mean=out[3])
        moe.moe_gate_bwd(L, idx, out[4], s, ws, w=w, dw=dw, counts=out[1], tokens=out[2], z_coef=1e-3,
                         seq_offsets=seqs)
        assert moe.moe_check(ws) == moe.MOE_OK
        return out

    got, want = step(room[:need]), step(moe.workspace_bwd(s, S))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert bool((room[need:] == 0xff).all())
    with pytest.raises(ValueError, match="ws has"):
        moe.moe_balance_loss(L, idx, *got[:3], s, room[:need - 256], seq_offsets=seqs)
    assert all(torch.equal(a, b) for a, b in zip(step(moe.workspace_balance(s, S)), want))
