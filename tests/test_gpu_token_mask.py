"""Token masks as comparisons give them: bool, beside the uint8 of the C calls."""

import pytest
import torch

import routing_dispatch_expert_softmax_b200 as moe
from routing_dispatch_expert_softmax_b200 import workloads as wl

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.mark.parametrize("T", [1, 37, 300])
def test_bool_mask_is_the_same_mask(T):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    cfg = wl.TINY.with_T(T)
    t = wl.make_layer(cfg, DEV, 2)
    layer = moe.MoELayer(t["w_g"], t["bias"], t["w13"], t["w2"], cfg.k)
    mask = torch.arange(T, device=DEV) % 3 != 1
    dy = torch.randn(T, cfg.d, device=DEV).bfloat16()
    got = []
    for m in (mask, mask.to(torch.uint8)):
        tr = moe.GateTrainer(layer, z_coef=1e-3)
        tr(t["x"], token_mask=m)
        g = tr.backward(dy)
        assert tr.check() == moe.MOE_OK
        got.append([tr.loss, tr.counts, tr.tokens, g.dw_g])
    assert all(torch.equal(a, b) for a, b in zip(*got))
    assert int(got[0][2][0]) == int(mask.sum())
    with pytest.raises(ValueError, match="token_mask must have shape"):
        moe.GateTrainer(layer)(t["x"], token_mask=torch.ones(T + 1, dtype=torch.bool, device=DEV))
    with pytest.raises(ValueError, match="token_mask must be contiguous" if T > 1 else "token_mask must have shape"):
        moe.GateTrainer(layer)(t["x"], token_mask=torch.ones(2 * T, dtype=torch.bool, device=DEV)[::2][:T]
                               if T > 1 else torch.ones(1, 1, dtype=torch.bool, device=DEV))
    with pytest.raises(TypeError, match="token_mask must be torch.uint8, got torch.int32"):
        moe.GateTrainer(layer)(t["x"], token_mask=mask.int())
