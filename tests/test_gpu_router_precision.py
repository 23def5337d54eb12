"""How exact the router's backward is: dx and dw_g as products of fp32 values.

u = 2^-24 is half a step of fp32.  The bounds of test_gpu_gate_train grow with the number
of terms and leave room for operands of fewer bits; the data here do not: terms that
cancel, where an operand's rounding is all that remains, and sums whose exact value is an
fp32 number."""

import math

import pytest
import torch

import routing_dispatch_expert_softmax_b200 as moe
from routing_dispatch_expert_softmax_b200.binding import MoEShape

from parity_utils import U32

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF16 = 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    moe.load_library()
    yield
    torch.cuda.synchronize()


def run(x, W, dl, dw=True, db=True, dx=True):
    """The call's outputs, poisoned before; its scratch holds NaN patterns."""
    T, d, E = x.shape[0], W.shape[0], W.shape[1]
    s = MoEShape.of(T, d, E, 1, 64)
    ws = moe.workspace_bwd(s)
    ws[256:] = 0xff
    out = dict(dw_g=torch.full((d, E), math.nan, device=DEV) if dw else None,
               dbias=torch.full((E,), math.nan, device=DEV) if db else None,
               dx=torch.full((T, d), math.nan, dtype=torch.bfloat16, device=DEV) if dx else None)
    moe.moe_router_bwd(x if dw else None, W if dx else None, dl, s, ws, **out)
    st = moe.moe_check(ws)
    assert st == moe.MOE_OK, moe.moe_error_string(st)
    return out


def dx_bound(dl, W):
    """(dx in 64 bits, what the call may be off by).  Each operand is held in two parts of
    11 bits: what the second part loses (2^-21 of the value; for fp16 parts of a row that
    was scaled to [2^13, 2^15) no less than 2^-25, 2^-38 of its largest) and the product
    of the second parts (2^-20) come to 2^-19 of a term at most.  The tensor cores may cut
    at each MMA, 2u of the sum and 2u of what is added: 12 MMAs for each 64 experts (or 8
    for the 64 of three products of 8), and 20 adds behind them."""
    E = W.shape[1]
    l64, W64 = dl.double(), W.double()
    ref, mag = l64 @ W64.t(), l64.abs() @ W64.abs().t()
    low = 2.0 ** -38 * (l64.abs().amax(1)[:, None] * W64.abs().sum(1)[None]
                        + l64.abs().sum(1)[:, None] * W64.abs().amax(1)[None])
    n = 24 * -(-E // 64) + 20
    return ref, BF16 * ref.abs() + (1 + BF16) * ((2.0 ** -19 + 4 * n * U32) * mag + low) + 1e-37


def cancelling(T, d, E, seed=0):
    """Gradients of a softmax sum to zero over a row's experts; weights whose experts have
    most of a column in common then leave next to nothing of each product."""
    g = torch.Generator(device=DEV).manual_seed(seed + T + d + E)
    x = torch.randn(T, d, generator=g, device=DEV).bfloat16()
    W = 1 + torch.randn(d, E, generator=g, device=DEV) * 2.0 ** -8
    dl = torch.randn(T, E, generator=g, device=DEV)
    return x, W, dl - dl.mean(1, keepdim=True)


@pytest.mark.parametrize("T", [1, 16, 50, 96, 130, 192, 300, 1000])
@pytest.mark.parametrize("d,E", [(64, 3), (64, 8), (448, 60), (128, 130), (64, 255), (320, 300)])
def test_dx_where_terms_cancel(T, d, E):
    x, W, dl = cancelling(T, d, E)
    ref, bound = dx_bound(dl, W)
    off = (run(x, W, dl)["dx"].double() - ref).abs()
    assert bool((off <= bound).all()), float((off / bound).max())


@pytest.mark.parametrize("T,d,E", [(20000, 64, 8), (4097, 448, 60), (1000, 2048, 128), (515, 128, 1000),
                                   (2000, 576, 256), (9000, 1088, 192)])
def test_dx_of_many_tokens_where_terms_cancel(T, d, E):
    x, W, dl = cancelling(T, d, E)
    ref, bound = dx_bound(dl, W)
    off = (run(x, W, dl, dw=E % 3 == 0)["dx"].double() - ref).abs()
    assert bool((off <= bound).all()), float((off / bound).max())
