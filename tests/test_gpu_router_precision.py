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
    was scaled to [2^13, 2^15) no less than 2^-25, 2^-38 of its largest; for tf32 parts no
    less than 2^-137, half of its lowest step) and the product of the second parts (2^-20) come to 2^-19 of a term at most.  The tensor cores may cut
    at each MMA, 2u of the sum and 2u of what is added: 12 MMAs for each 64 experts (or 8
    for the 64 of three products of 8), and 20 adds behind them."""
    E = W.shape[1]
    l64, W64 = dl.double(), W.double()
    ref, mag = l64 @ W64.t(), l64.abs() @ W64.abs().t()
    low = 2.0 ** -38 * (l64.abs().amax(1)[:, None] * W64.abs().sum(1)[None]
                        + l64.abs().sum(1)[:, None] * W64.abs().amax(1)[None])
    low += 2.0 ** -137 * (W64.abs().sum(1)[None] + l64.abs().sum(1)[:, None])
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


@pytest.mark.parametrize("T,E", [(40, 24), (300, 24), (300, 60), (2000, 130), (300, 260)])
@pytest.mark.parametrize("a,b", [(112, 0), (113, -15), (124, -20), (124, -124), (-100, 90), (-104, 115), (90, -99),
                                 (-60, -46), (60, 60), (0, 120), (1, -90)])
def test_dx_of_operands_far_from_one(T, E, a, b):
    # the results lie in fp32's and bf16's range, whatever the operands' sizes
    d = 128
    g = torch.Generator(device=DEV).manual_seed(T + E)
    x = torch.randn(T, d, generator=g, device=DEV).bfloat16()
    W, dl = torch.randn(d, E, generator=g, device=DEV) / math.sqrt(d), torch.randn(T, E, generator=g, device=DEV)
    one = run(x, W, dl, dw=False)["dx"]
    dl, W = dl * 2.0 ** a, W * 2.0 ** b
    got = run(x, W, dl, dw=False)["dx"]
    ref, bound = dx_bound(dl, W)
    off = (got.double() - ref).abs()
    assert bool((off <= bound).all()), float((off / bound).max())
    if a % 2 == b % 2 == 0 and a + b > -100 and min(a, b) >= -104:
        # (below that the operands themselves round: fp32's lowest normal is 2^-126)
        # rows are scaled by even powers of two: the same values go through the products
        assert torch.equal(got.double(), one.double() * 2.0 ** (a + b))


@pytest.mark.parametrize("T,E", [(300, 24), (700, 200)])
def test_dx_of_rows_and_columns_of_every_size(T, E):
    # one call whose rows and columns span fp32's range; a row of zeros and one far below the others
    d = 192
    g = torch.Generator(device=DEV).manual_seed(T)
    x = torch.randn(T, d, generator=g, device=DEV).bfloat16()
    up = torch.linspace(-110, 110, T, device=DEV).round()[:, None]
    across = torch.linspace(100, -100, d, device=DEV).round()[:, None]
    dl = torch.randn(T, E, generator=g, device=DEV) * torch.exp2(up)
    W = torch.randn(d, E, generator=g, device=DEV) * torch.exp2(across)
    dl[7], W[9] = 0, 0
    dl[11] *= 2.0 ** -10
    ref, bound = dx_bound(dl, W)
    got = run(x, W, dl, dw=False)["dx"].double()
    fits = ref.abs() < 2.0 ** 127
    assert int(fits.sum()) > T * d // 2 and bool(torch.isfinite(got[fits]).all())
    assert bool(((got - ref).abs() <= bound)[fits].all())
    assert not got[7].any() and not got[:, 9].any()
