"""How exact the router's backward is: dx and dw_g as products of fp32 values.

u = 2^-24 is half a step of fp32.  The bounds of test_gpu_gate_train grow with the number
of terms and leave room for operands of fewer bits; the data here do not: terms that
cancel, where an operand's rounding is all that remains, and sums whose exact value is an
fp32 number."""

import math

import pytest
import torch

import routing_dispatch_expert_softmax_b200 as moe

from parity_utils import U32
from router_utils import dw_bound, dx_bound, run

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    moe.load_library()
    yield
    torch.cuda.synchronize()


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


# few tokens; planes side by side three and two to a row; a plane each; partial sums and none
SHAPES = [(5, 64, 8), (150, 128, 24), (192, 64, 130), (300, 320, 24), (300, 192, 60), (200, 128, 60), (257, 320, 130),
          (515, 128, 1000), (1000, 512, 128), (4097, 448, 60), (20000, 64, 8), (5000, 2048, 256)]


@pytest.mark.parametrize("T,d,E", SHAPES)
def test_dw_of_one_token_a_column_is_its_gradient(T, d, E):
    # with a single 1 in each column of x the sum is one fp32 number: all its 24 bits arrive,
    # in whichever token range and place of a tile the token lies
    g = torch.Generator(device=DEV).manual_seed(T + E)
    dl = torch.randn(T, E, generator=g, device=DEV) * torch.exp2(torch.randint(-30, 30, (T, E), generator=g, device=DEV))
    W = torch.zeros(d, E, device=DEV)
    for seed in range(3):
        t = torch.randint(0, T, (d,), generator=g, device=DEV)
        t[0], t[-1] = 0, T - 1
        x = torch.zeros(T, d, dtype=torch.bfloat16, device=DEV)
        x[t, torch.arange(d, device=DEV)] = 1.0
        assert torch.equal(run(x, W, dl, dx=seed == 1)["dw_g"], dl[t])


@pytest.mark.parametrize("T,d,E", [(192, 64, 8), (300, 192, 24), (3000, 16384, 256), (3000, 64, 130), (4097, 448, 60),
                                   (20000, 64, 8), (20000, 4096, 200)])
def test_dw_of_long_sums_of_one_sign(T, d, E):
    # the tensor cores cut: left in their accumulator over 600 MMAs such a sum is 2.4e-5 short
    g = torch.Generator(device=DEV).manual_seed(T + E)
    x = (1 + torch.rand(T, d, generator=g, device=DEV)).bfloat16()
    dl = 0.5 + torch.rand(T, E, generator=g, device=DEV)
    got = run(x, torch.zeros(d, E, device=DEV), dl, dx=False)["dw_g"]
    ref, bound = dw_bound(x, dl)
    off = (got.double() - ref).abs()
    assert bool((off <= bound).all()), float((off / ref).max())
    assert float((bound / ref).max()) < 1.9e-5
