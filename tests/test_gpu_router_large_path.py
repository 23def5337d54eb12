"""moe_router_bwd through its three kernels, what the calls of few tokens do not reach: each
set of outputs, sizes of gradients, values that are not finite, operands at any alignment.
The numbers of experts cover planes three and two to a row and a plane each, the W tiles
that stay in shared memory and those that do not."""

import math

import pytest
import torch

import routing_dispatch_expert_softmax_b200 as moe
from routing_dispatch_expert_softmax_b200.binding import MoEShape

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


def inputs(T, d, E, scale=1.0):
    g = torch.Generator(device=DEV).manual_seed(T + d + E)
    x = torch.randn(T, d, generator=g, device=DEV).bfloat16()
    W = torch.randn(d, E, generator=g, device=DEV) / math.sqrt(d)
    return x, W, torch.randn(T, E, generator=g, device=DEV) * torch.rand(T, 1, generator=g, device=DEV) * scale


def check(x, W, dl, out):
    T = x.shape[0]
    if out["dw_g"] is not None:
        ref, bound = dw_bound(x, dl)
        assert bool(((out["dw_g"].double() - ref).abs() <= bound).all()), "dw_g"
    if out["dbias"] is not None:
        # a block of at most T / 592 + 32 rows in fp32, then 64 bits
        l64 = dl.double()
        bound = (T // 592 + 50) * U32 * l64.abs().sum(0) + 1e-37
        assert bool(((out["dbias"].double() - l64.sum(0)).abs() <= bound).all()), "dbias"
    if out["dx"] is not None:
        ref, bound = dx_bound(dl, W)
        assert bool(((out["dx"].double() - ref).abs() <= bound).all()), "dx"


TOKENS, EXPERTS = [193, 300, 2000], [3, 24, 60, 130, 300]


@pytest.mark.parametrize("which", [(1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 1, 0), (1, 0, 1), (0, 1, 1), (1, 1, 1)])
@pytest.mark.parametrize("T", TOKENS)
@pytest.mark.parametrize("E", EXPERTS)
def test_each_set_of_outputs(T, E, which):
    x, W, dl = inputs(T, 320, E)
    check(x, W, dl, run(x, W, dl, *map(bool, which)))


@pytest.mark.parametrize("scale", [1e-30, 3e-34, 1e30, 1e34, 3e37])
@pytest.mark.parametrize("T", [300, 2000])
@pytest.mark.parametrize("E", EXPERTS)
def test_tiny_and_huge_gradients(T, E, scale):
    # at 3e37 sums of 2000 tokens would pass fp32's range
    x, W, dl = inputs(T, 192, E, scale)
    out = run(x, W, dl, dw=scale < 1e34, db=scale < 3e37)
    check(x, W, dl, out)


@pytest.mark.parametrize("T", TOKENS)
@pytest.mark.parametrize("E", [8, 24, 60, 130, 300])
def test_values_that_are_not_finite_show_and_stay(T, E):
    d = 192
    x, W, dl = inputs(T, d, E)
    dl[3, 2], dl[T - 5, 4] = math.inf, math.nan
    x[70, 11], x[T - 1, 13] = math.inf, math.nan
    W[17, 1], W[d - 1, E - 1] = math.nan, -math.inf
    out = run(x, W, dl)
    experts = torch.tensor([e in (2, 4) for e in range(E)], device=DEV)
    columns = torch.tensor([i in (11, 13) for i in range(d)], device=DEV)
    reached = experts[None, :] | columns[:, None]
    assert torch.equal(torch.isfinite(out["dw_g"]), ~reached)
    assert torch.equal(torch.isfinite(out["dbias"]), ~experts)
    rows = torch.tensor([t in (3, T - 5) for t in range(T)], device=DEV)
    columns = torch.tensor([i in (17, d - 1) for i in range(d)], device=DEV)
    assert torch.equal(torch.isfinite(out["dx"]), ~(rows[:, None] | columns[None, :]))


@pytest.mark.parametrize("T,d,E", [(300, 256, 12), (300, 128, 60), (2000, 320, 128), (515, 64, 300), (257, 64, 33)])
def test_operands_at_any_alignment_and_the_same_bits(T, d, E):
    x, W, dl = inputs(T, d, E)
    want = run(x, W, dl)
    s = MoEShape.of(T, d, E, 1, 64)
    ws = moe.workspace_bwd(s)
    for off in (1, 2, 3):
        dl1 = torch.empty(dl.numel() + off, device=DEV)[off:].view_as(dl).copy_(dl)
        W1 = torch.empty(W.numel() + off, device=DEV)[off:].view_as(W).copy_(W)
        bufs = [torch.full((n + off + 2,), 7.0, device=DEV) for n in (d * E, E)]
        dw, db = bufs[0][off:-2].view(d, E), bufs[1][off:-2]
        dx = torch.full((T + 1, d), 7.0, device=DEV).bfloat16()
        moe.moe_router_bwd(x, W1, dl1, s, ws, dw_g=dw, dbias=db, dx=dx[:T])
        assert torch.equal(dw, want["dw_g"]) and torch.equal(db, want["dbias"]) and torch.equal(dx[:T], want["dx"])
        for b in bufs:
            assert bool((b[:off] == 7).all()) and bool((b[-2:] == 7).all())
        assert bool((dx[T] == 7).all())
    assert moe.moe_check(ws) == moe.MOE_OK
