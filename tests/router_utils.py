"""Calls of moe_router_bwd on poisoned outputs and scratch, and what they may be off by.

u = 2^-24 is half a step of fp32."""

import math

import torch

import routing_dispatch_expert_softmax_b200 as moe
from routing_dispatch_expert_softmax_b200.binding import MoEShape

from parity_utils import U32

DEV = "cuda"
BF16 = 2.0 ** -8


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
    less than 2^-137, half of its lowest step) and the product of the second parts (2^-20)
    come to 2^-19 of a term at most.  The tensor cores may cut at each MMA, 2u of the sum
    and 2u of what is added: 12 MMAs of 16 for each 64 experts (tf32: 24 of 8), and 20 adds
    behind them."""
    E = W.shape[1]
    l64, W64 = dl.double(), W.double()
    ref, mag = l64 @ W64.t(), l64.abs() @ W64.abs().t()
    low = 2.0 ** -38 * (l64.abs().amax(1)[:, None] * W64.abs().sum(1)[None]
                        + l64.abs().sum(1)[:, None] * W64.abs().amax(1)[None])
    low += 2.0 ** -137 * (W64.abs().sum(1)[None] + l64.abs().sum(1)[:, None])
    n = 24 * -(-E // 64) + 20
    return ref, BF16 * ref.abs() + (1 + BF16) * ((2.0 ** -19 + 4 * n * U32) * mag + low) + 1e-37


def dw_bound(x, dl):
    """(dw_g in 64 bits, what the call may be off by).  The products are exact.  At most 128
    tokens' sums stay on the tensor cores (few tokens: 192), 24 MMAs (36) that may each cut
    2u of the sum and 2u of what they add.  Then come adds that round, u of a sum that grows
    evenly, half of its end on average: one for each 128 tokens of a range, and one for each
    of the n partials, in a row below 16 and else in eight rows of n / 8 which 7 more join;
    148 ranges of three parts at most, n / 16 + 12 of them."""
    T = x.shape[0]
    n = 4 * (24 if T > 192 else 36) + T // 256 + 1 + 40
    x64, l64 = x.double(), dl.double()
    return x64.t() @ l64, n * U32 * (x64.abs().t() @ l64.abs()) + 1e-37
