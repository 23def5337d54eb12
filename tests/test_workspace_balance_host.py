"""Workspace sizes of the balance loss, on the CPU."""

import pytest

import routing_dispatch_expert_softmax_b200 as moe


def shape(T, E, d=64):
    return moe.MoEShape.of(T, d, E, min(E, 4), 64)


def test_balance_loss_asks_for_its_own_part():
    # partial sums of at most 592 blocks and each sequence: megabytes, whatever the tokens
    n = moe.moe_workspace_size_balance(shape(262144, 256))
    assert 0 < n <= 256 + 600 * (8 * 256 + 8) + 4096
    assert n < moe.moe_workspace_size_bwd(shape(262144, 256)) // 100


@pytest.mark.parametrize("T", [0, 1, 64, 65, 4095, 262144])
@pytest.mark.parametrize("E", [1, 8, 130, 1024])
@pytest.mark.parametrize("S", [1, 7, 65535])
def test_the_common_workspace_holds_it(T, E, S):
    assert 0 < moe.moe_workspace_size_balance(shape(T, E), S) <= moe.moe_workspace_size_bwd(shape(T, E), S)


def test_invalid_arguments():
    for s, S in ((shape(8, 8), 0), (shape(8, 8), 65536), (shape(8, 8, d=65), 1), (shape(8, 2000), 1)):
        assert moe.moe_workspace_size_balance(s, S) == 0
        with pytest.raises(moe.MoEError):
            moe.workspace_balance(s, S)
