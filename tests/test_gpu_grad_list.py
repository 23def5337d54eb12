"""A GradList whose tensors are replaced between calls, on the device."""

import math

import pytest
import torch

import routing_dispatch_expert_softmax_b200 as moe

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    moe.load_library()
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("n", [1, 10, 63])
def test_shorter_tensor_in_the_same_place(n):
    buf = torch.full((64,), 2.0, device=DEV)
    p = torch.empty(0, device=DEV)
    p.data = buf
    lst, norm = moe.GradList([p]), torch.empty(1, device=DEV)
    moe.moe_clip_grads(lst, math.inf, norm)
    assert norm.item() == 16.0
    p.data = buf[:n]
    moe.moe_clip_grads(lst, 1.0, norm)
    assert math.isclose(norm.item(), 2 * math.sqrt(n), rel_tol=1e-6)
    assert bool((buf[n:] == 2.0).all())  # what lies behind it is not the list's
    assert torch.allclose(buf[:n], torch.full_like(buf[:n], 1 / math.sqrt(n)), rtol=1e-5)


def test_refused_change_and_the_old_tensors_again():
    a, b = torch.full((8, 8), 1.0, device=DEV), torch.full((6, 4), 1.0, device=DEV)
    lst, norm = moe.GradList([a, b]), torch.empty(1, device=DEV)
    old_a, old_b = a.data, b.data
    other = torch.full((8, 8), 5.0, device=DEV)
    a.data, b.data = other, torch.zeros(4, 6, device=DEV).t()
    with pytest.raises(ValueError, match="contiguous"):
        moe.moe_clip_grads(lst, 1.0, norm)
    a.data, b.data = old_a, old_b
    moe.moe_clip_grads(lst, 1.0, norm)
    assert math.isclose(norm.item(), math.sqrt(88), rel_tol=1e-6)
    assert bool((other == 5.0).all()) and bool((a < 1.0).all()) and bool((b < 1.0).all())
