"""GradList's marshalled entries against the tensors they stand for, on the CPU: a stand-in
for the operand checks accepts CPU tensors; nothing is launched."""

import pytest
import torch

import routing_dispatch_expert_softmax_b200 as moe
from routing_dispatch_expert_softmax_b200 import binding as B


class Checks:
    """What the native checks do, for CPU tensors; ``device`` is where they are said to lie."""

    device = 0

    def __init__(self, where):
        self.where, self.index = where, None

    def ptr(self, t, dtype, shape, name, optional=False):
        if t.dtype != dtype or not t.is_contiguous():
            raise ValueError(f"{self.where}: {name} must be contiguous")
        self.index = Checks.device
        return t.data_ptr()


@pytest.fixture
def cpu_list(monkeypatch):
    B.load_library()
    monkeypatch.setattr(B, "_Operands", Checks)
    monkeypatch.setattr(Checks, "device", 0)
    zeros = torch.zeros
    monkeypatch.setattr(torch, "zeros", lambda *a, **kw: zeros(*a, **dict(kw, device="cpu")))
    return moe.GradList


def entries(lst):
    return [(e.data, e.out, e.n, e.dtype, e.out_dtype) for e in lst._entries]


def expected(tensors):
    code = {torch.float32: 0, torch.bfloat16: 1}
    return [(t.data_ptr(), t.data_ptr(), t.numel(), code[t.dtype], code[t.dtype]) for t in tensors]


def test_entries_survive_a_refused_change(cpu_list):
    a, b = torch.zeros(8, 8), torch.zeros(6, 4)
    lst = cpu_list([a, b])
    want = entries(lst)
    assert want == expected([a, b])
    old_a, old_b = a.data, b.data
    a.data, b.data = torch.zeros(8, 8), torch.zeros(4, 6).t()  # b is refused, a alone would do
    for _ in range(2):
        with pytest.raises(ValueError, match="contiguous"):
            lst.operands("call")
    a.data, b.data = old_a, old_b
    lst.operands("call")
    assert entries(lst) == want
    a.data = torch.zeros(8, 8)
    lst.operands("call")
    assert entries(lst) == expected([a, b])


def test_entries_survive_a_refused_overlap(cpu_list):
    a, b, buf = torch.zeros(50), torch.zeros(50), torch.zeros(100)
    lst = cpu_list([a, b])
    old_a, old_b = a.data, b.data
    a.data, b.data = buf[:50], buf[40:90]
    with pytest.raises(ValueError, match="overlaps"):
        lst.operands("call")
    a.data, b.data = old_a, old_b
    lst.operands("call")
    assert entries(lst) == expected([a, b])


def test_entries_follow_a_tensor_of_other_length_in_the_same_place(cpu_list):
    buf = torch.zeros(64)
    a, b = torch.zeros(0), torch.zeros(8)
    a.data = buf
    lst = cpu_list([a, b])
    assert entries(lst)[0][2] == 64
    a.data = buf[:10]  # a step's smaller gradient gets the old one's memory
    lst.operands("call")
    assert entries(lst) == expected([a, b]) and entries(lst)[0][2] == 10
    a.data = buf[:32].view(4, 8)
    lst.operands("call")
    assert entries(lst)[0][2] == 32
    a.data = buf[:32].view(4, 8).t()  # not contiguous any more: refused, in the same place too
    with pytest.raises(ValueError, match="contiguous"):
        lst.operands("call")


def test_entries_follow_a_separate_out_of_other_length(cpu_list):
    g, buf = torch.zeros(20), torch.zeros(64)
    out = torch.zeros(0)
    out.data = buf[:20]
    lst = cpu_list([g], [out])
    out.data = buf[:12]
    with pytest.raises(ValueError, match="out 0 has 12 elements"):
        lst.operands("call")
    g.data = g.data[:12]
    lst.operands("call")
    assert entries(lst) == [(g.data_ptr(), buf.data_ptr(), 12, 0, 0)]


def test_entries_follow_a_dtype_in_the_same_place(cpu_list):
    buf = torch.zeros(64)
    t = buf[:16]
    lst = cpu_list([t])
    lst.grads[0] = buf.view(torch.bfloat16)[:16]
    lst.operands("call")
    assert entries(lst) == expected([lst.grads[0]])


def test_layouts():
    B.load_library()
    f = B._native.layouts
    a, b = torch.zeros(4, 6), torch.zeros(4, 6)
    assert f([a], None) == f([b], None) == f([a.view(24)], None)
    others = [a[:3], a.bfloat16(), a.int(), a.t()]
    assert len({f([t], None) for t in [a, *others]}) == 5
    assert f([a, b], None) == f([a], [b]) == f([a], None) + f([b], None)
    for args in (((), None), ([3], None), ([], [None]), ([], 3)):
        with pytest.raises(TypeError):
            f(*args)


def test_tensors_on_another_device_are_refused(cpu_list):
    # the list's workspace stays where it was made
    a = torch.zeros(8)
    lst = cpu_list([a])
    Checks.device = 1
    a.data = torch.zeros(8)
    for _ in range(2):
        with pytest.raises(ValueError, match="cuda:1.*cuda:0"):
            lst.operands("call")
    Checks.device = 0
    lst.operands("call")
    assert entries(lst) == expected([a])
