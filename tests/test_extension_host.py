"""What of the package needs the Python extension of the operand checks, and which build of
it: each in a process of its own."""

import subprocess
import sys

import torch

from routing_dispatch_expert_softmax_b200 import binding as B

HIDE = """
import importlib, sys, types, torch
real = importlib.import_module
def fake(name, *a):
    if name.endswith('_operands'):
        if module is None: raise ImportError('no such file')
        return module
    return real(name, *a)
importlib.import_module = fake
module = None
import routing_dispatch_expert_softmax_b200 as moe
from routing_dispatch_expert_softmax_b200 import binding as B
def refused(*words):
    s = moe.MoEShape.of(1, 64, 1, 1, 64)
    try: moe.moe_combine_bwd(None, None, None, None, s)
    except RuntimeError as e:
        for w in ('_operands.so is not built',) + words: assert w in str(e), e
    else: assert False
"""


def run(code):
    p = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True)
    assert p.returncode == 0, p.stderr


def test_importing_the_package_loads_no_native_code():
    run("import sys\n"
        "import routing_dispatch_expert_softmax_b200 as moe\n"
        "assert not any(m.endswith('_operands') for m in sys.modules)\n"
        "maps = open('/proc/self/maps').read()\n"
        "assert '_operands.so' not in maps and 'libmoe_b200.so' not in maps\n")


def test_the_library_without_the_extension():
    run(HIDE + "lib = moe.load_library()\n"
               "assert lib.moe_version() >= 105 and B.moe_error_string(0)\n"
               "s = moe.MoEShape.of(4, 64, 8, 2, 64)\n"
               "assert moe.moe_workspace_size(s) > 0 and moe.moe_workspace_size_bwd(s) > 0\n"
               "refused()\n"
               "try: moe.GradList([torch.zeros(3)])\n"
               "except RuntimeError as e: assert '_operands.so is not built' in str(e), e\n"
               "else: assert False\n")


def test_an_extension_for_another_torch_is_refused_before_any_tensor():
    run(HIDE + "class Never:\n"
               "    def __init__(self, *a): raise SystemExit('made')\n"
               "module = types.SimpleNamespace(TORCH='2.11.0.dev20260101+cpu', Operands=Never)\n"
               "assert moe.load_library().moe_version() >= 105\n"
               "refused('2.11.0.dev20260101+cpu', str(torch.__version__))\n"
               "assert B._native is None\n")


def test_a_prerelease_torch_has_an_extension_too():
    for version in ("2.12.0a0+git1234567", "2.12.0.dev20260101", "2.11.0+vendor"):
        run(HIDE + f"torch.__version__ = {version!r}\n"
                   "class Operands:\n"
                   "    __slots__ = ('where',)\n"
                   "    def __init__(self, where): self.where = where\n"
                   "    def ptr(self, t, *a): raise KeyError('seen')\n"
                   f"module = types.SimpleNamespace(TORCH={version!r}, Operands=Operands)\n"
                   "try: moe.moe_combine_bwd(None, None, None, None, moe.MoEShape.of(1, 64, 1, 1, 64))\n"
                   "except KeyError: pass\n"
                   "else: assert False\n")


def test_the_built_extension_names_the_whole_version():
    B.load_library()
    assert B._native.TORCH == str(torch.__version__)


def test_a_bool_token_mask_is_checked_like_another():
    run("import torch\n"
        "import routing_dispatch_expert_softmax_b200 as moe\n"
        "from routing_dispatch_expert_softmax_b200 import binding as B\n"
        "moe.load_library()\n"
        "class O(B._native.Operands):\n"
        "    def ptr(self, t, dtype, shape, name, optional=False):\n"
        "        if name == 'token_mask': raise KeyError(t.dtype, dtype)\n"
        "        return 0\n"
        "B._Operands = O\n"
        "s = moe.MoEShape.of(4, 64, 8, 2, 64)\n"
        "for call in (lambda m: moe.moe_balance_loss(0, 0, 0, 0, 0, s, None, token_mask=m),\n"
        "             lambda m: moe.moe_gate_bwd(0, 0, 0, s, None, token_mask=m)):\n"
        "    for m, seen in ((torch.ones(4, dtype=torch.bool), torch.uint8), (torch.ones(4), torch.float32)):\n"
        "        try: call(m)\n"
        "        except KeyError as e: assert e.args == (seen, torch.uint8), e.args\n"
        "        else: assert False\n")
