"""What the first call of a kind sets up: a process that only adapts weights
neither loads the 8-bit product's kernels nor depends on them, and the other way
round."""
import os
import subprocess
import sys

import pytest

import dora_adapter_factored_b200 as dora

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_nothing_is_set_up_by_loading(built_library):
    code = "import sys; sys.path.insert(0, sys.argv[1])\n" \
           "import dora_adapter_factored_b200 as dora\n" \
           "dora.dora_linear_i8_plan(600, 1024, 4096, 148, 33, 15)\n" \
           "assert dora.dora_kernels_prepared() == 0\nprint('OK')\n"
    res = subprocess.run([sys.executable, "-c", code, ROOT], capture_output=True, text=True,
                         timeout=300)
    assert res.returncode == 0 and "OK" in res.stdout, res.stdout + res.stderr


_CHILD = r"""
import sys
sys.path.insert(0, sys.argv[1])
import torch
import dora_adapter_factored_b200 as dora
bf = dict(dtype=torch.bfloat16, device="cuda")

def norm():
    W0, A, B = torch.ones(256, 512, **bf), torch.ones(64, 512, **bf), torch.ones(256, 64, **bf)
    n, _ = dora.dora_factored_norm(W0, A, B, 1.0)
    assert torch.allclose(n, torch.full_like(n, 65.0 * 512 ** 0.5), rtol=1e-3)

def rows():
    x = torch.ones(40, 512, **bf)
    q, s, _ = dora.dora_rmsnorm_quant(x, x[0].contiguous(), 1e-6)
    assert (q == 127).all()
    return q, s

def linear():
    q, s = rows()
    y = dora.dora_linear_i8(q, s, q, s, dtype=torch.float32)
    assert torch.allclose(y, torch.full_like(y, 512.0), rtol=1e-4)

calls = {"norm": (norm, 1), "rows": (rows, 0), "linear": (linear, 2)}
have = 0
for name in sys.argv[2].split(","):
    call, bit = calls[name]
    call()
    have |= bit
    assert dora.dora_kernels_prepared() == have, (name, dora.dora_kernels_prepared())
torch.cuda.synchronize()
assert dora.dora_get_device_status() == 0
print("OK")
"""


@pytest.mark.gpu
@pytest.mark.parametrize("order", ["norm,rows,linear", "rows,linear,norm"])
def test_each_kind_of_call_sets_up_its_own_kernels(order):
    res = subprocess.run([sys.executable, "-c", _CHILD, ROOT, order], capture_output=True,
                         text=True, timeout=300)
    assert res.returncode == 0 and "OK" in res.stdout, res.stdout + res.stderr
