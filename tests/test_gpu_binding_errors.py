"""An argument that fails inside a serving call (tensors without memory, as a tracer passes them) raises in Python: the
interpreter is whole afterwards. In a process of its own."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROGRAM = """
import torch
from torch._subclasses.fake_tensor import FakeTensorMode
import fp8_quant_memory_gb300 as fq

def inputs():
    i = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
    f = lambda *s: torch.zeros(*s, device="cuda")
    c = lambda *s: torch.zeros(*s, dtype=torch.uint8, device="cuda")
    h = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")
    cache = lambda: (c(3, 2, 16, 64), c(3, 2, 16, 64), f(3, 2, 16), f(3, 2, 16))
    return {
        "sample": lambda: (h(4, 100), f(4)),
        "paged_extend": lambda: (i(2, 3), i(2), i(2), i(9), i(3), 16, 5),
        "fp8_matmul": lambda: (c(2, 128), f(2, 1), c(8, 128), f(1, 1)),
        "paged_attention": lambda: (c(2, 4, 64), f(2, 4), *cache(), i(2, 1), i(2)),
        "qkv_norm_rope_append": lambda: (h(2, 512), h(64), h(64), f(2, 32), f(2, 32), torch.zeros(2, dtype=torch.int64, device="cuda"), *cache(), 4, 2),
    }

for name, make in inputs().items():
    call = getattr(fq, name)
    real = make()
    call(*real)
    with FakeTensorMode():
        fake = make()
    for _ in range(3):
        try:
            call(*fake)
        except RuntimeError as e:
            error = str(e)
        else:
            raise SystemExit(name + " took tensors without memory")
    call(*real)
    print(name, "raised:", error.splitlines()[0])
torch.cuda.synchronize()
assert fq.device_status(clear=True) == 0
"""


def test_errors_inside_a_call_are_raised(cuda_ok):
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    assert r.stdout.count("raised:") == 5, r.stdout
