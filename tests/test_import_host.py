"""The package on a torch that lacks the private lookup of the current stream:
it imports, its host-side functions work, and streams come from the public
call."""
from __future__ import annotations

import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import types
import torch
if hasattr(torch._C, "_cuda_getCurrentRawStream"):
    del torch._C._cuda_getCurrentRawStream
import packed_xor_popcount_amd as bnn
import packed_xor_popcount_amd.fold
assert bnn.words(65) == 2 and bnn.f8_row_bytes(129) == 256
try:
    bnn.layernorm_fwd(torch.zeros(2, 3))
except TypeError:
    pass
else:
    raise AssertionError("a CPU tensor was taken")
torch.cuda.current_stream = lambda device=None: types.SimpleNamespace(cuda_stream=1000 + torch.device("cuda", device).index
                                                                      if isinstance(device, int) else 1000 + device.index)
for index in (0, 3):
    tensor = types.SimpleNamespace(device=torch.device("cuda", index))
    assert bnn._stream(tensor) == 1000 + index
print("fine")
"""


def test_without_the_private_stream_lookup():
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("fine"), r.stderr[-2000:]
