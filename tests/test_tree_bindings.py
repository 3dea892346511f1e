"""The Python bindings under a torch without its private allocation (CPU)."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LOST = {"name": "del torch._C._dynamo.guards._empty_strided_cuda",
        "module": "del torch._C._dynamo"}
BODY = """
import types, torch
{lose}
from head_latent_attention_qkv_gb300 import api
h = types.SimpleNamespace(device=torch.device("cpu"), device_index=0)
for shape, dtype in (((3, 5), torch.float16), ((7,), torch.int32), ((2, 0), torch.int32)):
    t = api._new(h, shape, dtype)
    assert t.shape == shape and t.dtype is dtype and t.is_contiguous()
"""


@pytest.mark.parametrize("what", LOST)
def test_bindings_import_and_allocate_without_the_private_name(what):
    r = subprocess.run([sys.executable, "-c", BODY.format(lose=LOST[what])], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
