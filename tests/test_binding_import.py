"""The binding on a torch without the private reads of the current device and stream that its
KV-cache calls prefer: it imports, the host-only functions work, and the calls use the public ones."""
import os
import subprocess
import sys

import pytest
import torch

import kv_plain as P

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
WITHOUT = """
import torch
for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
from mixed_precision_weight_b200 import binding as dv
assert dv._current_device is torch.cuda.current_device
shape = dv.AttnShape(4, 16, 4, 256, 32768, 1.1, 12.0)
assert dv.dvssq_bss_attention_q8_workspace_size(shape) > 0
assert dv.dvssq_encode_workspace_size(dv.Shape.make(2560, 10240, 256, 16)) > 0
print("ok")
"""


def test_import_without_private_torch_names():
    r = subprocess.run([sys.executable, "-c", WITHOUT], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stderr[-2000:]


@pytest.mark.gpu
def test_calls_with_the_public_names(monkeypatch):
    from mixed_precision_weight_b200 import binding as dv
    lens = [100, 30]
    q = P.queries(2, 8, 64, seed=1).cuda()
    pool, table, _ = P.filled(2, 2, 64, lens, seed=2)
    c = dv.KvCache(*(pool[n].cuda() for n in ("k", "v", "ks", "vs")), table.cuda())
    lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    want = dv.dvssq_bss_attention_q8(q, c, lens)
    monkeypatch.setattr(dv, "_current_device", torch.cuda.current_device)
    monkeypatch.setattr(dv, "_current_stream", lambda index: torch.cuda.current_stream(index).cuda_stream)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [dv.dvssq_bss_attention_q8(q, c, lens), dv.dvssq_bss_attention_q8(q, c, lens, stream=side)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for x in got)
    assert dv.dvssq_device_error(clear=True) == 0
