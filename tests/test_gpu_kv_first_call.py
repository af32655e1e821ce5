"""The first call of a process to each form of the KV-cache attention, which readies its kernels,
eager and captured into a graph: the same result either way, and as later calls give it."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FIRST = """
import sys, torch
sys.path.insert(0, "tests")
import kv_plain as P
from mixed_precision_weight_b200 import binding as dv
form, captured = sys.argv[1], sys.argv[2] == "captured"
lens, prefix = [100, 0, 7] * 8, {"short": 0, "long": 0, "joined": 100, "once": 6000}[form]
q = P.queries(24, 16, 128, seed=1)
pool, table, ptable = P.filled(24, 2, 128, lens, seed=2, prefix=prefix)
if form == "long":
    table = torch.cat([table, torch.full((24, 130), -1, dtype=torch.int32)], 1).contiguous()
c = dv.KvCache(*(pool[n].cuda() for n in ("k", "v", "ks", "vs")), table.cuda())
args = [q.cuda(), c, torch.tensor(lens, dtype=torch.int32, device="cuda")]
f = dv.dvssq_bss_attention_q8
if prefix:
    f, args = dv.dvssq_bss_attention_prefix, args + [ptable.cuda(), prefix]
if captured:
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = f(*args)
    g.replay()
else:
    out = f(*args)
assert torch.equal(out, f(*args))
ref = P.attention(q, pool, table, lens, ptable=ptable, prefix=prefix)
err = (out.double().cpu() - ref).norm(dim=-1)
assert (err <= (1e-3 if form == "once" else 1e-4) * ref.norm(dim=-1)).all()
assert dv.dvssq_device_error() == 0
print("ok")
"""


@pytest.mark.parametrize("how", ["eager", "captured"])
@pytest.mark.parametrize("form", ["short", "long", "joined", "once"])
def test_first_call(form, how):
    r = subprocess.run([sys.executable, "-c", FIRST, form, how], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stderr[-2000:]
