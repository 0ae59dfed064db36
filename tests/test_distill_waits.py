"""distill_loss where the waits of a row's blocks for one another run out: the call reports it, and no block leaves its cluster while another
may still store to it. The library is built so that every second block does not wait; the results of its calls are anything."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CALLS = """
import sys
import torch
from smc_reweight_resample_gb300 import _binding as B
B.load(sys.argv[1])
seen = set()
for R, V, K, dtype in ((300, 24_000, 40, torch.float32), (64, 43_000, 8, torch.bfloat16), (300, 128_256, 64, torch.bfloat16),
                       (40, 128_256, 200, torch.float32), (3, 819_000, 5, torch.bfloat16)):
    z = torch.randn(R, V, device="cuda").to(dtype)
    values, tokens = torch.log_softmax(z.float(), 1).topk(K, 1)
    tokens = tokens.int()
    tokens[::3] = -1
    weight = torch.ones(R, device="cuda")
    weight[1::4] = 0
    for rest in (False, True):
        for with_loss in (False, True):
            ws = B.Workspace(B.OP_DISTILL_LOSS, 1)
            for _ in range(4):
                B.distill_loss(z, tokens, values, V, rest=rest, weight=weight, with_loss=with_loss, ws=ws)
            seen.add(B.check_status(ws))
            assert B.check_status(ws) == 0
# the loss alone and rows of one block wait for nobody, and the context is as it was
ws = B.Workspace(B.OP_DISTILL_LOSS, 1)
z = torch.randn(5, 1000, device="cuda")
values, tokens = torch.log_softmax(z, 1).topk(1000, 1)
loss, grad = B.distill_loss(z, tokens[:, :200].int(), values[:, :200].contiguous(), 1000, ws=ws)
alone = B.distill_loss(z, tokens[:, :200].int(), values[:, :200].contiguous(), 1000, grad=False, ws=ws)[0]
assert B.check_status(ws) == 0 and bool(torch.isfinite(loss).all()) and torch.allclose(loss, alone, atol=1e-4)
print("statuses", sorted(seen))
assert B.ERR_TIMEOUT in seen and seen <= {0, B.ERR_TIMEOUT, B.ERR_NONFINITE}
"""


def test_waits_that_run_out(smcsd):
    from smc_reweight_resample_gb300 import build

    folder = os.path.join(build.BUILD, "impatient")
    lib = build.build(extra_flags=("-DSMCSD_IMPATIENT",), out=os.path.join(folder, "libsmcsd_impatient.so"), objdir=folder)
    r = subprocess.run([sys.executable, "-c", CALLS, lib], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-2000:]
