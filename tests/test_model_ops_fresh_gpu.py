"""Calls that must not depend on what the process called before."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

# each size is the first call of its kernel, with 48 KB of dynamic shared memory: rows by 256 threads
# of 12 vectors each, alone and in a cluster
FIRST_CALLS = """
import torch
import gradient_sync_zero_gb300 as dps
import model_reference as ref
for P, T, V, dtype in ((8, 64, 24576, torch.bfloat16), (8, 64, 12288, torch.float32),
                       (1, 200, 49152, torch.bfloat16), (1, 200, 24576, torch.float32)):
    g = torch.Generator(device="cuda").manual_seed(V)
    x = torch.randn(P, T, V, generator=g, device="cuda").to(dtype)
    tokens = torch.randint(0, V, (P, T), generator=g, device="cuda")
    want, _ = ref.logprob(x.double(), tokens, 1.0)
    old, adv = want.float(), torch.ones(P, T, device="cuda")
    logp, stats = torch.empty(P, T, device="cuda"), torch.empty(P, 4, device="cuda")
    dps.dp_policy_loss(x, tokens, old, adv, logp, stats)
    bound = ref.logprob_bound(x.double(), 1.0)
    assert ((logp.double() - want).abs() <= bound).all(), (V, dtype)
print("fine")
"""


def test_policy_loss_of_48_kb_rows_as_the_first_call():
    here = os.path.dirname(os.path.abspath(__file__))
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([os.path.dirname(here), here]))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS], env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "fine" in r.stdout, r.stderr[-2000:]
