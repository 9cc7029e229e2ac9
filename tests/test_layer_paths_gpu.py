"""Paths of the dense layer, the orthogonalisation and the Muon step that the shapes of
test_layer_gpu.py do not take, and what each leaves alone."""
import pytest
import torch

import gradient_sync_zero_gb300 as dps
from test_layer_gpu import BF, gen, no_timeouts   # noqa: F401

pytestmark = pytest.mark.gpu

# in shared memory, thin both ways, on the tensor cores with whole vectors and without
KINDS = [(61, 64), (131, 48), (40, 5000), (5000, 41), (320, 264), (264, 328), (300, 260)]


def muon_case(shapes, P=3, seed=30, gap=77):
    """A plan with a tensor that is no matrix between any two, and its state."""
    sizes = [s for r, c in shapes for s in (r * c, gap)]
    plan = dps.Plan(sizes, 1 << 17, P)
    g = gen(seed)
    mean, master, buf = (torch.randn(plan.L, generator=g) * s for s in (1e-3, 0.02, 1e-3))
    params = torch.randn(P, plan.stride, generator=g).to(BF)
    return plan, {2 * i: s for i, s in enumerate(shapes)}, (mean, master, buf, params)


def test_muon_writes_nothing_after_a_timeout():
    """The bit that a product's wait leaves when it gives up: sums that were not waited for must not
    reach the weights, in no kernel of the step."""
    plan, matrices, state = muon_case(KINDS)
    ws, m = plan.new_workspace(), dps.Muon(plan, matrices)
    at = dps.workspace_result_offsets()[3]
    status = ws[at:at + 4].view(torch.int32)
    status.fill_(dps.DP_STATUS_TIMEOUT)
    dev = [t.cuda() for t in state]
    dps.dp_muon_step(m, ws, m.new_workspace(), *dev)
    for a, b in zip(dev, state):
        assert torch.equal(a.cpu().view(torch.int16), b.view(torch.int16))
    with pytest.raises(dps.DPError) as e:
        dps.dp_read_norm(plan, ws)
    assert e.value.code == dps.DP_ETIMEOUT and int(status) == dps.DP_STATUS_TIMEOUT
    status.zero_()
    dps.dp_muon_step(m, ws, m.new_workspace(), *dev)
    assert int(status) == 0
    for t, (r, c) in matrices.items():
        o = plan.tensor(t)[1]
        assert (dev[1][o:o + r * c].cpu() != state[1][o:o + r * c]).float().mean() > 0.9
