"""The mixture of NF4 experts: routing of logits that are no numbers."""
import pytest
import torch

from test_gpu_moe import Moe, q, route64  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("nan,low", [(1, 4), (4, 1)])
@pytest.mark.parametrize("E", [6, 40])
def test_a_nan_logit_ranks_as_minus_infinity(q, E, nan, low):
    """NaN counts as minus infinity and ties go to the lower index, so of a NaN and a
    minus infinity the lower index comes first, whichever it is."""
    m = Moe(q, 3, E, 6, 128, 64)
    m.x[:, 0] = 1.0
    m.router[nan, 0], m.router[low, 0] = float("nan"), -float("inf")
    for dead in range(6, E):
        m.router[dead, 0] = -float("inf")
    _, ids, w = q.nf4_moe_fwd(m.gate_up, m.down, m.x, m.router, 6)
    assert torch.equal(ids.long(), route64(m, True)[0])
    assert ids[:, 4:].tolist() == [[1, 4]] * 3
    assert bool(w.isnan().all())
