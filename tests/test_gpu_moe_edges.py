"""The mixture of NF4 experts: routing of logits that are no numbers, and every
group size."""
import pytest
import torch

from test_gpu_moe import Moe, check_moe, q, route64  # noqa: F401

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


# groups of 4, 8 and 16 warps, each with scales in pairs (an even number of 8-bit
# ones to a row) and single
@pytest.mark.parametrize("M,E,k,H,F", [
    (40, 3, 2, 512, 512), (64, 12, 7, 576, 320), (20, 6, 2, 512, 640), (20, 6, 2, 512, 576),
    (4, 5, 3, 1152, 2560), (3, 8, 2, 2048, 2112),
])
def test_group_sizes(q, M, E, k, H, F):
    m = Moe(q, M, E, k, H, F)
    check_moe(q, m, q.nf4_moe_fwd(m.gate_up, m.down, m.x, m.router, k, residual=m.residual), "silu", True, m.residual)
    assert q.device_status() == q.NF4_OK
