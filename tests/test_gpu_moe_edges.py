"""The mixture of NF4 experts: routing of logits that are no numbers, every group
size, the products against the weights that the NF4 levels define, and the output
over the tokens."""
import pytest
import torch

from epilogue_ref import act64
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


@pytest.mark.parametrize("dq", [True, False])
@pytest.mark.parametrize("block", [64, 128])
@pytest.mark.parametrize("act", ["none", "silu"])
def test_against_the_nf4_levels(q, act, block, dq):
    """The kernel's table of levels is rounded, so against scale times level a product
    is off by 0.08% of a weight in the mean square (the table's rounding over the codes
    of normally distributed weights: 0.078% in blocks of 64, 0.083% of 128). In the
    2-norm, with the roundings independent of each other: gate, up and down by 0.00083
    each, gate times 1.1 for silu (the norm of act'(g) dg over that of act(g), g about
    normal: 0.616 / 0.597), and twice a bf16 rounding, 2^-8 / sqrt(3) at most in the
    mean. The length along the true result has no such noise: it is off by the table's
    fit (6.1e-5 per product in blocks of 128, 1e-6 of 64), and by the noise's share,
    0.0035 / sqrt(48 * 1024), five times over."""
    m = Moe(q, 48, 8, 2, 1024, 768, (dq, dq), (block, block))
    out, ids, w = q.nf4_moe_fwd(m.gate_up, m.down, m.x, m.router, 2, act)
    ids64, w64 = route64(m, True)
    assert torch.equal(ids.long(), ids64)
    W = q.nf4_dequantize(m.gate_up, bf16=False).double().view(8, 2 * 768, 1024)
    D = q.nf4_dequantize(m.down, bf16=False).double().view(8, 1024, 768)
    want = torch.zeros(48, 1024, dtype=torch.float64, device="cuda")
    for e in ids64.unique().tolist():
        tok, j = (ids64 == e).nonzero(as_tuple=True)
        gu = m.x[tok].double() @ W[e].T
        a = act64(gu[:, :768], act)[0] * gu[:, 768:]
        want.index_add_(0, tok, w64[tok, j][:, None] * (a @ D[e].T))
    got = out.double()
    rel = ((got - want).norm() / want.norm()).item()
    assert rel <= (0.00083 ** 2 * (1.1 ** 2 + 2) + 2 * 2.0 ** -16 / 3) ** 0.5, rel
    along = ((got * want).sum() / (want * want).sum()).item() - 1
    assert abs(along) <= 3 * (6.1e-5 if block == 128 else 1e-6) + 5 * 0.0035 / (48 * 1024) ** 0.5, along


@pytest.mark.parametrize("M,E,k,H,F", [(64, 32, 8, 256, 256), (5, 8, 2, 640, 320), (37, 4, 3, 1216, 1024)])
@pytest.mark.parametrize("with_residual", [False, True])
def test_the_output_over_the_tokens(q, M, E, k, H, F, with_residual):
    """out may be x, alone or with x as the residual; also captured, where each replay
    takes the output before as its tokens."""
    m = Moe(q, M, E, k, H, F)
    step = lambda x, out: q.nf4_moe_fwd(m.gate_up, m.down, x, m.router, k, residual=x if with_residual else None, out=out)
    want = [m.x]
    for _ in range(4):
        want.append(step(want[-1], None)[0])
    x = m.x.clone()
    for w in want[1:]:
        assert step(x, x)[0] is x and torch.equal(x, w)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(x, x)
    x.copy_(m.x)
    for w in want[1:]:
        g.replay()
        assert torch.equal(x, w)
    assert q.device_status() == q.NF4_OK
