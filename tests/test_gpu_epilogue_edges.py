"""The layer with its epilogue where its sums and its kept z are most exposed:
infinite tokens and overflowing operands under a ReLU that keeps z."""
import pytest
import torch

from test_gpu_epilogue import q  # noqa: F401

pytestmark = pytest.mark.gpu
INF = float("inf")


class Plain:
    """A layer whose weights take both signs in column 100, some of them exact in
    bf16 (the largest of their block: the fp32 scale itself), and whose adapter
    branch has the weight's sign in every row, so that an infinite element there
    gives one infinity and no difference of two."""

    def __init__(self, q, N, K, M, r, s):
        g = torch.Generator().manual_seed(N + K + M)
        mk = lambda *sh: torch.randn(*sh, generator=g)
        W = (mk(N, K) * 0.02).clamp(-0.4, 0.4)
        W[0::4, 100], W[1::4, 100] = 0.5, -0.5
        self.qw = q.nf4_quantize(W.bfloat16().cuda(), double_quant=False)
        self.W = q.nf4_dequantize(self.qw, bf16=False)
        self.x, self.A = mk(M, K).bfloat16().cuda(), (mk(r, K) * 0.05).bfloat16().cuda()
        self.sign = self.W[:, 100].sign()
        self.B = ((mk(N, r).abs() * 0.01 + 0.01).cuda() * self.sign[:, None]).bfloat16()
        self.alpha, self.s = s * r, s


@pytest.mark.parametrize("inf", [INF, -INF])
@pytest.mark.parametrize("N,K,M", [(264, 640, 5), (264, 640, 150), (4104, 320, 1100)])
def test_an_infinite_token_under_a_relu_that_keeps_z(q, N, K, M, inf):
    """Its z is the infinity that one pass gives, or NaN (where the two parts of the
    weight differ in sign); the other tokens keep their bits."""
    c = Plain(q, N, K, M, 16, 2.0)
    c.A[:, 100] = 2.0 ** -6
    c.x[3] = 0
    clean = q.qlora_linear_fwd_epilogue(c.qw, c.x, c.A, c.B, c.alpha, act="relu")
    c.x[3, 100] = inf
    h, u, z = q.qlora_linear_fwd_epilogue(c.qw, c.x, c.A, c.B, c.alpha, act="relu")
    want = torch.where(c.sign == 0, float("nan"), c.sign * inf)           # 0 times infinity
    one = q.qlora_linear_fwd_epilogue(c.qw, c.x, c.A, c.B, c.alpha)[2]    # z without a ReLU: one pass
    assert torch.equal(one[3].float().nan_to_num(nan=0.0), want.nan_to_num(nan=0.0))
    got = z[3].float()
    assert bool((got.isnan() | (got == want)).all()) and not bool(got.isnan().all())
    assert torch.equal(h[3].float().nan_to_num(nan=7.0), got.clamp_min(0).nan_to_num(nan=7.0))
    keep = [i for i in range(M) if i != 3]
    for a, b in zip((h, u, z), clean):
        assert torch.equal(a[keep], b[keep])


@pytest.mark.parametrize("s,x", [(4.0, 2.0 ** 127), (1.003, torch.finfo(torch.bfloat16).max)])
@pytest.mark.parametrize("M", [5, 150])
def test_adapter_activations_that_overflow_under_a_relu_that_keeps_z(q, M, s, x):
    """s u beyond fp32, and within fp32 but rounded to infinity in bf16: an infinity of
    the adapter's sign either way, as where z is not kept."""
    c = Plain(q, 264, 640, M, 16, s)
    c.x[3] = 0
    c.x[3, 100], c.A[:, 100] = x, 1.0
    h, u, z = q.qlora_linear_fwd_epilogue(c.qw, c.x, c.A, c.B, c.alpha, act="relu")
    at = c.sign != 0
    assert bool(u[3].isfinite().all()) and torch.equal(z[3, at].float(), c.sign[at] * INF)
    assert torch.equal(h[3, at].float(), (c.sign[at] * INF).clamp_min(0))


@pytest.mark.parametrize("M", [5, 150])
def test_scales_beyond_bf16_under_a_relu_that_keeps_z(q, M):
    """A block scale that bf16 rounds to infinity: its largest weight is infinite in the
    products, with its sign, as where z is not kept."""
    c = Plain(q, 264, 640, M, 16, 2.0)
    W = torch.zeros(264, 640)
    W[5, 128], W[9, 130] = 3.4e38, -3.4e38
    c.qw = q.nf4_quantize(W.cuda(), double_quant=False)
    c.x[:] = 1.0
    c.A[:] = 0
    for save in (False, True):
        h, _, z = q.qlora_linear_fwd_epilogue(c.qw, c.x, c.A, c.B, c.alpha, act="relu", save_z=save)
        assert bool((h[:, 5] == INF).all())
        assert not bool(h[:, [i for i in range(264) if i != 5]].any())
        if save:
            assert bool((z[:, 5] == INF).all()) and bool((z[:, 9] == -INF).all())
