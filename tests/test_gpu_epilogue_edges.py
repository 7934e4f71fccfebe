"""The layer with its epilogue where its sums and its kept z are most exposed:
infinite tokens and overflowing operands under a ReLU that keeps z, the
gradients against the formula at the unrounded z, the wider GEMM tiles, every
form of the streaming kernel, and offsets past 32 bits."""
import pytest
import torch

from epilogue_ref import ACT_EVAL, HALF_BF16, act64, backward64, check, forward64
from test_gpu_epilogue import ACTS, Case, check_forward, pick, q  # noqa: F401

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
    """Its z is the infinity that one pass gives, or NaN (where the weight's rest is zero
    or of the other sign); the other tokens keep their bits."""
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


def curvature(act):
    """Bounds of |act''| and |act'''| over all z (0 beyond |z| = 14 to 1e-15), from a
    fine grid; 1% for what lies between its points."""
    z = torch.linspace(-14, 14, 280001, dtype=torch.float64, requires_grad=True)
    d2, = torch.autograd.grad(act64(z, act)[1].sum(), z, create_graph=True)
    d3, = torch.autograd.grad(d2.sum(), z)
    return 1.01 * float(d2.detach().abs().max()), 1.01 * float(d3.abs().max())


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("N,K,M,r,dq,block", [
    (264, 640, 5, 16, True, 64), (136, 1152, 16, 64, True, 128), (264, 640, 17, 16, True, 64),
    (520, 1152, 300, 128, False, 128), (4104, 640, 1100, 16, True, 64),
])
def test_gradients_at_the_unrounded_z(q, N, K, M, r, dq, block, act):
    """Forward and backward together against the formula whose z is never rounded.
    The kept z is off by d = (the forward's own error) + half a bf16 step of z, so
    act(z) in dmul is off by |act'| d + max|act''| d^2 / 2 and act'(z) in dz by
    |act''| d + max|act'''| d^2 / 2: element by element that may be more than dz's own
    rounding. (A ReLU's sign survives the rounding of z, so act' errs only where |z|
    is within the forward's error.)"""
    c = Case(q, N, K, M, r, dq, block)
    W = q.nf4_dequantize(c.qw, bf16=True)
    for use in ("b", "bm"):
        bias, mul, _ = pick(c, use)
        h, u, z = q.qlora_linear_fwd_epilogue(c.qw, c.x, c.A, c.B, c.alpha, bias, act, mul)
        got = q.qlora_linear_bwd_epilogue(c.qw, c.x, c.A, c.B, c.alpha, c.dH, z, act, mul, u=u, need_dbias=True)
        exact = act == "relu"
        _, z64, _, tol = forward64(c.operand(q, exact), c.x, c.A, c.B, c.s, bias, act, mul, None, exact)
        want = backward64(W, c.x, c.A, c.B, c.s, c.dH, z64, act, mul, u)
        d = tol + HALF_BF16 * (z64.abs() + tol)
        dH, ma = c.dH.double().abs(), 1.0 if mul is None else mul.double().abs()
        if act == "none":
            e0, e1 = d, torch.zeros_like(d)
        elif act == "relu":
            e0, e1 = d, (z64.abs() <= tol).double()
        else:
            top2, top3 = curvature(act)
            zz = z64.detach().requires_grad_()
            d2, = torch.autograd.grad(act64(zz, act)[1].sum(), zz)
            e0 = act64(z64, act)[1].abs() * d + top2 / 2 * d * d
            e1 = d2.abs() * d + top3 / 2 * d * d
        # (evaluated at the kept z, which is up to d larger)
        ev = 0.0 if act in ("none", "relu") else ACT_EVAL
        ez = dH * ma * (e1 + ev * d)                                # of dz before its rounding
        er = ez * (1 + HALF_BF16)
        A, B, x = (t.double().abs() for t in (c.A, c.B, c.x))
        s = abs(c.s)
        # (rounding of s v, and the fp32 sums, act on the error's own share too)
        more = 1 + HALF_BF16 + (N + K + M + r + 16) * 2.0 ** -23
        eb = (er @ B) * more
        extra = dict(dX=(er @ W.double().abs() + s * eb @ A) * more, dA=s * (eb.T @ x) * more,
                     dB=s * (er.T @ u.double().abs()) * more, dbias=ez.sum(0) * more,
                     dmul=dH * (e0 + ev * d))
        for name, t in zip(("dX", "dA", "dB", "dbias", "dmul"), got):
            if t is not None:
                check(name, t, want[name][0], want[name][1] + extra[name])


# 192-wide tiles in one round of CTA pairs, and whole 256-wide tiles in one round
# (the other shapes of the tests take 128-wide tiles, or split 256-wide ones)
@pytest.mark.parametrize("act", ["relu", "silu", "gelu"])
@pytest.mark.parametrize("N,M", [(4104, 513), (5120, 517)])
def test_wider_tiles(q, N, M, act):
    c = Case(q, N, 320, M, 24)
    for use in ("bmr", ""):
        bias, mul, residual = pick(c, use)
        for save in (True, False):
            h, u, z = q.qlora_linear_fwd_epilogue(c.qw, c.x, c.A, c.B, c.alpha, bias, act, mul, residual, save_z=save)
            check_forward(q, c, act, use, h, u, z)
    h, u, z = q.qlora_linear_fwd_epilogue(c.qw, c.x, c.A, c.B, c.alpha, c.bias, act, c.mul)
    got = q.qlora_linear_bwd_epilogue(c.qw, c.x, c.A, c.B, c.alpha, c.dH, z, act, c.mul, u=u, need_dbias=True)
    want = backward64(q.nf4_dequantize(c.qw, bf16=True), c.x, c.A, c.B, c.s, c.dH, z, act, c.mul, u)
    for name, t in zip(("dX", "dA", "dB", "dbias", "dmul"), got):
        check(name, t, *want[name])
    inplace = c.residual.clone()
    h, _, _ = q.qlora_linear_fwd_epilogue(c.qw, c.x, c.A, c.B, c.alpha, c.bias, act, c.mul, inplace, h=inplace)
    assert torch.equal(h, q.qlora_linear_fwd_epilogue(c.qw, c.x, c.A, c.B, c.alpha, c.bias, act, c.mul, c.residual)[0])
    assert q.device_status() == q.NF4_OK


# every chunk width of the streaming kernel (1 to 5 blocks, from K), up to 8 and up to 16
# tokens, with half tiles (24 rows) and without (4608 rows: whole tiles on 144 CTAs)
@pytest.mark.parametrize("K", [640, 1152, 2560, 4096, 5120])
@pytest.mark.parametrize("N,M", [(24, 3), (24, 13), (4608, 3), (4608, 13)])
def test_every_chunk_width_of_few_tokens(q, N, M, K):
    c = Case(q, N, K, M, 16)
    h, u, z = q.qlora_linear_fwd_epilogue(c.qw, c.x, c.A, c.B, c.alpha, c.bias, "silu", c.mul, c.residual)
    check_forward(q, c, "silu", "bmr", h, u, z)
    assert q.device_status() == q.NF4_OK


def test_offsets_past_32_bits(q):
    """More than 2^31 elements in h, z, mul, the residual and the gradients: rows at the
    start, around element 2^31 and at the end against the formula, dbias over all rows."""
    N, K, M, r = 28672, 128, 75009, 8
    c = Case(q, N, K, 32, r)
    g = torch.Generator(device="cuda").manual_seed(5)
    mk = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=torch.bfloat16)
    c.M, c.x, c.mul, c.residual, c.dH = M, mk(M, K), mk(M, N), mk(M, N), mk(M, N)
    W = q.nf4_dequantize(c.qw, bf16=True)
    at = 2 ** 31 // N
    for act in ("silu", "relu"):
        h, u, z = q.qlora_linear_fwd_epilogue(c.qw, c.x, c.A, c.B, c.alpha, c.bias, act, c.mul, c.residual)
        dX, _, _, dbias, dmul = q.qlora_linear_bwd_epilogue(c.qw, c.x, c.A, c.B, c.alpha, c.dH, z, act, c.mul, u=u,
                                                            need_dbias=True, grad_dtype=torch.float32)
        for i in (0, at - 20, M - 40):
            s = slice(i, i + 40)
            p = Case.__new__(Case)
            p.__dict__.update(c.__dict__, M=M, x=c.x[s], mul=c.mul[s], residual=c.residual[s])
            check_forward(q, p, act, "bmr", h[s], u[s], z[s])
            want = backward64(W, c.x[s], c.A, c.B, c.s, c.dH[s], z[s], act, c.mul[s], u[s])
            check("dX", dX[s], *want["dX"])
            check("dmul", dmul[s], *want["dmul"])
        total, size = torch.zeros(N, dtype=torch.float64, device="cuda"), torch.zeros(N, dtype=torch.float64, device="cuda")
        err = torch.zeros_like(total)
        for i in range(0, M, 5000):
            s = slice(i, i + 5000)
            z64 = z[s].double()
            dz = c.dH[s].double() * act64(z64, act)[1] * c.mul[s].double()
            total += dz.sum(0)
            size += dz.abs().sum(0)
            if act == "silu":
                err += (c.dH[s].double() * c.mul[s].double() * z64.abs().clamp_min(1)).abs().sum(0) * ACT_EVAL
            del z64, dz
        # fp32 sums of at most M terms in some order
        check("dbias", dbias, total, err + (M + 4) * 2.0 ** -24 * size, out_half=2.0 ** -24)
        del h, u, z, dX, dbias, dmul
    assert q.device_status() == q.NF4_OK
