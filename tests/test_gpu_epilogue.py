"""The QLoRA layer with its epilogue (bias, activation, mul, residual), forward
and backward, against the formulas in 64 bits.

The oracle takes the operand the products use: the dequantised weight rounded to
bf16, or, for at most 16 tokens and rank at most 64 (the streaming kernel), the
block scale times the level rounded to bf16, or, for a ReLU that keeps z, the
fp32 weight. Every bound is worked out in
epilogue_ref.py from the roundings on the way."""
import pytest
import torch

import workloads
from epilogue_ref import ACT_EVAL, ACT_SLOPE, HALF_BF16, act64, backward64, check, forward64

pytestmark = pytest.mark.gpu
ACTS = ["none", "relu", "silu", "gelu_tanh", "gelu"]


@pytest.fixture(scope="module")
def q():
    import bit_nf4_quantized_05_b200 as mod
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    return mod


class Case:
    def __init__(self, q, N, K, M, r, dq=True, block=64, seed=0, alpha=32.0):
        w = workloads.LayerWorkload("t", N, K, M, r, alpha, 0.02, dq, 7000 + seed + N + M)
        inp = workloads.make_inputs(w)
        self.N, self.K, self.M, self.r, self.alpha = N, K, M, r, alpha
        self.s = alpha / r
        self.qw = q.nf4_quantize(inp["W0"].cuda(), double_quant=dq, block_size=block)
        self.x, self.A, self.B, self.dH = (inp[k].cuda() for k in ("x", "A", "B", "dY"))
        g = torch.Generator().manual_seed(11 + seed)
        mk = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).cuda()
        self.bias, self.mul, self.residual = mk(N), mk(M, N), mk(M, N)

    def operand(self, q, exact=False):
        """W~ as the products of the forward use it (exact: to 2^-17)."""
        if exact:
            return q.nf4_dequantize(self.qw, bf16=False)
        if self.M > 16 or self.r > 64:
            return q.nf4_dequantize(self.qw, bf16=True)
        qw = self.qw
        codes = torch.stack((qw.codes >> 4, qw.codes & 15), -1).view(self.N, self.K)
        levels = q_levels().bfloat16().double().cuda()
        nb = self.N * self.K // qw.block_size
        if qw.double_quant:
            c = (qw.absmax_c / 127.0).repeat_interleave(256)[:nb]
            s = qw.absmax_q8[:nb].float() * c
        else:
            s = qw.absmax[:nb]
        return levels[codes.long()] * s.double().repeat_interleave(qw.block_size).view(self.N, self.K)


def q_levels():
    from perf.operators import LEVELS
    return torch.tensor(LEVELS)


def pick(c, use):
    return (c.bias if "b" in use else None, c.mul if "m" in use else None, c.residual if "r" in use else None)


def check_forward(q, c, act, use, h, u, z):
    bias, mul, residual = pick(c, use)
    exact = act == "relu" and z is not None
    u64, z64, h64, tol = forward64(c.operand(q, exact), c.x, c.A, c.B, c.s, bias, act, mul, residual, exact)
    ma = 1.0 if mul is None else mul.double().abs()
    slope = 1.0 if act in ("none", "relu") else ACT_SLOPE
    ev = 0.0 if act in ("none", "relu") else ACT_EVAL
    th = (slope * tol + ev * (act64(z64, act)[0].abs() + tol)) * ma
    check("h", h, h64, th + 2.0 ** -22 * h64.abs())
    if z is not None:
        check("z", z, z64, tol)
    if u is not None:
        mag = c.x.double().abs() @ c.A.double().abs().T
        check("u", u, u64, (c.K + 4) * 2.0 ** -23 * mag, out_half=2.0 ** -24)


# streaming path; its rank limit; one tile; ragged rows and columns; several
# reduction steps of the adapter; more 256-wide tiles than CTA pairs (split tiles)
SHAPES = [
    (264, 640, 1, 16, True, 64), (136, 1152, 16, 64, True, 128), (8, 64, 5, 8, False, 64),
    (1032, 5120, 3, 24, True, 64),
    (264, 640, 16, 72, True, 64), (264, 640, 17, 16, True, 64), (520, 1152, 300, 128, False, 128),
    (8, 128, 129, 8, True, 128), (4104, 640, 1100, 16, True, 64), (2056, 320, 513, 40, False, 64),
]


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("N,K,M,r,dq,block", SHAPES)
def test_forward(q, N, K, M, r, dq, block, act):
    c = Case(q, N, K, M, r, dq, block)
    for use in ("b", "mr", "bmr", ""):
        bias, mul, residual = pick(c, use)
        h, u, z = q.qlora_linear_fwd_epilogue(c.qw, c.x, c.A, c.B, c.alpha, bias, act, mul, residual)
        check_forward(q, c, act, use, h, u, z)
    h, u, z = q.qlora_linear_fwd_epilogue(c.qw, c.x, c.A, c.B, c.alpha, c.bias, act, c.mul, c.residual, save_u=False,
                                          save_z=False)
    assert u is None and z is None
    check_forward(q, c, act, "bmr", h, None, None)
    assert q.device_status() == q.NF4_OK


@pytest.mark.parametrize("M", [4, 200])
def test_without_an_epilogue_it_is_the_layer(q, M):
    c = Case(q, 264, 640, M, 16)
    h, u, z = q.qlora_linear_fwd_epilogue(c.qw, c.x, c.A, c.B, c.alpha)
    h0, u0 = q.qlora_linear_fwd(c.qw, c.x, c.A, c.B, c.alpha)
    assert torch.equal(h, h0) and torch.equal(u, u0) and torch.equal(z, h0)
    g = q.qlora_linear_bwd_epilogue(c.qw, c.x, c.A, c.B, c.alpha, c.dH, u=u)
    g0 = q.qlora_linear_bwd(c.qw, c.x, c.A, c.B, c.alpha, c.dH, u=u)
    assert all(torch.equal(a, b) for a, b in zip(g, g0)) and g[3] is None and g[4] is None


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("N,K,M,r,dq,block", SHAPES)
def test_backward(q, N, K, M, r, dq, block, act):
    c = Case(q, N, K, M, r, dq, block)
    W = q.nf4_dequantize(c.qw, bf16=True)
    for use, gd in (("b", torch.bfloat16), ("bm", torch.float32), ("m", torch.bfloat16)):
        bias, mul, _ = pick(c, use)
        h, u, z = q.qlora_linear_fwd_epilogue(c.qw, c.x, c.A, c.B, c.alpha, bias, act, mul)
        got = q.qlora_linear_bwd_epilogue(c.qw, c.x, c.A, c.B, c.alpha, c.dH, z, act, mul, u=u,
                                          need_dbias="b" in use, grad_dtype=gd)
        want = backward64(W, c.x, c.A, c.B, c.s, c.dH, z, act, mul, u)
        half = HALF_BF16 if gd == torch.bfloat16 else 2.0 ** -24
        names = ("dX", "dA", "dB", "dbias", "dmul")
        for name, t in zip(names, got):
            if t is None:
                assert name == ("dbias" if "b" not in use else "dmul")
                continue
            check(name, t, *want[name], out_half=HALF_BF16 if name in ("dX", "dmul") else half)
            # the roundings are independent: far inside their worst case together
            ref = want[name][0]
            rel = ((t.double() - ref).norm() / ref.norm().clamp_min(1e-30)).item()
            assert rel <= 2 * HALF_BF16, (name, rel)
        # u recomputed, and no dX wanted
        again = q.qlora_linear_bwd_epilogue(c.qw, c.x, c.A, c.B, c.alpha, c.dH, z, act, mul, need_dX=False,
                                            need_dbias="b" in use, grad_dtype=gd)
        assert again[0] is None and torch.equal(again[1], got[1])
        check("dB", again[2], *want["dB"], out_half=half)
    assert q.device_status() == q.NF4_OK


def test_fp32_gradients_are_the_sums_that_bf16_rounds(q):
    c = Case(q, 264, 640, 300, 16)
    h, u, z = q.qlora_linear_fwd_epilogue(c.qw, c.x, c.A, c.B, c.alpha, c.bias, "silu", c.mul)
    a = q.qlora_linear_bwd_epilogue(c.qw, c.x, c.A, c.B, c.alpha, c.dH, z, "silu", c.mul, u=u, need_dbias=True)
    b = q.qlora_linear_bwd_epilogue(c.qw, c.x, c.A, c.B, c.alpha, c.dH, z, "silu", c.mul, u=u, need_dbias=True,
                                    grad_dtype=torch.float32)
    assert torch.equal(a[0], b[0]) and torch.equal(a[4], b[4])
    for i in (1, 2, 3):
        assert b[i].dtype == torch.float32 and torch.equal(a[i], b[i].bfloat16())


@pytest.mark.parametrize("M", [6, 150])
@pytest.mark.parametrize("act", ACTS)
def test_extreme_pre_activations(q, M, act):
    """z from the bias alone (x = 0): the largest values of the type, infinities
    and NaN keep to their own column, forward and backward."""
    c = Case(q, 264, 640, M, 16)
    x = torch.zeros_like(c.x)
    big = torch.finfo(torch.bfloat16).max
    vals = [0.0, -0.0, 1e-30, -1e-30, 88.0, -88.0, 104.0, -104.0, 1e4, -1e4, 1e18, -1e18, big, -big,
            float("inf"), float("-inf"), float("nan")]
    bias = torch.zeros(264)
    bias[:len(vals)] = torch.tensor(vals)
    bias = bias.to(torch.bfloat16).cuda()
    h, u, z = q.qlora_linear_fwd_epilogue(c.qw, x, c.A, c.B, c.alpha, bias, act, residual=c.residual)
    fin = torch.isfinite(bias)
    a64 = act64(bias.double()[fin], act)[0]
    check("h", h[:, fin], a64 + c.residual.double()[:, fin], ACT_EVAL * a64.abs() + 2.0 ** -23 * c.residual.double()[:, fin].abs())
    nan = len(vals) - 1
    assert bool(h[:, nan].isnan().all())
    assert bool((h[:, nan - 2] == float("inf")).all())            # act(inf) = inf
    if act == "relu":
        assert torch.equal(h[:, nan - 1], c.residual[:, nan - 1])
    _, dA, dB, dbias, _ = q.qlora_linear_bwd_epilogue(c.qw, x, c.A, c.B, c.alpha, c.dH, z, act, u=u,
                                                      need_dX=False, need_dbias=True)
    da = act64(bias.double(), act)[1]
    want = c.dH.double().sum(0) * da
    tol = (ACT_EVAL * 2 + 2.0 ** -18) * c.dH.double().abs().sum(0)
    check("dbias", dbias[fin], want[fin], tol[fin])


@pytest.mark.parametrize("N,M", [(520, 9), (520, 200), (4104, 1100)])
def test_residual_and_mul_updated_in_place(q, N, M):
    c = Case(q, N, 640, M, 16)
    want, _, _ = q.qlora_linear_fwd_epilogue(c.qw, c.x, c.A, c.B, c.alpha, c.bias, "silu", c.mul, c.residual)
    for t in (c.residual.clone(), c.mul.clone()):
        kw = dict(mul=c.mul, residual=c.residual)
        kw["residual" if torch.equal(t, c.residual) else "mul"] = t
        h, _, _ = q.qlora_linear_fwd_epilogue(c.qw, c.x, c.A, c.B, c.alpha, c.bias, "silu", h=t, **kw)
        assert h is t and torch.equal(h, want)


@pytest.mark.parametrize("N,K,M,r", [(264, 640, 5, 16), (264, 640, 77, 16), (4104, 640, 1100, 16)])
def test_writes_stay_in_their_buffers_and_calls_repeat_bit_for_bit(q, N, K, M, r):
    from test_gpu_guard import Guarded
    c = Case(q, N, K, M, r)
    G = {n: Guarded(s, torch.bfloat16) for n, s in dict(h=(M, N), z=(M, N), dX=(M, K), dA=(r, K), dB=(N, r),
                                                         dbias=(N,), dmul=(M, N)).items()}
    G["u"] = Guarded((M, r), torch.float32)
    G["ws"] = Guarded((q.fwd_epilogue_workspace_bytes(M, N, K, r),), torch.uint8)
    G["wb"] = Guarded((q.bwd_epilogue_workspace_bytes(M, N, K, r),), torch.uint8)
    import ctypes
    st = c.qw.struct()
    p = {n: g.t.data_ptr() for n, g in G.items()}
    ep = q.EpilogueStruct(q.ACTIVATIONS["gelu"], c.bias.data_ptr(), c.mul.data_ptr(), c.residual.data_ptr())
    stream = torch.cuda.current_stream().cuda_stream
    assert q.lib.qlora_linear_fwd_epilogue(ctypes.byref(st), c.x.data_ptr(), M, c.A.data_ptr(), c.B.data_ptr(), r,
                                           c.alpha, ctypes.byref(ep), p["h"], p["z"], p["u"], p["ws"],
                                           G["ws"].nbytes, stream) == 0
    assert q.lib.qlora_linear_bwd_epilogue(ctypes.byref(st), c.x.data_ptr(), M, c.A.data_ptr(), c.B.data_ptr(), r,
                                           c.alpha, ctypes.byref(ep), c.dH.data_ptr(), p["z"], p["u"], p["dX"],
                                           p["dA"], p["dB"], p["dbias"], p["dmul"], 0, p["wb"], G["wb"].nbytes,
                                           stream) == 0
    torch.cuda.synchronize()
    assert [n for n, g in G.items() if not g.intact()] == []
    h, u, z = q.qlora_linear_fwd_epilogue(c.qw, c.x, c.A, c.B, c.alpha, c.bias, "gelu", c.mul, c.residual)
    g = q.qlora_linear_bwd_epilogue(c.qw, c.x, c.A, c.B, c.alpha, c.dH, z, "gelu", c.mul, u=u, need_dbias=True)
    for n, t in zip(("h", "u", "z", "dX", "dA", "dB", "dbias", "dmul"), (h, u, z) + g):
        assert torch.equal(t, G[n].t), n


@pytest.mark.parametrize("M", [1, 8, 13])
@pytest.mark.parametrize("N", [24, 2312, 4616, 5128, 6904, 6928, 9232])
def test_few_tokens_with_every_dealing_of_rows_to_blocks(q, N, M):
    """Rows in 32- and 16-row tiles over the GPU's blocks: one whole round and a
    rest, a rest alone, a rest past one half tile each. Each row's sum is taken
    in the same order whichever it is, so without an epilogue the layer's own
    kernel, which has 32-row tiles only, gives the same bits."""
    c = Case(q, N, 320, M, 16, True, 64)
    want, uw = q.qlora_linear_fwd(c.qw, c.x, c.A, c.B, c.alpha)
    guard = torch.full((M * N + 512,), -3.0, device="cuda", dtype=torch.bfloat16)
    out = guard[256:256 + M * N].view(M, N)
    h, u, _ = q.qlora_linear_fwd_epilogue(c.qw, c.x, c.A, c.B, c.alpha, save_z=False, h=out)
    assert torch.equal(h, want) and torch.equal(u, uw)
    assert (guard[:256] == -3.0).all() and (guard[256 + M * N:] == -3.0).all()
    h, u, z = q.qlora_linear_fwd_epilogue(c.qw, c.x, c.A, c.B, c.alpha, c.bias, "silu", c.mul, c.residual)
    check_forward(q, c, "silu", "bmr", h, u, z)


def test_empty_batch(q):
    c = Case(q, 264, 640, 4, 16)
    e = lambda n: torch.empty(0, n, dtype=torch.bfloat16, device="cuda")
    h, u, z = q.qlora_linear_fwd_epilogue(c.qw, e(640), c.A, c.B, c.alpha, c.bias, "silu", e(264), e(264))
    assert h.shape == (0, 264) and u.shape == (0, 16) and z.shape == (0, 264)
    dX, dA, dB, dbias, dmul = q.qlora_linear_bwd_epilogue(c.qw, e(640), c.A, c.B, c.alpha, e(264), z, "silu",
                                                          e(264), need_dbias=True)
    assert dX.shape == (0, 640) and dmul.shape == (0, 264)
    assert not dA.any() and not dB.any() and not dbias.any()


@pytest.mark.parametrize("M", [7, 150])
def test_captured_and_replayed_on_new_inputs(q, M):
    c, d = Case(q, 264, 640, M, 16), Case(q, 264, 640, M, 16, seed=1)
    wf = torch.empty(q.fwd_epilogue_workspace_bytes(M, 264, 640, 16), dtype=torch.uint8, device="cuda")
    wb = torch.empty(q.bwd_epilogue_workspace_bytes(M, 264, 640, 16), dtype=torch.uint8, device="cuda")

    def step(x, dH, mul):
        h, u, z = q.qlora_linear_fwd_epilogue(c.qw, x, c.A, c.B, c.alpha, c.bias, "silu", mul, workspace=wf)
        return (h,) + q.qlora_linear_bwd_epilogue(c.qw, x, c.A, c.B, c.alpha, dH, z, "silu", mul, u=u,
                                                  need_dbias=True, workspace=wb)

    x, dH, mul = c.x.clone(), c.dH.clone(), c.mul.clone()
    step(x, dH, mul)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = step(x, dH, mul)
    for src in (c, d, c):
        x.copy_(src.x), dH.copy_(src.dH), mul.copy_(src.mul)
        g.replay()
        got = [t.clone() for t in outs]
        want = step(src.x, src.dH, src.mul)
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_two_streams_at_once(q):
    cs = [Case(q, 520, 1152, M, 16, seed=M) for M in (150, 7, 300, 12)]
    call = lambda c: q.qlora_linear_fwd_epilogue(c.qw, c.x, c.A, c.B, c.alpha, c.bias, "gelu", c.mul, c.residual)
    want = [call(c) for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    got = [[] for _ in cs]
    for _ in range(5):
        for i, (c, s) in enumerate(zip(cs, streams)):
            with torch.cuda.stream(s):
                got[i].append(call(c))
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        for one in g:
            assert all(torch.equal(a, b) for a, b in zip(w, one))


def test_a_gated_mlp_as_it_would_be_used(q):
    """up, gate (silu, times up), down (into the residual stream), and back."""
    M, H, F, r, alpha = 150, 640, 1152, 16, 32.0
    mk = lambda n, k, seed: Case(q, n, k, M, r, seed=seed, alpha=alpha)
    up, gate, down = mk(F, H, 1), mk(F, H, 2), mk(H, F, 3)
    x, res, dY = up.x, down.residual, down.dH
    hu, uu = q.qlora_linear_fwd(up.qw, x, up.A, up.B, alpha)
    hg, ug, zg = q.qlora_linear_fwd_epilogue(gate.qw, x, gate.A, gate.B, alpha, act="silu", mul=hu)
    y, ud, _ = q.qlora_linear_fwd_epilogue(down.qw, hg, down.A, down.B, alpha, residual=res, save_z=False)
    dg, dAd, dBd, _, _ = q.qlora_linear_bwd_epilogue(down.qw, hg, down.A, down.B, alpha, dY, u=ud)
    dx1, dAg, dBg, _, du = q.qlora_linear_bwd_epilogue(gate.qw, x, gate.A, gate.B, alpha, dg, zg, "silu", hu, u=ug)
    dx2, dAu, dBu = q.qlora_linear_bwd(up.qw, x, up.A, up.B, alpha, du, u=uu)

    W = [q.nf4_dequantize(c.qw, bf16=True).double() for c in (up, gate, down)]
    P = [[t.double().requires_grad_() for t in (c.A, c.B)] for c in (up, gate, down)]
    xd = x.double().requires_grad_()
    lin = lambda i, v: v @ W[i].T + alpha / r * (v @ P[i][0].T) @ P[i][1].T
    g = lin(1, xd)
    yd = lin(2, g * torch.sigmoid(g) * lin(0, xd)) + res.double()
    yd.backward(dY.double())
    want = dict(y=yd.detach(), dx=xd.grad, dAd=P[2][0].grad, dBd=P[2][1].grad, dAg=P[1][0].grad, dBg=P[1][1].grad,
                dAu=P[0][0].grad, dBu=P[0][1].grad)
    got = dict(y=y, dx=dx1.double() + dx2.double(), dAd=dAd, dBd=dBd, dAg=dAg, dBg=dBg, dAu=dAu, dBu=dBu)
    # at most nine bf16 roundings of random sign lie between an input and a gradient,
    # each 2^-8 / sqrt(3) of its value in the mean square: sqrt(9 / 3) 2^-8
    for n in want:
        rel = ((got[n].double() - want[n]).norm() / want[n].norm()).item()
        assert rel <= 3 ** 0.5 * HALF_BF16, (n, rel)
