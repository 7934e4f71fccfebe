"""The mixture of NF4 experts for a few tokens against its definition in 64 bits.

The oracle takes the weight as the kernel's products do: a multiple of the level
rounded to bf16, times the fp32 block scale over that multiple. Left are the rounding of act(gate) . up to
bf16, fp32 sums, and the output's rounding; the bound follows them through."""
import pytest
import torch

from epilogue_ref import ACT_EVAL, ACT_SLOPE, HALF_BF16, act64, check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    import bit_nf4_quantized_05_b200 as mod
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    return mod


def operand(qw, rows):
    """bf16(1.4367 level) * 0.69603324 scale of some rows, in 64 bits, on the GPU."""
    from perf.operators import LEVELS
    lv = (torch.tensor(LEVELS) * 1.4367).bfloat16().double().cuda() * 0.69603324
    c = qw.codes.view(qw.n, qw.k // 2)[rows]
    codes = torch.stack((c >> 4, c & 15), -1).view(c.shape[0], qw.k)
    nb = qw.n * qw.k // qw.block_size
    if qw.double_quant:
        s = qw.absmax_q8[:nb].double() * (qw.absmax_c.double() / 127).repeat_interleave(256)[:nb]
    else:
        s = qw.absmax[:nb].double()
    s = s.view(qw.n, -1)[rows]
    return lv[codes.long()] * s.repeat_interleave(qw.block_size, 1)


class Moe:
    def __init__(self, q, M, E, k, H, F, dq=(True, True), block=(64, 64), seed=0):
        g = torch.Generator().manual_seed(900 + seed + M * 7 + E)
        mk = lambda *s, std=1.0: torch.randn(*s, generator=g) * std
        self.M, self.E, self.k, self.H, self.F = M, E, k, H, F
        self.x = mk(M, H).bfloat16().cuda()
        self.residual = mk(M, H).bfloat16().cuda()
        self.router = mk(E, H, std=1 / H ** 0.5).bfloat16().cuda()
        self.gate_up = q.nf4_quantize(mk(E * 2 * F, H, std=1 / H ** 0.5).cuda(), dq[0], block_size=block[0])
        self.down = q.nf4_quantize(mk(E * H, F, std=1 / F ** 0.5).cuda(), dq[1], block_size=block[1])


def route64(m, renorm):
    l = m.x.double() @ m.router.double().T
    rank = l.nan_to_num(nan=-float("inf"), posinf=float("inf"), neginf=-float("inf"))
    ids = torch.sort(rank, dim=1, descending=True, stable=True)[1][:, :m.k]
    p = torch.softmax(l, 1).gather(1, ids)
    return ids, p / p.sum(1, keepdim=True) if renorm else p


def moe64(m, ids, w, act, residual):
    """(out, bound on the error before the output's rounding)."""
    f = 2.0 ** -23
    out = torch.zeros(m.M, m.H, dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(out)
    for e in ids.unique().tolist():
        tok, j = (ids == e).nonzero(as_tuple=True)
        x = m.x[tok].double()
        W = operand(m.gate_up, slice(e * 2 * m.F, (e + 1) * 2 * m.F))
        Wd = operand(m.down, slice(e * m.H, (e + 1) * m.H))
        gu = x @ W.T
        tgu = (m.H + 12) * f * (x.abs() @ W.abs().T)
        g, u, tg, tu = gu[:, :m.F], gu[:, m.F:], tgu[:, :m.F], tgu[:, m.F:]
        slope, ev = (1.0, 0.0) if act in ("none", "relu") else (ACT_SLOPE, ACT_EVAL)
        v, _ = act64(g, act)
        tv = slope * tg + ev * (v.abs() + slope * tg)
        a = v * u
        ta = tv * (u.abs() + tu) + v.abs() * tu
        ta = ta + HALF_BF16 * (a.abs() + ta)
        y = a @ Wd.T
        ty = ta @ Wd.abs().T + (m.F + 12) * f * ((a.abs() + ta) @ Wd.abs().T)
        s = w[tok, j][:, None]
        out.index_add_(0, tok, s * y)
        tol.index_add_(0, tok, s * (ty + (m.k + 24) * f * y.abs()))      # the weight's own fp32 error too
    if residual is not None:
        out = out + residual.double()
        tol = tol + f * out.abs()
    return out, tol


def check_moe(q, m, got, act, renorm, residual):
    out, ids, w = got
    ids64, w64 = route64(m, renorm)
    assert torch.equal(ids.long(), ids64)
    # expf and the division within a few 2^-23; l - max is rounded to fp32 (|l| below 2^7)
    assert ((w.double() - w64).abs() <= 2.0 ** -16 * w64 + 1e-37).all()
    want, tol = moe64(m, ids64, w64, act, residual)
    check("out", out, want, tol + 2.0 ** -16 * tol)
    rel = ((out.double() - want).norm() / want.norm()).item()
    assert rel <= 2 * HALF_BF16, rel            # two roundings, each at most 2^-8 in the norm


# one token to the limit; full, overfull and one-token chunks; odd block counts in
# both products; one block; as many experts as fit; every token at every expert
SHAPES = [
    (1, 8, 2, 256, 128), (2, 4, 4, 64, 64), (7, 16, 3, 320, 192), (8, 5, 1, 2048, 1408), (9, 2, 2, 448, 704),
    (16, 64, 6, 512, 320), (17, 256, 16, 128, 64), (33, 3, 2, 1088, 576), (64, 32, 8, 256, 256),
    (64, 1, 1, 128, 128), (3, 8, 2, 5120, 2112), (64, 256, 16, 64, 64),
]


@pytest.mark.parametrize("M,E,k,H,F", SHAPES)
def test_against_the_definition(q, M, E, k, H, F):
    m = Moe(q, M, E, k, H, F)
    for act, renorm, res in (("silu", True, None), ("gelu_tanh", False, m.residual)):
        got = q.nf4_moe_fwd(m.gate_up, m.down, m.x, m.router, k, act, renorm, res)
        check_moe(q, m, got, act, renorm, res)
    assert q.device_status() == q.NF4_OK


@pytest.mark.parametrize("dq", [(False, False), (True, False), (False, True)])
@pytest.mark.parametrize("block", [(64, 64), (128, 64), (64, 128), (128, 128)])
def test_scale_forms_and_block_sizes(q, dq, block):
    m = Moe(q, 11, 6, 2, 384, 640, dq, block)
    for act in ("none", "relu", "gelu"):
        check_moe(q, m, q.nf4_moe_fwd(m.gate_up, m.down, m.x, m.router, 2, act), act, True, None)


@pytest.mark.parametrize("M", [8, 9, 40, 64])
def test_every_token_at_the_same_experts(q, M):
    m = Moe(q, M, 12, 2, 256, 192)
    m.x[:, 0] = 8.0
    m.router[:, 0] = 0.0
    m.router[7, 0] = 4.0
    m.router[11, 0] = 2.0
    got = q.nf4_moe_fwd(m.gate_up, m.down, m.x, m.router, 2)
    assert bool((got[1] == torch.tensor([7, 11], device="cuda")).all())
    check_moe(q, m, got, "silu", True, None)


def test_ties_go_to_the_lower_index(q):
    m = Moe(q, 20, 40, 5, 192, 64)
    m.router[33] = m.router[2]
    m.router[20] = m.router[2]
    m.router[39] = m.router[0]
    m.x[3] = 0                                     # all experts tie
    got = q.nf4_moe_fwd(m.gate_up, m.down, m.x, m.router, 5, renormalise=False)
    assert got[1][3].tolist() == [0, 1, 2, 3, 4]
    assert torch.equal(got[2][3], torch.full((5,), 1 / 40, device="cuda"))
    check_moe(q, m, got, "silu", False, None)


def test_near_ties_follow_the_exact_logits(q):
    """Experts whose logits differ far below an fp32 sum's error."""
    m = Moe(q, 16, 24, 6, 4096, 64)
    m.x[:, 0] = 2.0 ** -20
    for e in range(1, 24):
        m.router[e] = m.router[0]
        m.router[e, 0] = m.router[0, 0].float() + 2.0 ** -6 * ((e * 7) % 24)
    got = q.nf4_moe_fwd(m.gate_up, m.down, m.x, m.router, 6)
    ids64, _ = route64(m, True)
    assert torch.equal(got[1].long(), ids64)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_a_bad_token_keeps_to_its_row(q, bad):
    m = Moe(q, 12, 8, 3, 256, 128)
    clean = q.nf4_moe_fwd(m.gate_up, m.down, m.x, m.router, 3)
    m.x[5, 17] = bad
    out, ids, w = q.nf4_moe_fwd(m.gate_up, m.down, m.x, m.router, 3)
    keep = [i for i in range(12) if i != 5]
    # (chunks may be cut elsewhere, but a token's sums do not depend on its neighbours)
    assert torch.equal(out[keep], clean[0][keep]) and torch.equal(ids[keep], clean[1][keep])
    assert torch.equal(w[keep], clean[2][keep])
    assert bool(out[5].isnan().all()) and bool(((ids >= 0) & (ids < 8)).all())
    assert len(set(ids[5].tolist())) == 3
    assert q.device_status() == q.NF4_OK


def test_bad_weights_of_experts_nobody_chose_do_not_show(q):
    m = Moe(q, 4, 8, 2, 256, 128, dq=(False, False))
    want = q.nf4_moe_fwd(m.gate_up, m.down, m.x, m.router, 2)
    idle = [e for e in range(8) if not bool((want[1] == e).any())]
    assert idle
    for e in idle:
        m.gate_up.absmax.view(8, -1)[e] = float("nan")
        m.down.absmax.view(8, -1)[e] = float("nan")
    got = q.nf4_moe_fwd(m.gate_up, m.down, m.x, m.router, 2)
    assert torch.equal(got[0], want[0])


def test_a_token_alone_and_in_a_batch(q):
    m = Moe(q, 24, 16, 4, 512, 320)
    out, ids, w = q.nf4_moe_fwd(m.gate_up, m.down, m.x, m.router, 4)
    for i in (0, 9, 23):
        o, d, v = q.nf4_moe_fwd(m.gate_up, m.down, m.x[i:i + 1], m.router, 4)
        assert torch.equal(d[0], ids[i]) and torch.equal(v[0], w[i]) and torch.equal(o[0], out[i])


@pytest.mark.parametrize("M,E,k,H,F", [(5, 8, 2, 256, 192), (40, 16, 4, 192, 320)])
def test_writes_stay_in_their_buffers_and_leftovers_do_not_matter(q, M, E, k, H, F):
    import ctypes
    from test_gpu_guard import Guarded
    m = Moe(q, M, E, k, H, F)
    want = q.nf4_moe_fwd(m.gate_up, m.down, m.x, m.router, k, residual=m.residual)
    G = dict(out=Guarded((M, H), torch.bfloat16), ids=Guarded((M, k), torch.int32),
             w=Guarded((M, k), torch.float32), ws=Guarded((q.moe_workspace_bytes(M, E, H, F, k),), torch.uint8))
    gu, dn = m.gate_up.struct(), m.down.struct()
    for fill in (0xFF, 0x00, None, 0x7F):
        if fill is not None:
            G["ws"].t.fill_(fill)
        assert q.lib.nf4_moe_fwd(ctypes.byref(gu), ctypes.byref(dn), m.x.data_ptr(), M, m.router.data_ptr(), E, k, 1,
                                 q.ACTIVATIONS["silu"], m.residual.data_ptr(), G["out"].t.data_ptr(),
                                 G["ids"].t.data_ptr(), G["w"].t.data_ptr(), G["ws"].t.data_ptr(), G["ws"].nbytes,
                                 torch.cuda.current_stream().cuda_stream) == 0
        torch.cuda.synchronize()
        assert [n for n, g in G.items() if not g.intact()] == []
        for n, t in zip(("out", "ids", "w"), want):
            assert torch.equal(G[n].t, t), (n, fill)
    # the routing outputs may be left out; the output may be the residual
    r = m.residual.clone()
    assert q.lib.nf4_moe_fwd(ctypes.byref(gu), ctypes.byref(dn), m.x.data_ptr(), M, m.router.data_ptr(), E, k, 1,
                             q.ACTIVATIONS["silu"], r.data_ptr(), r.data_ptr(), None, None, G["ws"].t.data_ptr(),
                             G["ws"].nbytes, torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    assert torch.equal(r, want[0])


def test_empty_batch(q):
    m = Moe(q, 1, 4, 2, 128, 64)
    out, ids, w = q.nf4_moe_fwd(m.gate_up, m.down, m.x[:0], m.router, 2)
    assert out.shape == (0, 128) and ids.shape == (0, 2) and w.shape == (0, 2)


def test_captured_and_replayed_on_new_inputs(q):
    m = Moe(q, 6, 16, 4, 256, 192)
    ws = torch.empty(q.moe_workspace_bytes(6, 16, 256, 192, 4), dtype=torch.uint8, device="cuda")
    x = m.x.clone()
    call = lambda x: q.nf4_moe_fwd(m.gate_up, m.down, x, m.router, 4, residual=x, workspace=ws)
    call(x)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):                 # two graphs on one workspace, replayed in turn
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call(x))
        graphs.append(g)
    for i in range(6):
        x.copy_(torch.randn(6, 256, generator=torch.Generator().manual_seed(i)).bfloat16())
        graphs[i % 2].replay()
        got = [t.clone() for t in outs[i % 2]]
        for a, b in zip(got, call(x)):
            assert torch.equal(a, b)


def test_several_streams_at_once(q):
    ms = [Moe(q, M, 16, 4, 512, 320, seed=M) for M in (1, 5, 16, 64)]
    call = lambda m: q.nf4_moe_fwd(m.gate_up, m.down, m.x, m.router, 4)
    want = [call(m) for m in ms]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ms]
    got = [[] for _ in ms]
    for _ in range(8):
        for i, (m, s) in enumerate(zip(ms, streams)):
            with torch.cuda.stream(s):
                got[i].append(call(m))
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        for one in g:
            assert all(torch.equal(a, b) for a, b in zip(w, one))
    assert q.device_status() == q.NF4_OK


def test_a_block_as_it_would_be_served(q):
    """A projection into the residual stream, then the experts into it, decoding."""
    from test_gpu_epilogue import Case
    M, H = 5, 640
    c = Case(q, H, 1152, M, 16)
    m = Moe(q, M, 8, 2, H, 320)
    stream = c.residual.clone()
    q.qlora_linear_fwd_epilogue(c.qw, c.x, c.A, c.B, c.alpha, residual=stream, h=stream, save_u=False, save_z=False)
    m.x = stream.clone()
    out, ids, w = q.nf4_moe_fwd(m.gate_up, m.down, stream, m.router, 2, residual=stream, out=stream)
    assert out is stream
    check_moe(q, m, (out, ids, w), "silu", True, m.x)


@pytest.mark.parametrize("M,E,k,H,F", [(3, 8, 2, 256, 192), (40, 16, 4, 192, 320)])
def test_wait_for_activations_runs_out_and_next_call_is_clean(q, M, E, k, H, F):
    """The gate-up items are not counted, so the down products' wait for them takes
    its (short) limit: the status says so, and the next call is as ever."""
    m = Moe(q, M, E, k, H, F)
    call = lambda: q.nf4_moe_fwd(m.gate_up, m.down, m.x, m.router, k)
    clean = call()
    assert q.device_status() == q.NF4_OK
    try:
        assert q.lib.nf4_debug_flag_wait(1, 20000) == q.NF4_OK
        bad = call()
        torch.cuda.synchronize()
        st = q.device_status()
    finally:
        assert q.lib.nf4_debug_flag_wait(0, 0) == q.NF4_OK
    assert st == q.NF4_ERR_TIMEOUT, q.status_string(st)
    assert q.device_status() == q.NF4_OK                  # read once, then cleared
    assert torch.equal(bad[1], clean[1]) and torch.equal(bad[2], clean[2])    # the routing had no part in it
    for _ in range(2):
        assert all(torch.equal(a, b) for a, b in zip(call(), clean))
    assert q.device_status() == q.NF4_OK
