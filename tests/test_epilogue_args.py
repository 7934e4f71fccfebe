"""Refusals of the layer with its epilogue (host checks: no GPU needed), and the
gradient formulas of the 64-bit reference against central differences."""
import ctypes

import pytest
import torch

from conftest import build_library
from epilogue_ref import act64, backward64, forward64

N, K, M, R = 64, 128, 5, 8
FAKE = 0x10000
FAR = 0x4000000
X = 0x40000000


@pytest.fixture(scope="module")
def q():
    build_library()
    import bit_nf4_quantized_05_b200 as mod
    return mod


def weight(q, n=N, k=K):
    return q.NF4WeightStruct(n, k, 64, 0, FAKE, FAKE, FAKE, FAKE)


def fwd(q, **kw):
    ep = q.EpilogueStruct(kw.get("act", 0), kw.get("bias"), kw.get("mul"), kw.get("residual"))
    return q.lib.qlora_linear_fwd_epilogue(
        ctypes.byref(kw.get("w", weight(q))), X, kw.get("M", M), FAKE, FAKE, kw.get("r", R), 16.0,
        None if kw.get("no_ep") else ctypes.byref(ep), kw.get("h", FAKE), kw.get("z"), None,
        kw.get("ws", FAKE), kw.get("wsb", 16), None)


def test_forward_argument_checks(q):
    assert fwd(q, no_ep=True) == q.NF4_ERR_INVALID_ARG
    assert fwd(q, act=5) == q.NF4_ERR_INVALID_ARG
    assert fwd(q, act=-1) == q.NF4_ERR_INVALID_ARG
    assert fwd(q, r=7) == q.NF4_ERR_UNSUPPORTED_SHAPE
    assert fwd(q, bias=FAKE + 2) == q.NF4_ERR_ALIGNMENT
    assert fwd(q, mul=FAKE + 8) == q.NF4_ERR_ALIGNMENT
    assert fwd(q, residual=FAR + 4) == q.NF4_ERR_ALIGNMENT
    assert fwd(q, z=FAR + 4) == q.NF4_ERR_ALIGNMENT
    assert fwd(q, h=None) == q.NF4_ERR_INVALID_ARG
    # h on top of the residual is the in-place update; half over it is not
    assert fwd(q, residual=FAKE) == q.NF4_ERR_WORKSPACE
    assert fwd(q, residual=FAKE + 16) == q.NF4_ERR_INVALID_ARG
    assert fwd(q, mul=FAKE + M * N * 2 - 16) == q.NF4_ERR_INVALID_ARG
    assert fwd(q, mul=FAKE + M * N * 2) == q.NF4_ERR_WORKSPACE
    assert fwd(q, z=FAKE) == q.NF4_ERR_INVALID_ARG
    assert fwd(q, z=FAR, mul=FAR) == q.NF4_ERR_INVALID_ARG
    assert fwd(q, z=FAR, residual=FAR + 32) == q.NF4_ERR_INVALID_ARG
    assert fwd(q, h=X) == q.NF4_ERR_INVALID_ARG                         # over the tokens
    assert fwd(q, h=X + M * K * 2 - 16) == q.NF4_ERR_INVALID_ARG
    assert fwd(q, h=X + M * K * 2) == q.NF4_ERR_WORKSPACE
    assert fwd(q, z=X - M * N * 2 + 16) == q.NF4_ERR_INVALID_ARG
    assert fwd(q, M=0, act=2, h=None) == q.NF4_OK


def bwd(q, **kw):
    ep = q.EpilogueStruct(kw.get("act", 0), None, kw.get("mul"), None)
    return q.lib.qlora_linear_bwd_epilogue(
        ctypes.byref(kw.get("w", weight(q))), X, kw.get("M", M), FAKE, FAKE, R, 16.0,
        None if kw.get("no_ep") else ctypes.byref(ep), kw.get("dH", FAKE), kw.get("z"), None, kw.get("dX"),
        kw.get("dA", FAKE), FAKE, kw.get("dbias"), kw.get("dmul"), kw.get("f32", 0), kw.get("ws", FAKE),
        kw.get("wsb", 16), None)


def test_backward_argument_checks(q):
    assert bwd(q, no_ep=True) == q.NF4_ERR_INVALID_ARG
    assert bwd(q, act=9) == q.NF4_ERR_INVALID_ARG
    assert bwd(q, act=2) == q.NF4_ERR_INVALID_ARG                       # z missing
    assert bwd(q, mul=FAKE, dmul=FAR) == q.NF4_ERR_INVALID_ARG          # z missing
    assert bwd(q, z=FAKE, dmul=FAR) == q.NF4_ERR_INVALID_ARG            # dmul without mul
    assert bwd(q, z=FAR, mul=FAKE, dmul=FAKE) == q.NF4_ERR_INVALID_ARG  # dmul over its inputs
    assert bwd(q, z=FAR, mul=2 * FAR, dmul=FAR + 16) == q.NF4_ERR_INVALID_ARG
    assert bwd(q, dX=FAKE) == q.NF4_ERR_INVALID_ARG                     # dX over dH
    assert bwd(q, dX=X + 16) == q.NF4_ERR_INVALID_ARG
    assert bwd(q, dX=FAR) == q.NF4_ERR_WORKSPACE
    assert bwd(q, z=FAR, mul=2 * FAR, dmul=3 * FAR, dX=3 * FAR) == q.NF4_ERR_INVALID_ARG
    assert bwd(q, dH=None) == q.NF4_ERR_INVALID_ARG
    assert bwd(q, dA=None) == q.NF4_ERR_INVALID_ARG
    assert bwd(q, f32=2) == q.NF4_ERR_INVALID_ARG
    assert bwd(q, dbias=FAKE + 4) == q.NF4_ERR_ALIGNMENT
    assert bwd(q, z=FAKE + 4, act=1) == q.NF4_ERR_ALIGNMENT
    assert bwd(q) == q.NF4_ERR_WORKSPACE
    assert bwd(q, ws=None, wsb=1 << 30) == q.NF4_ERR_WORKSPACE
    assert bwd(q, ws=FAKE + 16, wsb=1 << 30) == q.NF4_ERR_ALIGNMENT


def test_workspace_holds_the_scaled_gradient(q):
    a, b = q.bwd_workspace_bytes(100, 512, 256, 16), q.bwd_epilogue_workspace_bytes(100, 512, 256, 16)
    assert b >= a + 100 * 512 * 2 and b % 256 == 0


def bf16(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def test_binding_checks(q):
    qw = q.QuantizedWeight.empty(N, K, True, "cpu")
    x, A, B, dH = bf16(M, K), bf16(R, K), bf16(N, R), bf16(M, N)
    f = lambda **kw: q.qlora_linear_fwd_epilogue(qw, x, A, B, 16.0, **kw)
    g = lambda **kw: q.qlora_linear_bwd_epilogue(qw, x, A, B, 16.0, kw.pop("dH", dH), **kw)
    for match, call in [
        ("act must be", lambda: f(act="tanh")),
        ("bias", lambda: f(bias=bf16(M))),
        ("bias", lambda: f(bias=torch.zeros(N))),
        ("mul", lambda: f(mul=bf16(M + 1, N))),
        ("residual", lambda: f(residual=bf16(N, M).T)),
        ("h", lambda: f(h=bf16(M, K))),
        ("CUDA tensors", lambda: f(bias=bf16(N), act="gelu", mul=bf16(M, N), residual=bf16(M, N))),
        ("dH", lambda: g(dH=bf16(M, K))),
        ("z \\(the", lambda: g(act="silu")),
        ("z \\(the", lambda: g(mul=bf16(M, N))),
        ("z", lambda: g(z=torch.zeros(M, N), act="relu")),
        ("u", lambda: g(u=torch.zeros(M, R + 1))),
        ("bf16 or fp32", lambda: g(grad_dtype=torch.float16)),
        ("act must be", lambda: g(act="swish")),
        ("CUDA tensors", lambda: g(z=bf16(M, N), act="silu", mul=bf16(M, N))),
    ]:
        with pytest.raises(ValueError, match=match):
            call()


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu_tanh", "gelu"])
def test_reference_gradients_against_differences(act):
    """Directional central differences of sum(dH . h) in 64 bits."""
    g = torch.Generator().manual_seed(3)
    mk = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)
    M, N, K, r, s = 3, 5, 7, 2, 0.5
    W, x, A, B, bias, mul, res, dH = mk(N, K), mk(M, K), mk(r, K), mk(N, r), mk(N), mk(M, N), mk(M, N), mk(M, N)
    value = lambda x, A, B, bias, mul: float((dH * forward64(W, x, A, B, s, bias, act, mul, res)[2]).sum())
    u, z, _, _ = forward64(W, x, A, B, s, bias, act, mul, res)
    got = backward64(W, x, A, B, s, dH, z, act, mul, u)
    args = dict(x=x, A=A, B=B, bias=bias, mul=mul)
    for name, key in (("x", "dX"), ("A", "dA"), ("B", "dB"), ("bias", "dbias"), ("mul", "dmul")):
        d = mk(*args[name].shape)
        e = 1e-5
        hi, lo = ({**args, name: args[name] + t * d} for t in (e, -e))
        diff = (value(**hi) - value(**lo)) / (2 * e)
        want = float((got[key][0] * d).sum())
        assert abs(diff - want) <= 1e-6 * max(1.0, abs(want)), (name, diff, want)


def test_reference_activations_against_torch():
    z = torch.linspace(-12, 12, 4001, dtype=torch.float64)
    f = torch.nn.functional
    for act, ref in (("relu", f.relu), ("silu", f.silu), ("gelu", f.gelu),
                     ("gelu_tanh", lambda t: f.gelu(t, approximate="tanh"))):
        assert float((act64(z, act)[0] - ref(z)).abs().max()) <= 1e-13


def test_a_weight_takes_numpy_flags_and_names_the_array_it_lacks(q):
    import dataclasses

    import numpy as np
    qw = q.QuantizedWeight.empty(8, 64, True, "cpu")
    st = dataclasses.replace(qw, double_quant=np.bool_(True)).struct()
    assert st.double_quant == 1 and st.codes == qw.codes.data_ptr()
    for name in ("codes", "absmax", "absmax_q8", "absmax_c"):
        with pytest.raises(ValueError, match=name + " is required"):
            dataclasses.replace(qw, **{name: None}).struct()
