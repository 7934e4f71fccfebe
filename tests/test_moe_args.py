"""Refusals of the mixture of NF4 experts (host checks: no GPU needed)."""
import ctypes

import pytest
import torch

from conftest import build_library

FAKE = 0x10000
M, E, TOPK, H, F = 3, 4, 2, 128, 64


@pytest.fixture(scope="module")
def q():
    build_library()
    import bit_nf4_quantized_05_b200 as mod
    return mod


def weight(q, n, k, block=64, dq=0, codes=FAKE):
    return q.NF4WeightStruct(n, k, block, dq, codes, FAKE, FAKE, FAKE)


def call(q, **kw):
    gu = kw.get("gu", weight(q, E * 2 * F, H))
    dn = kw.get("dn", weight(q, E * H, F))
    return q.lib.nf4_moe_fwd(ctypes.byref(gu) if gu else None, ctypes.byref(dn) if dn else None,
                             kw.get("x", FAKE), kw.get("M", M), kw.get("router", FAKE), kw.get("E", E),
                             kw.get("k", TOPK), kw.get("renorm", 1), kw.get("act", 2), kw.get("res"),
                             kw.get("out", FAKE), kw.get("ids"), kw.get("w"), kw.get("ws", FAKE),
                             kw.get("wsb", 64), None)


def test_argument_checks(q):
    assert call(q) == q.NF4_ERR_WORKSPACE
    assert call(q, ws=None, wsb=1 << 30) == q.NF4_ERR_WORKSPACE
    assert call(q, ws=FAKE + 16, wsb=1 << 30) == q.NF4_ERR_ALIGNMENT
    assert call(q, gu=None) == q.NF4_ERR_INVALID_ARG
    assert call(q, dn=None) == q.NF4_ERR_INVALID_ARG
    assert call(q, M=0, wsb=0) == q.NF4_OK
    assert call(q, M=-1) == q.NF4_ERR_UNSUPPORTED_SHAPE
    assert call(q, M=65) == q.NF4_ERR_UNSUPPORTED_SHAPE
    assert call(q, E=0) == q.NF4_ERR_UNSUPPORTED_SHAPE
    assert call(q, E=3) == q.NF4_ERR_UNSUPPORTED_SHAPE                  # the stacks hold four
    big = dict(gu=weight(q, 257 * 2 * F, H), dn=weight(q, 257 * H, F))
    assert call(q, E=257, **big) == q.NF4_ERR_UNSUPPORTED_SHAPE
    assert call(q, k=0) == q.NF4_ERR_UNSUPPORTED_SHAPE
    assert call(q, k=E + 1) == q.NF4_ERR_UNSUPPORTED_SHAPE
    many = dict(gu=weight(q, 32 * 2 * F, H), dn=weight(q, 32 * H, F), E=32)
    assert call(q, k=17, **many) == q.NF4_ERR_UNSUPPORTED_SHAPE
    assert call(q, k=16, **many) == q.NF4_ERR_WORKSPACE
    assert call(q, dn=weight(q, E * H, 2 * F)) == q.NF4_ERR_UNSUPPORTED_SHAPE
    assert call(q, gu=weight(q, E * 2 * F, 2 * H)) == q.NF4_ERR_UNSUPPORTED_SHAPE
    assert call(q, dn=weight(q, E * H, F, block=128)) == q.NF4_ERR_UNSUPPORTED_SHAPE   # F % 128
    assert call(q, renorm=2) == q.NF4_ERR_INVALID_ARG
    assert call(q, act=5) == q.NF4_ERR_INVALID_ARG
    assert call(q, x=None) == q.NF4_ERR_INVALID_ARG
    assert call(q, router=None) == q.NF4_ERR_INVALID_ARG
    assert call(q, out=None) == q.NF4_ERR_INVALID_ARG
    assert call(q, x=FAKE + 2) == q.NF4_ERR_ALIGNMENT
    assert call(q, ids=FAKE + 4) == q.NF4_ERR_ALIGNMENT
    assert call(q, w=FAKE + 8) == q.NF4_ERR_ALIGNMENT
    assert call(q, res=FAKE) == q.NF4_ERR_WORKSPACE                     # the residual updated in place
    assert call(q, res=FAKE + 16) == q.NF4_ERR_INVALID_ARG
    assert call(q, x=FAKE + 16) == q.NF4_ERR_INVALID_ARG                # x half under out
    assert call(q, x=FAKE + M * H * 2) == q.NF4_ERR_WORKSPACE
    assert call(q, gu=weight(q, E * 2 * F, H, codes=FAKE + 8)) == q.NF4_ERR_ALIGNMENT


def test_workspace_query(q):
    a = q.moe_workspace_bytes(1, 8, 256, 128, 2)
    b = q.moe_workspace_bytes(64, 8, 256, 128, 2)
    # activations of every slot in bf16, their products in fp32, the logits in fp64
    assert a < b and b >= 64 * 2 * (128 * 2 + 256 * 4) + 64 * 8 * 8 and b % 256 == 0


def test_binding_checks(q):
    bf16 = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    gu = q.QuantizedWeight.empty(E * 2 * F, H, True, "cpu")
    dn = q.QuantizedWeight.empty(E * H, F, False, "cpu")
    x, r = bf16(M, H), bf16(E, H)
    for match, fn in [
        ("CUDA tensors", lambda: q.nf4_moe_fwd(gu, dn, x, r, 2, residual=bf16(M, H), out=bf16(M, H))),
        ("x", lambda: q.nf4_moe_fwd(gu, dn, bf16(M, F), r, 2)),
        ("2-D", lambda: q.nf4_moe_fwd(gu, dn, bf16(H), r, 2)),
        ("router", lambda: q.nf4_moe_fwd(gu, dn, x, torch.zeros(E, H), 2)),
        ("stacked experts", lambda: q.nf4_moe_fwd(gu, dn, x, bf16(E - 1, H), 2)),
        ("stacked experts", lambda: q.nf4_moe_fwd(gu, gu, x, r, 2)),
        ("top_k", lambda: q.nf4_moe_fwd(gu, dn, x, r, 0)),
        ("top_k", lambda: q.nf4_moe_fwd(gu, dn, x, r, E + 1)),
        ("residual", lambda: q.nf4_moe_fwd(gu, dn, x, r, 2, residual=bf16(M, F))),
        ("contiguous", lambda: q.nf4_moe_fwd(gu, dn, x, r, 2, out=bf16(H, M).T)),
        ("workspace", lambda: q.nf4_moe_fwd(gu, dn, x, r, 2, workspace=torch.zeros(8))),
    ]:
        with pytest.raises(ValueError, match=match):
            fn()
