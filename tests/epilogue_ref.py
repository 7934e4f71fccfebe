"""Plain 64-bit forms of the layer with its epilogue and of the activations, for
the tests. Written from the formulas; they share no code with the library."""
import math

import torch

# largest |act'(z)| over all z (silu 1.0998, both gelu 1.1290)
ACT_SLOPE = 1.13
HALF_BF16 = 2.0 ** -8          # half a step of bf16, relative
# error of an activation evaluated in fp32 with the hardware exponential, relative
# to max(|z|, 1) |.|: exp(-z) has its argument rounded (|z| 2^-24, and beyond
# |z| = 100 the result is 0 or z itself) plus a few units of 2^-22
ACT_EVAL = 2.0 ** -16


def act64(z, act):
    """(act(z), act'(z))."""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z)), (z > 0).to(z.dtype)
    if act == "silu":
        p = torch.sigmoid(z)
        return z * p, p + z * p * torch.sigmoid(-z)
    if act == "gelu":
        cdf = 0.5 * torch.erfc(-z / math.sqrt(2.0))
        return z * cdf, cdf + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    zc = z.clamp(-1e4, 1e4)
    v = c * (zc + 0.044715 * zc ** 3)
    p = torch.sigmoid(2 * v)
    return z * p, p + z * p * torch.sigmoid(-2 * v) * 2 * c * (1 + 3 * 0.044715 * zc ** 2)


def forward64(W, x, A, B, s, bias, act, mul, residual, exact=False):
    """u, z, h and the bound on the kernels' error of z before any output rounding.
    W is the operand the products use, so what is left is: the rounding of
    s (x A^T) to bf16, and fp32 sums of k + r products on the tensor cores
    (at most one 2^-23 of the running magnitude per addition). exact: weight and
    s (x A^T) go in as two bf16 parts (2^-16 left at most) in twice the sums."""
    W, x, A, B = (t.double() for t in (W, x, A, B))
    u = x @ A.T
    z = x @ W.T + s * (u @ B.T)
    mag = x.abs() @ W.abs().T + abs(s) * (u.abs() @ B.abs().T)
    lora = abs(s) * ((x.abs() @ A.abs().T) @ B.abs().T)
    terms = (x.shape[1] + A.shape[0] + 8) * 2.0 ** -23 * (mag + lora)
    if exact:
        tol = 2.0 ** -16 * mag + 2 * terms
    else:
        tol = HALF_BF16 * abs(s) * (u.abs() @ B.abs().T) + terms
    if bias is not None:
        z = z + bias.double()
        tol = tol + 2.0 ** -23 * z.abs()
    h, _ = act64(z, act)
    if mul is not None:
        h = h * mul.double()
    if residual is not None:
        h = h + residual.double()
    return u, z, h, tol


def backward64(W, x, A, B, s, dH, z, act, mul, u):
    """Gradients from the formula, and bounds: dz is rounded to bf16 before the
    products, s (dz B) and s u are too, then fp32 sums; outputs round once."""
    W, x, A, B, dH, z, u = (t.double() for t in (W, x, A, B, dH, z, u))
    a, da = act64(z, act)
    dz = dH * da
    dmul = None
    if mul is not None:
        dmul = dH * a
        dz = dz * mul.double()
    # act' in fp32: its terms are at most max(|z|, 1) in size
    edz = dH.abs() * ACT_EVAL * z.abs().clamp_min(1) * (1 if mul is None else mul.double().abs())
    if act in ("none", "relu"):
        edz = torch.zeros_like(dz)
    rdz = edz + HALF_BF16 * dz.abs() if (act != "none" or mul is not None) else torch.zeros_like(dz)
    M, N, K, r = x.shape[0], W.shape[0], W.shape[1], A.shape[0]
    f = 2.0 ** -23
    v, va = dz @ B, dz.abs() @ B.abs()
    ev = rdz @ B.abs() + (N + 2) * f * va + HALF_BF16 * v.abs()        # of the rounded s v, over s
    dX = dz @ W + s * (v @ A)
    tX = rdz @ W.abs() + (N + r + 8) * f * (dz.abs() @ W.abs() + abs(s) * (va @ A.abs())) + abs(s) * (ev @ A.abs())
    dA = s * (v.T @ x)
    tA = abs(s) * (ev.T @ x.abs() + (M + 4) * f * (va.T @ x.abs()))
    dB = s * (dz.T @ u)
    tB = abs(s) * (rdz.T @ u.abs() + (HALF_BF16 + (M + 4) * f + K * f) * (dz.abs().T @ u.abs()))
    dbias = dz.sum(0)
    tbias = edz.sum(0) + (M + 4) * 2.0 ** -24 * dz.abs().sum(0)
    return dict(dX=(dX, tX), dA=(dA, tA), dB=(dB, tB), dbias=(dbias, tbias),
                dmul=None if dmul is None else (dmul, dH.abs() * ACT_EVAL * z.abs().clamp_min(1)))


def check(name, got, want, tol, out_half=HALF_BF16):
    """|got - want| <= tol + half a step of the output type, element by element."""
    err = (got.double() - want).abs()
    bar = tol + out_half * (want.abs() + tol) + 1e-37
    bad = ~(err <= bar)
    if bool(bad.any()):
        i = int((err / bar).nan_to_num(float("inf")).argmax())
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} outside; worst at {i}: got "
                             f"{got.flatten()[i].item()}, want {want.flatten()[i].item()}, bar "
                             f"{bar.flatten()[i].item()}")
