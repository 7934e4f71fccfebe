"""What is measured of two operators next to the QLoRA linear layer.

  layer    the layer with its epilogue: z = x W~^T + (alpha/r)(x A^T) B^T + bias,
           h = act(z) * mul + residual; as a forward, and as a training step
           (forward and backward)
  moe      a mixture-of-experts layer for a few tokens over NF4 experts: router,
           top-k, gated experts, weighted sum

W~ is the dequantised weight, scale(block) * level(code), of an NF4 weight with
blocks of 64 or 128 elements and optional 8-bit block scales in groups of 256.

With `own` false the operators run in their plain form (fp32 torch operations,
rounded once); with `own` true they are the framework's calls.
"""
import math

import torch

own = False

LEVELS = (-1.0, -0.6961928009986877, -0.5250730514526367, -0.39491748809814453, -0.28444138169288635,
          -0.18477343022823334, -0.09105003625154495, 0.0, 0.07958029955625534, 0.16093020141124725,
          0.24611230194568634, 0.33791524171829224, 0.44070982933044434, 0.5626170039176941,
          0.7229568362236023, 1.0)


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def _layer(name, n, k, M, r, act, bias=False, mul=False, residual=False, step=False, block=64, dq=True):
    return dict(name=name, op="layer", n=n, k=k, M=M, r=r, act=act, bias=bias, mul=mul, residual=residual,
                step=step, block=block, dq=dq)


def _moe(name, M, E, top_k, H, F, act="silu", renorm=True, residual=False, block=64, dq=True):
    return dict(name=name, op="moe", M=M, E=E, top_k=top_k, H=H, F=F, act=act, renorm=renorm,
                residual=residual, block=block, dq=dq)


def listed():
    return [
        # one token through the gate projection of a gated MLP, times the up projection
        _layer("decode_gate_1", 13824, 5120, 1, 16, "silu", mul=True),
        # a ragged decode batch through the down projection, added to the residual stream
        _layer("decode_down_13", 5120, 13824, 13, 16, "none", residual=True),
        # a short prompt through a biased projection with its activation
        _layer("prefill_gelu_517", 5120, 5120, 517, 16, "gelu_tanh", bias=True, block=128, dq=False),
        # a prefill batch through the gate projection
        _layer("prefill_gate_4096", 13824, 5120, 4096, 16, "silu", mul=True),
        # training step of a small biased layer, odd token count
        _layer("train_small_100", 1024, 1024, 100, 8, "gelu", bias=True, residual=True, step=True, dq=False),
        # training step of an attention-sized projection with bias, activation and residual
        _layer("train_relu_2048", 5120, 5120, 2048, 16, "relu", bias=True, residual=True, step=True),
        # training step of the gate projection of a 70B-sized MLP
        _layer("train_gate_4096", 28672, 8192, 4096, 64, "silu", mul=True, step=True),
        # one token, many small experts
        _moe("moe_1_of_64x8", 1, 64, 8, 2048, 1024),
        # a few tokens, few large experts
        _moe("moe_4_of_8x2", 4, 8, 2, 5120, 13824),
        # a decode batch over many small experts of an odd width, added to the residual stream
        _moe("moe_16_of_64x6", 16, 64, 6, 2048, 1408, residual=True),
        # a larger ragged decode batch, weights as the softmax gave them, 128-element blocks
        _moe("moe_37_of_32x4", 37, 32, 4, 4096, 1792, act="gelu_tanh", renorm=False, block=128, dq=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.6:
        block = rng.choice((64, 64, 128))
        n = 8 * _log(rng, 16, 2400)
        k = block * _log(rng, 512 // block, 14336 // block)
        step = rng.random() < 0.5
        M = _log(rng, 1, 4096)
        if rng.random() < 0.3:
            M = rng.randint(1, 16)
        while M * n * k > 4096 * 28672 * 8192 // 4:
            M //= 2
        return dict(op="layer", n=n, k=k, M=M, r=8 * rng.randint(1, 16),
                    act=rng.choice(("none", "relu", "silu", "gelu_tanh", "gelu")), bias=rng.random() < 0.5,
                    mul=rng.random() < 0.5, residual=rng.random() < 0.5, step=step, block=block,
                    dq=rng.random() < 0.7)
    block = rng.choice((64, 64, 128))
    E = _log(rng, 2, 128)
    top_k = rng.randint(1, min(E, 8))
    H = block * _log(rng, 512 // block, 5120 // block)
    F = block * _log(rng, 256 // block, 8192 // block)
    while E * H * F > 8 * 5120 * 13824:
        F = max(block, F // 2 // block * block)
    return dict(op="moe", M=_log(rng, 1, 64), E=E, top_k=top_k, H=H, F=F,
                act=rng.choice(("silu", "silu", "gelu_tanh", "relu")), renorm=rng.random() < 0.5,
                residual=rng.random() < 0.5, block=block, dq=rng.random() < 0.7)


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(torch.bfloat16)


def _nf4(g, n, k, block, dq, std):
    """Random normal weights, quantised: codes, block scales and their 8-bit form."""
    nb = n * k // block
    lv = torch.tensor(LEVELS, device="cuda")
    mid = (lv[1:] + lv[:-1]) / 2
    codes = torch.empty(n * k // 2, dtype=torch.uint8, device="cuda")
    absmax = torch.empty(nb, device="cuda")
    rows = max(1, (1 << 26) // block)                    # bounded scratch
    for b0 in range(0, nb, rows):
        w = torch.randn(min(rows, nb - b0), block, generator=g, device="cuda") * std
        s = w.abs().amax(1)
        c = torch.bucketize(w / s[:, None], mid).to(torch.uint8).view(-1, 2)
        absmax[b0:b0 + len(s)] = s
        codes[b0 * block // 2:(b0 + len(s)) * block // 2] = c[:, 0] * 16 + c[:, 1]
    q8 = c8 = None
    if dq:
        ng = (nb + 255) // 256
        pad = torch.zeros(ng * 256, device="cuda")
        pad[:nb] = absmax
        c8 = pad.view(ng, 256).amax(1)
        q8 = (pad.view(ng, 256) / c8[:, None] * 127).round().to(torch.uint8).view(-1)[:nb].contiguous()
    return dict(n=n, k=k, block=block, dq=dq, codes=codes, absmax=absmax, q8=q8, c8=c8)


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case=case)
    if case["op"] == "layer":
        n, k, M, r = case["n"], case["k"], case["M"], case["r"]
        s["w"] = _nf4(g, n, k, case["block"], case["dq"], 0.02)
        s["x"] = _normal(g, M, k)
        s["A"] = ((torch.rand(r, k, generator=g, device="cuda") * 2 - 1) / math.sqrt(k)).to(torch.bfloat16)
        s["B"] = _normal(g, n, r, std=0.01)
        s["alpha"] = 2.0 * r
        s["bias"] = _normal(g, n, std=0.5) if case["bias"] else None
        s["mul"] = _normal(g, M, n) if case["mul"] else None
        s["residual"] = _normal(g, M, n) if case["residual"] else None
        s["dH"] = _normal(g, M, n) if case["step"] else None
    else:
        M, E, H, F = case["M"], case["E"], case["H"], case["F"]
        s["gate_up"] = _nf4(g, E * 2 * F, H, case["block"], case["dq"], 0.02)
        s["down"] = _nf4(g, E * H, F, case["block"], case["dq"], 0.02)
        s["x"] = _normal(g, M, H)
        s["router"] = _normal(g, E, H, std=0.02)
        s["residual"] = _normal(g, M, H) if case["residual"] else None
    return s


# ---------------------------------------------------------------------------
# The plain form
# ---------------------------------------------------------------------------
def _act(z, act):
    if act == "relu":
        return z.clamp_min(0)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    if act == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    return torch.ones_like(z)


def _scales(w):
    if not w["dq"]:
        return w["absmax"]
    c = (w["c8"] / 127).repeat_interleave(256)[:w["q8"].numel()]
    return w["q8"].float() * c


def _codes(c):
    return torch.stack((c >> 4, c & 15), -1).flatten(-2)


def _dequant(w):
    """W~ [n, k] in fp32."""
    lv = torch.tensor(LEVELS, device="cuda")
    return (lv[_codes(w["codes"].view(-1, w["block"] // 2)).int()] * _scales(w)[:, None]).view(w["n"], w["k"])


def _dequant_experts(w, E, chosen):
    """W~ of the chosen ones of E stacked weights, [len(chosen), n / E, k] in fp32."""
    lv = torch.tensor(LEVELS, device="cuda")
    c = _codes(w["codes"].view(E, -1)[chosen].view(len(chosen), -1, w["block"] // 2))
    s = _scales(w).view(E, -1)[chosen]
    return (lv[c.int()] * s[:, :, None]).view(len(chosen), w["n"] // E, w["k"])


def _plain_layer(s):
    c, x, A, B = s["case"], s["x"].float(), s["A"].float(), s["B"].float()
    W, sc = _dequant(s["w"]), s["alpha"] / c["r"]
    u = x @ A.T
    z = x @ W.T + sc * (u @ B.T)
    if c["bias"]:
        z = z + s["bias"].float()
    h = _act(z, c["act"])
    if c["mul"]:
        h = h * s["mul"].float()
    if c["residual"]:
        h = h + s["residual"].float()
    out = {"h": h.to(torch.bfloat16)}
    if not c["step"]:
        return out
    dH = s["dH"].float()
    dz = dH * _act_grad(z, c["act"])
    if c["mul"]:
        dz = dz * s["mul"].float()
        out["dmul"] = (dH * _act(z, c["act"])).to(torch.bfloat16)
    if c["bias"]:
        out["dbias"] = dz.sum(0).to(torch.bfloat16)
    v = dz @ B
    out["dX"] = (dz @ W + sc * (v @ A)).to(torch.bfloat16)
    out["dA"] = (sc * (v.T @ x)).to(torch.bfloat16)
    out["dB"] = (sc * (dz.T @ u)).to(torch.bfloat16)
    return out


def _plain_moe(s):
    c, x = s["case"], s["x"].float()
    E, F = c["E"], c["F"]
    logits = s["x"].double() @ s["router"].double().T            # next to a border: 64 bits
    ids = torch.sort(logits, dim=1, descending=True, stable=True)[1][:, :c["top_k"]]
    p = torch.softmax(logits, dim=1).gather(1, ids)
    if c["renorm"]:
        p = p / p.sum(1, keepdim=True)
    p = p.float()
    chosen = ids.unique()
    gu = x @ _dequant_experts(s["gate_up"], E, chosen).transpose(1, 2)          # [chosen, M, 2F]
    a = _act(gu[:, :, :F], c["act"]) * gu[:, :, F:]
    y = a @ _dequant_experts(s["down"], E, chosen).transpose(1, 2)              # [chosen, M, H]
    share = ((ids[None] == chosen[:, None, None]) * p[None]).sum(2)             # [chosen, M]
    out = (share[:, :, None] * y).sum(0)
    if c["residual"]:
        out = out + s["residual"].float()
    return {"out": out.to(torch.bfloat16), "ids": ids.int(), "weights": p}


# ---------------------------------------------------------------------------
# The framework's calls
# ---------------------------------------------------------------------------
def _handle(q, w):
    return q.QuantizedWeight(w["n"], w["k"], w["dq"], w["codes"], w["absmax"], w["q8"], w["c8"], w["block"])


def _own_layer(s):
    import bit_nf4_quantized_05_b200 as q
    c = s["case"]
    w = _handle(q, s["w"])
    h, u, z = q.qlora_linear_fwd_epilogue(w, s["x"], s["A"], s["B"], s["alpha"], bias=s["bias"], act=c["act"],
                                          mul=s["mul"], residual=s["residual"], save_u=c["step"],
                                          save_z=c["step"])
    out = {"h": h}
    if c["step"]:
        dX, dA, dB, dbias, dmul = q.qlora_linear_bwd_epilogue(w, s["x"], s["A"], s["B"], s["alpha"], s["dH"], z,
                                                              act=c["act"], mul=s["mul"], u=u,
                                                              need_dbias=c["bias"])
        if c["mul"]:
            out["dmul"] = dmul
        if c["bias"]:
            out["dbias"] = dbias
        out.update(dX=dX, dA=dA, dB=dB)
    return out


def _own_moe(s):
    import bit_nf4_quantized_05_b200 as q
    c = s["case"]
    out, ids, weights = q.nf4_moe_fwd(_handle(q, s["gate_up"]), _handle(q, s["down"]), s["x"], s["router"],
                                      c["top_k"], act=c["act"], renormalise=c["renorm"], residual=s["residual"])
    return {"out": out, "ids": ids, "weights": weights}


def run(state):
    if own:
        return _own_layer(state) if state["case"]["op"] == "layer" else _own_moe(state)
    return _plain_layer(state) if state["case"]["op"] == "layer" else _plain_moe(state)


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------
def _weight_bytes(n, k, block, dq):
    return n * k // 2 + n * k // block * (1 if dq else 4) + (n * k // block // 256 * 4 if dq else 0)


def work(case):
    if case["op"] == "layer":
        n, k, M, r = case["n"], case["k"], case["M"], case["r"]
        tall = case["mul"] + case["residual"]
        b = _weight_bytes(n, k, case["block"], case["dq"]) + 2 * M * k + 2 * r * (n + k) + 2 * M * n * (1 + tall)
        b += 2 * n * case["bias"]
        f = 2 * M * n * k + 2 * M * r * (n + k)
        if case["step"]:
            # dH in; dX, dmul, dA, dB, dbias out
            b += 2 * M * n * (1 + case["mul"]) + 2 * M * k + 2 * r * (n + k) + 2 * n * case["bias"]
            f += 2 * M * n * k + 4 * M * r * (n + k)
        return {"bytes": b, "flops": f}
    M, E, H, F, t = case["M"], case["E"], case["H"], case["F"], case["top_k"]
    # experts that M tokens are expected to choose
    used = E * (1 - (1 - t / E) ** M)
    b = used / E * (_weight_bytes(2 * E * F, H, case["block"], case["dq"]) +
                    _weight_bytes(E * H, F, case["block"], case["dq"]))
    b += 2 * E * H + 2 * M * H * (2 + case["residual"]) + 8 * M * t
    return {"bytes": int(b), "flops": 2 * M * E * H + 6 * M * t * H * F}


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------
def _d(t):
    return t.to(torch.float64)


def _weight64(w, first, rows):
    """Rows [first, first + rows) of W~ in 64 bits."""
    k, bs = w["k"], w["block"]
    byte = w["codes"].view(-1, k // 2)[first:first + rows].long()
    level = torch.tensor(LEVELS, dtype=torch.float64, device="cuda")
    block = torch.arange(first * k // bs, (first + rows) * k // bs, device="cuda")
    if w["dq"]:
        scale = _d(w["q8"])[block] * _d(w["c8"])[block // 256] / 127
    else:
        scale = _d(w["absmax"])[block]
    out = torch.empty(rows, k, dtype=torch.float64, device="cuda")
    out[:, 0::2] = level[byte // 16]
    out[:, 1::2] = level[byte % 16]
    return out * scale.view(rows, k // bs).repeat_interleave(bs, 1)


def _sigma(z):
    return torch.sigmoid(z)


def _act64(z, act):
    """(act, its derivative)."""
    if act == "relu":
        return torch.where(z > 0, z, 0.0), torch.where(z > 0, 1.0, 0.0).to(z.dtype)
    if act == "silu":
        return z * _sigma(z), _sigma(z) + z * _sigma(z) * _sigma(-z)
    if act == "gelu":
        cdf = 0.5 * torch.erfc(-z / 2 ** 0.5)
        return z * cdf, cdf + z * torch.exp(-z * z / 2) / (2 * math.pi) ** 0.5
    if act == "gelu_tanh":
        a = (2 / math.pi) ** 0.5
        v = 2 * a * (z + 0.044715 * z ** 3)              # (1 + tanh(v / 2)) / 2 = sigma(v)
        return z * _sigma(v), _sigma(v) + z * _sigma(v) * _sigma(-v) * 2 * a * (1 + 0.134145 * z ** 2)
    return z, torch.ones_like(z)


def exact(case, seed):
    s = prepare(case, seed)
    x = _d(s["x"])
    if case["op"] == "layer":
        n, k, M, r = case["n"], case["k"], case["M"], case["r"]
        if (3 if case["step"] else 1) * 2 * M * n * k > 1e13:
            return None                                   # over 20 seconds in 64 bits
        A, B, f = _d(s["A"]), _d(s["B"]), s["alpha"] / r
        h = torch.empty(M, n, dtype=torch.float64, device="cuda")
        dX = torch.zeros(M, k, dtype=torch.float64, device="cuda")
        dB = torch.empty(n, r, dtype=torch.float64, device="cuda")
        dbias = torch.empty(n, dtype=torch.float64, device="cuda")
        dmul = torch.empty(M, n, dtype=torch.float64, device="cuda") if case["mul"] else None
        u, v = x @ A.T, torch.zeros(M, r, dtype=torch.float64, device="cuda")
        for j in range(0, n, 4096):                       # columns of h, a stripe at a time
            e = min(n, j + 4096)
            W = _weight64(s["w"], j, e - j)
            z = x @ W.T + f * (u @ B[j:e].T)
            if case["bias"]:
                z += _d(s["bias"][j:e])
            a, da = _act64(z, case["act"])
            h[:, j:e] = a * _d(s["mul"][:, j:e]) if case["mul"] else a
            if case["residual"]:
                h[:, j:e] += _d(s["residual"][:, j:e])
            if case["step"]:
                g = _d(s["dH"][:, j:e])
                dz = g * da
                if case["mul"]:
                    dz *= _d(s["mul"][:, j:e])
                    dmul[:, j:e] = g * a
                dbias[j:e] = dz.sum(0)
                dB[j:e] = f * (dz.T @ u)
                dX += dz @ W
                v += dz @ B[j:e]
        out = {"h": h}
        if case["step"]:
            if case["mul"]:
                out["dmul"] = dmul
            if case["bias"]:
                out["dbias"] = dbias
            out.update(dX=dX + f * (v @ A), dA=f * (v.T @ x), dB=dB)
        return out
    E, H, F, t = case["E"], case["H"], case["F"], case["top_k"]
    logits = x @ _d(s["router"]).T
    # rank of expert e: how many are larger, or equal with a lower index
    e = torch.arange(E, device="cuda")
    above = (logits[:, None, :] > logits[:, :, None]) | ((logits[:, None, :] == logits[:, :, None]) & (e < e[:, None]))
    ids = torch.argsort(above.sum(2), 1)[:, :t]
    odds = torch.exp(logits - logits.amax(1, keepdim=True))
    share = odds.gather(1, ids)
    share = share / (share if case["renorm"] else odds).sum(1, keepdim=True)
    out = _d(s["residual"]) if case["residual"] else torch.zeros_like(x)
    for i in ids.unique().tolist():
        tok, slot = (ids == i).nonzero(as_tuple=True)
        xi = x[tok]
        gate, _ = _act64(xi @ _weight64(s["gate_up"], i * 2 * F, F).T, case["act"])
        up = xi @ _weight64(s["gate_up"], i * 2 * F + F, F).T
        y = (gate * up) @ _weight64(s["down"], i * H, H).T
        out.index_add_(0, tok, share[tok, slot][:, None] * y)
    return {"out": out, "ids": ids.int(), "weights": share}
