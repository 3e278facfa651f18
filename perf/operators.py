"""Cases, plain forms and 64-bit values of three operators of a 4-bit serving step.

  int4_pack    int4 codes of a weight matrix with one scale (and, if asked, one
               zero point) per group of 32, 64 or 128 weights of a row
  int4_linear  y = x . dequant(W)^T (+ bias) over such a matrix, for one row of
               activations up to a few hundred
  moe_layer    a whole mixture-of-experts layer for 1 to 64 tokens over NF4 or
               MXFP4 expert stacks: router top-k and softmax, gate_up, SwiGLU,
               down, the weighted sum over each token's experts, an optional
               residual

With ``own`` false, ``run`` computes them from elementary torch operations in 32
bits, rounded once at the end; with ``own`` true it makes the calls that a user
makes of ``grouped_nf4_expert_amd.gnf4``.
"""

import math

import torch

own = False

DEV = "cuda:0"

NF4 = (-1.0, -0.6961928009986877, -0.5250730514526367, -0.39491748809814453,
       -0.28444138169288635, -0.18477343022823334, -0.09105003625154495, 0.0,
       0.07958029955625534, 0.16093020141124725, 0.2461123913526535, 0.33791524171829224,
       0.44070982933044434, 0.5626170039176941, 0.7229568362236023, 1.0)
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)

SCALE_DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def _lib():
    from grouped_nf4_expert_amd import gnf4
    return gnf4


# ------------------------------------------------------------------- cases

def _pack(n, k, group, asym, w, scale):
    return {"op": "int4_pack", "n": n, "k": k, "group": group, "asym": asym, "w": w,
            "scale": scale}


def _linear(m, n, k, group, asym, scale, bias):
    return {"op": "int4_linear", "m": m, "n": n, "k": k, "group": group, "asym": asym,
            "scale": scale, "bias": bias}


def _moe(t, e, top_k, h, i, fmt, residual):
    return {"op": "moe_layer", "t": t, "e": e, "top_k": top_k, "h": h, "i": i, "fmt": fmt,
            "residual": residual}


def listed():
    cases = [
        # one square projection quantised as a checkpoint is loaded
        ("pack 2048x2048", _pack(2048, 2048, 128, False, "bf16", "bf16")),
        # a wide fp32 matrix with zero points and a K that 128 does not divide
        ("pack 5760x2880 zero points", _pack(5760, 2880, 32, True, "f32", "f32")),
        # a batch-1 decode step's small projection: the smallest call, all latency
        ("linear 1x2048x2048", _linear(1, 2048, 2048, 128, False, "bf16", False)),
        # batch-1 with fine groups, zero points and a bias, K not a multiple of 128
        ("linear 1x5760x2880 zero points", _linear(1, 5760, 2880, 32, True, "f32", True)),
        # an output head over a vocabulary of odd size: the largest weight stream
        ("linear 1x65537x8192", _linear(1, 65537, 8192, 128, False, "bf16", False)),
        # a small batch of decode tokens
        ("linear 13x4096x7168", _linear(13, 4096, 7168, 64, False, "bf16", False)),
        # a chunk of a prompt: matrix products rather than a weight stream
        ("linear 256x7168x2048", _linear(256, 7168, 2048, 128, True, "bf16", False)),
        # batch-1 decode of a 64-expert layer: the smallest layer call
        ("moe 1 token 64 experts", _moe(1, 64, 8, 2048, 1024, "nf4", False)),
        # two tokens over a native MXFP4 checkpoint's layer, odd widths
        ("moe 2 tokens mxfp4", _moe(2, 128, 4, 2880, 2880, "mxfp4", True)),
        # a small serving batch over 128 narrow experts
        ("moe 8 tokens 128 experts", _moe(8, 128, 8, 2048, 768, "nf4_bf16", True)),
        # the largest batch: nearly every expert read, several rows each
        ("moe 64 tokens 64 experts", _moe(64, 64, 8, 2048, 1024, "nf4", False)),
        # a small batch over a very large layer (256 experts, gigabytes read)
        ("moe 16 tokens 256 experts", _moe(16, 256, 8, 7168, 2048, "nf4", False)),
    ]
    return [dict(c, name=name) for name, c in cases]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


_LARGEST = {"int4_pack": 5760 * 2880, "int4_linear": 65537 * 8192, "moe_layer": 256 * 7168 * 2048}


def draw(rng):
    op = rng.choice(("int4_pack", "int4_linear", "int4_linear", "moe_layer", "moe_layer"))
    while True:
        group = rng.choice((32, 64, 128))
        if op == "int4_pack":
            n, k = _log(rng, 1, 8192), group * _log(rng, 1, 8192 // group)
            size = n * k
            case = _pack(n, k, group, rng.random() < 0.5, rng.choice(("bf16", "f32")),
                         rng.choice(("bf16", "f32")))
        elif op == "int4_linear":
            m, n = _log(rng, 1, 256), _log(rng, 64, 65537)
            k = group * _log(rng, 1, 8192 // group)
            size = n * k * max(1, m // 16)
            case = _linear(m, n, k, group, rng.random() < 0.5, rng.choice(("bf16", "f32")),
                           rng.random() < 0.5)
        else:
            e = _log(rng, 4, 256)
            top_k = rng.randint(1, min(e, 8))
            h, i = 64 * _log(rng, 2, 112), 64 * _log(rng, 1, 45)
            t = _log(rng, 1, 64)
            size = e * h * i * max(1, t // 16)
            case = _moe(t, e, top_k, h, i, rng.choice(("nf4", "nf4_bf16", "mxfp4")),
                        rng.random() < 0.5)
        if size <= _LARGEST[op]:
            return case


# ------------------------------------------------------------------ inputs

def _bell_bytes(shape, gen):
    """Bytes of two int4 codes each, distributed as rounded normal weights are."""
    def code():
        v = torch.randn(shape, device=DEV, generator=gen).mul_(2.6).round_().add_(8)
        return v.clamp_(0, 15).to(torch.uint8)
    return (code() << 4) | code()


def _int4_weights(case, gen):
    n, k, g = case["n"], case["k"], case["group"]
    packed = torch.empty((n, k // 2), dtype=torch.uint8, device=DEV)
    for r in range(0, n, 8192):
        rows = min(8192, n - r)
        packed[r:r + rows] = _bell_bytes((rows, k // 2), gen)
    scales = torch.rand((n, k // g), device=DEV, generator=gen) * 0.01 + 0.005
    zeros = None
    if case["asym"]:
        zeros = torch.randint(5, 12, (n, k // g), device=DEV, generator=gen, dtype=torch.uint8)
    return packed, scales.to(SCALE_DTYPES[case["scale"]]), zeros


def _expert_stack(e, n, k, fmt, gen):
    """Codes of a stack [e, n, k].  NF4's levels are quantiles of the normal
    distribution, so the codes of normal weights are close to uniform."""
    packed = torch.empty((e, n, k // 2), dtype=torch.uint8, device=DEV)
    flat = packed.view(-1)
    step = 1 << 30
    for a in range(0, flat.numel(), step):
        b = min(a + step, flat.numel())
        flat[a:b] = torch.randint(0, 256, (b - a,), dtype=torch.uint8, device=DEV, generator=gen)
    if fmt == "mxfp4":
        scales = torch.randint(118, 122, (e, n, k // 32), dtype=torch.uint8, device=DEV,
                               generator=gen)
    else:
        scales = torch.rand((e, n, k // 64), device=DEV, generator=gen) * 0.03 + 0.035
        if fmt == "nf4_bf16":
            scales = scales.to(torch.bfloat16)
    return packed, scales


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    state = {"case": case}
    if case["op"] == "int4_pack":
        w = torch.randn((case["n"], case["k"]), device=DEV, generator=gen) * 0.02
        state["w"] = w.to(torch.bfloat16) if case["w"] == "bf16" else w
    elif case["op"] == "int4_linear":
        state["weights"] = _int4_weights(case, gen)
        state["x"] = torch.randn((case["m"], case["k"]), device=DEV,
                                 generator=gen).to(torch.bfloat16)
        state["bias"] = None
        if case["bias"]:
            state["bias"] = torch.randn(case["n"], device=DEV, generator=gen).to(torch.bfloat16)
    else:
        t, e, h, i = case["t"], case["e"], case["h"], case["i"]
        state["logits"] = torch.randn((t, e), device=DEV, generator=gen)
        state["x"] = torch.randn((t, h), device=DEV, generator=gen).to(torch.bfloat16)
        state["gate_up"] = _expert_stack(e, 2 * i, h, case["fmt"], gen)
        state["down"] = _expert_stack(e, h, i, case["fmt"], gen)
        state["residual"] = None
        if case["residual"]:
            state["residual"] = torch.randn((t, h), device=DEV, generator=gen).to(torch.bfloat16)
        if own:
            state["buffers"] = _lib().MoeLayerBuffers(t, e, case["top_k"], h, i, DEV)
    return state


# ------------------------------------------------------------- plain forms

def _plain_pack(state):
    """Scale: the largest magnitude over 7 (or the range over 15, the range
    always holding zero), in 32 bits, stored in the scale's type.  Code: the
    level nearest to the weight, ties to the lower code, counted from the
    midpoints between levels in 64 bits, where their products are exact."""
    case, w = state["case"], state["w"].float()
    n, k, g = case["n"], case["k"], case["group"]
    w = w.view(n, k // g, g)
    if case["asym"]:
        lo, hi = w.amin(2).clamp_max(0.0), w.amax(2).clamp_min(0.0)
        d = torch.full_like(hi, 15.0)
        scale = (hi / d - lo / d).to(SCALE_DTYPES[case["scale"]])
    else:
        a = w.abs().amax(2)
        scale = (a / torch.full_like(a, 7.0)).to(SCALE_DTYPES[case["scale"]])
    s = scale.double()
    mids = torch.arange(15, device=w.device, dtype=torch.float64) + 0.5
    if case["asym"]:
        zero = (-lo.double().unsqueeze(2) > mids * s.unsqueeze(2)).sum(2)
        zero = torch.where(s == 0, torch.zeros_like(zero), zero)
    else:
        zero = torch.full_like(scale, 8, dtype=torch.int64)
    codes = torch.zeros(w.shape, dtype=torch.uint8, device=w.device)
    wd = w.double()
    for j in range(15):
        mid = (j + 0.5 - zero.double()) * s
        codes += (wd > mid.unsqueeze(2)).to(torch.uint8)
    codes = torch.where((s == 0).unsqueeze(2), zero.unsqueeze(2).to(torch.uint8), codes)
    codes = codes.view(n, k)
    packed = (codes[:, 0::2] << 4) | codes[:, 1::2]
    if case["asym"]:
        return packed, scale, zero.to(torch.uint8)
    return packed, scale


def _high_first(packed):
    codes = torch.stack((packed >> 4, packed & 15), dim=-1)
    return codes.view(packed.shape[:-1] + (packed.shape[-1] * 2,))


def _low_first(packed):
    codes = torch.stack((packed & 15, packed >> 4), dim=-1)
    return codes.view(packed.shape[:-1] + (packed.shape[-1] * 2,))


def _plain_linear(state):
    case, x = state["case"], state["x"].float()
    packed, scales, zeros = state["weights"]
    n, k, g = case["n"], case["k"], case["group"]
    parts = []
    for r in range(0, n, 16384):
        q = _high_first(packed[r:r + 16384]).float().view(-1, k // g, g)
        z = 8.0 if zeros is None else zeros[r:r + 16384].float().unsqueeze(2)
        w = (q - z) * scales[r:r + 16384].float().unsqueeze(2)
        parts.append(x @ w.view(-1, k).t())
    y = torch.cat(parts, dim=1)
    if state["bias"] is not None:
        y = y + state["bias"].float()
    return y.to(torch.bfloat16)


def _plain_weights(packed, scales):
    """An expert stack's weights in 32 bits."""
    if scales.dtype == torch.uint8:
        table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=packed.device)
        w = table[_low_first(packed).int()]
        s, block = torch.exp2(scales.float() - 127.0), 32
    else:
        table = torch.tensor(NF4, device=packed.device)
        w = table[_high_first(packed).int()]
        s, block = scales.float(), 64
    shape = w.shape
    return (w.view(shape[:-1] + (-1, block)) * s.unsqueeze(-1)).view(shape)


def _silu(v):
    return v / (1.0 + torch.exp(-v))


def _plain_moe(state):
    case = state["case"]
    logits, x = state["logits"], state["x"].float()
    t, e, k, h, i = case["t"], case["e"], case["top_k"], case["h"], case["i"]
    order = torch.sort(logits, dim=1, descending=True, stable=True)
    ids, best = order.indices[:, :k], order.values[:, :k]
    ex = torch.exp(best - best[:, :1])
    w = ex / ex.sum(1, keepdim=True)
    (gp, ga), (dp, da) = state["gate_up"], state["down"]
    out = torch.zeros((t, h), device=x.device)
    if state["residual"] is not None:
        out += state["residual"].float()
    if t * k <= e:  # few picks: each token's experts
        for r in range(t):
            for j in range(k):
                one = ids[r, j:j + 1]
                gu = x[r:r + 1] @ _plain_weights(gp[one], ga[one])[0].t()
                act = _silu(gu[:, :i]) * gu[:, i:]
                y = act @ _plain_weights(dp[one], da[one])[0].t()
                out[r] += w[r, j] * y[0]
    else:           # many: every expert over every token, unpicked ones at weight zero
        dense = torch.zeros((t, e), device=x.device).scatter(1, ids, w)
        for n in range(e):
            gu = x @ _plain_weights(gp[n], ga[n]).t()
            act = _silu(gu[:, :i]) * gu[:, i:]
            y = act @ _plain_weights(dp[n], da[n]).t()
            out += dense[:, n:n + 1] * y
    return out.to(torch.bfloat16), ids.int(), w


def run(state):
    case = state["case"]
    if case["op"] == "int4_pack":
        if not own:
            return _plain_pack(state)
        packed, scales, zeros = _lib().int4_pack(state["w"], case["group"],
                                                 zero_points=case["asym"],
                                                 scale_dtype=SCALE_DTYPES[case["scale"]])
        return (packed, scales, zeros) if case["asym"] else (packed, scales)
    if case["op"] == "int4_linear":
        if not own:
            return _plain_linear(state)
        packed, scales, zeros = state["weights"]
        return _lib().int4_linear(state["x"], packed, scales, zeros, bias=state["bias"])
    if not own:
        return _plain_moe(state)
    return _lib().moe_layer(state["logits"], state["x"], state["gate_up"], state["down"],
                            case["top_k"], residual=state["residual"], buffers=state["buffers"])


# -------------------------------------------------------------------- work

def work(case):
    if case["op"] == "int4_pack":
        n, k, g = case["n"], case["k"], case["group"]
        per_group = (2 if case["scale"] == "bf16" else 4) + (1 if case["asym"] else 0)
        in_bytes = (2 if case["w"] == "bf16" else 4) * n * k
        return {"bytes": in_bytes + n * k // 2 + per_group * n * (k // g), "flops": 4 * n * k}
    if case["op"] == "int4_linear":
        m, n, k, g = case["m"], case["n"], case["k"], case["group"]
        per_group = (2 if case["scale"] == "bf16" else 4) + (1 if case["asym"] else 0)
        bias = 2 * n if case["bias"] else 0
        return {"bytes": n * k // 2 + per_group * n * (k // g) + 2 * m * (n + k) + bias,
                "flops": 2 * m * n * k}
    t, e, k, h, i = case["t"], case["e"], case["top_k"], case["h"], case["i"]
    touched = e * (1.0 - (1.0 - k / e) ** t)  # expected distinct experts of independent tokens
    weights = 3 * h * i
    per = {"nf4": 4 / 64, "nf4_bf16": 2 / 64, "mxfp4": 1 / 32}[case["fmt"]]
    rows = 2 * t * h * (3 if case["residual"] else 2)
    return {"bytes": int(touched * weights * (0.5 + per)) + rows + 4 * t * e + 8 * t * k,
            "flops": 2 * t * k * weights}


# ----------------------------------------------------------- 64-bit values

def _exact_nibbles(packed, high_first):
    """Codes [..., K] from bytes, element by element of each byte."""
    b = packed.to(torch.int64)
    out = torch.empty(packed.shape[:-1] + (2 * packed.shape[-1],), dtype=torch.int64,
                      device=packed.device)
    out[..., 0::2] = b // 16 if high_first else b % 16
    out[..., 1::2] = b % 16 if high_first else b // 16
    return out


def _exact_expert(packed, scales):
    if scales.dtype == torch.uint8:
        code = _exact_nibbles(packed, False)
        exp, man, sign = (code // 2) % 4, code % 2, code // 8
        mag = torch.where(exp == 0, man * 0.5,
                          torch.ldexp(1.0 + man.double() * 0.5, (exp - 1).double()))
        val = torch.where(sign == 1, -mag, mag).double()
        scale = torch.ldexp(torch.ones_like(scales, dtype=torch.float64),
                            scales.double() - 127.0)
        return val * scale.repeat_interleave(32, dim=-1)
    val = torch.tensor(NF4, dtype=torch.float32, device=packed.device).double()
    return val[_exact_nibbles(packed, True)] * scales.double().repeat_interleave(64, dim=-1)


def _exact_pack(state):
    case, w = state["case"], state["w"].double()
    n, k, g = case["n"], case["k"], case["group"]
    blocks = w.reshape(-1, g)
    if case["asym"]:
        top = torch.relu(blocks.max(dim=1).values)
        low = torch.relu((-blocks).max(dim=1).values)
        stored = ((top / 15.0).float() + (low / 15.0).float()).to(SCALE_DTYPES[case["scale"]])
    else:
        stored = (blocks.abs().max(dim=1).values / 7.0).float().to(SCALE_DTYPES[case["scale"]])
    s = stored.double()
    safe = torch.where(s == 0, torch.ones_like(s), s)

    def nearest(v):  # nearest whole number to v / s, ties down, checked by exact products
        c = torch.floor(v / safe.unsqueeze(1))
        c = c - ((c * safe.unsqueeze(1)) > v).double()
        return c + ((c + 0.5) * safe.unsqueeze(1) < v).double()

    if case["asym"]:
        zero = nearest(low.unsqueeze(1)).clamp(0, 15).squeeze(1)
        zero = torch.where(s == 0, torch.zeros_like(zero), zero)
    else:
        zero = torch.full_like(s, 8.0)
    code = (nearest(blocks) + zero.unsqueeze(1)).clamp(0, 15)
    code = torch.where((s == 0).unsqueeze(1), zero.unsqueeze(1), code).to(torch.int64)
    code = code.reshape(n, k // 2, 2)
    packed = (code[:, :, 0] * 16 + code[:, :, 1]).to(torch.uint8)
    stored = stored.view(n, k // g)
    if case["asym"]:
        return packed, stored, zero.to(torch.uint8).view(n, k // g)
    return packed, stored


def _exact_linear(state):
    case, x = state["case"], state["x"].double()
    packed, scales, zeros = state["weights"]
    n, g = case["n"], case["group"]
    y = torch.empty((case["m"], n), dtype=torch.float64, device=x.device)
    for r in range(0, n, 4096):
        code = _exact_nibbles(packed[r:r + 4096], True).double()
        if zeros is None:
            code -= 8.0
        else:
            code -= zeros[r:r + 4096].double().repeat_interleave(g, dim=1)
        code *= scales[r:r + 4096].double().repeat_interleave(g, dim=1)
        y[:, r:r + 4096] = torch.mm(code, x.t().contiguous()).t()
    if state["bias"] is not None:
        y += state["bias"].double()
    return y


def _exact_moe(state):
    case = state["case"]
    k, i = case["top_k"], case["i"]
    logits, x = state["logits"].cpu().double(), state["x"].double()
    ids = [sorted(range(case["e"]), key=lambda n: (-row[n], n))[:k] for row in logits.tolist()]
    picks = torch.tensor(ids, dtype=torch.int64)
    w = torch.softmax(torch.gather(logits, 1, picks), dim=1)
    out = torch.zeros((case["t"], case["h"]), dtype=torch.float64, device=x.device)
    if state["residual"] is not None:
        out += state["residual"].double()
    rows_of = {}
    for r, row in enumerate(ids):
        for j, n in enumerate(row):
            rows_of.setdefault(n, []).append((r, j))
    for n, rows in rows_of.items():
        tok = torch.tensor([r for r, _ in rows], device=x.device)
        wt = torch.stack([w[r, j] for r, j in rows]).to(x.device)
        gu = torch.mm(_exact_expert(state["gate_up"][0][n], state["gate_up"][1][n]),
                      x[tok].t().contiguous())
        act = gu[:i] * torch.sigmoid(gu[:i]) * gu[i:]
        y = torch.mm(_exact_expert(state["down"][0][n], state["down"][1][n]), act)
        out.index_add_(0, tok, (y * wt).t().contiguous())
    return out, picks.int(), w


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "int4_pack":
        return _exact_pack(state)
    if case["op"] == "int4_linear":
        return _exact_linear(state)
    return _exact_moe(state)
