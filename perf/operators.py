"""Cases and plain forms of the few-token expert layer and of the fp8
block-scale operators (product, token quantisation, SiLU*mul quantisation)."""
import torch

own = False

BLOCK = 128        # one fp32 scale per 128 values of a token row, per 128 x 128 weights
E4M3_MAX = 448.0   # largest e4m3fn value
TINY = 1e-12       # smallest block maximum a scale is made from


def listed():
    return [
        # one sequence decoding on the 48-expert top-3 layer (5120 / 8 columns an expert)
        {"name": "few_1_e48", "op": "few", "T": 1, "valid": 1, "H": 7168, "E": 48, "k": 3,
         "I": 640, "shared": 0, "fp8": False, "packed": True},
        # one sequence on the 256-expert top-8 layer with its shared expert
        {"name": "few_1_e256_shared", "op": "few", "T": 1, "valid": 1, "H": 7168, "E": 256,
         "k": 8, "I": 256, "shared": 1, "fp8": False, "packed": True},
        # four sequences in a gathered batch with padding rows, fp8 weights
        {"name": "few_6_e256_fp8", "op": "few", "T": 6, "valid": 4, "H": 7168, "E": 256, "k": 8,
         "I": 256, "shared": 1, "fp8": True, "packed": True},
        # the largest few-token batch, weights as a checkpoint holds them
        {"name": "few_16_e256_rows", "op": "few", "T": 16, "valid": 16, "H": 7168, "E": 256,
         "k": 8, "I": 256, "shared": 1, "fp8": False, "packed": False},
        # a dense layer's gate/up projection for one decoded token
        {"name": "gemm_1", "op": "gemm", "M": 1, "N": 4096, "K": 7168, "f32": False},
        # a small ragged batch on odd sizes: K ends inside a scale block, N inside a tile
        {"name": "gemm_37_ragged", "op": "gemm", "M": 37, "N": 1001, "K": 5136, "f32": True},
        # a dense layer's down projection over a short prompt
        {"name": "gemm_1000", "op": "gemm", "M": 1000, "N": 7168, "K": 2048, "f32": False},
        # a prefill micro-batch through a dense gate/up projection
        {"name": "gemm_8192", "op": "gemm", "M": 8192, "N": 4096, "K": 7168, "f32": False},
        # the token rows of a small decode batch, ahead of an fp8 product
        {"name": "quant_16", "op": "quant", "M": 16, "K": 7168, "f32": False},
        # the token rows of a prefill micro-batch
        {"name": "quant_8192", "op": "quant", "M": 8192, "K": 7168, "f32": False},
        # between the two products of a dense layer: odd rows, a tail block, fp32 gate/up
        {"name": "silu_33_ragged", "op": "silu", "M": 33, "I": 1040, "f32": True},
        # the same for a prefill micro-batch
        {"name": "silu_8192", "op": "silu", "M": 8192, "I": 2048, "f32": False},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, round(lo * (hi / lo) ** rng.random())))


def draw(rng):
    op = rng.choice(("few", "few", "gemm", "gemm", "quant", "silu"))
    if op == "few":
        top = work(listed()[3])["bytes"]
        while True:
            fp8 = rng.random() < 0.5
            step = 128 if fp8 else 32
            T = _log(rng, 1, 16)
            E = _log(rng, 4, 256)
            c = {"op": "few", "T": T, "valid": rng.randint((T + 1) // 2, T),
                 "H": 128 * _log(rng, 2, 56), "E": E, "k": rng.randint(1, min(8, E)),
                 "I": step * _log(rng, 1, 640 // step), "shared": rng.randint(0, 1), "fp8": fp8,
                 "packed": rng.random() < 0.5}
            if work(c)["bytes"] <= top:
                return c
    if op == "gemm":
        return {"op": "gemm", "M": _log(rng, 1, 8192), "N": _log(rng, 16, 4096),
                "K": 16 * _log(rng, 8, 448), "f32": rng.random() < 0.3}
    if op == "quant":
        return {"op": "quant", "M": _log(rng, 1, 8192), "K": 16 * _log(rng, 1, 448),
                "f32": rng.random() < 0.3}
    return {"op": "silu", "M": _log(rng, 1, 8192), "I": 16 * _log(rng, 1, 128),
            "f32": rng.random() < 0.3}


def _blocks(n):
    return -(-n // BLOCK)


def _codes(shape, gen, spread):
    """e4m3fn codes of block-scaled normal values: a block's largest one lies at 448."""
    v = torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16)
    return v.mul_(E4M3_MAX / spread).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)


def _scales(shape, gen, std, spread):
    s = torch.rand(shape, generator=gen, device="cuda")
    return (0.9 + 0.2 * s) * (std * spread / E4M3_MAX)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    normal = lambda *shape: torch.randn(shape, generator=gen, device="cuda")  # noqa: E731
    c, s = case, {"case": case}
    if c["op"] == "few":
        T, H, E, I, ne = c["T"], c["H"], c["E"], c["I"], c["E"] + c["shared"]
        s["x"] = normal(T, H).bfloat16()
        rows = torch.randperm(T, generator=gen, device="cuda")[: c["valid"]]
        s["valid"] = torch.zeros(T, dtype=torch.uint8, device="cuda")
        s["valid"][rows] = 1
        s["router"] = (0.02 * normal(E, H)).bfloat16()
        if c["fp8"]:
            # the largest of a block's 16384 normal values lies near 4.1 deviations
            s["w13"] = _codes((ne, 2 * I, H), gen, 4.1)
            s["w2"] = _codes((ne, H, I), gen, 4.1)
            s["s13"] = _scales((ne, 2 * I // BLOCK, H // BLOCK), gen, 0.02, 4.1)
            s["s2"] = _scales((ne, H // BLOCK, I // BLOCK), gen, 0.02, 4.1)
        else:
            w = lambda *shape: torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16).mul_(0.02)  # noqa: E731
            s["w13"], s["w2"], s["s13"], s["s2"] = w(ne, 2 * I, H), w(ne, H, I), None, None
        if own:
            import expert_layer_moe_amd as moe
            s["layer"] = moe.DeviceLayer(s["router"], s["w13"], s["w2"], c["k"], c["shared"],
                                         s["s13"], s["s2"], packed=c["packed"])
    elif c["op"] == "gemm":
        M, N, K = c["M"], c["N"], c["K"]
        # the largest of a token row's 128 normal values lies near 2.6 deviations
        s["a"], s["sa"] = _codes((M, K), gen, 2.6), _scales((M, _blocks(K)), gen, 1.0, 2.6)
        s["b"], s["sb"] = _codes((N, K), gen, 4.1), _scales((_blocks(N), _blocks(K)), gen, 0.02, 4.1)
    elif c["op"] == "quant":
        s["x"] = normal(c["M"], c["K"]).to(torch.float32 if c["f32"] else torch.bfloat16)
    else:
        s["gu"] = normal(c["M"], 2 * c["I"]).mul_(1.7).to(torch.float32 if c["f32"] else torch.bfloat16)
    return s


# ---- the plain forms ---------------------------------------------------------
def _wide(scale, rows, cols):
    """Block scales [.., ceil(rows / 128), ceil(cols / 128)] -> [.., rows, cols]."""
    return scale.repeat_interleave(BLOCK, -2)[..., :rows, :].repeat_interleave(BLOCK, -1)[..., :cols]


def _weights(w, scale, pick):
    got = w[pick]
    if scale is None:
        return got.float()
    got = got.view(torch.float8_e4m3fn).float()
    return got * _wide(scale[pick], got.shape[-2], got.shape[-1])


def _few(s):
    c = s["case"]
    valid = s["valid"].bool()[:, None]
    x = torch.where(valid, s["x"].float(), 0.0)
    # the choice of experts turns on small differences of long sums: 64 bits
    logits = x.double() @ s["router"].double().T
    got = torch.sort(logits, dim=1, descending=True, stable=True)
    ids, top = got.indices[:, : c["k"]], got.values[:, : c["k"]]
    w = torch.exp(top - top[:, :1])
    w = (w / w.sum(1, keepdim=True)).float()
    if c["shared"]:
        ids = torch.cat([ids, torch.full_like(ids[:, :1], c["E"])], 1)
        w = torch.cat([w, torch.ones_like(w[:, :1])], 1)
    gu = torch.matmul(_weights(s["w13"], s["s13"], ids), x[:, None, :, None])[..., 0]
    g, u = gu[..., : c["I"]], gu[..., c["I"]:]
    h = g / (1 + torch.exp(-g)) * u
    y = torch.matmul(_weights(s["w2"], s["s2"], ids), h[..., None])[..., 0]
    return torch.where(valid, (w[..., None] * y).sum(1), 0.0).bfloat16()


def _gemm(s):
    c = s["case"]
    a = s["a"].view(torch.float8_e4m3fn).float()
    a = a * s["sa"].repeat_interleave(BLOCK, 1)[:, : c["K"]]
    b = s["b"].view(torch.float8_e4m3fn).float() * _wide(s["sb"], c["N"], c["K"])
    return (a @ b.T).to(torch.float32 if c["f32"] else torch.bfloat16)


def _quant(v):
    M, K = v.shape
    nb = _blocks(K)
    wide = torch.nn.functional.pad(v, (0, nb * BLOCK - K)).view(M, nb, BLOCK)
    scale = wide.abs().amax(2).clamp(min=TINY)
    # by a tensor: division by a plain number multiplies by its rounded reciprocal
    scale = scale / torch.full_like(scale, E4M3_MAX)
    codes = (wide / scale[..., None]).view(M, nb * BLOCK)[:, :K].contiguous()
    return codes.to(torch.float8_e4m3fn), scale


def _silu(s):
    I = s["case"]["I"]
    g, u = s["gu"][:, :I].float(), s["gu"][:, I:].float()
    return _quant(g / (1 + torch.exp(-g)) * u)


def run(s):
    op = s["case"]["op"]
    if own:
        import expert_layer_moe_amd as moe
        if op == "few":
            return s["layer"].forward_few(s["x"], s["valid"])
        if op == "gemm":
            return moe.moe_gemm_fp8(s["a"], s["sa"], s["b"], s["sb"],
                                    out_dtype=torch.float32 if s["case"]["f32"] else torch.bfloat16)
        if op == "quant":
            codes, scale = moe.moe_quant_fp8(s["x"])
        else:
            codes, scale = moe.moe_silu_mul_quant_fp8(s["gu"])
        return codes.view(torch.float8_e4m3fn), scale
    if op == "few":
        return _few(s)
    if op == "gemm":
        return _gemm(s)
    return _quant(s["x"].float()) if op == "quant" else _silu(s)


def _experts_read(c):
    """Expected number of distinct routed experts of the valid rows."""
    return c["E"] * (1 - (1 - c["k"] / c["E"]) ** c["valid"]) + c["shared"]


def work(case):
    c = case
    if c["op"] == "few":
        each = 3 * c["I"] * c["H"]
        weights = _experts_read(c) * (each * (1 + 4 / BLOCK ** 2) if c["fp8"] else each * 2)
        rows = c["valid"] * (c["k"] + c["shared"])
        return {"bytes": weights + 2 * c["E"] * c["H"] + 2 * (c["valid"] + c["T"]) * c["H"] + c["T"],
                "flops": 2.0 * rows * each + 2.0 * c["valid"] * c["E"] * c["H"]}
    if c["op"] == "gemm":
        M, N, K = c["M"], c["N"], c["K"]
        return {"bytes": (M + N) * K + 4.0 * (M + _blocks(N)) * _blocks(K) + M * N * (4 if c["f32"] else 2),
                "flops": 2.0 * M * N * K}
    size = 4 if c["f32"] else 2
    if c["op"] == "quant":
        n = c["M"] * c["K"]
        return {"bytes": n * (size + 1.0) + 4.0 * c["M"] * _blocks(c["K"]), "flops": 3.0 * n}
    n = c["M"] * c["I"]
    return {"bytes": n * (2.0 * size + 1) + 4.0 * c["M"] * _blocks(c["I"]), "flops": 8.0 * n}


# ---- the definitions in 64 bits ------------------------------------------------
def _decode64(codes, scale=None):
    """e4m3fn codes as the numbers their bits stand for, times their scales."""
    bits = torch.arange(256, device=codes.device)
    sign = 1.0 - 2.0 * (bits >> 7).double()
    e, m = (bits >> 3) & 15, (bits & 7).double()
    table = sign * torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * torch.exp2((e - 7).double()))
    v = table[codes.long()]
    if scale is not None:
        r, k = torch.arange(v.shape[0], device=v.device), torch.arange(v.shape[1], device=v.device)
        v = v * scale.double()[r // BLOCK][:, k // BLOCK]
    return v


def _round_e4m3(v):
    """Nearest e4m3fn value, ties to the even code, as a 64-bit number."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _quant64(v):
    M, K = v.shape
    scale = torch.empty(M, _blocks(K), dtype=torch.float64, device=v.device)
    codes = torch.empty_like(v)
    for b in range(_blocks(K)):
        part = v[:, b * BLOCK:(b + 1) * BLOCK]
        scale[:, b] = part.abs().max(1).values.clamp(min=TINY) / E4M3_MAX
        # the codes are those of the scale as it is stored, in 32 bits
        stored = scale[:, b:b + 1].float().double()
        codes[:, b * BLOCK:(b + 1) * BLOCK] = _round_e4m3(part / stored)
    return codes, scale


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "gemm":
        K = c["K"]
        a = _decode64(s["a"]) * s["sa"].double()[:, torch.arange(K, device="cuda") // BLOCK]
        return a @ _decode64(s["b"], s["sb"]).T
    if c["op"] == "quant":
        return _quant64(s["x"].double())
    if c["op"] == "silu":
        gu = s["gu"].double()
        g, u = gu[:, : c["I"]], gu[:, c["I"]:]
        return _quant64(g * torch.sigmoid(g) * u)
    out = torch.zeros(c["T"], c["H"], dtype=torch.float64, device="cuda")
    for t in range(c["T"]):
        if not int(s["valid"][t]):
            continue
        x = s["x"][t].double()
        logits = (s["router"].double() @ x).tolist()
        chosen = sorted(range(c["E"]), key=lambda e: (-logits[e], e))[: c["k"]]
        w = torch.softmax(torch.tensor([logits[e] for e in chosen], dtype=torch.float64), 0).tolist()
        for e, we in list(zip(chosen, w)) + [(c["E"], 1.0)] * c["shared"]:
            w13 = _decode64(s["w13"][e], s["s13"][e]) if c["fp8"] else s["w13"][e].double()
            w2 = _decode64(s["w2"][e], s["s2"][e]) if c["fp8"] else s["w2"][e].double()
            g, u = (w13 @ x).split(c["I"])
            out[t] += we * (w2 @ (torch.sigmoid(g) * g * u))
    return out
