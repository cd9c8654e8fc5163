"""The operators around the 4-bit linear layers as measured cases: what each is
given, its plain form in elementary torch operations, and its definition in
64 bits.

Four operators of one transformer block whose linear layers hold MXFP4 weights:

* ``quant``: activations to MXFP4 codes and block scales, with the LoRA-down
  product, in one pass over x (`quantize_mxfp4_act`);
* ``few``: the MXFP4 linear layer for few tokens (`gemm_mxfp4_few`);
* ``rotary``: rotary positions over several axes (`rotary_axes`);
* ``attend``: attention of queries to keys and values of another length, held
  by shared heads, with a length per sequence (`cross_attention`).

`run` computes the plain form where `own` is false and calls the package where
it is true. Sizes are those of the synthetic workloads (hidden 3072 in 24
heads of 128, MLP 12288, 4096 and 4352 tokens) and generic odd ones.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
# magnitudes of the E2M1 codes 0..7; bit 3 is the sign
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # the input of a QKV projection over a 64 x 64 latent image
        {"name": "quant_image", "op": "quant", "M": 4096, "K": 3072, "R": 32, "type": "bf16"},
        # the wide input of an MLP-down projection, odd token count, largest rank
        {"name": "quant_mlp_down_odd", "op": "quant", "M": 1001, "K": 12288, "R": 128, "type": "f16"},
        # the conditioning vectors of a batch of four: a call of a few microseconds
        {"name": "quant_vectors", "op": "quant", "M": 4, "K": 3072, "R": 32, "type": "bf16"},
        # one conditioning vector through a 3072 -> 12288 layer
        {"name": "few_one_vector", "op": "few", "M": 1, "N": 12288, "K": 3072, "R": 32, "type": "bf16"},
        # sixteen vectors through an MLP-down layer at the largest rank in use
        {"name": "few_mlp_down", "op": "few", "M": 16, "N": 3072, "K": 12288, "R": 128, "type": "bf16"},
        # an odd number of short-prompt tokens, odd columns, a K that ends inside a 128-wide step
        {"name": "few_odd", "op": "few", "M": 61, "N": 1001, "K": 3104, "R": 17, "type": "f16"},
        # q and k of a joint QKV output, rotated over (time, height, width)
        {"name": "rotary_image", "op": "rotary", "B": 1, "L": 4096, "H": 48, "HALL": 72, "D": 128,
         "s0": 8, "s1": 28, "s2": 28, "interleaved": True, "inverse": False, "type": "bf16"},
        # one new token for each of eight sequences, halves layout, a head with a part left unrotated
        {"name": "rotary_token", "op": "rotary", "B": 8, "L": 1, "H": 9, "HALL": 9, "D": 72,
         "s0": 4, "s1": 11, "s2": 17, "interleaved": False, "inverse": True, "type": "f16"},
        # image queries to a text encoder's 512 states
        {"name": "attend_text", "op": "attend", "B": 1, "LQ": 4096, "LK": 512, "HQ": 24, "HKV": 24,
         "D": 128, "lens": "full", "type": "bf16"},
        # one new token of each of eight sequences over a long encoder output, shared heads, ragged lengths
        {"name": "attend_token", "op": "attend", "B": 8, "LQ": 1, "LK": 8191, "HQ": 24, "HKV": 8,
         "D": 128, "lens": "ragged", "type": "bf16"},
        # odd lengths, a head size between the powers of two, one sequence with no states at all
        {"name": "attend_odd", "op": "attend", "B": 3, "LQ": 1001, "LK": 333, "HQ": 16, "HKV": 16,
         "D": 72, "lens": "ragged", "type": "f16"},
        # the largest: image queries to image and text states together
        {"name": "attend_joint", "op": "attend", "B": 1, "LQ": 4352, "LK": 4608, "HQ": 24, "HKV": 24,
         "D": 128, "lens": "full", "type": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quant", "few", "rotary", "attend"])
    kind = rng.choice(["bf16", "f16"])
    if op == "quant":
        return {"op": op, "M": _log_int(rng, 1, 4352), "K": 32 * _log_int(rng, 2, 384),
                "R": rng.choice([0, 128, rng.randint(1, 32), rng.randint(33, 127)]), "type": kind}
    if op == "few":
        return {"op": op, "M": rng.choice([1, rng.randint(2, 16), rng.randint(17, 64)]), "N": _log_int(rng, 64, 12288),
                "K": 32 * _log_int(rng, 2, 384), "R": rng.choice([0, 128, rng.randint(1, 64)]), "type": kind}
    if op == "rotary":
        heads = rng.randint(1, 48)
        dim = 8 * rng.randint(4, 16)
        cut = sorted(rng.randint(0, dim // 2) for _ in range(3))
        return {"op": op, "B": rng.randint(1, 4), "L": _log_int(rng, 1, 4352), "H": heads, "HALL": heads + rng.randint(0, 24),
                "D": dim, "s0": cut[0], "s1": cut[1] - cut[0], "s2": cut[2] - cut[1],
                "interleaved": rng.random() < 0.5, "inverse": rng.random() < 0.5, "type": kind}
    group = rng.choice([1, 1, 2, 4, 8])
    kv = rng.randint(1, 24 // group)
    lk = _log_int(rng, 1, 8191)
    most = max(1, min(4352, 4352 * 4608 * 24 // (2 * lk * kv * group)))
    lq = rng.choice([1, _log_int(rng, 1, most), most - rng.randint(0, most // 2)])
    b = max(1, min(rng.randint(1, 8), 4352 * 4608 * 24 // (lk * lq * kv * group)))
    return {"op": op, "B": b, "LQ": lq, "LK": lk, "HQ": kv * group, "HKV": kv, "D": 8 * rng.randint(4, 16),
            "lens": rng.choice(["full", "ragged"]), "type": kind}


# ---------------------------------------------------------------- inputs


def _lens(case):
    """Keys in use of each sequence: all of them, or growing from none at all (the first) to all (the last)."""
    b, lk = case["B"], case["LK"]
    if case["lens"] == "full":
        return [lk] * b
    return [lk * i // (b - 1) for i in range(b)] if b > 1 else [lk - lk // 3]


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    half = TYPES[case["type"]]

    def normal(*shape, std=1.0, dtype=half):
        return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)

    s = dict(case)
    if case["op"] == "quant":
        M, K, R = case["M"], case["K"], case["R"]
        # channels of unequal size, one in a hundred an outlier, as activations have
        channel = torch.exp2(torch.rand((K,), generator=g, device=DEV) * 6 - 3)
        channel = torch.where(torch.rand((K,), generator=g, device=DEV) < 0.01, channel * 32, channel)
        s["x"] = (torch.randn((M, K), generator=g, device=DEV) * channel).to(half)
        s["lora_down"] = normal(R, K, std=0.02) if R else None
    elif case["op"] == "few":
        M, N, K, R = case["M"], case["N"], case["K"], case["R"]
        s["act"], s["ascales"] = _mxfp4(normal(M, K))
        s["wgt"], s["wscales"] = _mxfp4(normal(N, K, std=0.02))
        s["wcscale"] = torch.rand((N,), generator=g, device=DEV) + 0.5
        s["bias"] = torch.randn((N,), generator=g, device=DEV)
        s["lora_act_in"] = normal(M, R, std=0.1) if R else None
        s["lora_up"] = normal(R, N, std=0.1) if R else None
    elif case["op"] == "rotary":
        B, L, D = case["B"], case["L"], case["D"]
        joint = normal(B, L, case["HALL"], D)
        s["x"] = joint[:, :, :case["H"]]                  # the rotated heads of a joint projection
        side = max(1, math.isqrt(L))
        at = torch.arange(L, device=DEV)
        grid = torch.stack([at // (side * side), at // side % side, at % side], -1)
        shift = torch.randint(0, 64, (B, 1, 3), generator=g, device=DEV)
        s["positions"] = (grid + shift).to(torch.int32).contiguous()
        s["sections"] = (case["s0"], case["s1"], case["s2"])
        freqs = [10000.0 ** (-torch.arange(n, device=DEV, dtype=torch.float64) / max(1, n)) for n in s["sections"]]
        s["inv_freq"] = torch.cat(freqs).to(torch.float32)
    else:
        B, D = case["B"], case["D"]
        s["q"] = normal(B, case["LQ"], case["HQ"], D)
        s["k"] = normal(B, case["LK"], case["HKV"], D)
        s["v"] = normal(B, case["LK"], case["HKV"], D)
        s["kv_lens"] = None if case["lens"] == "full" else torch.tensor(_lens(case), dtype=torch.int32, device=DEV)
    return s


# ---------------------------------------------------------------- plain forms


def _mxfp4(x):
    """x [rows, K] -> MXFP4 codes uint8 [rows, K/2] (low nibble = even k) and UE8M0 bytes [K/32, rows].

    A block of 32 values has the scale 2^(floor(log2 of its largest magnitude) - 2); a code is the nearest E2M1
    value of x / scale, ties to the even code, at most 6. A block with a NaN or an infinity: byte 255, codes 0."""
    rows, K = x.shape
    v = x.float().reshape(rows, K // 32, 32)
    top = v.abs().amax(-1)
    fine = torch.isfinite(v).all(-1)
    byte = torch.clamp((torch.where(fine, top, 0.0).view(torch.int32) >> 23) - 2, min=0)
    a = v.abs() * ((254 - byte) << 23).view(torch.float32)[..., None]
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = torch.where(fine[..., None], code + 8 * torch.signbit(v), 0).reshape(rows, K).to(torch.uint8)
    byte = torch.where(fine, byte, 255).to(torch.uint8)
    return code[:, 0::2] | (code[:, 1::2] << 4), byte.t().contiguous()


def _values(codes, scales):
    """The float32 values that MXFP4 codes [rows, K/2] and scales [K/32, rows] stand for."""
    table = torch.tensor(E2M1 + tuple(-m for m in E2M1), device=codes.device)
    v = table[torch.stack([codes & 15, codes >> 4], -1).flatten(1).long()]
    scale = torch.exp2(scales.t().float() - 127.0)
    return (v.reshape(v.shape[0], -1, 32) * scale[..., None]).reshape(v.shape)


def _plain_quant(s):
    act, ascales = _mxfp4(s["x"])
    if s["lora_down"] is None:
        return act, ascales, None
    return act, ascales, (s["x"].float() @ s["lora_down"].float().t()).to(s["x"].dtype)


def _plain_few(s):
    y = (_values(s["act"], s["ascales"]) @ _values(s["wgt"], s["wscales"]).t()) * s["wcscale"] + s["bias"]
    if s["lora_up"] is not None:
        y = y + s["lora_act_in"].float() @ s["lora_up"].float()
    return y.to(TYPES[s["type"]])


def _plain_rotary(s):
    x, sections = s["x"].float(), s["sections"]
    pairs = sum(sections)
    axis = torch.repeat_interleave(torch.arange(len(sections), device=x.device), torch.tensor(sections, device=x.device), output_size=pairs)
    angle = (s["positions"].float()[..., axis] * s["inv_freq"])[:, :, None, :]
    cos, sin = torch.cos(angle), torch.sin(angle)
    if s["inverse"]:
        sin = -sin
    part, rest = x[..., :2 * pairs], x[..., 2 * pairs:]
    a, b = (part[..., 0::2], part[..., 1::2]) if s["interleaved"] else (part[..., :pairs], part[..., pairs:])
    u, w = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack([u, w], -1).flatten(-2) if s["interleaved"] else torch.cat([u, w], -1)
    return torch.cat([turned, rest], -1).to(s["x"].dtype)


def _plain_attend(s):
    q, k, v = (s[n].float().transpose(1, 2) for n in ("q", "k", "v"))
    B, HQ, LQ, D = q.shape
    HKV, LK = k.shape[1], k.shape[2]
    q = q.reshape(B, HKV, HQ // HKV * LQ, D)
    score = (q @ k.transpose(2, 3).contiguous()) * (D ** -0.5)
    if s["kv_lens"] is not None:
        live = torch.arange(LK, device=q.device) < s["kv_lens"][:, None]
        score = score.masked_fill(~live[:, None, None, :], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(torch.isfinite(top), top, 0.0)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    out = (p @ v.contiguous()) / torch.where(total > 0, total, 1.0)
    out = out.reshape(B, HQ, LQ, D).transpose(1, 2).contiguous().to(s["q"].dtype)
    return out, (top + torch.log(total)).reshape(B, HQ, LQ)


def run(state):
    s = state
    if not own:
        return {"quant": _plain_quant, "few": _plain_few, "rotary": _plain_rotary, "attend": _plain_attend}[s["op"]](s)
    import bit_quantized_gemm_amd as w4
    if s["op"] == "quant":
        return w4.quantize_mxfp4_act(s["x"], s["lora_down"])
    if s["op"] == "few":
        return w4.gemm_mxfp4_few(s["act"], s["ascales"], s["wgt"], s["wscales"], s["wcscale"], s["bias"],
                                 s["lora_act_in"], s["lora_up"], dtype=TYPES[s["type"]])
    if s["op"] == "rotary":
        return w4.rotary_axes(s["x"], s["positions"], s["inv_freq"], s["sections"],
                              interleaved=s["interleaved"], inverse=s["inverse"])
    return w4.cross_attention(s["q"], s["k"], s["v"], kv_lens=s["kv_lens"], return_lse=True)


# ---------------------------------------------------------------- what a pass cannot do without


def work(case):
    if case["op"] == "quant":
        M, K, R = case["M"], case["K"], case["R"]
        return {"bytes": 2 * M * K + 2 * R * K + M * K // 2 + M * K // 32 + 2 * M * R, "flops": 2 * M * K * R + M * K}
    if case["op"] == "few":
        M, N, K, R = case["M"], case["N"], case["K"], case["R"]
        return {"bytes": (M + N) * (K // 2 + K // 32) + 8 * N + 2 * R * (M + N) + 2 * M * N,
                "flops": 2 * M * N * (K + R)}
    if case["op"] == "rotary":
        n = case["B"] * case["L"] * case["H"] * case["D"]
        return {"bytes": 4 * n + 12 * case["B"] * case["L"], "flops": 3 * n}
    B, LQ, HQ, HKV, D = case["B"], case["LQ"], case["HQ"], case["HKV"], case["D"]
    keys = sum(_lens(case))
    return {"bytes": 4 * B * LQ * HQ * D + 4 * keys * HKV * D + 4 * B * LQ * HQ, "flops": 4 * LQ * HQ * D * keys}


# ---------------------------------------------------------------- the definitions in 64 bits


def _exact_values(codes, scales):
    c = torch.stack([codes & 15, codes >> 4], 2).reshape(codes.shape[0], -1).to(torch.int64)
    e, m = (c >> 1) & 3, c & 1
    mag = torch.where(e == 0, 0.5 * m.double(), (1 + 0.5 * m.double()) * 2.0 ** (e.double() - 1))
    two = 2.0 ** (scales.double() - 127.0)
    return torch.where(c >= 8, -mag, mag) * two.repeat_interleave(32, dim=0).t()


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quant":
        if not case["R"]:
            return None                                   # codes and scale bytes alone: whole numbers
        return None, None, torch.einsum("mk,rk->mr", s["x"].double(), s["lora_down"].double())
    if case["op"] == "few":
        y = torch.einsum("mk,nk->mn", _exact_values(s["act"], s["ascales"]), _exact_values(s["wgt"], s["wscales"]))
        y = y * s["wcscale"].double()[None, :] + s["bias"].double()[None, :]
        if case["R"]:
            y += torch.einsum("mr,rn->mn", s["lora_act_in"].double(), s["lora_up"].double())
        return y
    if case["op"] == "rotary":
        out = s["x"].double().clone()
        pairs, j = sum(s["sections"]), 0
        for a, n in enumerate(s["sections"]):
            for _ in range(n):
                turn = s["positions"][..., a].double() * s["inv_freq"][j].double() * (-1.0 if case["inverse"] else 1.0)
                i0, i1 = (2 * j, 2 * j + 1) if case["interleaved"] else (j, j + pairs)
                z = torch.complex(s["x"][..., i0].double(), s["x"][..., i1].double()) * torch.polar(torch.ones_like(turn), turn)[..., None]
                out[..., i0], out[..., i1] = z.real, z.imag
                j += 1
        return out
    B, LQ, HQ, D = s["q"].shape
    group = HQ // case["HKV"]
    out = torch.zeros((B, LQ, HQ, D), dtype=torch.float64, device=DEV)
    lse = torch.full((B, HQ, LQ), -math.inf, dtype=torch.float64, device=DEV)
    for b, n in enumerate(_lens(case)):
        for h in range(HQ if n else 0):
            q, k, v = s["q"][b, :, h].double(), s["k"][b, :n, h // group].double(), s["v"][b, :n, h // group].double()
            score = q @ k.t() / math.sqrt(D)
            lse[b, h] = torch.logsumexp(score, 1)
            out[b, :, h] = torch.exp(score - lse[b, h][:, None]) @ v
    return out, lse
