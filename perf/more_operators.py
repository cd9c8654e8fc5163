"""The operators that serve many requests at once on the 4-bit layers, as
measured cases: what each is given, its plain form in elementary torch
operations, and its definition in 64 bits.

* ``norm``: the norms after and before a block with its gate and residual in
  between (`block_norm`);
* ``adapt``: low-rank adapters of many requests beside a shared projection
  (`lora_adapters`);
* ``prompt``: causal attention over packed prompts of different lengths, heads
  shared in groups (`packed_attention`);
* ``append``: keys and values of new tokens into a paged cache
  (`cache_append`);
* ``token``: attention of the newest tokens over that cache
  (`paged_attention`).

`run` computes the plain form where `own` is false and calls the package where
it is true. Sizes are those of the synthetic workloads (hidden 3072 in 24
heads of 128, MLP 12288, 4096 and 4352 tokens) and generic odd ones.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-6


def listed():
    return [
        # the step from one block half to the next over a 64 x 64 latent image: residual with the
        # gate of one half, layer norm with the scale and shift of the next
        {"name": "norm_image", "op": "norm", "B": 1, "L": 4096, "C": 3072, "kind": "layer", "y": True, "gate": "batch",
         "post": False, "affine": "none", "mod": "batch", "type": "bf16"},
        # one new token of each of eight requests, norms on both sides of the block: a call of a few microseconds
        {"name": "norm_tokens", "op": "norm", "B": 8, "L": 1, "C": 3072, "kind": "rms", "y": True, "gate": "none",
         "post": True, "affine": "weight", "mod": "none", "type": "bf16"},
        # odd token count and odd width, a gate, scale and shift for every token (frames at different noise levels)
        {"name": "norm_odd", "op": "norm", "B": 3, "L": 333, "C": 1001, "kind": "layer", "y": True, "gate": "token",
         "post": False, "affine": "both", "mod": "token", "type": "f16"},
        # one new token of each of 64 requests, 16 adapters among them, through a QKV projection
        {"name": "adapt_tokens", "op": "adapt", "S": 64, "M": 64, "A": 16, "K": 3072, "N": 9216, "R": 32,
         "ranks": "full", "type": "bf16"},
        # the prompts of 12 requests through an MLP-up layer, eight adapters of different ranks and requests without one
        {"name": "adapt_prompts", "op": "adapt", "S": 12, "M": 4352, "A": 8, "K": 3072, "N": 12288, "R": 64,
         "ranks": "mixed", "type": "bf16"},
        # odd rows, columns and rank, a K that ends inside a tile
        {"name": "adapt_odd", "op": "adapt", "S": 7, "M": 333, "A": 5, "K": 1000, "N": 1001, "R": 17,
         "ranks": "full", "type": "f16"},
        # prompts of a long request and of shorter ones, one of them empty, in one batch padded at its end
        {"name": "prompt_long", "op": "prompt", "S": 8, "T": 8192, "pad": 100, "HQ": 24, "HKV": 8, "D": 128,
         "causal": True, "type": "bf16"},
        # short prompts of a head size between the powers of two
        {"name": "prompt_short", "op": "prompt", "S": 5, "T": 1001, "pad": 0, "HQ": 16, "HKV": 16, "D": 72,
         "causal": True, "type": "f16"},
        # the keys and values of packed prompts into pages
        {"name": "append_prompts", "op": "append", "T": 4352, "HKV": 8, "D": 128, "page": 64, "type": "bf16"},
        # those of one new token of each of eight requests
        {"name": "append_tokens", "op": "append", "T": 8, "HKV": 8, "D": 128, "page": 16, "type": "f16"},
        # one new token of each of eight requests over caches of different lengths
        {"name": "token_long", "op": "token", "B": 8, "Q": 1, "LK": 8191, "HQ": 24, "HKV": 8, "D": 128, "page": 64,
         "type": "bf16"},
        # three tokens at a time (a draft being checked), small pages, one request without any
        {"name": "token_draft", "op": "token", "B": 3, "Q": 3, "LK": 1001, "HQ": 16, "HKV": 4, "D": 72, "page": 16,
         "type": "f16"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "adapt", "prompt", "append", "token"])
    half = rng.choice(["bf16", "f16"])
    if op == "norm":
        C = rng.choice([8 * _log_int(rng, 8, 1536), _log_int(rng, 64, 12288)])
        B = rng.choice([1, rng.randint(1, 8)])
        y = rng.random() < 0.8
        return {"op": op, "B": B, "L": _log_int(rng, 1, max(1, min(4352, 4096 * 3072 // (B * C)))), "C": C,
                "kind": rng.choice(["layer", "rms"]), "y": y, "gate": rng.choice(["none", "batch", "token"]) if y else "none",
                "post": y and rng.random() < 0.5, "affine": rng.choice(["none", "weight", "both"]),
                "mod": rng.choice(["none", "batch", "token"]), "type": half}
    if op == "adapt":
        M = _log_int(rng, 1, 4352)
        return {"op": op, "S": rng.randint(1, min(M, 64)), "M": M, "A": rng.randint(1, 16), "K": 8 * _log_int(rng, 8, 384),
                "N": _log_int(rng, 64, 12288), "R": rng.choice([16, 32, 64, rng.randint(1, 64)]),
                "ranks": rng.choice(["full", "mixed"]), "type": half}
    kv = rng.choice([1, 2, 4, 8, rng.randint(1, 8)])
    group = rng.choice([1, 2, 3, 4, 8])
    D = rng.choice([64, 128, 8 * rng.randint(4, 16)])
    if op == "prompt":
        causal = rng.random() < 0.75
        T = _log_int(rng, 1, 8192)
        if kv * group * T * T * D > 8192 * 1480 * 24 * 128:          # (the longest listed case, were all of it one prompt)
            T = max(1, math.isqrt(8192 * 1480 * 24 * 128 // (kv * group * D)))
        return {"op": op, "S": rng.randint(1, 16), "T": T, "pad": rng.choice([0, rng.randint(1, 64)]), "HQ": kv * group,
                "HKV": kv, "D": D, "causal": causal, "type": half}
    page = rng.choice([16, 32, 64, 128, 48])
    if op == "append":
        return {"op": op, "T": _log_int(rng, 1, 4352), "HKV": kv, "D": D, "page": page, "type": half}
    return {"op": op, "B": rng.randint(1, 8), "Q": rng.choice([1, 1, rng.randint(2, 8)]), "LK": _log_int(rng, 1, 8191),
            "HQ": kv * group, "HKV": kv, "D": D, "page": page, "type": half}


# ---------------------------------------------------------------- inputs


def _lengths(total, count):
    """`count` lengths that add up to `total`: one over half of it, the others shorter and shorter, the third of four
    or more none at all."""
    lens, left = [], total
    for i in range(count):
        n = left if i == count - 1 else min(left, left * 17 // 32 + 1)
        if i == 2 and count > 3:
            n = 0
        lens.append(n)
        left -= n
    return lens


def _requests(case):
    """Of `adapt`: (first row, rows, adapter) of each request; adapter -1: none (every fifth)."""
    lens = [1] * case["S"] if case["S"] == case["M"] else _lengths(case["M"], case["S"])
    at, reqs = 0, []
    for i, n in enumerate(lens):
        reqs.append((at, n, -1 if i % 5 == 4 else (7 * i) % case["A"]))
        at += n
    return reqs


def _ranks(case):
    """Of `adapt`: each adapter's rank."""
    R = case["R"]
    return [R if case["ranks"] == "full" else max(1, R >> (a % 3)) for a in range(case["A"])]


def _cache_lens(case):
    """Of `token`: the keys of each request, the new tokens' own among them, the last of three or more none at all."""
    B, LK = case["B"], case["LK"]
    lens = [max(min(LK, case["Q"]), LK * (B - b) // B) for b in range(B)]
    if B > 2:
        lens[-1] = 0
    return lens


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    half = TYPES[case["type"]]

    def normal(*shape, std=1.0, mean=0.0):
        return (torch.randn(shape, generator=g, device=DEV) * std + mean).to(half)

    s = dict(case)
    if case["op"] == "norm":
        B, L, C = case["B"], case["L"], case["C"]
        # a residual stream: channels of unequal size, one in a hundred an outlier
        channel = torch.exp2(torch.rand((C,), generator=g, device=DEV) * 4 - 2)
        channel = torch.where(torch.rand((C,), generator=g, device=DEV) < 0.01, channel * 16, channel)
        s["x"] = (torch.randn((B, L, C), generator=g, device=DEV) * channel + 0.25).to(half)
        s["y"] = normal(B, L, C) if case["y"] else None
        # gate, scale and shift as slices of one modulation tensor, for every request or every token
        parts = sum(case[k] != "none" for k in ("gate", "mod", "mod"))
        rows = L if "token" in (case["gate"], case["mod"]) else 1
        joint = normal(B, rows, max(1, parts) * C, std=0.5)
        pieces = [joint[..., i * C:(i + 1) * C] for i in range(parts)]
        wide = [p if kind == "token" else p[:, :1] for p, kind in
                zip(pieces, [case[k] for k in ("gate", "mod", "mod") if case[k] != "none"])]
        s["gate"] = wide.pop(0) if case["gate"] != "none" else None
        s["scale"], s["shift"] = wide if case["mod"] != "none" else (None, None)
        s["weight"] = normal(C, std=0.2, mean=1.0) if case["affine"] != "none" else None
        s["bias"] = normal(C, std=0.2) if case["affine"] == "both" else None
        s["post_weight"] = normal(C, std=0.2, mean=1.0) if case["post"] else None
    elif case["op"] == "adapt":
        M, A, K, N, R = (case[k] for k in ("M", "A", "K", "N", "R"))
        s["x"], s["y"] = normal(M, K), normal(M, N)
        s["down"], s["up"] = normal(A, R, K, std=K ** -0.5), normal(A, R, N, std=0.5)
        s["requests"], s["rank_list"] = _requests(case), _ranks(case)
        s["adapter"] = torch.tensor([a for _, n, a in s["requests"] for _ in range(n)], dtype=torch.int32, device=DEV)
        s["ranks"] = None if case["ranks"] == "full" else torch.tensor(s["rank_list"], dtype=torch.int32, device=DEV)
        s["scaling"] = torch.rand((A,), generator=g, device=DEV) + 0.5
    elif case["op"] == "prompt":
        S, D = case["S"], case["D"]
        rows = case["T"] + case["pad"]
        joint = normal(rows, case["HQ"] + 2 * case["HKV"], D)     # a joint QKV projection's output
        s["q"], s["k"], s["v"] = joint.split([case["HQ"], case["HKV"], case["HKV"]], 1)
        s["lens"] = _lengths(case["T"], S)
        s["starts"] = torch.tensor([sum(s["lens"][:i]) for i in range(S + 1)], dtype=torch.int32, device=DEV)
        s["out"] = torch.zeros((rows, case["HQ"], D), dtype=half, device=DEV)    # a program's buffer: padding stays zero
    elif case["op"] == "append":
        T, H, D, page = case["T"], case["HKV"], case["D"], case["page"]
        pages = -(-T // page) + 2
        joint = normal(T, 2 * H, D)
        s["k"], s["v"] = joint[:, :H], joint[:, H:]
        s["k_cache"], s["v_cache"] = normal(pages, page, H, D), normal(pages, page, H, D)
        # tokens in order in pages that lie anywhere; every ninth is padding, which has no slot
        order = torch.randperm(pages, generator=g, device=DEV)
        at = torch.arange(T, device=DEV)
        s["slots"] = torch.where(at % 9 == 8, -1, order[at // page] * page + at % page)
    else:
        B, H, D, page = case["B"], case["HKV"], case["D"], case["page"]
        lens = _cache_lens(case)
        most = max(1, -(-max(lens) // page))
        pages = sum(-(-n // page) for n in lens) + 3
        s["q"] = normal(B, case["Q"], case["HQ"], D)
        s["k_cache"], s["v_cache"] = normal(pages, page, H, D), normal(pages, page, H, D)
        order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
        table, at = torch.full((B, most), -1, dtype=torch.int32, device=DEV), 0
        for b, n in enumerate(lens):
            used = -(-n // page)
            table[b, :used] = order[at:at + used]
            at += used
        s["table"], s["lens"] = table, torch.tensor(lens, dtype=torch.int32, device=DEV)
    return s


# ---------------------------------------------------------------- plain forms


def _plain_norm(v, kind):
    if kind == "layer":
        v = v - v.mean(-1, keepdim=True)
    return v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS)


def _plain(s):
    op, half = s["op"], TYPES[s["type"]]
    if op == "norm":
        r = s["x"].float()
        if s["y"] is not None:
            y = s["y"].float()
            if s["post"]:
                y = _plain_norm(y, s["kind"]) * s["post_weight"].float()
            if s["gate"] is not None:
                y = y * s["gate"].float()
            r = r + y
        h = _plain_norm(r, s["kind"])
        if s["weight"] is not None:
            h = h * s["weight"].float()
        if s["bias"] is not None:
            h = h + s["bias"].float()
        if s["scale"] is not None:
            h = h * (1 + s["scale"].float()) + s["shift"].float()
        return (h.to(half), r.to(half)) if s["y"] is not None else h.to(half)
    if op == "adapt":
        rows = {}                                        # the rows of each adapter
        for at, n, a in s["requests"]:
            if a >= 0 and n:
                rows.setdefault(a, []).append(torch.arange(at, at + n, device=DEV))
        out = s["y"].float()
        for a, parts in rows.items():
            at, R = torch.cat(parts), s["rank_list"][a]
            low = s["x"][at].float() @ s["down"][a, :R].float().t()
            out[at] += (low @ s["up"][a, :R].float()) * s["scaling"][a]
        return out.to(half)
    if op == "prompt":
        out, at = torch.zeros(s["q"].shape, device=DEV), 0
        group = s["HQ"] // s["HKV"]
        for n in s["lens"]:
            if n:
                q = s["q"][at:at + n].float().transpose(0, 1).unflatten(0, (s["HKV"], group))
                k = s["k"][at:at + n].float().permute(1, 2, 0).contiguous()[:, None]
                v = s["v"][at:at + n].float().transpose(0, 1).contiguous()[:, None]
                score = torch.matmul(q, k) * s["D"] ** -0.5
                if s["causal"]:
                    i = torch.arange(n, device=DEV)
                    score = torch.where(i[None, :] <= i[:, None], score, -math.inf)
                p = torch.exp(score - score.amax(-1, keepdim=True))
                o = torch.matmul(p, v) / p.sum(-1, keepdim=True)
                out[at:at + n] = o.flatten(0, 1).transpose(0, 1)
            at += n
        return out.to(half)
    if op == "append":
        # (padding goes to one row past the end)
        H, D = s["HKV"], s["D"]
        for cache, new in ((s["k_cache"], s["k"]), (s["v_cache"], s["v"])):
            flat = torch.cat([cache.view(-1, H, D), cache.new_zeros(1, H, D)])
            flat[torch.where(s["slots"] < 0, flat.shape[0] - 1, s["slots"])] = new
            cache.copy_(flat[:-1].view(cache.shape))
        return s["k_cache"], s["v_cache"]
    B, Q, H, D = s["B"], s["Q"], s["HKV"], s["D"]
    group = s["HQ"] // H
    table = s["table"].long().clamp(min=0)
    k, v = (c[table].flatten(1, 2).float() for c in (s["k_cache"], s["v_cache"]))     # [B, keys, H, D]
    keys = torch.arange(k.shape[1], device=DEV)
    last = s["lens"].long()[:, None] - Q + torch.arange(Q, device=DEV)                # [B, Q]
    live = keys <= last[..., None]                                                   # [B, Q, keys]
    q = s["q"].float().transpose(1, 2).unflatten(1, (H, group)).flatten(2, 3)          # [B, H, group * Q, D]
    score = torch.matmul(q, k.permute(0, 2, 3, 1).contiguous()) * D ** -0.5
    live = live[:, None].expand(B, group, Q, -1).flatten(1, 2)[:, None]
    score = torch.where(live, score, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v.transpose(1, 2).contiguous()) / torch.where(total == 0, 1.0, total)
    lse = (top + torch.log(total)).view(B, H * group, Q)
    return o.unflatten(2, (group, Q)).flatten(1, 2).transpose(1, 2).to(half), lse


def run(state):
    s = state
    if not own:
        return _plain(s)
    import bit_quantized_gemm_amd as w4
    if s["op"] == "norm":
        h, r = w4.block_norm(s["x"], s["y"], gate=s["gate"], post_norm=s["post"], post_weight=s["post_weight"],
                             kind=s["kind"], weight=s["weight"], bias=s["bias"], scale=s["scale"], shift=s["shift"],
                             eps=EPS)
        return (h, r) if s["y"] is not None else h
    if s["op"] == "adapt":
        return w4.lora_adapters(s["y"], s["x"], s["down"], s["up"], s["adapter"], scaling=s["scaling"], ranks=s["ranks"])
    if s["op"] == "prompt":
        return w4.packed_attention(s["q"], s["k"], s["v"], s["starts"], causal=s["causal"], out=s["out"])
    if s["op"] == "append":
        w4.cache_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["slots"])
        return s["k_cache"], s["v_cache"]
    return w4.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], return_lse=True)


# ---------------------------------------------------------------- work


def work(case):
    if case["op"] == "norm":
        n, C = case["B"] * case["L"], case["C"]
        rows = {"none": 0, "batch": case["B"], "token": n}
        vectors = rows[case["gate"]] + 2 * rows[case["mod"]] + {"none": 0, "weight": 1, "both": 2}[case["affine"]] + case["post"]
        return {"bytes": 2 * C * (n * (4 if case["y"] else 2) + vectors), "flops": (16 if case["y"] else 8) * n * C}
    if case["op"] == "adapt":
        M, K, N, ranks = case["M"], case["K"], case["N"], _ranks(case)
        reqs = [(n, a) for _, n, a in _requests(case) if n and a >= 0]
        weights = sum(ranks[a] for a in {a for _, a in reqs})
        return {"bytes": 2 * (sum(n for n, _ in reqs) * K + weights * (K + N) + 2 * M * N) + 4 * M,
                "flops": 2 * sum(n * ranks[a] for n, a in reqs) * (K + N)}
    if case["op"] == "prompt":
        scores = sum(n * (n + 1) // 2 if case["causal"] else n * n for n in _lengths(case["T"], case["S"]))
        return {"bytes": 4 * case["T"] * (case["HQ"] + case["HKV"]) * case["D"], "flops": 4 * scores * case["HQ"] * case["D"]}
    if case["op"] == "append":
        live = case["T"] - case["T"] // 9
        return {"bytes": 8 * live * case["HKV"] * case["D"] + 8 * case["T"], "flops": 0}
    keys, Q, HQ, HKV, D = sum(_cache_lens(case)), case["Q"], case["HQ"], case["HKV"], case["D"]
    return {"bytes": 4 * keys * HKV * D + case["B"] * Q * HQ * (4 * D + 4), "flops": 4 * keys * Q * HQ * D}


# ---------------------------------------------------------------- the definitions in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        def normed(v):
            mean = v.sum(-1, keepdim=True) / v.shape[-1] if case["kind"] == "layer" else 0.0
            return (v - mean) / torch.sqrt(((v - mean) ** 2).sum(-1, keepdim=True) / v.shape[-1] + EPS)
        r = s["x"].double()
        if case["y"]:
            y = s["y"].double()
            if case["post"]:
                y = normed(y) * s["post_weight"].double()
            r = torch.addcmul(r, y, s["gate"].double().expand_as(r)) if s["gate"] is not None else r + y
        h = normed(r)
        h = h * (s["weight"].double() if s["weight"] is not None else 1.0)
        h = h + (s["bias"].double() if s["bias"] is not None else 0.0)
        if case["mod"] != "none":
            h = h + h * s["scale"].double() + s["shift"].double()
        return (h, r) if case["y"] else h
    if case["op"] == "adapt":
        out = s["y"].double()
        for at, n, a in _requests(case):
            if n and a >= 0:
                R = _ranks(case)[a]
                delta = s["down"][a, :R].double().t() @ s["up"][a, :R].double() if n > 4 * (case["K"] + R) else None
                x = s["x"][at:at + n].double()
                add = x @ delta if delta is not None else (x @ s["down"][a, :R].double().t()) @ s["up"][a, :R].double()
                out[at:at + n] += s["scaling"][a].double() * add
        return out
    if case["op"] == "prompt":
        out, at, group = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV), 0, case["HQ"] // case["HKV"]
        for n in _lengths(case["T"], case["S"]):
            for h in range(case["HQ"] if n else 0):
                q, k, v = (s[i][at:at + n, j].double() for i, j in (("q", h), ("k", h // group), ("v", h // group)))
                score = q @ k.t() / math.sqrt(case["D"])
                if case["causal"]:
                    score = score.masked_fill(torch.ones_like(score, dtype=torch.bool).triu(1), -math.inf)
                out[at:at + n, h] = torch.softmax(score, 1) @ v
            at += n
        return out
    if case["op"] == "append":
        k, v, page = s["k_cache"].double(), s["v_cache"].double(), case["page"]
        for t, slot in enumerate(s["slots"].tolist()):
            if slot >= 0:
                k[slot // page, slot % page] = s["k"][t].double()
                v[slot // page, slot % page] = s["v"][t].double()
        return k, v
    B, Q, HQ, D, page = case["B"], case["Q"], case["HQ"], case["D"], case["page"]
    group = HQ // case["HKV"]
    out = torch.zeros((B, Q, HQ, D), dtype=torch.float64, device=DEV)
    lse = torch.full((B, HQ, Q), -math.inf, dtype=torch.float64, device=DEV)
    for b, n in enumerate(_cache_lens(case)):
        pages = s["table"][b, :-(-n // page)].long()
        for i in range(Q):
            m = n - Q + 1 + i                             # keys that token i of the new ones sees
            for h in range(HQ if m > 0 else 0):
                k, v = (s[c][pages, :, h // group].reshape(-1, D)[:m].double() for c in ("k_cache", "v_cache"))
                score = k @ s["q"][b, i, h].double() / math.sqrt(D)
                lse[b, h, i] = torch.logsumexp(score, 0)
                out[b, i, h] = torch.exp(score - lse[b, h, i]) @ v
    return out, lse
