"""Measured cases of the decode operators around the 4-bit products: a paged
cache of keys and values held in 4 bits (kv4_append), attention over it
(kv4_attention), low-rank adapters of many requests beside a linear layer on
4-bit weights (linear_w4_lora), and penalties, biases and grammar masks on
logits (adjust_logits).

`run` computes a case in its plain form, elementary torch operations in fp32
(the cache's transforms in fp64: their values are rounded to 4 bits), or,
where `own` is true, through the package's entry points.  `exact` is the
operator's definition in float64.
"""

import math

import torch

own = False

GROUP = {"mxfp4": 32, "nvfp4": 16, "int4": 32}
TYPE = {"bf16": torch.bfloat16, "f32": torch.float32, "f16": torch.float16}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
CACHE_CAP = 16 * 131072 * 8 * 128     # tokens * kv heads * head width of the largest cache
PAIR_CAP = 2 * 1000 * 16384 * 32 * 128  # queries * tokens * heads * head width of the largest prompt
WEIGHT_CAP = 57344 * 8192             # N * K of the largest layer
LOGIT_CAP = 200 * 100003


def listed():
    return [
        # One short chat, one token: latency counts.
        _attend("attend one mxfp4", "mxfp4", 1, 400, 500, 1, 32, 8, 128, 16, 0, False),
        # A serving batch of chats of every length, wide groups, transformed keys.
        _attend("attend batch nvfp4 T", "nvfp4", 48, 1, 8192, 1, 32, 4, 128, 64, 0, True),
        # Long documents, the largest cache.
        _attend("attend long int4", "int4", 16, 40000, 131072, 1, 64, 8, 128, 128, 0, False),
        # Two prompts' chunks behind long prefixes.
        _attend("attend prompt mxfp4", "mxfp4", 2, 15000, 16384, 1000, 32, 8, 128, 64, 0, False),
        # Three drafted tokens per request in a sliding window, one head per key head, narrow heads.
        _attend("attend window mxfp4", "mxfp4", 33, 100, 9000, 3, 16, 16, 64, 32, 1000, False),
        # The new tokens of one decode step.
        _append("append step int4", "int4", 64, 8, 128, 16, False),
        # A prompt's keys and values with their online transforms.
        _append("append prompt mxfp4 T", "mxfp4", 8200, 8, 128, 64, True),
        # One request with its adapter through an attention output projection.
        _lora("adapter one token mxfp4", "mxfp4", 1, 4096, 4096, 16, 4, False, "bf16"),
        # A batch of requests over many adapters through a fused gate|up layer.
        _lora("adapters batch nvfp4", "nvfp4", 64, 24576, 4096, 32, 40, False, "bf16"),
        # Odd sizes, wide adapters, the online block transform, fp32 result.
        _lora("adapters odd int4 T", "int4", 13, 5003, 5152, 64, 5, True, "f32"),
        # The sampled token of one request with a long history.
        _adjust("penalties one bf16", 1, 131072, 0, "bf16", 3000, 1000, 20, True),
        # A batch under grammars: odd vocabulary, padded rows, fp32 logits.
        _adjust("penalties batch f32", 200, 100003, 5, "f32", 1500, 700, 100, True),
    ]


def _attend(name, fmt, B, lo, hi, queries, heads, kv_heads, D, page, window, transform):
    return {"name": name, "op": "attend", "fmt": fmt, "B": B, "lo": lo, "hi": hi, "queries": queries, "heads": heads,
            "kv_heads": kv_heads, "D": D, "page": page, "window": window, "transform": transform}


def _append(name, fmt, n, kv_heads, D, page, transform):
    return {"name": name, "op": "append", "fmt": fmt, "n": n, "kv_heads": kv_heads, "D": D, "page": page,
            "transform": transform}


def _lora(name, fmt, M, N, K, rank, adapters, transform, out):
    return {"name": name, "op": "lora", "fmt": fmt, "M": M, "N": N, "K": K, "rank": rank, "adapters": adapters,
            "transform": transform, "out": out}


def _adjust(name, R, V, pad, dtype, prompt, output, biases, masked):
    return {"name": name, "op": "adjust", "R": R, "V": V, "pad": pad, "dtype": dtype, "prompt": prompt, "output": output,
            "biases": biases, "masked": masked}


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("attend", "attend", "attend", "append", "lora", "lora", "adjust"))
    fmt = rng.choice(("mxfp4", "nvfp4", "int4"))
    if op in ("attend", "append"):
        D = rng.choice((64, 128, 128, 256))
        kv_heads = rng.choice((1, 2, 4, 8, 16))
        page = rng.choice((16, 32, 64, 128, 256))
    if op == "attend":
        heads = kv_heads * rng.choice((1, 2, 4, 5, 8))
        B = _log_uniform(rng, 1, 64)
        hi = _log_uniform(rng, 64, min(131072, CACHE_CAP // (B * kv_heads * D)))
        queries = rng.choice((1, 1, 1, rng.randint(2, 8), _log_uniform(rng, 9, 2000)))
        queries = min(queries, hi, max(1, PAIR_CAP // (B * hi * heads * D)))
        lo = _log_uniform(rng, max(1, queries, hi // 100), hi)
        window = rng.choice((0, 0, 0, _log_uniform(rng, 16, hi)))
        c = _attend("", fmt, B, lo, hi, queries, heads, kv_heads, D, page, window, rng.random() < 0.3)
    elif op == "append":
        n = _log_uniform(rng, 1, min(16384, 8200 * 8 * 128 // (kv_heads * D)))
        c = _append("", fmt, n, kv_heads, D, page, rng.random() < 0.5)
    elif op == "lora":
        K = max(256, _log_uniform(rng, 256, 16384) // 32 * 32)
        N = _log_uniform(rng, 64, min(57344, WEIGHT_CAP // 8 // K))
        c = _lora("", fmt, _log_uniform(rng, 1, 64), N, K, rng.choice((8, 16, 16, 32, 64)), _log_uniform(rng, 1, 40),
                  rng.random() < 0.3, rng.choice(("bf16", "bf16", "f32")))
    else:
        V = _log_uniform(rng, 1000, 200000)
        c = _adjust("", _log_uniform(rng, 1, min(256, LOGIT_CAP // V)), V, rng.choice((0, 0, 8, 11)),
                    rng.choice(("bf16", "bf16", "f16", "f32")), _log_uniform(rng, 1, 4000), _log_uniform(rng, 1, 2000),
                    rng.choice((0, 1, 20, 100)), rng.random() < 0.5)
    c.pop("name")
    return c


# ---------------------------------------------------------------- inputs

def _code_table(fmt, device):
    """65536 bytes to draw from: two codes each, of normal values scaled to their group's largest."""
    g = torch.Generator().manual_seed(6)
    v = torch.randn(65536, 2, generator=g)
    if fmt == "int4":
        nib = (v * 2.7).round().clamp(-7, 7).to(torch.int64) & 15
    else:
        mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
        v = v * 2.2
        nib = torch.bucketize(v.abs(), mid) + 8 * (v < 0).to(torch.int64)
    return (nib[:, 0] | (nib[:, 1] << 4)).to(torch.uint8).to(device)


def _quantized(fmt, lead, K, gen, size):
    """Codes [*lead, K/2] and scales [*lead, K/G] of values of about this size; NVFP4's are relative to a tensor scale."""
    dev = gen.device
    rows = math.prod(lead)
    pick = torch.randint(0, 65536, (rows * (K // 2),), generator=gen, device=dev, dtype=torch.int32)
    codes = _code_table(fmt, dev).index_select(0, pick).view(*lead, K // 2)
    shape = (*lead, K // GROUP[fmt])
    if fmt == "mxfp4":
        e = 126 + round(math.log2(size))
        scales = torch.randint(e - 1, e + 2, shape, generator=gen, device=dev, dtype=torch.int32).to(torch.uint8)
    elif fmt == "nvfp4":
        scales = torch.randint(104, 127, shape, generator=gen, device=dev, dtype=torch.int32).to(torch.uint8)
    else:
        scales = (size * (0.2 + 0.3 * torch.rand(shape, generator=gen, device=dev))).to(torch.float16)
    return codes, scales


def _tensor_scale(fmt, gen, size):
    return size * (1.5e-3 + 1e-3 * torch.rand(1, generator=gen, device=gen.device)) if fmt == "nvfp4" else None


def _bank(gen, *shape):
    """Well-conditioned dense block transforms."""
    return (torch.randn(*shape, generator=gen, device=gen.device) / math.sqrt(shape[-1])).to(torch.bfloat16)


def _outliers(x, gen):
    """A few persistent outlier channels."""
    at = torch.randint(0, x.shape[-1], (max(1, x.shape[-1] // 100),), generator=gen, device=gen.device)
    x[..., at] *= 8.0
    return x.to(torch.bfloat16)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dev, s, fmt = gen.device, dict(case), case.get("fmt")

    def rand(*shape):
        return torch.rand(*shape, generator=gen, device=dev)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    if case["op"] == "attend":
        B, lo, hi, Q, H, kv, D, P = (case[n] for n in ("B", "lo", "hi", "queries", "heads", "kv_heads", "D", "page"))
        u = rand(B)
        u[0] = 1.0  # one sequence of the largest length
        lengths = (lo * (hi / lo) ** u).round().clamp(lo, hi).to(torch.int32)
        # Prompts' chunks end where they end: up to a fifth fewer queries than the most.
        count = Q - Q // 5 * torch.arange(B, device=dev) // max(B - 1, 1)
        start = torch.zeros(B + 1, dtype=torch.int32, device=dev)
        start[1:] = count.cumsum(0)
        pages = ((lengths + P - 1) // P).long()
        width, total = int(pages.max()), int(pages.sum())
        # Pages in any order, with some of other requests between them.
        order = torch.randperm(total + 7, generator=gen, device=dev).to(torch.int32)
        col = torch.arange(width, device=dev)
        at = (pages.cumsum(0) - pages).unsqueeze(1) + col
        s["table"] = torch.where(col < pages.unsqueeze(1), order[at.clamp(max=total + 6)], 0).to(torch.int32)
        s["lengths"], s["start"] = lengths, start
        s["k"] = (*_quantized(fmt, (total + 7, kv, P), D, gen, 0.5), _tensor_scale(fmt, gen, 0.5))
        s["v"] = (*_quantized(fmt, (total + 7, kv, P), D, gen, 1.0), _tensor_scale(fmt, gen, 1.0))
        s["n"], s["most"] = int(start[-1]), Q
        s["q"] = normal(s["n"], H, D).to(torch.bfloat16)
        s["T"] = _bank(gen, kv, D // GROUP[fmt], GROUP[fmt], GROUP[fmt]) if case["transform"] else None
    elif case["op"] == "append":
        n, kv, D, P = (case[n] for n in ("n", "kv_heads", "D", "page"))
        pages = (n + P - 1) // P + 1
        qkv = normal(n, kv * 3, D)  # keys and values as views of one projection
        s["keys"] = _outliers(qkv, gen)[:, kv:2 * kv]
        s["values"] = normal(n, kv, D).to(torch.bfloat16)
        slots = torch.randperm(pages * P, generator=gen, device=dev)[:n]
        slots[3::17] = -1  # padding of the batch
        s["slots"] = slots
        s["k"] = (*_quantized(fmt, (pages, kv, P), D, gen, 0.5), _tensor_scale(fmt, gen, 8.0))
        s["v"] = (*_quantized(fmt, (pages, kv, P), D, gen, 0.5), _tensor_scale(fmt, gen, 2.0))
        G = GROUP[fmt]
        s["T_k"], s["T_v"] = (_bank(gen, kv, D // G, G, G) if case["transform"] else None for _ in range(2))
    elif case["op"] == "lora":
        M, N, K, r, E = (case[n] for n in ("M", "N", "K", "rank", "adapters"))
        G = GROUP[fmt]
        s["x"] = _outliers(normal(M, K), gen)
        s["codes"], s["scales"] = _quantized(fmt, (N,), K, gen, 0.02)
        s["gs"] = _tensor_scale(fmt, gen, 0.02)
        s["A"] = (normal(E, r, K) / math.sqrt(K)).to(torch.bfloat16)
        s["B"] = (normal(E, N, r) / math.sqrt(r)).to(torch.bfloat16)
        s["scale"] = 0.5 + rand(E)
        ids = torch.randint(0, E, (M,), generator=gen, device=dev).to(torch.int32)
        ids[2::9] = -1  # requests without an adapter
        s["ids"] = ids
        s["T"] = _bank(gen, K // G, G, G) if case["transform"] else None
    else:
        R, V = case["R"], case["V"]
        s["logits"] = (normal(R, V + case["pad"]) * 2.5).to(TYPE[case["dtype"]])[:, :V]
        # Texts repeat few of a vocabulary's tokens often.
        def text(length):
            t = (V ** rand(R, length)).to(torch.int32) - 1
            return t.masked_fill_(torch.arange(length, device=dev) >= (length * (0.5 + 0.5 * rand(R, 1))), -1)
        s["prompt_ids"], s["output_ids"] = text(case["prompt"]), text(case["output"])
        s["rep"], s["freq"], s["pres"] = 1 + 0.3 * rand(R), 0.5 * rand(R), 0.5 * rand(R)
        n = min(case["biases"], V)
        s["bias_ids"] = s["bias"] = s["allowed"] = None
        if n:
            step = V // n
            s["bias_ids"] = (torch.arange(n, device=dev) * step + (step * rand(R, n)).long().clamp(max=step - 1)).to(
                torch.int32)
            s["bias"] = 4 * normal(R, n)
        if case["masked"]:
            words = torch.randint(-2**31, 2**31, (R, (V + 31) // 32), generator=gen, device=dev)
            words[1::4] = -1  # no grammar
            words[3:4] = 0    # nothing is allowed
            s["allowed"] = words.to(torch.int32)
    return s


# ---------------------------------------------------------------- the operators

def run(state):
    return (_own if own else _plain)[state["op"]](state)


def _own_attend(s):
    import mxfp4_activation_amd as wush
    cache = wush.KV4Cache(s["k"][0], s["k"][1], s["v"][0], s["v"][1], s["k"][2], s["v"][2])
    return wush.kv4_attention(s["fmt"], s["q"], cache, s["table"], s["lengths"], q_start=s["start"], window=s["window"],
                              T_q=s["T"])


def _own_append(s):
    import mxfp4_activation_amd as wush
    fmt, D = s["fmt"], s["D"]
    cache = wush.KV4Cache(s["k"][0], s["k"][1], s["v"][0], s["v"][1], s["k"][2], s["v"][2])
    wush.kv4_append(fmt, s["keys"], s["values"], cache, s["slots"], T_k=s["T_k"], T_v=s["T_v"])
    return tuple(wush.dequant(fmt, c.view(-1, D // 2), sc.view(-1, D // GROUP[fmt]), g) for c, sc, g in (s["k"], s["v"]))


def _own_lora(s):
    import mxfp4_activation_amd as wush
    return wush.linear_w4_lora(s["fmt"], s["x"], s["codes"], s["scales"], wush.LoraAdapters(s["A"], s["B"], s["scale"]),
                               s["ids"], T=s["T"], global_scale=s["gs"], out_dtype=TYPE[s["out"]])


def _own_adjust(s):
    import mxfp4_activation_amd as wush
    return wush.adjust_logits(s["logits"], prompt=s["prompt_ids"], output=s["output_ids"], repetition=s["rep"],
                              frequency=s["freq"], presence=s["pres"], bias_ids=s["bias_ids"], bias=s["bias"],
                              allowed=s["allowed"])


def _e4m3(c):
    c = c.to(torch.int32)
    e, m = (c >> 3).float(), (c & 7).float()
    return torch.where(e > 0, (1 + m / 8) * torch.exp2(e - 7), m * 2.0 ** -9)


def _dequant(fmt, codes, scales, gs):
    """fp32 values of codes [..., K/2] with scales [..., K/G] and a tensor scale or None."""
    if fmt == "int4":
        table = [float(i) for i in range(8)] + [float(i) for i in range(-8, 0)]
    else:
        table = list(E2M1) + [-v for v in E2M1]
    # Both values of every byte at once.
    t = torch.tensor(table, device=codes.device)
    pair = torch.stack((t.repeat(16), t.repeat_interleave(16)), 1)
    v = pair.index_select(0, codes.reshape(-1).to(torch.int32)).view(*scales.shape, GROUP[fmt])
    if fmt == "mxfp4":
        sc = torch.exp2(scales.float() - 127.0)
    elif fmt == "nvfp4":
        sc = _e4m3(scales) * gs
    else:
        sc = scales.float()
    return (v * sc.unsqueeze(-1)).view(*codes.shape[:-1], codes.shape[-1] * 2)


def _quantize(fmt, y, gs):
    """Codes and scales of fp32 values [..., D], rounded to nearest, ties to even."""
    yb = y.unflatten(-1, (-1, GROUP[fmt]))
    amax = yb.abs().amax(-1, keepdim=True)
    if fmt == "int4":
        scales = (amax / 7).to(torch.float16)
        s = scales.float()
        v = torch.where(s > 0, yb * (1 / s), 0.0).clamp(-7, 7).round().to(torch.int32) & 15
    else:
        if fmt == "mxfp4":
            e = torch.where(amax > 0, torch.frexp(amax).exponent - 3, -127).clamp(-127, 127)
            scales = (e + 127).to(torch.uint8)
            v = torch.ldexp(yb, -e)
        else:
            e4m3 = (amax / 6 / gs).clamp(max=448.0).to(torch.float8_e4m3fn)
            scales, eff = e4m3.view(torch.uint8), e4m3.float() * gs
            v = torch.where(eff > 0, yb * (1 / eff), 0.0)
        # A tie goes to the even code: up from 0.75, 1.75 and 3.5.
        below = [math.nextafter(m, 0) if up else m for m, up in zip((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0), (0, 1) * 4)]
        mid = torch.tensor(below, dtype=torch.float64, device=y.device)
        v = torch.bucketize(v.abs().double(), mid).to(torch.int32) + 8 * torch.signbit(v).to(torch.int32)
    v = v.flatten(-2)
    return (v[..., ::2] | (v[..., 1::2] << 4)).to(torch.uint8), scales.squeeze(-1)


def _transform(x, T):
    """Block c of the last axis times T[..., c, :, :], in x's type."""
    C, G = T.shape[-3], T.shape[-1]
    return (T.to(x.dtype) * x.view(*x.shape[:-1], C, 1, G)).sum(-1).view(x.shape)


def _plain_attend(s):
    fmt, D, H, kv, Q = s["fmt"], s["D"], s["heads"], s["kv_heads"], s["most"]
    B, L = s["table"].shape[0], s["table"].shape[1] * s["page"]
    pages = s["table"].reshape(-1)

    def read(codes, scales, gs):
        x = _dequant(fmt, codes.index_select(0, pages), scales.index_select(0, pages), gs)
        return x.view(B, -1, kv, s["page"], D).transpose(1, 2).reshape(B, kv, L, D)

    count = (s["start"][1:] - s["start"][:-1]).unsqueeze(1)
    i = torch.arange(Q, device=pages.device)
    row = (s["start"][:-1].unsqueeze(1) + i).clamp(max=s["n"] - 1)
    q = s["q"].float()
    if s["T"] is not None:
        q = _transform(q.view(-1, kv, H // kv, D), s["T"].unsqueeze(1)).view(-1, H, D)
    q = q[row].view(B, Q, kv, H // kv, D).permute(0, 2, 1, 3, 4).reshape(B, kv, -1, D)
    w = torch.matmul(q, read(*s["k"]).transpose(2, 3)).mul_(D ** -0.5)
    at = s["lengths"].unsqueeze(1) - count + i  # each query's place
    t = torch.arange(L, device=pages.device)
    seen = t <= at.unsqueeze(2)
    if s["window"]:
        seen &= t > at.unsqueeze(2) - s["window"]
    w.view(B, kv, Q, H // kv, L).masked_fill_(~seen.view(B, 1, Q, 1, L), -math.inf)
    w.sub_(w.amax(-1, keepdim=True).clamp(min=-1e30)).exp_()
    out = torch.matmul(w, read(*s["v"])) / w.sum(-1, keepdim=True).clamp(min=1e-30)
    out = out.view(B, kv, Q, H // kv, D).permute(0, 2, 1, 3, 4).reshape(B, Q, H, D)
    return out[i < count].to(torch.bfloat16)


def _plain_append(s):
    fmt, D = s["fmt"], s["D"]
    use = (s["slots"] >= 0).nonzero().squeeze(1)
    slot = s["slots"][use]
    page, place = slot // s["page"], slot % s["page"]

    def write(x, T, held):
        x = x[use]
        y = x.float() if T is None else _transform(x.double(), T).float()
        codes, scales = _quantize(fmt, y, held[2])
        held[0][page, :, place] = codes
        held[1][page, :, place] = scales
        return _dequant(fmt, *held).view(-1, D)

    return write(s["keys"], s["T_k"], s["k"]), write(s["values"], s["T_v"], s["v"])


def _plain_lora(s):
    x = s["x"].float()
    xt = x if s["T"] is None else _transform(x, s["T"])
    y = xt @ _dequant(s["fmt"], s["codes"], s["scales"], s["gs"]).t()
    a = s["ids"].clamp(min=0)
    h = (s["A"][a].float() * x.unsqueeze(1)).sum(-1) * s["scale"][a].unsqueeze(1)
    h = h * (s["ids"] >= 0).unsqueeze(1)
    return (y + (s["B"][a].float() * h.unsqueeze(1)).sum(-1)).to(TYPE[s["out"]])


def _plain_adjust(s):
    l = s["logits"].float()
    R, V = l.shape

    def counts(ids):
        # Padding is counted behind the vocabulary.
        n = torch.zeros(R, V + 1, dtype=torch.int32, device=l.device)
        at = torch.where(ids < 0, V, ids).long()
        return n.scatter_add_(1, at, torch.ones_like(at, dtype=torch.int32))[:, :V]

    out = counts(s["output_ids"])
    seen = (out + counts(s["prompt_ids"])) > 0
    rep = s["rep"].unsqueeze(1)
    l = torch.where(seen, torch.where(l > 0, l / rep, l * rep), l)
    l = l - s["freq"].unsqueeze(1) * out.float() - s["pres"].unsqueeze(1) * (out > 0).float()
    if s["bias"] is not None:
        l = l.scatter_add(1, s["bias_ids"].long(), s["bias"])
    if s["allowed"] is not None:
        v = torch.arange(V, device=l.device)
        ok = (s["allowed"][:, v // 32] >> (v % 32).to(torch.int32)) & 1
        l = l.masked_fill(ok == 0, -math.inf)
    return l.to(s["logits"].dtype)


_plain = {"attend": _plain_attend, "append": _plain_append, "lora": _plain_lora, "adjust": _plain_adjust}
_own = {"attend": _own_attend, "append": _own_append, "lora": _own_lora, "adjust": _own_adjust}


# ---------------------------------------------------------------- work and definition

def _row_bytes(fmt, K):
    """Bytes of K values in 4 bits with their scales."""
    return K // 2 + K // GROUP[fmt] * (2 if fmt == "int4" else 1)


def work(case):
    fmt = case.get("fmt")
    if case["op"] == "attend":
        B, lo, hi, Q, H, kv, D = (case[n] for n in ("B", "lo", "hi", "queries", "heads", "kv_heads", "D"))
        mean = (hi - lo) / math.log(hi / lo) if hi > lo else hi
        rest = sum(Q - Q // 5 * b // max(B - 1, 1) for b in range(1, B))
        reach = case["window"] + Q if case["window"] else math.inf
        tokens = min(hi, reach) + (B - 1) * min(mean, reach)
        see = case["window"] or math.inf
        pairs = Q * min(see, hi - Q / 2) + rest * min(see, max(mean - Q / 2, Q / 2))
        n = Q + rest
        T = case["transform"]
        return {"bytes": int(tokens * kv * 2 * _row_bytes(fmt, D) + 4 * n * H * D + (2 * kv * D * GROUP[fmt] if T else 0)),
                "flops": int(4 * pairs * H * D + (2 * n * H * D * GROUP[fmt] if T else 0))}
    if case["op"] == "append":
        n, kv, D, P = (case[x] for x in ("n", "kv_heads", "D", "page"))
        T, rows = case["transform"], ((n + P - 1) // P + 1) * P * kv
        # Keys and values in, their codes out; then the whole small cache as fp32 values.
        return {"bytes": 2 * n * kv * (2 * D + _row_bytes(fmt, D)) + 2 * rows * (_row_bytes(fmt, D) + 4 * D)
                + (4 * kv * D * GROUP[fmt] if T else 0),
                "flops": 4 * n * kv * D * GROUP[fmt] if T else 0}
    if case["op"] == "lora":
        M, N, K, r, E = (case[n] for n in ("M", "N", "K", "rank", "adapters"))
        T = case["transform"]
        used = E * (1 - (1 - 1 / E) ** M)
        return {"bytes": int(N * _row_bytes(fmt, K) + 2 * M * K + used * 2 * r * (K + N)
                             + M * N * (4 if case["out"] == "f32" else 2) + (2 * K * GROUP[fmt] if T else 0)),
                "flops": 2 * M * N * K + 2 * M * r * (K + N) + (2 * M * K * GROUP[fmt] if T else 0)}
    R, V = case["R"], case["V"]
    return {"bytes": R * (2 * V * (4 if case["dtype"] == "f32" else 2) + 4 * (case["prompt"] + case["output"])
                          + 8 * case["biases"] + (V // 8 if case["masked"] else 0) + 12), "flops": 6 * R * V}


def _values64(fmt, codes, scales, gs):
    """Codes and scales from the bits of the formats' definitions, in float64."""
    n = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).to(torch.int16)
    if fmt == "int4":
        v = (n - 16 * (n >> 3)).double()
        s = scales.double()
    else:
        e, m = (n >> 1) & 3, (n & 1).double()
        v = torch.where(e == 0, 0.5 * m, torch.ldexp(1 + 0.5 * m, (e - 1).double())) * (1 - 2 * (n >> 3)).double()
        b = scales.double()
        if fmt == "mxfp4":
            s = torch.ldexp(torch.ones_like(b), b - 127)
        else:
            s = scales.view(torch.float8_e4m3fn).double() * gs.double()
    return (v.unflatten(-1, (-1, GROUP[fmt])) * s.unsqueeze(-1)).flatten(-2)


def _blocks64(x, T):
    xb = x.double().unflatten(-1, (T.shape[-3], T.shape[-1]))
    return torch.matmul(T.double(), xb.unsqueeze(-1)).squeeze(-1).flatten(-2)


def _grid64(v, levels):
    """Nearest of the ascending non-negative levels per |v|, the even place between two, with v's sign."""
    g = torch.tensor(levels, dtype=torch.float64, device=v.device)
    hi = torch.searchsorted(g, v.abs().clamp(max=levels[-1]).contiguous())
    lo = (hi - 1).clamp(min=0)
    a = v.abs().clamp(max=levels[-1])
    d = (a - g[lo]) - (g[hi] - a)
    up = (d > 0) | ((d == 0) & (hi % 2 == 0))
    return torch.where(up, g[hi], g[lo]) * torch.where(v < 0, -1.0, 1.0)


def _held64(fmt, y, gs):
    """What fp32 values [..., D] become in 4 bits."""
    y = y.double().unflatten(-1, (-1, GROUP[fmt]))
    top = y.abs().amax(-1, keepdim=True)
    if fmt == "mxfp4":
        s = torch.exp2((top.clamp(min=2.0 ** -140).log2().floor() - 2).clamp(min=-127))
        # log2 may round up to a whole number just below a power of two.
        s = torch.where(s * 4 > top, torch.clamp(s / 2, min=2.0 ** -127), s)
        out = _grid64(y / s, list(E2M1)) * s
    elif fmt == "nvfp4":
        fp8 = [m * 2.0 ** -9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:-1]
        ratio = ((top / 6).float().double() / gs.double()).float().double()
        s = (_grid64(ratio, fp8) * gs.double()).float().double()
        v = (y * (1 / s).float().double()).float().double()
        out = torch.where(s > 0, _grid64(v, list(E2M1)), 0.0) * s
    else:
        s = (top / 7).float().half().double()
        v = (y * (1 / s).float().double()).float().double()
        out = torch.where(s > 0, v.clamp(-7, 7).round(), 0.0) * s
    return out.flatten(-2)


def exact(case, seed):
    s = prepare(case, seed)
    fmt, D = case.get("fmt"), case.get("D")
    if case["op"] == "attend":
        H, kv, P = case["heads"], case["kv_heads"], case["page"]
        out = []
        for b in range(case["B"]):
            L, lo, hi = int(s["lengths"][b]), int(s["start"][b]), int(s["start"][b + 1])
            pages = s["table"][b, :(L + P - 1) // P].long()
            q = s["q"][lo:hi].double().view(hi - lo, kv, H // kv, D)
            rows = []
            for h in range(kv):
                qh = q[:, h] if s["T"] is None else _blocks64(q[:, h], s["T"][h])
                K, V = (_values64(fmt, c[pages, h].reshape(-1, D // 2)[:L], sc[pages, h].reshape(-1, D // GROUP[fmt])[:L],
                                  g) for c, sc, g in (s["k"], s["v"]))
                w = qh.reshape(-1, D) @ K.t() / math.sqrt(D)
                at = torch.arange(L - (hi - lo), L, device=w.device).repeat_interleave(H // kv).unsqueeze(1)
                t = torch.arange(L, device=w.device)
                hide = (t > at) | ((t <= at - case["window"]) if case["window"] else False)
                rows.append((torch.softmax(w.masked_fill(hide, -math.inf), 1) @ V).view(hi - lo, H // kv, D))
            out.append(torch.stack(rows, 1).view(hi - lo, H, D))
        return torch.cat(out)
    if case["op"] == "append":
        answer = []
        for x, T, (codes, scales, g) in ((s["keys"], s["T_k"], s["k"]), (s["values"], s["T_v"], s["v"])):
            y = x.float() if T is None else _blocks64(x, T).float()
            held = _values64(fmt, codes, scales, g).transpose(1, 2).flatten(0, 1)  # [slots, heads, D]
            use = s["slots"] >= 0
            held[s["slots"][use]] = _held64(fmt, y[use], g)
            answer.append(held.unflatten(0, (-1, case["page"])).transpose(1, 2).reshape(-1, D))
        return tuple(answer)
    if case["op"] == "lora":
        x = s["x"].double()
        xt = x if s["T"] is None else _blocks64(s["x"], s["T"])
        y = xt @ _values64(fmt, s["codes"], s["scales"], s["gs"]).t()
        for a in range(case["adapters"]):
            m = s["ids"] == a
            y[m] += s["scale"][a].double() * (x[m] @ s["A"][a].double().t()) @ s["B"][a].double().t()
        return y
    l = s["logits"].double()
    for r in range(case["R"]):
        said = s["output_ids"][r]
        n = torch.bincount(said[said >= 0], minlength=case["V"]).double()
        asked = s["prompt_ids"][r]
        seen = (n + torch.bincount(asked[asked >= 0], minlength=case["V"])) > 0
        row, rep = l[r], s["rep"][r].double()
        row = torch.where(seen, row * torch.where(row > 0, 1 / rep, rep), row)
        row = row - n * s["freq"][r].double() - torch.sign(n) * s["pres"][r].double()
        if s["bias"] is not None:
            row[s["bias_ids"][r].long()] += s["bias"][r].double()
        l[r] = row
    if s["allowed"] is not None:
        bits = (s["allowed"].unsqueeze(2) >> torch.arange(32, device=l.device, dtype=torch.int32)) & 1
        l[bits.flatten(1)[:, :case["V"]] == 0] = -math.inf
    return l
