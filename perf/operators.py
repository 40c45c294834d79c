"""Cases of the decoding-step operators: the 4-bit paged key/value cache (append, read back, attention) and the
processing of logits before their softmax.

``run`` computes a case through the library (``own``) or in a plain form of elementary torch operations.
"""
import math
import random

import numpy as np
import torch

own = False

GROUP = 32  # elements that share a scale and a zero
BLOCK = 16  # tokens of a head that lie together in the cache


def _dtype(case):
    return {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[case["dtype"]]


def _lengths(case):
    """Cache lengths (with this step's tokens) and new tokens of each sequence: a function of the case alone."""
    rng = random.Random(case["batch"] * 1000003 + case["length"] * 101 + case["new"])
    lens, news = [], []
    for b in range(case["batch"]):
        frac = 1.0 if b == 0 else rng.random() if case["ragged"] else 1.0 - 0.05 * rng.random()
        n = max(1, int(case["length"] * frac))
        new = n if case["new"] == 0 else max(1, int(case["new"] * (rng.random() if case["ragged"] and b else 1.0)))
        lens.append(n)
        news.append(min(n, new))
    return lens, news


def listed():
    serve = {"op": "attention", "ragged": False, "new": 1, "scale": 0.0}
    append = {"op": "append", "ragged": True}
    gather = {"op": "gather", "ragged": True, "new": 0}
    logits = {"op": "logits"}
    return [
        # one user's first tokens: a launch-bound step
        {**serve, "name": "attention_short", "batch": 1, "length": 200, "hq": 32, "hkv": 8, "d": 128, "page": 16, "dtype": "bf16"},
        # two long documents, few sequences: the work has to be split over the keys
        {**serve, "name": "attention_long", "batch": 2, "length": 262144, "hq": 64, "hkv": 8, "d": 128, "page": 64, "dtype": "bf16"},
        # a full batch of conversations of all lengths
        {**serve, "name": "attention_batch", "batch": 64, "length": 16384, "hq": 32, "hkv": 8, "d": 128, "page": 32, "dtype": "fp16", "ragged": True},
        # four drafted tokens per sequence checked at once, heads of 64
        {**serve, "name": "attention_draft", "batch": 16, "length": 8191, "hq": 64, "hkv": 8, "d": 64, "page": 16, "dtype": "bf16", "new": 4},
        # a decoding batch: one token per sequence, wherever its page ends
        {**append, "name": "append_decode", "batch": 128, "length": 4096, "new": 1, "hq": 32, "hkv": 8, "d": 128, "rot": 128, "pairs": "halves", "page": 16, "dtype": "bf16"},
        # chunks of prompts
        {**append, "name": "append_prompt", "batch": 4, "length": 20000, "new": 8192, "hq": 32, "hkv": 8, "d": 128, "rot": 128, "pairs": "halves", "page": 64, "dtype": "bf16"},
        # drafts and short prompts, a part of each head rotated, neighbouring pairs
        {**append, "name": "append_odd", "batch": 21, "length": 1500, "new": 77, "hq": 12, "hkv": 4, "d": 64, "rot": 32, "pairs": "neighbours", "page": 16, "dtype": "fp16"},
        # a short prompt's prefix read back
        {**gather, "name": "gather_short", "batch": 1, "length": 777, "hkv": 8, "d": 64, "page": 32, "dtype": "fp16"},
        # long prefixes read back for the next chunks of their prompts
        {**gather, "name": "gather_prefix", "batch": 4, "length": 65536, "hkv": 8, "d": 128, "page": 64, "dtype": "bf16"},
        # one sampled token: latency
        {**logits, "name": "logits_one", "rows": 1, "vocab": 131072, "dtype": "bf16", "history": 1000, "bias": 16, "mask": True, "out": "softmax"},
        # a batch with long histories
        {**logits, "name": "logits_batch", "rows": 256, "vocab": 131072, "dtype": "bf16", "history": 8192, "bias": 64, "mask": True, "out": "softmax"},
        # odd rows in 32 bits, log probabilities
        {**logits, "name": "logits_odd", "rows": 37, "vocab": 50021, "dtype": "fp32", "history": 333, "bias": 300, "mask": False, "out": "log_softmax"},
    ]


def draw(rng):
    def spread(lo, hi):
        return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))

    op = rng.choice(["attention", "attention", "attention", "append", "append", "gather", "logits", "logits"])
    if op == "logits":
        vocab = spread(1000, 262144)
        return {"op": op, "rows": spread(1, max(1, min(256, 256 * 131072 // vocab))), "vocab": vocab, "dtype": rng.choice(["bf16", "fp16", "fp32"]),
                "history": spread(1, 8192), "bias": rng.choice([0, 1, 17, 300]), "mask": rng.random() < 0.5,
                "out": rng.choice(["softmax", "log_softmax", "logits"])}
    hkv, d = rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
    case = {"op": op, "hkv": hkv, "d": d, "page": rng.choice([16, 32, 64, 128]), "dtype": rng.choice(["bf16", "fp16"]),
            "ragged": rng.random() < 0.6}
    if op == "attention":
        batch = spread(1, 128)
        return {**case, "batch": batch, "length": spread(1, 524288 // batch), "hq": hkv * rng.choice([1, 2, 3, 4, 7, 8, 16]),
                "new": rng.choice([1, 1, 1, 2, 5, 8]), "scale": rng.choice([0.0, 0.11])}
    if op == "append":
        batch = spread(1, 128)
        new = 1 if rng.random() < 0.4 else spread(1, 16384 // batch)
        return {**case, "batch": batch, "length": new + spread(1, 8192), "new": new, "hq": hkv * rng.choice([1, 3, 4, 8]),
                "rot": rng.choice([0, 32, d]), "pairs": rng.choice(["halves", "neighbours"])}
    batch = spread(1, 32)
    return {**case, "batch": batch, "length": spread(1, 262144 // batch), "new": 0}


# ---- inputs ---------------------------------------------------------------------------------------------------


def _paged(case, gen):
    """A filled cache, the pages of each sequence in a random order, lengths and offsets of the new tokens."""
    lens, news = _lengths(case)
    page, hkv, d = case["page"], case["hkv"], case["d"]
    width = -(-max(lens) // page)
    used = [-(-n // page) for n in lens]
    total = sum(used) + 3
    groups = d // GROUP
    cache = torch.randint(0, 256, (total, hkv, page // BLOCK, 20 * d), dtype=torch.uint8, device="cuda", generator=gen)
    shape = (total, hkv, page // BLOCK, 2, BLOCK * groups)
    # groups of 32 normal values of a varying amplitude: range about 4 sd, from about -2 sd
    sd = torch.exp(0.4 * torch.randn(shape, device="cuda", generator=gen))
    zero = -2.0 * sd * (1 + 0.1 * torch.randn(shape, device="cuda", generator=gen))
    tail = torch.stack([(sd * (4.0 / 15)).half(), zero.half()], dim=-2)  # K scales, K zeros, V scales, V zeros
    cache[..., 16 * d:] = tail.reshape(*shape[:3], -1).view(torch.uint8)
    order = torch.randperm(total, device="cuda", generator=gen)
    starts = np.concatenate([[0], np.cumsum(used)])
    table = np.zeros((len(lens), width), np.int64)
    for b, n in enumerate(used):
        table[b, :n] = np.arange(starts[b], starts[b] + n)
    table = order[torch.from_numpy(table).cuda()].to(torch.int32).contiguous()
    cu = torch.tensor(np.concatenate([[0], np.cumsum(news)]), dtype=torch.int32, device="cuda")
    return {"cache": cache, "table": table, "lens": torch.tensor(lens, dtype=torch.int32, device="cuda"),
            "cu": None if max(news) == 1 else cu, "tokens": int(sum(news)), "most": max(news)}


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = _dtype(case)
    if case["op"] == "logits":
        M, N, L = case["rows"], case["vocab"], case["history"]
        x = (2.5 * torch.randn(M, N, device="cuda", generator=gen)).to(dt)
        total = torch.randint(1, L + 1, (M,), device="cuda", generator=gen)
        total[0] = L
        prompt = (total * torch.rand(M, device="cuda", generator=gen)).long()
        # text repeats itself: tokens from a short part of the vocabulary, some many times
        u = torch.rand(M, L, device="cuda", generator=gen)
        tokens = (N * u ** 6).long().clamp(max=N - 1)
        tokens = torch.where(torch.arange(L, device="cuda")[None] < total[:, None], tokens, -1)
        s = {"case": case, "x": x, "tokens": tokens.int(), "prompt": prompt.int(), "total": total.int()}
        s["rep"] = 1 + 0.5 * torch.rand(M, device="cuda", generator=gen)
        s["freq"] = torch.rand(M, device="cuda", generator=gen) * 0.5
        s["pres"] = torch.rand(M, device="cuda", generator=gen)
        s["scale"] = 1 / (0.5 + torch.rand(M, device="cuda", generator=gen))
        K = case["bias"]
        ids = torch.rand(M, min(N, 4096), device="cuda", generator=gen).argsort(1)[:, :K]
        s["ids"] = (ids * (N // min(N, 4096))).int().contiguous() if K else None
        s["values"] = 3 * torch.randn(M, K, device="cuda", generator=gen) if K else None
        words = (N + 31) // 32
        s["mask"] = torch.randint(-(2 ** 31), 2 ** 31, (M, words), device="cuda", generator=gen).int() if case["mask"] else None
        return s
    s = {"case": case, **_paged(case, gen)}
    T, d = s["tokens"], case["d"]
    if case["op"] != "gather":
        s["q"] = (1.5 * torch.randn(T, case["hq"], d, device="cuda", generator=gen)).to(dt)
    if case["op"] == "append":
        # keys and values as a projection leaves them: side by side in one row a token
        kv = torch.randn(T, 2 * case["hkv"], d, device="cuda", generator=gen)
        kv = (kv * torch.exp(0.5 * torch.randn(1, 2 * case["hkv"], d, device="cuda", generator=gen))).to(dt)
        s["k"], s["v"] = kv[:, : case["hkv"]], kv[:, case["hkv"]:]
        if case["rot"]:
            half = case["rot"] // 2
            freq = torch.arange(half, dtype=torch.float64, device="cuda").mul(-math.log(10000.0) / half).exp()
            angle = torch.arange(case["length"], dtype=torch.float64, device="cuda")[:, None] * freq
            s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        else:
            s["cos_sin"] = None
    return s


# ---- plain forms ----------------------------------------------------------------------------------------------


def _where(s):
    """Sequence and position of each token of the step."""
    T = s["tokens"]
    i = torch.arange(T, device="cuda")
    lens = s["lens"].long()
    if s["cu"] is None:
        return i, lens - 1
    seq = torch.searchsorted(s["cu"][1:], i.int(), right=True)
    return seq, lens[seq] - (s["cu"].long()[seq + 1] - i)


def _nibbles(b):
    return torch.stack([b & 15, b >> 4], dim=-1)


def _unpack(blocks, d):
    """Keys and values [..., 16, d] in fp32 of blocks [..., 20 d]."""
    G, lead = d // GROUP, blocks.shape[:-1]
    n = len(lead)
    kc = _nibbles(blocks[..., : 8 * d].reshape(*lead, 16, 4, G, 4)).reshape(*lead, 16, 4, G, 8)
    kc = kc.transpose(n + 1, n + 2).reshape(*lead, 16, G, GROUP)
    vc = _nibbles(blocks[..., 8 * d: 16 * d].reshape(*lead, 2, 8, 4, G, 2, 2)).reshape(*lead, 2, 8, 4, G, 2, 4)
    order = [n + a for a in (0, 2, 4, 3, 1, 5)]  # f, t, e | j | g, n
    vc = vc.permute(*range(n), *order).reshape(*lead, 16, G, GROUP)
    h = blocks[..., 16 * d:].contiguous().view(torch.float16).reshape(*lead, 4, 16 * G).float()
    ks, kz = (h[..., a, :].reshape(*lead, 16, G, 1) for a in (0, 1))
    vs, vz = (h[..., a, :].reshape(*lead, 8, G, 2).transpose(n + 1, n + 2).reshape(*lead, 16, G, 1) for a in (2, 3))
    return (kc.float() * ks + kz).reshape(*lead, 16, d), (vc.float() * vs + vz).reshape(*lead, 16, d)


def _rotate(x, cs, rot, pairs):
    """x [T, H, d] fp32 rotated by cs [T, rot] (cosines, then sines)."""
    c, s = cs[:, None, : rot // 2], cs[:, None, rot // 2:]
    y = x.clone()
    a, b = (x[..., : rot // 2], x[..., rot // 2: rot]) if pairs == "halves" else (x[..., 0:rot:2], x[..., 1:rot:2])
    u, w = a * c - b * s, b * c + a * s
    if pairs == "halves":
        y[..., : rot // 2], y[..., rot // 2: rot] = u, w
    else:
        y[..., 0:rot:2], y[..., 1:rot:2] = u, w
    return y


def _quantise(x):
    """Codes, scales and zeros of x [T, H, d] fp32."""
    T, H, d = x.shape
    x = x.clamp(-65504, 65504).reshape(T, H, d // GROUP, GROUP)
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    z, s = lo.half(), ((hi - lo) / torch.full_like(lo, 15.0)).half()
    c = torch.round((x - z.float()) / s.float()).clamp(0, 15)  # a quotient half-way between two codes goes to the even one
    return torch.where(s > 0, c, torch.zeros_like(c)).to(torch.uint8), s[..., 0], z[..., 0]


def _plain_append(s):
    case = s["case"]
    hkv, d, page = case["hkv"], case["d"], case["page"]
    G = d // GROUP
    seq, pos = _where(s)
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    if case["rot"]:
        cs = s["cos_sin"][pos]
        q, k = (_rotate(x, cs, case["rot"], case["pairs"]) for x in (q, k))
    kc, ks, kz = _quantise(k)
    vc, vs, vz = _quantise(v)
    pages = s["table"].long()[seq, pos // page]
    blk, r = (pos % page) // BLOCK, (pos % BLOCK)[:, None, None]
    # halfwords of the cache: [block of a head][10 d]
    flat = s["cache"].view(-1).view(torch.int16)
    base = ((pages[:, None] * hkv + torch.arange(hkv, device="cuda")) * (page // BLOCK) + blk[:, None])[..., None] * (10 * d)

    def four(c):  # four codes to a halfword
        c = c.reshape(*c.shape[:2], -1, 4).int()
        return (c[..., 0] | c[..., 1] << 4 | c[..., 2] << 8 | c[..., 3] << 12).to(torch.int16)

    m = torch.arange(d // 4, device="cuda")  # quadruple m: dims 4 m ..
    j, g = m // 8, m % 8
    flat[base + r * (d // 4) + ((g // 2) * G + j) * 2 + g % 2] = four(kc.reshape(*k.shape))
    f, t, e = r // 8, (r % 8) // 2, r % 2
    flat[base + 4 * d + (((f * 8 + g) * 4 + t) * G + j) * 2 + e] = four(vc.reshape(*v.shape))
    j = torch.arange(G, device="cuda")
    for a, h in enumerate((ks, kz, vs, vz)):
        at = r * G + j if a < 2 else ((r // 2) * G + j) * 2 + e
        flat[base + 8 * d + a * 16 * G + at] = h.view(torch.int16)
    return q.to(s["q"].dtype)


def _plain_gather(s):
    case = s["case"]
    page = case["page"]
    seq, pos = _where(s)
    if case["op"] == "gather":  # whole sequences: every page of theirs, then their tokens
        k, v = _unpack(s["cache"][s["table"].long()], case["d"])  # [B, W, Hkv, blocks, 16, d]
        return tuple(x.transpose(2, 3).transpose(3, 4).reshape(*s["table"].shape, page, case["hkv"], case["d"])[seq, pos // page, pos % page].to(_dtype(case))
                     for x in (k, v))
    blocks = s["cache"][s["table"].long()[seq, pos // page], :, (pos % page) // BLOCK]  # [T, Hkv, 20 d]
    at = (pos % BLOCK)[:, None, None, None].expand(-1, case["hkv"], 1, case["d"])
    return tuple(x.gather(2, at)[:, :, 0].to(_dtype(case)) for x in _unpack(blocks, case["d"]))


def _plain_attention(s):
    case = s["case"]
    hq, hkv, d, dt = case["hq"], case["hkv"], case["d"], _dtype(case)
    B, W = s["table"].shape
    L = W * case["page"]
    k, v = _unpack(s["cache"][s["table"].long()], d)  # [B, W, Hkv, blocks, 16, d]
    k, v = (x.transpose(1, 2).reshape(B, hkv, L, d) for x in (k, v))
    scale = case["scale"] or 1 / math.sqrt(d)
    seq, pos = _where(s)
    slot = s["lens"].long()[seq] - 1 - pos  # from a sequence's last token back
    n = s["most"]
    q = torch.zeros(B, n, hkv, hq // hkv, d, device="cuda")
    q[seq, slot] = s["q"].float().reshape(-1, hkv, hq // hkv, d)
    q = q.permute(0, 2, 1, 3, 4).reshape(B, hkv, -1, d)
    z = (q @ k.transpose(-1, -2)) * scale  # [B, Hkv, n G, L]
    last = s["lens"].long()[:, None] - 1 - torch.arange(n, device="cuda")  # [B, n]
    last = last.repeat_interleave(hq // hkv, 1)[:, None, :, None]
    z = torch.where(torch.arange(L, device="cuda") <= last, z, -math.inf)
    m = z.amax(-1, keepdim=True)
    p = torch.exp(z - torch.where(m.isinf(), 0.0, m))
    l = p.sum(-1, keepdim=True)
    v = torch.where((torch.arange(L, device="cuda") < s["lens"].long()[:, None])[:, None, :, None], v, 0.0)
    o = torch.where(l > 0, p @ v / l, 0.0)
    lse = (m + torch.log(l)).reshape(B, hkv, n, -1)
    o = o.reshape(B, hkv, n, hq // hkv, d)
    o = o.permute(0, 2, 1, 3, 4).reshape(B, n, hq, d)[seq, slot]
    return o.to(dt), lse.permute(0, 2, 1, 3).reshape(B, n, hq)[seq, slot]


def _plain_logits(s):
    x = s["x"].float()
    M, N = x.shape
    L = s["tokens"].shape[1]
    at = torch.arange(L, device="cuda")[None]
    ids = s["tokens"].long().clamp(min=0)
    live = at < s["total"][:, None]
    written = live & (at >= s["prompt"][:, None])
    count = torch.zeros(M, N, device="cuda").scatter_add_(1, ids, written.float())
    seen = torch.zeros(M, N, device="cuda").scatter_add_(1, ids, live.float()) > 0
    rep = s["rep"][:, None]
    x = torch.where(seen, torch.where(x > 0, x / rep, x * rep), x)
    x = x - (s["freq"][:, None] * count + s["pres"][:, None] * (count > 0))
    if s["ids"] is not None:
        x = x.scatter_add(1, s["ids"].long(), s["values"])
    x = x * s["scale"][:, None]
    if s["mask"] is not None:
        col = torch.arange(N, device="cuda")
        x = torch.where((s["mask"][:, col // 32] >> (col % 32)) & 1 == 1, x, -math.inf)
    m = x.amax(1, keepdim=True)
    e = torch.exp(x - torch.where(m.isinf(), 0.0, m))
    d = e.sum(1, keepdim=True)
    lse = m + torch.log(d)
    y = x if s["case"]["out"] == "logits" else e / d if s["case"]["out"] == "softmax" else (x - m) - torch.log(d)
    return y.to(s["x"].dtype), lse[:, 0]


def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if own:
        import row_wise_online_gb300 as rwo

        if op == "logits":
            lse = torch.empty(case["rows"], device="cuda")
            y = rwo.logits_process_rows(s["x"], out=case["out"], lse_out=lse, tokens=s["tokens"], prompt_lens=s["prompt"], token_lens=s["total"],
                                        repetition=s["rep"], frequency=s["freq"], presence=s["pres"], bias_ids=s["ids"], bias_values=s["values"],
                                        mask=s["mask"], scale=s["scale"])
            return {"y": y, "lse": lse}
        paged = (s["cache"], s["table"], s["lens"])
        if op == "attention":
            lse = torch.empty(s["q"].shape[:2], device="cuda")
            o = rwo.attention_kv4(s["q"], *paged, cu_tokens=s["cu"], lse_out=lse, scale=case["scale"] or None)
            return {"o": o, "lse": lse}
        q = None
        if op == "append":
            q = rwo.kv4_append(s["k"], s["v"], *paged, cu_tokens=s["cu"], q=s["q"], cos_sin=s["cos_sin"], interleaved=case["pairs"] == "neighbours")
        k, v = rwo.kv4_gather(*paged, cu_tokens=s["cu"], num_tokens=s["tokens"], dtype=_dtype(case))
        return {"q": q, "k": k, "v": v}
    if op == "logits":
        y, lse = _plain_logits(s)
        return {"y": y, "lse": lse}
    if op == "attention":
        o, lse = _plain_attention(s)
        return {"o": o, "lse": lse}
    q = _plain_append(s) if op == "append" else None  # what a step appends is read back: the cache's values
    k, v = _plain_gather(s)
    return {"q": q, "k": k, "v": v}


def work(case):
    e = 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "logits":
        M, N = case["rows"], case["vocab"]
        return {"bytes": M * (2 * N * e + (N // 8 if case["mask"] else 0) + 4 * case["history"] + 8 * case["bias"] + 28), "flops": 6 * M * N}
    lens, news = _lengths(case)
    T, hkv, d = sum(news), case["hkv"], case["d"]
    held = 1.25 * d * hkv  # codes, scales and zeros of a token
    if case["op"] == "attention":
        keys = sum(n * k for n, k in zip(news, lens))
        return {"bytes": sum(lens) * held + T * case["hq"] * (2 * d * e + 4), "flops": 4 * case["hq"] * d * keys}
    back = T * (held + 2 * hkv * d * e)
    if case["op"] == "gather":
        return {"bytes": back, "flops": 4 * T * hkv * d}
    return {"bytes": back + T * (2 * hkv * d * e + held + 2 * case["hq"] * d * e + 4 * case["rot"]), "flops": T * d * (30 * hkv + 3 * case["hq"])}


# ---- 64 bits --------------------------------------------------------------------------------------------------


def _places(d):
    """Nibble of each (token, dim) of a block for keys and for values, and halfword of each (token, group)."""
    G = d // GROUP
    r, e = np.arange(16)[:, None], np.arange(d)[None]
    j, w = e // GROUP, e % GROUP
    k = (r * (d // 8) + G * (w // 8) + j) * 8 + w % 8
    v = 16 * d + ((((r // 8 * 8 + w // 4) * 4 + r % 8 // 2) * G + j) * 2 + r % 2) * 4 + w % 4
    return k, v, 8 * d + r * G + j, 8 * d + 32 * G + (r // 2 * G + j) * 2 + r % 2


def _decode64(blocks, d):
    """Keys and values [n, 16, d] of blocks [n, 20 d], in 64 bits."""
    kn, vn, kh, vh = (torch.from_numpy(a).to(blocks.device) for a in _places(d))
    half = blocks.contiguous().view(torch.float16).double()
    out = []
    for nib, h in ((kn, kh), (vn, vh)):
        c = (blocks[:, nib // 2].int() >> (4 * (nib % 2)).int()) & 15
        out.append(c.double() * half[:, h] + half[:, h + 16 * (d // GROUP)])
    return out


def _sequence64(s, b, h):
    """Keys and values of one sequence and head."""
    case = s["case"]
    n, page = int(s["lens"][b]), case["page"]
    pages = s["table"][b, : -(-n // page)].long()
    k, v = _decode64(s["cache"][pages, h].reshape(-1, 20 * case["d"]), case["d"])
    return k.reshape(-1, case["d"])[:n], v.reshape(-1, case["d"])[:n]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "logits":
        if case["rows"] * case["vocab"] > 40_000_000:
            return None
        ys, lses = [], []
        for r in range(case["rows"]):
            x = s["x"][r].double()
            toks = s["tokens"][r, : int(s["total"][r])].long()
            seen = torch.zeros_like(x).index_fill_(0, toks, 1.0) > 0
            count = torch.bincount(toks[int(s["prompt"][r]):], minlength=x.numel()).double()
            rep = s["rep"][r].double()
            x = torch.where(seen, torch.where(x > 0, x / rep, x * rep), x)
            x = x - s["freq"][r].double() * count - s["pres"][r].double() * (count > 0)
            if s["ids"] is not None:
                x = x.index_add(0, s["ids"][r].long(), s["values"][r].double())
            x = x * s["scale"][r].double()
            if s["mask"] is not None:
                bits = np.unpackbits(s["mask"][r].cpu().numpy().view(np.uint8), bitorder="little")[: x.numel()]
                x[torch.from_numpy(bits == 0).cuda()] = -math.inf
            lse = torch.logsumexp(x, 0)
            ys.append(x if case["out"] == "logits" else (x - lse).exp() if case["out"] == "softmax" else x - lse)
            lses.append(lse)
        return {"y": torch.stack(ys), "lse": torch.stack(lses)}
    lens, news = _lengths(case)
    starts = np.concatenate([[0], np.cumsum(news)])
    T, hkv, d = s["tokens"], case["hkv"], case["d"]
    if case["op"] == "attention":
        if sum(n * k for n, k in zip(news, lens)) * case["hq"] > 100_000_000 or case["batch"] * hkv > 2000:
            return None
        G = case["hq"] // hkv
        o = torch.zeros(T, case["hq"], d, dtype=torch.float64, device="cuda")
        lse = torch.zeros(T, case["hq"], dtype=torch.float64, device="cuda")
        for b, (n, new) in enumerate(zip(lens, news)):
            for h in range(hkv):
                k, v = _sequence64(s, b, h)
                rows, heads = slice(starts[b], starts[b + 1]), slice(h * G, h * G + G)
                z = s["q"][rows, heads].double() @ k.T * (case["scale"] or 1 / math.sqrt(d))
                hide = torch.arange(n, device="cuda")[None] > (n - new + torch.arange(new, device="cuda"))[:, None]
                z.masked_fill_(hide[:, None], -math.inf)
                lse[rows, heads] = torch.logsumexp(z, -1)
                o[rows, heads] = torch.softmax(z, -1) @ v
        return {"o": o, "lse": lse}
    if T * hkv * d > 60_000_000 or case["batch"] * hkv > 2000:
        return None
    if case["op"] == "gather":
        k = torch.zeros(T, hkv, d, dtype=torch.float64, device="cuda")
        v = torch.zeros_like(k)
        for b in range(case["batch"]):
            for h in range(hkv):
                k[starts[b]: starts[b + 1], h], v[starts[b]: starts[b + 1], h] = _sequence64(s, b, h)
        return {"q": None, "k": k, "v": v}
    pos = torch.cat([torch.arange(n - new, n) for n, new in zip(lens, news)]).cuda()

    def turned(x):
        x, rot = x.double().clone(), case["rot"]
        if rot:
            cs = s["cos_sin"][pos].double()
            w = torch.complex(cs[:, : rot // 2], cs[:, rot // 2:])[:, None]
            i = torch.arange(rot // 2, device="cuda")
            a, b = (i, i + rot // 2) if case["pairs"] == "halves" else (2 * i, 2 * i + 1)
            t = torch.complex(x[..., a], x[..., b]) * w
            x[..., a], x[..., b] = t.real, t.imag
        return x

    def held(x):
        x = x.clamp(-65504, 65504).unflatten(-1, (-1, GROUP))
        lo, hi = x.min(-1, keepdim=True).values, x.max(-1, keepdim=True).values
        z, step = lo.half().double(), ((hi - lo) / 15).half().double()
        c = torch.where(step > 0, ((x - z) / step.clamp(min=2.0 ** -30)).round().clamp(0, 15), 0.0)
        return (c * step + z).flatten(-2)

    return {"q": turned(s["q"]), "k": held(turned(s["k"])), "v": held(s["v"].double())}
