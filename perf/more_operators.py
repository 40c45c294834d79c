"""Cases of the operators of a training step around its matrix products: the loss of the logits with its gradient, the
root-mean-square norm of rows, embedding lookup with its gradient, and the global gradient norm with clipping.

``run`` computes a case through the library (``own``) or in a plain form of elementary torch operations.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _size(name):
    return 4 if name == "fp32" else 2


def listed():
    loss = {"op": "loss", "smoothing": 0.0, "z": 0.0, "pad": 0, "weighted": False}
    norm = {"op": "norm", "residual": True, "out": "same", "group": 0, "offset": 0.0}
    back = {"op": "norm_grad", "sum_grad": True, "offset": 0.0}
    grads = {"op": "embedding_grad", "out": "fp32"}
    return [
        # fine-tuning on one short answer: a launch-bound call
        {**loss, "name": "loss_short", "rows": 16, "vocab": 32768, "dtype": "bf16"},
        # a pre-training micro-batch of long sequences over a large vocabulary
        {**loss, "name": "loss_batch", "rows": 8192, "vocab": 131072, "dtype": "bf16"},
        # logits in 32 bits, an odd vocabulary, smoothed labels, a penalty on the log-sum-exp, weights for the rows
        {**loss, "name": "loss_odd", "rows": 1023, "vocab": 50021, "dtype": "fp32", "smoothing": 0.1, "z": 1e-4, "weighted": True},
        # a decoding step of four users: latency
        {**norm, "name": "norm_decode", "rows": 4, "dim": 4096, "dtype": "bf16"},
        # a training or prompt batch on its way to an 8-bit product
        {**norm, "name": "norm_e4m3", "rows": 16384, "dim": 8192, "dtype": "bf16", "out": "e4m3", "group": 128},
        # the backward pass of a micro-batch, the residual's gradient added on the way
        {**back, "name": "norm_grad_batch", "rows": 16384, "dim": 4096, "dtype": "bf16"},
        # rows of an odd length in 16 bits
        {**back, "name": "norm_grad_odd", "rows": 777, "dim": 5003, "dtype": "fp16", "sum_grad": False, "offset": 1.0},
        # tokens of a micro-batch looked up, the rows scaled
        {"op": "embedding", "name": "embedding_batch", "tokens": 32768, "vocab": 131072, "dim": 4096, "dtype": "bf16", "skew": 3.0, "scale": 64.0},
        # their gradient into 32 bits: few tokens make up much of a text
        {**grads, "name": "embedding_grad_batch", "tokens": 32768, "vocab": 131072, "dim": 4096, "dtype": "bf16", "skew": 3.0, "scale": 64.0},
        # a small model's batch with padding, where sorting is what takes time
        {**grads, "name": "embedding_grad_short", "tokens": 1500, "vocab": 5003, "dim": 512, "dtype": "fp32", "skew": 6.0, "scale": 1.0},
        # gradients of a model of a billion weights in 16 bits, clipped into 32 bits for its optimiser
        {"op": "clip", "name": "clip_model", "layers": 16, "hidden": 2048, "dtype": "bf16", "out": "fp32", "clips": True, "scale": 0.125},
        # a small model's gradients, nothing to clip: latency
        {"op": "clip", "name": "clip_short", "layers": 3, "hidden": 64, "dtype": "fp32", "out": "place", "clips": False, "scale": 1.0},
    ]


def draw(rng):
    def spread(lo, hi):
        return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))

    op = rng.choice(["loss", "loss", "norm", "norm", "norm_grad", "embedding", "embedding_grad", "embedding_grad", "clip"])
    case = {"op": op, "dtype": rng.choice(["bf16", "fp16", "fp32"])}
    if op == "loss":
        vocab = spread(100, 262144)
        if rng.random() < 0.6:
            vocab = -(-vocab // 64) * 64
        return {**case, "vocab": vocab, "rows": spread(1, min(65536, 8192 * 131072 // (2 * vocab))), "pad": rng.choice([0, 0, 24, 7]),
                "smoothing": rng.choice([0.0, 0.0, 0.1]), "z": rng.choice([0.0, 1e-4]), "weighted": rng.random() < 0.5}
    if op in ("norm", "norm_grad"):
        dim = spread(64, 16384)
        if rng.random() < 0.7:
            dim = -(-dim // 128) * 128
        case |= {"dim": dim, "rows": spread(1, min(65536, 16384 * 8192 // dim)), "offset": rng.choice([0.0, 1.0])}
        if op == "norm_grad":
            return {**case, "sum_grad": rng.random() < 0.6}
        out = rng.choice(["same", "same", "e4m3"])
        return {**case, "residual": rng.random() < 0.6, "out": out, "group": 128 if out == "e4m3" and rng.random() < 0.6 else 0}
    if op == "clip":
        hidden = spread(16, 2048)
        out = rng.choice(["place", "same", "fp32"])
        return {**case, "hidden": hidden, "layers": rng.randint(1, 16), "out": out, "clips": out != "place", "scale": 1.0 if out == "place" else rng.choice([1.0, 0.125])}
    dim, vocab = spread(32, 8192), spread(100, 262144)
    if rng.random() < 0.7:
        dim = -(-dim // 64) * 64
    while dim * vocab > 131072 * 4096:
        vocab //= 2
    case |= {"dim": dim, "vocab": vocab, "tokens": spread(1, min(262144, 131072 * 4096 // dim)), "skew": rng.choice([1.0, 3.0, 6.0]), "scale": rng.choice([1.0, 64.0])}
    return case if op == "embedding" else {**case, "out": rng.choice(["fp32", "same"])}


# ---- inputs ---------------------------------------------------------------------------------------------------


def _sizes(case):
    """Elements of each gradient: layers of square and four-fold matrices, their norms' weights and a bias of odd length."""
    h = case["hidden"]
    return ([h * h] * 4 + [4 * h * h] * 3 + [h, h, 3 * h + 1]) * case["layers"]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt, op = TYPES[case["dtype"]], case["op"]

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)

    if op == "loss":
        M, N = case["rows"], case["vocab"]
        # logits as a product leaves them, a pitch apart where the vocabulary was padded for it
        x = normal(M, N + case["pad"]).mul_(2.5).to(dt)[:, :N]
        labels = torch.randint(0, N, (M,), device="cuda", generator=gen)
        ignored = torch.rand(M, device="cuda", generator=gen) < 0.06
        labels = torch.where(ignored, -100, labels)  # prompts and padding
        weights = torch.rand(M, device="cuda", generator=gen) if case["weighted"] else None
        # the mean over the rows; in fp16 times the loss scale that keeps such gradients in range
        return {"case": case, "x": x, "labels": labels, "weights": weights, "grad_scale": (4096.0 if case["dtype"] == "fp16" else 1.0) / M}
    if op in ("norm", "norm_grad"):
        M, N = case["rows"], case["dim"]
        s = {"case": case, "w": (1.0 - case["offset"] + 0.2 * normal(N)).to(dt)}
        amplitude = torch.exp(normal(M, 1))
        if op == "norm":
            s["x"] = (normal(M, N) * amplitude).to(dt)
            s["r"] = (2.0 * normal(M, N)).to(dt) if case["residual"] else None
            return s
        s["h"] = (normal(M, N) * amplitude).to(dt)
        s["dy"] = (0.01 * normal(M, N)).to(dt)
        s["dsum"] = (0.01 * normal(M, N)).to(dt) if case["sum_grad"] else None
        s["rstd"] = torch.cat([torch.rsqrt(h.float().square().mean(1) + EPS) for h in s["h"].split(4096)])  # kept from the forward pass
        return s
    if op in ("embedding", "embedding_grad"):
        T, V, D = case["tokens"], case["vocab"], case["dim"]
        u = torch.rand(T, device="cuda", generator=gen, dtype=torch.float64)
        tokens = (V * u ** case["skew"]).long().clamp(max=V - 1)
        tokens = (tokens * 7919) % V if V % 7919 else tokens  # frequent tokens anywhere in the vocabulary
        tokens = torch.where(torch.rand(T, device="cuda", generator=gen) < 0.03, -1, tokens)  # padding
        if op == "embedding":
            return {"case": case, "tokens": tokens, "table": normal(V, D).mul_(0.02).to(dt)}
        return {"case": case, "tokens": tokens, "dy": normal(T, D).mul_(0.01).to(dt)}
    sizes = _sizes(case)
    # every gradient a view of one buffer, as they lie in a bucket
    flat = torch.empty(sum(sizes), dtype=dt, device="cuda")
    grads = list(flat.split(sizes))
    for k, g in enumerate(grads):
        g.copy_(torch.randn(g.numel(), device="cuda", generator=gen).mul_(0.002 * (1 + k % 7)))
    norm = 0.01 * math.sqrt(sum(sizes)) * case["scale"]  # not far from theirs
    s = {"case": case, "flat": flat, "grads": grads, "max_norm": norm / 8 if case["clips"] else 8 * norm, "out": None, "out_flat": flat}
    if case["out"] != "place":
        s["out_flat"] = torch.zeros(sum(sizes), dtype=torch.float32 if case["out"] == "fp32" else dt, device="cuda")
        s["out"] = list(s["out_flat"].split(sizes))
    return s


# ---- plain forms ----------------------------------------------------------------------------------------------


def _plain_loss(s):
    case = s["case"]
    x, labels, eps, z = s["x"].float(), s["labels"], case["smoothing"], case["z"]
    N, live = x.shape[1], labels >= 0
    at = labels.clamp(min=0)[:, None]
    m = x.amax(1, keepdim=True)
    x = x - m
    e = torch.exp(x)
    d = e.sum(1, keepdim=True)
    log_d = torch.log(d)
    lse = m + log_d
    loss = log_d - (1 - eps) * x.gather(1, at) - (eps * x.mean(1, keepdim=True) if eps else 0.0) + z * lse * lse
    g = torch.where(live, s["grad_scale"] * (s["weights"] if s["weights"] is not None else torch.ones_like(m[:, 0])), 0.0)[:, None]
    e *= g * (1 + 2 * z * lse) / d
    if eps:
        e -= g * (eps / N)
    e.scatter_add_(1, at, -(1 - eps) * g)
    return {"loss": torch.where(live, loss[:, 0], 0.0), "lse": lse[:, 0], "grad": e.to(s["x"].dtype)}


def _plain_norm(s):
    case, dt = s["case"], s["x"].dtype
    h = s["x"] if s["r"] is None else (s["x"].float() + s["r"].float()).to(dt)
    x = h.float()
    rstd = torch.rsqrt((x * x).mean(1, keepdim=True) + EPS)
    y = x * rstd * (s["w"].float() + case["offset"])
    out = {"rstd": rstd[:, 0], "sum": None if s["r"] is None else h}
    if case["out"] == "same":
        return {**out, "y": y.to(dt), "scales": None}
    M, N = y.shape
    group = case["group"] or N
    groups = -(-N // group)
    y = torch.nn.functional.pad(y, (0, groups * group - N)).reshape(M, groups, group)
    scales = (y.abs().amax(2) / 448.0).clamp(min=2.0 ** -126)
    y = (y / scales[:, :, None]).clamp(-448.0, 448.0).reshape(M, -1)[:, :N]
    return {**out, "y": y.to(torch.float8_e4m3fn), "scales": scales}


def _plain_norm_grad(s):
    h, dy, rstd = s["h"].float(), s["dy"].float(), s["rstd"][:, None]
    xhat = h * rstd
    g = dy * (s["w"].float() + s["case"]["offset"])
    dx = rstd * (g - xhat * (g * xhat).mean(1, keepdim=True))
    if s["dsum"] is not None:
        dx = dx + s["dsum"].float()
    return {"dx": dx.to(s["h"].dtype), "dweight": (dy * xhat).sum(0)}


def _plain_embedding(s):
    y = s["table"][s["tokens"].clamp(min=0)].float() * s["case"]["scale"]
    return torch.where((s["tokens"] >= 0)[:, None], y, 0.0).to(s["table"].dtype)


def _plain_embedding_grad(s):
    case = s["case"]
    dy = torch.where((s["tokens"] >= 0)[:, None], s["dy"].float() * case["scale"], 0.0)
    grad = torch.zeros(case["vocab"], case["dim"], device="cuda").index_add_(0, s["tokens"].clamp(min=0), dy)
    return grad if case["out"] == "fp32" else grad.to(s["dy"].dtype)


def _plain_clip(s):
    flat = torch.cat([g.reshape(-1) for g in s["grads"]]).float() * s["case"]["scale"]
    norm = torch.sqrt(flat.square().sum(dtype=torch.float64))
    flat = flat * torch.clamp(s["max_norm"] / norm, max=1.0).float()
    return {"norm": norm.float(), "grads": flat.to(s["out_flat"].dtype)}


def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if own:
        import row_wise_online_gb300 as rwo

        if op == "loss":
            lse = torch.empty(case["rows"], device="cuda")
            loss, grad = rwo.cross_entropy_rows_grad(s["x"], s["labels"], lse_out=lse, upstream=s["weights"], grad_scale=s["grad_scale"],
                                                     label_smoothing=case["smoothing"], z_loss=case["z"])
            return {"loss": loss, "lse": lse, "grad": grad}
        if op == "norm":
            rstd = torch.empty(case["rows"], device="cuda")
            a = {"residual": s["r"], "rstd_out": rstd, "eps": EPS, "offset": case["offset"]}
            if case["out"] == "same":
                y, h = rwo.rms_norm_rows(s["x"], s["w"], **a)
                return {"rstd": rstd, "sum": None if s["r"] is None else h, "y": y, "scales": None}
            y, scales, h = rwo.rms_norm_rows_e4m3(s["x"], s["w"], group=case["group"], **a)
            return {"rstd": rstd, "sum": None if s["r"] is None else h, "y": y, "scales": scales}
        if op == "norm_grad":
            dx, dw = rwo.rms_norm_rows_backward(s["dy"], s["h"], s["rstd"], s["w"], offset=case["offset"], sum_grad=s["dsum"])
            return {"dx": dx, "dweight": dw}
        if op == "embedding":
            return rwo.embedding_rows(s["table"], s["tokens"], scale=case["scale"])
        if op == "embedding_grad":
            dt = torch.float32 if case["out"] == "fp32" else s["dy"].dtype
            return rwo.embedding_rows_backward(s["dy"], s["tokens"], case["vocab"], scale=case["scale"], dtype=dt)
        norm = rwo.clip_grad_norm(s["grads"], s["max_norm"], out=s["out"], scale=case["scale"])
        return {"norm": norm, "grads": s["out_flat"]}
    plain = {"loss": _plain_loss, "norm": _plain_norm, "norm_grad": _plain_norm_grad, "embedding": _plain_embedding,
             "embedding_grad": _plain_embedding_grad, "clip": _plain_clip}
    return plain[op](s)


def _touched(case):
    """Rows of the table that the case's tokens are expected to name."""
    edges = (np.arange(case["vocab"] + 1) / case["vocab"]) ** (1 / case["skew"])
    return float(np.sum(-np.expm1(0.97 * case["tokens"] * np.log1p(-np.minimum(np.diff(edges), 1 - 1e-12)))))


def work(case):
    e, op = _size(case["dtype"]), case["op"]
    if op == "loss":
        M, N = case["rows"], case["vocab"]
        return {"bytes": M * (2 * N * e + 16 + (4 if case["weighted"] else 0)), "flops": 8 * M * N}
    if op == "norm":
        M, N = case["rows"], case["dim"]
        out = e if case["out"] == "same" else 1 + 4 / (case["group"] or N)
        return {"bytes": M * N * (e + (2 * e if case["residual"] else 0) + out) + N * e + 4 * M, "flops": 8 * M * N}
    if op == "norm_grad":
        M, N = case["rows"], case["dim"]
        return {"bytes": M * N * (3 + case["sum_grad"]) * e + N * (e + 4) + 4 * M, "flops": 12 * M * N}
    if op == "embedding":
        T, D = case["tokens"], case["dim"]
        return {"bytes": T * (D * e + 8) + _touched(case) * D * e, "flops": T * D}
    if op == "embedding_grad":
        T, D = case["tokens"], case["dim"]
        return {"bytes": T * (D * e + 8) + case["vocab"] * D * (4 if case["out"] == "fp32" else e), "flops": 2 * T * D}
    n = sum(_sizes(case))
    out = 0 if case["out"] == "place" and not case["clips"] else 4 if case["out"] == "fp32" else e
    return {"bytes": n * (e + out), "flops": 4 * n}


# ---- 64 bits --------------------------------------------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "loss":
        N, eps, z = case["vocab"], case["smoothing"], case["z"]
        grad = torch.empty(s["x"].shape, dtype=torch.float64, device="cuda")
        losses, lses, step = [], [], max(1, (1 << 27) // N)
        for r in range(0, case["rows"], step):
            x, labels = s["x"][r: r + step].double(), s["labels"][r: r + step]
            lse = torch.logsumexp(x, 1)
            # smoothed labels as a distribution of their own
            target = torch.full_like(x, eps / N)
            target[torch.arange(len(labels), device="cuda"), labels.clamp(min=0)] += 1 - eps
            live = (labels >= 0).double()
            losses.append(live * ((target * (lse[:, None] - x)).sum(1) + z * lse ** 2))
            g = live * s["grad_scale"]
            if s["weights"] is not None:
                g = g * s["weights"][r: r + step].double()
            grad[r: r + step] = g[:, None] * ((x - lse[:, None]).exp() * (1 + 2 * z * lse)[:, None] - target)
            lses.append(lse)
        return {"loss": torch.cat(losses), "lse": torch.cat(lses), "grad": grad}
    if op == "norm":
        x = s["x"].double()
        total = x if s["r"] is None else x + s["r"].double()
        h = total.to(s["x"].dtype).double()  # the norm is of the sum as it is kept
        rstd = (h.pow(2).sum(1) / case["dim"] + EPS) ** -0.5
        y = torch.einsum("mn,m,n->mn", h, rstd, s["w"].double() + case["offset"])
        out = {"rstd": rstd, "sum": None if s["r"] is None else total, "y": y, "scales": None}
        if case["out"] == "e4m3":
            parts = y.split(case["group"] or case["dim"], 1)
            tops = [p.abs().max(1, keepdim=True).values / 448 for p in parts]
            out |= {"y": torch.cat([p / t for p, t in zip(parts, tops)], 1), "scales": torch.cat(tops, 1)}
        return out
    if op == "norm_grad":
        N = case["dim"]
        dw, dxs = torch.zeros(N, dtype=torch.float64, device="cuda"), []
        w = s["w"].double() + case["offset"]
        for r in range(0, case["rows"], 2048):
            h, dy, rstd = (s[k][r: r + 2048].double() for k in ("h", "dy", "rstd"))
            g = dy * w
            dot = torch.einsum("mn,mn->m", g, h)
            dx = g * rstd[:, None] - h * (rstd ** 3 * dot / N)[:, None]
            dxs.append(dx if s["dsum"] is None else dx + s["dsum"][r: r + 2048].double())
            dw += torch.einsum("mn,mn,m->n", dy, h, rstd)
        return {"dx": torch.cat(dxs), "dweight": dw}
    if op == "embedding":
        y = s["table"].double().index_select(0, s["tokens"].clamp(min=0)).mul_(case["scale"])
        return y.masked_fill_((s["tokens"] < 0)[:, None], 0.0)
    if op == "embedding_grad":
        kept = s["tokens"] >= 0
        grad = torch.zeros(case["vocab"], case["dim"], dtype=torch.float64, device="cuda")
        return grad.index_put_((s["tokens"][kept],), s["dy"][kept].double(), accumulate=True).mul_(case["scale"])
    squares = sum(float(torch.dot(p, p)) for g in s["grads"] for p in (g.double() for g in g.split(1 << 27)))
    norm = abs(case["scale"]) * math.sqrt(squares)
    factor = case["scale"] * min(1.0, s["max_norm"] / norm)
    return {"norm": norm, "grads": torch.cat([g.double() * factor for g in s["grads"]])}
