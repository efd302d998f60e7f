"""The vocabulary losses as measured cases: what a training, scoring or distillation program asks of them.

Two operators over the output projection of a language model, z = scale * H W^T
with hidden states H (tokens x width) and a head W (vocabulary x width):

* ``xent``     softmax cross entropy against a label per token;
* ``distill``  the divergence from a teacher that is known by its top logits.

Each runs forward (loss and log-sum-exp per token) or as a training step, which
also returns the gradients of H and W. ``run`` computes them in elementary torch
operations, or with ``own`` set through the library's entry points.
"""

import math

import torch

own = False
_handle = None


def _sgemm():
    """The library handle that a program keeps (its workspace with it)."""
    global _handle
    if _handle is None:
        import dense_fp32_gemm_04_gb300 as sg

        _handle = sg.Sgemm()
    return _handle


def _case(name, op, train, tokens, vocab, width, dtype, k=1, temperature=1.0, masked=0.1, pad=0):
    return {"name": name, "op": op, "train": train, "tokens": tokens, "vocab": vocab, "width": width, "dtype": dtype,
            "k": k, "temperature": temperature, "masked": masked, "pad": pad}


def listed():
    return [
        # the probability of one token under a small model: latency, and one reading of the head
        _case("xent score 1 token", "xent", False, 1, 32768, 2048, "bfloat16", masked=0.0),
        # log-probabilities of a short answer under a large vocabulary: the head's bytes are the cost
        _case("xent score 60 tokens", "xent", False, 60, 131072, 4096, "bfloat16", masked=0.0),
        # the same in single precision, for a handful of tokens
        _case("xent score 5 tokens f32", "xent", False, 5, 50021, 2048, "float32", masked=0.0),
        # perplexity over a long document
        _case("xent evaluate 8192", "xent", False, 8192, 131072, 4096, "bfloat16", masked=0.02),
        # a fine-tuning micro-batch of a small model; half of its tokens are the prompt and masked
        _case("xent train 256", "xent", True, 256, 32768, 1024, "bfloat16", masked=0.5),
        # a pretraining micro-batch of a large model
        _case("xent train 4096", "xent", True, 4096, 131072, 4096, "bfloat16", masked=0.0),
        # ragged in every size, rows of the operands at odd strides
        _case("xent train ragged", "xent", True, 2047, 50021, 1531, "bfloat16", masked=0.3, pad=2),
        # a training step in single precision
        _case("xent train 2048 f32", "xent", True, 2048, 32768, 2048, "float32", masked=0.1),
        # divergence from a teacher on held-out text, its 32 best logits stored
        _case("distill evaluate 1024", "distill", False, 1024, 65536, 2048, "bfloat16", k=32, temperature=2.0, masked=0.05),
        # distillation of a small student, short sequences
        _case("distill train 512", "distill", True, 512, 32768, 1024, "bfloat16", k=16, temperature=1.0, masked=0.1),
        # distillation with a large vocabulary and many logits per token
        _case("distill train 4096", "distill", True, 4096, 131072, 2048, "bfloat16", k=64, temperature=2.0, masked=0.0),
        # single precision, ragged, some lists of the teacher short or empty
        _case("distill train ragged f32", "distill", True, 1000, 32003, 1001, "float32", k=10, temperature=4.0, masked=0.2, pad=3),
    ]


_MOST = 6 * 4096 * 131072 * 4096  # operations of the largest listed case


def _log_uniform(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    train = rng.random() < 0.6
    dtype = "float32" if rng.random() < 0.3 else "bfloat16"
    op = rng.choice(["xent", "distill"])
    # a training step has a micro-batch of tokens, a scoring call from one token on;
    # single precision is for the smaller models
    wide = dtype == "bfloat16"
    tokens = _log_uniform(rng, 200 if train else 1, 8192 if wide else 3000)
    vocab = _log_uniform(rng, 8000, 140000 if wide else 66000)
    width = _log_uniform(rng, 500, 4096 if wide else 2100)
    if rng.random() < 0.5:  # sizes as models choose them; odd ones otherwise
        vocab, width = (vocab + 63) // 64 * 64, (width + 63) // 64 * 64
    most = _MOST if wide else _MOST // 8
    tokens = max(1, min(tokens, most // ((6 if train else 2) * vocab * width)))
    case = _case("", op, train, tokens, vocab, width, dtype, masked=rng.choice([0.0, 0.1, 0.5]), pad=rng.choice([0, 0, 1, 8]))
    if op == "distill":
        case["k"] = _log_uniform(rng, 1, 100)
        case["temperature"] = rng.choice([1.0, 2.0, 4.0])
    del case["name"]
    return case


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bfloat16" else torch.float32


def _inputs(case, seed):
    """Hidden states as a final norm leaves them, a head whose logits have a spread of about two, targets that the
    hidden states point at more or less, and a gradient of the loss that averages over the tokens with weights."""
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    T, V, D, k, pad = case["tokens"], case["vocab"], case["width"], case["k"], case["pad"]
    W = torch.empty(V, D + pad, device=dev, dtype=_dtype(case))[:, :D]
    W.copy_(torch.randn(V, D, device=dev, generator=gen) * (2.0 / math.sqrt(D)))
    hidden = torch.randn(T, D, device=dev, generator=gen)
    start = torch.randint(V, (T, 1), device=dev, generator=gen)
    hidden += W[start[:, 0]].float() * (3.0 * torch.rand(T, 1, device=dev, generator=gen))
    H = torch.empty(T, D + pad, device=dev, dtype=_dtype(case))[:, :D]
    H.copy_(hidden)
    out = torch.rand(T, device=dev, generator=gen) < case["masked"]
    dloss = (0.5 + torch.rand(T, device=dev, generator=gen)) / T
    if case["op"] == "xent":
        return {"H": H, "W": W, "labels": torch.where(out, -100, start[:, 0]), "dloss": dloss}
    # distinct ids for each token, logits from the largest down, -1 past the end of a short or empty list
    stride = torch.randint(1, max(2, V // k), (T, 1), device=dev, generator=gen)
    at = torch.arange(k, device=dev)
    ids = (start + at * stride) % V
    steps = torch.rand(T, k, device=dev, generator=gen).clamp_min(1e-6).log().neg()
    logits = 12.0 - steps.cumsum(1) * (8.0 / k)
    length = torch.randint(1, k + 1, (T, 1), device=dev, generator=gen)
    length = torch.where(torch.rand(T, 1, device=dev, generator=gen) < 0.5, k, length)
    length = torch.where(out[:, None], 0, length) if case["masked"] else torch.full_like(length, k)
    return {"H": H, "W": W, "ids": torch.where(at < length, ids, -1), "logits": logits, "dloss": dloss}


def prepare(case, seed):
    return {"case": dict(case), **_inputs(case, seed)}


def _plain(case, x):
    H, W = x["H"].float(), x["W"].float()
    scale = 1.0 / case["temperature"]
    z = (H @ W.T) * scale
    top = z.max(1, keepdim=True).values
    lse = top[:, 0] + (z - top).exp().sum(1).log()
    if case["op"] == "xent":
        labels = x["labels"]
        used = (labels >= 0).float()
        ids = labels.clamp_min(0)[:, None]
        q = used[:, None]
        loss = (lse - z.gather(1, ids)[:, 0]) * used
        weight = scale
    else:
        some = x["ids"] >= 0
        ids = x["ids"].clamp_min(0)
        t = torch.where(some, x["logits"] * scale, -math.inf)
        best = t.max(1, keepdim=True).values
        t = t - torch.where(best > -math.inf, best, 0.0)
        e = t.exp()
        total = e.sum(1, keepdim=True)
        used = (total[:, 0] > 0).float()
        total = torch.where(total > 0, total, 1.0)
        q = e / total
        logq = torch.where(q > 0, t - total.log(), 0.0)
        squared = case["temperature"] ** 2
        loss = squared * ((q * (logq - z.gather(1, ids))).sum(1) + lse * used)
        weight = squared * scale
    if not case["train"]:
        return {"loss": loss, "lse": lse}
    g = (x["dloss"] * weight * used)[:, None]
    dz = (z - lse[:, None]).exp() * g
    dz.scatter_add_(1, ids, -g * q)
    return {"loss": loss, "lse": lse, "dH": (dz @ W).to(x["H"].dtype), "dW": (dz.T @ H).to(x["W"].dtype)}


def _own(case, x):
    h, H, W = _sgemm(), x["H"], x["W"]
    if case["op"] == "xent":
        scale = 1.0 / case["temperature"]
        loss, lse = h.xent(H, W, x["labels"], scale=scale)
        if not case["train"]:
            return {"loss": loss, "lse": lse}
        dH, dW = h.xent_grad(H, W, x["labels"], lse, x["dloss"], scale=scale)
    else:
        loss, lse = h.distill(H, W, x["ids"], x["logits"], temperature=case["temperature"])
        if not case["train"]:
            return {"loss": loss, "lse": lse}
        dH, dW = h.distill_grad(H, W, x["ids"], x["logits"], lse, x["dloss"], temperature=case["temperature"])
    return {"loss": loss, "lse": lse, "dH": dH, "dW": dW}


def run(state):
    return _own(state["case"], state) if own else _plain(state["case"], state)


def work(case):
    T, V, D, k = case["tokens"], case["vocab"], case["width"], case["k"]
    size = 2 if case["dtype"] == "bfloat16" else 4
    operands = (T + V) * D * size
    targets = T * (8 if case["op"] == "xent" else 12 * k)
    if not case["train"]:
        return {"bytes": operands + targets + 8 * T, "flops": 2 * T * V * D}
    return {"bytes": 2 * operands + targets + 12 * T, "flops": 6 * T * V * D}


def exact(case, seed):
    """The same from the definition in 64 bits: probabilities token block by token block, each loss as the sum over the
    targets of q (log q - log p), each gradient as that of log p."""
    T, V, D, k = case["tokens"], case["vocab"], case["width"], case["k"]
    if (6 if case["train"] else 2) * T * V * D > 15e12:
        return None
    x = _inputs(case, seed)
    W = x["W"].double()
    tau = float(case["temperature"])
    if case["op"] == "xent":
        ids, logits, factor = x["labels"][:, None], torch.zeros(T, 1, device="cuda", dtype=torch.float64), 1.0
    else:
        ids, logits, factor = x["ids"], x["logits"].double(), tau * tau
    losses, lses, dHs = [], [], []
    dW = torch.zeros(V, D, device="cuda", dtype=torch.float64) if case["train"] else None
    rows = max(1, min(T, (1 << 28) // V))
    for r in range(0, T, rows):
        h = x["H"][r:r + rows].double()
        logp = h @ W.T / tau
        norm = torch.logsumexp(logp, 1, keepdim=True)
        logp -= norm
        real = ids[r:r + rows] >= 0
        at = torch.where(real, ids[r:r + rows], 0)
        t = (logits[r:r + rows] / tau).masked_fill(~real, -math.inf)
        full = real.any(1, keepdim=True)
        q = torch.where(full, torch.softmax(t.masked_fill(~full, 0.0), 1), 0.0)
        term = torch.special.xlogy(q, q) - q * logp.gather(1, at)
        losses.append(factor * term.sum(1))
        lses.append(norm[:, 0])
        if case["train"]:
            g = (factor / tau) * x["dloss"][r:r + rows].double()[:, None]
            dz = logp.exp_().mul_(g * full)
            dz.scatter_add_(1, at, -(g * q))
            dHs.append(dz @ W)
            dW.addmm_(dz.T, h)
    out = {"loss": torch.cat(losses), "lse": torch.cat(lses)}
    if case["train"]:
        out.update(dH=torch.cat(dHs), dW=dW)
    return out
