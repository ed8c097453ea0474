"""The operators of a model's output head, as cases to measure: products with a 4-bit head or
projection, the distillation loss against a teacher's top logits, and the cross entropy of a
dense head whose logits are never kept.

Each case runs in a plain form (elementary torch operations in 32 bits) or, with ``own``,
through this package's calls.  ``exact`` gives the same outputs from the definitions in 64 bits.
"""
import math

import torch

own = False

# Vocabulary and hidden sizes: 4096 and 8192 are the hidden sizes of the package's decoder-block
# workloads, 28672 their MLP width, 512 x 512 the single small layer, 1024 and 4096 their
# calibration and prefill batches; 32000 to 128000 are usual vocabulary sizes (32001: one added
# token, 50257: a vocabulary that is no multiple of anything, padded to rows of 50304 logits).


def listed():
    return [
        # the small layer kept at 4 bits, one token: the cost of a call
        {"name": "q4_small_b1", "op": "q4", "m": 512, "n": 512, "group": 128, "batch": 1, "zeros": False},
        # an attention projection kept at 4 bits beside factorised ones, a few sequences
        {"name": "q4_proj_b3", "op": "q4", "m": 4096, "n": 4096, "group": 32, "batch": 3, "zeros": True},
        # the head of a decoder with one added token, one sequence: the logits of every step
        {"name": "q4_head_b1", "op": "q4", "m": 32001, "n": 4096, "group": 64, "batch": 1, "zeros": True},
        # an MLP projection of the large block, a full decode batch
        {"name": "q4_mlp_b8", "op": "q4", "m": 28672, "n": 8192, "group": 128, "batch": 8, "zeros": False},
        # distillation: the loss of a handful of tokens (validation of one short answer)
        {"name": "distill_fwd_few", "op": "distill_fwd", "tokens": 8, "vocab": 32000, "pitch": 32000, "k": 16,
         "rest": False, "temperature": 1.0, "logits": "f32", "grad": "none"},
        # ragged rows: a factorised head padded to a multiple of 128, the teacher's remaining mass kept
        {"name": "distill_fwd_ragged", "op": "distill_fwd", "tokens": 777, "vocab": 50257, "pitch": 50304, "k": 50,
         "rest": True, "temperature": 2.0, "logits": "f32", "grad": "none"},
        # one refinement step: fp32 logits of a factorised head in, the bf16 output gradient out
        {"name": "distill_bwd_step", "op": "distill_bwd", "tokens": 1024, "vocab": 32000, "pitch": 32000, "k": 64,
         "rest": False, "temperature": 1.0, "logits": "f32", "grad": "bf16"},
        # a large calibration batch over a large vocabulary, bf16 logits of a dense head
        {"name": "distill_bwd_large", "op": "distill_bwd", "tokens": 4096, "vocab": 128000, "pitch": 128000, "k": 128,
         "rest": True, "temperature": 2.0, "logits": "bf16", "grad": "bf16"},
        # cross entropy: the score of a few tokens (one pass over the head's weights)
        {"name": "ce_fwd_few", "op": "ce_fwd", "tokens": 8, "vocab": 32000, "d": 4096},
        # the perplexity of a calibration batch
        {"name": "ce_fwd_large", "op": "ce_fwd", "tokens": 4096, "vocab": 32000, "d": 4096},
        # gradients of a ragged batch, padding tokens among them, over a ragged vocabulary
        {"name": "ce_bwd_ragged", "op": "ce_bwd", "tokens": 1000, "vocab": 50257, "d": 2048},
        # gradients of a calibration batch
        {"name": "ce_bwd_large", "op": "ce_bwd", "tokens": 4096, "vocab": 32000, "d": 4096},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["q4", "distill_fwd", "distill_bwd", "ce_fwd", "ce_bwd"])
    if op == "q4":
        m, n = _log(rng, 64, 50000), 128 * _log(rng, 1, 64)
        return {"op": op, "m": m, "n": n, "group": rng.choice([32, 64, 128]), "batch": rng.randint(1, 16),
                "zeros": rng.random() < 0.5}
    if op.startswith("distill"):
        vocab = _log(rng, 500, 128000)
        tokens = min(_log(rng, 1, 4096), 4096 * 64000 // vocab)
        return {"op": op, "tokens": tokens, "vocab": vocab, "pitch": vocab + rng.choice([0, 0, -vocab % 128]),
                "k": min(vocab, _log(rng, 1, 256)), "rest": rng.random() < 0.5, "temperature": rng.choice([1.0, 2.0, 4.0]),
                "logits": rng.choice(["f32", "bf16"]),
                "grad": "none" if op == "distill_fwd" else rng.choice(["f32", "bf16"])}
    vocab, d = _log(rng, 500, 60000), 8 * _log(rng, 16, 512)
    tokens = min(_log(rng, 1, 4096), max(1, 4096 * 32000 * 4096 // (vocab * d)))
    return {"op": op, "tokens": tokens, "vocab": vocab, "d": d}


_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def _inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 1000003 + 17)

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=g)

    def uniform(*shape):
        return torch.rand(*shape, device="cuda", generator=g)

    s = {}
    if case["op"] == "q4":
        m, n, group, batch = case["m"], case["n"], case["group"], case["batch"]
        codes = torch.randint(0, 256, (m, n // 2), device="cuda", generator=g, dtype=torch.uint8)
        s["packed"] = codes.view(torch.int32)  # code c of a row in bits 4 (c % 8) of its word c / 8
        s["scales"] = ((uniform(m, n // group) + 0.5) * 0.02).half()
        if case["zeros"]:
            s["zeros"] = (uniform(m, n // group) * 6 + 5).half()
        x = normal(batch, n)
        x[:, 5::1024] *= 100.0  # a few large channels, as decoder activations have
        s["x"] = x.bfloat16()
        return s
    if case["op"].startswith("distill"):
        tokens, vocab, k = case["tokens"], case["vocab"], case["k"]
        full = torch.zeros(tokens, case["pitch"], device="cuda")
        full[:, :vocab] = normal(tokens, vocab) * 2.5
        s["logits"] = full.to(_TYPES[case["logits"]])
        teacher = full[:, :vocab] + normal(tokens, vocab)
        top, ids = torch.topk(teacher, k, dim=1)
        if case["rest"]:
            s["teacher_lse"] = torch.logsumexp(teacher / case["temperature"], dim=1)
        # some positions have fewer than k entries, some none (padding): their ids are -1
        kept = torch.where(uniform(tokens) < 0.1, (uniform(tokens) * k).int(), torch.full((tokens,), k, device="cuda").int())
        gone = torch.arange(k, device="cuda")[None, :] >= kept[:, None]
        s["ids"] = torch.where(gone, torch.full_like(ids, -1), ids).int().contiguous()
        s["teacher"] = top.float().contiguous()
        s["dloss"] = (uniform(tokens) + 0.5) / tokens
        return s
    tokens, vocab, d = case["tokens"], case["vocab"], case["d"]
    s["h"] = normal(tokens, d).bfloat16()
    s["W"] = (normal(vocab, d) * (1.6 / math.sqrt(d))).bfloat16()
    labels = torch.randint(0, vocab, (tokens,), device="cuda", generator=g, dtype=torch.int32)
    if tokens > 1:
        labels[uniform(tokens) < 0.1] = -100  # positions that do not count
    s["labels"] = labels
    if case["op"] == "ce_bwd":
        s["dloss"] = (uniform(tokens) + 0.5) / tokens
        s["lse"] = torch.logsumexp(s["h"].float() @ s["W"].float().T, dim=1)  # what the forward left
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    return s


def run(s):
    c = s["case"]
    if own:
        from binary_rank_linear_02_b200 import nq

        if c["op"] == "q4":
            return {"y": nq.q4_linear_fwd(s["x"], s["packed"], s["scales"], c["m"], c["n"], c["group"], zeros=s.get("zeros"))}
        if c["op"] == "distill_fwd":
            return {"loss": nq.distill_topk_fwd(s["logits"], s["ids"], s["teacher"], c["vocab"],
                                                temperature=c["temperature"], teacher_lse=s.get("teacher_lse"))}
        if c["op"] == "distill_bwd":
            dlogits, loss = nq.distill_topk_bwd(s["logits"], s["ids"], s["teacher"], c["vocab"], s["dloss"],
                                                temperature=c["temperature"], teacher_lse=s.get("teacher_lse"),
                                                dtype=_TYPES[c["grad"]])
            return {"dlogits": dlogits[:, :c["vocab"]], "loss": loss}
        if c["op"] == "ce_fwd":
            loss, lse = nq.linear_cross_entropy_fwd(s["h"], s["W"], s["labels"])
            return {"loss": loss, "lse": lse}
        dh, dW = nq.linear_cross_entropy_bwd(s["h"], s["W"], s["labels"], s["lse"], s["dloss"])
        return {"dh": dh, "dW": dW}
    if c["op"] == "q4":
        return {"y": _plain_q4(s, c)}
    if c["op"].startswith("distill"):
        return _plain_distill(s, c)
    if c["op"] == "ce_fwd":
        return _plain_ce_fwd(s)
    return _plain_ce_bwd(s)


def _plain_q4(s, c):
    shifts = torch.arange(0, 32, 4, device="cuda", dtype=torch.int32)
    codes = ((s["packed"][:, :, None] >> shifts) & 15).reshape(c["m"], -1, c["group"]).float()
    zeros = s["zeros"].float()[:, :, None] if "zeros" in s else 8.0
    w = ((codes - zeros) * s["scales"].float()[:, :, None]).reshape(c["m"], c["n"])
    return s["x"].float() @ w.T


def _plain_distill(s, c):
    # Over the classes in 32 bits; the few values of the teacher's list, the logarithms and the
    # differences between them in 64 (a small loss is left of terms that nearly cancel).
    vocab, t = c["vocab"], c["temperature"]
    z = s["logits"][:, :vocab].float()
    valid = s["ids"] >= 0
    at = s["ids"].long().clamp_min(0)
    u = torch.where(valid, s["teacher"].double() / t, -math.inf)
    if "teacher_lse" in s:
        q = torch.exp(u - s["teacher_lse"].double()[:, None])
        rest = (1.0 - q.sum(1)).clamp_min(0.0)
    else:
        e = torch.exp(u - u.amax(1, keepdim=True).clamp_min(-1e30))
        q = e / e.sum(1, keepdim=True).clamp_min(1e-30)
        rest = torch.zeros_like(q[:, 0])
    peak = z.amax(1, keepdim=True)
    e = torch.exp((z - peak) / t)
    norm = e.sum(1, keepdim=True, dtype=torch.float64)
    logp = (z.gather(1, at) - peak).double() / t - torch.log(norm)
    loss = torch.where(q > 0, q * (torch.log(q.clamp_min(1e-300)) - logp), 0.0).sum(1)
    # the classes outside the teacher's list, for the rest of its mass
    outside = torch.ones_like(e, dtype=torch.int8).scatter_add_(1, at, -valid.to(torch.int8)) > 0
    prest = (e * outside).sum(1, dtype=torch.float64) / norm[:, 0]
    rest = torch.where(prest > 0, rest, 0.0)  # the list may name every class
    loss = loss + torch.where(rest > 0, rest * (torch.log(rest.clamp_min(1e-300)) - torch.log(prest.clamp_min(1e-300))), 0.0)
    loss = (loss * (t * t)).float()
    if c["op"] == "distill_fwd":
        return {"loss": loss}
    total = (q.sum(1) + rest).float()[:, None]
    share = (rest / prest.clamp_min(1e-300)).float()[:, None]
    dz = e / norm.float() * (total - outside * share)
    dz.scatter_add_(1, at, -q.float())
    dz = dz * (t * s["dloss"])[:, None]
    return {"dlogits": dz.to(_TYPES[c["grad"]]), "loss": loss}


def _plain_ce_fwd(s):
    z = s["h"].float() @ s["W"].float().T
    peak = z.amax(1)
    lse = peak + torch.log(torch.exp(z - peak[:, None]).sum(1))
    counted = s["labels"] >= 0
    picked = z.gather(1, s["labels"].long().clamp_min(0)[:, None])[:, 0]
    return {"loss": torch.where(counted, lse - picked, torch.zeros_like(lse)), "lse": lse}


def _plain_ce_bwd(s):
    h, w = s["h"].float(), s["W"].float()
    dz = torch.exp(h @ w.T - s["lse"][:, None])
    counted = s["labels"] >= 0
    dz.scatter_add_(1, s["labels"].long().clamp_min(0)[:, None], -torch.ones_like(dz[:, :1]))
    dz = dz * torch.where(counted, s["dloss"], torch.zeros_like(s["dloss"]))[:, None]
    return {"dh": (dz @ w).bfloat16(), "dW": (dz.T @ h).bfloat16()}


def work(case):
    if case["op"] == "q4":
        m, n, batch = case["m"], case["n"], case["batch"]
        per_group = 4 if case["zeros"] else 2
        return {"bytes": m * n // 2 + m * (n // case["group"]) * per_group + batch * (2 * n + 4 * m),
                "flops": 2 * m * n * batch}
    if case["op"].startswith("distill"):
        tokens, vocab, k = case["tokens"], case["vocab"], case["k"]
        size = {"f32": 4, "bf16": 2, "none": 0}
        moved = tokens * vocab * (size[case["logits"]] + size[case["grad"]]) + tokens * (8 * k + 12)
        return {"bytes": moved, "flops": tokens * vocab * (4 if case["op"] == "distill_fwd" else 8)}
    tokens, vocab, d = case["tokens"], case["vocab"], case["d"]
    if case["op"] == "ce_fwd":
        return {"bytes": 2 * d * (tokens + vocab) + 12 * tokens, "flops": 2 * tokens * vocab * d}
    # the logits once more, then a product for each gradient
    return {"bytes": 4 * d * (tokens + vocab) + 12 * tokens, "flops": 6 * tokens * vocab * d}


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "q4":
        return {"y": _exact_q4(s, case)}
    if case["op"].startswith("distill"):
        return _exact_distill(s, case)
    h, w = s["h"].double(), s["W"].double()
    z = h @ w.T
    logp = torch.log_softmax(z, dim=1)
    rows = torch.arange(h.shape[0], device="cuda")
    counted = s["labels"] >= 0
    picked = torch.where(counted, s["labels"], torch.zeros_like(s["labels"])).long()
    if case["op"] == "ce_fwd":
        return {"loss": -logp[rows, picked] * counted, "lse": z[:, 0] - logp[:, 0]}
    dz = logp.exp_()
    dz[rows, picked] -= 1.0
    dz *= (s["dloss"].double() * counted)[:, None]
    return {"dh": dz @ w, "dW": dz.T @ h}


def _exact_q4(s, case):
    m, n, group = case["m"], case["n"], case["group"]
    nibbles = s["packed"].view(torch.uint8).reshape(m, n // 2)
    w = torch.empty(m, n, dtype=torch.float64, device="cuda")
    w[:, 0::2] = (nibbles & 15).double()
    w[:, 1::2] = (nibbles >> 4).double()
    zero = s["zeros"].double().repeat_interleave(group, dim=1) if "zeros" in s else 8.0
    return s["x"].double() @ ((w - zero) * s["scales"].double().repeat_interleave(group, dim=1)).T


def _exact_distill(s, case):
    vocab, t = case["vocab"], case["temperature"]
    logp = torch.log_softmax(s["logits"][:, :vocab].double() / t, dim=1)
    tokens = logp.shape[0]
    valid = s["ids"] >= 0
    u = (s["teacher"].double() / t).masked_fill(~valid, -math.inf)
    named = valid.any(1)
    if "teacher_lse" in s:
        logq = u - s["teacher_lse"].double()[:, None]
    else:
        logq = u - torch.logsumexp(u.masked_fill(~named[:, None], 0.0), dim=1, keepdim=True)
    q = logq.exp()
    spread = torch.zeros(tokens, vocab + 1, dtype=torch.float64, device="cuda")  # the last column takes what is absent
    column = torch.where(valid, s["ids"].long(), torch.full_like(s["ids"].long(), vocab))
    spread.scatter_add_(1, column, q)
    inside = torch.zeros(tokens, vocab + 1, dtype=torch.bool, device="cuda").scatter_(1, column, True)[:, :vocab]
    spread = spread[:, :vocab]
    at = column.clamp_max(vocab - 1)
    terms = (q * (logq - logp.gather(1, at))).masked_fill(~(q > 0), 0.0)
    loss = terms.sum(1)
    if "teacher_lse" in s:
        rest = (1.0 - q.sum(1)).clamp_min(0.0)
        log_rest_p = torch.logsumexp(logp.masked_fill(inside, -math.inf), dim=1)
        some = (rest > 0) & ~inside.all(1)
        loss = loss + torch.where(some, rest * (torch.log(rest.clamp_min(1e-300)) - log_rest_p), torch.zeros_like(rest))
        rest = torch.where(some, rest, torch.zeros_like(rest))
    else:
        rest, log_rest_p = torch.zeros_like(loss), torch.zeros_like(loss)
    out = {"loss": loss * t * t}
    if case["op"] == "distill_bwd":
        total = q.sum(1) + rest
        dz = logp.exp() * total[:, None] - spread
        dz -= (logp - log_rest_p[:, None]).exp() * rest[:, None] * ~inside
        out["dlogits"] = dz * (t * s["dloss"].double())[:, None]
    return out
