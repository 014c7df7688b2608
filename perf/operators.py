"""The operators at the two ends of a training step, as cases to be measured.

A step around the library's transformer blocks begins with the embedding
lookup, ends with the cross entropy over the vocabulary, and is closed by the
gradient of the embedding table and the clipping of all gradients by their
global norm:

  xent   loss_t = logsumexp_v(x_t . w_v) - x_t . w_target(t), and for the row
         gradients g_t of the losses dX = dZ W, dW = dZ^T X with
         dZ_tv = g_t (softmax(x_t W^T)_v - [v = target(t)]);
         rows with a negative target count for nothing
  embed  out_t = s E[token(t)], and dE_v = s sum_{t: token(t) = v} dout_t;
         rows with a negative token are zero and give no gradient
  clip   norm = sqrt(sum of all squares), out_i = min(1, max_norm / (norm + 1e-6)) g_i

`own` False computes them from elementary torch operations in 32 bits, `own`
True calls the library.
"""

import math
import random

import numpy as np
import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # The loss of one scored token: the vocabulary's matrix is read for a single row.
        {"name": "loss_one_token", "op": "xent", "train": False, "T": 1, "D": 768, "V": 50257, "dtype": "bf16"},
        # Evaluation (perplexity) of a batch.
        {"name": "loss_eval", "op": "xent", "train": False, "T": 4096, "D": 1024, "V": 32000, "dtype": "bf16"},
        # A training step's loss and gradients next to the GPT-2-small-shaped blocks, an odd vocabulary.
        {"name": "loss_train_small", "op": "xent", "train": True, "T": 4096, "D": 768, "V": 50257, "dtype": "bf16"},
        # Ragged in every size: a batch of unpadded sequences, a width that fills no tile.
        {"name": "loss_train_ragged", "op": "xent", "train": True, "T": 1037, "D": 2056, "V": 30011, "dtype": "bf16"},
        # A large model's step: a wide layer and a large vocabulary.
        {"name": "loss_train_large", "op": "xent", "train": True, "T": 8192, "D": 4096, "V": 128000, "dtype": "bf16"},
        # A step kept in 32 bits throughout.
        {"name": "loss_train_f32", "op": "xent", "train": True, "T": 1000, "D": 512, "V": 32001, "dtype": "f32"},
        # One token for each of a few sequences: latency.
        {"name": "embed_few_tokens", "op": "embed", "train": False, "T": 8, "D": 4096, "V": 128000, "dtype": "bf16"},
        # A small model's step, the gradient in 32 bits as the block's backward gives it.
        {"name": "embed_train_small", "op": "embed", "train": True, "T": 4096, "D": 768, "V": 50257, "dtype": "f32"},
        # A large batch and table; most rows of the table get no gradient.
        {"name": "embed_train_large", "op": "embed", "train": True, "T": 65536, "D": 4096, "V": 128000,
         "dtype": "bf16"},
        # The shard gradients of one small block.
        {"name": "clip_block", "op": "clip", "tensors": 8, "size": 589824, "spread": False, "mixed": False},
        # Many tensors of odd sizes and both types, one element to a few million.
        {"name": "clip_mixed", "op": "clip", "tensors": 56, "size": 3000001, "spread": True, "mixed": True},
        # The shard gradients of one large block (D = 8192, F = 32768, 8 shards).
        {"name": "clip_large", "op": "clip", "tensors": 16, "size": 33554432, "spread": False, "mixed": False},
    ]


def _log_between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("xent", "xent", "embed", "clip"))
    if op == "xent":
        return {"op": "xent", "train": rng.random() < 0.7, "T": _log_between(rng, 1, 8192),
                "D": 8 * _log_between(rng, 8, 512), "V": _log_between(rng, 300, 128000),
                "dtype": rng.choice(("bf16", "bf16", "bf16", "f32"))}
    if op == "embed":
        return {"op": "embed", "train": rng.random() < 0.7, "T": _log_between(rng, 1, 65536),
                "D": _log_between(rng, 16, 4096), "V": _log_between(rng, 100, 128000),
                "dtype": rng.choice(("bf16", "f32"))}
    return {"op": "clip", "tensors": rng.randint(1, 60), "size": _log_between(rng, 100, 8000000),
            "spread": rng.random() < 0.7, "mixed": rng.random() < 0.5}


def _sizes(case):
    """The element counts of a case's gradients: all alike, or from one element up to the largest, over the logarithm."""
    n, size = case["tensors"], case["size"]
    if not case["spread"]:
        return [size] * n
    r = random.Random(n * 1000003 + size)
    return [size] + [_log_between(r, 1, size) for _ in range(n - 1)]


def _types(case):
    return [torch.bfloat16 if case["mixed"] and i % 2 else torch.float32 for i in range(case["tensors"])]


def _token_ids(g, T, V):
    """Ids as frequent as words are (the k-th about as 1 / k), scattered over the table."""
    u = torch.rand(T, generator=g, device="cuda", dtype=torch.float64)
    rank = (torch.exp(u * math.log(V + 1.0)).long() - 1).clamp_(0, V - 1)
    return torch.randperm(V, generator=g, device="cuda")[rank]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    if case["op"] == "xent":
        T, D, V = case["T"], case["D"], case["V"]
        dt = _TYPES[case["dtype"]]
        W = (0.02 * randn(V, D)).to(dt)
        targets = _token_ids(g, T, V)
        # Rows between untrained and sure of their target (its logit 0 to 12 above the others).
        u = torch.rand(T, 1, generator=g, device="cuda")
        X = (randn(T, D) + u * (12.0 / (0.02 * 0.02 * D)) * W[targets].float()).to(dt)
        # One row in ten is padding or prompt, without a loss.
        skip = torch.rand(T, generator=g, device="cuda") < 0.1
        skip[0] = False
        targets = torch.where(skip, torch.full_like(targets, -100), targets)
        # The gradient of the mean over the rows that count.
        dloss = torch.full((T,), 1.0, device="cuda") / (~skip).sum()
        return {"case": case, "X": X, "W": W, "targets": targets, "dloss": dloss}
    if case["op"] == "embed":
        T, D, V = case["T"], case["D"], case["V"]
        dt = _TYPES[case["dtype"]]
        tokens = _token_ids(g, T, V)
        if T > 1:  # padding
            pad = torch.rand(T, generator=g, device="cuda") < 0.05
            tokens = torch.where(pad, torch.full_like(tokens, -1), tokens)
        return {"case": case, "E": (0.02 * randn(V, D)).to(dt), "tokens": tokens, "scale": math.sqrt(D),
                "dout": (randn(T, D) / max(T, 1)).to(dt) if case["train"] else None}
    scales = torch.exp(torch.rand(case["tensors"], generator=g, device="cuda") * 6.0 - 8.0)
    grads = [(randn(n) * scales[i]).to(dt) for i, (n, dt) in enumerate(zip(_sizes(case), _types(case)))]
    return {"case": case, "grads": grads, "max_norm": 1.0}


# ------------------------------------------------------------------ one pass


def run(s):
    if own:
        return _library(s)
    op = s["case"]["op"]
    return _plain_xent(s) if op == "xent" else _plain_embed(s) if op == "embed" else _plain_clip(s)


def _library(s):
    import tensor_transformer_mlp_column_gb300 as tp

    case = s["case"]
    if case["op"] == "xent":
        loss, lse = tp.tpmlp_xent_forward(s["X"], s["W"], s["targets"])
        if not case["train"]:
            return {"loss": loss, "lse": lse}
        dX, dW = tp.tpmlp_xent_backward(s["X"], s["W"], s["targets"], lse, s["dloss"])
        return {"loss": loss, "lse": lse, "dX": dX, "dW": dW}
    if case["op"] == "embed":
        out = tp.tpmlp_embed_forward(s["E"], s["tokens"], s["scale"])
        if not case["train"]:
            return {"out": out}
        return {"out": out, "dE": tp.tpmlp_embed_backward(s["dout"], s["tokens"], case["V"], s["scale"])}
    out = [torch.empty_like(g) for g in s["grads"]]
    norm = tp.tpmlp_grad_clip(s["grads"], s["max_norm"], out=out)
    return {"norm": norm, "out": out}


def _plain_xent(s):
    X, W, targets = s["X"], s["W"], s["targets"]
    x, w = X.float(), W.float()
    z = x @ w.T
    valid = targets >= 0
    at = targets.clamp(min=0)[:, None]
    top = z.max(dim=1, keepdim=True).values
    lse = top + torch.log(torch.exp(z - top).sum(dim=1, keepdim=True))
    zt = z.gather(1, at)
    loss = torch.where(valid, (lse - zt)[:, 0], torch.zeros_like(lse[:, 0]))
    if not s["case"]["train"]:
        return {"loss": loss, "lse": lse[:, 0]}
    g = torch.where(valid, s["dloss"], torch.zeros_like(s["dloss"]))[:, None]
    dz = torch.exp(z - lse) * g
    dz.scatter_add_(1, at, -g)
    return {"loss": loss, "lse": lse[:, 0], "dX": (dz @ w).to(X.dtype), "dW": (dz.T @ x).to(W.dtype)}


def _plain_embed(s):
    E, tokens, scale = s["E"], s["tokens"], s["scale"]
    valid = (tokens >= 0)[:, None]
    at = tokens.clamp(min=0)
    out = torch.where(valid, E[at].float() * scale, torch.zeros((), device="cuda")).to(E.dtype)
    if not s["case"]["train"]:
        return {"out": out}
    d = torch.where(valid, s["dout"].float() * scale, torch.zeros((), device="cuda"))
    dE = torch.zeros(E.shape, dtype=torch.float32, device="cuda").index_add_(0, at, d)
    return {"out": out, "dE": dE.to(s["dout"].dtype)}


def _plain_clip(s):
    sums = torch.stack([g.float().square().sum() for g in s["grads"]])
    norm = sums.sum().sqrt()
    c = torch.clamp(s["max_norm"] / (norm + 1e-6), max=1.0)
    return {"norm": norm.reshape(1), "out": [(g.float() * c).to(g.dtype) for g in s["grads"]]}


# ------------------------------------------------------------------ what a pass cannot do without


def _distinct(case):
    """Expected number of distinct table rows among a case's tokens."""
    k = np.arange(case["V"], dtype=np.float64)
    p = np.log((k + 2) / (k + 1)) / math.log(case["V"] + 1.0)
    return float(np.sum(-np.expm1(case["T"] * np.log1p(-np.minimum(p, 1 - 1e-12)))))


def work(case):
    if case["op"] == "xent":
        T, D, V = case["T"], case["D"], case["V"]
        es = 2 if case["dtype"] == "bf16" else 4
        bytes_ = (T + V) * D * es + 8 * T + 8 * T  # X, W, targets; loss and lse
        if not case["train"]:
            return {"bytes": bytes_, "flops": 2 * T * V * D}
        return {"bytes": bytes_ + (T + V) * D * es + 4 * T, "flops": 6 * T * V * D}
    if case["op"] == "embed":
        T, D, V = case["T"], case["D"], case["V"]
        es = 2 if case["dtype"] == "bf16" else 4
        bytes_ = 8 * T + _distinct(case) * D * es + T * D * es
        flops = T * D
        if case["train"]:
            bytes_ += T * D * es + V * D * es
            flops += 2 * T * D
        return {"bytes": bytes_, "flops": flops}
    n = sum(_sizes(case))
    b = sum(m * (2 if t == torch.bfloat16 else 4) for m, t in zip(_sizes(case), _types(case)))
    return {"bytes": 2 * b + 4, "flops": 3 * n}


# ------------------------------------------------------------------ the definitions in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "xent":
        T, D, V = case["T"], case["D"], case["V"]
        if (6 if case["train"] else 2) * T * D * V > 6e12:
            return None  # 64-bit products of that size take too long
        w = s["W"].double()
        dW = torch.zeros((V, D), dtype=torch.float64, device="cuda")
        loss, lse, dX = [], [], []
        for r in range(0, T, 1024):
            x = s["X"][r:r + 1024].double()
            t = s["targets"][r:r + 1024]
            counted = (t >= 0).double()
            logits = torch.mm(x, w.t())
            norm = torch.logsumexp(logits, 1)
            hot = torch.nn.functional.one_hot(t.clamp(min=0), V).double()
            lse.append(norm)
            loss.append((norm - (logits * hot).sum(1)) * counted)
            if case["train"]:
                d = (torch.softmax(logits, 1) - hot) * (s["dloss"][r:r + 1024].double() * counted)[:, None]
                dX.append(torch.mm(d, w))
                dW.addmm_(d.t(), x)
            del logits, hot
        got = {"loss": torch.cat(loss), "lse": torch.cat(lse)}
        if case["train"]:
            got.update(dX=torch.cat(dX), dW=dW)
        return got
    if case["op"] == "embed":
        t = s["tokens"]
        keep = torch.nonzero(t >= 0)[:, 0]
        out = torch.zeros((case["T"], case["D"]), dtype=torch.float64, device="cuda")
        out[keep] = s["E"].index_select(0, t[keep]).double() * s["scale"]
        if not case["train"]:
            return {"out": out}
        dE = torch.zeros((case["V"], case["D"]), dtype=torch.float64, device="cuda")
        dE.index_put_((t[keep],), s["dout"][keep].double() * s["scale"], accumulate=True)
        return {"out": out, "dE": dE}
    norm = math.sqrt(sum(float(torch.dot(g.double(), g.double())) for g in s["grads"]))
    c = min(1.0, s["max_norm"] / (norm + 1e-6))
    return {"norm": torch.tensor([norm], dtype=torch.float64), "out": [g.double() * c for g in s["grads"]]}
