"""The operators of the attention of a training step, as cases to be measured.

Queries, keys and values stand in one buffer [T, heads + 2 kv_heads, head_dim],
as a projection writes them; T tokens of one or more sequences back to back,
possibly with unused rows behind the last one.

  attn  per query head h (kv head h / (heads / kv_heads)) and sequence:
          s_ij = q_i . k_j / sqrt(head_dim)   (causal: only j <= i)
          lse_i = log sum_j exp(s_ij),  p_ij = exp(s_ij - lse_i),  o_i = sum_j p_ij v_j
        and for the gradient dO of o
          ds_ij = p_ij (do_i . v_j - do_i . o_i),
          dq_i = sum_j ds_ij k_j / sqrt(head_dim), dk_j = sum_i ds_ij q_i / sqrt(head_dim), dv_j = sum_i p_ij do_i,
        dk and dv summed over the query heads that share a kv head
  rope  for every head of q and k: x / sqrt(mean(x^2) + eps) * w, then the pairs of its first `rot` elements turned by
        pos[axis(i)] * theta^(-2i / rot); and the gradients of q, k and the two w

`own` False computes them from elementary torch operations in 32 bits (angles
in 64), `own` True calls the library.
"""

import math
import random

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_EPS = 1e-6


def listed():
    return [
        # A few short prompts, one of a single token: the time of the calls themselves.
        {"name": "attn_few_tokens", "op": "attn", "train": True, "batch": 3, "seq": 17, "ragged": True, "heads": 12,
         "kv_heads": 12, "head_dim": 64, "causal": True, "dtype": "bf16"},
        # Evaluation of a GPT-2-small-shaped model (8 x 512 tokens, D = 768).
        {"name": "attn_eval_small", "op": "attn", "train": False, "batch": 8, "seq": 512, "ragged": False, "heads": 12,
         "kv_heads": 12, "head_dim": 64, "causal": True, "dtype": "bf16"},
        # A training step of the sequence sweep's layer (8 x 512 tokens, D = 1024), every token sees every other one.
        {"name": "attn_train_full", "op": "attn", "train": True, "batch": 8, "seq": 512, "ragged": False, "heads": 16,
         "kv_heads": 16, "head_dim": 64, "causal": False, "dtype": "bf16"},
        # A batch of unpadded sequences, heads that fill no tile, keys shared by three heads, rows left over.
        {"name": "attn_train_ragged", "op": "attn", "train": True, "batch": 13, "seq": 1500, "ragged": True, "heads": 12,
         "kv_heads": 4, "head_dim": 80, "causal": True, "dtype": "bf16"},
        # A training step of the large layer (8 x 2048 tokens, D = 4096), keys shared by four heads.
        {"name": "attn_train_large", "op": "attn", "train": True, "batch": 8, "seq": 2048, "ragged": False, "heads": 32,
         "kv_heads": 8, "head_dim": 128, "causal": True, "dtype": "bf16"},
        # One long document, a few heads.
        {"name": "attn_train_long", "op": "attn", "train": True, "batch": 1, "seq": 16384, "ragged": False, "heads": 8,
         "kv_heads": 2, "head_dim": 128, "causal": True, "dtype": "bf16"},
        # A step kept in 32 bits throughout.
        {"name": "attn_train_f32", "op": "attn", "train": True, "batch": 4, "seq": 384, "ragged": False, "heads": 8,
         "kv_heads": 8, "head_dim": 64, "causal": True, "dtype": "f32"},
        # One token of one sequence: latency.
        {"name": "rope_one_token", "op": "rope", "train": False, "T": 1, "heads": 32, "kv_heads": 8, "head_dim": 128,
         "rot": 128, "axes": 1, "interleaved": False, "norm": True, "dtype": "bf16"},
        # A small model's step, forward and gradient.
        {"name": "rope_train_small", "op": "rope", "train": True, "T": 4096, "heads": 12, "kv_heads": 12, "head_dim": 64,
         "rot": 64, "axes": 1, "interleaved": False, "norm": True, "dtype": "bf16"},
        # A large layer's step.
        {"name": "rope_train_large", "op": "rope", "train": True, "T": 16384, "heads": 32, "kv_heads": 8, "head_dim": 128,
         "rot": 128, "axes": 1, "interleaved": False, "norm": True, "dtype": "bf16"},
        # Patches of a video (time, height, width), a part of each head turned, adjacent pairs, 32 bits.
        {"name": "rope_train_axes_f32", "op": "rope", "train": True, "T": 5037, "heads": 10, "kv_heads": 2, "head_dim": 80,
         "rot": 48, "axes": 3, "interleaved": True, "norm": True, "dtype": "f32"},
        # Rotation alone, images and far positions, forward only.
        {"name": "rope_eval_plain", "op": "rope", "train": False, "T": 8192, "heads": 16, "kv_heads": 16, "head_dim": 64,
         "rot": 64, "axes": 2, "interleaved": False, "norm": False, "dtype": "bf16"},
    ]


def _log_between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
    kv = rng.choice((1, 2, 3, 4, 8))
    heads = kv * rng.choice((1, 1, 2, 3, 4))
    if rng.random() < 0.55:
        f32 = dtype == "f32"
        seq = _log_between(rng, 1, 1024 if f32 else 8192)
        dim = rng.choice((64, 128, 64, 128, 8 * rng.randint(2, 16)))
        # At most 16384 tokens and about a quarter of the large step's work.
        most = max(1, min(16, 16384 // seq, int((2.0 ** 28 if f32 else 2.0 ** 31) / (float(seq) * seq * heads))))
        return {"op": "attn", "train": rng.random() < 0.7, "batch": _log_between(rng, 1, most), "seq": seq,
                "ragged": rng.random() < 0.5, "heads": heads, "kv_heads": kv, "head_dim": dim,
                "causal": rng.random() < 0.7, "dtype": dtype}
    dim = rng.choice((64, 128, 64, 128, 8 * rng.randint(2, 16)))
    return {"op": "rope", "train": rng.random() < 0.6, "T": _log_between(rng, 1, 16384), "heads": heads, "kv_heads": kv,
            "head_dim": dim, "rot": rng.choice((dim, dim, 8 * rng.randint(1, dim // 8))), "axes": rng.choice((1, 1, 2, 3)),
            "interleaved": rng.random() < 0.4, "norm": rng.random() < 0.7, "dtype": dtype}


def _lengths(case):
    """The sequences' lengths: all alike, or between one token and the longest."""
    n, seq = case["batch"], case["seq"]
    if not case["ragged"]:
        return [seq] * n
    r = random.Random(n * 1000003 + seq)
    return ([seq, 1] + [r.randint(1, seq) for _ in range(n)])[:n]


def _rows(case):
    """Tokens and rows of the buffers: a ragged batch has up to 63 rows that belong to no sequence."""
    tokens = sum(_lengths(case))
    return tokens, (tokens + 63) // 64 * 64 if case["ragged"] else tokens


def _axis_of(case):
    """The axis that turns each frequency: the axes take turns, so that each has slow and fast ones."""
    return [i % case["axes"] for i in range(case["rot"] // 2)]


def _freqs(case):
    return [10000.0 ** (-2.0 * i / case["rot"]) for i in range(case["rot"] // 2)]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    dt = _TYPES[case["dtype"]]
    heads, kv, dim = case["heads"], case["kv_heads"], case["head_dim"]

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    def split(x):
        return x[:, :heads], x[:, heads:heads + kv], x[:, heads + kv:]

    if case["op"] == "attn":
        lengths = _lengths(case)
        tokens, T = _rows(case)
        # Normed queries and keys: some heads look at few tokens (logits of a spread of 4), some at all alike.
        x = randn(T, heads + 2 * kv, dim)
        x[:, :heads] *= torch.exp(torch.rand(1, heads, 1, generator=g, device="cuda") * 2.0 - 0.6)
        q, k, v = split(x.to(dt))
        s = {"case": case, "q": q, "k": k, "v": v, "lengths": lengths, "starts": None, "rows": T}
        if case["ragged"]:
            ends = torch.tensor([0] + lengths).cumsum(0)
            s["starts"] = ends.to(torch.int32).cuda()
            # Buffers that the program keeps; the rows behind the last sequence stay zero.
            s["o"] = torch.zeros(T, heads, dim, dtype=dt, device="cuda")
            s["lse"] = torch.zeros(heads, T, device="cuda")
        if case["train"]:
            s["do"] = randn(T, heads, dim).to(dt)
            # The gradients go where the projection's backward reads them: one buffer of the projection's layout.
            s["d"] = split(torch.zeros(T, heads + 2 * kv, dim, dtype=dt, device="cuda"))
        return s
    T = case["T"]
    q, k, _ = split((randn(T, heads + 2 * kv, dim) * torch.exp(randn(T, heads + 2 * kv, 1) * 0.5)).to(dt))
    if case["axes"] == 1:  # a few sequences, the first of them far into a document
        at = torch.arange(T, device="cuda")
        pos = torch.where(at < T // 3, at + 800000, at % 1000)[None]
    else:
        pos = torch.randint(0, 4000, (case["axes"], T), generator=g, device="cuda")
    s = {"case": case, "q": q, "k": k, "pos": pos.contiguous(), "freqs": _freqs(case), "axis": _axis_of(case),
         "wq": None, "wk": None}
    if case["norm"]:
        s["wq"], s["wk"] = (1.0 + 0.2 * randn(dim)).to(dt), (1.0 + 0.2 * randn(dim)).to(dt)
    if case["train"]:
        s["dyq"], s["dyk"] = randn(T, heads, dim).to(dt), randn(T, kv, dim).to(dt)
    return s


# ------------------------------------------------------------------ one pass


def run(s):
    if own:
        return _library(s)
    return _plain_attn(s) if s["case"]["op"] == "attn" else _plain_rope(s)


def _library(s):
    import tensor_transformer_mlp_column_gb300 as tp

    case = s["case"]
    if case["op"] == "attn":
        seqs = {"starts": s["starts"], "max_seq": case["seq"]} if case["ragged"] else {"batch": case["batch"]}
        o, lse = tp.tpmlp_attn_core_forward(s["q"], s["k"], s["v"], causal=case["causal"], o=s.get("o"),
                                            lse=s.get("lse"), **seqs)
        if not case["train"]:
            return {"o": o, "lse": lse}
        dq, dk, dv = tp.tpmlp_attn_core_backward(s["q"], s["k"], s["v"], o, lse, s["do"], causal=case["causal"],
                                                 dq=s["d"][0], dk=s["d"][1], dv=s["d"][2], **seqs)
        return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}
    turn = {"freqs": s["freqs"], "axis": s["axis"], "interleaved": case["interleaved"], "wq": s["wq"], "wk": s["wk"],
            "eps": _EPS}
    yq, yk = tp.tpmlp_qk_rope_forward(s["q"], s["k"], s["pos"], **turn)
    if not case["train"]:
        return {"yq": yq, "yk": yk}
    dq, dk, dwq, dwk = tp.tpmlp_qk_rope_backward(s["dyq"], s["dyk"], s["q"], s["k"], s["pos"], **turn)
    out = {"yq": yq, "yk": yk, "dq": dq, "dk": dk}
    if case["norm"]:
        out.update(dwq=dwq, dwk=dwk)
    return out


def _plain_attn(s):
    case = s["case"]
    heads, kv, dim, T = case["heads"], case["kv_heads"], case["head_dim"], s["rows"]
    group, scale = heads // kv, 1.0 / math.sqrt(case["head_dim"])
    dt = s["q"].dtype
    o = torch.zeros(T, heads, dim, dtype=dt, device="cuda")
    lse = torch.zeros(heads, T, device="cuda")
    dq = torch.zeros(T, heads, dim, dtype=dt, device="cuda")
    dk = torch.zeros(T, kv, dim, dtype=dt, device="cuda")
    dv = torch.zeros(T, kv, dim, dtype=dt, device="cuda")
    at = 0
    for n in s["lengths"]:
        rows = slice(at, at + n)
        at += n
        # As many kv heads at a time as keep a score matrix within 2 GB.
        some = max(1, min(kv, int(2 ** 29 / (float(n) * n * group))))
        hidden = None
        if case["causal"]:
            hidden = torch.arange(n, device="cuda")[None, :] > torch.arange(n, device="cuda")[:, None]
        for h in range(0, kv, some):
            ks = slice(h, min(kv, h + some))
            qs = slice(ks.start * group, ks.stop * group)
            k = s["k"][rows, ks].float().transpose(0, 1)[:, None]  # [kv heads, 1, n, dim]
            v = s["v"][rows, ks].float().transpose(0, 1)[:, None]
            q = s["q"][rows, qs].float().transpose(0, 1).reshape(-1, group, n, dim)
            p = (q @ k.transpose(2, 3)) * scale
            if hidden is not None:
                p.masked_fill_(hidden, float("-inf"))
            top = p.amax(dim=3, keepdim=True)
            p = torch.exp(p - top)
            total = p.sum(dim=3, keepdim=True)
            p = p / total
            y = p @ v
            o[rows, qs] = y.reshape(-1, n, dim).transpose(0, 1).to(dt)
            lse[qs, rows] = (top + torch.log(total)).reshape(-1, n)
            if not case["train"]:
                continue
            do = s["do"][rows, qs].float().transpose(0, 1).reshape(-1, group, n, dim)
            dv[rows, ks] = (p.transpose(2, 3) @ do).sum(dim=1).transpose(0, 1).to(dt)
            ds = do @ v.transpose(2, 3)
            ds = p * (ds - (do * y).sum(dim=3, keepdim=True))
            dq[rows, qs] = ((ds @ k) * scale).reshape(-1, n, dim).transpose(0, 1).to(dt)
            dk[rows, ks] = ((ds.transpose(2, 3) @ q).sum(dim=1) * scale).transpose(0, 1).to(dt)
    return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv} if case["train"] else {"o": o, "lse": lse}


def _turn(x, cos, sin, rot, interleaved):
    """The pairs of the first `rot` elements of every head turned; cos and sin [T, 1, rot / 2]."""
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, a * sin + b * cos
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * cos - b * sin, a * sin + b * cos
    return y


def _plain_rope(s):
    case = s["case"]
    freqs = torch.tensor(s["freqs"], dtype=torch.float64).cuda()
    angle = s["pos"].double()[torch.tensor(s["axis"]).cuda()].T * freqs
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    out = {}
    for name in ("q", "k"):
        x, w = s[name].float(), s["w" + name]
        n = x
        if w is not None:
            r = 1.0 / torch.sqrt((x * x).mean(dim=2, keepdim=True) + _EPS)
            n = x * r
            y = _turn(n * w.float(), cos, sin, case["rot"], case["interleaved"])
        else:
            y = _turn(n, cos, sin, case["rot"], case["interleaved"])
        out["y" + name] = y.to(s[name].dtype)
        if not case["train"]:
            continue
        g = _turn(s["dy" + name].float(), cos, -sin, case["rot"], case["interleaved"])
        if w is not None:
            out["dw" + name] = (g * n).sum(dim=(0, 1))
            g = g * w.float()
            g = r * (g - n * (g * n).mean(dim=2, keepdim=True))
        out["d" + name] = g.to(s[name].dtype)
    return out


# ------------------------------------------------------------------ what a pass cannot do without


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    heads, kv, dim = case["heads"], case["kv_heads"], case["head_dim"]
    if case["op"] == "attn":
        tokens = sum(_lengths(case))
        pairs = sum(n * (n + 1) // 2 if case["causal"] else n * n for n in _lengths(case))
        q, k = tokens * heads * dim * es, tokens * kv * dim * es
        rows = 4 * heads * tokens
        if not case["train"]:  # q, k, v; o, lse
            return {"bytes": 2 * q + 2 * k + rows, "flops": 4 * pairs * heads * dim}
        # q, k, v, do; o, lse, dq, dk, dv
        return {"bytes": 4 * q + 4 * k + rows, "flops": 14 * pairs * heads * dim}
    T = case["T"]
    x = T * (heads + kv) * dim * es
    small = 8 * case["axes"] * T + (2 * dim * es if case["norm"] else 0)
    if not case["train"]:
        return {"bytes": 2 * x + small, "flops": 8 * T * (heads + kv) * dim}
    return {"bytes": 4 * x + small + (8 * dim if case["norm"] else 0), "flops": 24 * T * (heads + kv) * dim}


# ------------------------------------------------------------------ the definitions in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_attn(s) if case["op"] == "attn" else _exact_rope(s)


def _exact_attn(s):
    """Head by head from the softmax's definition; the gradients by differentiating it."""
    case = s["case"]
    heads, kv, dim, T = case["heads"], case["kv_heads"], case["head_dim"], s["rows"]
    if 14.0 * dim * heads * sum(float(n) * n for n in s["lengths"]) > 8e12:
        return None  # 64-bit products of that size take too long
    f64 = {"dtype": torch.float64, "device": "cuda"}
    got = {"o": torch.zeros(T, heads, dim, **f64), "lse": torch.zeros(heads, T, **f64)}
    if case["train"]:
        got.update(dq=torch.zeros(T, heads, dim, **f64), dk=torch.zeros(T, kv, dim, **f64), dv=torch.zeros(T, kv, dim, **f64))
    first = 0
    for n in s["lengths"]:
        last = first + n
        for h in range(heads):
            j = h * kv // heads
            q = s["q"][first:last, h].double().requires_grad_(case["train"])
            k = s["k"][first:last, j].double().requires_grad_(case["train"])
            v = s["v"][first:last, j].double().requires_grad_(case["train"])
            z = torch.mm(q, k.t()) * dim ** -0.5
            if case["causal"]:
                z = z + torch.full((n, n), -math.inf, **f64).triu_(1)
            y = torch.mm(torch.softmax(z, 1), v)
            got["o"][first:last, h] = y.detach()
            got["lse"][h, first:last] = torch.logsumexp(z.detach(), 1)
            if case["train"]:
                y.backward(s["do"][first:last, h].double())
                got["dq"][first:last, h] = q.grad
                got["dk"][first:last, j] += k.grad
                got["dv"][first:last, j] += v.grad
            del z, y
        first = last
    return got


def _exact_rope(s):
    """Pairs as complex numbers times exp(i angle); the gradients by differentiating that."""
    case = s["case"]
    rot, T = case["rot"], case["T"]
    turns = torch.stack([s["pos"][a].double() * f for f, a in zip(s["freqs"], s["axis"])], dim=1)[:, None]
    phase = torch.polar(torch.ones_like(turns), turns)
    got = {}
    for name in ("q", "k"):
        x = s[name].double().requires_grad_(case["train"])
        w = None if s["w" + name] is None else s["w" + name].double().requires_grad_(case["train"])
        n = x if w is None else x * torch.rsqrt(x.pow(2).mean(-1, keepdim=True) + _EPS) * w
        part = n[..., :rot]
        pairs = part.unflatten(-1, (-1, 2)) if case["interleaved"] else part.unflatten(-1, (2, -1)).transpose(-1, -2)
        z = torch.complex(pairs[..., 0], pairs[..., 1]) * phase
        pairs = torch.stack((z.real, z.imag), -1)
        part = pairs.flatten(-2) if case["interleaved"] else pairs.transpose(-1, -2).flatten(-2)
        y = torch.cat((part, n[..., rot:]), -1)
        got["y" + name] = y.detach()
        if case["train"]:
            y.backward(s["dy" + name].double())
            got["d" + name] = x.grad
            if w is not None:
                got["dw" + name] = w.grad
    return got
