"""The attention of a training step on the GPU, against its definitions in 64
bits: softmax attention on given queries, keys and values with its gradients,
the norms and rotation of queries and keys with theirs, and a run of both.

Tolerances are bounds by arithmetic, element by element. U16 = 2^-8 is half a
step of bf16 relative to the value, U32 = 2^-24 of fp32. A sum over n products
in fp32 is off by at most (n + 2) U32 of the sum of their magnitudes; on the
tensor cores 16 products at a time go to an accumulator that is rounded or
truncated, at most 2 U32 each time.
"""

import math

import pytest
import torch

pytestmark = pytest.mark.gpu

U16, U32 = 2.0 ** -8, 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def tp():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()
    import tensor_transformer_mlp_column_gb300 as tp

    torch.cuda.set_device(0)
    return tp


def _close(got, ref, tol, what):
    err = (got.double() - ref).abs()
    worst = (err / tol.clamp(min=1e-300)).max().item() if err.numel() else 0.0
    assert bool((err <= tol).all()), f"{what}: worst error is {worst:.3g} of its bound"


def _sum(n, dtype):
    """Bound of a sum over n products, relative to the sum of their magnitudes."""
    return (n / 16 + 2) * 2 * U32 if dtype == "bf16" else (n + 2) * U32


# ------------------------------------------------------------------ attention


def _inputs(T, heads, kv, dim, dtype, seed, spread=1.5, layout="packed"):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, heads + 2 * kv, dim, generator=g, device="cuda")
    x[:, :heads] *= spread
    do = torch.randn(T, heads, dim, generator=g, device="cuda").to(DT[dtype])
    x = x.to(DT[dtype])
    parts = [x[:, :heads], x[:, heads:heads + kv], x[:, heads + kv:]]
    if layout == "apart":
        parts = [p.contiguous() for p in parts]
    elif layout == "heads_first":
        parts = [p.transpose(0, 1).contiguous().transpose(0, 1) for p in parts]
        do = do.transpose(0, 1).contiguous().transpose(0, 1)
    return (*parts, do)


def _reference(q, k, v, do, lengths, first, causal, scale, dtype):
    """Values and bounds of every output, [T, ...] in 64 bits, zero outside of the sequences."""
    T, heads, dim = q.shape
    kv = k.shape[1]
    f64 = dict(dtype=torch.float64, device="cuda")
    shape = {"o": (T, heads, dim), "lse": (heads, T), "dq": (T, heads, dim), "dk": (T, kv, dim), "dv": (T, kv, dim)}
    val = {n: torch.zeros(s, **f64) for n, s in shape.items()}
    tol = {n: torch.zeros(s, **f64) for n, s in shape.items()}
    u_op = 1.01 * U16 if dtype == "bf16" else 0.0   # probabilities and ds as operands
    u_out = 1.01 * U16 if dtype == "bf16" else 1.01 * U32
    c_dim = _sum(dim, dtype)
    at = first
    for n in lengths:
        r = slice(at, at + n)
        at += n
        if n == 0:
            continue
        c_n = _sum(n, dtype)
        hide = torch.ones(n, n, dtype=torch.bool, device="cuda").triu(1) if causal else None
        for h in range(heads):
            j = h * kv // heads
            Q, K, V, G = (t[r, i].double() for t, i in ((q, h), (k, j), (v, j), (do, h)))
            s = Q @ K.T * scale
            mag = Q.abs() @ K.abs().T * scale
            if causal:
                s = s.masked_fill(hide, -math.inf)
                mag = mag.masked_fill(hide, 0.0)
            lse = torch.logsumexp(s, 1)
            p = torch.exp(s - lse[:, None])
            o = p @ V
            # Scores: their sums, the factor; exponentials: the argument's rounding (size up to |s| + |lse|) and 4 U32.
            big = mag.max(dim=1).values + lse.abs()
            e_s = mag.max(dim=1).values * (c_dim + 4 * U32) + 8 * U32 * (big + 1)
            e_l = 2 * e_s + (n + 4) * U32 + 8 * U32 * (lse.abs() + 1)
            e_p = 1.01 * (e_s + e_l) + 8 * U32
            pv = p @ V.abs()
            t_o = pv * (u_op + 2 * e_p + 2 * c_n)[:, None]
            t_o = t_o + u_out * o.abs()
            delta = (G * o).sum(1)
            e_d = (G.abs() * t_o).sum(1) + c_dim * (G.abs() * o.abs()).sum(1) + dim * U32 * (G.abs() * o.abs()).sum(1)
            dp = G @ V.T
            e_dp = (G.abs() @ V.abs().T) * c_dim + 2 * U32 * (dp.abs() + delta.abs()[:, None])
            ds = p * (dp - delta[:, None])
            e_ds = p * (e_dp + e_d[:, None]) * 1.02 + ds.abs() * (e_p[:, None] + u_op + 4 * U32) * 1.01
            e_pp = p * (e_p[:, None] + u_op) * 1.01
            val["o"][r, h], tol["o"][r, h] = o, t_o
            val["lse"][h, r], tol["lse"][h, r] = lse, e_l
            dq = ds @ K * scale
            val["dq"][r, h] = dq
            tol["dq"][r, h] = scale * (e_ds @ K.abs() + c_n * (ds.abs() @ K.abs())) + u_out * dq.abs() + 2 * U32 * dq.abs()
            val["dk"][r, j] += ds.T @ Q * scale
            tol["dk"][r, j] += scale * (e_ds.T @ Q.abs() + _sum(n * heads // kv, dtype) * (ds.abs().T @ Q.abs()))
            val["dv"][r, j] += p.T @ G
            tol["dv"][r, j] += e_pp.T @ G.abs() + _sum(n * heads // kv, dtype) * (p.T @ G.abs())
    for name in ("dk", "dv"):
        tol[name] += (u_out + 2 * U32) * val[name].abs()
    return val, tol


FILL = 7.0


def _check(tp, lengths, heads, kv, dim, dtype, causal=True, seed=0, first=0, behind=0, scale=None, layout="packed",
           spread=1.5, batch=None, max_seq=None):
    T = first + sum(lengths) + behind
    q, k, v, do = _inputs(T, heads, kv, dim, dtype, seed, spread, layout)
    outside = torch.ones(T, dtype=torch.bool, device="cuda")
    outside[first:first + sum(lengths)] = False
    for t in (q, k, v, do):
        t[outside] = math.nan  # rows of no sequence may hold anything
    sc = dim ** -0.5 if scale is None else scale
    val, tol = _reference(q, k, v, do, lengths, first, causal, sc, dtype)
    kw = dict(scale=scale, causal=causal)
    if batch is None:
        ends = torch.tensor([first] + list(lengths)).cumsum(0)
        kw.update(starts=ends.to(torch.int32).cuda(), max_seq=max(lengths) if max_seq is None else max_seq)
    else:
        kw.update(batch=batch)
    out = {n: torch.full_like(t, FILL) for n, t in (("o", q), ("dq", q), ("dk", k), ("dv", v))}
    out["lse"] = torch.full((heads, T), FILL, device="cuda")
    o, lse = tp.tpmlp_attn_core_forward(q, k, v, o=out["o"], lse=out["lse"], **kw)
    assert o.data_ptr() == out["o"].data_ptr() and lse.data_ptr() == out["lse"].data_ptr()
    tp.tpmlp_attn_core_backward(q, k, v, o, lse, do, dq=out["dq"], dk=out["dk"], dv=out["dv"], **kw)
    tp.tpmlp_check_status()
    for name, got in out.items():
        away = got[:, outside] if name == "lse" else got[outside]
        assert bool((away == FILL).all()), f"{name}: rows of no sequence were written"
        rows = (slice(None), ~outside) if name == "lse" else (~outside,)
        _close(got[rows], val[name][rows], tol[name][rows] + 1e-30, f"{name} {lengths}")
    return out


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lengths", [[1], [2], [63], [64], [65], [127], [128], [129], [257], [1, 1, 1], [5, 1, 130, 17],
                                     [300, 0, 40, 0, 0, 129]])
def test_lengths(tp, lengths, causal, dtype):
    _check(tp, lengths, 2, 2, 64, dtype, causal, seed=sum(lengths))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("count", [31, 32, 33, 63, 64, 65, 150])
def test_many_sequences(tp, count, causal, dtype):
    # bf16 hands them out by their lengths, 64 at a time.
    lengths = [(37 * i * i + 11 * i) % 300 for i in range(count)]
    lengths[count // 2] = 700
    _check(tp, lengths, 2, 1, 64 if count % 2 else 128, dtype, causal, seed=count)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lengths", [[5, 300] + [0] * 130 + [257, 1, 0, 40], [0] * 200 + [130], [0] * 64 + [1] * 64 + [0] * 64,
                                     [200] * 64 + [3] + [0] * 63])
def test_many_empty_sequences(tp, lengths, dtype):
    _check(tp, lengths, 2, 2, 64, dtype, seed=len(lengths), max_seq=sum(lengths))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lengths", [[5, 300] + [0] * 130 + [257, 1, 0, 40], [700] + [1] * 70 + [33], [0] * 70 + [65] * 5,
                                     [64] * 40, [1, 2, 1000]])
@pytest.mark.parametrize("dim", [64, 96])
def test_longest_length_left_at_all_tokens(tp, lengths, causal, dim, dtype):
    _check(tp, lengths, 6, 2, dim, dtype, causal, seed=len(lengths) + 3, first=3, behind=45, max_seq=48 + sum(lengths))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [8, 16, 24, 40, 56, 64, 72, 80, 96, 120, 128])
def test_head_sizes(tp, dim, dtype):
    _check(tp, [150, 33], 2, 1, dim, dtype, True, seed=dim)
    _check(tp, [150, 33], 2, 1, dim, dtype, False, seed=dim + 1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_sequences_of_no_stated_length(tp, dtype):
    # max_seq for every sequence would be 2^32 tiles of 32 rows; what there is to do is as with the longest length given.
    T, n, heads = 1 << 17, 1 << 15, 32
    g = torch.Generator().manual_seed(3)
    ends = torch.cat([torch.zeros(1, dtype=torch.long), torch.randint(0, 8, (n,), generator=g).cumsum(0)])
    longest, starts = int((ends[1:] - ends[:-1]).max()), ends.to(torch.int32).cuda()
    q, k, v, do = _inputs(T, heads, 1, 8, dtype, 31)
    got = []
    for most in (longest, None):
        o, lse = tp.tpmlp_attn_core_forward(q, k, v, starts=starts, max_seq=most, o=torch.zeros_like(q),
                                            lse=torch.zeros(heads, T, device="cuda"))
        dq, _, dv = tp.tpmlp_attn_core_backward(q, k, v, o, lse, do, starts=starts, max_seq=most, dq=torch.zeros_like(q),
                                                dv=torch.zeros_like(v))
        got.append((o, lse, dq, dv))
    tp.tpmlp_check_status()
    assert all(torch.equal(a, b) for a, b in zip(*got)) and got[0][0].float().abs().sum().item() > 0


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lengths,dim", [([1, 2, 3, 9, 40, 64], 64), ([64, 33], 8), ([128, 127, 5, 1], 128), ([100] * 5, 72),
                                         ([700], 16), ([130, 64, 1, 1000], 40), ([65, 300], 56)])
def test_both_pieces_of_ds(tp, lengths, dim, causal):
    # Short sequences' dq and dk, and narrow heads' dq, are as far off as their own rounding to bf16 and fp32 sums make
    # them: ds enters in two bf16 pieces (off by U16^2), and what delta is off (U16 of sum |do o|, rows of more than a
    # tile) is taken out again with probabilities rounded to bf16, which leaves U16 of it.
    T = sum(lengths)
    q, k, v, do = _inputs(T, 3, 3, dim, "bf16", 77 + dim)
    ends = torch.tensor([0] + lengths).cumsum(0).to(torch.int32).cuda()
    kw = dict(starts=ends, max_seq=max(lengths), causal=causal)
    o, lse = tp.tpmlp_attn_core_forward(q, k, v, **kw)
    dq, dk, _ = tp.tpmlp_attn_core_backward(q, k, v, o, lse, do, **kw)
    scale, c_dim, at = dim ** -0.5, _sum(dim, "bf16"), 0
    short = max(lengths) <= (64 if dim <= 64 else 128)
    for n in lengths:
        r = slice(at, at + n)
        at += n
        c_n = _sum(n, "bf16")
        hide = torch.ones(n, n, dtype=torch.bool, device="cuda").triu(1) & causal
        for h in range(3):
            Q, K, V, G = (t[r, h].double() for t in (q, k, v, do))
            s = (Q @ K.T * scale).masked_fill(hide, -math.inf)
            mag = (Q.abs() @ K.abs().T * scale).masked_fill(hide, 0.0).max(dim=1).values
            l = torch.logsumexp(s, 1)
            p = torch.exp(s - l[:, None])
            e_s = mag * (c_dim + 4 * U32) + 8 * U32 * (mag + l.abs() + 1)
            e_p = (1.01 * (3 * e_s + (n + 4) * U32 + 8 * U32 * (l.abs() + 1)) + 8 * U32)[:, None]
            O = p @ V
            dp = G @ V.T
            delta = (G * O).sum(1)[:, None]
            e_dp = (G.abs() @ V.abs().T) * c_dim + 2 * U32 * (dp.abs() + delta.abs())
            E = ((G.abs() * O.abs()).sum(1) * 1.02 * U16 + (G.abs() * (p @ V.abs())).sum(1) * 1.02 * U16)[:, None]
            e_d = (p * e_dp).sum(1, True) + 2 * (e_p + c_n) * (p * (dp.abs() + delta.abs() + E)).sum(1, True) + 1.02 * U16 * E
            ds = p * (dp - delta)
            big = ds.abs() + p * E
            e_ds = 1.02 * p * (e_dp + e_d) + big * (e_p + 8 * U32 + 1.02 * U16 * U16)
            ref = ds @ K * scale
            _close(dq[r, h], ref, scale * ((e_ds + c_n * big) @ K.abs() + c_n * E * (p @ K.abs())) + 1.01 * U16 * ref.abs() + 1e-30,
                   f"dq {n}")
            if short:
                ref = ds.T @ Q * scale
                _close(dk[r, h], ref, scale * ((e_ds + c_n * big).T @ Q.abs()) + 1.01 * U16 * ref.abs() + 1e-30, f"dk {n}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("heads,kv", [(1, 1), (3, 1), (8, 2), (6, 3), (12, 4), (5, 5), (16, 1)])
def test_shared_heads(tp, heads, kv, dtype):
    _check(tp, [70, 200], heads, kv, 64, dtype, True, seed=heads)
    _check(tp, [140], heads, kv, 128, dtype, False, seed=heads + 1)


@pytest.mark.parametrize("dim", [40, 64, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lengths,heads,kv", [([1000], 8, 1), ([700, 130, 1, 0, 300], 16, 1), ([520, 520], 12, 2),
                                              ([2100], 2, 1), ([1], 16, 1), ([129] * 3, 32, 1)])
def test_few_keys_for_many_queries(tp, lengths, heads, kv, causal, dim):
    # The passes over a key tile are cut into runs, some of them without a pass, whose sums are added.
    _check(tp, lengths, heads, kv, dim, "bf16", causal, seed=heads + dim, first=3, behind=5)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["packed", "apart", "heads_first"])
def test_layouts(tp, layout, dtype):
    _check(tp, [100, 129, 3], 4, 2, 72, dtype, True, seed=3, layout=layout)
    _check(tp, [100] * 3, 4, 2, 64, dtype, False, seed=4, layout=layout, batch=3)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 128])
def test_rows_of_no_sequence(tp, dim, dtype):
    # NaNs before the first and behind the last sequence, inside the tiles of its first and last rows.
    _check(tp, [65, 1, 60], 2, 1, dim, dtype, True, seed=5, first=37, behind=50)
    _check(tp, [130], 2, 1, dim, dtype, False, seed=6, first=1, behind=1, max_seq=150)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_sequence_does_not_see_its_neighbours(tp, dtype):
    lengths, heads, kv, dim = [100, 70, 90], 2, 2, 64
    q, k, v, do = _inputs(260, heads, kv, dim, dtype, 11)
    for t in (q, k, v, do):
        t[100:170] = math.inf
    starts = torch.tensor([0, 100, 170, 260], dtype=torch.int32, device="cuda")
    for causal in (True, False):
        o, lse = tp.tpmlp_attn_core_forward(q, k, v, starts=starts, max_seq=100, causal=causal)
        got = (o, *tp.tpmlp_attn_core_backward(q, k, v, o, lse, do, starts=starts, max_seq=100, causal=causal))
        for t in got:
            assert bool(torch.isfinite(t[:100]).all()) and bool(torch.isfinite(t[170:]).all())
        # The same as each of them alone.
        for a, b in ((0, 100), (170, 260)):
            p = [t[a:b] for t in (q, k, v)]
            o1, l1 = tp.tpmlp_attn_core_forward(*p, causal=causal)
            g1 = tp.tpmlp_attn_core_backward(*p, o1, l1, do[a:b], causal=causal)
            for x, y in zip(got, (o1, *g1)):
                assert torch.equal(x[a:b], y)
            assert torch.equal(lse[:, a:b], l1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("spread,scale", [(30.0, None), (0.0, None), (1.0, 3.0), (1.0, 1e-6)])
def test_scores_large_and_small(tp, spread, scale, dtype):
    _check(tp, [200, 64], 2, 1, 64, dtype, True, seed=7, spread=spread, scale=scale)
    _check(tp, [200, 64], 2, 1, 64, dtype, False, seed=8, spread=spread, scale=scale)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scores_that_grow_along_the_keys(tp, dtype):
    # The running maximum moves in every tile, up and, in the other order, never again.
    T, dim = 600, 64
    for order in (1, -1):
        q, k, v, do = _inputs(T, 1, 1, dim, dtype, 9)
        ramp = torch.linspace(0.0, 12.0, T, device="cuda")[:, None, None]
        ramp = ramp.flip(0) if order < 0 else ramp
        q[:], k[:] = (q.float() * 0.1 + 1.0).to(q.dtype), (k.float() * 0.1 + ramp).to(k.dtype)
        for causal in (True, False):
            val, tol = _reference(q, k, v, do, [T], 0, causal, dim ** -0.5, dtype)
            o, lse = tp.tpmlp_attn_core_forward(q, k, v, causal=causal)
            dq, dk, dv = tp.tpmlp_attn_core_backward(q, k, v, o, lse, do, causal=causal)
            for name, got in (("o", o), ("lse", lse), ("dq", dq), ("dk", dk), ("dv", dv)):
                _close(got, val[name], tol[name] + 1e-30, name)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_infinite_scores(tp, dtype):
    # A key of -inf scores counts for nothing (as in the definition), whichever tile it stands in.
    q, k, v, do = _inputs(300, 1, 1, 64, dtype, 10)
    q[:] = q.abs()
    k[:200:7] = -math.inf
    for causal in (False, True):
        o, lse = tp.tpmlp_attn_core_forward(q, k, v, causal=causal)
        s = q[:, 0].double() @ k[:, 0].double().T * 0.125
        if causal:
            s = s.masked_fill(torch.ones(300, 300, dtype=torch.bool, device="cuda").triu(1), -math.inf)
        ref = torch.logsumexp(s, 1)
        seen = torch.isfinite(ref)
        assert bool(seen[1:].all()) and bool(seen[0]) == (not causal)
        assert bool(((lse[0].double() - ref)[seen].abs() < 1e-4).all())
        y = torch.softmax(s, 1) @ v[:, 0].double()
        assert bool(((o[:, 0].double() - y)[seen].abs() < 0.05).all())
        assert bool(torch.isnan(o[~seen]).all())  # a row without a key, as a softmax over nothing is


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_long(tp, dtype):
    _check(tp, [1500, 700], 2, 1, 128, dtype, True, seed=12, layout="apart")
    _check(tp, [2100], 1, 1, 64, dtype, False, seed=13)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_bitwise_reproducible(tp, dtype):
    q, k, v, do = _inputs(1200, 8, 2, 64, dtype, 14)
    first = None
    for _ in range(3):
        o, lse = tp.tpmlp_attn_core_forward(q, k, v, batch=2)
        got = (o, lse, *tp.tpmlp_attn_core_backward(q, k, v, o, lse, do, batch=2))
        first = got if first is None else first
        assert all(torch.equal(a, b) for a, b in zip(got, first))


def test_gradients_against_differences(tp):
    # fp32: the loss is off by about 2^-24 of its terms' size; steps of 2^-6 make the difference's third-order part small.
    lengths, heads, kv, dim = [9, 30], 2, 1, 16
    T = sum(lengths)
    q, k, v, do = _inputs(T, heads, kv, dim, "f32", 15, layout="apart")
    starts = torch.tensor([0, 9, 39], dtype=torch.int32, device="cuda")

    def loss(q, k, v):
        o, lse = tp.tpmlp_attn_core_forward(q, k, v, starts=starts, max_seq=30)
        return (o.double() * do.double()).sum().item()

    o, lse = tp.tpmlp_attn_core_forward(q, k, v, starts=starts, max_seq=30)
    grads = tp.tpmlp_attn_core_backward(q, k, v, o, lse, do, starts=starts, max_seq=30)
    g = torch.Generator(device="cuda").manual_seed(1)
    for i in range(3):
        for _ in range(4):
            d = torch.randn(grads[i].shape, generator=g, device="cuda")
            d = d / d.norm()
            h = 2.0 ** -6
            x = [q, k, v]
            up, down = list(x), list(x)
            up[i], down[i] = x[i] + h * d, x[i] - h * d
            num = (loss(*up) - loss(*down)) / (2 * h)
            ana = (grads[i].double() * d.double()).sum().item()
            size = grads[i].double().norm().item()
            assert abs(num - ana) <= 2e-3 * size, (i, num, ana)


def test_sequences_that_are_none(tp):
    q, k, v, do = _inputs(300, 2, 1, 64, "bf16", 16)
    for bad in ([0, 100, 90, 300], [0, 100, 301, 400], [0, 100, -5, 100]):
        starts = torch.tensor(bad, dtype=torch.int32, device="cuda")
        o, lse = torch.full_like(q, FILL), torch.full((2, 300), FILL, device="cuda")
        tp.tpmlp_attn_core_forward(q, k, v, starts=starts, max_seq=300, o=o, lse=lse)
        with pytest.raises(tp.TpmlpError) as e:
            tp.tpmlp_check_status()
        assert e.value.code == tp.TPMLP_ERR_BOUNDS and "sequence" in str(e.value)
        one, _ = tp.tpmlp_attn_core_forward(q[:100], k[:100], v[:100])
        # Rows 90 .. 99 of the first list belong to two sequences, [0, 100) and [90, 300): undefined.
        alone = 90 if bad[2] == 90 else 100
        assert torch.equal(o[:alone], one[:alone])
    # Longer than max_seq: left out; the rest is done.
    starts = torch.tensor([0, 100, 200, 300], dtype=torch.int32, device="cuda")
    long = torch.tensor([0, 100, 230, 300], dtype=torch.int32, device="cuda")
    for back in (False, True):
        o, lse = tp.tpmlp_attn_core_forward(q, k, v, starts=starts, max_seq=100)
        dq, dk, dv = (torch.full_like(t, FILL) for t in (q, k, v))
        if back:
            tp.tpmlp_attn_core_backward(q, k, v, o, lse, do, starts=long, max_seq=100, dq=dq, dk=dk, dv=dv)
            assert bool((dq[100:230] == FILL).all()) and bool((dk[100:230] == FILL).all())
        else:
            o2 = torch.full_like(q, FILL)
            tp.tpmlp_attn_core_forward(q, k, v, starts=long, max_seq=100, o=o2)
            assert bool((o2[100:230] == FILL).all()) and torch.equal(o2[:100], o[:100])
        with pytest.raises(tp.TpmlpError):
            tp.tpmlp_check_status()
    tp.tpmlp_check_status()


def test_nothing_to_do(tp):
    e = torch.empty(0, 2, 64, device="cuda", dtype=torch.bfloat16)
    o, lse = tp.tpmlp_attn_core_forward(e, e, e)
    assert o.shape == (0, 2, 64) and lse.shape == (2, 0)
    assert [t.shape for t in tp.tpmlp_attn_core_backward(e, e, e, o, lse, e)] == [e.shape] * 3
    q, k, v, do = _inputs(10, 2, 1, 64, "bf16", 17)
    for starts in ([0], [3, 3], [0, 0, 0, 10, 10]):
        s = torch.tensor(starts, dtype=torch.int32, device="cuda")
        o = torch.full_like(q, FILL)
        tp.tpmlp_attn_core_forward(q, k, v, starts=s, o=o)
        assert bool((o == FILL).all()) == (len(starts) < 5)
    tp.tpmlp_check_status()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("back", [False, True])
def test_sequences_where_nothing_is_computed(tp, back, dtype):
    # No rows, or a longest length of 0: nothing is written, and a sequence that has tokens all the same is recorded.
    def call(q, k, v, do, starts, max_seq):
        out = [torch.full_like(t, FILL) for t in (q, q, k, v)]
        lse = torch.full((q.shape[1], q.shape[0]), FILL, device="cuda")
        s = torch.tensor(starts, dtype=torch.int32, device="cuda")
        if back:
            tp.tpmlp_attn_core_backward(q, k, v, q, lse, do, starts=s, max_seq=max_seq, dq=out[1], dk=out[2], dv=out[3])
        else:
            tp.tpmlp_attn_core_forward(q, k, v, starts=s, max_seq=max_seq, o=out[0], lse=lse)
        torch.cuda.synchronize()
        assert all(bool((t == FILL).all()) for t in (*out, lse))

    some, none = _inputs(300, 2, 1, 64, dtype, 42), _inputs(0, 2, 1, 64, dtype, 42)
    for x, starts, max_seq, fine in ((some, [0, 0, 0], 0, True), (some, [7], 0, True), (some, [300, 300], 0, True),
                                     (some, [0, 100, 300], 0, False), (some, [5] * 999 + [6], 0, False),
                                     (some, [0, 0, -1, -1], 0, False), (some, [301, 301], 0, False),
                                     (none, [0, 0, 0], None, True), (none, [0], None, True), (none, [0, 5], None, False),
                                     (none, [0, 0, 0, 1], 0, False)):
        call(*x, starts, max_seq)
        if fine:
            tp.tpmlp_check_status()
            continue
        with pytest.raises(tp.TpmlpError) as e:
            tp.tpmlp_check_status()
        assert e.value.code == tp.TPMLP_ERR_BOUNDS and "sequence" in str(e.value)
    # Captured into a graph, the check is one of its nodes.
    s, o = torch.tensor([0, 100, 300], dtype=torch.int32, device="cuda"), torch.full_like(some[0], FILL)
    lse = torch.zeros(2, 300, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        if back:
            tp.tpmlp_attn_core_backward(*some[:3], o, lse, some[3], starts=s, max_seq=0)
        else:
            tp.tpmlp_attn_core_forward(*some[:3], starts=s, max_seq=0, o=o, lse=lse)
    tp.tpmlp_check_status()
    g.replay()
    with pytest.raises(tp.TpmlpError):
        tp.tpmlp_check_status()
    s.zero_()
    g.replay()
    tp.tpmlp_check_status()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_one_token_of_a_large_layout(tp, dtype):
    # One token of buffers [heads, tokens, 64]: the token stride is less than a row of all heads, and not used.
    big = torch.full((9, 5000, 64), math.nan, device="cuda", dtype=DT[dtype])
    big[:, 4999] = torch.randn(9, 64, generator=torch.Generator("cuda").manual_seed(5), device="cuda").to(DT[dtype])
    one = big.transpose(0, 1)[4999:]
    q, k, v, do = one[:, :4], one[:, 4:6], one[:, 6:8], one[:, 5:9]
    pos, f = torch.full((1,), 77, device="cuda"), _freqs(64)

    def run(q, k, v, do, out):
        yq, yk = tp.tpmlp_qk_rope_forward(q, k, pos, f, yq=out(4), yk=out(2))
        o, lse = tp.tpmlp_attn_core_forward(yq, yk, v, o=out(4))
        dq, dk, dv = tp.tpmlp_attn_core_backward(yq, yk, v, o, lse, do, dq=out(4), dk=out(2), dv=out(2))
        return o, lse, dv, *tp.tpmlp_qk_rope_backward(dq, dk, q, k, pos, f, dq=out(4), dk=out(2))[:2]

    far = run(q, k, v, do, lambda n: torch.empty(n, 3000, 64, device="cuda", dtype=DT[dtype]).transpose(0, 1)[2999:])
    near = run(*(t.contiguous() for t in (q, k, v, do)), lambda n: None)
    tp.tpmlp_check_status()
    assert all(torch.equal(a, b) for a, b in zip(far, near)) and bool(torch.isfinite(far[0]).all())


# ------------------------------------------------------------------ norms and rotation


def _rope_reference(x, dy, w, pos, freqs, axis, inter, eps, dtype):
    """y, dx, dw in 64 bits with their bounds."""
    T, heads, dim = x.shape
    half = len(freqs)
    rot = 2 * half
    X, G = x.double(), dy.double()
    u_out = 1.01 * U16 if dtype == "bf16" else 1.01 * U32
    ang = torch.stack([pos[a].double() * f for f, a in zip(freqs, axis)], 1)[:, None] if half else None

    def turn(z, back):
        if not half:
            return z
        z = z.clone()
        c, s = torch.cos(ang), torch.sin(ang) * (-1.0 if back else 1.0)
        ia = torch.arange(0, rot, 2) if inter else torch.arange(half)
        ib = ia + 1 if inter else ia + half
        a, b = z[..., ia].clone(), z[..., ib].clone()
        z[..., ia], z[..., ib] = a * c - b * s, a * s + b * c
        return z

    def pair(z):  # |a| + |b| in both places of a pair
        z = z.abs().clone()
        if half:
            ia = torch.arange(0, rot, 2) if inter else torch.arange(half)
            ib = ia + 1 if inter else ia + half
            both = z[..., ia] + z[..., ib]
            z[..., ia], z[..., ib] = both, both
        return z

    if w is None:
        n, z, r, W = X, X, torch.ones_like(X[..., :1]), torch.ones(dim, dtype=torch.float64, device="cuda")
    else:
        r = 1.0 / torch.sqrt((X * X).mean(-1, keepdim=True) + eps)
        n, W = X * r, w.double()
        z = n * W
    rel = (dim + 30) * U32  # of r (a sum of dim squares), the products, the angles and the turn
    y = turn(z, False)
    t_y = pair(z) * rel + u_out * y.abs()
    g = turn(G, True)
    t_g = pair(G) * 30 * U32
    if w is None:
        return y, t_y, g, t_g + u_out * g.abs(), None, None
    dn = g * W
    mean = (dn * n).mean(-1, keepdim=True)
    dx = r * (dn - n * mean)
    mag = r * (pair(G) * W.abs() + n.abs() * (pair(G) * W.abs() * n.abs()).mean(-1, keepdim=True))
    t_dx = mag * 2 * rel + u_out * dx.abs()
    dw = (g * n).sum((0, 1))
    t_dw = ((pair(G) * n.abs()).sum((0, 1))) * (rel + (T * heads + 20) * U32) + 1.01 * U32 * dw.abs()
    return y, t_y, dx, t_dx, dw, t_dw


def _rope_inputs(T, heads, kv, dim, dtype, axes, seed, norm=True):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*s):
        return torch.randn(s, generator=g, device="cuda")

    x = (randn(T, heads + 2 * kv, dim) * torch.exp(randn(T, heads + 2 * kv, 1))).to(DT[dtype])
    pos = torch.randint(-50, 5000, (axes, T), generator=g, device="cuda")
    w = [(1.0 + 0.3 * randn(dim)).to(DT[dtype]) for _ in range(2)] if norm else [None, None]
    dy = randn(T, heads, dim).to(DT[dtype]), randn(T, kv, dim).to(DT[dtype])
    return x[:, :heads], x[:, heads:heads + kv], pos, w, dy


def _freqs(rot, theta=10000.0):
    return [theta ** (-2.0 * i / rot) for i in range(rot // 2)]


def _check_rope(tp, T, heads, kv, dim, rot, dtype, axes=1, inter=False, norm=True, seed=0, pos=None, eps=1e-6):
    q, k, p, w, dy = _rope_inputs(T, heads, kv, dim, dtype, axes, seed, norm)
    pos = p if pos is None else pos
    freqs, axis = _freqs(rot), [(3 * i + 1) % axes for i in range(rot // 2)]
    kw = dict(freqs=freqs, axis=axis, interleaved=inter, wq=w[0], wk=w[1], eps=eps)
    y = tp.tpmlp_qk_rope_forward(q, k, pos, **kw)
    dq, dk, dwq, dwk = tp.tpmlp_qk_rope_backward(*dy, q, k, pos, **kw)
    tp.tpmlp_check_status()
    for name, x, g, wt, yy, dx, dw in (("q", q, dy[0], w[0], y[0], dq, dwq), ("k", k, dy[1], w[1], y[1], dk, dwk)):
        ry, ty, rdx, tdx, rdw, tdw = _rope_reference(x, g, wt, pos, freqs, axis, inter, eps, dtype)
        _close(yy, ry, ty + 1e-30, f"y{name}")
        _close(dx, rdx, tdx + 1e-30, f"d{name}")
        if norm:
            assert dw.dtype == torch.float32
            _close(dw, rdw, tdw + 1e-30, f"dw{name}")
        else:
            assert dw is None


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dim,rot", [(8, 8), (16, 8), (64, 64), (64, 32), (72, 40), (80, 80), (128, 128), (128, 64),
                                     (136, 136), (200, 104), (256, 256), (64, 0), (256, 8)])
def test_rope_head_sizes(tp, dim, rot, inter, dtype):
    _check_rope(tp, 37, 3, 2, dim, rot, dtype, axes=2, inter=inter, seed=dim + rot)
    _check_rope(tp, 5, 2, 1, dim, rot, dtype, inter=inter, norm=False, seed=dim + rot + 1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 2, 7, 100, 3001])
@pytest.mark.parametrize("heads,kv", [(1, 1), (32, 8), (12, 12), (5, 1), (2, 3)])
def test_rope_tokens_and_heads(tp, T, heads, kv, dtype):
    _check_rope(tp, T, heads, kv, 64 if T > 100 else 128, 64, dtype, axes=3, seed=T + heads)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rope_far_positions(tp, dtype):
    # The definition's own angle in 64 bits is off by 2^-53 of its size; far ones are turned by their fraction of a turn.
    pos = torch.tensor([[0, 1, -1, 1000003, -999983, 2 ** 24 + 1, 123456789, -2 ** 31]], device="cuda")
    _check_rope(tp, 8, 2, 2, 64, 64, dtype, pos=pos, seed=21)


def test_rope_in_place_and_layouts(tp):
    for dtype in ("bf16", "f32"):
        q, k, pos, w, dy = _rope_inputs(300, 6, 2, 80, dtype, 2, 22)
        kw = dict(freqs=_freqs(48), axis=[i % 2 for i in range(24)], wq=w[0], wk=w[1])
        y = tp.tpmlp_qk_rope_forward(q, k, pos, **kw)
        back = tp.tpmlp_qk_rope_backward(*dy, q, k, pos, **kw)
        qt, kt = (t.transpose(0, 1).contiguous().transpose(0, 1) for t in (q, k))
        yt = [torch.empty_like(t) for t in (qt, kt)]
        tp.tpmlp_qk_rope_forward(qt, kt, pos, yq=yt[0], yk=yt[1], **kw)
        assert torch.equal(yt[0], y[0]) and torch.equal(yt[1], y[1])
        g = [t.clone() for t in dy]
        got = tp.tpmlp_qk_rope_backward(*g, qt, kt, pos, dq=g[0], dk=g[1], **kw)
        assert all(torch.equal(a, b) for a, b in zip(got, back))
        tp.tpmlp_qk_rope_forward(q, k, pos, yq=q, yk=k, **kw)
        assert torch.equal(q, y[0]) and torch.equal(k, y[1])


def test_rope_no_tokens(tp):
    e = torch.empty(0, 4, 64, device="cuda", dtype=torch.bfloat16)
    pos = torch.empty(0, device="cuda", dtype=torch.int64)
    w = torch.ones(64, device="cuda", dtype=torch.bfloat16)
    y = tp.tpmlp_qk_rope_forward(e, e, pos, _freqs(64), wq=w, wk=w)
    assert y[0].shape == e.shape
    dw = [torch.full((64,), FILL, device="cuda") for _ in range(2)]
    tp.tpmlp_qk_rope_backward(e, e, e, e, pos, _freqs(64), wq=w, wk=w, dwq=dw[0], dwk=dw[1])
    assert bool((dw[0] == 0).all()) and bool((dw[1] == 0).all())


def test_rope_zero_and_infinite_rows(tp):
    # A row of zeros stays zero (eps > 0); a row that is not finite spoils no other one.
    q, k, pos, w, dy = _rope_inputs(50, 3, 1, 64, "f32", 1, 23)
    kw = dict(freqs=_freqs(64), wq=w[0], wk=w[1])
    ref = tp.tpmlp_qk_rope_forward(q, k, pos, **kw)
    q[7], q[9, 1] = 0.0, math.nan
    y, _ = tp.tpmlp_qk_rope_forward(q, k, pos, **kw)
    assert bool((y[7] == 0).all()) and bool(torch.isnan(y[9, 1]).all())
    rest = torch.ones(50, 3, dtype=torch.bool, device="cuda")
    rest[7], rest[9, 1] = False, False
    assert torch.equal(y[rest], ref[0][rest])


@pytest.mark.parametrize("T,heads,kv", [(1, 1, 1), (3, 2, 1), (37, 5, 2), (1001, 3, 1)])
def test_rope_without_eps(tp, T, heads, kv):
    # Lanes and groups without a head add nothing to the weights' gradients, whatever 1 / sqrt(0) is.
    for dim in (8, 40, 136):
        _check_rope(tp, T, heads, kv, dim, dim, "f32", seed=T, eps=0.0)


def test_rope_reproducible(tp):
    q, k, pos, w, dy = _rope_inputs(2000, 8, 2, 128, "bf16", 1, 24)
    a = tp.tpmlp_qk_rope_backward(*dy, q, k, pos, _freqs(128), wq=w[0], wk=w[1])
    b = tp.tpmlp_qk_rope_backward(*dy, q, k, pos, _freqs(128), wq=w[0], wk=w[1])
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_rope_gradients_against_differences(tp):
    q, k, pos, w, dy = _rope_inputs(6, 2, 1, 16, "f32", 1, 25)
    q, k = q.contiguous(), k.contiguous()
    freqs = _freqs(8)

    def loss(q, k, wq, wk):
        y = tp.tpmlp_qk_rope_forward(q, k, pos, freqs, wq=wq, wk=wk)
        return sum((a.double() * b.double()).sum().item() for a, b in zip(y, dy))

    grads = tp.tpmlp_qk_rope_backward(*dy, q, k, pos, freqs, wq=w[0], wk=w[1])
    x = [q, k, *w]
    g = torch.Generator(device="cuda").manual_seed(2)
    for i in range(4):
        d = torch.randn(x[i].shape, generator=g, device="cuda")
        d = d / d.norm() * x[i].norm()
        h = 2.0 ** -9  # relative step
        up, down = list(x), list(x)
        up[i], down[i] = x[i] + h * d, x[i] - h * d
        num = (loss(*up) - loss(*down)) / (2 * h)
        ana = (grads[i].double() * d.double()).sum().item()
        assert abs(num - ana) <= 5e-3 * (grads[i].double().norm() * d.double().norm()).item(), (i, num, ana)


# ------------------------------------------------------------------ a run of them


def _step(tp, x, w, pos, starts, max_seq, heads, kv, do, stream=None, d=None):
    """Norm and rotation, attention, and back into one buffer of the projection's layout."""
    q, k, v = x[:, :heads], x[:, heads:heads + kv], x[:, heads + kv:]
    kw = dict(freqs=_freqs(q.shape[2]), wq=w[0], wk=w[1], stream=stream)
    seqs = dict(starts=starts, max_seq=max_seq, stream=stream)
    yq, yk = tp.tpmlp_qk_rope_forward(q, k, pos, **kw)
    o, lse = tp.tpmlp_attn_core_forward(yq, yk, v, **seqs)
    d = torch.zeros_like(x) if d is None else d
    dq, dk, dv = d[:, :heads], d[:, heads:heads + kv], d[:, heads + kv:]
    tp.tpmlp_attn_core_backward(yq, yk, v, o, lse, do, dq=dq, dk=dk, dv=dv, **seqs)
    _, _, dwq, dwk = tp.tpmlp_qk_rope_backward(dq, dk, q, k, pos, dq=dq, dk=dk, **kw)
    return o, lse, d, dwq, dwk


def _step_inputs(dtype, lengths, heads, kv, dim, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    T = sum(lengths)
    x = torch.randn(T, heads + 2 * kv, dim, generator=g, device="cuda").to(DT[dtype])
    w = [(1.0 + 0.2 * torch.randn(dim, generator=g, device="cuda")).to(DT[dtype]) for _ in range(2)]
    do = torch.randn(T, heads, dim, generator=g, device="cuda").to(DT[dtype])
    starts = torch.tensor([0] + lengths).cumsum(0).to(torch.int32).cuda()
    pos = torch.cat([torch.arange(n) for n in lengths]).cuda()
    return x, w, pos, starts, max(lengths), heads, kv, do


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("heads,kv,dim", [(4, 2, 64), (3, 1, 128), (2, 2, 40)])
def test_a_run_of_them(tp, heads, kv, dim, dtype):
    lengths = [130, 1, 77]
    args = _step_inputs(dtype, lengths, heads, kv, dim, 31)
    o, lse, d, dwq, dwk = _step(tp, *args)
    x, w, pos, starts, _, _, _, do = args
    X = x.double().requires_grad_()
    W = [t.double().requires_grad_() for t in w]
    half = dim // 2
    ang = pos.double()[:, None] * torch.tensor(_freqs(dim), dtype=torch.float64, device="cuda")
    c, s = torch.cos(ang)[:, None], torch.sin(ang)[:, None]

    def rope(z, wt):
        z = z * torch.rsqrt((z * z).mean(-1, keepdim=True) + 1e-6) * wt
        a, b = z[..., :half], z[..., half:]
        return torch.cat((a * c - b * s, a * s + b * c), -1)

    q, k, v = rope(X[:, :heads], W[0]), rope(X[:, heads:heads + kv], W[1]), X[:, heads + kv:]
    outs, at = [], 0
    for n in lengths:
        r = slice(at, at + n)
        at += n
        kk, vv = (t[r].repeat_interleave(heads // kv, 1).transpose(0, 1) for t in (k, v))
        z = q[r].transpose(0, 1) @ kk.transpose(1, 2) * dim ** -0.5
        z = z.masked_fill(torch.ones(n, n, dtype=torch.bool, device="cuda").triu(1), -math.inf)
        outs.append((torch.softmax(z, -1) @ vv).transpose(0, 1))
    ref = torch.cat(outs)
    ref.backward(do.double())
    # Norms of the errors: bf16 rounds yq, yk, p, o, ds, the gradients of both calls: ten roundings of at most 2^-8 each,
    # their effects on the gradients of the scores at most twice their size.
    bound = 20 * U16 if dtype == "bf16" else 2.0 ** -16
    for name, got, want in (("o", o, ref.detach()), ("d", d, X.grad), ("dwq", dwq, W[0].grad), ("dwk", dwk, W[1].grad)):
        err = (got.double() - want).norm() / want.norm()
        assert err.item() <= bound, (name, err.item())
    tp.tpmlp_check_status()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_captured_and_replayed(tp, dtype):
    # Two graphs of different sizes that share nothing, replayed in turn, beside eager calls.
    cases = [_step_inputs(dtype, lengths, 4, 2, 64, seed) for lengths, seed in (([200, 60], 32), ([33, 300, 1], 33))]
    want = [_step(tp, *a) for a in cases]
    graphs = []
    for a in cases:
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.stream(s):
            _step(tp, *a)
        torch.cuda.current_stream().wait_stream(s)
        with torch.cuda.graph(g):
            out = _step(tp, *a)
        graphs.append((g, out))
    for _ in range(3):
        for g, _ in graphs:
            g.replay()
        eager = _step(tp, *cases[0])
        torch.cuda.synchronize()
        for (_, out), w in zip(graphs, want):
            assert all(torch.equal(a, b) for a, b in zip(out, w))
        assert all(torch.equal(a, b) for a, b in zip(eager, want[0]))
    # New inputs in the captured buffers.
    cases[0][0].copy_(cases[0][0].flip(0))
    graphs[0][0].replay()
    again = _step(tp, *cases[0])
    assert all(torch.equal(a, b) for a, b in zip(graphs[0][1], again))
    tp.tpmlp_check_status()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_side_by_side_on_two_streams(tp, dtype):
    cases = [_step_inputs(dtype, [400, 100], 4, 2, 64, seed) for seed in (34, 35)]
    want = [_step(tp, *a) for a in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for s, a in zip(streams, cases):
            with torch.cuda.stream(s):
                d = torch.zeros_like(a[0])
            got.append(_step(tp, *a, stream=s, d=d))
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(torch.equal(a, b) for a, b in zip(g, w))


def test_rows_beyond_32_bit_offsets(tp):
    # A buffer of more than 2^32 elements: the last sequence starts behind 2^31 elements, and 2^32 bytes.
    heads, kv, dim = 64, 2, 64
    T = 2 ** 32 // (68 * 64) + 300
    x = torch.empty(T, heads + 2 * kv, dim, dtype=torch.bfloat16, device="cuda")
    n = 130
    g = torch.Generator(device="cuda").manual_seed(36)
    tail = torch.randn(n, heads + 2 * kv, dim, generator=g, device="cuda").bfloat16()
    x[T - n:] = tail
    starts = torch.tensor([T - n, T], dtype=torch.int32, device="cuda")
    do = torch.empty(T, heads, dim, dtype=torch.bfloat16, device="cuda")
    do[T - n:] = tail[:, 3:3 + heads]
    q, k, v = x[:, :heads], x[:, heads:heads + kv], x[:, heads + kv:]
    o, lse = tp.tpmlp_attn_core_forward(q, k, v, starts=starts, max_seq=n)
    dq, dk, dv = tp.tpmlp_attn_core_backward(q, k, v, o, lse, do, starts=starts, max_seq=n)
    p = tail[:, :heads], tail[:, heads:heads + kv], tail[:, heads + kv:]
    o1, l1 = tp.tpmlp_attn_core_forward(*p)
    g1 = tp.tpmlp_attn_core_backward(*p, o1, l1, tail[:, 3:3 + heads])
    assert torch.equal(o[T - n:], o1) and torch.equal(lse[:, T - n:], l1)
    for a, b in zip((dq, dk, dv), g1):
        assert torch.equal(a[T - n:], b)
    pos = torch.full((T,), 5, dtype=torch.int64, device="cuda")
    del o, lse, dq, dk, dv, do
    yq, yk = tp.tpmlp_qk_rope_forward(q, k, pos, _freqs(64))
    zq, zk = tp.tpmlp_qk_rope_forward(p[0], p[1], pos[:n], _freqs(64))
    assert torch.equal(yq[T - n:], zq) and torch.equal(yk[T - n:], zk)
    tp.tpmlp_check_status()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("load", [1, 2, 5])
def test_a_load_that_never_comes(tp, load, backward, dim):
    # Every wait has a limit: the CTAs give up, report it, and the next calls are as before.
    q, k, v, do = _inputs(700, 4, 4, dim, "bf16", 41, layout="apart")
    o, lse = tp.tpmlp_attn_core_forward(q, k, v, causal=False)
    want = (o, lse, *tp.tpmlp_attn_core_backward(q, k, v, o, lse, do, causal=False))
    tp.tpmlp_check_status()
    tp.tpmlp_selftest_attn_core_timeout(q, k, v, backward, load, 50)
    with pytest.raises(tp.TpmlpError) as e:
        tp.tpmlp_check_status()
    assert e.value.code == tp.TPMLP_ERR_TIMEOUT
    o, lse = tp.tpmlp_attn_core_forward(q, k, v, causal=False)
    got = (o, lse, *tp.tpmlp_attn_core_backward(q, k, v, o, lse, do, causal=False))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    tp.tpmlp_check_status()


def test_captured_before_any_other_call(tp):
    # The first calls of a process may be captured: nothing is allocated or looked up on the stream.
    import subprocess
    import sys

    code = """
import torch
import tensor_transformer_mlp_column_gb300 as tp
x = torch.randn(300, 6, 64, device="cuda").bfloat16()
q, k, v = x[:, :4], x[:, 4:5], x[:, 5:]
do = torch.randn(300, 4, 64, device="cuda").bfloat16()
pos = torch.arange(300, device="cuda")
freqs = [10000.0 ** (-i / 32) for i in range(32)]
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
def step():
    a, b = tp.tpmlp_qk_rope_forward(q, k, pos, freqs)
    o, lse = tp.tpmlp_attn_core_forward(a, b, v)
    return (o, lse, *tp.tpmlp_attn_core_backward(a, b, v, o, lse, do))
with torch.cuda.graph(g):
    out = step()
g.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(out, step()))
tp.tpmlp_check_status()
print("captured")
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


_PI = 3141592653589793238462643383279502884197169399375105820974944592307816  # 10^69 pi


def _angle(pos, f):
    """pos * f without its whole turns, from integers: off by less than 2^-50 of a turn for |pos f| < 2^150."""
    n, d = f.as_integer_ratio()
    unit = 2 * _PI * d  # a whole turn, in units of 1 / (10^69 d)
    part = pos * n * 10 ** 69 % unit
    return 2 * math.pi * (part / unit)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("inter", [False, True])
def test_rope_fast_frequencies_and_far_positions(tp, inter, dtype):
    # The turn is off by 2^-64 |pos| (2^-24 here), whatever the frequency. fp32: the angle as a fraction of half a turn and
    # sincospi's argument, pi U32, its result 2 U32, the turn's products and sum 3 U32 of |a| + |b|. bf16: 32 bits of the
    # turn, a rounded argument, pi U32 twice, and 2^-21.19 of the special-function unit: below 2^-20.
    freqs = [1.0, 7.0, 6.283185307179586, 100.3, 1.0e4, 123456.789, 3.1e9, 2.0 ** 40, -3.7, -1.0e4, -1e-12, 1e-12, -2.0 ** -60,
             0.1, 1 / 3, 0.0]
    pos = [0, 1, -1, 5, 10 ** 9 + 7, -10 ** 9 + 1, 2 ** 38 + 12345, -2 ** 38 + 3, 2 ** 40 - 1, -2 ** 40 + 77, 2 ** 39 + 1]
    dim, rot, T = 40, 2 * len(freqs), len(pos)
    q, k, _, _, dy = _rope_inputs(T, 3, 2, dim, dtype, 1, 51, norm=False)
    p = torch.tensor(pos, device="cuda")
    ang = torch.tensor([[_angle(at, f) for f in freqs] for at in pos], dtype=torch.float64, device="cuda")[:, None]
    c, s = torch.cos(ang), torch.sin(ang)
    far = 2 * math.pi * 2.0 ** -64 * p.abs().double()[:, None, None]
    unit = (10 * U32 if dtype == "f32" else 2.0 ** -20 + 10 * U32) + far
    u_out = 1.01 * (U32 if dtype == "f32" else U16)
    ia = torch.arange(0, rot, 2) if inter else torch.arange(rot // 2)
    ib = ia + 1 if inter else ia + rot // 2
    y = tp.tpmlp_qk_rope_forward(q, k, p, freqs, interleaved=inter)
    d = tp.tpmlp_qk_rope_backward(*dy, q, k, p, freqs, interleaved=inter)
    for name, x, got, sn in (("yq", q, y[0], s), ("yk", k, y[1], s), ("dq", dy[0], d[0], -s), ("dk", dy[1], d[1], -s)):
        a, b = x[..., ia].double(), x[..., ib].double()
        ref, tol = x.double().clone(), torch.zeros_like(x, dtype=torch.float64)
        ref[..., ia], ref[..., ib] = a * c - b * sn, a * sn + b * c
        tol[..., ia] = tol[..., ib] = (a.abs() + b.abs()) * unit
        _close(got, ref, tol + u_out * ref.abs() + 1e-30, name)
    tp.tpmlp_check_status()
