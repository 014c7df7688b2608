"""Refusals of the attention of a training step: argument checks that run before
any CUDA call, through the C ABI with addresses that are never dereferenced,
and the binding's own checks."""

import ctypes
import math
from array import array

import pytest

FAKE = 0x7F0000000000  # 16-byte aligned, never dereferenced
WS = 1 << 40


@pytest.fixture(scope="module")
def tp():
    import __graft_entry__

    __graft_entry__.build()
    import tensor_transformer_mlp_column_gb300 as tp

    return tp


def _strides(rows, pairs, change):
    s = [x for h in pairs for x in (rows * 64, 64)] if isinstance(pairs, list) else None
    for i, v in (change or {}).items():
        s[i] = v
    return array("q", s)


def _core(tp, back=False, q=FAKE, k=FAKE, v=FAKE, o=FAKE, lse=FAKE, do=FAKE, starts=None, T=24, batch=2, max_seq=12, heads=4,
          kv=2, dim=64, scale=0.125, causal=1, dt=1, dq=FAKE, dk=FAKE, dv=FAKE, ws=FAKE, nb=WS, strides=None, change=None):
    s = _strides(8, [1] * 8, change) if strides is None else strides
    p = s.buffer_info()[0] if s is not False else None
    l = tp.lib()
    if back:
        rc = l.tpmlp_attn_core_backward(q, k, v, o, lse, do, p, starts, T, batch, max_seq, heads, kv, dim, scale, causal, dt,
                                        dq, dk, dv, ws, nb, None)
    else:
        rc = l.tpmlp_attn_core_forward(q, k, v, p, starts, T, batch, max_seq, heads, kv, dim, scale, causal, dt, o, lse, None)
    return tp.STATUS_NAMES[rc]


CORE = [
    (dict(T=-1), "TPMLP_ERR_ARG"),
    (dict(T=(1 << 30) + 1), "TPMLP_ERR_ARG"),
    (dict(heads=0), "TPMLP_ERR_ARG"),
    (dict(heads=5000, kv=5000), "TPMLP_ERR_ARG"),
    (dict(kv=0), "TPMLP_ERR_ARG"),
    (dict(kv=3), "TPMLP_ERR_DIVISIBILITY"),
    (dict(kv=8), "TPMLP_ERR_DIVISIBILITY"),
    (dict(dim=0), "TPMLP_ERR_SHAPE"),
    (dict(dim=60), "TPMLP_ERR_SHAPE"),
    (dict(dim=136), "TPMLP_ERR_SHAPE"),
    (dict(dt=2), "TPMLP_ERR_ARG"),
    (dict(batch=-1), "TPMLP_ERR_ARG"),
    (dict(max_seq=-1), "TPMLP_ERR_ARG"),
    (dict(max_seq=25), "TPMLP_ERR_ARG"),
    (dict(batch=3), "TPMLP_ERR_ARG"),                    # 3 * 12 != 24 without starts
    (dict(starts=FAKE + 2), "TPMLP_ERR_ALIGN"),
    (dict(starts=FAKE, batch=1 << 30, max_seq=24, heads=64), "TPMLP_ERR_ARG"),
    (dict(scale=0.0), "TPMLP_ERR_ARG"),
    (dict(scale=-1.0), "TPMLP_ERR_ARG"),
    (dict(scale=math.inf), "TPMLP_ERR_ARG"),
    (dict(scale=math.nan), "TPMLP_ERR_ARG"),
    (dict(strides=False), "TPMLP_ERR_ARG"),
    (dict(q=None), "TPMLP_ERR_ARG"),
    (dict(k=None), "TPMLP_ERR_ARG"),
    (dict(v=None), "TPMLP_ERR_ARG"),
    (dict(o=None), "TPMLP_ERR_ARG"),
    (dict(lse=None), "TPMLP_ERR_ARG"),
    (dict(q=FAKE + 8), "TPMLP_ERR_ALIGN"),
    (dict(v=FAKE + 2), "TPMLP_ERR_ALIGN"),
    (dict(lse=FAKE + 2), "TPMLP_ERR_ALIGN"),
    (dict(change={0: 516}), "TPMLP_ERR_ALIGN"),          # bf16 rows off 16 bytes
    (dict(change={0: 514}, dt=0), "TPMLP_ERR_ALIGN"),
    (dict(change={3: 0}), "TPMLP_ERR_ALIGN"),            # a broadcast kv head
    (dict(change={0: 0}), "TPMLP_ERR_ALIGN"),
    (dict(change={0: -512}), "TPMLP_ERR_ALIGN"),
    (dict(change={0: 128}), "TPMLP_ERR_ARG"),            # the tokens' rows overlap
    (dict(change={7: 32}), "TPMLP_ERR_ARG"),             # the heads' rows overlap
    (dict(change={0: 1 << 40}), "TPMLP_ERR_ALIGN"),
    (dict(T=0, batch=1, max_seq=0, q=None, o=None, lse=None, strides=False), "TPMLP_OK"),
    (dict(T=0, batch=0, max_seq=0, q=None, o=None, lse=None, strides=False), "TPMLP_OK"),
    (dict(starts=FAKE, batch=0, q=None), "TPMLP_OK"),
]


@pytest.mark.parametrize("kw,code", CORE)
def test_forward_argument_errors(tp, kw, code):
    assert _core(tp, **kw) == code, tp.tpmlp_last_error()


@pytest.mark.parametrize("kw,code", CORE + [
    (dict(do=None), "TPMLP_ERR_ARG"),
    (dict(dq=None), "TPMLP_ERR_ARG"),
    (dict(dk=FAKE + 8), "TPMLP_ERR_ALIGN"),
    (dict(dv=None), "TPMLP_ERR_ARG"),
    (dict(ws=None), "TPMLP_ERR_ARG"),
    (dict(ws=FAKE + 8), "TPMLP_ERR_ALIGN"),
    (dict(nb=16), "TPMLP_ERR_WORKSPACE"),
    (dict(change={14: 64}), "TPMLP_ERR_ARG"),
])
def test_backward_argument_errors(tp, kw, code):
    assert _core(tp, back=True, **kw) == code, tp.tpmlp_last_error()


def test_strides_of_one_token_or_head_do_not_count(tp):
    # A single head's head stride and a single token's token stride may be anything: the next check is reached.
    one = array("q", [512, 3] * 8)
    assert _core(tp, strides=one, heads=1, kv=1, lse=None) == "TPMLP_ERR_ARG" and "lse" in tp.tpmlp_last_error()
    one = array("q", [3, 64] * 8)
    assert _core(tp, strides=one, T=1, batch=1, max_seq=1, lse=None) == "TPMLP_ERR_ARG" and "lse" in tp.tpmlp_last_error()


def _rope(tp, back=False, q=FAKE, k=FAKE, wq=FAKE, wk=FAKE, eps=1e-6, pos=FAKE, freqs=(1.0,) * 32, axis=None, T=24, heads=4,
          kv=2, dim=64, rot=64, axes=1, inter=0, dt=1, yq=FAKE, yk=FAKE, dyq=FAKE, dyk=FAKE, dwq=FAKE, dwk=FAKE, ws=FAKE,
          nb=WS, change=None, strides=None):
    s = _strides(8, [1] * 6, change) if strides is None else strides
    f = None if freqs is None else array("d", freqs)
    a = None if axis is None else array("B", axis)
    common = (q, k, s.buffer_info()[0], wq, wk, eps, pos, None if f is None else f.buffer_info()[0],
              None if a is None else a.buffer_info()[0], T, heads, kv, dim, rot, axes, inter, dt, yq, yk)
    l = tp.lib()
    rc = l.tpmlp_qk_rope_backward(dyq, dyk, *common, dwq, dwk, ws, nb, None) if back else l.tpmlp_qk_rope_forward(*common, None)
    return tp.STATUS_NAMES[rc]


ROPE = [
    (dict(T=-1), "TPMLP_ERR_ARG"),
    (dict(heads=0), "TPMLP_ERR_ARG"),
    (dict(kv=5000), "TPMLP_ERR_ARG"),
    (dict(dim=60), "TPMLP_ERR_SHAPE"),
    (dict(dim=264), "TPMLP_ERR_SHAPE"),
    (dict(rot=60), "TPMLP_ERR_SHAPE"),
    (dict(rot=72), "TPMLP_ERR_SHAPE"),
    (dict(rot=-8), "TPMLP_ERR_SHAPE"),
    (dict(axes=0), "TPMLP_ERR_ARG"),
    (dict(axes=9), "TPMLP_ERR_ARG"),
    (dict(axis=[0] * 31 + [1]), "TPMLP_ERR_ARG"),
    (dict(axis=[0] * 31 + [3], axes=3), "TPMLP_ERR_ARG"),
    (dict(freqs=None), "TPMLP_ERR_ARG"),
    (dict(freqs=(1.0,) * 31 + (math.inf,)), "TPMLP_ERR_ARG"),
    (dict(freqs=(math.nan,) * 32), "TPMLP_ERR_ARG"),
    (dict(wq=None), "TPMLP_ERR_ARG"),
    (dict(wk=None), "TPMLP_ERR_ARG"),
    (dict(wq=FAKE + 8), "TPMLP_ERR_ALIGN"),
    (dict(eps=-1.0), "TPMLP_ERR_ARG"),
    (dict(eps=math.nan), "TPMLP_ERR_ARG"),
    (dict(pos=None), "TPMLP_ERR_ARG"),
    (dict(pos=FAKE + 4), "TPMLP_ERR_ALIGN"),
    (dict(dt=7), "TPMLP_ERR_ARG"),
    (dict(q=None), "TPMLP_ERR_ARG"),
    (dict(yk=None), "TPMLP_ERR_ARG"),
    (dict(k=FAKE + 8), "TPMLP_ERR_ALIGN"),
    (dict(change={2: 516}), "TPMLP_ERR_ALIGN"),
    (dict(change={0: 64}), "TPMLP_ERR_ARG"),
]


@pytest.mark.parametrize("kw,code", ROPE + [(dict(T=0, q=None, pos=None, yq=None), "TPMLP_OK")])
def test_rope_forward_argument_errors(tp, kw, code):
    assert _rope(tp, **kw) == code, tp.tpmlp_last_error()


@pytest.mark.parametrize("kw,code", ROPE + [
    (dict(dyq=None), "TPMLP_ERR_ARG"),
    (dict(dyk=FAKE + 8), "TPMLP_ERR_ALIGN"),
    (dict(dwq=None), "TPMLP_ERR_ARG"),
    (dict(dwk=FAKE + 2), "TPMLP_ERR_ALIGN"),
    (dict(ws=None), "TPMLP_ERR_ARG"),
    (dict(ws=FAKE + 8), "TPMLP_ERR_ALIGN"),
    (dict(nb=16), "TPMLP_ERR_WORKSPACE"),
    (dict(T=0, wq=None, wk=None, q=None, dwq=None, ws=None), "TPMLP_OK"),  # no weights: nothing to clear
])
def test_rope_backward_argument_errors(tp, kw, code):
    assert _rope(tp, back=True, **kw) == code, tp.tpmlp_last_error()


def test_rope_in_place_needs_the_same_strides(tp):
    # (token, head) of q, k, (dyq, dyk,) and the outputs, of which every address is the same here.
    for back, n, places in ((False, 4, (0, 2, 4, 6)), (True, 6, (0, 2, 4, 6, 8, 10))):
        for i in places:
            s = array("q", [512, 64] * n)
            s[i] = 1024
            assert _rope(tp, back, strides=s) == "TPMLP_ERR_ARG" and "place" in tp.tpmlp_last_error()


def test_many_sequences_of_no_stated_length(tp):
    # What counts is the tiles that T rows can have, not max_seq for every sequence.
    l = tp.lib()
    assert l.tpmlp_attn_core_workspace_bytes(1 << 18, 1 << 14, 1 << 18, 32, 8, 64, 1) > 0
    assert l.tpmlp_attn_core_workspace_bytes(1 << 18, 1 << 14, 1 << 18, 32, 8, 64, 0) > 0
    assert l.tpmlp_attn_core_workspace_bytes(1 << 18, 1 << 28, 1 << 18, 32, 8, 64, 0) == 0


def test_workspace_sizes(tp):
    l = tp.lib()
    core = l.tpmlp_attn_core_workspace_bytes
    assert core(0, 1, 0, 4, 2, 64, 1) == 0 and core(100, 1, 100, 4, 3, 64, 1) == 0 and core(100, 1, 100, 4, 2, 60, 1) == 0
    assert core(100, 1, 100, 4, 2, 64, 5) == 0 and core(-1, 1, 0, 4, 2, 64, 1) == 0 and core(100, 1, 101, 4, 2, 64, 1) == 0
    assert core(100, -1, 100, 4, 2, 64, 1) == 0 and core(100, 0, 100, 4, 2, 64, 1) == 0
    assert core(100, 1, 100, 4, 2, 64, 1) >= 1600 and core(100, 2, 50, 4, 2, 64, 0) == 1792
    assert core(1 << 20, 1, 1 << 20, 32, 32, 128, 1) == 128 << 20
    rope = l.tpmlp_qk_rope_workspace_bytes
    assert rope(0, 4, 2, 64) == 0 and rope(10, 4, 2, 65) == 0 and rope(10, 0, 2, 64) == 0
    assert rope(1, 4, 2, 64) == 512
    assert rope(1 << 20, 32, 8, 128) <= 1 << 20


@pytest.mark.parametrize("kw", [dict(load=0), dict(limit=0), dict(limit=10001), dict(T=0), dict(dim=60), dict(heads=0),
                                dict(nb=0, backward=1)])
def test_timeout_hook_refuses(tp, kw):
    a = dict(T=300, heads=2, dim=64, backward=0, load=1, limit=50, nb=WS)
    a.update(kw)
    assert tp.lib().tpmlp_selftest_attn_core_timeout(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, a["T"], a["heads"], a["dim"], FAKE,
                                                     FAKE, FAKE, FAKE, a["nb"], a["backward"], a["load"], a["limit"],
                                                     None) < 0


def test_binding_refuses(tp):
    import torch

    T, H, K, D = 6, 4, 2, 64
    f = [1.0] * 32
    q, k = torch.zeros(T, H, D), torch.zeros(T, K, D)
    pos = torch.zeros(T, dtype=torch.int64)
    with pytest.raises(ValueError):
        tp._qkv_shape(q[0], k)
    with pytest.raises(TypeError):
        tp.tpmlp_attn_core_forward(q.double(), k.double(), k.double())
    s = []
    with pytest.raises(ValueError, match="shape"):
        tp._heads(k, T, H, D, torch.float32, 0, s, "k")
    with pytest.raises(ValueError, match="torch.bfloat16"):
        tp._heads(q, T, H, D, torch.bfloat16, 0, s, "q")
    with pytest.raises(ValueError, match="is on cpu"):
        tp._heads(q, T, H, D, torch.float32, 0, s, "q")
    with pytest.raises(ValueError, match="equal sequences"):
        tp._sequences(None, None, 4, T, 0)
    with pytest.raises(ValueError, match="equal sequences"):
        tp._sequences(None, 2, 2, T, 0)
    with pytest.raises(ValueError, match="int32"):
        tp._sequences(torch.zeros(3, dtype=torch.int64), None, None, T, 0)
    with pytest.raises(ValueError, match="disagree"):
        tp._sequences(torch.zeros(3, dtype=torch.int32), None, 3, T, 0)
    with pytest.raises(ValueError, match="axis"):
        tp._turns((1.0, 2.0), (0,), 1)
    with pytest.raises(ValueError, match="axis"):
        tp._turns((1.0, 2.0), (0, 2), 2)
    with pytest.raises(ValueError, match="positions"):
        tp._rope_args(q, k, pos[:3], f, None, False, None, None, 1e-6, 0)
    with pytest.raises(ValueError, match="positions"):
        tp._rope_args(q, k, pos.int(), f, None, False, None, None, 1e-6, 0)
    assert tp._turns((1.0, 2.0), (0, 1), 2)[0].tolist() == [1.0, 2.0]


def test_frequencies_of_any_kind(tp):
    import numpy as np
    import torch

    # Lists, tuples, arrays and tensors, one after another and again: the values count, not where they stand.
    q, k, pos = torch.zeros(6, 4, 64), torch.zeros(6, 2, 64), torch.zeros(2, 6, dtype=torch.int64)

    def made(f, a):
        keep = tp._rope_args(q, k, pos, f, a, False, None, None, 1e-6, -1)[2]
        return keep[0].tolist(), None if keep[1] is None else keep[1].tolist()

    f, a = [2.0 ** -i for i in range(16)], [i % 2 for i in range(16)]
    for ff, aa in [(f, a), (np.array(f), a), (f, np.array(a)), (torch.tensor(f), torch.tensor(a)), (tuple(f), tuple(a)),
                   (np.array(f, np.float32), None), (f, a)] * 2:
        assert made(ff, aa) == (f, None if aa is None else a)
    f[3] = 0.5
    assert made(f, a) == (f, a)
    a[3] = 0
    assert made(f, a) == (f, a)
    with pytest.raises(ValueError, match="axis"):
        tp._turns((1.0, 2.0), (0, 299), 300)


def test_sizes_of_no_sequences_and_hook_shapes(tp):
    import torch

    assert tp.tpmlp_attn_core_workspace_bytes(16, 4, 2, 64, torch.bfloat16, batch=0) == 0
    q = torch.zeros(6, 4, 64, dtype=torch.bfloat16)
    for k in (q[:5], q.float(), q[0]):
        with pytest.raises(ValueError, match="one shape"):
            tp.tpmlp_selftest_attn_core_timeout(q, k, q, False, 1, 50)


def test_one_token_of_a_large_layout(tp):
    # One token of [heads, tokens, 64]: the head stride is large, and no other one counts.
    for head in (1 << 20, 1 << 33):
        one = array("q", [8, head] * 8)
        rc = _core(tp, strides=one, T=1, batch=1, max_seq=1, heads=64, kv=64, lse=None)
        assert rc == "TPMLP_ERR_ARG" and "lse" in tp.tpmlp_last_error()
    assert _core(tp, strides=array("q", [64, 1 << 62] * 8), T=1, batch=1, max_seq=1) == "TPMLP_ERR_ALIGN"
    assert _core(tp, strides=array("q", [64, 56] * 8), T=1, batch=1, max_seq=1) == "TPMLP_ERR_ARG"


def test_frequencies_changed_in_place(tp):
    import numpy as np
    import torch

    # Elements that are views (0-dim tensors, arrays) change with their tensor: every call takes the values of its time.
    q, k, pos = torch.zeros(6, 4, 64), torch.zeros(6, 2, 64), torch.zeros(2, 6, dtype=torch.int64)

    def made(f, a):
        keep = tp._rope_args(q, k, pos, f, a, False, None, None, 1e-6, -1)[2]
        return keep[0].tolist(), None if keep[1] is None else keep[1].tolist()

    want = [2.0 ** -i for i in range(16)]
    for make in (lambda: torch.tensor(want), lambda: torch.tensor(want, dtype=torch.float64)):
        for kind in (list, tuple):
            t, a = make(), torch.arange(16) % 2
            f, ax = kind(t), kind(a)
            assert made(f, ax) == (want, [i % 2 for i in range(16)])
            t.mul_(0.5)
            a[0] = 1
            half = ([0.5 * w for w in want], [1] + [i % 2 for i in range(1, 16)])
            assert made(kind(t), kind(a)) == half  # new views of the same memory
            assert made(f, ax) == half             # the same list as before
    f = [np.array(w) for w in want]
    assert made(f, None)[0] == want
    f[2][...] = 9.0
    assert made(f, None)[0] == want[:2] + [9.0] + want[3:]
    # Numbers that compare equal in 32 bits but are not: 0.1 and the nearest 32-bit number.
    assert made([0.1] * 4, None)[0] == [0.1] * 4
    assert made(list(np.full(4, 0.1, np.float32)), None)[0] == [float(np.float32(0.1))] * 4
    assert made([0.1] * 4, None)[0] == [0.1] * 4


@pytest.mark.parametrize("name,least", [("attn_core.cu", 1), ("attn_core_tc.cu", 6), ("attn_core_walk.cuh", 1), ("qk_rope.cu", 2)])
def test_debug_checks_stand_in_the_kernels(name, least):
    # Items and shared-memory areas, sums of runs, elements of heads: what the debug build is said to check.
    import os
    import re

    csrc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "tensor_transformer_mlp_column_gb300", "csrc")
    with open(os.path.join(csrc, name)) as f:
        text = f.read()
    assert len(re.findall(r"\b(?:TPMLP_DCHECK|in_bounds|fits|part_exists)\(", text)) >= least


def test_axes_by_value(tp):
    import torch

    q, k, pos = torch.zeros(6, 4, 64), torch.zeros(6, 2, 64), torch.zeros(2, 6, dtype=torch.int64)

    def made(a):
        return tp._rope_args(q, k, pos, [1.0] * 4, a, False, None, None, 1e-6, -1)[2][1]

    for _ in range(2):
        assert made(None) is None
        for bad in ([], [0], [0, 0, 0, 2], [0, 0, 0, -1], [0, 0, 0, 300], [0, 0, 0, 2 ** 70], [0] * 5):
            with pytest.raises(ValueError, match="axis"):
                made(bad)
        for a in ([0, 1, 0, 1], (0, 1, 0, 1), [0.0, 1.0, 0.0, 1.0], torch.tensor([0, 1, 0, 1]), list(torch.tensor([0, 1, 0, 1])),
                  [False, True, False, True]):
            assert made(a).tolist() == [0, 1, 0, 1]
        assert made([1, 1, 0, 0]).tolist() == [1, 1, 0, 0]
