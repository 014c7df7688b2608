"""Refusals of the calls at the two ends of a training step (embedding, cross
entropy over the vocabulary, gradient clipping): argument checks that run
before any CUDA call, through the C ABI with addresses that are never
dereferenced, and the binding's own checks."""

import ctypes

import pytest
import torch

FAKE = 0x7F0000000000  # 16-byte aligned, never dereferenced
WS = 1 << 40


@pytest.fixture(scope="module")
def tp():
    import __graft_entry__

    __graft_entry__.build()
    import tensor_transformer_mlp_column_gb300 as tp

    return tp


def _xent_forward(tp, X=FAKE, W=FAKE, t=FAKE, T=8, D=64, V=100, dt=1, loss=FAKE, lse=FAKE, ws=FAKE, nb=WS):
    return tp.STATUS_NAMES[tp.lib().tpmlp_xent_forward(X, W, t, T, D, V, dt, loss, lse, ws, nb, None)]


def _xent_backward(tp, X=FAKE, W=FAKE, t=FAKE, lse=FAKE, dloss=FAKE, T=8, D=64, V=100, dt=1, dX=FAKE, dW=FAKE, ws=FAKE,
                   nb=WS):
    return tp.STATUS_NAMES[tp.lib().tpmlp_xent_backward(X, W, t, lse, dloss, T, D, V, dt, dX, dW, ws, nb, None)]


def _embed_forward(tp, E=FAKE, ids=FAKE, T=8, D=64, V=100, dt=1, out=FAKE):
    return tp.STATUS_NAMES[tp.lib().tpmlp_embed_forward(E, ids, T, D, V, dt, 1.0, out, None)]


def _embed_backward(tp, dout=FAKE, ddt=1, ids=FAKE, T=8, D=64, V=100, dE=FAKE, edt=1, acc=0, ws=FAKE, nb=WS):
    return tp.STATUS_NAMES[tp.lib().tpmlp_embed_backward(dout, ddt, ids, T, D, V, 1.0, dE, edt, acc, ws, nb, None)]


SIZES = [
    (dict(T=-1), "TPMLP_ERR_ARG"),
    (dict(T=(1 << 30) + 1), "TPMLP_ERR_ARG"),
    (dict(D=0), "TPMLP_ERR_ARG"),
    (dict(D=(1 << 20) + 8), "TPMLP_ERR_ARG"),
    (dict(V=0), "TPMLP_ERR_ARG"),
    (dict(V=(1 << 30) + 1), "TPMLP_ERR_ARG"),
]


@pytest.mark.parametrize("kw,code", SIZES + [
    (dict(dt=2), "TPMLP_ERR_ARG"),
    (dict(D=60), "TPMLP_ERR_SHAPE"),
    (dict(D=4, dt=0), "TPMLP_ERR_SHAPE"),
    (dict(X=None), "TPMLP_ERR_ARG"),
    (dict(W=None), "TPMLP_ERR_ARG"),
    (dict(t=None), "TPMLP_ERR_ARG"),
    (dict(loss=None), "TPMLP_ERR_ARG"),
    (dict(lse=None), "TPMLP_ERR_ARG"),
    (dict(ws=None), "TPMLP_ERR_ARG"),
    (dict(X=FAKE + 2), "TPMLP_ERR_ALIGN"),
    (dict(t=FAKE + 4), "TPMLP_ERR_ALIGN"),
    (dict(lse=FAKE + 2), "TPMLP_ERR_ALIGN"),
    (dict(nb=0), "TPMLP_ERR_WORKSPACE"),
    (dict(T=0, X=None, loss=None, ws=None, nb=0), "TPMLP_OK"),  # no rows: nothing enqueued
])
def test_xent_forward_argument_errors(tp, kw, code):
    assert _xent_forward(tp, **kw) == code, tp.tpmlp_last_error()


@pytest.mark.parametrize("kw,code", SIZES + [
    (dict(dt=-1), "TPMLP_ERR_ARG"),
    (dict(D=12), "TPMLP_ERR_SHAPE"),
    (dict(dX=None), "TPMLP_ERR_ARG"),
    (dict(dW=None), "TPMLP_ERR_ARG"),
    (dict(dW=None, T=0), "TPMLP_ERR_ARG"),
    (dict(dloss=None), "TPMLP_ERR_ARG"),
    (dict(dW=FAKE + 8), "TPMLP_ERR_ALIGN"),
    (dict(dloss=FAKE + 2), "TPMLP_ERR_ALIGN"),
    (dict(nb=16), "TPMLP_ERR_WORKSPACE"),
])
def test_xent_backward_argument_errors(tp, kw, code):
    assert _xent_backward(tp, **kw) == code, tp.tpmlp_last_error()


@pytest.mark.parametrize("kw,code", SIZES + [
    (dict(dt=3), "TPMLP_ERR_ARG"),
    (dict(E=None), "TPMLP_ERR_ARG"),
    (dict(ids=None), "TPMLP_ERR_ARG"),
    (dict(out=None), "TPMLP_ERR_ARG"),
    (dict(out=FAKE + 8), "TPMLP_ERR_ALIGN"),
    (dict(T=0, ids=None, out=None), "TPMLP_OK"),
])
def test_embed_forward_argument_errors(tp, kw, code):
    assert _embed_forward(tp, **kw) == code, tp.tpmlp_last_error()


@pytest.mark.parametrize("kw,code", SIZES + [
    (dict(ddt=3), "TPMLP_ERR_ARG"),
    (dict(edt=3), "TPMLP_ERR_ARG"),
    (dict(dE=None), "TPMLP_ERR_ARG"),
    (dict(dE=None, T=0), "TPMLP_ERR_ARG"),
    (dict(dout=None), "TPMLP_ERR_ARG"),
    (dict(ids=FAKE + 4), "TPMLP_ERR_ALIGN"),
    (dict(dE=FAKE + 4), "TPMLP_ERR_ALIGN"),
    (dict(nb=8), "TPMLP_ERR_WORKSPACE"),
    (dict(T=0, acc=1, dout=None, ids=None, ws=None, nb=0), "TPMLP_OK"),  # adds nothing
])
def test_embed_backward_argument_errors(tp, kw, code):
    assert _embed_backward(tp, **kw) == code, tp.tpmlp_last_error()


def test_workspace_sizes(tp):
    l = tp.lib()
    assert l.tpmlp_xent_workspace_bytes(0, 64, 100, 1, 0) == 0
    assert l.tpmlp_xent_workspace_bytes(8, 60, 100, 1, 0) == 0
    assert l.tpmlp_xent_workspace_bytes(8, 64, 100, 1, 2) == 0
    # The logits never exist: forward takes 8 bytes per 128 of them.
    T, D, V = 8192, 4096, 128000
    assert T * V / 16 <= l.tpmlp_xent_workspace_bytes(T, D, V, 1, 0) <= T * V / 16 + 4 * T + 1024
    # Backward holds a piece of dz (at most 512 MB here) and sums of dX.
    assert l.tpmlp_xent_workspace_bytes(T, D, V, 1, 1) < (1 << 29) + 64 * T * D
    assert l.tpmlp_embed_workspace_bytes(0, 64, 100) == 0
    assert l.tpmlp_embed_workspace_bytes(100, 64, 0) == 0
    assert l.tpmlp_embed_workspace_bytes(100, 64, 10) >= 1600
    assert l.tpmlp_grad_workspace_bytes(-1) == 0
    assert l.tpmlp_grad_workspace_bytes(0) == l.tpmlp_grad_workspace_bytes(1) > 0
    assert l.tpmlp_grad_workspace_bytes(10000) > l.tpmlp_grad_workspace_bytes(1)


def _clip(tp, grads, counts, dts, n=None, max_norm=1.0, out=None, norm=FAKE - 4096, ws=FAKE - 8192, nb=WS, clip=True):
    P = ctypes.c_void_p
    k = len(grads)
    g, c, d = (P * k)(*grads), (ctypes.c_int64 * k)(*counts), (ctypes.c_int * k)(*dts)
    o = None if out is None else (P * k)(*out)
    n = k if n is None else n
    if clip:
        return tp.STATUS_NAMES[tp.lib().tpmlp_grad_clip(g, c, d, n, max_norm, o, norm, ws, nb, None)]
    return tp.STATUS_NAMES[tp.lib().tpmlp_grad_norm(g, c, d, n, norm, ws, nb, None)]


def test_clip_argument_errors(tp):
    ok = dict(grads=[FAKE, FAKE + 4096], counts=[16, 16], dts=[0, 1])
    assert _clip(tp, **ok, n=-1) == "TPMLP_ERR_ARG"
    assert _clip(tp, [FAKE], [-1], [0]) == "TPMLP_ERR_ARG"
    assert _clip(tp, [FAKE], [4], [7]) == "TPMLP_ERR_ARG"
    assert _clip(tp, [None], [4], [0]) == "TPMLP_ERR_ARG"
    assert _clip(tp, [FAKE + 4], [4], [0]) == "TPMLP_ERR_ALIGN"
    assert _clip(tp, [FAKE], [4], [0], out=[None]) == "TPMLP_ERR_ARG"
    assert _clip(tp, [FAKE], [4], [0], out=[FAKE + 8]) == "TPMLP_ERR_ALIGN"
    for bad in (-1.0, float("nan"), float("inf")):
        assert _clip(tp, **ok, max_norm=bad) == "TPMLP_ERR_ARG"
    assert _clip(tp, **ok, norm=None) == "TPMLP_ERR_ARG"
    assert _clip(tp, **ok, ws=None) == "TPMLP_ERR_ARG"
    assert _clip(tp, **ok, norm=FAKE - 4094) == "TPMLP_ERR_ALIGN"
    assert _clip(tp, **ok, nb=8) == "TPMLP_ERR_WORKSPACE"
    assert _clip(tp, **ok, nb=8, clip=False) == "TPMLP_ERR_WORKSPACE"
    assert _clip(tp, [FAKE], [4], [7], clip=False) == "TPMLP_ERR_ARG"


def test_clip_refuses_overlapping_tensors(tp):
    # The same tensor twice, a part of another one, and an output over another tensor.
    f32 = [0, 0]
    assert _clip(tp, [FAKE, FAKE], [16, 16], f32) == "TPMLP_ERR_ARG"
    assert _clip(tp, [FAKE, FAKE + 32], [16, 4], f32) == "TPMLP_ERR_ARG"
    assert _clip(tp, [FAKE + 32, FAKE], [4, 16], f32) == "TPMLP_ERR_ARG"
    assert "overlaps" in tp.tpmlp_last_error()
    a, b = FAKE, FAKE + 4096
    assert _clip(tp, [a, b], [16, 16], f32, out=[b, b + 4096]) == "TPMLP_ERR_ARG"
    assert _clip(tp, [a, b], [16, 16], f32, out=[a + 8192, a + 8192]) == "TPMLP_ERR_ARG"
    if torch.cuda.is_available():
        return
    # These are sound: they get as far as the missing device.
    for kw in (dict(), dict(out=[a, b]), dict(out=[a + 8192, b + 8192])):
        assert _clip(tp, [a, b], [16, 16], f32, **kw) in ("TPMLP_ERR_CUDA", "TPMLP_ERR_DEVICE")
    # Reading the same tensor twice for the norm alone is sound too.
    assert _clip(tp, [a, a], [16, 16], f32, clip=False) in ("TPMLP_ERR_CUDA", "TPMLP_ERR_DEVICE")
    # An empty tensor's pointer is not looked at.
    assert _clip(tp, [a, None], [16, 0], f32) in ("TPMLP_ERR_CUDA", "TPMLP_ERR_DEVICE")


def test_calls_without_a_gpu_report_errors(tp):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    bad = ("TPMLP_ERR_CUDA", "TPMLP_ERR_DEVICE")
    assert _xent_forward(tp) in bad
    assert _xent_backward(tp) in bad
    assert _xent_backward(tp, T=0) in bad  # clears dW
    assert _embed_forward(tp) in bad
    assert _embed_backward(tp) in bad
    assert _embed_backward(tp, T=0) in bad


@pytest.mark.parametrize("kw,code", SIZES + [
    (dict(loss=None), "TPMLP_ERR_ARG"),
    (dict(loss=FAKE + 2), "TPMLP_ERR_ALIGN"),
    (dict(lse=None), "TPMLP_ERR_ARG"),
    (dict(dloss=FAKE + 2), "TPMLP_ERR_ALIGN"),
    (dict(D=12), "TPMLP_ERR_SHAPE"),
    (dict(dW=None, T=0), "TPMLP_ERR_ARG"),
    (dict(nb=16), "TPMLP_ERR_WORKSPACE"),
])
def test_xent_backward_saved_argument_errors(tp, kw, code):
    a = dict(X=FAKE, W=FAKE, t=FAKE, loss=FAKE, lse=FAKE, dloss=FAKE, T=8, D=64, V=100, dt=1, dX=FAKE, dW=FAKE, ws=FAKE, nb=WS)
    a.update(kw)
    assert tp.STATUS_NAMES[tp.lib().tpmlp_xent_backward_saved(*a.values(), None)] == code, tp.tpmlp_last_error()


@pytest.mark.parametrize("kw,code", SIZES + [
    (dict(T=0), "TPMLP_ERR_ARG"),
    (dict(stage=0), "TPMLP_ERR_ARG"),
    (dict(stage=4), "TPMLP_ERR_ARG"),
    (dict(limit_ms=0), "TPMLP_ERR_ARG"),
    (dict(limit_ms=10001), "TPMLP_ERR_ARG"),
    (dict(lse=None), "TPMLP_ERR_ARG"),
    (dict(X=FAKE + 2), "TPMLP_ERR_ALIGN"),
    (dict(nb=0), "TPMLP_ERR_WORKSPACE"),
])
def test_xent_stage_timeout_argument_errors(tp, kw, code):
    a = dict(X=FAKE, W=FAKE, t=FAKE, T=8, D=64, V=100, dt=1, loss=FAKE, lse=FAKE, stage=1, limit_ms=100, ws=FAKE, nb=WS)
    a.update(kw)
    assert tp.STATUS_NAMES[tp.lib().tpmlp_selftest_xent_stage_timeout(*a.values(), None)] == code, tp.tpmlp_last_error()


@pytest.mark.parametrize("dt", [0, 1])
@pytest.mark.parametrize("T,D,V", [(1, 64, 100), (64, 4096, 2000), (64, 8, 100000), (8192, 512, 300), (192, 1024, 64000),
                                   (300, 4096, 5000), (34000, 16, 9000), (4096, 768, 50257), (65, 1 << 15, 300)])
def test_xent_backward_workspace_is_within_what_the_header_says(tp, T, D, V, dt):
    got = tp.lib().tpmlp_xent_workspace_bytes(T, D, V, dt, 1)
    planes = 3 if dt == 0 else 2 if T <= 64 else 1
    few = T <= (192 if dt == 0 else 64)
    C = min(V, max(8192, 2 ** 28 // (T * planes)))
    dz = T * C * 2 * planes
    copies = 6 * (T + V) * (D + 64) if dt == 0 else 2 * T * (D + 64)
    s = max(64, 1 + 512 * 152 // D) if few else 64
    # Rows of whole 64 columns, partial sums of whole 32 rows, parts on 256 bytes.
    assert got <= copies + dz + 64 * 2 * planes * T + s * (T + 32) * D * 4 + 64 * (C + 32) * D * 4 + 4096
    assert got >= dz - 256 * 2 * planes * T + (T * D * 4 if few or C < V else 0)
