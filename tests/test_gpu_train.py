"""The two ends of a training step on the GPU, against their definitions in 64
bits: the cross entropy over the vocabulary with its gradients, the embedding
lookup with its gradient, the gradients' global norm and clipping; and a whole
step of them around the library's block.

Tolerances are bounds by arithmetic, element by element. U16 = 2^-8 is half a
step of bf16 relative to the value, U32 = 2^-24 of fp32. A tensor-core sum adds
16 products at a time to an fp32 accumulator that is rounded (possibly
truncated: a whole step, 2 U32) each time.
"""

import math

import pytest
import torch

pytestmark = pytest.mark.gpu

U16, U32 = 2.0 ** -8, 2.0 ** -24


@pytest.fixture(scope="module")
def tp():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()
    import tensor_transformer_mlp_column_gb300 as tp

    torch.cuda.set_device(0)
    return tp


DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _close(got, ref, tol, what):
    err = (got.double() - ref).abs()
    worst = (err / tol.clamp(min=1e-300)).max().item() if err.numel() else 0.0
    assert bool((err <= tol).all()), f"{what}: worst error is {worst:.3g} of its bound"


# ------------------------------------------------------------------ cross entropy


def _xent_inputs(T, D, V, dtype, seed, masked=0.1, sure=12.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    W = (torch.randn(V, D, generator=g, device="cuda") / math.sqrt(D)).to(DT[dtype])
    t = torch.randint(0, V, (T,), generator=g, device="cuda")
    u = torch.rand(T, 1, generator=g, device="cuda") * sure
    X = (torch.randn(T, D, generator=g, device="cuda") + u * W[t].float()).to(DT[dtype])
    t[torch.rand(T, generator=g, device="cuda") < masked] = -100
    dloss = torch.rand(T, generator=g, device="cuda") - 0.3
    return X, W, t, dloss


def _xent_reference(X, W, t, dloss):
    x, w, on = X.double(), W.double(), (t >= 0) & (t < W.shape[0])
    at = torch.where(on, t, torch.zeros_like(t))
    z = x @ w.T
    lse = torch.logsumexp(z, 1)
    loss = torch.where(on, lse - z.gather(1, at[:, None])[:, 0], torch.zeros_like(lse))
    dz = torch.exp(z - lse[:, None])
    dz[torch.arange(len(t), device="cuda"), at] -= 1
    dz = dz * torch.where(on, dloss.double(), torch.zeros_like(lse))[:, None]
    return z, lse, loss, dz


def _sum_bound(k, dtype):
    """Relative (to the sum of magnitudes) bound of a tensor-core sum over k products."""
    if dtype == "bf16":
        return (k / 16 + 2) * 2 * U32
    # Three planes: the dropped products are below 3 * 2^-24, six products are summed.
    return (6 * k / 16 + 2) * 2 * U32 + 4 * U32


def _check_xent(tp, X, W, t, dloss, dtype):
    T, D = X.shape
    V = W.shape[0]
    z, lse, loss, dz = _xent_reference(X, W, t, dloss)
    got_loss, got_lse = tp.tpmlp_xent_forward(X, W, t)
    # Logits: their own sums; the exponentials and logarithms add a few U32 of the exponents' size.
    mag = (X.double().abs() @ W.double().abs().T).max(dim=1).values
    ez = mag * _sum_bound(D, dtype) + 8 * U32 * (z.abs().max(dim=1).values + 1)
    el = ez + (V / 128 + 64) * 2 * U32 + 4 * U32 * lse.abs()
    _close(got_lse, lse, el, "lse")
    _close(got_loss, loss, ez + el + U32 * loss.abs(), "loss")
    off = (t < 0) | (t >= V)
    assert bool((got_loss[off] == 0).all())

    dX, dW = tp.tpmlp_xent_backward(X, W, t, got_lse, dloss)
    tp.tpmlp_check_status() if not bool((t >= V).any()) else None
    assert dX.dtype == dW.dtype == X.dtype
    # dz: relative error of the exponential from the logits and lse, then (bf16) one rounding.
    on = ~off
    p = torch.where(on[:, None], torch.exp(z - lse[:, None]) * dloss.double().abs()[:, None], torch.zeros_like(z))
    edz = p * (ez + el + 16 * U32)[:, None] * 1.01
    edz = edz + dz.abs() * ((1.01 * U16 if dtype == "bf16" else 4 * U32) + 4 * U32)
    out = U16 * 1.01 if dtype == "bf16" else 2 * U32
    ref = dz @ W.double()
    tol = edz @ W.double().abs() + (dz.abs() @ W.double().abs()) * (_sum_bound(V, dtype) + 80 * U32) + out * ref.abs()
    _close(dX, ref, tol + 1e-30, "dX")
    assert bool((dX[off] == 0).all())
    ref = dz.T @ X.double()
    tol = edz.T @ X.double().abs() + (dz.abs().T @ X.double().abs()) * (_sum_bound(T, dtype) + 80 * U32) + out * ref.abs()
    _close(dW, ref, tol + 1e-30, "dW")
    return got_loss, got_lse, dX, dW


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,D,V", [
    (1, 8, 1), (1, 64, 257), (3, 72, 31), (129, 64, 127), (257, 136, 1000), (256, 256, 256), (300, 768, 5003),
    (33, 64, 20000), (1000, 8, 130), (64, 2056, 640),
])
def test_xent_against_64_bits(tp, T, D, V, dtype):
    X, W, t, dloss = _xent_inputs(T, D, V, dtype, seed=T + D + V)
    _check_xent(tp, X, W, t, dloss, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [264, 288, 296, 320, 328, 376, 384, 392, 416, 448, 504, 512])
def test_xent_widths_of_the_last_tiles(tp, D, dtype):
    # The gradients' products have a last column of tiles of every width, in steps of 32.
    X, W, t, dloss = _xent_inputs(270, D, 520, dtype, seed=D)
    _check_xent(tp, X, W, t, dloss, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,D,V", [(600, 1032, 8300), (2100, 56, 70001), (70, 7400, 8300), (9000, 24, 30001)])
def test_xent_rows_off_the_sectors(tp, T, D, V, dtype):
    # The products read X (fp32: and W) from copies on rows of whole lines.
    X, W, t, dloss = _xent_inputs(T, D, V, dtype, seed=D)
    _check_xent(tp, X, W, t, dloss, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,D,V", [
    (1, 1000, 5000), (2, 72, 15), (3, 4104, 700), (4, 64, 16), (5, 8, 17), (7, 520, 2049), (8, 1032, 4000), (9, 72, 64),
    (16, 4096, 300), (17, 256, 1000), (31, 40, 129), (32, 768, 3000), (6, 12000, 90), (32, 6400, 200), (2, 60000, 40),
    (33, 264, 1000), (64, 1024, 2000), (65, 72, 500), (128, 136, 1300), (150, 520, 700), (193, 64, 900), (256, 48, 260),
    (257, 64, 300), (129, 4200, 4001), (192, 2048, 8200),
])
def test_xent_of_a_few_rows(tp, T, D, V, dtype):
    X, W, t, dloss = _xent_inputs(T, D, V, dtype, seed=T + D + V)
    a = _check_xent(tp, X, W, t, dloss, dtype)
    b = _check_xent(tp, X, W, t, dloss, dtype)
    assert all(torch.equal(u, v) for u, v in zip(a, b))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,D", [(64, 1024), (64, 512), (20, 512)])
def test_xent_of_a_few_rows_is_the_same_every_time(tp, dtype, T, D):
    # Several tiles a CTA, many calls: a stage of operands that is filled again while it is still being read shows in one
    # call of some thousands.
    V = 50257
    X, W, t, dloss = _xent_inputs(T, D, V, dtype, seed=T + D)
    ref = tp.tpmlp_xent_forward(X, W, t)
    gref = tp.tpmlp_xent_backward(X, W, t, ref[1], dloss)
    differs = torch.zeros((), dtype=torch.int64, device="cuda")
    for i in range(8000):
        for a, b in zip(tp.tpmlp_xent_forward(X, W, t), ref):
            differs += (a != b).any()
        if i % 4 == 0:
            for a, b in zip(tp.tpmlp_xent_backward(X, W, t, ref[1], dloss), gref):
                differs += (a != b).any()
    assert differs.item() == 0
    tp.tpmlp_check_status()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_xent_of_a_few_rows_that_do_not_count(tp, dtype):
    X, W, t, dloss = _xent_inputs(6, 64, 300, dtype, seed=18, masked=0.0)
    t[1], t[4], dloss[1], dloss[4] = -100, 300, float("nan"), float("inf")
    loss, lse = tp.tpmlp_xent_forward(X, W, t)
    with pytest.raises(tp.TpmlpError) as e:
        tp.tpmlp_check_status()
    assert e.value.code == tp.TPMLP_ERR_BOUNDS
    dX, dW = tp.tpmlp_xent_backward(X, W, t, lse, dloss)
    assert bool((loss[[1, 4]] == 0).all()) and bool(torch.isfinite(lse).all())
    assert bool((dX[[1, 4]] == 0).all()) and bool(torch.isfinite(dW).all())
    keep = [0, 2, 3, 5]
    loss2, lse2 = tp.tpmlp_xent_forward(X[keep], W, t[keep])
    dX2, dW2 = tp.tpmlp_xent_backward(X[keep], W, t[keep], lse2, dloss[keep])
    assert torch.equal(loss2, loss[keep]) and torch.equal(dX2, dX[keep]) and torch.equal(dW2, dW)
    tp.tpmlp_check_status()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_xent_in_pieces_of_the_vocabulary(tp, dtype):
    # 34000 rows: 2^28 / 34000 < 8192 columns a piece; 9000 ids make two, the second ragged.
    X, W, t, dloss = _xent_inputs(34000, 16, 9000, dtype, seed=5)
    T, D, V = 34000, 16, 9000
    assert tp.tpmlp_xent_workspace_bytes(T, D, V, X.dtype, 1) < T * V * (2 if dtype == "bf16" else 6)
    _check_xent(tp, X, W, t, dloss, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_xent_rows_that_do_not_count(tp, dtype):
    # Every row masked: no loss, gradients exactly zero, whatever dloss holds there.
    X, W, t, dloss = _xent_inputs(70, 64, 300, dtype, seed=8)
    t[:] = -1
    dloss[::2] = float("nan")
    dloss[1::2] = float("inf")
    loss, lse = tp.tpmlp_xent_forward(X, W, t)
    dX, dW = tp.tpmlp_xent_backward(X, W, t, lse, dloss)
    assert bool((loss == 0).all()) and bool(torch.isfinite(lse).all())
    assert bool((dX == 0).all()) and bool((dW == 0).all())
    # One row counts; the others' dloss must not reach it.
    t[5] = 7
    dloss[5] = 0.25
    ref = dloss.clone()
    ref[t < 0] = 0
    loss, lse = tp.tpmlp_xent_forward(X, W, t)
    dX, dW = tp.tpmlp_xent_backward(X, W, t, lse, dloss)
    dX2, dW2 = tp.tpmlp_xent_backward(X, W, t, lse, ref)
    assert torch.equal(dX, dX2) and torch.equal(dW, dW2) and bool(torch.isfinite(dW).all())
    # Zero upstream gradients.
    dX, dW = tp.tpmlp_xent_backward(X, W, t, lse, torch.zeros_like(dloss))
    assert bool((dX == 0).all()) and bool((dW == 0).all())
    tp.tpmlp_check_status()


def test_xent_target_out_of_range_is_left_out_and_reported(tp):
    X, W, t, dloss = _xent_inputs(50, 64, 300, "bf16", seed=9, masked=0.0)
    ref_t = t.clone()
    t[3], t[17], ref_t[3], ref_t[17] = 300, 1 << 40, -1, -1
    loss, lse = tp.tpmlp_xent_forward(X, W, t)
    with pytest.raises(tp.TpmlpError) as e:
        tp.tpmlp_check_status()
    assert e.value.code == tp.TPMLP_ERR_BOUNDS
    tp.tpmlp_check_status()
    loss2, lse2 = tp.tpmlp_xent_forward(X, W, ref_t)
    assert torch.equal(loss, loss2) and torch.equal(lse, lse2)
    a, b = tp.tpmlp_xent_backward(X, W, t, lse, dloss), tp.tpmlp_xent_backward(X, W, ref_t, lse, dloss)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("T,D,V", [(100, 8, 1), (300, 16, 3), (70, 64, 257), (513, 24, 65)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_xent_small_vocabularies(tp, T, D, V, dtype):
    X, W, t, dloss = _xent_inputs(T, D, V, dtype, seed=T + V)
    _check_xent(tp, X, W, t, dloss, dtype)


@pytest.mark.parametrize("T", [9, 100])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_xent_extreme_row_gradients(tp, dtype, T):
    # An infinite row gradient spoils its own row of dX only; tiny ones keep their precision.
    X, W, t, dloss = _xent_inputs(T, 64, 300, dtype, seed=70, masked=0.0)
    _, lse = tp.tpmlp_xent_forward(X, W, t)
    ref, _ = tp.tpmlp_xent_backward(X, W, t, lse, torch.where(torch.arange(T, device="cuda") == 4, 0.0, dloss))
    dloss[4] = float("inf")
    dX, _ = tp.tpmlp_xent_backward(X, W, t, lse, dloss)
    keep = torch.arange(T, device="cuda") != 4
    assert torch.equal(dX[keep], ref[keep]) and not bool(torch.isfinite(dX[4]).all())
    for scale in (1e-38, 1e-30, 1e30):
        _check_xent(tp, X, W, t, torch.full_like(dloss, scale), dtype) if scale > 1e-35 else None
        dX, dW = tp.tpmlp_xent_backward(X, W, t, lse, torch.full_like(dloss, scale))
        assert bool(torch.isfinite(dX).all()) and bool(torch.isfinite(dW).all()) and bool((dX != 0).any())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_xent_large_logits(tp, dtype):
    # Logits of some hundreds: exponentials that over- and underflow fp32 unless they are taken below the maximum.
    X, W, t, dloss = _xent_inputs(40, 64, 700, dtype, seed=10)
    X = (X.float() * 100).to(X.dtype)
    loss, lse = tp.tpmlp_xent_forward(X, W, t)
    assert bool(torch.isfinite(loss).all()) and bool(torch.isfinite(lse).all()) and lse.max() > 150
    _check_xent(tp, X, W, t, dloss, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,V", [(1, 300), (3, 5000), (40, 5000), (100, 300), (300, 5000), (2100, 300)])
def test_xent_loss_of_nearly_certain_rows(tp, T, V, dtype):
    # Entries -1, 0 and 1 and X_t = W_target: every logit is an exact integer, the target's about 40, and the losses are
    # down to 1e-12: differences of fp32 numbers near 40 could not show them.
    g = torch.Generator(device="cuda").manual_seed(T + V)
    W = torch.randint(-1, 2, (V, 64), generator=g, device="cuda").to(DT[dtype])
    t = torch.randint(0, V, (T,), generator=g, device="cuda")
    X = W[t].contiguous()
    loss, lse = tp.tpmlp_xent_forward(X, W, t)
    z = X.double() @ W.double().T
    e = z - z.gather(1, t[:, None])
    gap = e.abs().max(dim=1).values
    e.scatter_(1, t[:, None], -math.inf)
    ref = torch.log1p(torch.exp(e).sum(1))
    # log2 e as an fp32 constant and each exponent's rounding are off by the exponent times U32, an exponential by 4, the
    # sums of parts and their joining by 64 U32 (as above), the result's functions by 8.
    _close(loss, ref, ref * (3 * gap + 80) * U32, "loss")
    _close(lse, z.gather(1, t[:, None])[:, 0] + ref, 2 * U32 * (lse.double().abs() + ref), "lse")


class _WithLoss:
    """The library with the forward's loss handed to the backward."""

    def __init__(self, tp):
        self.tp = tp

    def __getattr__(self, name):
        return getattr(self.tp, name)

    def tpmlp_xent_forward(self, *a, **kw):
        self.loss, lse = self.tp.tpmlp_xent_forward(*a, **kw)
        return self.loss, lse

    def tpmlp_xent_backward(self, *a, **kw):
        return self.tp.tpmlp_xent_backward(*a, loss=self.loss, **kw)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,D,V", [(1, 64, 257), (1, 8, 1), (9, 1032, 4000), (33, 264, 1000), (150, 520, 700), (257, 136, 1000),
                                   (192, 2048, 8200), (600, 1032, 8300), (34000, 16, 9000)])
def test_xent_gradients_from_the_loss(tp, T, D, V, dtype):
    X, W, t, dloss = _xent_inputs(T, D, V, dtype, seed=T + D + V)
    _check_xent(_WithLoss(tp), X, W, t, dloss, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,V", [(1, 300), (3, 5000), (40, 5000), (64, 300), (150, 600), (300, 5000), (2100, 300)])
def test_xent_gradients_of_nearly_certain_rows(tp, T, V, dtype):
    # The rows of the loss's test above: 1 - p down to 1e-12, which the fp32 exp(z - lse) - 1 near 40 does not hold, and
    # which is as large as all other ids' parts together. Bounds relative to each entry of dz.
    g = torch.Generator(device="cuda").manual_seed(T + V)
    W = torch.randint(-1, 2, (V, 64), generator=g, device="cuda").to(DT[dtype])
    t = torch.randint(0, V, (T,), generator=g, device="cuda")
    X = W[t].contiguous()
    dloss = torch.rand(T, generator=g, device="cuda") + 0.5
    loss, lse = tp.tpmlp_xent_forward(X, W, t)
    dX, dW = tp.tpmlp_xent_backward(X, W, t, lse, dloss, loss=loss)
    tp.tpmlp_check_status()
    z = X.double() @ W.double().T
    e = z - z.gather(1, t[:, None])
    gap = e.abs().max(dim=1).values[:, None]
    e.scatter_(1, t[:, None], -math.inf)
    ref = torch.log1p(torch.exp(e).sum(1))[:, None]
    dz = torch.exp(e - ref)
    dz.scatter_(1, t[:, None], torch.expm1(-ref))
    dz *= dloss.double()[:, None]
    # Exponents: lse's rounding, log2 e as a constant, its products and the difference, each off by its size times U32;
    # the exponential by 4 U32; the loss as in its test, expm1 2 U32 more; dloss / max and the product 2. Then dz's rounding.
    size = gap + z.abs().max(dim=1).values[:, None]
    half = 4 * U32 if dtype == "f32" else 1.01 * U16 if T > 64 else 1.01 * U16 ** 2
    edz = dz.abs() * ((4 * size + 3 * gap + 90) * U32 + half)
    out = U16 * 1.01 if dtype == "bf16" else 2 * U32
    for got, a, b, k, what in ((dX, dz, W.double(), V, "dX"), (dW, dz.T, X.double(), T, "dW")):
        want = a @ b
        err = edz if what == "dX" else edz.T
        tol = err @ b.abs() + (a.abs() @ b.abs()) * (_sum_bound(k, dtype) + 80 * U32) + out * want.abs()
        _close(got, want, tol + 1e-30, what)


def test_xent_infinities_stay_in_their_row(tp):
    X, W, t, dloss = _xent_inputs(40, 64, 300, "bf16", seed=12, masked=0.0)
    loss, lse = tp.tpmlp_xent_forward(X, W, t)
    Y = X.clone()
    Y[11, 3] = float("inf")
    Y[12, 3] = float("nan")
    loss2, lse2 = tp.tpmlp_xent_forward(Y, W, t)
    keep = torch.ones(40, dtype=torch.bool, device="cuda")
    keep[11:13] = False
    assert torch.equal(loss[keep], loss2[keep]) and torch.equal(lse[keep], lse2[keep])
    assert bool(torch.isnan(loss2[11:13]).all())


@pytest.mark.parametrize("T", [1, 100])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_xent_infinities_and_nans_among_the_logits(tp, dtype, T):
    # One column each: of every row's logits, the targets at id 0.
    X = torch.zeros(T, 64, device="cuda", dtype=DT[dtype])
    X[:, 0] = 1
    t = torch.zeros(T, dtype=torch.int64, device="cuda")
    inf, nan = float("inf"), float("nan")
    for column, want in (([0.0, nan], (nan, nan)), ([nan, 0.0], (nan, nan)), ([0.0, -inf], (0.0, 0.0)),
                         ([-inf, 0.0], (inf, 0.0)), ([0.0, inf], (nan, nan)), ([inf, 0.0], (nan, nan)),
                         ([0.0, 0.0, -inf], (math.log(2.0), math.log(2.0))), ([2.0], (0.0, 2.0)), ([nan], (nan, nan))):
        W = torch.zeros(len(column), 64, device="cuda", dtype=DT[dtype])
        W[:, 0] = torch.tensor(column, device="cuda")
        if dtype == "f32" and any(map(math.isinf, column)):
            continue  # the pieces of an infinity are not numbers
        loss, lse = tp.tpmlp_xent_forward(X, W, t)
        for got, ref in zip((loss, lse), want):
            ref = torch.full((T,), ref, device="cuda")
            assert torch.allclose(got, ref, rtol=1e-6, atol=0, equal_nan=True), (column, got[0].item(), ref[0].item())


def test_xent_gradient_against_differences(tp):
    # d/de L(X + e U, W + e V') at 0, by central differences of the fp32 losses. With s the
    # largest change rate of a logit, the third derivative of a row's loss is at most 2 s^3
    # (third cumulant of numbers within [-s, s], with room), so the step e leaves e^2 s^3 / 3
    # a row; the fp32 losses are good to 4e-6 here and leave 4e-6 / e.
    T, D, V = 60, 64, 500
    X, W, t, dloss = _xent_inputs(T, D, V, "f32", seed=13)
    g = torch.Generator(device="cuda").manual_seed(14)
    U = torch.randn(T, D, generator=g, device="cuda")
    Q = torch.randn(V, D, generator=g, device="cuda") / math.sqrt(D)
    loss, lse = tp.tpmlp_xent_forward(X, W, t)
    dX, dW = tp.tpmlp_xent_backward(X, W, t, lse, dloss)
    on = t >= 0
    for dx, dw in ((U, torch.zeros_like(Q)), (torch.zeros_like(U), Q)):
        e = 2.0 ** -6
        s = (dx.double() @ W.double().T + X.double() @ dw.double().T).abs().max().item()
        hi, _ = tp.tpmlp_xent_forward(X + e * dx, W + e * dw, t)
        lo, _ = tp.tpmlp_xent_forward(X - e * dx, W - e * dw, t)
        diff = ((hi.double() - lo.double()) / (2 * e) * dloss.double()).sum().item()
        want = (dX.double() * dx.double()).sum().item() + (dW.double() * dw.double()).sum().item()
        weight = dloss[on].double().abs().sum().item()
        assert abs(diff - want) <= weight * (e * e * s ** 3 / 3 + 4e-6 / e + 2e-5 * s), (diff, want)


# ------------------------------------------------------------------ embedding


def _ids(T, V, seed, kind):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if kind == "one":  # a single id T times
        return torch.full((T,), V // 2, device="cuda", dtype=torch.int64)
    if kind == "each":  # every id at most once, in disorder
        return torch.randperm(max(T, V), generator=g, device="cuda")[:T] % V
    u = torch.rand(T, generator=g, device="cuda", dtype=torch.float64)
    ids = (torch.exp(u * math.log(V + 1.0)).long() - 1).clamp(0, V - 1)  # frequent as words are
    ids[torch.rand(T, generator=g, device="cuda") < 0.1] = -1
    return ids


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,D,V", [(1, 1, 1), (1, 4096, 50), (7, 768, 1000), (300, 40, 65536), (1000, 33, 77),
                                   (5000, 8, 300), (130, 12, 9), (3, 2047, 4)])
def test_embed_lookup(tp, T, D, V, dtype):
    g = torch.Generator(device="cuda").manual_seed(T)
    E = torch.randn(V, D, generator=g, device="cuda").to(DT[dtype])
    ids = _ids(T, V, T + 1, "words")
    out = tp.tpmlp_embed_forward(E, ids, 1.7)
    # One product in fp32 and at most one rounding to bf16: the same as torch's.
    ref = torch.where((ids >= 0)[:, None], E[ids.clamp(min=0)].float() * 1.7, torch.zeros((), device="cuda")).to(E.dtype)
    assert torch.equal(out, ref)
    assert torch.equal(tp.tpmlp_embed_forward(E, ids), torch.where((ids >= 0)[:, None], E[ids.clamp(min=0)],
                                                                   torch.zeros((), device="cuda", dtype=E.dtype)))


def _check_embed_grad(tp, dout, ids, V, scale, dtype_out, dE0=None):
    T, D = dout.shape
    on = ids >= 0
    want = torch.zeros(V, D, dtype=torch.float64, device="cuda")
    mag = torch.zeros(V, D, dtype=torch.float64, device="cuda")
    want.index_add_(0, ids[on], dout[on].double() * scale)
    mag.index_add_(0, ids[on], (dout[on].double() * scale).abs())
    n = torch.bincount(ids[on], minlength=V).double()[:, None]
    if dE0 is not None:
        want = want + dE0.double()
        mag = mag + dE0.double().abs()
    dE = dE0.clone() if dE0 is not None else None
    got = tp.tpmlp_embed_backward(dout, ids, V, scale, dE=dE, accumulate=dE0 is not None,
                                  dtype=None if dE is not None else dtype_out)
    tp.tpmlp_check_status()
    out = 1.01 * U16 if dtype_out == torch.bfloat16 else U32
    _close(got, want, mag * (n + 3) * U32 + out * want.abs(), "dE")
    absent = n[:, 0] == 0
    assert torch.equal(got[absent], dE0[absent] if dE0 is not None else torch.zeros_like(got[absent]))
    return got


@pytest.mark.parametrize("types", [("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16"), ("bf16", "f32")],
                         ids=lambda t: f"{t[0]}-{t[1]}")
@pytest.mark.parametrize("kind", ["words", "one", "each"])
@pytest.mark.parametrize("T,D,V", [(1, 8, 1), (1, 5, 300), (63, 16, 10), (64, 768, 70000), (65, 40, 7), (700, 33, 500),
                                   (5000, 264, 3000), (20000, 8, 40)])
def test_embed_gradient(tp, T, D, V, kind, types):
    g = torch.Generator(device="cuda").manual_seed(T + D)
    dout = torch.randn(T, D, generator=g, device="cuda").to(DT[types[0]])
    ids = _ids(T, V, T + 2, kind)
    got = _check_embed_grad(tp, dout, ids, V, 1.5, DT[types[1]])
    # The order of every addition is fixed.
    again = tp.tpmlp_embed_backward(dout, ids, V, 1.5, dtype=DT[types[1]])
    assert torch.equal(got, again)


@pytest.mark.parametrize("kind", ["words", "one", "each"])
@pytest.mark.parametrize("T,D,V", [
    (8192, 8, 511), (8193, 8, 512), (32769, 16, 70000), (60000, 4, 262143), (65536, 136, 1000),  # one cluster sorts
    (65537, 8, 262144), (300001, 8, 90), (70000, 5, 3000),                                       # three launches a digit
])
def test_embed_gradient_of_many_tokens(tp, T, D, V, kind):
    # Around the limits of the two sorts and of their digits.
    g = torch.Generator(device="cuda").manual_seed(T + D)
    dout = torch.randn(T, D, generator=g, device="cuda")
    ids = _ids(T, V, T + 2, kind)
    got = _check_embed_grad(tp, dout, ids, V, 1.0, torch.float32)
    assert torch.equal(got, tp.tpmlp_embed_backward(dout, ids, V))
    dE0 = torch.randn(V, D, generator=g, device="cuda")
    _check_embed_grad(tp, dout, ids, V, 1.0, torch.float32, dE0)


@pytest.mark.parametrize("types", [("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16"), ("bf16", "f32")], ids="-".join)
@pytest.mark.parametrize("T,D,V", [(391, 1074, 40001), (100, 1075, 36000), (5000, 4095, 12345), (70000, 1001, 3000),
                                   (66000, 3, 100001), (9, 1, 70), (40, 2, 30000000), (300, 8201, 4000)])
def test_embed_gradient_of_rows_off_16_bytes(tp, T, D, V, types):
    # Rows that begin anywhere: summed with strided columns, cleared in 16 bytes at a time across the rows' borders;
    # the table's last bytes and what lies behind them too.
    g = torch.Generator(device="cuda").manual_seed(T + D)
    ids = torch.randint(0, V, (T,), generator=g, device="cuda")
    ids[0], ids[-1] = V - 1, -1
    dout = torch.randint(-8, 9, (T, D), generator=g, device="cuda").to(DT[types[0]])  # sums of small integers are exact
    whole = torch.full((V * D + 64,), 7.0, device="cuda", dtype=DT[types[1]])
    dE = whole[:V * D].view(V, D)
    keep = ids >= 0
    ref = torch.zeros(V, D, device="cuda").index_add_(0, ids[keep], dout[keep].float() * 0.5).to(DT[types[1]])
    tp.tpmlp_embed_backward(dout, ids, V, 0.5, dE=dE)
    assert torch.equal(dE, ref) and bool((whole[V * D:] == 7).all())
    got = tp.tpmlp_embed_forward(ref, ids, 2.0)
    want = torch.where(keep[:, None], ref[ids.clamp(min=0)].float() * 2, torch.zeros((), device="cuda")).to(ref.dtype)
    assert torch.equal(got, want)
    tp.tpmlp_embed_backward(dout, ids, V, 0.5, dE=dE, accumulate=True)
    assert torch.equal(dE, (ref.float() * 2).to(ref.dtype))
    tp.tpmlp_check_status()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_embed_lookup_of_many_tokens(tp, dtype):
    g = torch.Generator(device="cuda").manual_seed(2)
    for T, D, V in ((70001, 136, 500), (20000, 1500, 3000)):
        E = torch.randn(V, D, generator=g, device="cuda").to(DT[dtype])
        ids = _ids(T, V, T, "words")
        ref = torch.where((ids >= 0)[:, None], E[ids.clamp(min=0)].float() * 0.3, torch.zeros((), device="cuda")).to(E.dtype)
        assert torch.equal(tp.tpmlp_embed_forward(E, ids, 0.3), ref)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_embed_gradient_added_to_a_tied_table(tp, dtype):
    g = torch.Generator(device="cuda").manual_seed(3)
    T, D, V = 900, 72, 400
    dout = torch.randn(T, D, generator=g, device="cuda")
    dE0 = torch.randn(V, D, generator=g, device="cuda").to(DT[dtype])
    _check_embed_grad(tp, dout, _ids(T, V, 4, "words"), V, 0.5, DT[dtype], dE0)
    # No tokens: nothing is added; without accumulate the table's gradient is cleared.
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    dE = dE0.clone()
    tp.tpmlp_embed_backward(dout[:0], none, V, dE=dE, accumulate=True)
    assert torch.equal(dE, dE0)
    tp.tpmlp_embed_backward(dout[:0], none, V, dE=dE)
    assert bool((dE == 0).all())


def test_embed_gradient_differences(tp):
    # The lookup is linear, so differences give the gradient up to rounding:
    # <dE, Q> = <dout, lookup(Q)>, sums of T D products with errors below 2^-20 of their magnitudes.
    g = torch.Generator(device="cuda").manual_seed(6)
    T, D, V = 500, 96, 60
    dout, Q = torch.randn(T, D, generator=g, device="cuda"), torch.randn(V, D, generator=g, device="cuda")
    ids = _ids(T, V, 7, "words")
    dE = tp.tpmlp_embed_backward(dout, ids, V, 2.0)
    out = tp.tpmlp_embed_forward(Q, ids, 2.0)
    a, b = (dE.double() * Q.double()).sum(), (dout.double() * out.double()).sum()
    assert abs((a - b).item()) <= (dout.double() * out.double()).abs().sum().item() * 2.0 ** -16


def test_embed_token_out_of_range_is_left_out_and_reported(tp):
    g = torch.Generator(device="cuda").manual_seed(8)
    E = torch.randn(30, 24, generator=g, device="cuda")
    dout = torch.randn(20, 24, generator=g, device="cuda")
    ids = torch.arange(20, device="cuda")
    ref = ids.clone()
    ids[4], ids[9], ref[4], ref[9] = 30, 1 << 50, -5, -5
    for call in (lambda i: tp.tpmlp_embed_forward(E, i), lambda i: tp.tpmlp_embed_backward(dout, i, 30)):
        got = call(ids)
        with pytest.raises(tp.TpmlpError) as e:
            tp.tpmlp_check_status()
        assert e.value.code == tp.TPMLP_ERR_BOUNDS
        assert torch.equal(got, call(ref))
        tp.tpmlp_check_status()


# ------------------------------------------------------------------ clipping


def _check_clip(tp, grads, max_norm, in_place):
    ref = math.sqrt(sum(g.double().square().sum().item() for g in grads))
    c = min(1.0, max_norm / (ref + 1e-6))
    before = [g.clone() for g in grads]
    n2 = tp.tpmlp_grad_norm(grads)
    out = None if in_place else [torch.full_like(g, 7.0) for g in grads]
    norm = tp.tpmlp_grad_clip(grads, max_norm, out=out)
    # 32 fp32 additions in a chain and one rounding of the square each, halved by the root, and the final rounding.
    rel = 18 * U32
    assert norm.shape == (1,) and abs(norm.item() - ref) <= rel * ref + 1e-44
    assert torch.equal(norm, n2)
    for g0, got in zip(before, grads if in_place else out):
        want = g0.double() * c
        half = U16 if got.dtype == torch.bfloat16 else U32
        _close(got, want, want.abs() * (rel + 4 * U32 + half * 1.001), "clipped")
    if not in_place:
        assert all(torch.equal(a, b) for a, b in zip(before, grads))


SETS = {
    "one": [(1, "f32")],
    "one_bf16": [(1, "bf16")],
    "odd": [(3, "f32"), (8191, "bf16"), (8193, "f32"), (1, "bf16"), (16385, "bf16"), (5, "f32")],
    "empty_among": [(0, "f32"), (100, "bf16"), (0, "bf16"), (70000, "f32"), (0, "f32")],
    "large": [(5000001, "f32"), (3000007, "bf16"), (12, "f32")],
    "many": [(1 + 37 * i % 911, "f32" if i % 3 else "bf16") for i in range(700)],
}


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("name", list(SETS))
def test_clip(tp, name, in_place):
    g = torch.Generator(device="cuda").manual_seed(17)
    for max_norm in (0.5, 1e6, 0.0):
        grads = [torch.randn(n, generator=g, device="cuda").to(DT[dt]) for n, dt in SETS[name]]
        _check_clip(tp, grads, max_norm, in_place)


def test_clip_of_nothing_and_of_zeros(tp):
    for grads in ([], [torch.empty(0, device="cuda")]):
        assert tp.tpmlp_grad_norm(grads).item() == 0 and tp.tpmlp_grad_clip(grads, 1.0).item() == 0
    z = [torch.zeros(1000, device="cuda"), torch.zeros(7, device="cuda", dtype=torch.bfloat16)]
    assert tp.tpmlp_grad_clip(z, 1.0).item() == 0
    assert all(bool((t == 0).all()) for t in z)


def test_clip_norm_beyond_the_range(tp):
    # An infinite or NaN gradient shows in the norm; the clipped values follow the formula.
    a = torch.ones(100, device="cuda")
    a[3] = float("inf")
    assert tp.tpmlp_grad_norm([a]).item() == float("inf")
    a[3] = float("nan")
    assert math.isnan(tp.tpmlp_grad_norm([a]).item())
    out = [torch.empty_like(a)]
    tp.tpmlp_grad_clip([a], 1.0, out=out)
    assert bool(torch.isnan(out[0]).all())


def test_clip_of_views_and_refusals(tp):
    flat = torch.randn(4096, device="cuda")
    views = [flat[:1000], flat[1000:1004], flat[1024:4096]]  # each on a 16-byte boundary
    _check_clip(tp, views, 0.25, True)
    with pytest.raises(tp.TpmlpError) as e:
        tp.tpmlp_grad_clip([flat[1:100]], 1.0)
    assert e.value.code == tp.TPMLP_ERR_ALIGN
    with pytest.raises(tp.TpmlpError) as e:
        tp.tpmlp_grad_clip([flat, flat[:8]], 1.0)
    assert e.value.code == tp.TPMLP_ERR_ARG
    with pytest.raises(ValueError):
        tp.tpmlp_grad_clip([flat.view(64, 64).t()], 1.0)
    with pytest.raises(TypeError):
        tp.tpmlp_grad_norm([flat.double()])
    with pytest.raises(ValueError):
        tp.tpmlp_grad_clip([flat], 1.0, out=[flat[:10]])


# ------------------------------------------------------------------ beyond 2^31 elements


@pytest.mark.parametrize("T", [3, 70])
def test_xent_of_more_than_2_31_weights(tp, T):
    D, V = 8, (1 << 28) + 77
    g = torch.Generator(device="cuda").manual_seed(T)
    W = torch.randn(V, D, generator=g, device="cuda").bfloat16()
    X = torch.randn(T, D, generator=g, device="cuda").bfloat16()
    t = torch.randint(0, V, (T,), generator=g, device="cuda")
    t[0], t[1], t[2] = V - 1, 0, (1 << 28) + 3
    dloss = torch.rand(T, generator=g, device="cuda") + 0.5
    loss, lse = tp.tpmlp_xent_forward(X, W, t)
    dX, dW = tp.tpmlp_xent_backward(X, W, t, lse, dloss)
    tp.tpmlp_check_status()
    x, step = X.double(), 1 << 22
    sums = torch.zeros(T, dtype=torch.float64, device="cuda")
    for v in range(0, V, step):
        sums += torch.exp(x @ W[v:v + step].double().T).sum(1)
    ref = torch.log(sums)
    zt = (x * W[t].double()).sum(1)
    # A thread adds at most 2^21 / 128 parts one after the other (3 rows: fewer); logits and logarithm as above.
    ez = 16 * U32 * ((x.abs() @ W[:step].double().abs().T).max(1).values + 40)
    el = (1 << 14) * 2 * U32 + ez
    _close(lse, ref, el, "lse")
    _close(loss, ref - zt, el + ez, "loss")
    rX, mag = torch.zeros_like(x), torch.zeros_like(x)
    for v in range(0, V, step):
        w = W[v:v + step].double()
        dz = torch.exp(x @ w.T - ref[:, None])
        here = (t >= v) & (t < v + step)
        dz[here, t[here] - v] -= 1
        dz *= dloss.double()[:, None]
        rX += dz @ w
        mag += dz.abs() @ w.abs()
        if v == 0 or v + 2 * step > V:  # the first piece and what lies around and behind 2^31 elements
            r, m = dz.T @ x, dz.abs().T @ x.abs()
            _close(dW[v:v + step], r, m * (1.01 * U16 + 2 * (ez + el).max() + 1e-5) + 1.01 * U16 * r.abs() + 1e-30, "dW")
    # dX: dz's rounding, and sums in slices of under 2^22 ids, 16 to an addition, then of at most 80 pieces.
    _close(dX, rX, mag * (1.01 * U16 + 2 * (ez + el).max() + (2 ** 18 + 80) * 2 * U32) + 1.01 * U16 * rX.abs(), "dX")


def test_embed_of_more_than_2_31_elements(tp):
    D, V = 4096, (1 << 19) + 1000
    g = torch.Generator(device="cuda").manual_seed(5)
    E = torch.randn(V, D, generator=g, device="cuda", dtype=torch.bfloat16)
    ids = torch.randperm(V, generator=g, device="cuda")
    assert torch.equal(tp.tpmlp_embed_forward(E, ids), E[ids])
    dE = tp.tpmlp_embed_backward(E, ids, V)
    assert torch.equal(dE[ids], E)  # each id once: its row of dout
    few = torch.tensor([V - 1, 3, V - 1, 1 << 19], device="cuda")
    dE = tp.tpmlp_embed_backward(E[:4], few, V)
    ref = torch.zeros_like(E)
    ref[V - 1], ref[3], ref[1 << 19] = (E[0].float() + E[2].float()).bfloat16(), E[1], E[3]
    assert torch.equal(dE, ref)
    tp.tpmlp_check_status()


def test_clip_of_more_than_2_31_elements(tp):
    a = torch.full(((1 << 31) + 4099,), 0.5, device="cuda", dtype=torch.bfloat16)
    a[-1] = -1.5
    norm = tp.tpmlp_grad_clip([a[:8], a[8:]], 2.0 ** 13)
    want = math.sqrt(0.25 * (a.numel() - 1) + 2.25)  # every partial sum is exact
    assert abs(norm.item() - want) <= U32 * want
    c = 2.0 ** 13 / (want + 1e-6)
    for got, v in ((a[:-1].amax(), 0.5), (a[:-1].amin(), 0.5), (a[-1], -1.5)):
        assert abs(got.item() - c * v) <= (1.01 * U16 + 4 * U32) * abs(c * v)


# ------------------------------------------------------------------ together


def _step(tp, E, ids, targets, shards, eps, max_norm):
    """Embedding, one block, the tied table as the loss's matrix, and back; all gradients clipped."""
    dt = E.dtype
    V, D = E.shape
    x = tp.tpmlp_embed_forward(E, ids, math.sqrt(D))
    h = tp.tpmlp_block_forward(x, shards, "fused", eps=eps).to(dt)
    loss, lse = tp.tpmlp_xent_forward(h, E, targets)
    dloss = torch.full((len(ids),), 1.0, device="cuda") / (targets >= 0).sum()
    dh, dE = tp.tpmlp_xent_backward(h, E, targets, lse, dloss)
    dx, dA, dB = tp.tpmlp_block_backward(x, dh, shards, "fused", eps=eps)
    tp.tpmlp_embed_backward(dx, ids, V, math.sqrt(D), dE=dE, accumulate=True)
    grads = [dE] + list(dA) + list(dB)
    norm = tp.tpmlp_grad_clip(grads, max_norm)
    return loss, norm, grads


def _step_reference(E, ids, targets, A, B, eps, max_norm):
    D = E.shape[1]
    e, a, b = (v.double().requires_grad_() for v in (E, A, B))
    on = (ids >= 0)[:, None]
    x = torch.where(on, e[ids.clamp(min=0)] * math.sqrt(D), torch.zeros((), device="cuda", dtype=torch.float64))
    y = (x - x.mean(1, keepdim=True)) / torch.sqrt(x.var(1, unbiased=False, keepdim=True) + eps)
    h = x + torch.nn.functional.gelu(y @ a, approximate="tanh") @ b
    z = h @ e.T
    counts = targets >= 0
    loss = torch.logsumexp(z, 1) - z.gather(1, targets.clamp(min=0)[:, None])[:, 0]
    loss = torch.where(counts, loss, torch.zeros_like(loss))
    (loss.sum() / counts.sum()).backward()
    norm = torch.sqrt(sum(v.grad.square().sum() for v in (e, a, b)))
    c = min(1.0, max_norm / (norm.item() + 1e-6))
    return loss.detach(), norm.item(), e.grad * c, a.grad * c, b.grad * c


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_training_step_of_all_of_them(tp, dtype):
    # Norm-wise bounds. fp32: every step is good to about 2^-18 of its magnitudes and there are
    # fewer than 16 in a row, none of which amplifies by more than the layer norm's factor (the
    # embedded rows have unit size, so about 1): 2^-14. bf16: x, LN(x), H, h, dz, dh (also the
    # block's operand), dP and dE are rounded to bf16, eight roundings of at most U16 relative to
    # their tensors, and the logits' rounding error through h, |h| |E| U16 at logits of size
    # about 1, doubles one of them: 9 U16.
    T, D, F, V, n = 500, 128, 512, 700, 4
    g = torch.Generator(device="cuda").manual_seed(21)
    E = (torch.randn(V, D, generator=g, device="cuda") / math.sqrt(D)).to(DT[dtype])
    A = (torch.randn(D, F, generator=g, device="cuda") * 0.05).to(DT[dtype])
    B = (torch.randn(F, D, generator=g, device="cuda") * 0.05).to(DT[dtype])
    ids = _ids(T, V, 22, "words")
    ids[0] = 3
    # Zero rows have an undefined direction under the layer norm's root only through eps; give them none here.
    ids = ids.clamp(min=0)
    targets = torch.roll(ids, -1)
    targets[-7:] = -100
    shards = tp.tpmlp_shard(A, B, n)
    loss, norm, grads = _step(tp, E, ids, targets, shards, 1e-5, 0.7)
    tp.tpmlp_check_status()
    rloss, rnorm, rE, rA, rB = _step_reference(E, ids, targets, A, B, 1e-5, 0.7)
    bound = 9 * U16 if dtype == "bf16" else 2.0 ** -14
    dE, dA, dB = grads[0], torch.cat(grads[1:1 + n], 1), torch.cat(grads[1 + n:], 0)
    assert rnorm > 0.7, "the step clips"
    for got, ref, what in ((loss, rloss, "loss"), (dE, rE, "dE"), (dA, rA, "dA"), (dB, rB, "dB")):
        rel = ((got.double() - ref).norm() / ref.norm()).item()
        assert rel <= bound, (what, rel)
    assert abs(norm.item() - rnorm) <= bound * rnorm


def _train_calls(tp, seed=31):
    X, W, t, dloss = _xent_inputs(300, 256, 3000, "bf16", seed=seed)
    Xf, Wf = X.float(), W.float()
    ids = _ids(3000, 500, seed + 1, "words")
    g = torch.Generator(device="cuda").manual_seed(seed)
    E = torch.randn(500, 128, generator=g, device="cuda").bfloat16()
    dout = torch.randn(3000, 128, generator=g, device="cuda")
    grads = [torch.randn(n, generator=g, device="cuda") for n in (70000, 3, 20001)]
    _, lse = tp.tpmlp_xent_forward(X, W, t)
    _, lsef = tp.tpmlp_xent_forward(Xf, Wf, t)
    return {
        "xent forward": lambda s=None: list(tp.tpmlp_xent_forward(X, W, t, stream=s)),
        "xent backward": lambda s=None: list(tp.tpmlp_xent_backward(X, W, t, lse, dloss, stream=s)),
        "xent forward f32": lambda s=None: list(tp.tpmlp_xent_forward(Xf, Wf, t, stream=s)),
        "xent backward f32": lambda s=None: list(tp.tpmlp_xent_backward(Xf, Wf, t, lsef, dloss, stream=s)),
        "embed forward": lambda s=None: [tp.tpmlp_embed_forward(E, ids, 3.0, stream=s)],
        "embed backward": lambda s=None: [tp.tpmlp_embed_backward(dout, ids, 500, 3.0, stream=s)],
        "clip": lambda s=None: (lambda o: [tp.tpmlp_grad_clip(grads, 0.5, out=o, stream=s)] + o)(
            [torch.empty_like(v) for v in grads]),
        "norm": lambda s=None: [tp.tpmlp_grad_norm(grads, stream=s)],
    }


def test_calls_are_reproducible_and_run_on_the_given_stream(tp):
    import time

    for name, fn in _train_calls(tp).items():
        ref = fn()
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        torch.cuda._sleep(2_000_000_000)  # about one second on the default stream (a bounded spin)
        done = torch.cuda.Event()
        with torch.cuda.stream(side):
            out = fn(side)
            done.record(side)
        t0 = time.time()
        while not done.query() and time.time() - t0 < 0.5:
            time.sleep(0.001)
        finished = done.query()
        torch.cuda.synchronize()
        assert finished, f"{name}: waited for the default stream"
        assert all(torch.equal(a, b) for a, b in zip(out, ref)), f"{name}: differs on the side stream"
    tp.tpmlp_check_status()


def test_calls_captured_into_graphs_and_replayed(tp):
    for name, fn in _train_calls(tp, seed=41).items():
        ref = [v.clone() for v in fn()]
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            fn(side)  # warm-up
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = fn(torch.cuda.current_stream())
        for _ in range(3):
            for v in out:
                v.fill_(5.0)
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, ref)), f"{name}: differs when replayed"
    tp.tpmlp_check_status()


def _other_calls(tp):
    calls = {}

    def xent(T, D, V, dtype):
        X, W, t, dloss = _xent_inputs(T, D, V, dtype, seed=T + V)
        _, lse = tp.tpmlp_xent_forward(X, W, t)
        calls[f"xent {T} {D} {V} {dtype}"] = lambda s=None: [
            *tp.tpmlp_xent_forward(X, W, t, stream=s), *tp.tpmlp_xent_backward(X, W, t, lse, dloss, stream=s)]

    def embed(T, D, V, dtype):
        g = torch.Generator(device="cuda").manual_seed(T)
        ids, dout = _ids(T, V, T, "words"), torch.randn(T, D, generator=g, device="cuda").to(DT[dtype])
        calls[f"embed {T} {D} {V} {dtype}"] = lambda s=None: [tp.tpmlp_embed_backward(dout, ids, V, 2.0, stream=s)]

    for dtype in DT:
        for T, D, V in ((1, 64, 3000), (7, 200, 5000), (40, 1000, 700), (150, 72, 900), (9000, 24, 30001)):
            xent(T, D, V, dtype)
        for T, D, V in ((1, 768, 3000), (600, 33, 100), (5000, 256, 60000), (70000, 64, 5000)):
            embed(T, D, V, dtype)
    xent(600, 1032, 8300, "bf16")
    return calls


def test_other_sizes_captured_replayed_and_side_by_side(tp):
    calls = _other_calls(tp)
    ref = {k: [v.clone() for v in f()] for k, f in calls.items()}
    torch.cuda.synchronize()
    graphs = {}
    for k, f in calls.items():
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            graphs[k] = graph, f(torch.cuda.current_stream())
    s, r = torch.cuda.Stream(), torch.cuda.Stream()
    names = list(calls)
    for _ in range(2):
        for k in names:
            for v in graphs[k][1]:
                v.fill_(3.0)
        torch.cuda.synchronize()
        got = []
        for a, b in zip(names, reversed(names)):  # one replayed while another runs
            with torch.cuda.stream(s):
                graphs[a][0].replay()
            with torch.cuda.stream(r):
                got.append((b, calls[b](r)))
        torch.cuda.synchronize()
        for k, out in got + [(k, graphs[k][1]) for k in names]:
            assert all(torch.equal(u, v) for u, v in zip(out, ref[k])), k
    tp.tpmlp_check_status()


FIRST_IN_A_GRAPH = r'''
import torch
import tensor_transformer_mlp_column_gb300 as tp
X, W = torch.randn(100, 64, device="cuda"), torch.randn(300, 64, device="cuda")
t = torch.arange(100, device="cuda")
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    loss, lse = tp.tpmlp_xent_forward(X, W, t)
    dX, dW = tp.tpmlp_xent_backward(X, W, t, lse, torch.ones_like(loss))
    dE = tp.tpmlp_embed_backward(X, t, 300, dE=dW, accumulate=True)
    norm = tp.tpmlp_grad_clip([dW, dX], 1e6)
graph.replay()
torch.cuda.synchronize()
out = [v.clone() for v in (loss, dX, dW, norm)]
loss, lse = tp.tpmlp_xent_forward(X, W, t)
dX, dW = tp.tpmlp_xent_backward(X, W, t, lse, torch.ones_like(loss))
tp.tpmlp_embed_backward(X, t, 300, dE=dW, accumulate=True)
norm = tp.tpmlp_grad_clip([dW, dX], 1e6)
assert all(torch.equal(a, b) for a, b in zip(out, (loss, dX, dW, norm)))
tp.tpmlp_check_status()
print("ok")
'''


def test_first_calls_of_a_process_in_a_graph(tp):
    import os
    import subprocess
    import sys

    r = subprocess.run([sys.executable, "-c", FIRST_IN_A_GRAPH], capture_output=True, text=True, timeout=600,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout[-2000:] + r.stderr[-4000:]


def test_calls_in_two_streams_at_once(tp):
    a, b = _train_calls(tp, seed=51), _train_calls(tp, seed=52)
    ra, rb = {k: f() for k, f in a.items()}, {k: f() for k, f in b.items()}
    torch.cuda.synchronize()
    s, r = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        got = []
        for k in a:
            with torch.cuda.stream(s):
                x = a[k](s)
            with torch.cuda.stream(r):
                y = b[k](r)
            got.append((k, x, y))
        torch.cuda.synchronize()
        for k, x, y in got:
            assert all(torch.equal(u, v) for u, v in zip(x, ra[k])), k
            assert all(torch.equal(u, v) for u, v in zip(y, rb[k])), k
    tp.tpmlp_check_status()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,D,V", [(63, 64, 300), (300, 264, 1000), (2101, 72, 700)])
def test_ids_and_rows_on_their_own_boundaries(tp, T, D, V, dtype):
    # The targets of next-token prediction are the ids one further on; loss, lse and dloss parts of larger tensors.
    X, W, t, dloss = _xent_inputs(T, D, V, dtype, seed=T)
    row = torch.cat([t[:1], t])

    def shifted(v):
        return torch.cat([v[:1], v])[1:]

    loss, lse = (torch.zeros(T + 2, device="cuda") for _ in range(2))
    tp.tpmlp_xent_forward(X, W, row[1:], loss=loss[1:-1], lse=lse[1:-1])
    ref = tp.tpmlp_xent_forward(X, W, t)
    assert torch.equal(loss[1:-1], ref[0]) and torch.equal(lse[1:-1], ref[1])
    assert loss[0] == loss[-1] == lse[0] == lse[-1] == 0
    got = tp.tpmlp_xent_backward(X, W, row[1:], lse[1:-1], shifted(dloss))
    for a, b in zip(got, tp.tpmlp_xent_backward(X, W, t, ref[1], dloss)):
        assert torch.equal(a, b)
    ids = t.clamp(min=0)
    assert torch.equal(tp.tpmlp_embed_forward(W, shifted(ids)), tp.tpmlp_embed_forward(W, ids))
    assert torch.equal(tp.tpmlp_embed_backward(X, shifted(ids), V), tp.tpmlp_embed_backward(X, ids, V))
    norms = torch.zeros(3, device="cuda")
    tp.tpmlp_grad_norm([X, W], norm=norms[1:2])
    assert norms[1] == tp.tpmlp_grad_norm([X, W])[0] and norms[0] == norms[2] == 0
    tp.tpmlp_check_status()


def test_binding_refuses_wrong_tensors(tp):
    X, W, t, dloss = _xent_inputs(16, 64, 50, "bf16", seed=61)
    with pytest.raises(ValueError):
        tp.tpmlp_xent_forward(X, W[:, :32].contiguous(), t)
    with pytest.raises(ValueError):
        tp.tpmlp_xent_forward(X, W.float(), t)
    with pytest.raises(ValueError):
        tp.tpmlp_xent_forward(X, W, t.int())
    with pytest.raises(ValueError):
        tp.tpmlp_xent_forward(X, W, t[:5])
    with pytest.raises(ValueError):
        tp.tpmlp_xent_forward(X.t(), W, t)
    with pytest.raises(ValueError):
        tp.tpmlp_xent_forward(X.cpu(), W, t)
    with pytest.raises(ValueError):
        tp.tpmlp_xent_forward(X, W, t, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        tp.tpmlp_xent_backward(X, W, t, dloss, dloss, dX=torch.empty(16, 64, device="cuda"))
    with pytest.raises(ValueError):
        tp.tpmlp_embed_backward(X, t, 50, accumulate=True)
    with pytest.raises(ValueError):
        tp.tpmlp_embed_forward(W, t.to(torch.int32))
    tp.tpmlp_check_status()


def test_binding_refuses_a_wrong_loss(tp):
    X, W, t, dloss = _xent_inputs(16, 64, 50, "bf16", seed=62)
    loss, lse = tp.tpmlp_xent_forward(X, W, t)
    for bad in (loss[:5], loss.double(), loss.cpu(), torch.stack([loss, loss], 1)[:, 0]):
        with pytest.raises(ValueError):
            tp.tpmlp_xent_backward(X, W, t, lse, dloss, loss=bad)
    tp.tpmlp_check_status()


def test_ids_out_of_range_are_named(tp):
    X, W, t, _ = _xent_inputs(9, 64, 50, "bf16", seed=63, masked=0.0)
    ids = t.clone()
    ids[3] = 50
    for call, what in ((lambda: tp.tpmlp_xent_forward(X, W, ids), "target id"), (lambda: tp.tpmlp_embed_forward(W, ids), "token id"),
                       (lambda: tp.tpmlp_embed_backward(X, ids, 50), "token id")):
        call()
        with pytest.raises(tp.TpmlpError, match=what) as e:
            tp.tpmlp_check_status()
        assert e.value.code == tp.TPMLP_ERR_BOUNDS
        tp.tpmlp_check_status()

def test_xent_backward_workspace_holds_partial_sums(tp):
    # How many follows the SMs. Sizes at which they are the largest part: dX's of few rows, dW's of many rows and a small vocabulary.
    ws = tp.lib().tpmlp_xent_workspace_bytes
    assert ws(64, 4096, 2000, 1, 1) > 64 * 2000 * 4 + 2 * 64 * 4096 * 4
    assert ws(8192, 512, 300, 1, 1) > 8192 * 300 * 2 + 2 * 300 * 512 * 4


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,D,V", [(1, 64, 3000), (40, 512, 50257), (150, 1000, 20000), (300, 264, 3000), (70, 4200, 2000)])
def test_gradients_from_the_loss_captured_replayed_and_side_by_side(tp, T, D, V, dtype):
    X, W, t, dloss = _xent_inputs(T, D, V, dtype, seed=T + D)
    loss, lse = tp.tpmlp_xent_forward(X, W, t)

    def call(s=None):
        return list(tp.tpmlp_xent_backward(X, W, t, lse, dloss, loss=loss, stream=s))

    ref = [v.clone() for v in call()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(torch.cuda.current_stream())
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        for v in out:
            v.fill_(5.0)
        torch.cuda.synchronize()
        with torch.cuda.stream(a):
            graph.replay()
        with torch.cuda.stream(b):
            other = call(b)
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(out, ref)) and all(torch.equal(u, v) for u, v in zip(other, ref))
    tp.tpmlp_check_status()
