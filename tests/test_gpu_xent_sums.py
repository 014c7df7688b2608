"""What the cross entropy's sums keep of their digits, on the GPU.

The tensor core cuts off, always towards zero, what it shifts out when it adds
16 products to its fp32 accumulator, so a long sum of one sign drifts with its
length: by 1.4 N U32 of itself over N such additions (measured, N = 4096). Long
sums are therefore cut into runs. The bounds here follow from the runs' length,
not from the sum's, so a sum that is not cut does not meet them.

X and W have entries from 1 to 1.125 (W times a power of two), so products are
within a factor q = 1.27 of one another and the i-th of n partial sums is at
most q i / n of the whole. Allowed are
  for a run of n additions a step, 2 U32, each:  2 U32 q (n + 1) / 2 of the run
  (bf16 products are multiples of 2^-14 here, so the first 512 of a run are added
  exactly and the next 512 lose at most their last bits),
  for R additions of runs, rounded to nearest:   U32 q (R + 1) / 2 of the sum,
  and 2 U32 where what an addition leaves out is carried over.
U16 = 2^-8 is half a step of bf16, U32 = 2^-24 of fp32.
"""

import pytest
import torch

pytestmark = pytest.mark.gpu

U16, U32 = 2.0 ** -8, 2.0 ** -24
Q = 1.27
V = 40
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


def _ones(g, shape, dtype):
    """Entries from 1 to 1.125, of all mantissas that the type has there."""
    if dtype == "bf16":
        return (1 + torch.randint(0, 16, shape, generator=g, device="cuda") / 128.0).bfloat16()
    return 1 + torch.rand(shape, generator=g, device="cuda") / 8


def _scale(D):
    return 2.0 ** -(D.bit_length() - 7)  # D times it: 64, logits of about 72


def _run(n):
    return Q * (n + 1)


def _joined(R):
    return Q * (R + 1) / 2


# (rows, D, bound in U32 of the sum). A K block is 64 products, four additions.
LONG = [
    # Up to 2 rows: runs of 4 K blocks over four accumulators, one addition of a block each; carried over.
    ("bf16", 1, 1 << 20, _run(4) + 2), ("bf16", 2, 1 << 20, _run(4) + 2),
    # Up to 32: of 8.
    ("bf16", 3, 1 << 20, _run(8) + 2), ("bf16", 32, 1 << 20, _run(8) + 2),
    # Up to 64: of 16, four sums each to be joined.
    ("bf16", 64, 1 << 18, _run(16) + _joined(4 * (1 << 18) // 1024)),
    # One accumulator. Up to 256 rows 8 K blocks, above that 16.
    ("bf16", 200, 1 << 16, _run(32) + _joined((1 << 16) // 512)),
    ("bf16", 1000, 1 << 16, _run(64) + _joined((1 << 16) // 1024)),
    # fp32: six products of bf16 pieces; three that are dropped, together below 4 U32. Few rows: three sums a run, of which
    # the two of the lower pieces are below 2^-7 of the first.
    ("f32", 1, 1 << 16, _run(16) + _run(32) * 2.0 ** -6 + _joined(3 * (1 << 16) // 256) + 4),
    ("f32", 32, 1 << 16, _run(16) + _run(32) * 2.0 ** -6 + _joined(3 * (1 << 16) // 256) + 4),
    ("f32", 64, 1 << 16, _run(32) + _run(64) * 2.0 ** -6 + _joined(3 * (1 << 16) // 512) + 4),
    # Many rows: the lower pieces' products first, in runs of 128 K blocks, then the high ones' in runs of 8.
    ("f32", 300, 1 << 16, _run(32) + _run(512) * 2.0 ** -6 + _joined((1 << 16) // 512 + 40) + 4),
]


@pytest.mark.parametrize("dtype,T,D,bound", LONG, ids=lambda v: str(v) if not isinstance(v, float) else "")
def test_statistics_of_long_sums(tp, dtype, T, D, bound):
    # One id with a long sum, all others and the target with none: lse is that sum, and so is the loss. Few rows take
    # several ids in turn, since a sum rounded at random may come out well by chance.
    g = torch.Generator(device="cuda").manual_seed(D + T)
    X = _ones(g, (T, D), dtype)
    t = torch.full((T,), V - 1, device="cuda")
    for at in range(1 if T > 8 else 16 // T):
        W = torch.zeros(V, D, device="cuda", dtype=DT[dtype])
        W[at] = _ones(g, (D,), dtype) * _scale(D)
        loss, lse = tp.tpmlp_xent_forward(X, W, t)
        want = X.double() @ W[at].double()
        # Beside the sum: z times log2 e and back, the logarithm, the result's rounding, each a U32; 39 ids at exp(-64).
        tol = want * (bound + 6) * U32 + 1e-20
        for got, what in ((lse, "lse"), (loss, "loss")):
            err = (got.double() - want).abs()
            assert bool((err <= tol).all()), (what, at, (err / want / U32).max().item(), bound + 6)
    tp.tpmlp_check_status()


@pytest.mark.parametrize("dtype,T", [("bf16", 1), ("bf16", 20), ("bf16", 64), ("bf16", 100), ("bf16", 600), ("f32", 1),
                                     ("f32", 64), ("f32", 300)])
def test_gradients_of_long_sums(tp, dtype, T):
    # Two ids with long sums share each row's softmax about evenly, the target has neither: dX is their rows times their
    # shares. The backward's own logits have to be about as good as those of lse: 16384 uncut additions lose 1.4 * 16384
    # U32 of 72, and the shares 10 %.
    D = 1 << 18 if dtype == "bf16" else 1 << 16
    g = torch.Generator(device="cuda").manual_seed(T)
    X = _ones(g, (T, D), dtype)
    W = torch.zeros(V, D, device="cuda", dtype=DT[dtype])
    W[3], W[17] = _ones(g, (D,), dtype) * _scale(D), _ones(g, (D,), dtype) * _scale(D)
    t = torch.full((T,), V - 1, device="cuda")
    dloss = torch.rand(T, generator=g, device="cuda") + 0.5
    loss, lse = tp.tpmlp_xent_forward(X, W, t)
    dX, dW = tp.tpmlp_xent_backward(X, W, t, lse, dloss)
    tp.tpmlp_check_status()
    z = X.double() @ W.double().T
    ref = torch.logsumexp(z, 1)[:, None]
    dz = torch.exp(z - ref)
    dz.scatter_add_(1, t[:, None], -torch.ones_like(ref))
    dz *= dloss.double()[:, None]
    # lse: the loosest of the forward's bounds above at this length; the logits: bf16 runs of 16 K blocks, fp32 as above.
    if dtype == "bf16":
        lse_bound, z_bound = _run(64) + _joined(4 * D // 1024), _run(64) + _joined(D // 1024)
        half = 1.01 * (U16 if T > 64 else U16 ** 2)
    else:
        lse_bound = z_bound = _run(32) + _run(512) * 2.0 ** -6 + _joined(3 * D // 256) + 4
        half = 4 * U32
    share = (lse_bound + z_bound + 12) * U32 * z.max()
    edz = dz.abs() * (torch.expm1(share) + half + 16 * U32)
    out = 1.01 * U16 if dtype == "bf16" else 2 * U32
    for got, a, e, b, k in ((dX, dz, edz, W.double(), V), (dW, dz.T, edz.T, X.double(), T)):
        want = a @ b
        # Sums of few terms, T or V of them: as many whole steps at most.
        tol = e @ b.abs() + (a.abs() @ b.abs()) * (6 * k / 16 + 84) * 2 * U32 + out * want.abs() + 1e-30
        err = (got.double() - want).abs()
        assert bool((err <= tol).all()), ((err / tol).max().item(), share.item())


def test_gradient_of_a_long_vocabulary(tp):
    # X = 0: every share is 2^-18 and dX the mean of W's rows (the targets' is zero), sums of one sign over 16384 additions
    # in tiles that fill the GPU, so that nothing is gained by slices of them. The rounding to bf16 averages out over the
    # columns, whose sums have all mantissas: U16 / sqrt(3 * 19456) and less. A run of 256 K blocks has 1024 additions, which
    # lose 1.4 * 1024 U32 = 8.5e-5 of it at most (the products have few bits here); in one sum they lost 4.0e-4.
    T, D, V = 100, 19456, 1 << 18
    g = torch.Generator(device="cuda").manual_seed(1)
    f = 1 + torch.rand(D, generator=g, device="cuda")
    W = torch.empty(V, D, device="cuda", dtype=torch.bfloat16)
    total = torch.zeros(D, device="cuda", dtype=torch.float64)
    for v in range(0, V, 8192):
        W[v:v + 8192] = _ones(g, (8192, D), "bf16") * f
        W[V - 1] = 0
        total += W[v:v + 8192].sum(0, dtype=torch.float64)
    X = torch.zeros(T, D, device="cuda", dtype=torch.bfloat16)
    t = torch.full((T,), V - 1, device="cuda")
    loss, lse = tp.tpmlp_xent_forward(X, W, t)
    dX, dW = tp.tpmlp_xent_backward(X, W, t, lse, torch.ones_like(loss), loss=loss)
    tp.tpmlp_check_status()
    assert bool((dW == 0).all())
    rel = dX.double() / (total / V) - 1
    assert rel.abs().max().item() <= 1.01 * U16 + 1e-3
    assert rel.mean(1).abs().max().item() <= 2 * 8.5e-5 + 5 * U16 / (3 * D) ** 0.5


@pytest.mark.parametrize("T,D,V", [(1, 264, 300), (2, 1032, 1000), (3, 264, 2000), (32, 520, 1000), (64, 264, 3000)])
def test_gradients_of_few_bf16_rows_are_rounded_once(tp, T, D, V):
    # dz of up to 64 rows is two bf16 pieces, off by U16^2 at most, so that what shows in the gradients is their own
    # rounding, U16; one piece would add its U16 to that, the same for all of a row, which some of a row's D columns show.
    g = torch.Generator(device="cuda").manual_seed(T + D)
    W = (torch.randn(V, D, generator=g, device="cuda") / D ** 0.5).bfloat16()
    X = torch.randn(T, D, generator=g, device="cuda").bfloat16()
    t = torch.randperm(V, generator=g, device="cuda")[:T]
    dloss = torch.rand(T, generator=g, device="cuda") + 0.5
    loss, lse = tp.tpmlp_xent_forward(X, W, t)
    dX, dW = tp.tpmlp_xent_backward(X, W, t, lse, dloss, loss=loss)
    tp.tpmlp_check_status()
    z = X.double() @ W.double().T
    ref = torch.logsumexp(z, 1)[:, None]
    dz = torch.exp(z - ref)
    dz.scatter_add_(1, t[:, None], -torch.ones_like(ref))
    dz *= dloss.double()[:, None]
    # Logits and lse: sums of D products, all additions a whole step; exponentials and logarithms a few U32.
    mag = (X.double().abs() @ W.double().abs().T).max()
    ez = mag * (D / 16 + 2) * 2 * U32 + 16 * U32 * (z.abs().max() + 1) + (V / 128 + 64) * 2 * U32
    p = torch.exp(z - ref) * dloss.double()[:, None]
    edz = p * 2.02 * ez + dz.abs() * (1.01 * U16 ** 2 + 16 * U32)
    for got, a, e, b, k in ((dX, dz, edz, W.double(), V), (dW, dz.T, edz.T, X.double(), T)):
        want = a @ b
        tol = e @ b.abs() + (a.abs() @ b.abs()) * (2 * k / 16 + 84) * 2 * U32 + 1.001 * U16 * want.abs() + 1e-30
        err = (got.double() - want).abs()
        assert bool((err <= tol).all()), (err / tol).max().item()
