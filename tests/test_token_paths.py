"""The token operators' variants that only large work reaches: streamed stores and loads, and a vocabulary that
is gone over in pieces."""
import math

import pytest
import torch

from coo_spmm_fwd_amd import binding as csp
from coo_spmm_fwd_amd import token_ops as ops
from tests.test_token_ops import BF16, F32, U32, ce_check, ce_inputs, gen, u, within


def beyond(n, dtype, seed):
    """n random elements that start one element past a 16-byte boundary."""
    return torch.randn(n + 1, generator=gen(seed), device="cuda").to(dtype)[1:]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,N,V,D", [(F32, 9001, 700, 1001), (BF16, 18001, 700, 1001), (BF16, 8192, 300, 2048)])
def test_lookup_of_more_than_the_cache(dtype, N, V, D):
    """Y of 32 MiB and more is streamed."""
    assert N * D * dtype.itemsize >= 32 << 20
    E, Y = beyond(V * D, dtype, 1).view(V, D), beyond(N * D, dtype, 2).view(N, D)
    ids = torch.randint(-1, V + 1, (N,), generator=gen(3), device="cuda")
    part = (ids >= 0) & (ids < V)
    csp.embed_fwd(E, ids, 0.25, Y=Y)
    want = torch.where(part[:, None], E[ids.clamp(0, V - 1)] * 0.25, torch.zeros((), dtype=dtype, device="cuda"))
    assert torch.equal(Y, want)                        # exact: a power of two


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,N,V,D", [(F32, 5003, 60_001, 1001), (BF16, 5003, 125_001, 1001), (BF16, 40_000, 300, 2000)])
def test_lookup_gradient_of_more_than_the_cache(dtype, N, V, D):
    """dE and twice dY past 256 MiB: dE is streamed.  Small integers, so that every sum is exact."""
    assert (V + 2 * N) * D * dtype.itemsize > 256 << 20
    dY = torch.randint(-2, 3, (N * D + 1,), generator=gen(4), device="cuda").to(dtype)[1:].view(N, D)
    ids = torch.randint(0, V, (N,), generator=gen(5), device="cuda")
    ids[::3] = 17                                       # a token that is cut into pieces
    ids[1::100] = -1
    dE = beyond(V * D, dtype, 6).view(V, D)
    csp.embed_bwd(dY, ids, V, 0.5, dE=dE)
    part = (ids >= 0).nonzero()[:, 0]
    want = torch.zeros(V, D, device="cuda").index_add_(0, ids[part], dY[part].float()) * 0.5
    assert torch.equal(dE, want.to(dtype))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,N,V,D", [(F32, 100, 66_001, 1025), (BF16, 33, 66_001, 2051), (BF16, 3, 33_000, 4160)])
def test_few_tokens_beside_a_head_of_more_than_the_cache(dtype, N, V, D):
    """W past 256 MiB is streamed in the backward."""
    assert V * D * dtype.itemsize > 256 << 20
    X, W, t = ce_inputs(N, V, D, dtype, 7, "some")
    t[0] = V - 1
    odd = torch.empty(V * D + 1, dtype=dtype, device="cuda")[1:].view(V, D).copy_(W)
    ce_check(X, odd, t)


@pytest.mark.gpu
@pytest.mark.parametrize("inplace", [False, True])
def test_clipping_more_than_the_cache(inplace):
    """More than 64 tensors, more than 128 MiB: the table in the workspace, and streamed outputs."""
    sizes = [400_001 + 37 * i for i in range(110)]
    dtypes = [BF16 if i % 3 == 1 else F32 for i in range(110)]
    gs = [beyond(n, t, 100 + i) for i, (n, t) in enumerate(zip(sizes, dtypes))]
    assert sum(n * t.itemsize for n, t in zip(sizes, dtypes)) > 128 << 20
    ref = math.sqrt(sum(float(g.double().square().sum()) for g in gs))
    m = 2.0 ** math.floor(math.log2(ref * 0.5))
    c = m / (ref + 1e-6)
    want = [g.double() * c for g in gs]
    outs = gs if inplace else [torch.full_like(g, 7.0) for g in gs]
    norm = csp.grad_clip(gs, m, outs=None if inplace else outs)
    assert abs(float(norm) - ref) <= 2 * U32 * ref
    for o, w in zip(outs, want):
        tol = 6 * U32 * w.abs()
        within(o, w, tol + u(o.dtype) * (w.abs() + tol) + 2.0 ** -149, "clipped")


def pieces(N, V, D, dtype, backward):
    """Whether a call goes over the vocabulary in pieces: of its workspace, what still grows with it are the maxima
    and sums (the backward: four sums), 8 (16) bytes a token (of a multiple of 256) and 256 vocabulary rows."""
    L, dt = csp.load(), csp.CSP_BF16 if dtype is BF16 else csp.CSP_F32
    more = L.linear_ce_workspace(N, V + 512, D, dt, backward) - L.linear_ce_workspace(N, V, D, dt, backward)
    return more == 2 * (16 if backward else 8) * (-(-N // 256) * 256)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,N,V,D,how", [
    (BF16, 16_500, 66_001, 64, (False, True)),      # W as it is, P in pieces
    (BF16, 16_500, 66_001, 65, (False, True)),      # W copied
    (BF16, 130, 240_001, 513, (True, True)),      # copies of W in pieces
    (F32, 11_000, 66_001, 40, (False, True)),
    (F32, 130, 360_001, 500, (True, True))])
def test_linear_ce_in_pieces(dtype, N, V, D, how):
    assert (pieces(N, V, D, dtype, 0), pieces(N, V, D, dtype, 1)) == how
    X, W, t = ce_inputs(N, V, D, dtype, 8, "some")
    t[0], t[1] = V - 1, 0
    ce_check(X, W, t)


@pytest.mark.gpu
def test_more_tiles_than_a_launch_holds():
    """2^21 tokens, few of which take part, and 300001 vocabulary rows: 9.6 million tiles, 4.9e9 threads."""
    N, V, D = 2**21 + 300, 300_001, 64
    assert -(-N // 256) * -(-V // 256) * 512 > 2**32
    W = (torch.randn(V, D, generator=gen(9), device="cuda") / 4).bfloat16()
    X = torch.randn(N, D, generator=gen(10), device="cuda").bfloat16()
    t = torch.full((N,), -100, device="cuda")
    rows = torch.arange(5, N, 9973, device="cuda")
    t[rows] = torch.randint(0, V, rows.shape, generator=gen(11), device="cuda")
    t[rows[0]], t[rows[-1]] = V - 1, 0
    loss, lse, total = csp.linear_ce_fwd(X, W, t)
    one, oness, _ = csp.linear_ce_fwd(X[rows], W, t[rows])     # the same tokens alone
    assert torch.equal(loss[rows], one) and torch.equal(lse[rows], oness)
    assert float(total[1]) == rows.numel() and not loss[t < 0].any()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("N,V,D", [(0, 40, 24), (1, 500, 33), (40, 300, 100), (64, 1000, 64), (100, 700, 72),
                                   (200, 300, 65), (300, 9000, 64), (700, 30_000, 128)])
def test_one_gradient_alone_is_that_of_both(N, V, D, dtype):
    X, W, t = ce_inputs(N, V, D, dtype, 12, "some")
    _, lse, total = csp.linear_ce_fwd(X, W, t)
    args = X, W, t, lse, torch.full((1,), 0.5, device="cuda"), total
    dX, dW = csp.linear_ce_bwd(*args)
    assert torch.equal(csp.linear_ce_bwd_input(*args), dX) and torch.equal(csp.linear_ce_bwd_weight(*args), dW)


@pytest.mark.gpu
def test_a_frozen_head_costs_no_gradient_of_it():
    N, V, D = 48, 50_000, 512
    X, W, t = ce_inputs(N, V, D, F32, 13, "none")
    peak = {}
    for frozen in (False, True):
        x, w = X.clone().requires_grad_(), W.clone().requires_grad_(not frozen)
        loss = ops.linear_cross_entropy(x, w, t)
        torch.cuda.reset_peak_memory_stats()
        before = torch.cuda.memory_allocated()
        loss.backward()
        peak[frozen] = torch.cuda.max_memory_allocated() - before
        assert (w.grad is None) == frozen and torch.isfinite(x.grad).all()
    assert peak[False] - peak[True] > 0.9 * V * D * 4


@pytest.mark.gpu
def test_lookup_of_more_rows_than_a_launch_holds():
    """4 rows of 33 vectors a workgroup: 2^26 rows and some are two launches (35 GB)."""
    N, V, D = 2**26 + 1001, 5, 132
    E = torch.randn(V, D, generator=gen(14), device="cuda")
    ids = torch.arange(N, device="cuda") % (V + 1)              # the last is none
    Y = csp.embed_fwd(E, ids, 2.0)
    want = torch.cat([E * 2.0, torch.zeros(1, D, device="cuda")])
    for n in range(0, N, 6 << 20):                              # a multiple of V + 1
        part = Y[n:n + (6 << 20)]
        assert torch.equal(part, want.repeat(-(-part.shape[0] // (V + 1)), 1)[:part.shape[0]]), n
