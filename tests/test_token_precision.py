"""What the linear cross entropy and its gradient hold on to: the digits of P, of small losses and of
long sums, and infinite logits, against 64-bit forms.

u(t) = finfo(t).eps / 2 is the largest relative error of one rounding to t.
"""
import math

import pytest
import torch

from coo_spmm_fwd_amd import binding as csp
from coo_spmm_fwd_amd import token_ops as ops
from tests.test_token_ops import BF16, F32, U32, ce_inputs, gen, u, within

# P stands beside bf16 operands as a sum of two bf16 numbers: the rest of the first rounding, 2^-8 of P
# at most, is rounded again.  Beside fp32 operands three of them hold all 24 bits.
P_ERROR = {BF16: u(BF16) ** 2, F32: 0.0}


def gradient_reference(X, W, t, target_error=None):
    """dX and dW of the mean loss in 64 bits, and how far fp32 sums and P_ERROR may put them off.
    target_error: relative error of the target's element of G, otherwise that of p - 1."""
    N, V, D = X.shape[0], W.shape[0], X.shape[1]
    rows = ((t >= 0) & (t < V)).nonzero()[:, 0]
    at = (torch.arange(rows.numel(), device="cuda"), t[rows])
    Xd, Wd = X.double()[rows], W.double()
    z = Xd @ Wd.T
    lse = torch.logsumexp(z, 1)
    ez = (D + 8) * U32 * (Xd.abs() @ Wd.abs().T)
    el = ez.amax(1) + (V + 16) * U32 + 4 * U32 * (z.abs().amax(1) + lse.abs())
    G = torch.exp(z - lse[:, None])
    dG = G * (torch.expm1(ez + el[:, None]) + 8 * U32)
    zt = z[at]
    G[at] = torch.expm1(-torch.nn.functional.softplus(torch.logsumexp(z.index_put(at, torch.full_like(zt, -math.inf)), 1) - zt))
    dG = dG + U32 * G.abs()
    if target_error is not None:
        dG[at] = (target_error(ez, z, lse) + 8 * U32) * G[at].abs()
    dG = dG + P_ERROR[X.dtype] * (G.abs() + dG)
    k = 1.0 / max(1, rows.numel())
    dX, eX = torch.zeros(2, N, D, dtype=torch.float64, device="cuda")
    dX[rows] = G @ Wd * k
    eX[rows] = (dG @ Wd.abs() + (V + 8) * U32 * (G.abs() @ Wd.abs())) * k
    Gt, dGt = G.T.contiguous(), dG.T.contiguous()
    dW = Gt @ Xd * k
    eW = (dGt @ Xd.abs() + (rows.numel() + 8) * U32 * (Gt.abs() @ Xd.abs())) * k
    uo = u(X.dtype)
    return dX, eX + uo * (dX.abs() + eX), dW, eW + uo * (dW.abs() + eW)


def gradients(X, W, t):
    X, W = X.clone().requires_grad_(), W.clone().requires_grad_()
    ops.linear_cross_entropy(X, W, t).backward()
    return X.grad, W.grad


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("N,V,D,mask", [(1, 300, 64, "none"), (16, 129, 40, "some"), (33, 260, 96, "none"),
                                        (64, 300, 64, "some"), (65, 300, 64, "none"), (128, 257, 100, "some"),
                                        (129, 300, 64, "none"), (200, 4000, 64, "none"), (600, 40, 32, "some"),
                                        (300, 9000, 33, "some"), (1500, 20000, 64, "none")])
def test_gradients_hold_the_digits_of_p(N, V, D, mask, dtype):
    """Each form (few tokens, logits kept in parts, tiles): one rounding of P to bf16 would show."""
    X, W, t = ce_inputs(N, V, D, dtype, N + V + D, mask)
    dX, eX, dW, eW = gradient_reference(X, W, t)
    gX, gW = gradients(X, W, t)
    within(gX, dX, eX, "dX")
    within(gW, dW, eW, "dW")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("N,V,D", [(1, 700, 96), (40, 700, 96), (100, 700, 96), (200, 30000, 96), (300, 300, 96)])
def test_gradients_of_small_losses_keep_their_digits(N, V, D, dtype):
    """Losses down to 1e-7 beside logits of 25: the target's element of G is 1 - p = 1 - e^-loss, which p - 1
    with p = exp(z - lse) has lost.  It is off by what the loss is off by: d loss = (1 - e^-loss) dd, with d
    the others' log-sum less the target's logit."""
    g = gen(38)
    t = torch.randint(0, V, (N,), generator=g, device="cuda")
    W = torch.randn(V, D, generator=g, device="cuda").to(dtype)
    lift = torch.linspace(0.1, 0.3, N, device="cuda")[:, None] if N > 1 else torch.full((1, 1), 0.25, device="cuda")
    X = (W.float()[t] * lift).to(dtype)

    def error(ez, z, lse):
        return torch.expm1(2 * ez.amax(1) + (V + 16) * U32 + 4 * U32 * (z.abs().amax(1) + lse.abs()))

    dX, eX, dW, eW = gradient_reference(X, W, t, error)
    gX, gW = gradients(X, W, t)
    within(gX, dX, eX, "dX")
    within(gW, dW, eW, "dW")


@pytest.mark.gpu
@pytest.mark.parametrize("N", [1, 16, 17, 32, 33, 64, 65, 130])
def test_an_infinite_logit_counts_as_nothing(N):
    """bf16 rows of W with -inf where X is positive: logits of -inf, whichever part of the width they are in."""
    V, D = 1100, 700
    X, W, t = ce_inputs(N, V, D, BF16, 40, "none")
    X = X.abs() + 1.0
    t = t // 8 * 8 + 1                                          # never one of the rows below
    W = W / 16                                                  # sums of positive terms stay moderate
    at = torch.arange(0, V, 8, device="cuda")
    W[at, (at * 37) % D] = -math.inf
    loss, lse, total = csp.linear_ce_fwd(X, W, t)
    keep = torch.ones(V, dtype=torch.bool, device="cuda")
    keep[at] = False
    z = X.double() @ W[keep].double().T
    want = torch.logsumexp(z, 1)
    zt = (X.double() * W[t].double()).sum(1)
    ez = (D + 8) * U32 * (X.double() @ W[keep].double().abs().T).amax(1)
    tol = ez + (V + 16) * U32 + 4 * U32 * (z.abs().amax(1) + want.abs())
    within(lse, want, tol, "lse")
    within(loss, want - zt, tol + ez + U32 * (want - zt).abs(), "loss")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("N", [1, 16, 17, 32])
def test_logits_of_up_to_32_tokens_carry_their_lost_digits(N, dtype):
    """z_0 = 2^14 and 31 terms of 3/8 of its step 2^-9, each in a part of the width of its own: added one by one
    to 2^14 in fp32 they vanish, together they are 11.6 steps.  z_1 = 2^14 alone, so that loss = softplus(z_1 -
    z_0) moves by at least (1 - p) of what is lost.  Off by half a step for each logit."""
    D, small = 32 * 128, 3 * 2.0 ** -12
    X = torch.ones(N, D, device="cuda", dtype=dtype)
    W = torch.zeros(2, D, device="cuda", dtype=dtype)
    W[:, 0] = 2.0 ** 14
    W[0, 128::128] = small
    t = torch.zeros(N, dtype=torch.int64, device="cuda")
    loss, _, _ = csp.linear_ce_fwd(X, W, t)
    want = torch.nn.functional.softplus(torch.full((N,), -31 * small, dtype=torch.float64, device="cuda"))
    within(loss, want, torch.full_like(want, 2.0 ** -9 + 8 * U32), "loss")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("N", [0, 5, 100, 300])
def test_no_target_takes_part_whatever_dmean_is(N, dtype):
    """No targets: zero gradients, also where the gradient of the mean is no finite number."""
    X, W, t = ce_inputs(N, 90, 40, dtype, 41, "all")
    _, lse, total = csp.linear_ce_fwd(X, W, t)
    for dmean in (math.inf, math.nan):
        dX, dW = csp.linear_ce_bwd(X, W, t, lse, torch.full((1,), dmean, device="cuda"), total)
        assert not dX.any() and not dW.any()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D", [3, 40])
def test_rows_that_no_id_names_are_zero_whatever_the_scale(D, dtype):
    ids = torch.tensor([2, -1, 7, 2], device="cuda")
    E = torch.ones(5, D, device="cuda", dtype=dtype)
    for scale in (math.inf, math.nan):
        Y = csp.embed_fwd(E, ids, scale)
        assert not Y[[1, 2]].any() and not torch.isfinite(Y[[0, 3]]).any()
        dE = csp.embed_bwd(torch.ones(4, D, device="cuda", dtype=dtype), ids, 5, scale)
        assert not dE[[0, 1, 3, 4]].any() and not torch.isfinite(dE[2]).any()
