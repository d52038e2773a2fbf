"""Token operators (embedding lookup and gradient, linear cross entropy and gradient, gradient norm
and clipping) against plain implementations in 64 bits, at the sizes and masks where they can go
wrong.

Tolerances count roundings, u(t) = finfo(t).eps / 2 each, per output element:
  sums of m fp32 terms      (m + 8) u32 * sum |terms|  (any order; 8 for the scaling and the joins)
  an output in type t       u(t) * |value|
  logits                    ez = (D + 8) u32 * sum_c |X W|
  lse                       max_v ez + (V + 16) u32 + 4 u32 (max |z| + |lse|): the logits, the sum of
                            V exponentials (each off by some u32 of itself), the log and the join
  G                         p (exp(ez + elz) - 1 + 8 u32) and, where G is rounded to bf16 to enter
                            the matrix products of bf16 operands, u(bf16) |G|
  dX, dW                    the errors of G times |W| (|X|), the sums' roundings, the output's
"""
import ctypes
import math

import numpy as np
import pytest
import torch

from coo_spmm_fwd_amd import binding as csp

F32, BF16 = torch.float32, torch.bfloat16
U32 = torch.finfo(F32).eps / 2


def u(t):
    return torch.finfo(t).eps / 2


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def within(got, ref, tol, what):
    err = (got.double() - ref).abs()
    bad = ~(err <= tol)
    if bad.any():
        i = int((err - tol).flatten().nan_to_num(nan=math.inf).argmax())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside; worst at {i}: "
                             f"{got.flatten()[i].item()!r} for {ref.flatten()[i].item()!r}, "
                             f"tolerance {(tol + 0 * err).flatten()[i].item()!r}")


# ------------------------------------------------------------------------------- refusals (CPU)
P = ctypes.c_void_p(4096)


@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(csp.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return csp.load()


def test_embed_refusals(lib):
    assert lib.embed_fwd(P, P, 4, 0, 8, 0, 1.0, P, None) == -1                    # V
    assert lib.embed_fwd(P, P, -1, 5, 8, 0, 1.0, P, None) == -1                   # N
    assert lib.embed_fwd(P, P, 4, 5, 0, 0, 1.0, P, None) == -1                    # D
    assert lib.embed_fwd(P, P, 4, 2**31, 8, 0, 1.0, P, None) == -1
    assert lib.embed_fwd(P, P, 4, 5, 8, 7, 1.0, P, None) == -6                    # dtype
    assert lib.embed_fwd(None, P, 4, 5, 8, 0, 1.0, P, None) == -1
    assert lib.embed_fwd(P, None, 4, 5, 8, 0, 1.0, P, None) == -1
    assert lib.embed_fwd(P, P, 4, 5, 8, 0, 1.0, None, None) == -1
    assert lib.embed_fwd(ctypes.c_void_p(4098), P, 4, 5, 8, 0, 1.0, P, None) == -1   # fp32 at 2 bytes
    assert lib.embed_fwd(P, ctypes.c_void_p(4100), 4, 5, 8, 0, 1.0, P, None) == -1   # int64 at 4 bytes
    assert lib.embed_fwd(P, P, 0, 5, 8, 0, 1.0, P, None) == 0                     # no tokens: nothing to do
    need = lib.embed_bwd_workspace(4, 5, 8, 0)
    assert need > 0
    assert lib.embed_bwd(P, P, 4, 5, 8, 0, 1.0, P, P, need - 1, None) == -1
    assert "workspace" in csp.sparse_layer_last_error()
    assert lib.embed_bwd(P, P, 4, 5, 8, 0, 1.0, P, None, need, None) == -1
    assert lib.embed_bwd(P, P, 4, 5, 8, 0, 1.0, None, P, need, None) == -1
    assert lib.embed_bwd(None, P, 4, 5, 8, 0, 1.0, P, P, need, None) == -1
    assert lib.embed_bwd(P, P, 4, 5, 8, 9, 1.0, P, P, need, None) == -6
    assert lib.embed_bwd_workspace(4, 0, 8, 0) == -1


def test_linear_ce_refusals(lib):
    need = lib.linear_ce_workspace(4, 5, 8, 0, 0)
    fwd = lambda X=P, W=P, t=P, N=4, V=5, D=8, dt=0, loss=P, lse=P, total=P, w=P, nb=need: lib.linear_ce_fwd(
        X, W, t, N, V, D, dt, loss, lse, total, w, nb, None)
    for bad in ({"X": None}, {"W": None}, {"t": None}, {"loss": None}, {"lse": None}, {"total": None}, {"w": None},
                {"nb": need - 1}, {"N": -1}, {"V": 0}, {"D": 0}, {"V": 2**31}, {"X": ctypes.c_void_p(4098)},
                {"t": ctypes.c_void_p(4100)}, {"w": ctypes.c_void_p(4104)}):
        assert fwd(**bad) == -1, bad
    assert fwd(dt=3) == -6
    need_b = lib.linear_ce_workspace(4, 5, 8, 0, 1)
    bwd = lambda X=P, W=P, t=P, N=4, V=5, D=8, dt=0, lse=P, dmean=P, total=P, dX=P, dW=P, w=P, nb=need_b: \
        lib.linear_ce_bwd(X, W, t, N, V, D, dt, lse, dmean, total, dX, dW, w, nb, None)
    for bad in ({"X": None}, {"W": None}, {"t": None}, {"lse": None}, {"dmean": None}, {"total": None}, {"dX": None},
                {"dW": None}, {"w": None}, {"nb": need_b - 1}, {"N": -1}, {"V": 0}, {"D": 0}):
        assert bwd(**bad) == -1, bad
    assert bwd(dt=3) == -6
    assert lib.linear_ce_workspace(4, 5, 0, 0, 0) == -1


def test_grad_clip_refusals(lib):
    need = lib.grad_clip_workspace(2)
    ptrs = (ctypes.c_void_p * 2)(4096, 8192)
    n = (ctypes.c_int64 * 2)(4, 4)
    dt = (ctypes.c_int32 * 2)(0, 1)
    call = lambda g=ptrs, o=ptrs, n=n, dt=dt, c=2, m=1.0, norm=P, w=P, nb=need: lib.grad_clip(
        g, o, n, dt, c, ctypes.c_float(m), norm, w, nb, None)
    for bad in ({"g": None}, {"o": None}, {"n": None}, {"dt": None}, {"c": -1}, {"m": -1.0}, {"m": math.nan},
                {"norm": None}, {"w": None}, {"nb": need - 1}, {"n": (ctypes.c_int64 * 2)(4, -1)},
                {"g": (ctypes.c_void_p * 2)(4098, 8192)}, {"o": (ctypes.c_void_p * 2)(4096, None)}):
        assert call(**bad) == -1, bad
    assert call(dt=(ctypes.c_int32 * 2)(0, 2)) == -6
    assert lib.grad_norm(None, n, dt, 2, P, P, need, None) == -1
    assert lib.grad_clip_workspace(-1) == -1


def test_python_refuses_host_tensors_and_bad_lists():
    t = torch.zeros(4, 8)
    with pytest.raises(TypeError):
        csp.embed_fwd(t, torch.zeros(2, dtype=torch.int64))
    with pytest.raises(TypeError):
        csp.embed_bwd(t, torch.zeros(4, dtype=torch.int64), 5)
    with pytest.raises(TypeError):
        csp.linear_ce_fwd(t, t, torch.zeros(4, dtype=torch.int64))
    with pytest.raises(TypeError):
        csp.grad_clip([t], 1.0)
    with pytest.raises(TypeError):
        csp.grad_norm([t])


# ------------------------------------------------------------------------------- embedding
def embed_inputs(N, V, seed, how):
    g = gen(seed)
    if how == "uniform":
        ids = torch.randint(0, V, (N,), generator=g, device="cuda")
    elif how == "one":      # every token the same
        ids = torch.full((N,), V // 2, device="cuda", dtype=torch.int64)
    elif how == "skewed":   # about 1 / rank
        r = torch.rand(N, generator=g, device="cuda", dtype=torch.float64)
        ids = (torch.exp(r * math.log(V + 1)) - 1).long().clamp_(0, V - 1)
    else:                   # none takes part
        ids = torch.full((N,), -1, device="cuda", dtype=torch.int64)
        ids[::2] = V
        ids[::3] = 2**62
        return ids
    if N > 2 and how != "one":
        ids[torch.rand(N, generator=g, device="cuda") < 0.1] = -1
        ids[N // 2] = V
        ids[N // 3] = -2**63
    return ids


EMBED_CASES = [(1, 1, 1, "uniform"), (1, 300, 768, "uniform"), (2, 5, 3, "uniform"), (7, 13, 1001, "uniform"),
               (64, 3, 64, "uniform"), (65, 1000, 100, "skewed"), (300, 257, 4096, "skewed"), (1000, 1, 129, "one"),
               (4097, 50, 72, "one"), (4097, 3000, 40, "skewed"), (333, 97, 8, "none"), (20000, 700, 48, "skewed"),
               (40000, 65536, 16, "skewed"), (0, 9, 5, "uniform"), (129, 70000, 24, "uniform")]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("N,V,D,how", EMBED_CASES)
def test_embed(N, V, D, how, dtype):
    ids = embed_inputs(N, V, N + V + D, how)
    part = (ids >= 0) & (ids < V)
    scale = float(np.float32(math.sqrt(D) / 3))
    E = torch.randn(V, D, generator=gen(1), device="cuda").to(dtype)
    Y = csp.embed_fwd(E, ids, scale)
    ref = torch.zeros(N, D, dtype=torch.float64, device="cuda")
    ref[part] = E.double()[ids[part]] * scale
    within(Y, ref, (u(dtype) + U32) * (1 + u(dtype)) * ref.abs(), "Y")
    dY = torch.randn(N, D, generator=gen(2), device="cuda").to(dtype)
    dE = csp.embed_bwd(dY, ids, V, scale)
    ref, S = (torch.zeros(V, D, dtype=torch.float64, device="cuda") for _ in range(2))
    ref.index_add_(0, ids[part], dY.double()[part] * scale)
    S.index_add_(0, ids[part], dY.double()[part].abs() * abs(scale))
    m = torch.bincount(ids[part], minlength=V)[:, None]
    t = (m + 8) * U32 * S
    within(dE, ref, t + u(dtype) * (ref.abs() + t), "dE")
    again = csp.embed_bwd(dY, ids, V, scale)
    assert torch.equal(dE.view(torch.int16), again.view(torch.int16)), "not reproducible"


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("N,V,D,how", [
    (70001, 65536, 8, "skewed"), (150_000, 40_000, 5, "uniform"), (33_000, 200_000, 9, "one"),   # sorted by digits
    (3, 17_000_000, 1, "uniform"), (0, 17_000_000, 2, "uniform"),                                # a very long table
    (64, 9, 31, "one"), (65, 9, 31, "one"), (128, 9, 31, "one"), (129, 300, 516, "one"),         # whole pieces of an id
    (5000, 3, 260, "uniform"), (2049, 256, 2056, "skewed"), (900, 512, 7, "skewed"), (40, 513, 2, "skewed")])
def test_embed_paths(N, V, D, how, dtype):
    """Both sorts, ids of many tokens cut into pieces at and around the cuts, tables of several id ranges."""
    test_embed(N, V, D, how, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("lead", [0, 1, 37, 63])
def test_embed_long_ids_between_short_ones(lead):
    """Pieces of ids of 63 to 200 tokens that begin anywhere between the cuts, exact in integers."""
    sizes = [lead, 64, 65, 1, 63, 128, 129, 0, 200, 3, 66]
    ids = torch.repeat_interleave(torch.arange(len(sizes)), torch.tensor(sizes)).cuda()
    ids = ids[torch.randperm(ids.numel(), generator=torch.Generator().manual_seed(lead)).cuda()]
    dY = torch.randint(-8, 9, (ids.numel(), 20), generator=gen(lead), device="cuda").float()
    want = torch.zeros(len(sizes) + 2, 20, dtype=torch.float64, device="cuda").index_add_(0, ids, dY.double())
    assert torch.equal(csp.embed_bwd(dY, ids, len(sizes) + 2).double(), want)
    got = csp.embed_bwd(dY.bfloat16(), ids, len(sizes) + 2)
    assert torch.equal(got, want.float().bfloat16())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_embed_at_element_alignment(dtype):
    """Tables, gradients and outputs that start one element past a 16-byte boundary."""
    N, V, D = 70, 40, 96
    ids = embed_inputs(N, V, 5, "uniform")
    part = (ids >= 0) & (ids < V)
    off = lambda r, seed: torch.randn(r * D + 1, generator=gen(seed), device="cuda").to(dtype)[1:].view(r, D)
    E, dY = off(V, 3), off(N, 4)
    Y = csp.embed_fwd(E, ids, 0.5, Y=off(N, 5))
    dE = csp.embed_bwd(dY, ids, V, 0.5, dE=off(V, 6))
    assert torch.equal(Y[part], E[ids[part]] * 0.5) and not Y[~part].any()   # exact: a power of two
    ref = torch.zeros(V, D, dtype=torch.float64, device="cuda").index_add_(0, ids[part], dY.double()[part] * 0.5)
    S = torch.zeros_like(ref).index_add_(0, ids[part], dY.double()[part].abs() * 0.5)
    t = (torch.bincount(ids[part], minlength=V)[:, None] + 8) * U32 * S
    within(dE, ref, t + u(dtype) * (ref.abs() + t), "dE")


@pytest.mark.gpu
def test_embed_keeps_infinities_and_nan_to_their_rows():
    V, D = 37, 80
    E = torch.randn(V, D, device="cuda")
    E[3], E[4] = math.inf, math.nan
    ids = torch.tensor([3, 5, 4, -1, 6], device="cuda")
    Y = csp.embed_fwd(E, ids, 2.0)
    assert torch.isposinf(Y[0]).all() and torch.isnan(Y[2]).all()
    assert torch.isfinite(Y[[1, 3, 4]]).all() and not Y[3].any()
    dY = torch.ones(5, D, device="cuda")
    dY[3], dY[0] = math.nan, math.inf   # the token that takes no part holds NaN
    dE = csp.embed_bwd(dY, ids, V)
    assert torch.isposinf(dE[3]).all() and torch.isfinite(dE[[i for i in range(V) if i != 3]]).all()


# ------------------------------------------------------------------------------- linear cross entropy
def ce_inputs(N, V, D, dtype, seed, mask):
    g = gen(seed)
    t = torch.randint(0, V, (N,), generator=g, device="cuda")
    W = torch.randn(V, D, generator=g, device="cuda") * (2.0 / math.sqrt(D))
    X = torch.randn(N, D, generator=g, device="cuda")
    X += W[t] * torch.rand(N, 1, generator=g, device="cuda") * 4
    if mask == "some" and N:
        t = torch.where(torch.rand(N, generator=g, device="cuda") < 0.4, torch.full_like(t, -100), t)
        t[N // 2] = V
    elif mask == "all":
        t = torch.full_like(t, -1)
    elif mask == "last" and N:
        t[:-1] = -100
    return X.to(dtype), W.to(dtype), t


def ce_reference(X, W, t, dmean):
    """Loss, lse, total, dX, dW in 64 bits from the definition, and their tolerances."""
    dtype = X.dtype
    N, V, D = X.shape[0], W.shape[0], X.shape[1]
    up = u(BF16) if dtype == BF16 else 0.0
    part = (t >= 0) & (t < V)
    z64 = lambda *s: torch.zeros(*s, dtype=torch.float64, device="cuda")
    r = {"loss": z64(N), "lse": z64(N), "dX": z64(N, D), "dW": z64(V, D)}
    tol = {"loss": z64(N), "lse": z64(N), "dX": z64(N, D), "dW": z64(V, D)}
    count = int(part.sum())
    k = dmean / max(1, count)
    Wd, rows = W.double(), part.nonzero()[:, 0]
    sw, sx = z64(V, D), z64(V, D)
    for rr in rows.split(512):
        Xd = X.double()[rr]
        z = Xd @ Wd.T
        ez = (D + 8) * U32 * (Xd.abs() @ Wd.abs().T)
        lse = torch.logsumexp(z, 1)
        el = ez.amax(1) + (V + 16) * U32 + 4 * U32 * (z.abs().amax(1) + lse.abs())
        zt = z.gather(1, t[rr][:, None])[:, 0]
        r["lse"][rr], tol["lse"][rr] = lse, el
        r["loss"][rr] = lse - zt
        tol["loss"][rr] = el + ez.gather(1, t[rr][:, None])[:, 0] + U32 * (lse - zt).abs()
        p = torch.exp(z - lse[:, None])
        G = p.clone()
        G[torch.arange(rr.numel(), device="cuda"), t[rr]] -= 1.0
        dG = p * (torch.expm1(ez + el[:, None]) + 8 * U32) + U32 * G.abs()
        dG = dG + up * (G.abs() + dG)
        r["dX"][rr] = G @ Wd * k
        e = (dG @ Wd.abs() + (V + 8) * U32 * (G.abs() @ Wd.abs())) * abs(k)
        tol["dX"][rr] = e + u(dtype) * (r["dX"][rr].abs() + e)
        r["dW"] += G.T.contiguous() @ Xd * k
        sw += dG.T.contiguous() @ Xd.abs()
        sx += G.abs().T.contiguous() @ Xd.abs()
    e = (sw + (count + 8) * U32 * sx) * abs(k)
    tol["dW"] = e + u(dtype) * (r["dW"].abs() + e)
    s = r["loss"].sum()
    r["total"] = torch.stack([s, torch.full_like(s, count), s / max(1, count)])
    es = tol["loss"].sum() + 4 * U32 * s.abs()
    tol["total"] = torch.stack([es, torch.zeros_like(s), es / max(1, count)])
    return r, tol


def ce_check(X, W, t, dmean=0.75):
    r, tol = ce_reference(X, W, t, dmean)
    loss, lse, total = csp.linear_ce_fwd(X, W, t)
    g = torch.full((1,), dmean, device="cuda")
    dX, dW = csp.linear_ce_bwd(X, W, t, lse, g, total)
    got = {"loss": loss, "lse": lse, "total": total, "dX": dX, "dW": dW}
    for name in ("lse", "loss", "total", "dX", "dW"):
        within(got[name], r[name], tol[name], name)
    again = csp.linear_ce_fwd(X, W, t)
    dX2, dW2 = csp.linear_ce_bwd(X, W, t, lse, g, total)
    for a, b in zip((loss, lse, total, dX, dW), (*again, dX2, dW2)):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16)), "not reproducible"
    return got


CE_CASES = [(1, 1, 1, "none"), (1, 2, 3, "none"), (1, 1000, 64, "none"), (1, 50257, 96, "none"), (2, 65, 17, "some"),
            (5, 257, 200, "some"), (16, 300, 128, "none"), (31, 64, 100, "some"), (32, 1000, 257, "none"),
            (33, 63, 64, "last"), (63, 129, 33, "some"), (64, 500, 320, "none"), (65, 511, 64, "some"),
            (100, 1500, 96, "all"), (127, 256, 130, "some"), (128, 1024, 192, "none"), (129, 1025, 448, "some"),
            (255, 300, 64, "none"), (257, 513, 65, "some"), (300, 2000, 520, "last"), (513, 1031, 200, "some"),
            (777, 3001, 129, "some"), (1024, 768, 256, "none"), (0, 40, 24, "none"), (300, 1, 40, "some"),
            (600, 8, 8, "none")]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("N,V,D,mask", CE_CASES)
def test_linear_ce(N, V, D, mask, dtype):
    got = ce_check(*ce_inputs(N, V, D, dtype, N + 3 * V + D, mask))
    if mask == "all":
        assert not got["dX"].any() and not got["dW"].any() and not got["total"].any()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("N,V,D,mask", [(1, 127, 65, "none"), (3, 128, 2100, "some"), (15, 129, 127, "none"),
                                        (16, 31, 1001, "some"), (17, 4097, 768, "some"), (32, 33, 513, "last"),
                                        (40, 700, 2100, "some"), (48, 2049, 36, "all"), (64, 12800, 1024, "some"),
                                        (64, 5, 4100, "none"), (64, 40, 7, "some"), (61, 9001, 129, "some"),
                                        (65, 129, 127, "some"), (100, 700, 2100, "some"), (128, 12800, 512, "none"),
                                        (128, 5, 4100, "some"), (97, 260, 65, "last"), (111, 4097, 48, "all")])
def test_linear_ce_few_tokens(N, V, D, mask, dtype):
    """Up to 64 tokens (128 in fp32): parts of a wave's 32 and a workgroup's 128 vocabulary rows, chunks and groups of columns
    that end inside or at a 16-byte load."""
    got = ce_check(*ce_inputs(N, V, D, dtype, N + 3 * V + D, mask))
    if mask == "all":
        assert not got["dX"].any() and not got["dW"].any() and not got["total"].any()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("N,V,D,mask", [(129, 500, 2241, "none"), (300, 257, 1100, "some"), (1030, 255, 700, "some"),
                                        (2056, 707, 1472, "some"), (700, 3, 600, "last"), (4000, 600, 130, "some"),
                                        (150, 1025, 1030, "all"), (5000, 33, 64, "some"), (260, 1, 1500, "none")])
def test_linear_ce_cut_along_the_depth(N, V, D, mask, dtype):
    """Few tiles: the logits' depth (the width), dX's (the vocabulary) and dW's (the tokens) are cut into parts,
    some of them empty when most targets are masked."""
    got = ce_check(*ce_inputs(N, V, D, dtype, N + 3 * V + D, mask))
    if mask == "all":
        assert not got["dX"].any() and not got["dW"].any() and not got["total"].any()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_linear_ce_over_several_pieces(dtype):
    """So many logits that the backward goes over the vocabulary in pieces."""
    ce_check(*ce_inputs(3000, 66001, 24, dtype, 9, "some"))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D", [64, 96])
def test_linear_ce_at_element_alignment(dtype, D):
    """Matrices that start one element past a 16-byte boundary."""
    N, V = 90, 333
    X, W, t = ce_inputs(N, V, D, dtype, 21, "some")
    shift = lambda a: torch.cat([a.flatten()[:1], a.flatten()])[1:].view(a.shape)
    X, W = shift(X), shift(W)
    assert X.data_ptr() % 16 and W.data_ptr() % 16
    ce_check(X, W, t)
    _, lse, total = csp.linear_ce_fwd(X, W, t)
    g = torch.ones(1, device="cuda")
    want = csp.linear_ce_bwd(X, W, t, lse, g, total)
    got = csp.linear_ce_bwd(X, W, t, lse, g, total, dX=shift(X), dW=shift(W))
    assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("N", [12, 300])
def test_masked_rows_may_hold_anything(dtype, N):
    X, W, t = ce_inputs(N, 700, 72, dtype, 33, "some")
    bad = (t < 0) | (t >= 700)
    clean = ce_check(X, W, t)
    Y = X.clone()
    Y[bad] = math.nan
    Y[bad.nonzero()[:1, 0]] = math.inf
    loss, lse, total = csp.linear_ce_fwd(Y, W, t)
    dX, dW = csp.linear_ce_bwd(Y, W, t, lse, torch.full((1,), 0.75, device="cuda"), total)
    for a, name in ((loss, "loss"), (lse, "lse"), (total, "total"), (dX, "dX"), (dW, "dW")):
        assert torch.equal(a, clean[name]), name


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("N", [4, 200])
def test_nan_stays_visible(dtype, N):
    """A NaN in a row that takes part shows in that row's loss and in the total, and in no other row."""
    X, W, t = ce_inputs(N, 260, 64, dtype, 34, "none")
    X[1, 5] = math.nan
    loss, lse, total = csp.linear_ce_fwd(X, W, t)
    assert torch.isnan(loss[1]) and torch.isnan(total[0]) and torch.isfinite(loss[torch.arange(N) != 1]).all()
    dX, dW = csp.linear_ce_bwd(X, W, t, lse, torch.ones(1, device="cuda"), total)
    assert torch.isnan(dX[1]).all() and torch.isfinite(dX[torch.arange(N) != 1]).all() and torch.isnan(dW).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("N", [3, 150])
def test_large_logits_do_not_overflow(dtype, N):
    X, W, t = ce_inputs(N, 400, 64, dtype, 35, "none")
    X, W = X * 64, W * 32   # logits of thousands: exp overflows without the maximum
    loss, lse, total = csp.linear_ce_fwd(X, W, t)
    assert torch.isfinite(loss).all() and torch.isfinite(lse).all() and (lse.abs().max() > 1000)
    r, tol = ce_reference(X, W, t, 1.0)
    within(lse, r["lse"], tol["lse"], "lse")
    within(loss, r["loss"], tol["loss"], "loss")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("N,V,D", [(1, 700, 96), (40, 700, 96), (200, 30000, 96), (300, 300, 96)])
def test_small_losses_keep_their_digits(N, V, D, dtype):
    """Losses down to 1e-6 beside logits of 20.  loss = log(1 + e^d) with d the others' log-sum less the target's
    logit moves by sigmoid(d) = 1 - e^-loss for each unit of d, and d is off by the logits' errors, as lse is."""
    g = gen(37)
    t = torch.randint(0, V, (N,), generator=g, device="cuda")
    W = torch.randn(V, D, generator=g, device="cuda").to(dtype)
    raise_ = torch.linspace(0.1, 0.35, N, device="cuda")[:, None] if N > 1 else torch.full((1, 1), 0.25, device="cuda")
    X = (W.float()[t] * raise_).to(dtype)
    loss, lse, total = csp.linear_ce_fwd(X, W, t)
    Xd, Wd = X.double(), W.double()
    z = Xd @ Wd.T
    zt = z.gather(1, t[:, None])[:, 0]
    others = z.scatter(1, t[:, None], -math.inf)
    d = torch.logsumexp(others, 1) - zt
    want = torch.nn.functional.softplus(d)
    assert want.min() < 1e-3
    ez = (D + 8) * U32 * (Xd.abs() @ Wd.abs().T).amax(1)
    off = 2 * ez + (V + 16) * U32 + 4 * U32 * (z.abs().amax(1) + torch.logsumexp(z, 1).abs())
    within(loss, want, torch.expm1(off) * (1 - torch.exp(-want)) + 8 * U32 * want, "loss")
    assert (loss[want > 1e-12] > 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("N", [3, 100])
def test_gradient_against_differences(N):
    """(f(x + h d) - f(x - h d)) / 2h along random directions.  With logits moved by at most a = h |d.w|
    the central difference is off by at most the third derivative of the loss along it, |d3| <= 2 (range
    of the logits' change per h)^3, times h^2 / 6, and by the losses' own error over h."""
    X, W, t = ce_inputs(N, 300, 40, F32, 36, "none")
    one = torch.ones(1, device="cuda")
    _, lse, total = csp.linear_ce_fwd(X, W, t)
    dX, dW = csp.linear_ce_bwd(X, W, t, lse, one, total)
    _, tol = ce_reference(X, W, t, 1.0)
    f = lambda X, W: csp.linear_ce_fwd(X, W, t)[2][2].double()
    h = 2.0 ** -6
    for seed in range(4):
        d = torch.randn(X.shape, generator=gen(seed), device="cuda") / 8
        zr = 2 * (d.double() @ W.double().T).abs().amax()
        want = (dX.double() * d.double()).sum()
        slack = 2 * zr**3 * h * h / 6 + 4 * tol["total"][2] / h + (tol["dX"] * d.double().abs()).sum()
        assert abs((f(X + h * d, W) - f(X - h * d, W)) / (2 * h) - want) <= slack
        d = torch.randn(W.shape, generator=gen(9 + seed), device="cuda") / 8
        zr = 2 * (X.double() @ d.double().T).abs().amax()
        want = (dW.double() * d.double()).sum()
        slack = 2 * zr**3 * h * h / 6 + 4 * tol["total"][2] / h + (tol["dW"] * d.double().abs()).sum()
        assert abs((f(X, W + h * d) - f(X, W - h * d)) / (2 * h) - want) <= slack


# ------------------------------------------------------------------------------- norm and clipping
def clip_tensors(sizes, dtypes, seed, offset=0):
    g = gen(seed)
    out = []
    for i, n in enumerate(sizes):
        t = dtypes[i % len(dtypes)]
        out.append((torch.randn(n + offset, generator=g, device="cuda") * 10.0 ** (i % 5 - 2)).to(t)[offset:])
    return out


CLIP_CASES = [([], [F32]), ([1], [F32]), ([1], [BF16]), ([0, 5, 0], [F32, BF16]), ([4096, 4095, 4097, 3], [F32]),
              ([8192, 8191, 8193, 7, 0], [BF16]), ([100_003], [F32]), ([3_000_001, 5, 70_001], [BF16, F32]),
              ([17] * 64, [F32, BF16]), ([17] * 65, [F32, BF16]), ([1000 + 37 * i for i in range(700)], [F32, BF16]),
              ([0] * 130 + [9] + [0] * 130, [F32, BF16]), ([40_000_003], [F32])]


@pytest.mark.gpu
@pytest.mark.parametrize("offset", [0, 1])
@pytest.mark.parametrize("sizes,dtypes", CLIP_CASES, ids=[f"{len(s)}x{sum(s)}" for s, _ in CLIP_CASES])
def test_clip(sizes, dtypes, offset):
    gs = clip_tensors(sizes, dtypes, 50, offset)
    ref = math.sqrt(sum(float(g.double().square().sum()) for g in gs))
    norm = csp.grad_norm(gs)
    assert abs(float(norm) - ref) <= 2 * U32 * ref   # fp64 sum, one rounding to fp32 (2 for the root)
    for max_norm in (ref * 0.5 + 1e-3, ref * 2 + 1.0, 0.0):
        m = float(np.float32(max_norm))
        c = min(1.0, m / (ref + 1e-6))
        outs = [torch.full_like(g, 7.0) for g in gs]
        got = csp.grad_clip(gs, m, outs=outs)
        assert torch.equal(got, norm)
        for o, g in zip(outs, gs):
            want = g.double() * c
            tol = 6 * U32 * want.abs()   # norm 2, sum, quotient, product, constant
            within(o, want, tol + u(g.dtype) * (want.abs() + tol) + 2.0 ** -149, "clipped")
        mine = [g.clone() for g in gs]
        csp.grad_clip(mine, m)
        assert all(torch.equal(a, b) for a, b in zip(mine, outs))


@pytest.mark.gpu
def test_clip_squares_do_not_overflow_and_nan_shows():
    g = torch.full((1000,), 1e30, device="cuda")
    assert abs(float(csp.grad_norm([g])) / (1e30 * math.sqrt(1000)) - 1) < 1e-6
    g[3] = math.nan
    out = torch.zeros_like(g)
    assert math.isnan(float(csp.grad_clip([g], 1.0, outs=[out]))) and torch.isnan(out).all()
    g[3] = math.inf
    assert math.isinf(float(csp.grad_clip([g], 1.0, outs=[out])))
    assert torch.isnan(out[3]) and not out[4:].any()   # inf * 0, and finite values * 0


# ------------------------------------------------------------------------------- arguments, streams, graphs
@pytest.mark.gpu
def test_python_argument_checks():
    X, W, t = ce_inputs(8, 30, 16, F32, 60, "none")
    with pytest.raises(ValueError):
        csp.linear_ce_fwd(X, W[:, :8].contiguous(), t)
    with pytest.raises(ValueError):
        csp.linear_ce_fwd(X, W.T, t)                      # not contiguous
    with pytest.raises(TypeError):
        csp.linear_ce_fwd(X, W.bfloat16(), t)
    with pytest.raises(TypeError):
        csp.linear_ce_fwd(X, W, t.int())
    with pytest.raises(ValueError):
        csp.linear_ce_fwd(X, W, t[:4])
    with pytest.raises(TypeError):
        csp.linear_ce_fwd(X.half(), W.half(), t)
    with pytest.raises(ValueError):
        csp.embed_fwd(W, t, Y=torch.empty(8, 15, device="cuda"))
    with pytest.raises(ValueError):
        csp.embed_fwd(W.flatten(), t)
    with pytest.raises(csp.CspError):
        csp.embed_bwd(X, t, 0)
    with pytest.raises(ValueError):
        csp.grad_clip([X], 1.0, outs=[])
    with pytest.raises(ValueError):
        csp.grad_clip([X], 1.0, outs=[W])
    with pytest.raises(csp.CspError):
        csp.grad_clip([X], -1.0)


def token_step(E, W, ids, t, one):
    Y = csp.embed_fwd(E, ids, 2.0)
    loss, lse, total = csp.linear_ce_fwd(Y, W, t)
    dY, dW = csp.linear_ce_bwd(Y, W, t, lse, one, total)
    dE = csp.embed_bwd(dY, ids, E.shape[0], 2.0)
    norm = csp.grad_clip([dE, dW], 0.01)
    return loss, total, dE, dW, norm


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("N,V,D", [(1, 1000, 64), (33, 901, 72), (300, 700, 128)])
def test_on_another_stream_and_in_a_graph(N, V, D, dtype):
    g = gen(70)
    E = torch.randn(V, D, generator=g, device="cuda").to(dtype)
    W = (torch.randn(V, D, generator=g, device="cuda") / math.sqrt(D)).to(dtype)
    ids = torch.randint(-1, V, (N,), generator=g, device="cuda")
    t = torch.randint(-1, V, (N,), generator=g, device="cuda")
    ids[0] = t[0] = V - 1
    one = torch.ones(1, device="cuda")
    want = [a.clone() for a in token_step(E, W, ids, t, one)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = token_step(E, W, ids, t, one)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    Y = csp.embed_fwd(E, ids, 2.0, stream=s)         # the stream as an argument, outputs of its pool
    loss, _, _ = csp.linear_ce_fwd(Y, W, t, stream=s)
    s.synchronize()
    assert torch.equal(loss, want[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = token_step(E, W, ids, t, one)
    for k in range(4):   # other inputs in the same place each time, eager work in between
        ids2 = torch.roll(ids, k)
        t2 = torch.roll(t, 2 * k)
        eager = [a.clone() for a in token_step(E, W, ids2, t2, one)]
        keep = ids.clone(), t.clone()
        ids.copy_(ids2)
        t.copy_(t2)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(eager, outs)), f"replay {k}"
        ids.copy_(keep[0])
        t.copy_(keep[1])
