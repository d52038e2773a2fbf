"""The torch functions of token_ops.py under autograd's and clipping's own rules, on the CPU: the library's
calls are replaced by plain torch ones, so what is tested is what the functions make of them."""
import pytest
import torch

from coo_spmm_fwd_amd import token_ops as ops


@torch.no_grad()  # as the library: torch sees no part of it
def plain_embed_fwd(E, ids, scale):
    return E[ids] * scale


@torch.no_grad()
def plain_embed_bwd(dY, ids, V, scale):
    return torch.zeros(V, dY.shape[1]).index_add_(0, ids, dY * scale)


@torch.no_grad()
def plain_ce_fwd(X, W, t):
    z = X @ W.T
    lse = torch.logsumexp(z, 1)
    loss = lse - z.gather(1, t[:, None])[:, 0]
    return loss, lse, torch.stack([loss.sum(), torch.tensor(float(t.numel())), loss.mean()])


@torch.no_grad()
def plain_ce_bwd(X, W, t, lse, dmean, total, **more):
    G = torch.exp(X @ W.T - lse[:, None])
    G[torch.arange(t.numel()), t] -= 1.0
    G = G * dmean / total[1]
    need = more.get("need", (True, True))
    return G @ W if need[0] else None, G.T @ X if need[1] else None


@pytest.fixture
def plain(monkeypatch):
    monkeypatch.setattr(ops.csp, "embed_fwd", plain_embed_fwd)
    monkeypatch.setattr(ops.csp, "embed_bwd", plain_embed_bwd)
    monkeypatch.setattr(ops.csp, "linear_ce_fwd", plain_ce_fwd)
    monkeypatch.setattr(ops.csp, "linear_ce_bwd", plain_ce_bwd)


def leaves():
    g = torch.Generator().manual_seed(0)
    X, W = (torch.randn(n, 5, generator=g).requires_grad_() for n in (4, 7))
    return X, W, torch.tensor([0, 6, 2, 2])


def test_first_gradients_agree_with_torch(plain):
    X, W, t = leaves()
    mine = torch.autograd.grad(ops.linear_cross_entropy(X, W, t), (X, W))
    want = torch.autograd.grad(torch.nn.functional.cross_entropy(X @ W.T, t), (X, W))
    assert all(torch.allclose(a, b, atol=1e-6) for a, b in zip(mine, want))
    (mine,) = torch.autograd.grad(ops.embedding(t, W, 2.0).square().sum(), W)
    (want,) = torch.autograd.grad((W[t] * 2.0).square().sum(), W)
    assert torch.allclose(mine, want)


def test_second_gradients_of_the_loss_raise(plain):
    """A penalty on a gradient differentiates the backward pass, which has no derivative of its own: an error,
    never a gradient without the penalty's part."""
    X, W, t = leaves()
    loss = ops.linear_cross_entropy(X, W, t)
    gX, gW = torch.autograd.grad(loss, (X, W), create_graph=True)
    for g in (gX, gW):
        with pytest.raises(RuntimeError, match="cannot be differentiated"):
            torch.autograd.grad(loss + g.square().sum(), (X, W), retain_graph=True)
    gX, gW = torch.autograd.grad(loss, (X, W))   # and no graph where none was asked for
    assert not gX.requires_grad and not gW.requires_grad


def test_second_gradients_pass_through_the_embedding(plain):
    for f in (ops.embedding, lambda ids, E, scale: E[ids] * scale):
        _, E, ids = leaves()
        y = f(ids, E, 2.0)
        (g,) = torch.autograd.grad(y.pow(3).sum(), E, create_graph=True)
        (second,) = torch.autograd.grad(y.sum() + g.square().sum(), E)
        if f is ops.embedding:
            mine = second
    assert torch.allclose(mine, second)


@pytest.fixture
def clipped(monkeypatch):
    """The lists of gradients that clip_grad_norm hands to the library."""
    lists = []

    def grad_clip(grads, max_norm):
        lists.append(list(grads))
        for g in grads:
            g.numpy()[...] *= 0.5  # as the library does: torch does not see the write
        return torch.ones(1)

    monkeypatch.setattr(ops.csp, "grad_clip", grad_clip)
    return lists


def test_clipping_takes_one_tensor_too(clipped):
    p = torch.nn.Parameter(torch.ones(3, 2))
    p.grad = torch.ones(3, 2)
    ops.clip_grad_norm(p, 1.0)
    assert [g is p.grad for g in clipped[0]] == [True]
    q = torch.nn.Parameter(torch.ones(2))
    ops.clip_grad_norm((r for r in (p, q)), 1.0)  # and any iterable; q has no gradient
    assert [g is p.grad for g in clipped[1]] == [True]


def test_clipping_counts_as_a_write(clipped):
    """A graph that saved a gradient before it was clipped refuses to use it, as after any write in place."""
    p = torch.nn.Parameter(torch.ones(3, 2))
    (g,) = torch.autograd.grad(p.pow(3).sum(), p, create_graph=True)
    loss = g.square().sum()  # saves g
    p.grad = g.detach()
    ops.clip_grad_norm([p], 1.0)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


@pytest.mark.parametrize("need", [(True, False), (False, True), (True, True)])
def test_only_the_gradients_that_are_asked_for(plain, monkeypatch, need):
    """A frozen head, or hidden states that are inputs: the other gradient is neither computed nor allocated."""
    asked = []
    for name, which in (("linear_ce_bwd", (True, True)), ("linear_ce_bwd_input", (True, False)),
                        ("linear_ce_bwd_weight", (False, True))):
        def call(*a, which=which):
            asked.append(which)
            got = plain_ce_bwd(*a)
            return got if all(which) else got[which.index(True)]
        monkeypatch.setattr(ops.csp, name, call, raising=False)
    X, W, t = leaves()
    both = torch.autograd.grad(ops.linear_cross_entropy(X, W, t), (X, W))
    asked.clear()
    X, W = X.detach().requires_grad_(need[0]), W.detach().requires_grad_(need[1])
    ops.linear_cross_entropy(X, W, t).backward()
    assert asked == [need]
    assert all(p.grad is None if not n else torch.equal(p.grad, g) for p, n, g in zip((X, W), need, both))


@pytest.mark.gpu
def test_second_gradients_on_the_library():
    g = torch.Generator(device="cuda").manual_seed(1)
    E, W = (torch.randn(9, 6, generator=g, device="cuda").requires_grad_() for _ in range(2))
    ids, t = torch.tensor([3, -1, 3, 8], device="cuda"), torch.tensor([0, 5, -100, 8], device="cuda")
    part = (ids >= 0)[:, None]
    got = []
    for look in (lambda: ops.embedding(ids, E, 2.0), lambda: torch.where(part, E[ids.clamp(min=0)] * 2.0, 0.0)):
        y = look()
        (first,) = torch.autograd.grad(y.pow(3).sum(), E, create_graph=True)
        got.append(torch.autograd.grad(y.sum() + first.square().sum(), E)[0])
    assert torch.allclose(*got, rtol=1e-5)
    loss = ops.linear_cross_entropy(ops.embedding(ids, E, 2.0), W, t)
    (first,) = torch.autograd.grad(loss, W, create_graph=True)
    with pytest.raises(RuntimeError, match="cannot be differentiated"):
        (loss + first.square().sum()).backward()
