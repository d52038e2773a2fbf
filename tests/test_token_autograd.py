"""The token operators as torch functions (token_ops.py) and the model that runs them together."""
import math

import pytest
import torch

from coo_spmm_fwd_amd import binding as csp
from coo_spmm_fwd_amd import token_ops as ops

F32, BF16 = torch.float32, torch.bfloat16


def test_shapes_are_checked_before_the_gpu():
    with pytest.raises(ValueError):
        ops.linear_cross_entropy(torch.zeros(2, 3, 8), torch.zeros(5, 8), torch.zeros(2, 4, dtype=torch.int64))
    with pytest.raises(TypeError):
        ops.embedding(torch.zeros(3, dtype=torch.int64), torch.zeros(4, 8))


def inputs(N, V, D, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    E = torch.randn(V, D, generator=g, device="cuda").to(dtype).requires_grad_()
    W = (torch.randn(V, D, generator=g, device="cuda") / math.sqrt(D)).to(dtype).requires_grad_()
    ids = torch.randint(-1, V, (N,), generator=g, device="cuda")
    t = torch.randint(-1, V, (N,), generator=g, device="cuda")
    t[0] = V - 1
    return E, W, ids, t


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("N,V,D", [(6, 50, 16), (96, 300, 72)])
def test_gradients_are_those_of_the_calls(N, V, D, dtype):
    E, W, ids, t = inputs(N, V, D, dtype)
    loss = 3.0 * ops.linear_cross_entropy(ops.embedding(ids.view(2, -1), E, 2.0), W, t.view(2, -1))
    loss.backward()
    Y = csp.embed_fwd(E.detach(), ids, 2.0)
    _, lse, total = csp.linear_ce_fwd(Y, W.detach(), t)
    dY, dW = csp.linear_ce_bwd(Y, W.detach(), t, lse, torch.full((1,), 3.0, device="cuda"), total)
    assert torch.equal(loss.detach(), 3.0 * total[2])
    assert torch.equal(W.grad, dW) and torch.equal(E.grad, csp.embed_bwd(dY, ids, V, 2.0))
    norm = ops.clip_grad_norm([E, W, torch.nn.Parameter(torch.zeros(3, device="cuda"))], 1e-3)
    assert torch.equal(norm, csp.grad_norm([csp.embed_bwd(dY, ids, V, 2.0), dW]))


@pytest.mark.gpu
def test_strided_and_broadcast_inputs_and_gradients():
    E, W, ids, t = inputs(64, 40, 24, F32, 3)
    two = torch.stack([ids, ids.flip(0)], 1)           # ids[:, 0] is strided
    Y = ops.embedding(two[:, 0], E)
    Y.sum().backward()                                 # the gradient of a sum is an expanded scalar
    n = torch.bincount(ids[ids >= 0], minlength=40).float()
    assert torch.equal(E.grad, n[:, None].expand(40, 24))
    X = torch.randn(24, 64, device="cuda", requires_grad=True)
    a = ops.linear_cross_entropy(X.T, W, t)            # rows that are columns
    b = ops.linear_cross_entropy(X.detach().T.contiguous(), W, t)
    assert torch.equal(a, b)
    a.backward()
    assert X.grad.shape == X.shape and torch.isfinite(X.grad).all()
    loss = ops.linear_cross_entropy(X.T, W, t)
    keep = loss.detach().clone()
    loss.mul_(0.5)                                     # in place on the loss: the backward still divides by the count
    W.grad = None
    loss.backward()
    want = csp.linear_ce_bwd(X.detach().T.contiguous(), W.detach(), t, *_lse_and_half(X, W, t))[1]
    assert torch.equal(loss.detach(), keep * 0.5) and torch.equal(W.grad, want)


def _lse_and_half(X, W, t):
    _, lse, total = csp.linear_ce_fwd(X.detach().T.contiguous(), W.detach(), t)
    return lse, torch.full((1,), 0.5, device="cuda"), total


@pytest.mark.gpu
def test_all_targets_masked_gives_zero_loss_and_gradients():
    E, W, ids, t = inputs(70, 33, 16, F32, 4)
    loss = ops.linear_cross_entropy(ops.embedding(ids, E), W, torch.full_like(t, -100))
    loss.backward()
    assert float(loss) == 0.0 and not E.grad.any() and not W.grad.any()


@pytest.mark.gpu
@pytest.mark.parametrize("N", [48, 200])
def test_captured_training_step(N):
    """Forward, backward, clipping and update as one graph, replayed against eager steps."""
    V, D, lr = 301, 64, 0.5
    E, W, ids, t = inputs(N, V, D, F32, 5)

    def step(E, W):
        loss = ops.linear_cross_entropy(ops.embedding(ids, E, 1.5), W, t)
        gE, gW = torch.autograd.grad(loss, (E, W))
        csp.grad_clip([gE, gW], 0.1)
        with torch.no_grad():
            E.sub_(gE, alpha=lr)
            W.sub_(gW, alpha=lr)
        return loss.detach()

    eager = [p.detach().clone().requires_grad_() for p in (E, W)]
    want = []
    for _ in range(4):
        loss = step(*eager)
        want.append((loss.clone(), eager[0].detach().clone(), eager[1].detach().clone()))
    own = [p.detach().clone().requires_grad_() for p in (E, W)]   # leaves no eager graph was made of
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):                                     # warm-up, on copies
        step(*[p.detach().clone().requires_grad_() for p in own])
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(*own)
    for k in range(4):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[k][0]), f"replay {k}"
        assert torch.equal(own[0].detach(), want[k][1]) and torch.equal(own[1].detach(), want[k][2]), f"replay {k}"
        csp.grad_norm([own[0].detach()])                           # eager work in between


@pytest.mark.gpu
def test_token_model_learns():
    from coo_spmm_fwd_amd import token_lm
    losses = token_lm.train(steps=120, vocab=500, width=64, tokens=256, restructure_every=40, log=None)
    assert all(math.isfinite(x) for x in losses)
    assert abs(losses[0] - math.log(500)) < 0.5 and losses[-1] < 0.6 * losses[0]
