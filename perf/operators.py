"""What the token operators cost: the embedding lookup and its gradient, the loss over a large
vocabulary and its gradient, and the global gradient norm with clipping.

`run` computes each in its plain form (elementary torch operations in fp32, rounded once at the
end), or, where `own` is true, through the library's calls.  `exact` gives the same results from
the definitions in fp64.

Definitions (ids and targets outside [0, V) take no part):
  lookup       Y[n, :] = scale * E[ids[n], :]                      (a zero row for an id that takes no part)
  lookup_grad  dE[v, :] = scale * sum over n with ids[n] = v of dY[n, :]
  loss         z = X W^T, lse[n] = log sum_v exp z[n, v], loss[n] = lse[n] - z[n, t_n], and
               {sum, count, sum / count} over the targets that take part
  loss_train   the same, then dX and dW of that mean
  norm         sqrt of the sum of all squares of all tensors
  clip         that norm, and every tensor times min(1, max_norm / (norm + 1e-6))
"""
import math

import torch

own = False

F32, BF16 = "f32", "bf16"


def listed():
    return [
        # decoding: the one token just drawn is looked up before the first layer
        {"name": "lookup_one_f32", "op": "lookup", "n": 1, "v": 50257, "d": 768, "dtype": F32},
        # a prompt of 16384 tokens into a wide model
        {"name": "lookup_prompt_bf16", "op": "lookup", "n": 16384, "v": 65536, "d": 4096, "dtype": BF16},
        # a training step of 16 short sequences, odd count, GPT-2-small width
        {"name": "lookup_grad_f32", "op": "lookup_grad", "n": 4093, "v": 50257, "d": 768, "dtype": F32},
        # a training step of a large batch
        {"name": "lookup_grad_bf16", "op": "lookup_grad", "n": 32768, "v": 65536, "d": 4096, "dtype": BF16},
        # scoring one token while decoding
        {"name": "loss_one_f32", "op": "loss", "n": 1, "v": 50257, "d": 768, "dtype": F32},
        # scoring a text of 2048 tokens (perplexity), no gradient
        {"name": "loss_text_bf16", "op": "loss", "n": 2048, "v": 65536, "d": 2048, "dtype": BF16},
        # a step at the batch of the sparse MLP workload (32 rows, width 768)
        {"name": "loss_train_b32_f32", "op": "loss_train", "n": 32, "v": 50257, "d": 768, "dtype": F32, "skip": 0.0},
        # the small-batch regime at full width: 64 rows
        {"name": "loss_train_b64_bf16", "op": "loss_train", "n": 64, "v": 65536, "d": 4096, "dtype": BF16, "skip": 0.0},
        # odd sizes everywhere, a third of the targets masked (prompt tokens of a fine-tuning batch)
        {"name": "loss_train_odd_bf16", "op": "loss_train", "n": 777, "v": 30011, "d": 1001, "dtype": BF16, "skip": 0.33},
        # a large training step
        {"name": "loss_train_large_bf16", "op": "loss_train", "n": 8192, "v": 65536, "d": 4096, "dtype": BF16,
         "skip": 0.02},
        # the gradients of the two sparse MLP layers and a bias: three small tensors
        {"name": "clip_mlp_f32", "op": "clip", "tensors": 3, "total": 472_000, "dtype": F32, "max_norm": 0.5},
        # all gradients of a model of 400 tensors, fp32 and bf16 mixed
        {"name": "clip_model_mixed", "op": "clip", "tensors": 400, "total": 500_000_000, "dtype": "mixed",
         "max_norm": 1.0},
    ]


def _log_between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["lookup", "lookup_grad", "loss", "loss_train", "loss_train", "norm", "clip"])
    if op in ("norm", "clip"):
        tensors = _log_between(rng, 1, 600)
        total = max(tensors, _log_between(rng, 1_000, 400_000_000))
        return {"op": op, "tensors": tensors, "total": total, "dtype": rng.choice([F32, BF16, "mixed"]),
                "max_norm": rng.choice([0.5, 1.0, 1e9])}
    dtype = rng.choice([F32, BF16])
    v = _log_between(rng, 500, 70_000)
    d = _log_between(rng, 48, 4096)
    if rng.random() < 0.6:
        d = -(-d // 64) * 64  # most models have a width like this; the others stay odd
    if op in ("lookup", "lookup_grad"):
        return {"op": op, "n": _log_between(rng, 1, 32768), "v": v, "d": d, "dtype": dtype}
    n = _log_between(rng, 1, 8192)
    while n * v * d > 4096 * 50257 * 2048:  # fp32 costs more a product: stay below the largest case
        n = max(1, n // 2)
    return {"op": op, "n": n, "v": v, "d": d, "dtype": dtype,
            **({"skip": rng.choice([0.0, 0.0, 0.1, 0.5, 0.9])} if op == "loss_train" else {})}


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == BF16 else torch.float32


def _tokens(n, v, g):
    """Token ids as text has them: about as many of rank r as 1 / r, the ranks scattered over the ids."""
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    rank = (torch.exp(u * math.log(v + 1)) - 1).long().clamp_(0, v - 1)
    return torch.randperm(v, generator=g, device="cuda")[rank]


def _sizes(tensors, total, seed):
    """Tensor sizes spread over three decades that add up to about `total`, odd ones among them."""
    w = torch.exp(torch.rand(tensors, generator=torch.Generator().manual_seed(seed), dtype=torch.float64) * math.log(1000.0))
    return torch.clamp((w / w.sum() * total).long(), min=1).tolist()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    if op in ("norm", "clip"):
        sizes = _sizes(case["tensors"], case["total"], 7)
        mixed = [torch.bfloat16 if case["dtype"] == BF16 or case["dtype"] == "mixed" and i % 2 else torch.float32
                 for i in range(len(sizes))]
        state = {"op": op, "max_norm": case["max_norm"], "grads": [], "outs": [], "flat": []}
        # one bucket of gradients a type, and one that takes the clipped ones, as a data-parallel step keeps them
        views, outs = {}, {}
        for t in sorted(set(mixed), key=str):
            n = [s for s, m in zip(sizes, mixed) if m == t]
            bucket = torch.randn(sum(n), generator=g, device="cuda", dtype=t).mul_(1e-3)
            flat = torch.empty_like(bucket)
            state["flat"].append(flat)
            views[t], outs[t] = iter(bucket.split(n)), iter(flat.split(n))
        state["grads"] = [next(views[t]) for t in mixed]
        state["outs"] = [next(outs[t]) for t in mixed]
        return state
    n, v, d, t = case["n"], case["v"], case["d"], _dtype(case)
    ids = _tokens(n, v, g)
    if op == "lookup":
        if n > 1:  # padding
            ids = torch.where(torch.rand(n, generator=g, device="cuda") < 0.02, torch.full_like(ids, -1), ids)
        return {"op": op, "scale": math.sqrt(d), "ids": ids,
                "E": torch.randn(v, d, generator=g, device="cuda", dtype=t).mul_(0.02)}
    if op == "lookup_grad":
        if n > 1:
            ids = torch.where(torch.rand(n, generator=g, device="cuda") < 0.02, torch.full_like(ids, -1), ids)
        return {"op": op, "scale": math.sqrt(d), "ids": ids, "v": v,
                "dY": torch.randn(n, d, generator=g, device="cuda", dtype=t).mul_(1e-3)}
    # logits of standard deviation 2, and the target's raised by 0 to 16, so that losses run from near 0 up
    W = torch.randn(v, d, generator=g, device="cuda", dtype=torch.float32).mul_(2.0 / math.sqrt(d))
    X = torch.randn(n, d, generator=g, device="cuda", dtype=torch.float32)
    X += W[ids] * (4.0 * torch.rand(n, 1, generator=g, device="cuda"))
    skip = torch.rand(n, generator=g, device="cuda") < case.get("skip", 0.0)
    skip[0] = False  # a batch has something to learn
    return {"op": op, "X": X.to(t), "W": W.to(t), "targets": torch.where(skip, torch.full_like(ids, -100), ids),
            "one": torch.ones(1, device="cuda")}


def _plain_lookup(s):
    E, ids = s["E"], s["ids"]
    part = (ids >= 0) & (ids < E.shape[0])
    Y = E[torch.where(part, ids, torch.zeros_like(ids))].float() * s["scale"]
    return torch.where(part[:, None], Y, torch.zeros_like(Y)).to(E.dtype)


def _plain_lookup_grad(s):
    dY, ids, v = s["dY"], s["ids"], s["v"]
    part = (ids >= 0) & (ids < v)
    rows = torch.where(part[:, None], dY.float(), torch.zeros((), device=dY.device))
    dE = torch.zeros(v, dY.shape[1], device=dY.device)
    dE.index_add_(0, torch.where(part, ids, torch.zeros_like(ids)), rows)
    return (dE * s["scale"]).to(dY.dtype)


def _plain_loss(s, train):
    X, W, t = s["X"].float(), s["W"].float(), s["targets"]
    part = (t >= 0) & (t < W.shape[0])
    at = torch.where(part, t, torch.zeros_like(t))[:, None]
    z = X @ W.T
    m = z.amax(1, keepdim=True)
    lse = m + torch.log(torch.exp(z - m).sum(1, keepdim=True))
    loss = torch.where(part, (lse - z.gather(1, at))[:, 0], torch.zeros((), device=X.device))
    count = part.sum().float()
    total = torch.stack([loss.sum(), count, loss.sum() / count.clamp(min=1.0)])
    out = {"loss": loss, "lse": torch.where(part, lse[:, 0], torch.zeros((), device=X.device)), "total": total}
    if train:
        p = torch.exp(z.sub_(lse))
        p.scatter_add_(1, at, torch.full_like(lse, -1.0))
        p *= (part.float() / count.clamp(min=1.0) * s["one"])[:, None]
        out["dX"] = (p @ W).to(s["X"].dtype)
        out["dW"] = (p.T @ X).to(s["W"].dtype)
    return out


def _plain_norm(s):
    return torch.sqrt(torch.stack([g.float().square().sum() for g in s["grads"]]).sum())[None]


def _plain_clip(s):
    norm = _plain_norm(s)
    c = torch.clamp(s["max_norm"] / (norm + 1e-6), max=1.0)
    [o.copy_(g.float() * c) for g, o in zip(s["grads"], s["outs"])]
    return {"norm": norm, "clipped": s["flat"]}


def run(state):
    op = state["op"]
    if own:
        from coo_spmm_fwd_amd import binding as csp
        if op == "lookup":
            return csp.embed_fwd(state["E"], state["ids"], state["scale"])
        if op == "lookup_grad":
            return csp.embed_bwd(state["dY"], state["ids"], state["v"], state["scale"])
        if op in ("loss", "loss_train"):
            loss, lse, total = csp.linear_ce_fwd(state["X"], state["W"], state["targets"])
            out = {"loss": loss, "lse": lse, "total": total}
            if op == "loss_train":
                out["dX"], out["dW"] = csp.linear_ce_bwd(state["X"], state["W"], state["targets"], lse, state["one"],
                                                         total)
            return out
        if op == "norm":
            return csp.grad_norm(state["grads"])
        return {"norm": csp.grad_clip(state["grads"], state["max_norm"], outs=state["outs"]),
                "clipped": state["flat"]}
    if op == "lookup":
        return _plain_lookup(state)
    if op == "lookup_grad":
        return _plain_lookup_grad(state)
    if op in ("loss", "loss_train"):
        return _plain_loss(state, op == "loss_train")
    return _plain_norm(state) if op == "norm" else _plain_clip(state)


def work(case):
    op = case["op"]
    if op in ("norm", "clip"):
        sizes = _sizes(case["tensors"], case["total"], 7)
        b = sum(n * (2 if case["dtype"] == BF16 or case["dtype"] == "mixed" and i % 2 else 4)
                for i, n in enumerate(sizes))
        return {"bytes": b * (2 if op == "clip" else 1) + 4, "flops": sum(sizes) * (3 if op == "clip" else 2)}
    n, v, d, e = case["n"], case["v"], case["d"], 2 if case["dtype"] == BF16 else 4
    if op == "lookup":
        return {"bytes": 8 * n + min(n, v) * d * e + n * d * e, "flops": n * d}
    if op == "lookup_grad":
        return {"bytes": 8 * n + n * d * e + v * d * e, "flops": 2 * n * d}
    b, f = 8 * n + n * d * e + v * d * e + 8 * n + 12, 2 * n * v * d + 2 * n * v
    if op == "loss_train":
        b, f = b + n * d * e + v * d * e, 3 * f
    return {"bytes": b, "flops": f}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "lookup":
        E, ids = s["E"].double(), s["ids"]
        Y = torch.zeros(ids.numel(), E.shape[1], dtype=torch.float64, device="cuda")
        has = (ids >= 0).nonzero()[:, 0]
        Y[has] = E[ids[has]] * s["scale"]
        return Y
    if op == "lookup_grad":
        has = (s["ids"] >= 0).nonzero()[:, 0]
        order = has[torch.argsort(s["ids"][has], stable=True)]
        dE = torch.zeros(s["v"], s["dY"].shape[1], dtype=torch.float64, device="cuda")
        dE.index_put_((s["ids"][order],), s["dY"][order].double() * s["scale"], accumulate=True)
        return dE
    if op in ("loss", "loss_train"):
        X, W, t = s["X"].double(), s["W"].double(), s["targets"]
        n = X.shape[0]
        out = {"loss": torch.zeros(n, dtype=torch.float64, device="cuda"),
               "lse": torch.zeros(n, dtype=torch.float64, device="cuda")}
        has = ((t >= 0) & (t < W.shape[0])).nonzero()[:, 0]
        count = max(1, has.numel())
        dX, dW = torch.zeros_like(X), torch.zeros_like(W)
        for rows in has.split(1024):  # the logits of 1024 tokens at a time
            z = X[rows] @ W.T
            lse = torch.logsumexp(z, 1)
            out["lse"][rows] = lse
            out["loss"][rows] = lse - z[torch.arange(rows.numel(), device="cuda"), t[rows]]
            if op == "loss_train":
                p = torch.exp(z - lse[:, None]) / count
                p[torch.arange(rows.numel(), device="cuda"), t[rows]] -= 1.0 / count
                dX[rows] = p @ W
                dW += p.T.contiguous() @ X[rows]
        total = out["loss"].sum()
        out["total"] = torch.stack([total, torch.full_like(total, has.numel()), total / count])
        if op == "loss_train":
            out["dX"], out["dW"] = dX, dW
        return out
    norm = math.sqrt(sum(float(g.double().square().sum()) for g in s["grads"]))
    if op == "norm":
        return torch.tensor([norm], dtype=torch.float64, device="cuda")
    c = min(1.0, s["max_norm"] / (norm + 1e-6))
    for g, o in zip(s["grads"], s["outs"]):  # in the state's own layout, in 64 bits
        o.copy_(g)
    return {"norm": torch.tensor([norm], dtype=torch.float64, device="cuda"),
            "clipped": [f.double() * c for f in s["flat"]]}
