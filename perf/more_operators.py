"""Cases of what stands at both ends of a language model's stack of linear units: the token
embedding (fsdp_embedding_forward, fsdp_embedding_backward), the layer norm
(fsdp_layernorm_forward, fsdp_layernorm_backward) and the loss over the vocabulary
(fsdp_vocab_loss_forward, fsdp_vocab_loss_backward).

Each case is one call. `run` with `own` false computes the same in elementary torch operations
in 32 bits, rounded once at the end; `exact` computes it in 64 bits. Sizes are those of this
repository's workloads (widths 768 and 2304 with a vocabulary of 50257, 4096 with one of 32000,
8 ranks, 8192 tokens) and ragged ones beside them.

A case: op; m tokens; k the width; for the embedding and the loss, v the vocabulary and n the
row shards that hold it (rows past the vocabulary's end pad the shards); out: the type of the
embedding's gradient; bits: the width of a token id; the layer norm's res: a gradient that is
added; the loss's mean: whether the gradient is the mean loss's or comes with one factor a token.
"""
import math

import torch

own = False
EPS = 1e-5
MOST = 8192 * 32000 * 4096  # m v k of the largest listed case


def listed():
    return [
        # a sequence's next token through a 768-wide model's embedding: latency
        {"name": "embed one token", "op": "embed", "m": 1, "v": 50257, "k": 768, "n": 1, "bits": 64},
        # a micro-batch of 8192 tokens through a 4096-wide embedding held as 8 row shards
        {"name": "embed 4096", "op": "embed", "m": 8192, "v": 32000, "k": 4096, "n": 8, "bits": 64},
        # a short last batch over a small vocabulary, padded, gradient in bf16
        {"name": "embed grad ragged", "op": "embed_grad", "m": 1003, "v": 1157, "k": 520, "n": 5, "bits": 32,
         "out": "bf16"},
        # the 768-wide model's embedding gradient, fp32, 8192 tokens of a natural text's frequencies
        {"name": "embed grad 768", "op": "embed_grad", "m": 8192, "v": 50257, "k": 768, "n": 8, "bits": 64,
         "out": "fp32"},
        # one token's hidden state, 4096 wide: latency
        {"name": "norm one token", "op": "norm", "m": 1, "k": 4096},
        # a micro-batch of the 4096-wide model
        {"name": "norm 4096", "op": "norm", "m": 8192, "k": 4096},
        # a short last micro-batch, 2304 wide
        {"name": "norm grad short", "op": "norm_grad", "m": 777, "k": 2304, "res": False},
        # the same micro-batch backwards, the skip path's gradient joined in
        {"name": "norm grad 4096", "op": "norm_grad", "m": 8192, "k": 4096, "res": True},
        # a small vocabulary in five shards, every size ending inside a tile
        {"name": "loss ragged", "op": "loss", "m": 1003, "v": 1157, "k": 520, "n": 5, "bits": 32},
        # the 768-wide model's loss over its vocabulary of 50257, one micro-batch
        {"name": "loss 768", "op": "loss", "m": 8192, "v": 50257, "k": 768, "n": 8, "bits": 64},
        # the gradient of a short last micro-batch, tokens weighted one by one
        {"name": "loss grad short", "op": "loss_grad", "m": 777, "v": 50257, "k": 768, "n": 8, "bits": 64,
         "mean": False},
        # the 4096-wide model's output layer over a vocabulary of 32000: its gradients
        {"name": "loss grad 4096", "op": "loss_grad", "m": 8192, "v": 32000, "k": 4096, "n": 8, "bits": 64,
         "mean": True},
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["embed", "embed_grad", "embed_grad", "norm", "norm_grad", "norm_grad", "loss", "loss", "loss_grad",
                     "loss_grad"])
    m, k = log(1, 65536), 8 * log(8, 2048)
    if op in ("norm", "norm_grad"):
        c = {"op": op, "m": max(1, min(m, 8192 * 14336 // k)), "k": k}
        if op == "norm_grad":
            c["res"] = rng.choice([True, False])
        return c
    v = log(16, 131072)
    if op in ("embed", "embed_grad"):
        while v * k > 1 << 28:
            v, k = log(16, 131072), 8 * log(8, 2048)
        c = {"op": op, "m": max(1, min(m, 8192 * 14336 // k)), "v": v, "k": k}
        if op == "embed_grad":
            c["out"] = rng.choice(["fp32", "bf16"])
    else:
        while m * v * k > MOST or v * k > 1 << 28 or m * v > 1 << 29:
            m, v, k = log(1, 16384), log(16, 131072), 8 * log(8, 1024)
        c = {"op": op, "m": m, "v": v, "k": k}
        if op == "loss_grad":
            c["mean"] = rng.choice([True, False])
    c["n"], c["bits"] = rng.choice([1, 2, 5, 8, 16]), rng.choice([32, 64])
    return c


# ---- inputs ----

def _rows(case):
    """Rows of one shard: the vocabulary's share, rounded up to whole groups of 8."""
    per = -(-case["v"] // case["n"])
    return -(-per // 8) * 8


def _ids(case, gen, dev):
    """Token ids with the frequencies of text (the i-th most frequent about as 1 / i, at places of
    their own in the vocabulary); one in fifty, and the batch's end, are padding (-100)."""
    m, v = case["m"], case["v"]
    u = torch.rand(m, generator=gen, device=dev, dtype=torch.float64)
    rank = (torch.exp(u * math.log(v + 1.0)).long() - 1).clamp_(0, v - 1)
    ids = torch.randperm(v, generator=gen, device=dev)[rank]
    pad = torch.rand(m, generator=gen, device=dev) < 0.02
    pad[m - m // 16:] = True
    ids = torch.where(pad, torch.full_like(ids, -100), ids)
    return ids.to(torch.int64 if case["bits"] == 64 else torch.int32)


def prepare(case, seed):
    dev, bf = "cuda", torch.bfloat16
    gen = torch.Generator(device=dev).manual_seed(seed)

    def randn(*shape, std=1.0):
        return torch.randn(*shape, generator=gen, device=dev) * std

    m, k, op = case["m"], case["k"], case["op"]
    s = {"case": case}
    if op in ("norm", "norm_grad"):
        # a residual stream: every token its own size and offset
        x = (randn(m, k) * torch.exp(randn(m, 1, std=0.5)) + randn(m, 1, std=0.3)).to(bf)
        s["x"], s["gamma"], s["beta"] = x, (1.0 + randn(k, std=0.2)).to(bf), randn(k, std=0.1).to(bf)
        if op == "norm":
            s["y"], s["mean"], s["rstd"] = torch.empty_like(x), torch.empty(m, device=dev), torch.empty(m, device=dev)
        else:
            d = x.double()
            mean = d.mean(1)
            s["mean"] = mean.float()
            s["rstd"] = ((d - mean[:, None]).square().mean(1) + EPS).rsqrt().float()
            s["dy"] = randn(m, k, std=1e-2).to(bf)
            s["res"] = randn(m, k, std=1e-2).to(bf) if case["res"] else None
            s["dx"] = torch.empty_like(x)
            s["dgamma"], s["dbeta"] = torch.empty(k, device=dev), torch.empty(k, device=dev)
        return s
    n, rows = case["n"], _rows(case)
    s["ids"] = _ids(case, gen, dev)
    if op == "embed_grad":
        s["dy"] = randn(m, k, std=1e-2).to(bf)
        s["de"] = torch.empty(n * rows, k, device=dev, dtype=torch.float32 if case["out"] == "fp32" else bf)
        return s
    w = randn(n * rows, k, std=2.0 * k ** -0.5 if op != "embed" else 0.02).to(bf)
    w[case["v"]:] = 0
    s["shards"] = [t.clone() for t in w.chunk(n)]
    if op == "embed":
        s["y"] = torch.empty(m, k, dtype=bf, device=dev)
        return s
    s["x"] = randn(m, k).to(bf)
    if op == "loss":
        s["loss"], s["lse"] = torch.empty(m, device=dev), torch.empty(m, device=dev)
        s["total"] = torch.empty(2, device=dev)
        return s
    s["lse"] = torch.logsumexp(s["x"].float() @ w[:case["v"]].float().t(), 1)
    counted = s["ids"] >= 0
    s["total"] = torch.stack([torch.zeros((), device=dev), counted.sum().float()]) if case["mean"] else None
    s["dloss"] = None if case["mean"] else torch.rand(m, generator=gen, device=dev) / m
    s["dx"], s["dw"] = torch.empty(m, k, dtype=bf, device=dev), torch.empty(n * rows, k, dtype=bf, device=dev)
    return s


SCALE = 0.5  # of the loss's gradient (a loss scale, or one of two micro-batches)


# ---- one pass ----

def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import fsdp_sharded_optimizer_zero_gb300 as z

    case = s["case"]
    op = case["op"]
    if op == "norm":
        z.fsdp_layernorm_forward(s["x"], s["y"], gamma=s["gamma"], beta=s["beta"], eps=EPS, mean=s["mean"],
                                 rstd=s["rstd"])
        return {"y": s["y"], "mean": s["mean"], "rstd": s["rstd"]}
    if op == "norm_grad":
        z.fsdp_layernorm_backward(s["dy"], s["x"], s["mean"], s["rstd"], s["dx"], gamma=s["gamma"], residual=s["res"],
                                  dgamma=s["dgamma"], dbeta=s["dbeta"])
        return {"dx": s["dx"], "dgamma": s["dgamma"], "dbeta": s["dbeta"]}
    if op == "embed":
        z.fsdp_embedding_forward(s["shards"], s["ids"], s["y"], vocab=case["v"], scale=case["k"] ** 0.5)
        return {"y": s["y"]}
    if op == "embed_grad":
        z.fsdp_embedding_backward(s["dy"], s["ids"], s["de"], vocab=case["v"], scale=case["k"] ** 0.5)
        return {"de": s["de"]}
    if op == "loss":
        z.fsdp_vocab_loss_forward(s["shards"], s["x"], s["ids"], s["loss"], s["lse"], total=s["total"], vocab=case["v"])
        return {"loss": s["loss"], "lse": s["lse"], "total": s["total"]}
    z.fsdp_vocab_loss_backward(s["shards"], s["x"], s["ids"], s["lse"], s["dx"], s["dw"], vocab=case["v"],
                               dloss=s["dloss"], total=s["total"], scale=SCALE)
    return {"dx": s["dx"], "dw": s["dw"]}


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "norm":
        x = s["x"].float()
        mean = x.mean(1, keepdim=True)
        c = x - mean
        rstd = torch.rsqrt((c * c).mean(1, keepdim=True) + EPS)
        y = c * rstd * s["gamma"].float() + s["beta"].float()
        return {"y": y.bfloat16(), "mean": mean[:, 0], "rstd": rstd[:, 0]}
    if op == "norm_grad":
        dy = s["dy"].float()
        xhat = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
        g = dy * s["gamma"].float()
        dx = (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True)) * s["rstd"][:, None]
        if s["res"] is not None:
            dx = dx + s["res"].float()
        # long sums: in 64 bits
        return {"dx": dx.bfloat16(), "dgamma": (dy * xhat).sum(0, dtype=torch.float64).float(),
                "dbeta": dy.sum(0, dtype=torch.float64).float()}
    ids = s["ids"].long()
    real = (ids >= 0) & (ids < case["v"])
    at = torch.where(real, ids, torch.zeros_like(ids))
    if op == "embed":
        rows = torch.cat(s["shards"])[at].float() * case["k"] ** 0.5
        return {"y": torch.where(real[:, None], rows, torch.zeros_like(rows)).bfloat16()}
    if op == "embed_grad":
        g = s["dy"].float() * case["k"] ** 0.5
        g = torch.where(real[:, None], g, torch.zeros_like(g))
        de = torch.zeros(s["de"].shape, device=g.device)
        return {"de": de.index_add_(0, at, g).to(s["de"].dtype)}
    w, x = torch.cat(s["shards"])[:case["v"]].float(), s["x"].float()
    logits = x @ w.t()
    if op == "loss":
        top = logits.max(1, keepdim=True).values
        lse = top[:, 0] + torch.log(torch.exp(logits - top).sum(1))
        loss = torch.where(real, lse - logits.gather(1, at[:, None])[:, 0], torch.zeros_like(lse))
        return {"loss": loss, "lse": lse, "total": torch.stack([loss.double().sum(), real.sum().double()]).float()}
    weight = torch.full_like(s["lse"], SCALE) if s["dloss"] is None else s["dloss"] * SCALE
    if s["total"] is not None:
        weight = weight / torch.clamp(s["total"][1], min=1.0)
    weight = torch.where(real, weight, torch.zeros_like(weight))
    p = torch.exp(logits - s["lse"][:, None]) * weight[:, None]
    p.scatter_add_(1, at[:, None], -weight[:, None])
    dw = torch.zeros(s["dw"].shape, dtype=torch.bfloat16, device=x.device)
    dw[:case["v"]] = (p.t() @ x).bfloat16()
    return {"dx": (p @ w).bfloat16(), "dw": dw}


def work(case):
    m, k, op = case["m"], case["k"], case["op"]
    x = 2 * m * k
    if op == "norm":
        return {"bytes": 2 * x + 4 * k + 8 * m, "flops": 8 * m * k}
    if op == "norm_grad":
        return {"bytes": (4 if case["res"] else 3) * x + 8 * m + 2 * k + 8 * k, "flops": 14 * m * k}
    ids = m * case["bits"] // 8
    v, rows = case["v"], case["n"] * _rows(case)
    if op == "embed":
        return {"bytes": 2 * x + ids, "flops": m * k}
    if op == "embed_grad":  # every row of the gradient is written, those of no token with zeros
        return {"bytes": x + ids + rows * k * (4 if case["out"] == "fp32" else 2), "flops": 2 * m * k}
    if op == "loss":
        return {"bytes": x + 2 * v * k + ids + 8 * m, "flops": 2 * m * v * k + 4 * m * v}
    # the logits are not kept: one product to have them again, one for each gradient
    return {"bytes": 2 * x + 2 * v * k + 2 * rows * k + ids + 8 * m, "flops": 6 * m * v * k + 4 * m * v}


# ---- the same in 64 bits, from the definitions ----

def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    op, m, k = case["op"], case["m"], case["k"]
    d = lambda t: t.to(f64)  # noqa: E731
    if op == "norm":
        x = d(s["x"])
        mean = x.sum(1) / k
        var = sum(((x[:, j:j + 4096] - mean.unsqueeze(1)) ** 2).sum(1) for j in range(0, k, 4096)) / k
        sigma = torch.sqrt(var + EPS)
        return {"y": (x - mean.unsqueeze(1)) / sigma.unsqueeze(1) * d(s["gamma"]) + d(s["beta"]), "mean": mean,
                "rstd": 1.0 / sigma}
    if op == "norm_grad":
        r, u = d(s["rstd"]).unsqueeze(1), d(s["dy"]) * d(s["gamma"])
        xn = r * (d(s["x"]) - d(s["mean"]).unsqueeze(1))
        dx = r * u - r * (u.sum(1, keepdim=True) / k) - r * xn * ((u * xn).sum(1, keepdim=True) / k)
        if case["res"]:
            dx += d(s["res"])
        return {"dx": dx, "dgamma": torch.einsum("ij,ij->j", d(s["dy"]), xn), "dbeta": d(s["dy"]).sum(0)}
    ids, v = s["ids"].to(torch.int64), case["v"]
    keep = torch.nonzero((ids >= 0) & (ids < v)).squeeze(1)
    if op == "embed":
        y = torch.zeros(m, k, dtype=f64, device=ids.device)
        per = s["shards"][0].shape[0]
        for q, e in enumerate(s["shards"]):
            mine = keep[torch.div(ids[keep], per, rounding_mode="floor") == q]
            y[mine] = d(e[ids[mine] - q * per]) * math.sqrt(k)
        return {"y": y}
    if op == "embed_grad":
        de = torch.zeros(s["de"].shape, dtype=f64, device=ids.device)
        de.index_put_((ids[keep],), d(s["dy"][keep]) * math.sqrt(k), accumulate=True)
        return {"de": de}
    z = torch.cat([d(s["x"]) @ d(w).t() for w in s["shards"]], 1)[:, :v]
    if op == "loss":
        lse = torch.logsumexp(z, 1)
        loss = torch.zeros_like(lse)
        loss[keep] = lse[keep] - z[keep, ids[keep]]
        total = torch.tensor([float(loss.sum()), float(keep.numel())], dtype=f64)
        return {"loss": loss, "lse": lse, "total": total}
    share = 1.0 / max(1, keep.numel()) if case["mean"] else d(s["dloss"])[keep]
    g = torch.zeros(m, dtype=f64, device=z.device)
    g[keep] = SCALE * share
    dz = z.sub_(d(s["lse"]).unsqueeze(1)).exp_().mul_(g.unsqueeze(1))
    dz[g == 0] = 0.0
    dz[keep, ids[keep]] -= g[keep]
    dx, at = torch.zeros(m, k, dtype=f64, device=z.device), 0
    dw = torch.zeros(s["dw"].shape, dtype=f64, device=z.device)
    for w in s["shards"]:
        cols = max(0, min(w.shape[0], v - at))
        part = dz[:, at:at + cols]
        dx += part @ d(w[:cols])
        dw[at:at + cols] = part.t() @ d(s["x"])
        at += cols
    return {"dx": dx, "dw": dw}
