"""A small language model trained from tokens to loss: token embedding, layer norms, an MLP of linear
units with its skip path, the loss over the vocabulary, and the fused ZeRO step.

    X0 = E[tokens],  X1 = X0 + gelu(norm1(X0) W1^T + b1) W2^T + b2,  loss = cross entropy of norm2(X1) E^T

The table E is the output layer too, held as row shards whose end is padding (the vocabulary is no
multiple of the shards). Two data-parallel ranks are simulated as separate gradient buffers, each with
its own batch, the end of which is padded. The logits are never kept: the loss keeps one number a token, from
which its backward computes them again, piece by piece. Weights, biases and the norms' parameters live in one flat
bf16 parameter buffer, gradients in one flat bf16 buffer per rank, and zero_fused_step reduces, updates
and casts them in one pass. Run with
`python -m fsdp_sharded_optimizer_zero_gb300.example_language` on a GPU."""
import torch

import fsdp_sharded_optimizer_zero_gb300 as z

BF16 = torch.bfloat16
EPS = 1e-5


class Model:
    """Sizes, and the views of flat buffers as the model's tensors."""

    def __init__(self, vocab=1003, d=128, f=512, shards=4):
        self.vocab, self.d, self.f, self.shards = vocab, d, f, shards
        rows = -(-vocab // (8 * shards)) * 8 * shards  # whole groups of 8 rows in each shard
        self.sizes = {"e": (rows, d), "g1": (d,), "c1": (d,), "w1": (f, d), "b1": (f,), "w2": (d, f), "b2": (d,), "g2": (d,),
                      "c2": (d,)}
        self.psi = sum(torch.Size(s).numel() for s in self.sizes.values())

    def views(self, flat):
        out, at = {}, 0
        for name, s in self.sizes.items():
            out[name] = flat[at:at + torch.Size(s).numel()].view(s)
            at += torch.Size(s).numel()
        return out

    def params(self, flat):
        p = self.views(flat)
        return {**p, **{k: list(p[k].chunk(self.shards)) for k in ("e", "w1", "w2")}}

    def buffers(self, m, dev):
        """What a rank allocates once for batches of m tokens."""
        def new(cols, dtype=BF16):
            return torch.empty(m, cols, dtype=dtype, device=dev)

        d, f, one = self.d, self.f, dict(device=dev)
        spaces = [z.fsdp_vocab_loss_forward_workspace(m, self.vocab), z.fsdp_vocab_loss_backward_workspace(m, self.vocab, d),
                  z.fsdp_layernorm_backward_workspace(m, d), z.fsdp_embedding_backward_workspace(m, self.vocab, d)]
        return {"x0": new(d), "h1": new(d), "pre": new(f), "hid": new(f), "x1": new(d), "h2": new(d), "dh2": new(d), "dx1": new(d),
                "dpre": new(f), "dh1": new(d), "dx0": new(d), "loss": torch.empty(m, **one), "lse": torch.empty(m, **one),
                "total": torch.empty(2, **one), "stat1": torch.empty(2, m, **one), "stat2": torch.empty(2, m, **one),
                "db1": torch.empty(f, **one), "small": torch.empty(5, d, **one),
                "ws": torch.empty(max(spaces), dtype=torch.uint8, device=dev)}


def forward(model, p, tokens, labels, b):
    """Leaves the batch's sum of losses and count in b["total"]."""
    z.fsdp_embedding_forward(p["e"], tokens, b["x0"], vocab=model.vocab)
    z.fsdp_layernorm_forward(b["x0"], b["h1"], gamma=p["g1"], beta=p["c1"], eps=EPS, mean=b["stat1"][0], rstd=b["stat1"][1])
    z.fsdp_linear_forward(p["w1"], b["h1"], b["hid"], bias=p["b1"], act=z.FSDP_ACT_GELU, z=b["pre"])
    z.fsdp_linear_forward(p["w2"], b["hid"], b["x1"], bias=p["b2"], residual=b["x0"])
    z.fsdp_layernorm_forward(b["x1"], b["h2"], gamma=p["g2"], beta=p["c2"], eps=EPS, mean=b["stat2"][0], rstd=b["stat2"][1])
    z.fsdp_vocab_loss_forward(p["e"], b["h2"], labels, b["loss"], b["lse"], total=b["total"], vocab=model.vocab, workspace=b["ws"])


def backward(model, p, tokens, labels, g, b):
    """Gradients of the mean loss into g (every tensor of the model, bf16)."""
    ws, small = b["ws"], b["small"]
    z.fsdp_vocab_loss_backward(p["e"], b["h2"], labels, b["lse"], b["dh2"], g["e"], vocab=model.vocab, total=b["total"], workspace=ws)
    z.fsdp_layernorm_backward(b["dh2"], b["x1"], b["stat2"][0], b["stat2"][1], b["dx1"], gamma=p["g2"], dgamma=small[0],
                              dbeta=small[1], workspace=ws)
    z.fsdp_linear_dw(b["dx1"], g["w2"], x=b["hid"])
    z.fsdp_act_backward(b["dx1"], db=small[2])
    z.fsdp_linear_dx(p["w2"], b["dx1"], b["dpre"], z=b["pre"], act=z.FSDP_ACT_GELU)  # through the GELU
    z.fsdp_linear_dw(b["dpre"], g["w1"], x=b["h1"])
    z.fsdp_act_backward(b["dpre"], db=b["db1"])
    z.fsdp_linear_dx(p["w1"], b["dpre"], b["dh1"])
    z.fsdp_layernorm_backward(b["dh1"], b["x0"], b["stat1"][0], b["stat1"][1], b["dx0"], gamma=p["g1"], residual=b["dx1"],
                              dgamma=small[3], dbeta=small[4], workspace=ws)  # joined with the skip path
    # the table's gradient as the embedding, on top of its gradient as the output layer
    z.fsdp_embedding_backward(b["dx0"], tokens, g["e"], vocab=model.vocab, accumulate=True, workspace=ws)
    for name, value in (("g2", small[0]), ("c2", small[1]), ("b2", small[2]), ("g1", small[3]), ("c1", small[4]), ("b1", b["db1"])):
        g[name].copy_(value)


def setup(model, n, m, dev, seed=0):
    """Master parameters, moments, each rank's gradients, batches and buffers. The text: each word is followed by one of its
    own; a batch's last tokens are padding."""
    gen = torch.Generator(device=dev).manual_seed(seed)
    plan = z.zero_plan(model.psi, n, "zero2", 1 << 20)
    P = plan.psi_padded
    master, mom, var = torch.zeros(P, device=dev), torch.zeros(P, device=dev), torch.zeros(P, device=dev)
    for name, t in model.views(master[:model.psi]).items():
        if name in ("g1", "g2"):
            t.fill_(1.0)
        elif name in ("e", "w1", "w2"):
            t.copy_(torch.randn(*t.shape, generator=gen, device=dev) * t.shape[1] ** -0.5)
    follows = torch.randperm(model.vocab, generator=gen, device=dev)
    batches = []
    for _ in range(n):
        tokens = torch.randint(0, model.vocab, (m,), generator=gen, device=dev)
        labels = follows[tokens]
        tokens[m - m // 8:], labels[m - m // 8:] = -100, -100
        batches.append((tokens, labels))
    return {"plan": plan, "master": master, "m": mom, "v": var, "param": master.to(BF16),
            "grads": [torch.zeros(P, dtype=BF16, device=dev) for _ in range(n)], "batches": batches,
            "bufs": [model.buffers(m, dev) for _ in range(n)]}


def main(steps=20, n=2, m=384):
    model, dev = Model(), torch.device("cuda")
    s = setup(model, n, m, dev)
    p = model.params(s["param"][:model.psi])
    hp = {"lr": 3e-3, "beta1": 0.9, "beta2": 0.95, "eps": 1e-8, "weight_decay": 0.0}
    losses = []
    for step in range(1, steps + 1):
        for r in range(n):
            forward(model, p, *s["batches"][r], s["bufs"][r])
            backward(model, p, *s["batches"][r], model.views(s["grads"][r][:model.psi]), s["bufs"][r])
        z.zero_fused_step(s["plan"], z.ZERO_ALL_RANKS, s["grads"], s["master"], s["m"], s["v"], s["param"], hp, step)
        losses.append(sum(b["total"][0] / b["total"][1] for b in s["bufs"]) / n)
    z.zero_device_status()   # synchronises; raises ZeroError if a device-side check fired
    return [float(t) for t in losses]


if __name__ == "__main__":
    for i, loss in enumerate(main()):
        print(f"step {i + 1:3d}  loss {loss:.4f}")
