"""A residual MLP block trained with the linear unit, its activations kept in 8 bits, and the
fused ZeRO step.

    H = gelu(X W1^T + b1),   Y = H W2^T + b2 + X

Two data-parallel ranks are simulated as separate gradient buffers, each with its own batch.
Between forward and backward a rank keeps 8-bit checkpoints alone: of its input X and of the
first layer's pre-activation (from which H is recomputed). Weights and biases live in one flat
bf16 parameter buffer, gradients in one flat bf16 buffer per rank, and zero_fused_step reduces,
updates and casts them in one pass. Run with
`python -m fsdp_sharded_optimizer_zero_gb300.example_linear` on a GPU."""
import torch

import fsdp_sharded_optimizer_zero_gb300 as z

BF16 = torch.bfloat16


def block_buffers(m, d, f, dev):
    """What a rank allocates once: the kept checkpoints and the passes' buffers."""
    def new(rows, cols, dtype=BF16):
        return torch.empty(rows, cols, dtype=dtype, device=dev)

    def checkpoint(rows, cols):
        groups = -(-cols // z.FSDP_CHECKPOINT8_GROUP)
        return new(rows, cols, torch.int8), new(rows, groups, torch.uint8)

    return {"x8": checkpoint(m, d), "z8": checkpoint(m, f), "h": new(m, f), "y": new(m, d), "dz": new(m, f),
            "dx": new(m, d), "db1": torch.empty(f, device=dev), "db2": torch.empty(d, device=dev),
            "ws": torch.empty(z.fsdp_linear_dw_workspace(m, d), dtype=torch.uint8, device=dev)}


def forward(p, x, b):
    """p: w1, b1, w2, b2 (each weight a list of row shards). Keeps X and Z in 8 bits."""
    z.fsdp_checkpoint8_pack(x, *b["x8"])
    z.fsdp_linear_forward(p["w1"], x, b["h"], bias=p["b1"], act=z.FSDP_ACT_GELU, z8=b["z8"])
    z.fsdp_linear_forward(p["w2"], b["h"], b["y"], bias=p["b2"], residual=x)
    return b["y"]


def backward(p, dy, g, b):
    """Gradients of the block from dY and the checkpoints, into g (w1, b1, w2, b2, bf16);
    returns dX."""
    z.fsdp_checkpoint8_unpack(*b["z8"], b["h"], act=z.FSDP_ACT_GELU)          # H again
    z.fsdp_linear_dw(dy, g["w2"], x=b["h"])
    z.fsdp_act_backward(dy, db=b["db2"])
    z.fsdp_linear_dx(p["w2"], dy, b["dz"], z8=b["z8"], act=z.FSDP_ACT_GELU)   # through the GELU
    z.fsdp_linear_dw(b["dz"], g["w1"], x8=b["x8"], workspace=b["ws"])
    z.fsdp_act_backward(b["dz"], db=b["db1"])
    z.fsdp_linear_dx(p["w1"], b["dz"], b["dx"], residual=dy)                  # joined with the skip path
    g["b1"].copy_(b["db1"])
    g["b2"].copy_(b["db2"])
    return b["dx"]


def main(steps=20, n=2, m=256, d=128, f=512, shards=2, seed=0):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)

    def randn(*shape, std=1.0):
        return torch.randn(*shape, generator=gen, device=dev) * std

    sizes = {"w1": (f, d), "b1": (f,), "w2": (d, f), "b2": (d,)}
    psi = sum(torch.Size(s).numel() for s in sizes.values())
    plan = z.zero_plan(psi, n, "zero2", 1 << 20)
    P = plan.psi_padded

    def views(flat):
        out, at = {}, 0
        for name, s in sizes.items():
            out[name] = flat[at:at + torch.Size(s).numel()].view(s)
            at += torch.Size(s).numel()
        return out

    master, mom, var = torch.zeros(P, device=dev), torch.zeros(P, device=dev), torch.zeros(P, device=dev)
    for name, t in views(master[:psi]).items():
        if name.startswith("w"):
            t.copy_(randn(*t.shape, std=t.shape[1] ** -0.5))
    param = master.to(BF16)
    grads = [torch.zeros(P, dtype=BF16, device=dev) for _ in range(n)]
    v = views(param[:psi])
    p = {"w1": list(v["w1"].chunk(shards)), "b1": v["b1"], "w2": list(v["w2"].chunk(shards)), "b2": v["b2"]}
    bufs = [block_buffers(m, d, f, dev) for _ in range(n)]
    batches = [(randn(m, d).to(BF16), randn(m, d)) for _ in range(n)]  # each rank's inputs and targets
    hp = {"lr": 3e-3, "beta1": 0.9, "beta2": 0.95, "eps": 1e-8, "weight_decay": 0.0}

    losses = []
    for step in range(1, steps + 1):
        total = 0.0
        for r in range(n):
            x, target = batches[r]
            diff = forward(p, x, bufs[r]).float() - target
            total = total + 0.5 * diff.square().mean()
            backward(p, (diff / diff.numel()).to(BF16), views(grads[r][:psi]), bufs[r])
        z.zero_fused_step(plan, z.ZERO_ALL_RANKS, grads, master, mom, var, param, hp, step)
        losses.append(total / n)
    z.zero_device_status()   # synchronises; raises ZeroError if a device-side check fired
    return [float(t) for t in losses]


if __name__ == "__main__":
    for i, loss in enumerate(main()):
        print(f"step {i + 1:3d}  loss {loss:.4f}")
