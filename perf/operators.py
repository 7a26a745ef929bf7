"""Cases of the linear unit with its epilogue (fsdp_linear_forward, fsdp_act_backward,
fsdp_linear_dx, fsdp_linear_dw) and of the 8-bit activation checkpoints it saves and reads
(fsdp_checkpoint8_pack, fsdp_checkpoint8_unpack).

Each case is one call (or, where an 8-bit checkpoint is part of the answer, the call and
the read of the checkpoint: codes are returned as the values they stand for). `run` with
`own` false computes the same in elementary torch operations in 32 bits, rounded once at the
end; `exact` computes it in 64 bits. Sizes are those of this repository's workloads (widths
768 and 2304, 4096, 14336 and 1024, 8 ranks, 8192 tokens) and ragged ones beside them.

A case: op; m tokens; r x k the weight [r, k] (ops fwd, dx, dw) or k the width (actb, ckpt);
n row shards of the weight; act; bits: how activations are kept (16: bf16, 8: codes with one
power-of-two scale per 32 columns); bias, res: whether the call adds a bias and a residual;
out: the type of dW.
"""
import math

import torch

own = False
G = 32  # columns that share a scale
ACTS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
MOST = 8192 * 4096 * 14336  # m r k of the largest listed case


def listed():
    return [
        # one token through a 4096 -> 1024 projection: latency, 8 MB of weight
        {"name": "fwd one token", "op": "fwd", "m": 1, "r": 1024, "k": 4096, "n": 8, "act": "none", "bits": 16,
         "bias": True, "res": False},
        # widths and a token count that end inside every tile, five shards of 232 rows
        {"name": "fwd ragged", "op": "fwd", "m": 1003, "r": 1160, "k": 520, "n": 5, "act": "gelu_tanh", "bits": 16,
         "bias": True, "res": True},
        # a 768-wide model's first linear, one 4096-token micro-batch, checkpoint in 8 bits
        {"name": "fwd 768", "op": "fwd", "m": 4096, "r": 2304, "k": 768, "n": 8, "act": "gelu_tanh", "bits": 8,
         "bias": True, "res": False},
        # a 4096-wide model's MLP up projection over 8192 tokens, checkpoint in 8 bits
        {"name": "fwd 4096", "op": "fwd", "m": 8192, "r": 14336, "k": 4096, "n": 8, "act": "silu", "bits": 8,
         "bias": True, "res": False},
        # a short last micro-batch of the 768-wide model, pre-activation kept in bf16
        {"name": "actb short", "op": "actb", "m": 777, "k": 2304, "act": "gelu", "bits": 16},
        # the 4096-wide model's MLP activation, 8192 tokens, from 8 bits
        {"name": "actb 14336", "op": "actb", "m": 8192, "k": 14336, "act": "silu", "bits": 8},
        # a 768-wide model's second linear: its input gradient through the first one's activation
        {"name": "dx 768", "op": "dx", "m": 1000, "r": 768, "k": 2304, "n": 8, "act": "gelu_tanh", "bits": 8,
         "res": False},
        # the 4096-wide model's down projection: the same over 8192 tokens
        {"name": "dx 4096", "op": "dx", "m": 8192, "r": 4096, "k": 14336, "n": 8, "act": "silu", "bits": 8,
         "res": False},
        # weight gradient of a 768 x 768 projection over an odd number of tokens, fp32 for the fp32-gradient step
        {"name": "dw 768", "op": "dw", "m": 2041, "r": 768, "k": 768, "n": 1, "bits": 16, "out": "fp32"},
        # weight gradient of the up projection from the 8-bit checkpoint of its input, bf16 for the bf16-gradient step
        {"name": "dw 4096", "op": "dw", "m": 8192, "r": 14336, "k": 4096, "n": 1, "bits": 8, "out": "bf16"},
        # a checkpoint of a ragged block input, written and read back
        {"name": "ckpt ragged", "op": "ckpt", "m": 333, "k": 1160, "act": "none", "bits": 8},
        # the MLP's hidden state recomputed from the checkpoint of its pre-activation
        {"name": "ckpt 14336", "op": "ckpt", "m": 8192, "k": 14336, "act": "silu", "bits": 8},
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["fwd", "fwd", "actb", "dx", "dw", "ckpt"])
    m = log(1, 16384)
    width = lambda: 8 * log(8, 1792)  # noqa: E731
    k = width()
    c = {"op": op, "m": m, "k": k, "bits": rng.choice([8, 16])}
    if op in ("actb", "ckpt"):
        c["m"] = max(1, min(m, 8192 * 14336 // k))
        c["act"] = rng.choice(sorted(ACTS))
        c["bits"] = 8 if op == "ckpt" else c["bits"]
        return c
    r = width()
    while m * r * k > MOST:
        r = width()
        m = c["m"] = log(1, 16384)
    n = rng.choice([1, 2, 4, 5, 8, 16])
    r = max(8 * n, r // (8 * n) * 8 * n)  # whole groups of 8 rows in each shard
    c["r"], c["n"] = r, n if op != "dw" else 1
    if op == "dw":
        c["out"] = rng.choice(["fp32", "bf16"])
        return c
    c["act"], c["res"] = rng.choice(sorted(ACTS)), rng.choice([True, False])
    if op == "fwd":
        c["bias"] = rng.choice([True, False])
    return c


# ---- inputs ----

def _power(b):
    """2^(b - 127) in fp32, exactly, b in 1..254 (an exp2 may be an ulp off, which breaks ties)."""
    return (b.to(torch.int32) << 23).view(torch.float32)


def _pack(x):
    """Codes and scale bytes of x [rows, cols] fp32, elementary operations (input making)."""
    rows, cols = x.shape
    pad = -cols % G
    g = torch.nn.functional.pad(x, (0, pad)).view(rows, -1, G)
    b = ((g.abs().amax(-1).view(torch.int32) + 0x10000) >> 23) - 6
    b = b.clamp(1, 248)
    c = torch.round(g * _power(254 - b).unsqueeze(-1)).clamp(-127, 127)
    return c.view(rows, -1)[:, :cols].to(torch.int8).contiguous(), b.to(torch.uint8)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed * 7919 + 17)
    bf = torch.bfloat16

    def normal(rows, cols, std, outliers=False):
        t = torch.randn(rows, cols, generator=gen, device=dev) * std
        if outliers:  # a few channels an order larger than the rest, as trained models have
            t[:, torch.randint(0, cols, (max(1, cols // 256),), generator=gen, device=dev)] *= 12.0
        return t.to(bf)

    op, m, k = case["op"], case["m"], case["k"]
    s = {"case": dict(case)}
    new = lambda rows, cols, dt=bf: torch.empty(rows, cols, dtype=dt, device=dev)  # noqa: E731

    def new8(rows, cols):
        return new(rows, cols, torch.int8), new(rows, -(-cols // G), torch.uint8)

    def kept(rows, cols, outliers=False):  # an activation as the forward kept it
        t = normal(rows, cols, 1.3, outliers)
        return t if case["bits"] == 16 else _pack(t.float())

    if op in ("fwd", "dx"):
        r, n = case["r"], case["n"]
        s["shards"] = [normal(r // n, k, 0.02) for _ in range(n)]
    if op == "fwd":
        s["x"] = normal(m, k, 1.0, True)
        s["bias"] = normal(1, r, 0.1)[0].contiguous() if case["bias"] else None
        s["res"] = normal(m, r, 1.0) if case["res"] else None
        s["y"] = new(m, r)
        s["z"] = new(m, r)
        s["z8"] = new8(m, r) if case["bits"] == 8 else None
    elif op == "actb":
        s["dy"] = normal(m, k, 1e-2)
        s["act_in"] = kept(m, k)
        s["dz"], s["db"] = new(m, k), torch.empty(k, device=dev)
    elif op == "dx":
        s["dz"] = normal(m, r, 1e-2)
        s["act_in"] = kept(m, k)
        s["res"] = normal(m, k, 1e-2) if case["res"] else None
        s["dx"] = new(m, k)
    elif op == "dw":
        s["dz"] = normal(m, case["r"], 1e-2)
        s["act_in"] = kept(m, k, True)
        s["dw"] = new(case["r"], k, torch.float32 if case["out"] == "fp32" else bf)
    else:
        s["x"] = normal(m, k, 1.3, True)
        s["z8"] = new8(m, k)
        s["out"] = new(m, k)
    return s


# ---- the plain form ----

def _act(z, act):
    if act == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _dact(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if act == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3.0 * 0.044715 * z * z)
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-z))
        return s * (1.0 + z * (1.0 - s))
    return torch.ones_like(z)


def _values(codes, scales):
    rows, cols = codes.shape
    return codes.float() * _power(scales).repeat_interleave(G, 1)[:, :cols]


def _through8(z):
    return _values(*_pack(z))


def _kept(t):
    return _values(*t) if isinstance(t, tuple) else t.float()


def _plain(s):
    c = s["case"]
    op, bf = c["op"], torch.bfloat16
    if op == "fwd":
        z = s["x"].float() @ torch.cat(s["shards"]).float().t()
        if s["bias"] is not None:
            z += s["bias"].float()
        y = _act(z, c["act"])
        if s["res"] is not None:
            y = y + s["res"].float()
        return {"y": y.to(bf), "z": (_through8(z) if c["bits"] == 8 else z).to(bf)}
    if op == "actb":
        dz = s["dy"].float() * _dact(_kept(s["act_in"]), c["act"])
        return {"dz": dz.to(bf), "db": dz.sum(0)}
    if op == "dx":
        dx = (s["dz"].float() @ torch.cat(s["shards"]).float()) * _dact(_kept(s["act_in"]), c["act"])
        if s["res"] is not None:
            dx = dx + s["res"].float()
        return {"dx": dx.to(bf)}
    if op == "dw":
        dw = (s["dz"].float().t() @ _kept(s["act_in"])) * 0.125
        return {"dw": dw if c["out"] == "fp32" else dw.to(bf)}
    return {"values": _act(_through8(s["x"].float()), c["act"]).to(bf)}


# ---- the calls a user makes ----

def _calls(s):
    import fsdp_sharded_optimizer_zero_gb300 as z

    c = s["case"]
    op = c["op"]
    act = ACTS[c.get("act", "none")]
    kept = s.get("act_in")
    as16, as8 = (None, kept) if isinstance(kept, tuple) else (kept, None)
    if op == "fwd":
        if c["bits"] == 8:
            z.fsdp_linear_forward(s["shards"], s["x"], s["y"], bias=s["bias"], act=act, residual=s["res"], z8=s["z8"])
            z.fsdp_checkpoint8_unpack(*s["z8"], s["z"])
        else:
            z.fsdp_linear_forward(s["shards"], s["x"], s["y"], bias=s["bias"], act=act, residual=s["res"], z=s["z"])
        return {"y": s["y"], "z": s["z"]}
    if op == "actb":
        z.fsdp_act_backward(s["dy"], s["dz"], db=s["db"], z=as16, z8=as8, act=act)
        return {"dz": s["dz"], "db": s["db"]}
    if op == "dx":
        z.fsdp_linear_dx(s["shards"], s["dz"], s["dx"], z=as16, z8=as8, act=act, residual=s["res"])
        return {"dx": s["dx"]}
    if op == "dw":
        z.fsdp_linear_dw(s["dz"], s["dw"], x=as16, x8=as8, scale=0.125)
        return {"dw": s["dw"]}
    z.fsdp_checkpoint8_pack(s["x"], *s["z8"])
    z.fsdp_checkpoint8_unpack(*s["z8"], s["out"], act=act)
    return {"values": s["out"]}


def run(state):
    return _calls(state) if own else _plain(state)


def work(case):
    op, m, k = case["op"], case["m"], case["k"]
    r = case.get("r", 0)
    kept = lambda cols: 2 * m * cols if case["bits"] == 16 else m * (cols + -(-cols // G))  # noqa: E731
    if op == "fwd":  # X, W, bias, residual; Y, Z (in 8 bits: the checkpoint and the values read from it)
        b = 2 * (m * k + r * k + 2 * m * r) + 2 * r * case["bias"] + 2 * m * r * case["res"]
        return {"bytes": b + (kept(r) if case["bits"] == 8 else 0), "flops": 2 * m * r * k}
    if op == "actb":
        return {"bytes": 4 * m * k + kept(k) + 4 * k, "flops": 0}
    if op == "dx":
        b = 2 * (m * r + r * k + m * k) + kept(k) * (case["act"] != "none") + 2 * m * k * case["res"]
        return {"bytes": b, "flops": 2 * m * r * k}
    if op == "dw":
        return {"bytes": 2 * m * r + kept(k) + r * k * (4 if case["out"] == "fp32" else 2), "flops": 2 * m * r * k}
    return {"bytes": 4 * m * k + kept(k), "flops": 0}


# ---- 64 bits, from the definitions ----

def exact(case, seed):
    s = prepare(case, seed)
    op, act = case["op"], case.get("act", "none")
    d = lambda t: t.double()  # noqa: E731

    def power(e):  # 2^e, exactly
        return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)

    def sigmoid(x):
        return 1.0 / (1.0 + torch.exp(-x))

    def f(x):
        if act == "relu":
            return x.clamp(min=0)
        if act == "gelu":  # x Phi(x)
            return 0.5 * x * torch.erfc(-x / 2.0 ** 0.5)
        if act == "gelu_tanh":  # (1 + tanh u) / 2 = sigmoid(2 u)
            return x * sigmoid(2.0 * (2.0 / math.pi) ** 0.5 * (x + 0.044715 * x ** 3))
        return x * sigmoid(x) if act == "silu" else x

    def df(x):
        if act == "relu":
            return torch.heaviside(x, torch.zeros((), dtype=x.dtype, device=x.device))
        if act == "gelu":
            return 0.5 * torch.erfc(-x / 2.0 ** 0.5) + x * torch.exp(-x * x / 2.0) / (2.0 * math.pi) ** 0.5
        if act == "gelu_tanh":
            a = 2.0 * (2.0 / math.pi) ** 0.5
            p = sigmoid(a * (x + 0.044715 * x ** 3))
            return p + x * p * (1.0 - p) * a * (1.0 + 3.0 * 0.044715 * x * x)
        if act == "silu":
            p = sigmoid(x)
            return p + x * p * (1.0 - p)
        return torch.ones_like(x)

    def through8(x):  # the nearest multiples of 2^e, 2^e the least power of two >= amax / 127.5 (2^-126 at least)
        out = x.clone()
        for j in range(0, x.shape[1], G):
            part = x[:, j:j + G]
            amax = part.abs().amax(1, keepdim=True)
            mant, e = torch.frexp(amax)  # amax = mant 2^e, mant in [0.5, 1)
            e = e - 7 + (mant >= 127.5 / 128.0).to(e.dtype)
            e = torch.where(amax == 0, torch.full_like(e, -126), e).clamp(-126, 121)
            u = power(e)
            out[:, j:j + G] = torch.round(part / u).clamp(-127, 127) * u
        return out

    def value(t):
        if not isinstance(t, tuple):
            return d(t)
        codes, scales = t
        col = torch.arange(codes.shape[1], device=codes.device) // G
        return d(codes) * power(scales.to(torch.int64) - 127)[:, col]

    if op == "fwd":
        z = torch.cat([d(s["x"]) @ d(w).t() for w in s["shards"]], 1)
        if s["bias"] is not None:
            z = z + d(s["bias"])
        y = f(z)
        if s["res"] is not None:
            y = y + d(s["res"])
        return {"y": y, "z": through8(z) if case["bits"] == 8 else z}
    if op == "actb":
        dz = d(s["dy"]) * df(value(s["act_in"]))
        return {"dz": dz, "db": dz.sum(0)}
    if op == "dx":
        rows = s["shards"][0].shape[0]
        g = sum(d(s["dz"][:, i * rows:(i + 1) * rows]) @ d(w) for i, w in enumerate(s["shards"]))
        g = g * df(value(s["act_in"]))
        return {"dx": g if s["res"] is None else g + d(s["res"])}
    if op == "dw":
        return {"dw": d(s["dz"]).t() @ value(s["act_in"]) / 8.0}
    return {"values": f(through8(d(s["x"])))}
