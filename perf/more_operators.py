"""What is measured of the 4-bit weights: storing a matrix (quantize, and reading it back), the linear layer over a stored
matrix, optionally with the RMSNorm before it and the residual behind it (linear), and the first half of a gated
feed-forward block over two stored matrices (glu).

A stored matrix [n, k] holds codes -8 .. 7, two in a byte (the even column in the low half), and one bf16 scale for each
`group` columns of a row; it stands for code * scale.  Each case says its sizes; values follow from the seed."""
import math

import torch

own = False

EPS = 1e-5


# ---- the cases ----

def listed():
    def store(name, n, k, group, dtype):
        return dict(name=name, op="store", dtype=dtype, tokens=0, n=n, k=k, group=group, norm=False, residual=False, act="")

    def linear(name, tokens, n, k, group, dtype, norm=False, residual=False):
        return dict(name=name, op="linear", dtype=dtype, tokens=tokens, n=n, k=k, group=group, norm=norm, residual=residual,
                    act="")

    def glu(name, tokens, n, k, group, dtype, norm=True, act="silu"):
        return dict(name=name, op="glu", dtype=dtype, tokens=tokens, n=n, k=k, group=group, norm=norm, residual=False, act=act)
    return [
        # the key projection of the 1B-class model, fp32 as it was trained
        store("store_key", 512, 2048, 32, "f32"),
        # a feed-forward matrix of the 8B-shape model
        store("store_ffn", 14336, 4096, 128, "bf16"),
        # one sequence decodes: the output projection of the 1B-class model into its residual stream, nothing but latency
        linear("token_small", 1, 2048, 2048, 128, "f32", residual=True),
        # the stacked query, key and value projections of the 8B-shape model for one token
        linear("token_qkv", 1, 6144, 4096, 128, "f32", norm=True),
        # the logits of one token over the 8B-shape model's vocabulary: as many bytes as a decode step reads at once
        linear("token_head", 1, 128256, 4096, 64, "f32", norm=True),
        # three sequences through a matrix of odd sizes and small groups
        linear("tokens_odd", 3, 1001, 1120, 32, "bf16"),
        # a serving batch of eight: the down projection into the residual stream
        linear("batch_down", 8, 4096, 14336, 128, "f32", residual=True),
        # eight sequences with drafts of five tokens each
        linear("drafts_qkv", 40, 6144, 4096, 128, "bf16", norm=True),
        # a long prompt, of odd length: the largest contraction
        linear("prompt_down", 4095, 4096, 14336, 128, "bf16", residual=True),
        # one token through the 1B-class model's feed-forward block
        glu("glu_token", 1, 8192, 2048, 64, "f32"),
        # a serving batch of eight through the 8B-shape model's
        glu("glu_batch", 8, 14336, 4096, 32, "f32"),
        # a prompt of 1000 tokens, fp32 activations, the other activation function
        glu("glu_prompt", 1000, 14336, 4096, 128, "f32", act="gelu_tanh"),
    ]


def draw(rng):
    def log(a, b):
        return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))
    op = rng.choice(["store", "linear", "linear", "linear", "glu", "glu"])
    group = rng.choice([32, 64, 128])
    k = group * max(1, log(64, 16384) // group)
    n = log(1, 32768)
    tokens = 0 if op == "store" else log(1, 12) if rng.random() < 0.6 else log(13, 4095)
    while n * k > 14336 * 4096 or max(1, tokens) * n * k > 4095 * 4096 * 14336 // 4:
        n = max(1, n * 2 // 3)
    return dict(op=op, dtype=rng.choice(["f32", "bf16"]), tokens=tokens, n=n, k=k, group=group,
                norm=op != "store" and rng.random() < 0.5, residual=op == "linear" and rng.random() < 0.5,
                act=rng.choice(["silu", "gelu_tanh"]) if op == "glu" else "")


def work(c):
    n, k, t, size = c["n"], c["k"], c["tokens"], 4 if c["dtype"] == "f32" else 2
    held = n * k // 2 + 2 * n * (k // c["group"])              # codes and scales
    if c["op"] == "store":
        # the matrix read, its codes and scales written and read, the values that they stand for written
        return {"bytes": 2 * n * k * size + 2 * held, "flops": 3 * n * k}
    matrices = 2 if c["op"] == "glu" else 1
    return {"bytes": matrices * held + size * (t * k + t * n * (2 if c["residual"] else 1) + (k if c["norm"] else 0)),
            "flops": 2 * matrices * t * n * k}


# ---- inputs ----

def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    g = torch.Generator(dev).manual_seed(seed)
    dt = torch.float32 if c["dtype"] == "f32" else torch.bfloat16
    n, k, t = c["n"], c["k"], c["tokens"]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    def matrix():
        # rows of unlike size, and a few columns larger than the rest, as they are in trained models
        w = normal(n, k).mul_(0.02)
        w.mul_(torch.exp(0.3 * normal(n, 1)))
        return w.mul_(1.0 + 4.0 * (torch.rand(1, k, generator=g, device=dev) > 0.98))
    s = dict(case=c)
    if c["op"] == "store":
        s["w"] = matrix().to(dt)
        s["codes"] = torch.empty(n, k // 2, dtype=torch.uint8, device=dev)
        s["scales"] = torch.empty(n, k // c["group"], dtype=torch.bfloat16, device=dev)
        s["values"] = torch.empty_like(s["w"])
        return s
    s["stored"] = [plain_quantize(matrix(), c["group"]) for _ in range(2 if c["op"] == "glu" else 1)]
    # activations of unlike size, a few channels larger than the rest
    wide = 1.0 + 9.0 * (torch.rand(k, generator=g, device=dev) > 0.99)
    s["x"] = (normal(t, k) * wide * torch.exp(0.5 * normal(t, 1))).to(dt)
    s["norm"] = (1.0 + 0.1 * normal(k)).to(dt) if c["norm"] else None
    s["residual"] = normal(t, n).to(dt) if c["residual"] else None
    s["out"] = torch.empty(t, n, dtype=dt, device=dev)
    if own:
        from graph_replay_gb300 import W4Weight
        s["weights"] = [W4Weight(codes, scales) for codes, scales in s["stored"]]
    return s


# ---- one pass ----

def run(state):
    s, c = state, state["case"]
    if own:
        if c["op"] == "store":
            from graph_replay_gb300 import W4Weight
            w = W4Weight.quantize(s["w"], group=c["group"], codes=s["codes"], scales=s["scales"])
            return {"values": w.dequantize(out=s["values"]), "scales": s["scales"]}
        if c["op"] == "linear":
            return s["weights"][0].linear(s["x"], norm=s["norm"], eps=EPS, residual=s["residual"], out=s["out"])
        gate, up = s["weights"]
        return gate.glu(up, s["x"], act=c["act"], norm=s["norm"], eps=EPS, out=s["out"])
    if c["op"] == "store":
        codes, scales = plain_quantize(s["w"], c["group"])
        s["codes"].copy_(codes)
        s["scales"].copy_(scales)
        s["values"].copy_(plain_values(s["codes"], s["scales"]))
        return {"values": s["values"], "scales": s["scales"]}
    x = s["x"].float()
    if c["norm"]:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * s["norm"].float()
    y = x @ plain_values(*s["stored"][0]).T
    if c["op"] == "glu":
        up = x @ plain_values(*s["stored"][1]).T
        if c["act"] == "silu":
            y = y / (1.0 + torch.exp(-y)) * up
        else:
            y = 0.5 * y * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (y + 0.044715 * y * y * y))) * up
    elif c["residual"]:
        y = y + s["residual"].float()
    s["out"].copy_(y)
    return s["out"]


def plain_quantize(w, group):
    """(codes [n, k / 2], scales [n, k / group]) of w: scale = bf16(max |w| / 7) over a group, code = w / scale to the
    nearest whole number, ties to even.  A group whose scale is below 2^-100 holds zeros at scale 0."""
    n, k = w.shape
    x = w.float().view(n, k // group, group)
    scale = (x.abs().amax(-1) / torch.full((), 7.0, device=w.device)).to(torch.bfloat16)   # a scalar would multiply by 1 / 7
    scale[scale < 2.0 ** -100] = 0.0
    s = scale.float()[..., None]
    q = torch.where(s > 0, torch.round(x / torch.where(s > 0, s, 1.0)), 0.0).to(torch.int8).view(n, k // 2, 2)
    return ((q[..., 0] & 15) | (q[..., 1] << 4)).view(torch.uint8), scale


def plain_values(codes, scales):
    """The fp32 matrix that codes and scales stand for."""
    n, groups = scales.shape
    q = codes.view(torch.int8)
    q = torch.stack([(q << 4) >> 4, q >> 4], -1).view(n, groups, -1)
    return (q.float() * scales.float()[..., None]).view(n, -1)


# ---- the definition in 64 bits ----

def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["op"] == "store":
        w = s["w"].double().unflatten(1, (-1, c["group"]))
        scale = to_bf16(torch.linalg.vector_norm(w, math.inf, dim=2) / 7.0)
        scale = torch.where(scale < 2.0 ** -100, 0.0, scale)
        code = torch.round(w / scale.clamp_min(2.0 ** -200)[..., None])
        value = code * scale[..., None]
        if c["dtype"] == "bf16":
            value = to_bf16(value)
        return {"values": value.flatten(1), "scales": scale}
    x = s["x"].double()
    if c["norm"]:
        x = x / torch.sqrt(x.square().sum(1, keepdim=True) / c["k"] + EPS) * s["norm"].double()
    y = [product(x, codes, scales, c["group"]) for codes, scales in s["stored"]]
    if c["op"] == "linear":
        return y[0] + s["residual"].double() if c["residual"] else y[0]
    if c["act"] == "silu":
        return y[0] * torch.sigmoid(y[0]) * y[1]
    u = math.sqrt(2.0 / math.pi) * (y[0] + 0.044715 * y[0] ** 3)
    return y[0] * torch.sigmoid(2.0 * u) * y[1]                   # (1 + tanh u) / 2


def to_bf16(x):
    """64-bit values to 8 significant bits, to the nearest, ties to even (bf16's normal range is enough here)."""
    b = x.contiguous().view(torch.int64)
    return ((b + (2 ** 44 - 1) + ((b >> 45) & 1)) >> 45 << 45).view(torch.float64)


def product(x, codes, scales, group):
    """x [t, k] times the stored matrix, group by group: each group's products with its codes, times its scales."""
    y = torch.zeros(x.shape[0], codes.shape[0], dtype=torch.float64, device=x.device)
    for i in range(scales.shape[1]):
        b = codes[:, i * group // 2:(i + 1) * group // 2].long()
        q = torch.empty(b.shape[0], group, dtype=torch.float64, device=x.device)
        q[:, 0::2] = (b % 16 - 16 * (b % 16 >= 8)).double()
        q[:, 1::2] = (b // 16 - 16 * (b // 16 >= 8)).double()
        y.addcmul_(x[:, i * group:(i + 1) * group] @ q.T, scales[:, i].double())
    return y
