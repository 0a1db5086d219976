"""What is measured of the 8-bit K/V cache: storing new tokens (append) and attention over the cache (attend) for single
tokens and for prompts, causal, optionally within a sliding window beside the first tokens of a sequence (sinks).

The cache holds K and V as e4m3 with one power-of-two scale for each block of `block` positions and K/V head.  Each case
says its sizes; lengths of a batch follow from the case alone, values from the seed."""
import math

import torch

own = False

LOW, HIGH = -40, 60   # exponents a scale may take


# ---- the cases ----

def listed():
    def case(name, op, dtype, rows, heads, kv_heads, dim, length, new=1, page=64, block=64, window=0, sinks=0, ragged=True):
        return dict(name=name, op=op, dtype=dtype, rows=rows, heads=heads, kv_heads=kv_heads, dim=dim, length=length,
                    new=new, page=page, block=block, window=window, sinks=sinks, ragged=ragged)
    return [
        # one sequence decodes its next token: the new K/V enters a half-filled block
        case("append_token", "append", "f32", 1, 32, 8, 128, 8000, ragged=False),
        # eight sequences of a serving batch, one token each, small pages
        case("append_batch", "append", "bf16", 8, 32, 8, 128, 8192, page=16, block=16),
        # the prompts of four requests, of odd lengths, are stored at once
        case("append_prompts", "append", "bf16", 4, 32, 8, 128, 8191, new=8191, page=64, block=64),
        # a short chat's next token on the small model: nothing but latency
        case("token_short", "attend", "f32", 1, 32, 8, 64, 129, page=16, block=16, ragged=False),
        # one sequence near the capacity of the 8B-shape model
        case("token_8k", "attend", "bf16", 1, 32, 8, 128, 8191, ragged=False),
        # a serving batch of the 8B-shape model over pages of 16, lengths as they come
        case("token_batch", "attend", "f32", 8, 32, 8, 128, 8192, page=16, block=16),
        # a wide batch of long sequences: as many bytes as a decode step reads in earnest
        case("token_wide", "attend", "bf16", 32, 32, 8, 128, 32768, page=256, block=64),
        # long streams that keep a window of 4096 and four first tokens
        case("token_window", "attend", "bf16", 16, 32, 4, 128, 65536, window=4096, sinks=4),
        # a prompt of 1024 tokens from nothing
        case("prompt_1k", "attend", "bf16", 1, 32, 8, 128, 1024, new=1024, ragged=False),
        # a long prompt from nothing: the largest contraction
        case("prompt_8k", "attend", "bf16", 1, 32, 8, 128, 8191, new=8191, page=16, block=16, ragged=False),
        # the next 64 tokens of two long documents, fp32 activations on the small model's heads
        case("chunk_32k", "attend", "f32", 2, 32, 8, 64, 32767, new=64),
        # prompts of odd lengths in one batch, window and sinks
        case("prompts_window", "attend", "bf16", 3, 24, 8, 128, 6000, new=6000, window=1000, sinks=20, block=32),
    ]


def draw(rng):
    def log(a, b):
        return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))
    op = rng.choice(["append", "attend", "attend", "attend", "attend"])
    prompt = rng.random() < 0.5
    dim = rng.choice([64, 128])
    kv_heads = rng.choice([1, 2, 3, 4, 8])
    heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 8])
    block = rng.choice([16, 32, 64, 128])
    page = block * rng.choice([1, 1, 2, 4])
    if prompt:
        rows, new = log(1, 6), log(2, 4000)
        length = new + (log(1, 8000) if rng.random() < 0.5 else 0)
        while rows * heads * new * length * dim > 32 * 8191 * 8191 * 128 // 4:
            rows, new = max(1, rows // 2), max(1, new * 2 // 3)
    else:
        rows, new, length = log(1, 48), 1, log(1, 50000)
        while rows * kv_heads * length * dim > 32 * 8 * 32768 * 128 // 2:
            rows, length = max(1, rows * 2 // 3), max(1, length * 2 // 3)
    windowed = rng.random() < 0.4
    return dict(op=op, dtype=rng.choice(["f32", "bf16"]), rows=rows, heads=heads, kv_heads=kv_heads, dim=dim,
                length=max(length, new), new=new, page=page, block=block, window=log(1, 5000) if windowed else 0,
                sinks=rng.choice([0, 1, 4, 33]) if windowed else 0, ragged=rng.random() < 0.7)


def lengths(c):
    """Of each row: (positions after the call, new tokens)."""
    got = []
    for r in range(c["rows"]):
        f = 1.0 - 0.7 * ((r * 0.6180339887) % 1.0) if c["ragged"] else 1.0
        n = max(1, int(c["new"] * f))
        got.append((max(n, int(c["length"] * f)), n))
    return got


def seen(c, p):
    """How many positions a token at position p sees."""
    if not c["window"]:
        return p + 1
    first = max(0, p + 1 - c["window"])
    return p + 1 - first + min(first, c["sinks"])


def work(c):
    rows = lengths(c)
    size = 4 if c["dtype"] == "f32" else 2
    total = sum(n for _, n in rows)
    kv = c["kv_heads"] * c["dim"]
    if c["op"] == "append":
        # the new K and V read, their bytes and the blocks' scales written
        scales = sum((l - 1) // c["block"] - (l - n) // c["block"] + 1 for l, n in rows) * c["kv_heads"]
        return {"bytes": 2 * (total * kv * (size + 1) + scales), "flops": 2 * total * kv}
    pairs, held = 0, 0
    for l, n in rows:
        w = c["window"]
        low = l - n + 1                      # positions seen by the first token of the row, if it sees all
        if not w:
            pairs += (low + l) * n // 2
            held += l
        else:
            pairs += sum(seen(c, p) for p in range(l - n, l))
            first = max(0, l - n + 1 - w)
            held += l - first + min(first, c["sinks"])
    return {"bytes": 2 * held * (kv + c["kv_heads"] / c["block"]) + 2 * total * c["heads"] * c["dim"] * size,
            "flops": 4 * pairs * c["heads"] * c["dim"]}


# ---- inputs ----

def stored(x, block):
    """(e4m3 bytes, scale bytes) of x [pages, heads, page, dim], one scale a block."""
    p, h, n, d = x.shape
    b = x.view(p, h, n // block, block * d)
    e = exponent(b.abs().amax(-1))
    q = (b * torch.exp2(-e.float())[..., None]).to(torch.float8_e4m3fn)
    return q.view(torch.uint8).view(p, h, n, d), (e + 127).to(torch.uint8)


def exponent(top):
    """The smallest exponent e with top <= 448 * 2^e, within the scales' range."""
    m, x = torch.frexp(top)
    return torch.where(top > 0, x - 9 + (m > 0.875).int(), LOW).clamp(LOW, HIGH)


def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    g = torch.Generator(dev).manual_seed(seed)
    rows = lengths(c)
    total = sum(n for _, n in rows)
    per_row = -(-max(l for l, _ in rows) // c["page"])
    pages = c["rows"] * per_row
    dt = torch.float32 if c["dtype"] == "f32" else torch.bfloat16

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    # a few channels of K are larger than the rest, as they are in trained models
    wide = 1.0 + 3.0 * (torch.rand(c["kv_heads"], 1, c["dim"], generator=g, device=dev) > 0.95)
    kb, ks = stored(normal(pages, c["kv_heads"], c["page"], c["dim"]) * wide, c["block"])
    vb, vs = stored(normal(pages, c["kv_heads"], c["page"], c["dim"]), c["block"])
    starts = [0]
    for _, n in rows:
        starts.append(starts[-1] + n)
    s = dict(case=c, k=kb, v=vb, k_scale=ks, v_scale=vs,
             table=torch.randperm(pages, generator=g, device=dev).view(c["rows"], per_row).int(),
             kv_len=torch.tensor([l for l, _ in rows], device=dev, dtype=torch.int32),
             q_start=torch.tensor(starts, device=dev, dtype=torch.int32), max_new=max(n for _, n in rows))
    if c["op"] == "append":
        s["new_k"] = (normal(total, c["kv_heads"], c["dim"]) * wide[:, 0] * 1.3).to(dt)
        s["new_v"] = normal(total, c["kv_heads"], c["dim"]).to(dt)
    else:
        s["q"] = normal(total, c["heads"], c["dim"]).to(dt)
        s["out"] = torch.empty_like(s["q"])
    if own:
        from graph_replay_gb300 import KV8Cache
        s["cache"] = KV8Cache(s["k"], s["v"], s["k_scale"], s["v_scale"], page_table=s["table"])
    return s


# ---- one pass ----

def run(state):
    s, c = state, state["case"]
    if own:
        starts = None if c["new"] == 1 else s["q_start"]
        if c["op"] == "append":
            s["cache"].append(s["new_k"], s["new_v"], s["kv_len"], q_start=starts, max_new=s["max_new"])
        else:
            return s["cache"].attend(s["q"], s["kv_len"], q_start=starts, max_new=s["max_new"], window=c["window"],
                                     sinks=c["sinks"], out=s["out"])
    elif c["op"] == "append":
        plain_append(s, s["new_k"], s["k"], s["k_scale"])
        plain_append(s, s["new_v"], s["v"], s["v_scale"])
    else:
        return plain_attend(s)
    return {"k": s["k"].view(torch.float8_e4m3fn), "k_scale": s["k_scale"].view(torch.float8_e8m0fnu),
            "v": s["v"].view(torch.float8_e4m3fn), "v_scale": s["v_scale"].view(torch.float8_e8m0fnu)}


def places(s):
    """Of each packed token: its row and its position."""
    total = s["q" if "q" in s else "new_k"].shape[0]
    t = torch.arange(total, device=s["k"].device)
    row = torch.searchsorted(s["q_start"][1:].long(), t, right=True)
    n = (s["q_start"][1:] - s["q_start"][:-1]).long()
    return row, s["kv_len"].long()[row] - n[row] + t - s["q_start"].long()[row]


def plain_append(s, x, store, scale):
    """x [tokens, heads, dim] into the cache: a block that new tokens enter takes the largest exponent that it needs;
    what it holds of earlier positions is rounded again where that grew."""
    c = s["case"]
    block, page, heads = c["block"], c["page"], c["kv_heads"]
    row, pos = places(s)
    where, inside, off = s["table"].long()[row, pos // page], pos % page // block, pos % block
    x = x.float()
    at = where * (page // block) + inside                         # the block of each token
    top = torch.zeros(store.shape[0] * (page // block), heads, device=x.device)
    e = exponent(top.scatter_reduce_(0, at[:, None].expand(-1, heads), x.abs().amax(-1), "amax"))
    # the block that a row's first token enters may hold earlier positions
    first = s["q_start"].long()[:-1]
    pg, b, n = where[first], inside[first], off[first]
    view = store.view(store.shape[0], heads, page // block, block, c["dim"])
    old, had = view[pg, :, b], scale[pg, :, b].int() - 127
    now = torch.where(n[:, None] > 0, torch.maximum(e[at[first]], had), e[at[first]])
    held = old.view(torch.float8_e4m3fn).float() * torch.exp2((had - now).float())[..., None, None]
    held = held.to(torch.float8_e4m3fn).view(torch.uint8)
    live = torch.arange(block, device=x.device)[None, :] < n[:, None]
    view[pg, :, b] = torch.where(live[:, None, :, None], held, old)
    e[at[first]] = now
    e = e[at]
    scale[where, :, inside] = (e + 127).to(torch.uint8)
    store[where, :, pos % page] = (x * torch.exp2(-e.float())[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)


def values(store, scale, table, block):
    """The fp32 values [rows, heads, positions, dim] that the pages of each row stand for."""
    p, h, n, d = store.shape
    x = store.view(torch.float8_e4m3fn).float().view(p, h, n // block, block * d)
    x = (x * torch.exp2(scale.float() - 127.0)[..., None]).view(p, h, n, d)
    return x[table.long()].transpose(1, 2).reshape(table.shape[0], h, -1, d)


def plain_attend(s):
    c = s["case"]
    rows, group, m = c["rows"], c["heads"] // c["kv_heads"], s["max_new"]
    k = values(s["k"], s["k_scale"], s["table"], c["block"])
    v = values(s["v"], s["v_scale"], s["table"], c["block"])
    row, pos = places(s)
    slot = torch.arange(row.numel(), device=row.device) - s["q_start"].long()[row]
    q = torch.zeros(rows, m, c["heads"], c["dim"], device=k.device)
    q[row, slot] = s["q"].float()
    at = torch.full((rows, m), -1, device=k.device)               # positions; -1 sees nothing
    at[row, slot] = pos
    q = q.view(rows, m, c["kv_heads"], group, c["dim"]).permute(0, 2, 1, 3, 4).reshape(rows, c["kv_heads"], m * group, -1)
    j = torch.arange(k.shape[2], device=k.device)
    see = j <= at[..., None]
    if c["window"]:
        see &= (j > at[..., None] - c["window"]) | (j < c["sinks"])
    x = (q @ k.transpose(2, 3)) * (1.0 / math.sqrt(c["dim"]))
    x = x.view(rows, c["kv_heads"], m, group, -1).masked_fill_(~see[:, None, :, None], float("-inf"))
    top = x.amax(-1, keepdim=True)
    x = x.sub_(torch.where(top > float("-inf"), top, 0.0)).exp_()
    x = x.div_(x.sum(-1, keepdim=True).clamp_min(1e-30))
    o = (x.view(rows, c["kv_heads"], m * group, -1) @ v).view(rows, c["kv_heads"], m, group, c["dim"])
    o = o.permute(0, 2, 1, 3, 4).reshape(rows, m, c["heads"], c["dim"])
    s["out"].copy_(o[row, slot])
    return s["out"]


# ---- the definition in 64 bits ----

def exact(case, seed):
    c = case
    s = prepare(case, seed)
    rows, group, out = lengths(c), c["heads"] // c["kv_heads"], []
    if c["op"] == "append":
        # one block at a time, from the definition; where that is too many blocks, nothing is said
        if sum(n for _, n in rows) * c["kv_heads"] > 4096:
            return None
        got = {}
        for name in "kv":
            store = s[name].view(torch.float8_e4m3fn).double().cpu()
            scale = s[name + "_scale"].cpu()
            new, table = s["new_" + name].double().cpu(), s["table"].cpu().tolist()
            scale, t = scale.clone(), 0
            for r, (l, n) in enumerate(rows):
                for h in range(c["kv_heads"]):
                    for b in range((l - n) // c["block"], (l - 1) // c["block"] + 1):
                        lo, hi = max(l - n, b * c["block"]), min(l, (b + 1) * c["block"])
                        x = new[t + lo - (l - n):t + hi - (l - n), h]
                        top = float(x.abs().max())
                        e = LOW if top == 0 else min(HIGH, max(LOW, math.ceil(math.log2(top / 448.0))))
                        at, off = table[r][b * c["block"] // c["page"]], b * c["block"] % c["page"]
                        was = int(scale[at, h, off // c["block"]]) - 127
                        keep = lo - b * c["block"]
                        e = max(e, was) if keep else e
                        held = store[at, h, off:off + keep] * 2.0 ** (was - e)
                        store[at, h, off:off + keep] = rounded(held)
                        store[at, h, off + keep:off + keep + hi - lo] = rounded(x * 2.0 ** -e)
                        scale[at, h, off // c["block"]] = e + 127
                t += n
            got[name], got[name + "_scale"] = store, torch.exp2(scale.double() - 127.0)
        return got
    if work(c)["flops"] > 4e12:
        return None
    k, v = s["k"].view(torch.float8_e4m3fn), s["v"].view(torch.float8_e4m3fn)
    ks, vs = s["k_scale"].double() - 127.0, s["v_scale"].double() - 127.0
    res = torch.zeros(s["q"].shape, dtype=torch.float64, device=k.device)
    t = 0
    for r, (l, n) in enumerate(rows):
        at = s["table"][r].long()
        j = torch.arange(l, device=k.device)
        p = torch.arange(l - n, l, device=k.device)[:, None]
        hide = j[None] > p
        if c["window"]:
            hide |= (j[None] <= p - c["window"]) & (j[None] >= c["sinks"])
        for h in range(c["kv_heads"]):
            kk = (k[at, h].double() * torch.exp2(ks[at, h]).repeat_interleave(c["block"], 1)[..., None]).flatten(0, 1)[:l]
            vv = (v[at, h].double() * torch.exp2(vs[at, h]).repeat_interleave(c["block"], 1)[..., None]).flatten(0, 1)[:l]
            for a in range(h * group, (h + 1) * group):
                x = (s["q"][t:t + n, a].double() @ kk.T) / math.sqrt(c["dim"])
                res[t:t + n, a] = torch.softmax(x.masked_fill(hide, -math.inf), -1) @ vv
        t += n
    return res


def rounded(x):
    """x (64 bits) to the nearest e4m3 value, ties to even, from the format's definition: 3 bits behind the point, least exponent -6."""
    _, e = torch.frexp(x)
    step = torch.exp2((e - 1).clamp_min(-6).double() - 3.0)
    return torch.round(x / step) * step
