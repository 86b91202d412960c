"""What is measured of the operators of a verify pass: a target layer's attention over a cache held in 4 bits.

After `dspark_assemble` the target model runs the admitted tokens of every request through its layers. In each
layer the queries and keys are normed by head and rotated (`qk_norm_rope`), the keys and values go into a paged
cache of 4-bit codes (`cache_append`; `cache_read` gives back the values), and the queries attend over the cache
(`cache_attend`), some models with a sliding window and a few first tokens that stay visible. A case of `op`
"pass" runs them together as one layer does.

The cache: pool[page][kv head][block], a block being, for `page` tokens of D channels, the K codes [page][D/2],
the V codes [page][D/2], the K scales [page][D/32] and the V scales [page/16][D/32][16]. Two channels share a byte,
the even one in the low half; a code of u stands for (u - 8) * scale. A scale serves 32 channels: their largest
magnitude over 7, rounded to 8 significant bits (as bf16 does) and held in fp16, 9344 at most, so that a code times
its scale is exact in fp16.
"""
import math

import torch

own = False

GROUP = 32
SCRATCH = 64 << 20     # what a program keeps as workspace for every call

# (query heads, kv heads) and head widths
HEADS = ((4, 1), (8, 8), (12, 3), (16, 4), (16, 2), (32, 8), (32, 4), (40, 8))


def listed():
    return [
        # queries and keys of a draft round's smallest verify batch (4 requests, 4 drafts and the anchor), fp32
        {"name": "rope tiny", "op": "rope", "T": 20, "Hq": 16, "Hkv": 4, "D": 64, "rot": 64, "inter": False,
         "dtype": "f32", "far": 4096},
        # the verify batch of 128 requests with 16 drafts each
        {"name": "rope verify", "op": "rope", "T": 2176, "Hq": 32, "Hkv": 8, "D": 128, "rot": 128, "inter": False,
         "dtype": "bf16", "far": 4096},
        # a long prompt at far positions, half of each head rotated, neighbouring channels paired
        {"name": "rope prompt", "op": "rope", "T": 32749, "Hq": 32, "Hkv": 8, "D": 128, "rot": 64, "inter": True,
         "dtype": "bf16", "far": 1 << 20},
        # keys and values of the 128-request verify batch into the cache, and read back
        {"name": "append verify", "op": "append", "T": 2176, "R": 128, "Hkv": 8, "D": 128, "page": 64,
         "dtype": "bf16"},
        # a prompt's keys and values into the cache in fp32, odd length, small pages
        {"name": "append prompt", "op": "append", "T": 49999, "R": 3, "Hkv": 4, "D": 64, "page": 16, "dtype": "f32"},
        # the smallest attention: 4 requests, 5 queries each, a short context, fp32
        {"name": "attend tiny", "op": "attend", "R": 4, "Q": 5, "ctx_lo": 100, "ctx_hi": 512, "Hq": 16, "Hkv": 4,
         "D": 64, "page": 16, "window": 0, "sinks": 0, "dtype": "f32"},
        # one token a request: plain decoding beside the draft rounds
        {"name": "attend decode", "op": "attend", "R": 128, "Q": 1, "ctx_lo": 512, "ctx_hi": 4096, "Hq": 32,
         "Hkv": 8, "D": 128, "page": 64, "window": 0, "sinks": 0, "dtype": "bf16"},
        # one token of few requests over a long context: the long axis has to be split
        {"name": "attend long", "op": "attend", "R": 2, "Q": 1, "ctx_lo": 120001, "ctx_hi": 131072, "Hq": 32,
         "Hkv": 4, "D": 128, "page": 64, "window": 0, "sinks": 0, "dtype": "bf16"},
        # the round's verify batch: up to 16 admitted drafts and the anchor a request, ragged
        {"name": "attend verify", "op": "attend", "R": 128, "Q": 17, "ctx_lo": 512, "ctx_hi": 4096, "Hq": 32,
         "Hkv": 8, "D": 128, "page": 64, "window": 0, "sinks": 0, "dtype": "bf16"},
        # a windowed layer's verify batch over longer contexts, small pages
        {"name": "attend window", "op": "attend", "R": 64, "Q": 9, "ctx_lo": 2000, "ctx_hi": 16384, "Hq": 16,
         "Hkv": 8, "D": 128, "page": 16, "window": 1024, "sinks": 4, "dtype": "bf16"},
        # a chunk of two prompts over what came before
        {"name": "attend prompt", "op": "attend", "R": 2, "Q": 2048, "ctx_lo": 1, "ctx_hi": 4096, "Hq": 32,
         "Hkv": 8, "D": 128, "page": 64, "window": 0, "sinks": 0, "dtype": "bf16"},
        # a layer's whole attention for a verify batch of 32 requests
        {"name": "pass verify", "op": "pass", "R": 32, "Q": 17, "ctx_lo": 512, "ctx_hi": 2048, "Hq": 32, "Hkv": 8,
         "D": 128, "rot": 128, "inter": False, "page": 32, "window": 0, "sinks": 0, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(("rope", "append", "attend", "attend", "attend", "pass"))
    Hq, Hkv = rng.choice(HEADS)
    D = rng.choice((64, 128))
    dtype = "f32" if rng.random() < 0.25 else "bf16"
    if op == "rope":
        D = rng.choice((32, 64, 96, 128, 256))
        T = _log(rng, 1, 32749 * 40 * 128 // ((Hq + Hkv) * D * (2 if dtype == "f32" else 1)))
        return {"op": op, "T": min(T, 40000), "Hq": Hq, "Hkv": Hkv, "D": D, "rot": rng.choice((D, D // 2)),
                "inter": rng.random() < 0.5, "dtype": dtype, "far": _log(rng, 64, 1 << 20)}
    page = rng.choice((16, 32, 64, 128))
    if op == "append":
        D = rng.choice((32, 64, 96, 128, 256))
        T = min(60000, _log(rng, 1, 49999 * 4 * 64 * 4 // (Hkv * D * (4 if dtype == "f32" else 2))))
        return {"op": op, "T": T, "R": min(T, rng.choice((1, 3, 32, 128))), "Hkv": Hkv, "D": D, "page": page,
                "dtype": dtype}
    if dtype == "f32":
        R, Q, hi = _log(rng, 1, 8), rng.choice((1, 2, 5, 9)), _log(rng, 16, 2048)
    else:
        R = _log(rng, 1, 128)
        Q = rng.choice((1, 1, 2, 5, 9, 17))
        if rng.random() < 0.15:
            R, Q = rng.randint(1, 2), rng.randint(64, 1500)
        # at most the work of the 128-request verify batch and the 16384-token windowed one, in keys and in scores
        most = min(128 * 4096 * 8 // (R * Hkv), 128 * 17 * 32 * 4096 // (R * Q * Hq), 65536)
        hi = _log(rng, 16, max(64, most))
    windowed = rng.random() < 0.4
    case = {"op": op, "R": R, "Q": Q, "ctx_lo": max(1, hi // 8), "ctx_hi": hi, "Hq": Hq, "Hkv": Hkv, "D": D,
            "page": page, "window": _log(rng, 16, 2048) if windowed else 0,
            "sinks": rng.randint(0, 20) if windowed else 0, "dtype": dtype}
    if op == "pass":
        case.update(rot=rng.choice((D, D // 2)), inter=rng.random() < 0.5)
    return case


def _type(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def _tokens(case):
    return case["T"] if "T" in case else case["R"] * case["Q"]


def _frequencies(rot, base=10000.0):
    """Turns a position of each pair, in units of 2^-64."""
    return torch.tensor([int(base ** (-2.0 * i / rot) / (2.0 * math.pi) * 2.0 ** 64) for i in range(rot // 2)],
                        dtype=torch.int64, device="cuda")


def _scale(top):
    return (top / 7).bfloat16().float().clamp(max=9344.0).half()


def _pool(gen, pages, Hkv, page, D):
    """A cache that normal keys and values were written to."""
    codes = page * D // 2
    scales = page * D // GROUP * 2
    pool = torch.empty((pages, Hkv, 2 * (codes + scales)), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 26) // (Hkv * page * D))
    for p in range(0, pages, step):
        n = min(step, pages - p)
        for half in range(2):
            x = torch.randn((n, Hkv, page, D // GROUP, GROUP), device="cuda", generator=gen)
            s = _scale(x.abs().amax(-1, keepdim=True))
            u = (torch.round(x / s.float()).clamp(-7, 7) + 8).to(torch.uint8).view(n, Hkv, page, D // 2, 2)
            pool[p:p + n, :, half * codes:(half + 1) * codes] = (u[..., 0] | (u[..., 1] << 4)).reshape(n, Hkv, codes)
            s = s.squeeze(-1) if half == 0 else s.squeeze(-1).unflatten(2, (-1, 16)).transpose(3, 4)
            pool[p:p + n, :, 2 * codes + half * scales:2 * codes + (half + 1) * scales] = \
                s.contiguous().view(torch.uint8).reshape(n, Hkv, scales)
    return pool


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    host = torch.Generator()
    host.manual_seed(seed)
    op, dt, T, Hkv, D = case["op"], _type(case), _tokens(case), case["Hkv"], case["D"]
    Hq = case.get("Hq", 0)
    s = {"case": dict(case), "workspace": torch.zeros(SCRATCH, dtype=torch.uint8, device="cuda")}
    # one projection's rows: the heads of the queries, the keys and the values beside one another
    qkv = torch.randn((T, (Hq + 2 * Hkv) * D), device="cuda", generator=gen).to(dt)
    s["q"] = qkv[:, :Hq * D].view(T, Hq, D)
    s["k"] = qkv[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D)
    s["v"] = qkv[:, (Hq + Hkv) * D:].view(T, Hkv, D)
    if op in ("rope", "pass"):
        s["freq"] = _frequencies(case["rot"])
        s["q_gain"] = 1 + 0.1 * torch.randn(D, device="cuda", generator=gen)
        s["k_gain"] = 1 + 0.1 * torch.randn(D, device="cuda", generator=gen)
        s["rope_out"] = {"q": torch.empty((T, Hq, D), dtype=dt, device="cuda"),
                         "k": torch.empty((T, Hkv, D), dtype=dt, device="cuda")}
    if op == "rope":
        s["position"] = torch.randint(0, case["far"], (T,), generator=host).to(torch.int32).cuda()
        return s
    R = case["R"]
    if op == "append":
        # the tokens of each request in a run, after a context of its own
        each = torch.full((R,), T // R, dtype=torch.int64)
        each[:T % R] += 1
        ctx = torch.randint(0, 200, (R,), generator=host)
        most = 200 + int(each.max())
    else:
        Q = case["Q"]
        each = torch.randint(1, Q + 1, (R,), generator=host) if 1 < Q <= 33 else torch.full((R,), Q, dtype=torch.int64)
        ctx = torch.randint(case["ctx_lo"], case["ctx_hi"] + 1, (R,), generator=host)
        most = case["ctx_hi"] + Q
    page = case["page"]
    width = -(-most // page)
    need = (ctx + each + page - 1) // page
    table = torch.randperm(R * width, generator=host).view(R, width).to(torch.int32)
    table[torch.arange(width)[None, :] >= need[:, None]] = -1
    request = torch.full((T,), -1, dtype=torch.int64)
    position = torch.full((T,), -1, dtype=torch.int64)
    total = int(each.sum())
    start = torch.cumsum(each, 0) - each
    request[:total] = torch.repeat_interleave(torch.arange(R), each)
    position[:total] = torch.arange(total) - start[request[:total]]
    for name, t in (("table", table), ("ctx_len", ctx), ("request", request), ("position", position),
                    ("offsets", torch.cat([start, torch.tensor([total])]))):
        s[name] = t.to(torch.int32).cuda()
    s["pool"] = _pool(gen, R * width, Hkv, page, D)
    if op in ("append", "pass"):
        s["read_out"] = {n: torch.empty((T, Hkv, D), dtype=dt, device="cuda") for n in ("k", "v")}
    if op in ("attend", "pass"):
        s["attend_out"] = {"out": torch.empty((T, Hq, D), dtype=dt, device="cuda"),
                           "lse": torch.empty((T, Hq), dtype=torch.float32, device="cuda")}
    return s


# ------------------------------------------------------------------ the plain forms

def _rotated(x, gain, position, freq, inter, eps=1e-6):
    f = x.float()
    y = f * torch.rsqrt(f.square().mean(-1, keepdim=True) + eps) * gain
    turns = torch.frac(position.double()[:, None] * (freq.double() * 2.0 ** -64))   # far positions: 64 bits
    angle = turns * (2.0 * math.pi)
    c, s = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    rot = 2 * freq.numel()
    a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if inter else (y[..., :rot // 2], y[..., rot // 2:rot])
    p, q = a * c - b * s, a * s + b * c
    turned = torch.stack((p, q), -1).flatten(-2) if inter else torch.cat((p, q), -1)
    return torch.cat((turned, y[..., rot:]), -1).to(x.dtype)


def _rope(s):
    case = s["case"]
    position = s["position"]
    if "request" in s:
        position = torch.where(s["request"] < 0, 0, position + s["ctx_len"][s["request"].long().clamp(min=0)])
    return tuple(_rotated(s[n], s[n + "_gain"], position, s["freq"], case["inter"]) for n in ("q", "k"))


def _parts(blocks, D):
    """The four parts of cache blocks [..., block]: K and V codes [..., page, D/2] and scales [..., page, D/32]."""
    page = blocks.shape[-1] * 8 // (9 * D)
    lead = blocks.shape[:-1]
    codes, scales = page * D // 2, page * D // GROUP * 2
    kc, vc, ks, vs = torch.split(blocks, [codes, codes, scales, scales], -1)
    return (kc.reshape(*lead, page, D // 2), vc.reshape(*lead, page, D // 2),
            ks.contiguous().view(torch.float16).view(*lead, page, D // GROUP),
            vs.contiguous().view(torch.float16).view(*lead, -1, D // GROUP, 16).transpose(-1, -2).flatten(-3, -2))


def _values(codes, scales):
    u = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).float() - 8
    return (u.unflatten(-1, (-1, GROUP)) * scales.float()[..., None]).flatten(-2)


def _packed(x):
    """The codes [..., D/2] and scales [..., D/32] of rows x; codes in 64 bits, where a value is next to a border."""
    g = x.float().unflatten(-1, (-1, GROUP))
    s = _scale(g.abs().amax(-1))
    u = torch.round(g.double() / s.double()[..., None]).nan_to_num(0.0).clamp(-7, 7) + 8
    u = u.to(torch.uint8).flatten(-2).unflatten(-1, (-1, 2))
    return u[..., 0] | (u[..., 1] << 4), s


def _append(s, k, v):
    case, pool = s["case"], s["pool"]
    D, page = case["D"], case["page"]
    live = torch.nonzero(s["request"] >= 0).squeeze(-1)
    request = s["request"][live].long()
    at = s["ctx_len"][request].long() + s["position"][live].long()
    block, slot = s["table"][request, at // page].long(), at % page
    codes, scales = page * D // 2, page * D // GROUP * 2
    pages, Hkv = pool.shape[:2]
    for half, x in enumerate((k, v)):
        c, sc = _packed(x[live])
        pool[..., half * codes:(half + 1) * codes].unflatten(-1, (page, D // 2))[block, :, slot] = c
        part = pool[..., 2 * codes + half * scales:2 * codes + (half + 1) * scales]
        b = sc.contiguous().view(torch.uint8).unflatten(-1, (-1, 2))
        if half == 0:
            part.unflatten(-1, (page, D // GROUP, 2))[block, :, slot] = b
        else:
            part.unflatten(-1, (page // 16, D // GROUP, 16, 2))[block, :, slot // 16, :, slot % 16] = b
    kc, vc, ks, vs = _parts(pool[block], D)
    n = torch.arange(live.numel(), device=live.device)
    out = []
    for c, sc in ((kc, ks), (vc, vs)):
        y = torch.zeros(k.shape, dtype=k.dtype, device=k.device)
        y[live] = _values(c[n, :, slot], sc[n, :, slot]).to(k.dtype)
        out.append(y)
    return out


def _attend(s, q):
    case = s["case"]
    D, G, Q, Hkv = case["D"], case["Hq"] // case["Hkv"], case["Q"], case["Hkv"]
    ctx, offsets = s["ctx_len"].long(), s["offsets"].long()
    R, T = ctx.numel(), q.shape[0]
    kc, vc, ks, vs = _parts(s["pool"][s["table"].long().clamp(min=0)], D)          # [R][width][Hkv][page][..]
    k = _values(kc, ks).transpose(1, 2).flatten(2, 3)                               # [R][Hkv][L][D]
    v = _values(vc, vs).transpose(1, 2).flatten(2, 3)
    each = offsets[1:] - offsets[:-1]
    j = torch.arange(Q, device=q.device)
    row = (offsets[:-1, None] + j).clamp(max=T - 1)                                 # [R][Q]
    x = q.float()[row].unflatten(2, (Hkv, G)).permute(0, 2, 1, 3, 4).flatten(2, 3)  # [R][Hkv][Q*G][D]
    z = torch.matmul(x, k.transpose(-1, -2)).unflatten(2, (Q, G)) * (1.0 / math.sqrt(D))
    here = (ctx[:, None] + j)[:, :, None]                                           # [R][Q][1]
    key = torch.arange(k.shape[2], device=q.device)
    seen = key <= here
    if case["window"]:
        seen = seen & ((key > here - case["window"]) | (key < case["sinks"]))
    z = z.masked_fill(~seen[:, None, :, None, :], -math.inf)
    top = z.amax(-1, keepdim=True)
    e = torch.exp(z - top)
    total = e.sum(-1, keepdim=True)
    o = torch.matmul((e / total).flatten(2, 3), v).unflatten(2, (Q, G))             # [R][Hkv][Q][G][D]
    lse = (top + torch.log(total)).squeeze(-1)
    real = j < each[:, None]
    out = torch.zeros(q.shape, dtype=q.dtype, device=q.device)
    l_out = torch.full(q.shape[:2], -math.inf, device=q.device)
    out[row[real]] = o.permute(0, 2, 1, 3, 4).flatten(2, 3)[real].to(q.dtype)
    l_out[row[real]] = lse.permute(0, 2, 1, 3).flatten(2, 3)[real]
    return out, l_out


def _run_plain(s):
    op = s["case"]["op"]
    if op == "rope":
        q, k = _rope(s)
        return {"q": q, "k": k}
    if op == "append":
        k, v = _append(s, s["k"], s["v"])
        return {"k": k, "v": v}
    if op == "attend":
        out, lse = _attend(s, s["q"])
        return {"out": out, "lse": lse}
    q, k = _rope(s)
    k, v = _append(s, k, s["v"])
    out, lse = _attend(s, q)
    return {"out": out, "lse": lse, "k": k, "v": v}


# ------------------------------------------------------------------ the framework's calls

def _run_own(s):
    import speculative_decoding_draft_round_gb300 as ds

    case, ws = s["case"], s["workspace"]
    op, got = case["op"], {}
    q, k = s["q"], s["k"]
    if op in ("rope", "pass"):
        got = ds.qk_norm_rope(q, k, s["freq"], s["position"], request=s.get("request"), ctx_len=s.get("ctx_len"),
                              q_gain=s["q_gain"], k_gain=s["k_gain"], eps=1e-6, interleaved=case["inter"],
                              out=s["rope_out"], workspace=ws)
        q, k = got["q"], got["k"]
        if op == "rope":
            return {"q": q, "k": k}
    where = (s["pool"], s["table"])
    if op in ("append", "pass"):
        ds.cache_append(k, s["v"], *where, s["request"], s["position"], s["ctx_len"], workspace=ws)
        got = ds.cache_read(*where, s["request"], s["position"], s["ctx_len"], D=case["D"], dtype=_type(case),
                            out=s["read_out"], workspace=ws)
        if op == "append":
            return {"k": got["k"], "v": got["v"]}
    att = ds.cache_attend(q, *where, s["offsets"], s["ctx_len"], window=case["window"], sinks=case["sinks"],
                          max_q=case["Q"], out=s["attend_out"], workspace=ws)
    if op == "attend":
        return {"out": att["out"], "lse": att["lse"]}
    return {"out": att["out"], "lse": att["lse"], "k": got["k"], "v": got["v"]}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    op, D, Hkv, T = case["op"], case["D"], case["Hkv"], _tokens(case)
    Hq = case.get("Hq", 0)
    row = D * 9 // 16                       # a cached row: codes and scales
    bytes_ = flops = 0
    if op == "pass" or op == "attend":
        each = (case["Q"] + 1) / 2 if 1 < case["Q"] <= 33 else case["Q"]
        live = case["R"] * each
    else:
        live = T
    if op in ("rope", "pass"):
        bytes_ += live * (Hq + Hkv) * D * size * 2 + live * 4
        flops += live * (Hq + Hkv) * D * 8
    if op in ("append", "pass"):
        # k (v) in, codes out; codes in, values out
        bytes_ += live * Hkv * 2 * (D * size + row + row + D * size)
        flops += live * Hkv * 2 * D * 6
    if op in ("attend", "pass"):
        ctx = (case["ctx_lo"] + case["ctx_hi"]) / 2
        reach = ctx + (each + 1) / 2        # keys that a query sees, on average
        keys = ctx + each
        if case["window"]:
            keys = min(keys, case["window"] + each + case["sinks"])
            reach = min(reach, case["window"] + case["sinks"])
        bytes_ += case["R"] * keys * Hkv * 2 * row + live * Hq * D * size * 2
        flops += live * Hq * reach * D * 4
    return {"bytes": bytes_, "flops": flops}


# ------------------------------------------------------------------ in 64 bits

def _exact_turn(x, gain, at, freq, inter):
    x = x.double()
    D, rot = x.shape[-1], 2 * freq.numel()
    y = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / D + 1e-6) * gain.double()
    step = [int(f) for f in freq.tolist()]
    # whole turns leave by integer arithmetic: 32 bits of a turn's fraction at a time
    hi = torch.tensor([f >> 32 for f in step], dtype=torch.int64, device=x.device)
    lo = torch.tensor([f & 0xFFFFFFFF for f in step], dtype=torch.int64, device=x.device)
    p = at.long()[:, None]
    whole = ((p * hi) & 0xFFFFFFFF).double() * 2.0 ** -32 + (p * lo).double() * 2.0 ** -64
    z = torch.polar(torch.ones_like(whole), whole * (2 * math.pi))[:, None]
    first = torch.arange(0, rot, 2, device=x.device) if inter else torch.arange(0, rot // 2, device=x.device)
    second = first + 1 if inter else first + rot // 2
    w = torch.complex(y[..., first], y[..., second]) * z
    y[..., first], y[..., second] = w.real, w.imag
    return y


def _exact_stored(x, dt):
    """What the cache holds of rows x of its own type."""
    x = x.to(dt).double()
    rows = x.reshape(-1, GROUP)
    step = torch.clamp((rows.abs().max(1).values.float() / 7).to(torch.bfloat16).double(), max=9344.0)
    step = step.half().double()[:, None]
    count = torch.where(step > 0, rows / step, torch.zeros_like(rows))
    return (count.round().clamp(-7, 7) * step).reshape(x.shape)


def exact(case, seed):
    s = prepare(case, seed)
    op, dt, D, Hkv = case["op"], _type(case), case["D"], case["Hkv"]
    q, k = s["q"].double(), s["k"].double()
    live = s["request"] >= 0 if "request" in s else None
    if op in ("rope", "pass"):
        at = s["position"].long()
        if live is not None:
            at = torch.where(live, at + s["ctx_len"].long()[s["request"].long().clamp(min=0)], torch.zeros_like(at))
        q = _exact_turn(s["q"], s["q_gain"], at, s["freq"], case["inter"])
        k = _exact_turn(s["k"], s["k_gain"], at, s["freq"], case["inter"])
        if op == "rope":
            return {"q": q, "k": k}
        q = q.to(dt).double()               # what one call leaves to the next has the cache's type
    if op in ("append", "pass"):
        k = _exact_stored(k, dt) * live[:, None, None]
        v = _exact_stored(s["v"], dt) * live[:, None, None]
        if op == "append":
            return {"k": k, "v": v}
    page, G = case["page"], case["Hq"] // case["Hkv"]
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=q.device)
    offsets, ctx, table = s["offsets"].tolist(), s["ctx_len"].tolist(), s["table"].long()
    cb, sb, ng = page * D // 2, page * D // 16, D // GROUP
    for r in range(case["R"]):
        a, b = offsets[r], offsets[r + 1]
        n = ctx[r] + b - a
        blocks = s["pool"][table[r, :-(-n // page)]]                       # [pages][Hkv][block]
        got = []
        for half in range(2):
            u = blocks[:, :, half * cb:(half + 1) * cb].reshape(-1, Hkv, page, D // 2).long()
            c = torch.empty((*u.shape[:3], D), dtype=torch.float64, device=q.device)
            c[..., 0::2], c[..., 1::2] = (u % 16 - 8).double(), (u // 16 - 8).double()
            w = blocks[:, :, 2 * cb + half * sb:2 * cb + (half + 1) * sb].contiguous().view(torch.float16).double()
            if half:
                w = w.view(-1, Hkv, page // 16, ng, 16).mT
            w = w.reshape(-1, Hkv, page, ng)
            c = c * w.repeat_interleave(GROUP, -1)
            c = c.permute(1, 0, 2, 3).reshape(Hkv, -1, D)[:, :n].clone()
            if op == "pass":                                               # this batch's rows are written by the pass
                c[:, ctx[r]:] = (k if half == 0 else v)[a:b].permute(1, 0, 2)
            got.append(c)
        i = torch.arange(n, device=q.device)
        for lo in range(a, b, 256):
            hi = min(b, lo + 256)
            p = (ctx[r] + torch.arange(lo - a, hi - a, device=q.device))[:, None]
            hide = i > p
            if case["window"]:
                hide = hide | ((i <= p - case["window"]) & (i >= case["sinks"]))
            z = torch.einsum("thgd,hkd->thgk", q[lo:hi].view(hi - lo, Hkv, G, D), got[0]) / math.sqrt(D)
            z = z.masked_fill(hide[:, None, None, :], -math.inf)
            lse[lo:hi] = torch.logsumexp(z, -1).view(hi - lo, -1)
            out[lo:hi] = torch.einsum("thgk,hkd->thgd", torch.softmax(z, -1), got[1]).reshape(hi - lo, -1, D)
    return {"out": out, "lse": lse, "k": k, "v": v} if op == "pass" else {"out": out, "lse": lse}
