"""What is measured of the target's pass beside its attention: norms, projections in 8 bits and the logits' adjustment.

Before and after `cache_attend` a target layer adds the residual, norms the rows and quantises them (`add_norm_quant`),
and multiplies them with weights held in 8 bits (`linear_i8`); so does the head that gives the logits. Between the
logits and `dspark_verify` stand the penalties for tokens a request has seen, its biases and its grammar's mask
(`adjust_logits`), for which a table of counts is kept (`seen_add`). A case of `op` "pass" runs the end of a target's
pass: norm, head, and the adjustment of its logits in place.

The table: int16 [R][V rounded up to 8], bit 15 for a token of the prompt, the low 15 bits the times that the request
has put it out. A mask's bit v % 32 of word v / 32 says that token v may follow.
"""
import math

import torch

own = False

SCRATCH = 256 << 20    # what a program keeps as workspace for every call, but for weights of odd widths


def listed():
    return [
        # a layer's norm for the verify batch of 128 requests with 16 drafts each
        {"name": "norm verify", "op": "norm", "T": 2176, "N": 4096, "dtype": "bf16", "residual": True, "norm": True,
         "codes": True},
        # a prompt's rows of odd number, normed for a projection that is not in 8 bits
        {"name": "norm prompt", "op": "norm", "T": 32749, "N": 5120, "dtype": "bf16", "residual": True, "norm": True,
         "codes": False},
        # 16 requests of one token: the weights are all there is to read
        {"name": "linear decode", "op": "linear", "T": 16, "K": 4096, "N": 6144, "dtype": "bf16"},
        # the queries, keys and values of the 128-request verify batch
        {"name": "linear verify", "op": "linear", "T": 2176, "K": 4096, "N": 6144, "dtype": "bf16"},
        # odd sizes, fp32: rows of weights that begin on no boundary
        {"name": "linear odd", "op": "linear", "T": 333, "K": 1001, "N": 1537, "dtype": "f32"},
        # the logits of 128 requests, one row each
        {"name": "linear head", "op": "linear", "T": 128, "K": 4096, "N": 151936, "dtype": "bf16"},
        # a chunk of prompts through a wide projection
        {"name": "linear prompt", "op": "linear", "T": 6007, "K": 8192, "N": 8192, "dtype": "bf16"},
        # four new requests, short prompts, small vocabulary
        {"name": "seen few", "op": "seen", "R": 4, "W": 300, "G": 4, "V": 1003},
        # 128 new requests with prompts of up to 4096 tokens
        {"name": "seen prompt", "op": "seen", "R": 128, "W": 4096, "G": 16, "V": 151936},
        # the smallest round's logits, odd vocabulary, fp32
        {"name": "adjust tiny", "op": "adjust", "R": 4, "S": 5, "V": 1003, "dtype": "f32"},
        # the target's logits of the 128-request verify batch
        {"name": "adjust verify", "op": "adjust", "R": 128, "S": 17, "V": 151936, "dtype": "bf16"},
        # the end of a target's pass for the verify batch of 32 requests
        {"name": "pass verify", "op": "pass", "R": 32, "S": 17, "K": 4096, "V": 151936, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def _width(rng, lo, hi, unit):
    """A size whose logarithm is uniform, mostly a multiple of `unit`."""
    n = _log(rng, lo, hi)
    return max(unit, n // unit * unit) if rng.random() < 0.75 else n


def draw(rng):
    op = rng.choice(("norm", "norm", "linear", "linear", "linear", "seen", "adjust", "adjust", "pass"))
    dtype = "f32" if rng.random() < 0.25 else "bf16"
    if op == "norm":
        N = _width(rng, 32, 16384, 8)
        T = _log(rng, 1, min(100000, 32749 * 5120 // (N * (2 if dtype == "f32" else 1))))
        return {"op": op, "T": T, "N": N, "dtype": dtype, "residual": rng.random() < 0.7, "norm": rng.random() < 0.8,
                "codes": rng.random() < 0.7}
    if op == "linear":
        K, T = _width(rng, 64, 12288, 64), _log(rng, 1, 8192)
        most = min(200000, 6007 * 8192 * 8192 // (T * K), 128 * 4096 * 151936 // (T * K) * 8, 151936 * 4096 // K,
                   2176 * 151936 // T)
        return {"op": op, "T": T, "K": K, "N": _width(rng, 64, max(64, most), 64), "dtype": dtype}
    V = _width(rng, 300, 200000, 8)
    if op == "seen":
        R = _log(rng, 1, min(512, max(1, 128 * 151936 // V)))
        return {"op": op, "R": R, "W": _log(rng, 1, min(32768, 128 * 4096 // R)), "G": rng.randint(1, 32), "V": V}
    if op == "adjust":
        S = rng.choice((1, 1, 2, 5, 9, 17, 33))
        R = _log(rng, 1, min(256, max(1, 128 * 17 * 151936 // (V * S * (2 if dtype == "f32" else 1)))))
        return {"op": op, "R": R, "S": S, "V": V, "dtype": dtype}
    K, S = 64 * rng.randint(4, 64), rng.choice((1, 2, 5, 9, 17))
    R = _log(rng, 1, max(1, min(64, 32 * 17 * 151936 * 4096 // (V * K * S), 32 * 17 * 151936 // (V * S))))
    return {"op": op, "R": R, "S": S, "K": K, "V": V, "dtype": "bf16"}


def _type(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def _codes(gen, rows, cols):
    """Rows of normal values in 8 bits, and their scales."""
    codes = torch.empty((rows, cols), dtype=torch.int8, device="cuda")
    scale = torch.empty(rows, device="cuda")
    step = max(1, (1 << 26) // cols)
    for a in range(0, rows, step):
        x = torch.randn((min(step, rows - a), cols), device="cuda", generator=gen)
        top = x.abs().amax(1)
        codes[a:a + step] = torch.round(x * (127 / top)[:, None]).to(torch.int8)
        scale[a:a + step] = top / 127
    return codes, scale


def _ids(gen, shape, V):
    """Tokens as text has them: few of them often, most of them seldom."""
    u = torch.rand(shape, device="cuda", generator=gen, dtype=torch.float64)
    return (torch.exp(u * math.log(V + 1.0)) - 1).long().clamp(0, V - 1)


def _counts(tokens, n, V):
    """[R][V] times that each id is among the first n[r] of row r of tokens (int32)."""
    R, W = tokens.shape
    live = torch.arange(W, device="cuda") < n[:, None]
    out = torch.zeros((R, V), dtype=torch.int32, device="cuda")
    return out.scatter_add_(1, tokens.long().clamp(0, V - 1), live.int())


def _table(prompt, out):
    R, V = prompt.shape
    t = torch.zeros((R, -(-V // 8) * 8), dtype=torch.int16, device="cuda")
    t[:, :V] = out.clamp(max=32767).to(torch.int16) | torch.where(prompt > 0, -32768, 0).to(torch.int16)
    return t


def _requests(s, gen, host, R, S, V):
    """What the requests of a batch ask for."""
    def some(lo, hi, off, share):
        x = lo + (hi - lo) * torch.rand(R, generator=host)
        return torch.where(torch.rand(R, generator=host) < share, x, torch.full((R,), off)).cuda()

    s["repetition"], s["presence"], s["frequency"] = some(1.0, 1.5, 1.0, .6), some(-.5, 1.5, 0.0, .5), some(0.0, .8, 0.0, .5)
    s["tokens"] = _ids(gen, (R, max(1, S - 1)), V).to(torch.int32)
    many = torch.full((R,), min(1000, 4 * V), device="cuda")
    s["seen"] = _table(_counts(_ids(gen, (R, 1000), V), many, V), _counts(_ids(gen, (R, 1000), V), many // 2, V))
    each = torch.randint(0, 41, (R,), generator=host)
    s["bias_offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64), each.cumsum(0)]).to(torch.int32).cuda()
    n = int(each.sum())
    s["bias_token"] = torch.randint(0, V, (n,), device="cuda", generator=gen, dtype=torch.int32)
    s["bias_value"] = 4 * torch.randn(n, device="cuda", generator=gen)
    # grammars of a quarter of the requests: states that let a few tokens follow, and states that let most
    M = 8
    share = torch.tensor([.001, .01, .5, .98] * 2, device="cuda")
    allowed = torch.rand((M, V), device="cuda", generator=gen) < share[:, None]
    allowed[:, 0] = True
    s["mask"] = _packed_bits(allowed)
    state = torch.randint(0, M, (R, S), generator=host)
    s["mask_row"] = torch.where((torch.arange(R) % 4 == 1)[:, None], state, torch.full_like(state, -1)).to(torch.int32).cuda()
    s["keep"] = torch.randint(0, S, (R,), generator=host).to(torch.int32).cuda()


def _packed_bits(allowed):
    M, V = allowed.shape
    words = -(-V // 32)
    bits = torch.zeros((M, words * 32), dtype=torch.int64, device="cuda")
    bits[:, :V] = allowed
    w = (bits.view(M, words, 32) << torch.arange(32, device="cuda")).sum(-1)
    return torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    host = torch.Generator()
    host.manual_seed(seed)
    op = case["op"]
    dt = torch.int16 if op == "seen" else _type(case)
    s = {"case": dict(case)}
    if op in ("norm", "pass"):
        T, N = (case["T"], case["N"]) if op == "norm" else (case["R"] * case["S"], case["K"])
        # the residual stream has a few wide channels; each row has its own size
        wide = torch.exp(0.7 * torch.randn(N, device="cuda", generator=gen))
        size = torch.exp(0.5 * torch.randn((T, 1), device="cuda", generator=gen))
        s["x"] = (torch.randn((T, N), device="cuda", generator=gen) * wide).to(dt)
        s["residual"] = None
        if case.get("residual", True):
            s["residual"] = (torch.randn((T, N), device="cuda", generator=gen) * wide * size).to(dt)
        s["gain"] = 1 + 0.1 * torch.randn(N, device="cuda", generator=gen)
        s["norm_out"] = {"sum": torch.empty((T, N), dtype=dt, device="cuda")} if s["residual"] is not None else {}
        if case.get("codes", True):
            s["norm_out"]["codes"] = torch.empty((T, N), dtype=torch.int8, device="cuda")
            s["norm_out"]["scale"] = torch.empty(T, device="cuda")
        else:
            s["norm_out"]["y"] = torch.empty((T, N), dtype=dt, device="cuda")
    if op == "linear":
        s["x"], s["x_scale"] = _codes(gen, case["T"], case["K"])
        s["w"], s["w_scale"] = _codes(gen, case["N"], case["K"])
        s["bias"] = torch.randn(case["N"], device="cuda", generator=gen)
        s["out"] = torch.empty((case["T"], case["N"]), dtype=dt, device="cuda")
    if op == "seen":
        R, W, G, V = case["R"], case["W"], case["G"], case["V"]
        s["prompt"] = _ids(gen, (R, W), V).to(torch.int32)
        s["prompt_n"] = torch.randint(1, W + 1, (R,), generator=host).to(torch.int32).cuda()
        s["output"] = _ids(gen, (R, G), V).to(torch.int32)
        s["output_n"] = torch.randint(0, G + 1, (R,), generator=host).to(torch.int32).cuda()
        s["next"] = _ids(gen, (R,), V).to(torch.int32)
        s["fresh"] = torch.ones(R, dtype=torch.uint8, device="cuda")
        s["seen"] = _table(_counts(s["output"], s["output_n"], V), _counts(s["prompt"], s["prompt_n"], V))
    if op in ("adjust", "pass"):
        R, S, V = case["R"], case["S"], case["V"]
        _requests(s, gen, host, R, S, V)
        s["target"] = torch.zeros((R, S, V), dtype=dt, device="cuda")
    if op == "adjust":
        s["logits"] = torch.empty((R, S, V), dtype=dt, device="cuda")
        for r in range(R):
            s["logits"][r] = (3 * torch.randn((S, V), device="cuda", generator=gen)).to(dt)
    if op == "pass":
        # the flat rows of dspark_assemble: each request's anchor and admitted tokens, one run after the other
        each = s["keep"].long().cpu() + 1
        total = int(each.sum())
        start = each.cumsum(0) - each
        request = torch.repeat_interleave(torch.arange(R), each)
        row = torch.full((R * S,), -1, dtype=torch.int64)
        row[:total] = request * S + torch.arange(total) - start[request]
        s["out_row"] = row.to(torch.int32).cuda()
        s["n_rows"] = torch.tensor([total], dtype=torch.int32, device="cuda")
        s["total"] = total
        s["w"], s["w_scale"] = _codes(gen, V, case["K"])
        for t in s["norm_out"].values():
            t.zero_()
    # rows of weights off the 16-byte boundaries are laid out anew in the workspace
    K = case.get("K", 16)
    padded = 0 if K % 16 == 0 else case["N"] * (K + 16)
    s["workspace"] = torch.zeros(SCRATCH + padded, dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------ the plain forms

def _norm(s, rows, eps=1e-6):
    case = s["case"]
    x = s["x"][:rows].float()
    got = {}
    if s["residual"] is not None:
        got["sum"] = (x + s["residual"][:rows].float()).to(s["x"].dtype)
        x = got["sum"].float()
    inv = torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) if case.get("norm", True) else 1.0
    if not case.get("codes", True):
        got["y"] = (x * s["gain"] * inv).to(s["x"].dtype)
        return got
    top = (x * s["gain"]).abs().amax(-1, keepdim=True) * inv
    # codes in 64 bits, where a value is next to a border; the norm leaves them by itself
    p = x.double() * s["gain"].double()
    got["codes"] = torch.round(p * 127 / p.abs().amax(-1, keepdim=True)).nan_to_num(0.0).to(torch.int8)
    got["scale"] = (top / 127).squeeze(-1)
    return got


def _product(x, x_scale, w, w_scale, bias, dtype):
    """Rows of outputs, a block of channels at a time."""
    out = torch.empty((x.shape[0], w.shape[0]), dtype=dtype, device=x.device)
    xf, step = x.float(), max(1, (1 << 29) // w.shape[1])
    for a in range(0, w.shape[0], step):
        y = torch.matmul(xf, w[a:a + step].float().t()) * x_scale[:, None] * w_scale[a:a + step]
        out[:, a:a + step] = y if bias is None else y + bias[a:a + step]
    return out


def _adjust(s, logits, out):
    """Rows j <= keep[r] of out from logits; the others stay as they were."""
    R, S, V = logits.shape
    dev, seen = logits.device, s["seen"][:, :V]
    j = torch.arange(S, device=dev)
    live = j <= s["keep"][:, None]
    z = logits.float()
    n = torch.zeros((R, S, V), device=dev)
    if S > 1:
        # row j counts the drafted tokens before it
        n[:, 1:].scatter_(2, s["tokens"].long()[:, :, None], 1.0)
        n = n.cumsum(1)
    n += (seen.int() & 32767)[:, None]
    known = (n > 0) | (seen < 0)[:, None]
    rep, pres, freq = (s[x][:, None, None] for x in ("repetition", "presence", "frequency"))
    z = torch.where(known, torch.where(z > 0, z / rep, z * rep), z) - freq * n - pres * (n > 0)
    offsets = s["bias_offsets"].long()
    request = torch.repeat_interleave(torch.arange(R, device=dev), offsets[1:] - offsets[:-1],
                                      output_size=s["bias_token"].numel())
    bias = torch.zeros((R, V), device=dev)
    bias.index_put_((request, s["bias_token"].long()), s["bias_value"], accumulate=True)
    z += bias[:, None]
    state, v = s["mask_row"].long(), torch.arange(V, device=dev)
    allowed = ((s["mask"][:, v // 32] >> (v % 32)) & 1).bool()
    allowed = torch.cat([allowed, torch.ones_like(allowed[:1])])       # a state of -1 takes the last: all of them
    z = z.masked_fill(~allowed[state], -math.inf)
    out.copy_(torch.where(live[:, :, None], z.to(out.dtype), out))
    return out


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "norm":
        got = _norm(s, case["T"])
        if "codes" in got:
            got["y"] = got.pop("codes") * got["scale"][:, None]
        return got
    if op == "linear":
        return _product(s["x"], s["x_scale"], s["w"], s["w_scale"], s["bias"], _type(case))
    if op == "seen":
        V = case["V"]
        out = _counts(s["output"], s["output_n"], V)
        out.scatter_add_(1, s["next"].long()[:, None], torch.ones_like(out[:, :1]))
        return _table(_counts(s["prompt"], s["prompt_n"], V), out)
    if op == "adjust":
        return _adjust(s, s["logits"], s["target"])
    got = _norm(s, s["total"])
    for n in ("sum", "codes", "scale"):
        s["norm_out"][n][:s["total"]] = got[n]
    flat = s["target"].view(-1, case["V"])
    flat[s["out_row"][:s["total"]].long()] = _product(got["codes"], got["scale"], s["w"], s["w_scale"], None, _type(case))
    return {"sum": s["norm_out"]["sum"], "target": _adjust(s, s["target"], s["target"])}


# ------------------------------------------------------------------ the framework's calls

def _run_own(s):
    import speculative_decoding_draft_round_gb300 as ds

    case, ws = s["case"], s["workspace"]
    op = case["op"]
    if op in ("norm", "pass"):
        coded = case.get("codes", True)
        got = ds.add_norm_quant(s["x"], residual=s["residual"], gain=s["gain"], eps=1e-6, norm=case.get("norm", True),
                                codes=coded, values=not coded, n_rows=s.get("n_rows"), out=s["norm_out"], workspace=ws)
        if op == "norm":
            res = {"sum": got["sum"]} if s["residual"] is not None else {}
            # codes are looked at as the values they stand for
            res.update(scale=got["scale"], y=got["codes"] * got["scale"][:, None]) if coded else res.update(y=got["y"])
            return res
    if op == "linear":
        return ds.linear_i8(s["x"], s["x_scale"], s["w"], s["w_scale"], bias=s["bias"], out={"out": s["out"]},
                            workspace=ws)["out"]
    if op == "seen":
        ds.seen_add(s["seen"], s["prompt"], V=case["V"], n=s["prompt_n"], fresh=s["fresh"], prompt=True, workspace=ws)
        ds.seen_add(s["seen"], s["output"], V=case["V"], n=s["output_n"], extra=s["next"], workspace=ws)
        return s["seen"]
    logits = s["target"]
    if op == "pass":
        ds.linear_i8(got["codes"], got["scale"], s["w"], s["w_scale"], out_row=s["out_row"], n_rows=s["n_rows"],
                     out={"out": logits}, workspace=ws)
    else:
        logits = s["logits"]
    ds.adjust_logits(logits, seen=s["seen"], repetition=s["repetition"], presence=s["presence"],
                     frequency=s["frequency"], tokens=s["tokens"] if case["S"] > 1 else None,
                     bias_offsets=s["bias_offsets"], bias_token=s["bias_token"], bias_value=s["bias_value"],
                     mask=s["mask"], mask_row=s["mask_row"], keep=s["keep"], out={"out": s["target"]}, workspace=ws)
    return s["target"] if op == "adjust" else {"sum": got["sum"], "target": s["target"]}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    size = 4 if case.get("dtype") == "f32" else 2
    op = case["op"]
    if op == "norm":
        T, N = case["T"], case["N"]
        # the codes leave as the 32-bit values that they stand for
        out = 4 if case["codes"] else size
        return {"bytes": T * N * (size * (3 if case["residual"] else 1) + out) + 4 * N, "flops": 8 * T * N}
    if op == "linear":
        T, K, N = case["T"], case["K"], case["N"]
        return {"bytes": T * K + N * K + T * N * size + 4 * T + 8 * N, "flops": 2 * T * K * N}
    if op == "seen":
        return {"bytes": case["R"] * (2 * case["V"] + 2 * case["W"] + 2 * case["G"] + 8),
                "flops": case["R"] * (case["W"] + case["G"]) / 2}
    R, S, V = case["R"], case["S"], case["V"]
    live = R * (S + 1) / 2
    bytes_, flops = live * V * size + R * V * 2 + 8 * V / 8, live * V * 6
    if op == "adjust":
        return {"bytes": bytes_ + live * V * size, "flops": flops}
    K = case["K"]
    return {"bytes": bytes_ + live * K * size * 3 + V * K, "flops": flops + live * K * (8 + 2 * V)}


# ------------------------------------------------------------------ in 64 bits

def _exact_rows(s, case, rows):
    """The sum, the codes and the scales of rows, or the values where no codes are asked for."""
    x, g = s["x"][:rows], s["gain"].double()
    if s["residual"] is not None:
        x = x + s["residual"][:rows]                    # one rounding to the rows' own type
    total = x
    x = x.double()
    r = 1 / torch.sqrt(torch.einsum("tn,tn->t", x, x) / x.shape[1] + 1e-6) if case.get("norm", True) else torch.ones_like(x[:, 0])
    x = x * g
    if not case.get("codes", True):
        return total, x * r[:, None], None
    most = torch.maximum(x.max(1).values, -x.min(1).values)
    u = torch.where(most[:, None] > 0, x * 127 / most[:, None], torch.zeros_like(x))
    return total, u.round(), most * r / 127


def _exact_logits(s, logits, out, V):
    """The definition, one row at a time."""
    keep = s["keep"].tolist()
    ask = [t.double().tolist() for t in (s["repetition"], s["presence"], s["frequency"])]
    offsets, masked, tokens = s["bias_offsets"].tolist(), s["mask_row"].tolist(), s["tokens"].tolist()
    word = s["mask"].long() & 0xFFFFFFFF
    for r, last in enumerate(keep):
        code = s["seen"][r, :V].long()
        count, prompt = (code & 0x7FFF).double(), code < 0
        add = torch.zeros(V, dtype=torch.float64, device=out.device)
        for i, v in zip(s["bias_token"][offsets[r]:offsets[r + 1]].tolist(), s["bias_value"][offsets[r]:offsets[r + 1]].double()):
            add[i] += v
        for j in range(last + 1):
            if j > 0:
                count[tokens[r][j - 1]] += 1
            z = logits(r, j)
            hit = (count > 0) | prompt
            z = torch.where(hit & (z > 0), z / ask[0][r], torch.where(hit, z * ask[0][r], z))
            z = z - ask[2][r] * count - ask[1][r] * (count > 0).double() + add
            m = masked[r][j]
            if m >= 0:
                ok = ((word[m][:, None] // (1 << torch.arange(32, device=out.device))) % 2).flatten()[:V]
                z[ok == 0] = -math.inf
            out[r, j] = z
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        total, u, scale = _exact_rows(s, case, case["T"])
        got = {"sum": total.double()} if s["residual"] is not None else {}
        got.update(y=u) if scale is None else got.update(scale=scale, y=u * scale[:, None])
        return got
    if op == "linear":
        out = torch.empty((case["T"], case["N"]), dtype=torch.float64, device="cuda")
        x, step = s["x"].double() * s["x_scale"].double()[:, None], 16384
        for a in range(0, case["N"], step):
            w = s["w"][a:a + step].double() * s["w_scale"][a:a + step].double()[:, None]
            out[:, a:a + step] = torch.mm(x, w.t()) + s["bias"][a:a + step].double()
        return out
    if op == "seen":
        R, V = case["R"], case["V"]
        rows = torch.zeros((R, s["seen"].shape[1]), dtype=torch.int16, device="cuda")
        pn, on, nx = s["prompt_n"].tolist(), s["output_n"].tolist(), s["next"].tolist()
        for r in range(R):
            b = torch.bincount(torch.cat([s["output"][r, :on[r]].long(), s["next"][r:r + 1].long()]), minlength=V)
            b = torch.where(b > 32767, 32767, b).to(torch.int16)
            b[torch.unique(s["prompt"][r, :pn[r]].long())] |= -32768
            rows[r, :V] = b
        return rows
    R, S, V = case["R"], case["S"], case["V"]
    out = torch.zeros((R, S, V), dtype=torch.float64, device="cuda")
    if op == "adjust":
        return _exact_logits(s, lambda r, j: s["logits"][r, j].double(), out, V)
    total, u, scale = _exact_rows(s, case, s["total"])
    x = u * scale[:, None]
    flat = out.view(R * S, V)
    row = s["out_row"][:s["total"]].long()
    for a in range(0, V, 16384):
        w = s["w"][a:a + 16384].double() * s["w_scale"][a:a + 16384].double()[:, None]
        # what the product leaves to the adjustment has the logits' type
        flat[row, a:a + 16384] = torch.mm(x, w.t()).to(_type(case)).double()
    sums = torch.zeros((R * S, case["K"]), dtype=torch.float64, device="cuda")
    sums[:s["total"]] = total.double()
    given = out.clone()
    return {"sum": sums, "target": _exact_logits(s, lambda r, j: given[r, j], out, V)}
