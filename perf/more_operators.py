"""What is measured of the attention layers of a hybrid model: the paged cache of keys and values, and the attention that
reads it, for the same ragged batches that the prefill of the recurrent layers takes.

* ``write``   the batch's keys and values into the cache's pages, as they are (bf16) or as e4m3 with a power of two for
              each token and head; with 8 bits the rows are read back after;
* ``read``    cached rows out of the pages again, as packed bf16 rows;
* ``attend``  causal attention of the batch's rows over the cache, query heads in groups on shared key heads: one new
              token a request, a few drafts, prompts, and prompts behind a cached context;
* ``layer``   what an attention layer runs for a batch: the plan, the norms with rotation, the write, the attention.

Each case is a dict of plain values; lengths follow from the case alone, the data from the seed.
"""
import math
import random

import torch

own = False

F32, F64, BF16, I32, E4M3 = torch.float32, torch.float64, torch.bfloat16, torch.int32, torch.float8_e4m3fn
MIN_EXP = -60  # the least power of two of an 8-bit head


# ----------------------------------------------------------------------------- cases
def listed():
    h = {"Hq": 32, "Hk": 4, "D": 128}
    return [
        # one decode step's keys and values into an 8-bit cache, 256 requests
        {"name": "write_step", "op": "write", "R": 256, "lo": 1, "hi": 1, "c_lo": 1, "c_hi": 8000, "ls": 1, "type": "e4m3", "page": 64, **h},
        # a batch of prompts into a bf16 cache, out of one fused projection
        {"name": "write_prompts", "op": "write", "R": 16, "lo": 300, "hi": 4000, "c_lo": 0, "c_hi": 0, "ls": 2, "type": "bf16", "page": 64, **h},
        # cached conversations taken out of an 8-bit cache, to be kept elsewhere
        {"name": "read_cached", "op": "read", "R": 21, "lo": 200, "hi": 8000, "c_lo": 0, "c_hi": 0, "ls": 3, "type": "e4m3", "page": 64, **h},
        # the smallest step: four young conversations
        {"name": "decode_few", "op": "attend", "R": 4, "lo": 1, "hi": 1, "c_lo": 50, "c_hi": 900, "ls": 4, "type": "bf16", "page": 64, **h},
        # a decode step of a full batch
        {"name": "decode_step", "op": "attend", "R": 256, "lo": 1, "hi": 1, "c_lo": 20, "c_hi": 8000, "ls": 5, "type": "bf16", "page": 64, **h},
        # the same from an 8-bit cache with small pages
        {"name": "decode_8bit", "op": "attend", "R": 256, "lo": 1, "hi": 1, "c_lo": 20, "c_hi": 8000, "ls": 6, "type": "e4m3", "page": 16, **h},
        # one request with a long document behind it
        {"name": "decode_long", "op": "attend", "R": 1, "lo": 1, "hi": 1, "c_lo": 131071, "c_hi": 131071, "ls": 7, "type": "bf16", "page": 256, **h},
        # speculative verification: four drafts a request
        {"name": "drafts", "op": "attend", "R": 64, "lo": 4, "hi": 4, "c_lo": 100, "c_hi": 6000, "ls": 8, "type": "bf16", "page": 32, **h},
        # a batch of prompts
        {"name": "prompts", "op": "attend", "R": 16, "lo": 300, "hi": 4000, "c_lo": 0, "c_hi": 0, "ls": 9, "type": "bf16", "page": 64, **h},
        # one long document
        {"name": "document", "op": "attend", "R": 1, "lo": 32768, "hi": 32768, "c_lo": 0, "c_hi": 0, "ls": 10, "type": "bf16", "page": 128, "Hq": 16, "Hk": 2, "D": 128},
        # turns of conversations, a few tokens to two hundred behind an 8-bit context; some bring one token
        {"name": "turns_8bit", "op": "attend", "R": 61, "lo": 1, "hi": 200, "c_lo": 100, "c_hi": 8000, "ls": 11, "type": "e4m3", "page": 64, **h},
        # everything that an attention layer runs for a mixed batch
        {"name": "layer_mixed", "op": "layer", "R": 40, "lo": 1, "hi": 900, "c_lo": 0, "c_hi": 3000, "ls": 12, "type": "bf16", "page": 64, "rot": 64, **h},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["write", "read", "attend", "attend", "attend", "attend", "layer"])
    Hk = rng.choice([1, 2, 4, 8])
    Hq = Hk * rng.choice([1, 2, 3, 4, 5, 8, 8, 16])
    if Hq > 64:
        Hq = Hk * 4
    D = rng.choice([64, 128, 128])
    c = {"op": op, "ls": rng.randrange(1 << 20), "Hq": Hq, "Hk": Hk, "D": D, "page": rng.choice([16, 32, 64, 128, 256]),
         "type": rng.choice(["bf16", "e4m3"]) if op != "layer" else "bf16"}
    if op == "layer":
        c["rot"] = rng.choice([D // 4, D // 2, D])
    if op in ("write", "read"):
        c["R"] = _log_int(rng, 1, 256)
        c["hi"] = _log_int(rng, 1, max(1, min(16_000, 6_000_000 // (c["R"] * Hk))))
        c["lo"] = rng.choice([1, max(1, c["hi"] // 4)])
        c["c_lo"], c["c_hi"] = rng.choice([(0, 0), (0, 500), (1, 3000)]) if op == "write" else (0, 0)
        return c
    kind = rng.choice(["token", "drafts", "prompts", "turns"])
    if kind == "token":
        R = _log_int(rng, 1, 256)
        most = _log_int(rng, 8, max(8, min(131_071, 4_000_000 // (R * Hk))))
        c.update(R=R, lo=1, hi=1, c_lo=rng.choice([1, max(1, most // 3)]), c_hi=most)
    elif kind == "drafts":
        R = _log_int(rng, 1, 128)
        n = rng.choice([2, 3, 4, 8])
        most = _log_int(rng, 8, max(8, min(65_000, 4_000_000 // (R * Hk * n))))
        c.update(R=R, lo=n, hi=n, c_lo=0, c_hi=most)
    else:
        R = _log_int(rng, 1, 40)
        pairs = 4_000_000_000 // (Hq * R)  # rows x keys of a request
        hi = _log_int(rng, 2, max(2, min(12_000, int(math.sqrt(pairs)))))
        most = 0 if kind == "prompts" else _log_int(rng, 8, max(8, min(30_000, pairs // hi)))
        c.update(R=R, lo=rng.choice([1, max(1, hi // 3)]), hi=hi, c_lo=0, c_hi=most)
    return c


# ----------------------------------------------------------------------------- what a batch looks like
def _batch(case):
    """Lengths and contexts of the requests, and the pages that they need."""
    r = random.Random(case["ls"])
    lengths, context = [], []
    c0, c1 = case["c_lo"], case["c_hi"]
    for _ in range(case["R"]):
        lengths.append(int(round(math.exp(r.uniform(math.log(case["lo"]), math.log(case["hi"]))))))
        context.append(r.randint(c0, c1))
    page = case["page"]
    need = [(n + c + page - 1) // page for n, c in zip(lengths, context)]
    cu = [0]
    for n in lengths:
        cu.append(cu[-1] + n)
    return {"lengths": lengths, "context": context, "need": need, "cu": cu, "tokens": cu[-1], "longest": max(lengths)}


def _pairs(b):
    """Rows times the keys that each sees, over all requests."""
    return sum(n * c + n * (n + 1) // 2 for n, c in zip(b["lengths"], b["context"]))


def work(case):
    b = _batch(case)
    T, Hq, Hk, D = b["tokens"], case["Hq"], case["Hk"], case["D"]
    head = 2 * D if case["type"] == "bf16" else D + 1  # bytes of a cached head
    if case["op"] in ("write", "read"):
        bytes_ = 2.0 * T * Hk * (2 * D + head) + 8 * T + 4 * sum(b["need"])
        if case["op"] == "write" and case["type"] == "e4m3":  # read back
            bytes_ += 2.0 * T * Hk * (2 * D + head)
        return {"bytes": bytes_, "flops": 0.0}
    keys = sum(n + c for n, c in zip(b["lengths"], b["context"]))
    bytes_ = 4.0 * T * Hq * D + 2.0 * keys * Hk * head + 4 * sum(b["need"]) + 8 * T
    flops = 4.0 * D * Hq * _pairs(b)
    if case["op"] == "layer":  # the new keys and values come in, and go to the cache
        bytes_ += 4.0 * T * Hk * D
        flops += 8.0 * T * (Hq + Hk) * D
    return {"bytes": bytes_, "flops": flops}


# ----------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape, dtype=F32):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype)


def _exponent(a):
    """The least e with a <= 448 * 2^e (448 = 0.875 * 2^9), at least MIN_EXP."""
    m, x = torch.frexp(a)
    e = x - 9 + (m > 0.875)
    return torch.where(a > 0, e, MIN_EXP).clamp_min(MIN_EXP)


def _quantise(x):
    """e4m3 codes and powers of two of heads x [..., D]."""
    x = x.float()
    e = _exponent(x.abs().amax(-1))
    return torch.ldexp(x, -e[..., None]).to(E4M3), e


def _values(codes, e):
    return torch.ldexp(codes.float(), e[..., None])


def _inputs(case, seed):
    b = _batch(case)
    g = _gen(seed)
    op, R, T, Hq, Hk, D, page = case["op"], case["R"], b["tokens"], case["Hq"], case["Hk"], case["D"], case["page"]
    s = {"case": case, "b": b}
    i32 = lambda x: torch.tensor(x, dtype=I32, device="cuda")
    s["lengths"], s["context"] = i32(b["lengths"]), i32(b["context"])
    s["req"] = torch.repeat_interleave(torch.arange(R, device="cuda"), s["lengths"].long())
    s["pos"] = torch.arange(T, device="cuda") - i32(b["cu"][:-1]).long()[s["req"]] + s["context"].long()[s["req"]]
    # every request's pages, anywhere in the cache
    total, most = sum(b["need"]), max(b["need"])
    s["n_pages"], s["max_pages"] = total + 3, most
    order = torch.randperm(s["n_pages"], generator=g, device="cuda").to(I32)
    table = torch.full((R, most), -1, dtype=I32, device="cuda")
    at = 0
    need = i32(b["need"])
    filled = torch.arange(most, device="cuda")[None, :] < need[:, None]
    table[filled] = order[:total]
    s["pages"] = table
    # one projection's rows: queries, keys and values side by side
    rows = _normal(g, T, (Hq + 2 * Hk) * D, dtype=BF16)
    s["q"] = rows[:, : Hq * D].unflatten(1, (Hq, D))
    s["k"], s["v"] = (rows[:, (Hq + i * Hk) * D : (Hq + (i + 1) * Hk) * D].unflatten(1, (Hk, D)) for i in (0, 1))
    # what the cache holds; heads differ in size, and some tokens stand out
    shape = (s["n_pages"], Hk, page, D)
    for name in ("ck", "cv"):
        size = torch.exp2(torch.randint(-1, 2, (1, Hk, 1, 1), generator=g, device="cuda").float())
        if op in ("write", "layer") and not any(b["context"]):
            x = torch.zeros(shape, dtype=BF16, device="cuda")
        else:
            x = torch.empty(shape, dtype=BF16, device="cuda")
            for i in range(0, shape[0], 4096):  # in pieces, for the memory
                n = min(4096, shape[0] - i)
                x[i : i + n] = _normal(g, n, *shape[1:]) * size
        if case["type"] == "e4m3":
            codes, e = _quantise_cache(x)
            s[name], s[name + "_e"] = codes, e
        else:
            s[name], s[name + "_e"] = x, None
        del x
    if op == "layer":
        s["wq"], s["wk"] = (1 + 0.2 * _normal(g, D)).to(BF16), (1 + 0.2 * _normal(g, D)).to(BF16)
        s["inv_freq"] = (10000.0 ** (-torch.arange(0, case["rot"], 2, device="cuda", dtype=F64) / case["rot"])).to(F32)
    else:
        # queries and keys are normed by then: scores of a few units, where some tokens matter
        s["q"].mul_(1.5)
    return s


def _quantise_cache(x):
    codes = torch.empty(x.shape, dtype=E4M3, device=x.device)
    e = torch.empty(x.shape[:-1], dtype=I32, device=x.device)
    for i in range(0, x.shape[0], 4096):
        codes[i : i + 4096], e[i : i + 4096] = _quantise(x[i : i + 4096])
    return codes, e


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:  # what a serving loop keeps: the batch's plan, the cache, and the attention's plan and workspace
        from rs_decode_gb300.attention import KVCache
        from rs_decode_gb300.prefill import Ragged

        b = s["b"]
        s["ragged"] = Ragged(case["R"], b["tokens"])
        s["ragged"].plan(s["lengths"], s["context"])
        s["cache"] = c = KVCache(case["Hq"], case["Hk"], case["D"], s["n_pages"], s["max_pages"], page=case["page"], type=case["type"])
        if case["type"] == "e4m3":
            c.k.view(torch.uint8).copy_(s["ck"].view(torch.uint8))
            c.v.view(torch.uint8).copy_(s["cv"].view(torch.uint8))
            c.k_exp.copy_(s["ck_e"] + 127)
            c.v_exp.copy_(s["cv_e"] + 127)
        else:
            c.k.copy_(s["ck"])
            c.v.copy_(s["cv"])
        del s["ck"], s["cv"]
        if case["op"] in ("attend", "layer"):
            s["plan"] = c.plan(s["ragged"], b["longest"])
            s["work"] = c.workspace(s["ragged"], b["longest"])
            s["y"] = torch.empty(b["tokens"], case["Hq"], case["D"], dtype=BF16, device="cuda")
    return s


# ----------------------------------------------------------------------------- the plain forms
def _slots(s):
    """Page and place in it of the batch's rows."""
    page = s["case"]["page"]
    return s["pages"][s["req"], s["pos"] // page].long(), s["pos"] % page


def _plain_write(s):
    at, place = _slots(s)
    if s["case"]["type"] == "bf16":
        s["ck"][at, :, place], s["cv"][at, :, place] = s["k"], s["v"]
        return {"k": s["ck"], "v": s["cv"]}
    out = {}
    for name, x in (("ck", s["k"]), ("cv", s["v"])):
        codes, e = _quantise(x)
        s[name].view(torch.uint8)[at, :, place] = codes.view(torch.uint8)
        s[name + "_e"][at, :, place] = e.to(I32)
        out[name[1]] = _values(codes, e).to(BF16)
    return out


def _plain_read(s):
    at, place = _slots(s)
    out = {}
    for name in ("ck", "cv"):
        if s["case"]["type"] == "bf16":
            out[name[1]] = s[name][at, :, place]
        else:
            codes = s[name].view(torch.uint8)[at, :, place].view(E4M3)
            out[name[1]] = _values(codes, s[name + "_e"][at, :, place]).to(BF16)
    return out


def _cached(s, name, r, n, dtype):
    """The first n keys or values of request r, [Hk, n, D]."""
    page = s["case"]["page"]
    at = s["pages"][r, : (n + page - 1) // page].long()
    if s["case"]["type"] == "bf16":
        x = s[name][at].to(dtype)
    else:
        x = torch.ldexp(s[name].view(torch.uint8)[at].view(E4M3).to(dtype), s[name + "_e"][at][..., None])
    return x.transpose(0, 1).flatten(1, 2)[:, :n]


def _plain_attend(s, q):
    case, b = s["case"], s["b"]
    Hq, Hk, D = case["Hq"], case["Hk"], case["D"]
    g, c = Hq // Hk, D ** -0.5
    y = torch.empty(b["tokens"], Hq, D, dtype=BF16, device=q.device)
    for r, (n, ctx, row) in enumerate(zip(b["lengths"], b["context"], b["cu"])):
        k, v = _cached(s, "ck", r, n + ctx, F32), _cached(s, "cv", r, n + ctx, F32)
        step = max(1, min(n, (1 << 28) // (Hq * (n + ctx))))
        for a in range(0, n, step):
            m = min(step, n - a)
            end = ctx + a + m
            qq = q[row + a : row + a + m].float().unflatten(1, (Hk, g)).permute(1, 2, 0, 3).reshape(Hk, g * m, D)
            p = torch.matmul(qq, k[:, :end].transpose(1, 2)) * c
            if m > 1:
                seen = torch.arange(end, device=q.device)[None, :] <= ctx + a + torch.arange(m, device=q.device)[:, None]
                p = p.view(Hk, g, m, end).masked_fill_(~seen, -math.inf).view(Hk, g * m, end)
            p = p.sub_(p.amax(-1, keepdim=True)).exp_()
            o = torch.matmul(p, v[:, :end]) / p.sum(-1, keepdim=True)
            y[row + a : row + a + m] = o.view(Hk, g, m, D).permute(2, 0, 1, 3).reshape(m, Hq, D).to(BF16)
    return y


def _norm_rotate(x, w, positions, inv_freq, dtype):
    x = x.to(dtype)
    x = x * (x.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * w.to(dtype)
    n = inv_freq.numel()
    angle = positions.to(F64)[:, None] * inv_freq.to(F64)  # far positions: in 64 bits
    cos, sin = angle.cos().to(dtype)[:, None, :], angle.sin().to(dtype)[:, None, :]
    a, b = x[..., :n], x[..., n : 2 * n]
    return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., 2 * n :]], -1)


def _plain_layer(s):
    n, c = s["lengths"].long(), s["context"].long()
    cu = torch.cat([n.new_zeros(1), n.cumsum(0)])
    row = torch.arange(s["b"]["tokens"], device=n.device)
    req = torch.searchsorted(cu, row, right=True) - 1
    s["req"], s["pos"] = req, row - cu[req] + c[req]
    q = _norm_rotate(s["q"], s["wq"], s["pos"], s["inv_freq"], F32).to(BF16)
    k = _norm_rotate(s["k"], s["wk"], s["pos"], s["inv_freq"], F32).to(BF16)
    at, place = _slots(s)
    s["ck"][at, :, place], s["cv"][at, :, place] = k, s["v"]
    return {"y": _plain_attend(s, q), "k": s["ck"], "v": s["cv"]}


# ----------------------------------------------------------------------------- the framework's calls
def _own_attend(s, q):
    return s["cache"].attend(s["ragged"], q, s["pages"], s["plan"], max_len=s["b"]["longest"], y=s["y"], work=s["work"])


def _own(s):
    case, cache, ragged = s["case"], s["cache"], s["ragged"]
    if case["op"] == "write":
        cache.write(ragged, s["k"], s["v"], s["pages"])
        if case["type"] == "bf16":
            return {"k": cache.k, "v": cache.v}
    if case["op"] in ("write", "read"):
        k, v = cache.read(ragged, s["pages"])
        return {"k": k, "v": v}
    if case["op"] == "attend":
        return {"y": _own_attend(s, s["q"])}
    from rs_decode_gb300.prefill import qk_norm

    ragged.plan(s["lengths"], s["context"])
    cache.plan(ragged, s["b"]["longest"], out=s["plan"])
    q, k = qk_norm(s["q"], s["k"], norm="rms", eps=1e-6, wq=s["wq"], wk=s["wk"], positions=ragged.token_pos, inv_freq=s["inv_freq"])
    cache.write(ragged, k, s["v"], s["pages"])
    return {"y": _own_attend(s, q), "k": cache.k, "v": cache.v}


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "write":
        return _plain_write(state)
    if op == "read":
        return _plain_read(state)
    if op == "attend":
        return {"y": _plain_attend(state, state["q"])}
    return _plain_layer(state)


# ----------------------------------------------------------------------------- in 64 bits
def _exact_attend(s, q, k_of, v_of):
    """Row blocks of one head at a time: log of the sum of exponentials, then the weights themselves."""
    case, b = s["case"], s["b"]
    g = case["Hq"] // case["Hk"]
    y = torch.zeros(b["tokens"], case["Hq"], case["D"], dtype=F64, device="cuda")
    for r in range(case["R"]):
        n, ctx, row = b["lengths"][r], b["context"][r], b["cu"][r]
        kk, vv = k_of(r), v_of(r)
        step = max(1, min(n, (1 << 25) // (n + ctx)))
        for a in range(0, n, step):
            m = min(step, n - a)
            end = ctx + a + m
            hidden = torch.ones(m, end, dtype=torch.bool, device="cuda").triu(ctx + a + 1)
            for h in range(case["Hq"]):
                score = q[row + a : row + a + m, h].to(F64) @ kk[h // g, :end].T / math.sqrt(case["D"])
                score[hidden] = -math.inf
                weight = (score - torch.logsumexp(score, -1, keepdim=True)).exp()
                y[row + a : row + a + m, h] = weight @ vv[h // g, :end]
    return y


def exact(case, seed):
    if case["op"] in ("write", "read"):
        s = _inputs(case, seed)
        if case["type"] == "bf16" and case["op"] == "write":
            at, place = _slots(s)
            s["ck"][at, :, place], s["cv"][at, :, place] = s["k"], s["v"]
            return {"k": s["ck"], "v": s["cv"]}
        out = {}
        for name in ("k", "v"):
            if case["op"] == "write":  # the codes' values: what the rounding to 8 bits leaves
                x = s[name].to(F64)
                a = x.abs().amax(-1, keepdim=True)
                unit = torch.exp2(torch.ceil(torch.log2(a / 448.0)).clamp_min(float(MIN_EXP)))
                out[name] = (x / unit).to(F32).to(E4M3).to(F64) * unit
            else:
                at, place = _slots(s)
                x = s["c" + name]
                if case["type"] == "bf16":
                    out[name] = x[at, :, place].to(F64)
                else:
                    e = s["c" + name + "_e"][at, :, place][..., None]
                    out[name] = x.view(torch.uint8)[at, :, place].view(E4M3).to(F64) * torch.exp2(e.to(F64))
        return out
    b = _batch(case)
    if 4.0 * case["D"] * case["Hq"] * _pairs(b) > 5e12 or case["R"] * case["Hq"] * max(1, b["longest"] // 1000) > 200_000:
        return None
    s = _inputs(case, seed)
    if case["op"] == "attend":
        return {"y": _exact_attend(s, s["q"], lambda r: _cached(s, "ck", r, b["lengths"][r] + b["context"][r], F64),
                                   lambda r: _cached(s, "cv", r, b["lengths"][r] + b["context"][r], F64))}
    q = _norm_rotate(s["q"], s["wq"], s["pos"], s["inv_freq"], F64)
    k = _norm_rotate(s["k"], s["wk"], s["pos"], s["inv_freq"], F64)
    at, place = _slots(s)
    # the attention reads the norms as they are stored, in bf16
    s["ck"][at, :, place], s["cv"][at, :, place] = k.to(BF16), s["v"]
    y = _exact_attend(s, q.to(BF16), lambda r: _cached(s, "ck", r, b["lengths"][r] + b["context"][r], F64),
                      lambda r: _cached(s, "cv", r, b["lengths"][r] + b["context"][r], F64))
    ck = s["ck"].to(F64)
    ck[at, :, place] = k
    return {"y": y, "k": ck, "v": s["cv"]}
