"""What is measured of the ragged prefill of a Gated DeltaNet layer.

Three operators, as a serving loop calls them for one batch of requests whose
lengths are known on the GPU:

* ``plan``   token offsets, rows' requests and positions, the chunk table and the table of state-cache blocks, from the
             requests' lengths (once for a batch, used by every layer);
* ``qk``     the norm of each head's query and key, with the rotation by position in the same pass;
* ``gdn``    the gated delta rule over the packed tokens of all requests, into the decode state, with the states at
             block boundaries kept for prefix reuse: chunked for long requests, recurrent for a few tokens;
* ``layer``  the three of them in a row.

Each case is a dict of plain values; request lengths follow from the case alone, the data from the seed.
"""
import math
import random

import torch

own = False

CHUNK = 64          # tokens of a chunk; chunks are aligned to multiples of it in a request's own positions
F32, F64, BF16, I32 = torch.float32, torch.float64, torch.bfloat16, torch.int32


# ----------------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of a full batch: every request brings one token
        {"name": "plan_step", "op": "plan", "R": 256, "lo": 1, "hi": 1, "ls": 1, "zeros": 0, "ctx": 4096, "block": 512},
        # prompts and decode tokens mixed in one batch, some requests idle, about half a million rows
        {"name": "plan_prompts", "op": "plan", "R": 1021, "lo": 1, "hi": 4500, "ls": 2, "zeros": 0.1, "ctx": 3000, "block": 256},
        # one decode step: 16 query and 16 key heads of 256 tokens, unit length
        {"name": "qk_step", "op": "qk", "T": 256, "Hq": 16, "Hk": 16, "D": 128, "norm": "l2", "rot": 0, "inter": False, "fused": True},
        # a long prompt's queries and keys for the delta rule, out of one fused projection
        {"name": "qk_prompt", "op": "qk", "T": 32768, "Hq": 16, "Hk": 16, "D": 128, "norm": "l2", "rot": 0, "inter": False, "fused": True},
        # the same for the attention layers between: weighted rms norm, half of each head rotated, shared key heads
        {"name": "qk_rotated", "op": "qk", "T": 8191, "Hq": 32, "Hk": 4, "D": 128, "norm": "rms", "rot": 64, "inter": False, "fused": True},
        # one token for each of 256 cached requests: the state is read and written once
        {"name": "gdn_tokens", "op": "gdn", "R": 256, "lo": 1, "hi": 1, "ls": 3, "zeros": 0, "H": 32, "G": 16, "d": 128, "prec": "fp32", "block": 0, "cached": 1.0, "fused": False},
        # short turns of cached conversations, a few tokens to two hundred each
        {"name": "gdn_turns", "op": "gdn", "R": 61, "lo": 1, "hi": 200, "ls": 4, "zeros": 0.05, "H": 32, "G": 16, "d": 128, "prec": "two", "block": 0, "cached": 0.8, "fused": True},
        # a batch of prompts, with the state kept every 512 tokens for prefix reuse
        {"name": "gdn_prompts", "op": "gdn", "R": 16, "lo": 300, "hi": 4000, "ls": 5, "zeros": 0, "H": 32, "G": 16, "d": 128, "prec": "fp32", "block": 512, "cached": 0.25, "fused": True},
        # one long document
        {"name": "gdn_long", "op": "gdn", "R": 1, "lo": 32768, "hi": 32768, "ls": 6, "zeros": 0, "H": 32, "G": 16, "d": 128, "prec": "fp32", "block": 0, "cached": 0, "fused": True},
        # a small layer with 64-wide heads and a bf16 state
        {"name": "gdn_small", "op": "gdn", "R": 24, "lo": 1, "hi": 1500, "ls": 7, "zeros": 0.1, "H": 8, "G": 4, "d": 64, "prec": "shared_bf16", "block": 0, "cached": 0.5, "fused": False},
        # everything that a layer runs for a mixed batch, with a bf16 state
        {"name": "layer_mixed", "op": "layer", "R": 40, "lo": 1, "hi": 900, "ls": 8, "zeros": 0.05, "H": 32, "G": 16, "d": 128, "prec": "shared_bf16", "block": 256, "cached": 0.5, "fused": True},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["plan", "qk", "gdn", "gdn", "layer"])
    if op == "plan":
        R = _log_int(rng, 1, 4096)
        hi = _log_int(rng, 1, max(1, min(8000, 600_000 // R)))
        return {"op": op, "R": R, "lo": rng.choice([1, max(1, hi // 4)]), "hi": hi, "ls": rng.randrange(1 << 20), "zeros": rng.choice([0, 0.1, 0.5]),
                "ctx": rng.choice([0, 100, 5000]), "block": rng.choice([0, 64, 192, 256, 512])}
    if op == "qk":
        D = rng.choice([64, 128, 128, 256])
        Hq = rng.choice([1, 4, 8, 16, 32])
        Hk = rng.choice([h for h in (1, 2, 4, 8, 16) if h <= Hq])
        T = _log_int(rng, 1, max(1, min(40_000, 32768 * 32 * 128 // ((Hq + Hk) * D))))
        return {"op": op, "T": T, "Hq": Hq, "Hk": Hk, "D": D, "norm": rng.choice(["l2", "rms"]), "rot": rng.choice([0, D // 4, D // 2, D]),
                "inter": rng.random() < 0.3, "fused": rng.random() < 0.6}
    d = rng.choice([64, 128, 128])
    G = rng.choice([2, 3, 4, 8, 16])
    H = G * rng.choice([1, 2, 2, 4])
    H = min(H, 32) // G * G or G
    R = _log_int(rng, 1, 256)
    most = max(1, 1_000_000 * 128 * 128 // (H * d * d))  # tokens x heads no more than the long document's
    hi = _log_int(rng, 1, max(1, min(16_000, most // R)))
    return {"op": op, "R": R, "lo": rng.choice([1, max(1, hi // 3)]), "hi": hi, "ls": rng.randrange(1 << 20), "zeros": rng.choice([0, 0, 0.1]), "H": H, "G": G, "d": d,
            # a rounding of a normed key that falls the other way is more than an fp32 state is held to
            "prec": rng.choice(["fp32", "fp32", "two", "shared_bf16"]) if op == "gdn" else "shared_bf16", "block": rng.choice([0, 64, 256, 512]) if R * hi * H <= 400_000 else 0,
            "cached": rng.choice([0.0, 0.5, 1.0]), "fused": rng.random() < 0.5}


# ----------------------------------------------------------------------------- what a batch looks like
def _batch(case):
    """The batch's integers, on the host: lengths, tokens before them, chunks and blocks."""
    r = random.Random(case["ls"])
    R, block = case["R"], case["block"]
    lengths, context = [], []
    for i in range(R):
        n = 0 if r.random() < case["zeros"] else int(round(math.exp(r.uniform(math.log(case["lo"]), math.log(case["hi"])))))
        lengths.append(n)
        if "ctx" in case:
            context.append(r.randrange(case["ctx"] + 1) if case["ctx"] and r.random() < 0.8 else 0)
        else:  # a cached prefix ends where a block ends
            c = case["cached"] > 0 and r.random() < case["cached"]
            context.append((block or CHUNK) * r.randint(1, 8) if c else 0)
    if not any(lengths):
        lengths[0] = case["hi"]
    cached = [c > 0 for c in context]
    chunks, cu, cuc = [], [0], [0]
    for i, (n, c) in enumerate(zip(lengths, context)):
        at = c
        while at < c + n:
            end = min(c + n, (at // CHUNK + 1) * CHUNK)
            chunks.append((i, cu[-1] + at - c, end - at, at // CHUNK))
            at = end
        cu.append(cu[-1] + n)
        cuc.append(len(chunks))
    taken = [((c + n) // block - c // block) if block else 0 for n, c in zip(lengths, context)]
    max_blocks = max([(c + n) // block for n, c in zip(lengths, context)] + [1]) if block else 0
    return {"lengths": lengths, "context": context, "cached": cached, "cu": cu, "cuc": cuc, "chunks": chunks, "taken": taken, "max_blocks": max_blocks,
            "tokens": cu[-1], "longest": max(lengths)}


def _spare(case):
    """Rows that a batch leaves free: a captured step has a fixed number of rows."""
    return 37 if case["op"] == "plan" else 0


def work(case):
    if case["op"] == "qk":
        n = case["T"] * (case["Hq"] + case["Hk"]) * case["D"]
        return {"bytes": 4.0 * n + (4 * case["T"] + 2 * case["rot"] if case["rot"] else 0) + (4 * case["D"] if case["norm"] == "rms" else 0),
                "flops": n * (4.0 if not case["rot"] else 4.0 + 3.0 * case["rot"] / case["D"])}
    b = _batch(case)
    R, T = case["R"], b["tokens"]
    cap = T + _spare(case)
    plan = 8 * R + 8 * (R + 1) + 8 * cap + 16 * (cap // CHUNK + 2 * R) + 8 * sum(b["taken"]) + 16
    if case["op"] == "plan":
        return {"bytes": float(plan), "flops": 0.0}
    H, G, d = case["H"], case["G"], case["d"]
    active = [n > 0 for n in b["lengths"]]
    size = 2 if case["prec"] == "shared_bf16" else 4  # of the pool's values
    reads = sum(a and c for a, c in zip(active, b["cached"])) * size
    writes = sum(active) * {"fp32": 4, "two": 6, "shared_bf16": 2}[case["prec"]] + sum(b["taken"]) * size
    bytes_ = T * (2 * G * d * 2 + 2 * H * d * 2 + 8 * H) + H * d * d * (reads + writes)
    flops = 6.0 * T * H * d * d
    if case["op"] == "layer":  # the raw queries and keys are read and the normed ones are needed nowhere else
        bytes_ += plan
        flops += 8.0 * T * G * d
    return {"bytes": float(bytes_), "flops": flops}


# ----------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape, dtype=F32):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype)


def _plan_inputs(case, seed):
    b = _batch(case)
    g = _gen(seed)
    s = {"case": case, "b": b}
    # the data of a plan are its integers: which block numbers are free comes from the seed
    total = sum(b["taken"])
    s["free"] = torch.randperm(total + 5, generator=g, device="cuda").to(I32) if case["block"] else None
    s["lengths"] = torch.tensor(b["lengths"], dtype=I32, device="cuda")
    s["context"] = torch.tensor(b["context"], dtype=I32, device="cuda")
    s["cap"] = b["tokens"] + _spare(case)
    s["no_chunk"] = torch.tensor([-1, 0, 0, 0], device="cuda")
    if case["op"] == "plan":
        # another seed hands the same lengths to the requests in another order
        order = torch.randperm(case["R"], generator=g, device="cuda")
        s["lengths"], s["context"] = s["lengths"][order].contiguous(), s["context"][order].contiguous()
    s["table"] = torch.full((case["R"], b["max_blocks"]), -1, dtype=I32, device="cuda") if case["block"] else None
    return s


def _unit(x):
    f = x.float()
    return (f / f.square().sum(-1, keepdim=True).sqrt().clamp_min(1e-6)).to(x.dtype)


def _gdn_inputs(case, seed):
    s = _plan_inputs(case, seed)
    g = _gen(seed + 7_777_777)
    b, R, H, G, d, T = s["b"], case["R"], case["H"], case["G"], case["d"], s["b"]["tokens"]
    if case["fused"]:  # one projection's rows hold queries, keys and values side by side
        rows = _normal(g, T, (2 * G + H) * d, dtype=BF16)
        q, k = rows[:, : G * d].unflatten(1, (G, d)), rows[:, G * d : 2 * G * d].unflatten(1, (G, d))
        v = rows[:, 2 * G * d :].unflatten(1, (H, d))
    else:
        q, k, v = _normal(g, T, G, d, dtype=BF16), _normal(g, T, G, d, dtype=BF16), _normal(g, T, H, d, dtype=BF16)
    if case["op"] == "gdn":  # the layer norms them itself
        q.copy_(_unit(q))
        k.copy_(_unit(k))
    s.update(q=q, k=k, v=v)
    # heads forget at rates from a hundred tokens to one; a token's gate moves around its head's
    rate = torch.exp(torch.rand(H, generator=g, device="cuda") * math.log(1024.0) - math.log(64.0))
    s["alpha"] = torch.exp(-torch.nn.functional.softplus(_normal(g, T, H)) * rate)
    s["beta"] = torch.sigmoid(_normal(g, T, H))
    # cached requests start from a state of the pool: its first slots; the others are for this batch's blocks
    n = sum(b["cached"])
    s["pool"] = torch.zeros(n + sum(b["taken"]) + 6, H, d, d, device="cuda", dtype=BF16 if case["prec"] == "shared_bf16" else F32)
    s["pool"][:n] = _normal(g, n, H, d, d) * 0.1
    at = iter(range(n))
    s["start"] = torch.tensor([next(at) if c else -1 for c in b["cached"]], dtype=I32, device="cuda")
    s["rows"] = torch.randperm(R, generator=g, device="cuda").to(I32)
    if case["block"]:
        s["free"] += n
        s["table_now"] = _plain_plan(s)["block_table"]
    # the batch's integers again, in the order that suits a loop over chunks: requests with the most chunks first
    order = sorted(range(R), key=lambda i: b["cuc"][i] - b["cuc"][i + 1])
    s["count"] = [b["cuc"][i + 1] - b["cuc"][i] for i in order]
    s["first"] = torch.tensor([b["cuc"][i] for i in order], device="cuda")
    s["order"] = torch.tensor(order, device="cuda")
    s["chunks"] = torch.tensor(b["chunks"], device="cuda")
    return s


def _qk_inputs(case, seed):
    g = _gen(seed)
    T, Hq, Hk, D = case["T"], case["Hq"], case["Hk"], case["D"]
    s = {"case": case}
    if case["fused"]:  # queries, keys and the values that this operator leaves alone, in one row
        rows = _normal(g, T, (Hq + 2 * Hk) * D, dtype=BF16)
        s["q"], s["k"] = rows[:, : Hq * D].unflatten(1, (Hq, D)), rows[:, Hq * D : (Hq + Hk) * D].unflatten(1, (Hk, D))
    else:
        s["q"], s["k"] = _normal(g, T, Hq, D, dtype=BF16), _normal(g, T, Hk, D, dtype=BF16)
    rms = case["norm"] == "rms"
    s["wq"] = (1 + 0.2 * _normal(g, D)).to(BF16) if rms else None
    s["wk"] = (1 + 0.2 * _normal(g, D)).to(BF16) if rms else None
    s["scale_q"] = 1.0 if rms else D ** -0.5
    s["positions"] = s["inv_freq"] = None
    if case["rot"]:
        s["positions"] = torch.randint(0, 40_000, (T,), generator=g, device="cuda", dtype=I32)
        s["inv_freq"] = (10000.0 ** (-torch.arange(0, case["rot"], 2, device="cuda", dtype=F64) / case["rot"])).to(F32)
    return s


def prepare(case, seed):
    op = case["op"]
    if op == "qk":
        return _qk_inputs(case, seed)
    s = _plan_inputs(case, seed) if op == "plan" else _gdn_inputs(case, seed)
    if own:  # what a serving loop keeps: the plan's arrays and the layer's decode state
        from rs_decode_gb300.layer import Layer
        from rs_decode_gb300.prefill import Ragged
        from rs_decode_gb300 import binding as rb

        s["ragged"] = Ragged(case["R"], s["cap"], block=case["block"], max_blocks=s["b"]["max_blocks"], n_free=0 if s["free"] is None else s["free"].numel())
        if s["table"] is not None:
            s["ragged"].block_table.fill_(-1)
        if op != "plan":
            s["layer"] = Layer("gdn", case["R"], case["H"], case["G"], case["d"], case["d"], 16, precision=rb.PRECISIONS[case["prec"]])
            s["y"] = torch.empty(s["b"]["tokens"], case["H"], case["d"], dtype=BF16, device="cuda")
            s["work"] = s["layer"].prefill_workspace(s["ragged"], s["b"]["longest"])
        if op == "gdn":
            s["ragged"].plan(s["lengths"], s["context"], s["free"])
    return s


# ----------------------------------------------------------------------------- plan: the plain form
def _excl(x):
    return torch.cat([x.new_zeros(1), x.cumsum(0)])


def _plain_plan(s):
    case, cap = s["case"], s["cap"]
    n, c = s["lengths"].long(), s["context"].long()
    R = n.numel()
    cu = _excl(n)
    first, last = c // CHUNK, (c + n + CHUNK - 1) // CHUNK
    nch = torch.where(n > 0, last - first, 0)
    cuc = _excl(nch)
    row = torch.arange(cap, device=n.device)
    req = torch.searchsorted(cu, row, right=True) - 1
    live = row < cu[-1]
    req = torch.where(live, req, R - 1)
    pos = torch.where(live, row - cu[req] + c[req], -1)
    token_req = torch.where(live, req, -1)
    ccap = cap // CHUNK + 2 * R
    ch = torch.arange(ccap, device=n.device)
    creq = torch.searchsorted(cuc, ch, right=True) - 1
    clive = ch < cuc[-1]
    creq = torch.where(clive, creq, R - 1)
    cabs = first[creq] + ch - cuc[creq]
    lo = torch.maximum(cabs * CHUNK, c[creq])
    hi = torch.minimum((cabs + 1) * CHUNK, (c + n)[creq])
    table = torch.stack([creq, cu[creq] + lo - c[creq], hi - lo, cabs], 1)
    table = torch.where(clive[:, None], table, s["no_chunk"])
    out = {"cu_tokens": cu, "cu_chunks": cuc, "token_req": token_req, "token_pos": pos, "chunks": table}
    used = cu.new_zeros(())
    if case["block"]:
        bs, blocks = case["block"], s["table"].clone()
        j0 = c // bs
        new = (c + n) // bs - j0
        off = _excl(new)
        used = off[-1]
        j = torch.arange(blocks.shape[1], device=n.device)[None, :]
        at = off[:-1, None] + j - j0[:, None]
        mine = (j >= j0[:, None]) & (j < (j0 + new)[:, None])
        free = s["free"]
        got = torch.where(at < free.numel(), free[at.clamp(0, free.numel() - 1)], -1)
        out["block_table"] = torch.where(mine, got, blocks).to(I32)
    out["counts"] = torch.stack([cu[-1], cuc[-1], used, (n > 0).sum()])
    return {k: v.to(I32) for k, v in out.items()}


def _own_plan(s):
    r = s["ragged"]
    r.plan(s["lengths"], s["context"], s["free"])
    out = {"cu_tokens": r.cu_tokens, "cu_chunks": r.cu_chunks, "token_req": r.token_req, "token_pos": r.token_pos, "chunks": r.chunks}
    if s["case"]["block"]:
        out["block_table"] = r.block_table
    out["counts"] = r.counts
    return out


# ----------------------------------------------------------------------------- qk: the plain form
def _rotate(x, positions, inv_freq, inter):
    rot = 2 * inv_freq.numel()
    angle = positions.to(inv_freq.dtype)[:, None] * inv_freq
    cos, sin = angle.cos()[:, None, :], angle.sin()[:, None, :]
    if inter:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    else:
        a, b = x[..., : rot // 2], x[..., rot // 2 : rot]
    y = x.clone()
    ra, rb_ = a * cos - b * sin, b * cos + a * sin
    if inter:
        y[..., 0:rot:2], y[..., 1:rot:2] = ra, rb_
    else:
        y[..., : rot // 2], y[..., rot // 2 : rot] = ra, rb_
    return y


def _norm_one(x, w, norm, scale, positions, inv_freq, inter, dtype):
    x = x.to(dtype)
    ss = x.square().sum(-1, keepdim=True)
    if norm == "l2":
        x = x / ss.sqrt().clamp_min(1e-6)
    else:
        x = x * (ss / x.shape[-1] + 1e-6).rsqrt()
    if w is not None:
        x = x * w.to(dtype)
    x = x * scale
    if inv_freq is not None:
        x = _rotate(x, positions, inv_freq.to(dtype), inter)
    return x


def _plain_qk(s):
    case = s["case"]
    return [_norm_one(x, w, case["norm"], sc, s["positions"], s["inv_freq"], case["inter"], F32).to(BF16)
            for x, w, sc in ((s["q"], s["wq"], s["scale_q"]), (s["k"], s["wk"], 1.0))]


def _own_qk(s):
    from rs_decode_gb300.prefill import qk_norm

    case = s["case"]
    return list(qk_norm(s["q"], s["k"], norm=case["norm"], eps=1e-6, wq=s["wq"], wk=s["wk"], scale_q=s["scale_q"], positions=s["positions"], inv_freq=s["inv_freq"], interleaved=case["inter"]))


# ----------------------------------------------------------------------------- gdn: the plain form
def _inverse(A):
    """(I + A)^-1 of strictly lower triangular blocks, by doubling the size of the inverted diagonal blocks."""
    n = A.shape[-1]
    i = torch.arange(n, device=A.device)
    X = torch.eye(n, device=A.device, dtype=A.dtype).expand_as(A)
    size = 1
    while size < n:
        below = (i[:, None] // size % 2 == 1) & (i[:, None] // size - 1 == i[None, :] // size)
        X = X - X @ (A * below) @ X
        size *= 2
    return X


def _end_slots(s, table):
    """The pool slot that the state after each chunk goes to, -1 for none."""
    block, (req, at, n, _) = s["case"]["block"], s["chunks"].unbind(1)
    cu = _excl(s["lengths"].long())
    end = s["context"].long()[req] + at - cu[req] + n
    return torch.where(end % block == 0, table[req, (end // block - 1).clamp_min(0)].long(), -1)


def _plain_gdn(s):
    case, b = s["case"], s["b"]
    R, H, G, d, T = case["R"], case["H"], case["G"], case["d"], b["tokens"]
    dev = s["q"].device
    chunks = s["chunks"]
    t = torch.arange(CHUNK, device=dev)
    idx = torch.where(t < chunks[:, 2:3], chunks[:, 1:2] + t, T)  # [chunks, 64], T: no token

    def rows(x, pad=0.0):
        x = torch.cat([x.float(), torch.full_like(x[:1], pad, dtype=F32)])
        return x[idx].transpose(1, 2)  # [chunks, heads, 64(, d)]

    q, k = (rows(s[n]).repeat_interleave(H // G, 1) for n in ("q", "k"))
    v = rows(s["v"])
    g = rows(s["alpha"], 1.0).log().cumsum(-1)  # [chunks, H, 64]
    beta = rows(s["beta"])
    lower = t[:, None] >= t[None, :]
    decay = torch.where(lower, g[..., :, None] - g[..., None, :], -math.inf).exp()
    kt = k.transpose(-1, -2)
    A = (k @ kt) * decay * (t[:, None] > t[None, :]) * beta[..., None]
    Tm = _inverse(A) * beta[..., None, :]
    del A
    P = (q @ kt) * decay
    del decay
    eg = g.exp()[..., None]
    last = g[..., -1:]
    ke = (k * (last - g).exp()[..., None]).transpose(-1, -2)
    y = torch.empty_like(v)
    pool = s["pool"]
    S = torch.where((s["start"] >= 0)[:, None, None, None], pool[s["start"].clamp_min(0).long()].float(), 0.0)
    slots = _end_slots(s, s["table_now"]) if case["block"] else None
    order, count = s["order"], s["count"]
    S = S[order]
    n = R
    for c in range(count[0]):
        while count[n - 1] <= c:
            n -= 1
        at = s["first"][:n] + c
        Sn = S[:n]
        u = Tm[at] @ (v[at] - eg[at] * (k[at] @ Sn))
        y[at] = eg[at] * (q[at] @ Sn) + P[at] @ u
        S[:n] = last[at].exp()[..., None] * Sn + ke[at] @ u
        if slots is not None:
            to = slots[at]  # the last slot of the pool is no block's
            pool[torch.where(to >= 0, to, pool.shape[0] - 1)] = torch.where((to >= 0)[:, None, None, None], S[:n].to(pool.dtype), pool[-1])
    out = {"y": torch.empty(T + 1, H, d, device=dev)}
    out["y"][idx.reshape(-1)] = y.transpose(1, 2).reshape(-1, H, d)
    out["y"] = out["y"][:T].to(BF16)
    live = s["lengths"][order] > 0
    hp = torch.zeros(R, H, d, d, device=dev)
    hp[s["rows"].long()[order]] = torch.where(live[:, None, None, None], S, 0.0)
    if case["prec"] != "shared_bf16":
        out["state"] = hp
    if case["prec"] != "fp32":
        out["state_bf16"] = hp.to(BF16)
    if case["block"]:
        out["pool"] = pool
    return out


def _own_gdn(s, q, k):
    case, layer = s["case"], s["layer"]
    y = layer.prefill(s["ragged"], q, k, s["v"], s["alpha"], s["beta"], max_len=s["b"]["longest"], rows=s["rows"], start=s["start"], pool=s["pool"], y=s["y"], work=s["work"])
    out = {"y": y}
    if case["prec"] != "shared_bf16":
        out["state"] = layer.checkpoint_hp()
    if case["prec"] != "fp32":
        out["state_bf16"] = layer.ckpt_lp.view(BF16).view(layer.shape)
    if case["block"]:
        out["pool"] = s["pool"]
    return out


def run(state):
    s, case = state, state["case"]
    if case["op"] == "plan":
        return _own_plan(s) if own else _plain_plan(s)
    if case["op"] == "qk":
        return _own_qk(s) if own else _plain_qk(s)
    if case["op"] == "gdn":
        if own:
            return _own_gdn(s, s["q"], s["k"])
        return _plain_gdn(s)
    d = case["d"]
    if own:
        from rs_decode_gb300.prefill import qk_norm

        plan = _own_plan(s)
        q, k = qk_norm(s["q"], s["k"], norm="l2", eps=1e-6, scale_q=d ** -0.5)
        out = _own_gdn(s, q, k)
    else:
        plan = _plain_plan(s)
        q = _norm_one(s["q"], None, "l2", d ** -0.5, None, None, False, F32).to(BF16)
        k = _norm_one(s["k"], None, "l2", 1.0, None, None, False, F32).to(BF16)
        out = _plain_gdn({**s, "q": q, "k": k, "table_now": plan.get("block_table")})
    return {**out, "counts": plan["counts"], "q": q, "k": k}


# ----------------------------------------------------------------------------- in 64 bits
def _steps(s, q, k):
    """The recurrence itself, token by token, for all requests at once, in 64 bits."""
    case, b = s["case"], s["b"]
    R, H, G, d, T = case["R"], case["H"], case["G"], case["d"], b["tokens"]
    dev = q.device
    n = s["lengths"].long()
    order = torch.argsort(n, descending=True, stable=True)
    cu = torch.tensor(b["cu"][:-1], device=dev)[order]
    ctx = s["context"].long()[order]
    S = torch.zeros(R, H, d, d, dtype=F64, device=dev)
    cached = s["start"][order] >= 0
    S[cached] = s["pool"].double()[s["start"][order][cached].long()]
    y = torch.zeros(T, H, d, dtype=F64, device=dev)
    pool = s["pool"].double()
    live = sorted(b["lengths"], reverse=True)
    m = sum(x > 0 for x in live)
    block = case["block"]
    at_step = {}  # token index -> (request's place in the order, pool slot) of the blocks that end with it
    if block:
        table = s["table_now"].tolist()
        for i, r in enumerate(order.tolist()):
            x, c = b["lengths"][r], b["context"][r]
            for end in range((c // block + 1) * block, c + x + 1, block):
                at_step.setdefault(end - c - 1, []).append((i, table[r][end // block - 1]))
    for t in range(live[0]):
        while live[m - 1] <= t:
            m -= 1
        rows = cu[:m] + t
        kk, qq = (x[rows].double().repeat_interleave(H // G, 1) for x in (k, q))  # [m, H, d]
        Sn = S[:m]
        Sn *= s["alpha"][rows].double()[..., None, None]
        u = s["beta"][rows].double()[..., None] * (s["v"][rows].double() - (kk[..., None, :] @ Sn)[..., 0, :])
        Sn += kk[..., :, None] * u[..., None, :]
        y[rows] = (qq[..., None, :] @ Sn)[..., 0, :]
        for i, slot in at_step.get(t, ()):
            pool[slot] = S[i]
    out = {"y": y}
    full = torch.zeros(R, H, d, d, dtype=F64, device=dev)
    full[s["rows"].long()[order]] = torch.where((n[order] > 0)[:, None, None, None], S, 0.0)
    if case["prec"] != "shared_bf16":
        out["state"] = full
    if case["prec"] != "fp32":
        out["state_bf16"] = full
    if block:
        out["pool"] = pool
    return out


def exact(case, seed):
    op = case["op"]
    if op == "plan":
        return None  # whole numbers
    s = _qk_inputs(case, seed) if op == "qk" else _gdn_inputs(case, seed)
    if op == "qk":
        return [_norm_one(x, w, case["norm"], sc, s["positions"], s["inv_freq"], case["inter"], F64)
                for x, w, sc in ((s["q"], s["wq"], s["scale_q"]), (s["k"], s["wk"], 1.0))]
    if op == "gdn":
        return _steps(s, s["q"], s["k"])
    q = _norm_one(s["q"], None, "l2", case["d"] ** -0.5, None, None, False, F64)
    k = _norm_one(s["k"], None, "l2", 1.0, None, None, False, F64)
    # the rule reads the norms as they are stored, in bf16
    out = _steps(s, q.to(BF16), k.to(BF16))
    return {**out, "counts": None, "q": q, "k": k}
