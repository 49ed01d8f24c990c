"""Ragged prefill on the GPU against plain 64-bit implementations: the batch
plan (whole numbers, equal), the head norms with rotation, and the gated delta
rule from every kind of starting state into the decode state.

Tolerances, fixed before the first run:
* norms: one bf16 rounding of the result (2^-9 relative; 2^-8 where the fp32
  value may fall to the other neighbour) plus 4e-6 of the magnitudes that
  enter, for a sum of at most 256 squares, a root, a division and an angle in fp32;
* states: 2-norm per request and head, 5e-6: operands held to 22 bits (S, R, T
  and u, 2^-23 each) and fp32 sums, times 8 for what 64 rows of the same key
  may add up;
* outputs y: 2-norm per request and head, 6e-3: y itself rounded to bf16 (2^-9),
  and S, u and P to fp16 (2^-12 each, times the same 8, half of it on average).
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
from rs_decode_gb300 import binding as rb
from rs_decode_gb300.layer import Layer
from rs_decode_gb300.prefill import Ragged, qk_norm

pytestmark = pytest.mark.gpu

TOL_S, TOL_Y, TOL_BF16 = 5e-6, 6e-3, 2.0 ** -8


def dev(a, dtype=None):
    t = torch.as_tensor(np.asarray(a))
    return (t if dtype is None else t.to(dtype)).cuda()


# ----------------------------------------------------------------------------- plan
def plan_ref(lengths, context, cap, block, max_blocks, free, table):
    """The plan by plain loops; returns the arrays and the status bits."""
    R, bits = len(lengths), 0
    cu, cuc, cub = [0], [0], [0]
    chunks, token_req, token_pos = [], [], []
    table = table.copy() if table is not None else None
    raw = 0
    for r in range(R):
        n, c = int(lengths[r]), int(context[r]) if context is not None else 0
        if n < 0 or c < 0 or n + c > 2 ** 30:
            bits |= rb.DEV_LENGTH
            n = 0
        raw += n
        if raw > cap:
            if n:
                bits |= rb.DEV_CAPACITY
            n = 0
        at = c
        while at < c + n:
            end = min(c + n, (at // 64 + 1) * 64)
            chunks.append((r, cu[-1] + at - c, end - at, at // 64))
            at = end
        token_req += [r] * n
        token_pos += list(range(c, c + n))
        taken = 0
        if block and n:
            for j in range(c // block, (c + n) // block):
                k = cub[-1] + taken
                if k >= len(free) or j >= max_blocks:
                    bits |= rb.DEV_BLOCKS
                if j < max_blocks:
                    table[r, j] = free[k] if k < len(free) else -1
                taken += 1
        cu.append(cu[-1] + n)
        cuc.append(len(chunks))
        cub.append(cub[-1] + taken)
    ccap = cap // 64 + 2 * R
    active = sum(b > a for a, b in zip(cu, cu[1:]))
    counts = [cu[-1], cuc[-1], cub[-1], active]
    chunks += [(-1, 0, 0, 0)] * (ccap - len(chunks))
    token_req += [-1] * (cap - cu[-1])
    token_pos += [-1] * (cap - cu[-1])
    return dict(cu_tokens=cu, cu_chunks=cuc, cu_blocks=cub, token_req=token_req, token_pos=token_pos,
                chunks=np.array(chunks).reshape(-1, 4), counts=counts, block_table=table), bits


PLANS = {
    "one token": dict(lengths=[1], context=[0], cap=1),
    "nothing": dict(lengths=[0, 0, 0], context=[5, 0, 64], cap=7),
    "edges": dict(lengths=[63, 64, 65, 0, 1, 128, 127], context=[0, 64, 63, 9, 191, 1, 65], cap=501, block=64),
    "no context": dict(lengths=[300, 2, 70], context=None, cap=400, block=128),
    "odd capacity": dict(lengths=[3, 6], context=[0, 0], cap=13),
    "too many rows": dict(lengths=[50, 60, 0, 5, 1], context=[0, 0, 3, 0, 0], cap=100, block=64),
    "bad requests": dict(lengths=[5, -1, 7, 2 ** 31 - 1, 4], context=[0, 0, -3, 1, 2 ** 30], cap=64),
    "huge positions": dict(lengths=[64, 200], context=[2 ** 30 - 64, 2 ** 30 - 201], cap=300),
    "free list runs out": dict(lengths=[256, 640], context=[0, 128], cap=1000, block=128, free=3),
    "table too narrow": dict(lengths=[640], context=[64], cap=640, block=64, max_blocks=5),
}


@pytest.mark.parametrize("name", PLANS)
def test_plan(name):
    c = PLANS[name]
    run_plan(np.array(c["lengths"], np.int32), None if c["context"] is None else np.array(c["context"], np.int32),
             c["cap"], c.get("block", 0), c.get("free", 64), c.get("max_blocks"))


@pytest.mark.parametrize("R,seed", [(7, 0), (255, 1), (1025, 2), (4000, 3), (4001, 4), (9001, 5)])
def test_plan_of_many_requests(R, seed):
    rng = np.random.default_rng(seed)
    lengths = rng.integers(0, 300, R).astype(np.int32) * (rng.random(R) < 0.8)
    context = rng.integers(0, 1000, R).astype(np.int32)
    total = int(lengths.sum())
    run_plan(lengths.astype(np.int32), context, total + 3, 192, 10 * R, None)
    # the same with a capacity that ends in the middle
    run_plan(lengths.astype(np.int32), context, max(1, total * 2 // 3), 0, 0, None)


def run_plan(lengths, context, cap, block, n_free, max_blocks):
    R = len(lengths)
    rng = np.random.default_rng(R)
    free = rng.permutation(n_free).astype(np.int32) if block else np.zeros(0, np.int32)
    if block and max_blocks is None:
        c = context if context is not None else np.zeros_like(lengths)
        max_blocks = int(max(1, np.max((c.astype(np.int64) + np.maximum(lengths, 0)) // block)))
    rg = Ragged(R, cap, block, max_blocks or 0, len(free))
    before = None
    if block:
        before = rng.integers(100, 200, (R, max_blocks)).astype(np.int32)
        rg.block_table.copy_(dev(before))
    ref, bits = plan_ref(lengths, context, cap, block, max_blocks or 0, free, before)
    rg.plan(dev(lengths), None if context is None else dev(context), dev(free) if block else None)
    for k, want in ref.items():
        if want is not None:
            np.testing.assert_array_equal(getattr(rg, k).cpu().numpy(), np.asarray(want), err_msg=k)
    assert rg.status() == bits
    return rg


# ----------------------------------------------------------------------------- norms
def qk_ref(x, norm, eps, w, w0, scale, positions, inv_freq, inter):
    """64-bit; also the magnitude that bounds the fp32 error."""
    x = x.double()
    ss = x.square().sum(-1, keepdim=True)
    if norm == "l2":
        x = x / ss.sqrt().clamp_min(eps)
    elif norm == "rms":
        x = x / (ss / x.shape[-1] + eps).sqrt()
    if w is not None:
        x = x * (w.double() + w0)
    x = x * scale
    mag = x.abs().clone()
    if inv_freq is not None:
        rot = 2 * inv_freq.numel()
        # exact angles: whole turns are taken off in integers
        f = [int(round(float(v) / (2 * np.pi) * 2 ** 96)) for v in inv_freq.double().cpu()]
        ang = torch.tensor([[((int(p) * k) % 2 ** 96) / 2 ** 96 * 2 * np.pi for k in f] for p in positions.cpu()],
                           dtype=torch.float64, device=x.device)[:, None, :]
        a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if inter else (x[..., : rot // 2], x[..., rot // 2: rot])
        ra, rb_ = a * ang.cos() - b * ang.sin(), b * ang.cos() + a * ang.sin()
        m = a.abs() + b.abs()
        y = x.clone()
        for t, va, vb in ((y, ra, rb_), (mag, m, m)):
            if inter:
                t[..., 0:rot:2], t[..., 1:rot:2] = va, vb
            else:
                t[..., : rot // 2], t[..., rot // 2: rot] = va, vb
        x = y
    return x, mag


QK = [  # T, Hq, Hk, D, norm, rot, interleaved, weights, fused
    (1, 1, 1, 64, "l2", 0, False, False, False),
    (3, 5, 2, 64, "rms", 16, False, True, True),
    (17, 16, 16, 128, "l2", 0, False, False, True),
    (33, 7, 1, 128, "rms", 128, True, True, False),
    (700, 8, 2, 128, "rms", 64, False, True, True),
    (5, 3, 3, 256, "none", 256, False, False, False),
    (1001, 4, 4, 256, "l2", 64, True, True, True),
    (40, 0, 3, 128, "l2", 32, False, False, False),
    (40, 3, 0, 64, "rms", 64, True, True, False),
]


@pytest.mark.parametrize("T,Hq,Hk,D,norm,rot,inter,weights,fused", QK)
def test_qk_norm(T, Hq, Hk, D, norm, rot, inter, weights, fused):
    g = torch.Generator(device="cuda").manual_seed(T)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda", dtype=torch.bfloat16)
    if fused:
        row = rnd(T, (Hq + Hk) * D + 24)
        q, k = row[:, :Hq * D].unflatten(1, (Hq, D)), row[:, Hq * D:(Hq + Hk) * D].unflatten(1, (Hk, D))
    else:
        q, k = rnd(T, Hq, D) if Hq else None, rnd(T, Hk, D) if Hk else None
    for t in (q, k):
        if t is not None:
            t[T // 2, 0] = 0  # a head without a direction
            t[T // 3, -1] *= 1000
    wq, wk = (rnd(D), rnd(D)) if weights else (None, None)
    inv = pos = None
    if rot:
        inv = (10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)).float()
        pos = torch.randint(-50_000, 500_000, (T,), generator=g, device="cuda", dtype=torch.int32)
        pos[0] = 2 ** 31 - 1
    kw = dict(norm=norm, eps=1e-6, wq=wq, wk=wk, weight_offset=1.0 if weights else 0.0, scale_q=D ** -0.5, scale_k=1.5,
              positions=pos, inv_freq=inv, interleaved=inter)
    qo, ko = qk_norm(q, k, **kw)
    for x, o, w, sc in ((q, qo, wq, D ** -0.5), (k, ko, wk, 1.5)):
        if x is None:
            assert o is None
            continue
        ref, mag = qk_ref(x, norm, 1e-6, w, kw["weight_offset"], sc, pos, inv, inter)
        err = (o.double() - ref).abs()
        assert o.dtype == torch.bfloat16 and bool((err <= TOL_BF16 * ref.abs() + 4e-6 * mag + 1e-30).all())
    # in place, and the same from another stream
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        qk_norm(q, k, out=(q, k), **kw)
    st.synchronize()
    for t, o in ((q, qo), (k, ko)):
        assert t is None or torch.equal(t, o)


def test_qk_norm_keeps_nan_to_its_head():
    q = torch.randn(9, 4, 128, device="cuda").bfloat16()
    clean, _ = qk_norm(q, None, norm="rms")
    q[3, 2, 7] = float("nan")
    q[5, 1, 0] = float("inf")
    for norm in ("rms", "l2"):
        out, _ = qk_norm(q, None, norm=norm)
        assert bool(out[3, 2].isnan().all()) and bool(out[5, 1, 0].isnan())
        bad = torch.zeros(9, 4, dtype=torch.bool, device="cuda")
        bad[3, 2] = bad[5, 1] = True
        assert bool(out[~bad].isfinite().all())
        if norm == "rms":
            assert torch.equal(out[~bad], clean[~bad])


# ----------------------------------------------------------------------------- gated delta rule
def gdn_ref(S, q, k, v, alpha, beta, ends=()):
    """One request, 64-bit: S [H, N, P], q, k [n, H, N], v [n, H, P] -> y, S, states after `ends` rows."""
    S, ys, kept = S.clone(), [], {}
    for t in range(q.shape[0]):
        S = alpha[t][:, None, None] * S
        u = beta[t][:, None] * (v[t] - torch.einsum("hn,hnp->hp", k[t], S))
        S = S + k[t][:, :, None] * u[:, None, :]
        ys.append(torch.einsum("hn,hnp->hp", q[t], S))
        if t + 1 in ends:
            kept[t + 1] = S.clone()
    return (torch.stack(ys) if ys else v[:0]), S, kept


class Case:
    def __init__(self, lengths, H=4, G=2, d=128, prec="fp32", context=None, block=0, fused=True, seed=0, spare=0,
                 alpha="mixed", beta="mixed", keys="unit", B=None):
        self.lengths, self.H, self.G, self.d, self.block, self.prec = list(lengths), H, G, d, block, prec
        R, T = len(lengths), sum(lengths)
        self.context = list(context) if context is not None else [0] * R
        g = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s: torch.randn(s, generator=g, device="cuda")
        cap = T + spare
        if fused:
            row = rnd(cap, (2 * G + H) * d + 8).bfloat16()
            self.q, self.k = row[:, :G * d].unflatten(1, (G, d)), row[:, G * d:2 * G * d].unflatten(1, (G, d))
            self.v = row[:, 2 * G * d:(2 * G + H) * d].unflatten(1, (H, d))
        else:
            self.q, self.k, self.v = rnd(cap, G, d).bfloat16(), rnd(cap, G, d).bfloat16(), rnd(cap, H, d).bfloat16()
        if keys == "same":
            self.k.copy_(self.k[:1].expand_as(self.k).clone())
        qk_norm(self.q, self.k, norm="l2", out=(self.q, self.k))
        rate = torch.exp(torch.rand(H, generator=g, device="cuda") * 7 - 4.2)
        self.alpha = torch.exp(-torch.nn.functional.softplus(rnd(cap, H)) * rate)
        self.beta = torch.sigmoid(rnd(cap, H))
        if alpha == "one":
            self.alpha.fill_(1)
        elif alpha == "zeros":  # resets in the middle, and several in a row
            self.alpha[torch.rand(cap, H, generator=g, device="cuda") < 0.2] = 0
        elif alpha == "slow":  # states that remember thousands of rows
            self.alpha.pow_(0.01)
        elif alpha == "tiny":
            self.alpha.fill_(1e-30)
        if beta == "one":
            self.beta.fill_(1)
        elif beta == "zero":
            self.beta.zero_()
        self.cap = cap
        B = B or R + 2
        self.layer = Layer("gdn", B, H, G, d, d, 16, precision=rb.PRECISIONS[prec])
        self.S0 = rnd(B, H, d, d) * 0.1
        self.layer.init(self.S0)
        self.rows = torch.randperm(B, generator=g, device="cuda")[:R].to(torch.int32)
        self.pool_dtype = torch.bfloat16 if prec == "shared_bf16" else torch.float32
        free = 0
        if block:
            free = sum((c + n) // block - c // block for c, n in zip(self.context, lengths))
        self.pool = (rnd(R + free + 1, H, d, d) * 0.1).to(self.pool_dtype)
        self.free = (torch.randperm(free, generator=g, device="cuda") + R).to(torch.int32)
        mb = max([1] + [(c + n) // block for c, n in zip(self.context, lengths)]) if block else 0
        self.rg = Ragged(R, cap, block, mb, free)
        self.rg.plan(dev(np.array(self.lengths, np.int32)), dev(np.array(self.context, np.int32)),
                     self.free if block else None)
        assert self.rg.status() == 0

    def run(self, start=None, max_len=None, **kw):
        self.start = start
        self.pool0 = self.pool.clone()
        self.y = self.layer.prefill(self.rg, self.q, self.k, self.v, self.alpha, self.beta,
                                    max_len=max(self.lengths) if max_len is None else max_len, rows=self.rows,
                                    start=None if start is None else dev(np.array(start, np.int32)), pool=self.pool, **kw)
        return self.y

    def state(self):
        return self.layer.checkpoint_lp_f32() if self.prec == "shared_bf16" else self.layer.checkpoint_hp()

    def first_state(self, r):
        s = -2 if self.start is None else self.start[r]
        if s == -1:
            return torch.zeros_like(self.S0[0]).double()
        x = self.S0[self.rows[r]] if s == -2 else self.pool0[s]
        return (x.bfloat16() if self.prec == "shared_bf16" else x).double()

    def check(self, skip=()):
        rep, at = self.H // self.G, 0
        got = self.state()
        cub = self.rg.cu_blocks.tolist()
        touched = set()
        for r, n in enumerate(self.lengths):
            row = int(self.rows[r])
            if n == 0 or r in skip:
                if r not in skip:
                    assert torch.equal(got[row], self.S0[row].bfloat16().float() if self.prec == "shared_bf16" else self.S0[row])
                at += n
                continue
            s = slice(at, at + n)
            c, b = self.context[r], self.block
            ends = [e - c for e in range((c // b + 1) * b, c + n + 1, b)] if b else []
            q, k = (x[s].double().repeat_interleave(rep, 1) for x in (self.q, self.k))
            y, S, kept = gdn_ref(self.first_state(r), q, k, self.v[s].double(), self.alpha[s].double(),
                                 self.beta[s].double(), ends)
            self.near(self.y[s].double().transpose(0, 1), y.transpose(0, 1), TOL_Y, f"y of request {r}")
            tol = TOL_S + (TOL_BF16 if self.prec == "shared_bf16" else 0)
            self.near(got[row].double(), S, tol, f"state of request {r}")
            if self.prec == "two":
                assert torch.equal(self.layer.checkpoint_lp_f32()[row], got[row].bfloat16().float())
            for i, e in enumerate(ends):
                slot = int(self.free[cub[r] + i])
                touched.add(slot)
                self.near(self.pool[slot].double(), kept[e], tol, f"block {i} of request {r}")
            at += n
        for slot in range(self.pool.shape[0]):
            if slot not in touched and not skip:
                assert torch.equal(self.pool[slot], self.pool0[slot])
        p = self.layer.pointers()
        assert not p["h"].any() and not p["nd"].any()

    def near(self, got, ref, tol, what):
        e = (got - ref).flatten(1).norm(dim=1)
        m = ref.flatten(1).norm(dim=1)
        assert bool((e <= tol * m + 1e-30).all()), f"{what}: {(e / m).tolist()}"


LENGTHS = [1, 0, 2, 15, 16, 17, 31, 63, 64, 65, 129, 200, 0]


@pytest.mark.parametrize("H,G,d,prec,fused", [
    (4, 2, 128, "fp32", True), (3, 3, 128, "two", False), (4, 1, 128, "shared_bf16", True), (32, 16, 128, "fp32", True),
    (4, 2, 64, "fp32", False), (6, 2, 64, "two", True), (5, 5, 64, "shared_bf16", True)])
def test_gdn_shapes(H, G, d, prec, fused):
    c = Case(LENGTHS, H, G, d, prec, fused=fused, seed=H)
    c.run()  # continues the layer's checkpoint
    c.check()
    assert c.layer.status() == 0


@pytest.mark.parametrize("n", [1, 3, 7, 8, 9, 24, 33, 127, 128, 192, 1000])
@pytest.mark.parametrize("d", [64, 128])
def test_gdn_one_request(n, d):
    c = Case([n], 2, 1, d, seed=n)
    c.run([-1])
    c.check()


@pytest.mark.parametrize("context", [0, 1, 63, 64, 100])
def test_gdn_starts_and_blocks(context):
    lengths = [64, 1, 63, 130, 300, 65, 2]
    c = Case(lengths, 4, 2, 64, context=[context] * len(lengths), block=64, seed=context)
    c.run([-1, 0, -2, 3, 1, -2, -1])
    c.check()


@pytest.mark.parametrize("prec", ["two", "shared_bf16"])
def test_gdn_blocks_of_other_precisions(prec):
    lengths = [200, 5, 400]
    c = Case(lengths, 4, 4, 128, prec, context=[128, 250, 0], block=128, seed=3)
    c.run([0, 1, -1])
    c.check()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lengths,start,prec,block", [
    ([2600], [-1], "fp32", 0), ([2600], [-2], "fp32", 256), ([3000, 1, 700, 2100], [-2, -1, 0, 1], "two", 512),
    ([2113, 64], [0, -2], "shared_bf16", 64)])
def test_gdn_long_requests(d, lengths, start, prec, block):
    """Few chains of many chunks: these run in segments."""
    c = Case(lengths, 2, 1, d, prec, context=[37] + [0] * (len(lengths) - 1), block=block, seed=len(lengths) + d, alpha="slow")
    c.run(start)
    c.check()
    assert c.layer.status() == 0


@pytest.mark.parametrize("alpha,beta,keys", [
    ("one", "mixed", "unit"), ("zeros", "mixed", "unit"), ("tiny", "one", "unit"), ("one", "one", "same"),
    ("mixed", "zero", "unit"), ("zeros", "one", "same")])
def test_gdn_extreme_gates(alpha, beta, keys):
    """Decays of one, of nothing and of 1e-30, full and no writes, one key all along."""
    c = Case([200, 64, 5, 70], 4, 2, 128, alpha=alpha, beta=beta, keys=keys, seed=11)
    c.run()
    c.check()


def test_gdn_keys_of_other_sizes():
    """Keys and values far from unit size (and rows of very different sizes in
    one chunk): alpha and beta keep the rule stable."""
    c = Case([150, 9], 4, 2, 128, seed=5)
    n = c.cap
    size = torch.exp2(torch.randint(-12, 1, (n, 1, 1), device="cuda").float())
    c.k.copy_((c.k.float() * size).bfloat16())
    c.v.copy_((c.v.float() * 2.0 ** 20).bfloat16())
    c.q.copy_((c.q.float() * 2.0 ** -20).bfloat16())
    c.run([-1, -1])
    c.check()


def test_gdn_bad_values_stay_in_their_request():
    lengths = [70, 40, 3, 90, 1, 2]
    clean = Case(lengths, 4, 2, 128, seed=2)
    clean.run()
    c = Case(lengths, 4, 2, 128, seed=2)
    at = np.cumsum([0] + lengths)
    c.v[at[1] + 5] = float("nan")
    c.k[at[3] + 64] = float("inf")
    c.alpha[at[4]] = float("nan")
    c.run()
    for r in (0, 2, 5):
        assert torch.equal(c.y[at[r]:at[r + 1]], clean.y[at[r]:at[r + 1]])
        row = int(c.rows[r])
        assert torch.equal(c.state()[row], clean.state()[row])
    for r in (1, 3, 4):
        assert not bool(c.state()[int(c.rows[r])].isfinite().all())
    assert bool(c.y[at[3]:at[3] + 64].isfinite().all())  # chunks before the bad row


def test_gdn_same_bits_again():
    """No result depends on the order of atomics or on what ran before."""
    outs = []
    for _ in range(2):
        c = Case(LENGTHS, 8, 4, 128, seed=9)
        c.run()
        outs.append((c.y, c.state().clone()))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


def test_gdn_spare_rows_and_other_stream():
    c = Case([33, 64, 5], 4, 2, 64, spare=77, seed=4)
    y = torch.full((c.cap, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    work = c.layer.prefill_workspace(c.rg, 64)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    c.run(y=y, work=work, stream=st)
    st.synchronize()
    c.check()
    assert bool((c.y[sum(c.lengths):] == 7).all())


def test_gdn_captured_in_a_graph():
    """The three calls in one graph, replayed on other lengths of the same capacity."""
    c = Case([100, 28], 4, 2, 64, seed=6)
    lengths = dev(np.array([100, 28], np.int32))
    start = dev(np.array([-1, -1], np.int32))
    y, work = torch.empty_like(c.v, memory_format=torch.contiguous_format), c.layer.prefill_workspace(c.rg, 128)

    def step():
        c.rg.plan(lengths)
        c.layer.prefill(c.rg, c.q, c.k, c.v, c.alpha, c.beta, max_len=128, rows=c.rows, start=start, y=y, work=work)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for lens in ([100, 28], [1, 127], [0, 64], [128, 0]):
        lengths.copy_(dev(np.array(lens, np.int32)))
        c.layer.init(c.S0)
        g.replay()
        torch.cuda.synchronize()
        c.lengths, c.start, c.y, c.pool0 = lens, [-1, -1], y, c.pool.clone()
        c.check()


def test_gdn_status_bits():
    c = Case([5, 6, 7, 8, 9, 10], 4, 2, 64, seed=8)
    before = c.layer.checkpoint_hp().clone()
    c.layer.h[int(c.rows[1])] = 2       # records buffered
    c.layer.nd[int(c.rows[2])] = 1      # drafts pending
    c.rows[3] = 8                       # no such row (B = 8)
    c.run([-2, -2, -2, -2, 99, -2], max_len=9)
    assert c.layer.status() == rb.DEV_RECORDS | rb.DEV_SLOT | rb.DEV_LENGTH
    c.layer.h.zero_(), c.layer.nd.zero_()
    for r in (1, 2, 4, 5):  # a refused request leaves its row alone
        assert torch.equal(c.layer.checkpoint_hp()[int(c.rows[r])], before[int(c.rows[r])])
    c.rows[3] = c.rows[0]
    c.lengths[3] = 8
    c.check(skip=(1, 2, 3, 4, 5))


def test_gdn_fresh_start_drops_records_and_decode_goes_on():
    """Prefill, then decode steps from the same state, against the oracle."""
    H, G, d, n = 4, 2, 64, 100
    c = Case([n, n], H, G, d, seed=12, B=2)
    c.rows = dev(np.array([0, 1], np.int32))
    c.layer.h.fill_(3), c.layer.base.fill_(2)
    c.run([-1, -1])
    c.check()
    model = oracle.Model("gdn", np.zeros((2, H, d, d), np.float32), {})
    bits = lambda t: t.view(torch.int16).cpu().numpy().view(np.uint16)
    pair = lambda t, i: t[[i, n + i]].contiguous()
    for i in range(n):
        model.step(dict(q=bits(pair(c.q, i)), k=bits(pair(c.k, i)), v=bits(pair(c.v, i)),
                        alpha=pair(c.alpha, i).cpu().numpy(), beta=pair(c.beta, i).cpu().numpy()))
    for i in range(20):  # crosses a fold
        x = {k: pair(getattr(c, k), i) for k in ("q", "k", "v", "alpha", "beta")}
        y = c.layer.decode(x, {}).cpu().numpy()
        ref = model.step({k: (bits(t) if k in "qkv" else t.cpu().numpy()) for k, t in x.items()})
        assert np.max(np.abs(y - ref)) <= 2e-3 * np.max(np.abs(ref))


def test_gdn_offsets_past_32_bits():
    """Row strides and pool slots whose offsets pass 2^31 elements."""
    H, G, d = 2, 2, 128
    T, ld = 130, 1 << 24
    c = Case([T - 2, 2], H, G, d, fused=False, seed=1)
    for name, heads in (("q", G), ("k", G), ("v", H)):
        x = getattr(c, name)
        big = torch.empty(T * ld, dtype=torch.bfloat16, device="cuda").view(T, ld)[:, :heads * d].unflatten(1, (heads, d))
        big.copy_(x)
        setattr(c, name, big)
    slots = (1 << 31) // (H * d * d) + 2
    small = c.pool
    c.pool = torch.empty(slots, H, d, d, device="cuda")
    c.pool[-1], c.pool[0] = small[0], small[1]
    start = dev(np.array([slots - 1, 0], np.int32))
    y = c.layer.prefill(c.rg, c.q, c.k, c.v, c.alpha, c.beta, max_len=T, rows=c.rows, start=start, pool=c.pool)
    c.pool0, c.pool, c.start, c.y = small, small, [0, 1], y
    c.check()


def test_gdn_scratch_needs_no_clearing():
    """Whatever the workspace held before, also where segments are joined."""
    for lengths in ([200, 64, 13], [3000]):
        outs = []
        for fill in (0, 255):
            c = Case(lengths, 2, 1, 128, seed=1)
            work = c.layer.prefill_workspace(c.rg, max(lengths))
            work.fill_(fill)
            c.run([-1] * len(lengths), work=work)
            outs.append((c.y, c.state().clone()))
        assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


@pytest.mark.parametrize("R,H,n", [(20, 16, 150), (10, 32, 20), (80, 32, 40)])
def test_gdn_many_chains_back_to_back(R, H, n):
    """Enough chains for the scan to start before the launch ahead of it ends, with short requests among
    them, called twice in a row and from a graph, results read by the next kernel on the stream."""
    rng = np.random.default_rng(R)
    lengths = [int(x) for x in rng.integers(0, n, R)]
    lengths[0] = 1
    c = Case(lengths, H, H // 2, 64 if R == 10 else 128, seed=R)
    start = [-1] * R
    c.run(start)
    first = (c.y.clone(), c.state().clone())
    c.check()
    work = c.layer.prefill_workspace(c.rg, n)
    st, y = dev(np.array(start, np.int32)), torch.empty_like(c.y)
    call = lambda: c.layer.prefill(c.rg, c.q, c.k, c.v, c.alpha, c.beta, max_len=n, rows=c.rows, start=st, pool=c.pool, y=y, work=work)
    call()
    call()
    assert torch.equal(y, first[0]) and torch.equal(c.state(), first[1])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
        twice = y + y
    y.zero_()
    c.layer.ckpt_hp.zero_()
    g.replay()
    torch.cuda.synchronize()
    for r, m in enumerate(lengths):
        if m:
            assert torch.equal(c.state()[int(c.rows[r])], first[1][int(c.rows[r])])
    assert torch.equal(y, first[0]) and torch.equal(twice, first[0] + first[0])


def test_gdn_only_short_requests_where_long_ones_may_come():
    """max_len allows chunks, no request has one: the recurrence alone, seen by the next kernel."""
    c = Case([1, 3, 12, 0, 7] * 20, 16, 8, 128, seed=2)
    y = c.run(max_len=500)
    twice = y + y
    torch.cuda.synchronize()
    c.check()
    assert torch.equal(twice, c.y + c.y)


def test_example_runs():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "prefill_decode.py")
    spec = importlib.util.spec_from_file_location("prefill_decode", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    out = m.main()
    assert out["taken"] == 2 + 0 + 5 + 1
    assert out["prefix"] <= 2 * TOL_S       # two states within the tolerance of the same one
    assert out["step"] <= TOL_Y + 2e-3      # a bf16 row against decode's fp32 one
