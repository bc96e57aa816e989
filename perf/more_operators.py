"""The training-side operators' cases: attention over whole sequences with its backward
pass, and dropout (with the residual's addition) whose mask is never stored.

``run`` computes a case in plain torch operations (``own`` false) or through the
library's entry points (``own`` true); ``exact`` is the definition in 64 bits.

Lengths of a ragged batch follow from the case alone (spread evenly between the
smallest and the largest); values and random keys come from the seed.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}


# ---------------------------------------------------------------- cases

def _attend(name, **kw):
    # k_min, k_max 0: self-attention, the keys are the queries' own tokens
    c = dict(op="attend", step="bwd", batch=1, q_min=1, q_max=1, k_min=0, k_max=0, heads=32,
             kv_heads=8, dim=128, dtype="bf16", causal=True, window=0)
    return {"name": name, **c, **kw}


def _dropout(name, **kw):
    c = dict(op="dropout", step="fwd", rows=1, hidden=4096, p=0.1, dtype="bf16", residual=True)
    return {"name": name, **c, **kw}


def listed():
    return [
        # the backward pass of a training batch, heads that share keys
        _attend("attend bwd train", batch=2, q_min=4096, q_max=4096),
        # documents of different lengths packed into one row, small heads, a sliding window
        _attend("attend bwd documents", batch=9, q_min=17, q_max=3001, heads=16, kv_heads=4,
                dim=64, dtype="f16", window=1000),
        # a small encoder's batch of short texts: latency
        _attend("attend bwd encoder", batch=4, q_min=128, q_max=128, heads=8, kv_heads=8, dim=64,
                dtype="f16", causal=False),
        # a decoder's queries over an encoder's output, ragged on both sides
        _attend("attend bwd cross", batch=7, q_min=3, q_max=509, k_min=211, k_max=1500, heads=12,
                kv_heads=12, dim=96, causal=False),
        # one long document
        _attend("attend bwd long", q_min=16384, q_max=16384, heads=8, kv_heads=2),
        # forward and backward of a training batch, every head with its own keys
        _attend("attend step train", step="both", batch=4, q_min=2048, q_max=2048, heads=16,
                kv_heads=16),
        # forward and backward of short packed sequences
        _attend("attend step short", step="both", batch=24, q_min=1, q_max=200, heads=8,
                kv_heads=2, dim=80, dtype="f16"),
        # the output of a block's last projection on its way into the residual stream
        _dropout("dropout add train", rows=16384),
        # its gradient
        _dropout("dropout bwd train", step="bwd", rows=16384),
        # the same of a small fp32 network: latency
        _dropout("dropout add small", rows=64, hidden=1024, dtype="f32"),
        # embeddings, odd sizes
        _dropout("dropout odd", rows=1021, hidden=4001, p=0.5, dtype="f16", residual=False),
        # a gradient in fp32, wide rows
        _dropout("dropout bwd f32", step="bwd", rows=4096, hidden=5120, p=0.25, dtype="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cost(case):
    w = work(case)
    return max(w["bytes"] / 6.8e12, w["flops"] / 1.9e15)


def draw(rng):
    if rng.random() < 0.3:
        step = rng.choice(["fwd", "bwd"])
        c = _dropout("", step=step, rows=_log(rng, 1, 16384), hidden=_log(rng, 64, 8192),
                     p=rng.choice([0.1, 0.05, 0.2, 0.5, 0.9]),
                     dtype=rng.choice(["bf16", "bf16", "f16", "f32"]),
                     residual=step == "fwd" and rng.random() < 0.7)
        most, small = _cost(listed()[7]), "rows"
    else:
        kv = rng.choice([1, 2, 4, 8])
        cross = rng.random() < 0.25
        q_max = _log(rng, 1, 8192)
        q_min = rng.choice([q_max, rng.randint(1, q_max)])
        batch = _log(rng, 1, max(1, min(64, 32768 // q_max)))
        k_max = _log(rng, 1, 4096) if cross else 0
        c = _attend("", step=rng.choice(["bwd", "bwd", "both"]), batch=batch, q_min=q_min,
                    q_max=q_max, k_min=rng.randint(1, k_max) if cross else 0, k_max=k_max,
                    heads=kv * rng.choice([1, 1, 2, 4, 5]), kv_heads=kv,
                    dim=rng.choice([128, 128, 64, 64, 96, 80, 32]),
                    dtype=rng.choice(["bf16", "bf16", "f16"]),
                    causal=not cross and rng.random() < 0.8,
                    window=rng.choice([0, 0, 0, 500]) if not cross else 0)
        most, small = _cost(listed()[4]), "batch"
    del c["name"]
    while _cost(c) > most and c[small] > 1:
        c[small] = max(1, c[small] * 3 // 4)
    if c["op"] == "attend":  # the plain form holds a sequence's whole score matrices
        while _cost(c) > most or c["heads"] * c["q_max"] * max(c["q_max"], c["k_max"]) > 2.2e9:
            c["q_max"] = c["q_max"] * 3 // 4
            c["q_min"] = min(c["q_min"], c["q_max"])
    return c


# ---------------------------------------------------------------- lengths and work

def _spread(lo, hi, n, step):
    """n whole numbers between lo and hi, both among them (n > 1), in a mixed order."""
    if n == 1:
        return [hi]
    while math.gcd(step, n) != 1:
        step += 1
    return [lo + (hi - lo) * (i * step % n) // (n - 1) for i in range(n)]


def _lengths(case):
    """Queries and keys of each sequence."""
    q = _spread(case["q_min"], case["q_max"], case["batch"], 7)
    return q, _spread(case["k_min"], case["k_max"], case["batch"], 3) if case["k_max"] else q


def _uniform(case):
    return not case["k_max"] and case["q_min"] == case["q_max"]


def _range(nq, nk, case, i):
    """First and last key + 1 that queries i (int64) of a sequence keep."""
    at = i + (nk - nq)
    high = (at + 1).clamp(0, nk) if case["causal"] else torch.full_like(i, nk)
    low = (at - case["window"] + 1).clamp(0, nk) if case["window"] else torch.zeros_like(i)
    return low, high


def _pairs(case):
    total = 0
    for nq, nk in zip(*_lengths(case)):
        low, high = _range(nq, nk, case, torch.arange(nq))
        total += int((high - low).clamp(min=0).sum())
    return total


def work(case):
    e = SIZE[case["dtype"]]
    if case["op"] == "dropout":
        n = case["rows"] * case["hidden"]
        # ten rounds of two products and four bitwise operations for four elements
        return {"bytes": n * e * (3 if case["residual"] and case["step"] == "fwd" else 2) + 16,
                "flops": n * 17}
    q, k = _lengths(case)
    tq, tk, h, hk, d = sum(q), sum(k), case["heads"], case["kv_heads"], case["dim"]
    q_bytes, k_bytes = tq * h * d * e, tk * hk * d * e
    pairs = _pairs(case)
    bytes_ = 4 * q_bytes + 4 * k_bytes + 4 * tq * h  # q, out, dout, lse, k, v; dq, dk, dv
    if not _uniform(case):
        bytes_ += 8 * (case["batch"] + 1)
    if case["step"] == "both":  # out and lse are results: written, then read
        bytes_ += 2 * q_bytes + 2 * k_bytes + 4 * tq * h
        return {"bytes": bytes_, "flops": 14 * pairs * h * d}
    return {"bytes": bytes_, "flops": 10 * pairs * h * d}


# ---------------------------------------------------------------- inputs

def _normal(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * std).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(1000003 * (seed + 1) + 23)
    dt = DT[case["dtype"]]
    s = dict(case)
    if case["op"] == "dropout":
        shape = (case["rows"], case["hidden"])
        s["x"] = _normal(g, shape, dt)  # (a step backward: the output's gradient)
        s["r"] = _normal(g, shape, dt, 2.0) if case["residual"] and case["step"] == "fwd" else None
        # the generator's key, and how often it was used before
        s["rng"] = torch.randint(0, 1 << 62, (2,), generator=g, device="cuda")
        return s
    q, k = _lengths(case)
    h, hk, d = case["heads"], case["kv_heads"], case["dim"]
    if case["k_max"]:
        s["q"] = _normal(g, (sum(q), h, d), dt)
        s["k"], s["v"] = _normal(g, (sum(k), 2 * hk, d), dt).split([hk, hk], dim=1)
    else:  # views of one projection's output
        lead = (case["batch"], case["q_max"]) if _uniform(case) else (sum(q),)
        s["q"], s["k"], s["v"] = _normal(g, (*lead, h + 2 * hk, d), dt).split([h, hk, hk], dim=-2)
    # f16 gradients carry a loss scale
    s["dout"] = _normal(g, s["q"].shape, dt, 1.0 if case["dtype"] == "f16" else 0.02)
    s["q_lens"], s["k_lens"] = q, k
    s["max_q"], s["max_k"] = max(q), max(k)
    s["cu_q"] = s["cu_k"] = None
    if not _uniform(case):
        s["cu_q"], s["cu_k"] = (torch.tensor([0, *n], device="cuda").cumsum(0).to(torch.int32)
                                for n in (q, k))
    if case["step"] == "bwd":
        s["out"], s["lse"] = _plain_forward(s)
    return s


# ---------------------------------------------------------------- plain forms

def _sequences(s):
    """Slices of the packed queries and keys."""
    a = b = 0
    for nq, nk in zip(s["q_lens"], s["k_lens"]):
        yield slice(a, a + nq), slice(b, b + nk)
        a, b = a + nq, b + nk


def _flat(x):
    return x.flatten(0, 1) if x.dim() == 4 else x


def _by_kv_head(x, hk):
    """[n, heads, d] as [kv heads, group * n, d] in 32 bits."""
    n, h, d = x.shape
    return x.float().view(n, hk, h // hk, d).permute(1, 2, 0, 3).reshape(hk, -1, d)


def _back(y, n):
    """[kv heads, group * n, d] as [n, heads, d]."""
    hk, _, d = y.shape
    return y.view(hk, -1, n, d).permute(2, 0, 1, 3).reshape(n, -1, d)


def _plain_scores(q, k, nq, s):
    """Masked scores [kv heads, group * queries, keys]."""
    nk = k.shape[1]
    z = (q @ k.transpose(1, 2)).mul_(s["dim"] ** -0.5)
    low, high = _range(nq, nk, s, torch.arange(nq, device=q.device))
    j = torch.arange(nk, device=q.device)
    drop = (j < low[:, None]) | (j >= high[:, None])
    z.view(q.shape[0], -1, nq, nk).masked_fill_(drop, -math.inf)
    return z


def _plain_forward(s):
    hk = s["kv_heads"]
    q, k, v = _flat(s["q"]), _flat(s["k"]), _flat(s["v"])
    out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    lse = torch.empty(q.shape[:2], device=q.device)
    for a, b in _sequences(s):
        n = a.stop - a.start
        z = _plain_scores(_by_kv_head(q[a], hk), _by_kv_head(k[b], hk), n, s)
        top = z.amax(-1, keepdim=True)
        top = torch.where(top == -math.inf, 0.0, top)
        p = z.sub_(top).exp_()
        total = p.sum(-1, keepdim=True)
        o = (p @ _by_kv_head(v[b], hk)) / torch.where(total == 0, 1.0, total)
        out[a] = _back(o, n).to(out.dtype)
        lse[a] = _back(top + total.log(), n).squeeze(-1)
    return out.view(s["q"].shape), lse.view(s["q"].shape[:-1])


def _plain_backward(s, out, lse):
    hk, scale = s["kv_heads"], s["dim"] ** -0.5
    q, k, v, do, o = (_flat(x) for x in (s["q"], s["k"], s["v"], s["dout"], out))
    lse = lse.reshape(q.shape[:2])
    dq, dk, dv = (torch.empty(x.shape, dtype=x.dtype, device=x.device) for x in (q, k, v))
    for a, b in _sequences(s):
        n, m = a.stop - a.start, b.stop - b.start
        qf, kf, vf, df = (_by_kv_head(x, hk) for x in (q[a], k[b], v[b], do[a]))
        p = _plain_scores(qf, kf, n, s)
        norm = _by_kv_head(lse[a].unsqueeze(-1), hk)
        p = p.sub_(torch.where(norm == -math.inf, 0.0, norm)).exp_()
        dv[b] = _back(p.transpose(1, 2) @ df, m).to(dv.dtype)
        ds = df @ vf.transpose(1, 2)
        ds.sub_((df * _by_kv_head(o[a], hk)).sum(-1, keepdim=True)).mul_(p)
        dq[a] = _back(ds @ kf * scale, n).to(dq.dtype)
        dk[b] = _back(ds.transpose(1, 2) @ qf * scale, m).to(dk.dtype)
    return {n: g.view(s[n[1]].shape) for n, g in (("dq", dq), ("dk", dk), ("dv", dv))}


def _mul_hi_lo(a, b):
    """The two 32-bit halves of products of 32-bit numbers held in int64 (which wrap)."""
    r = a * b
    return (r >> 32) & 0xFFFFFFFF, r & 0xFFFFFFFF


def _plain_words(n, rng):
    """32 random bits for each of n elements: element e takes word e % 4 of Philox 4x32-10
    (Salmon et al., 2011) of counter (e / 4, rng[1]) and key rng[0]."""
    i = torch.arange((n + 3) // 4, device=rng.device)
    low, high = rng & 0xFFFFFFFF, (rng >> 32) & 0xFFFFFFFF
    c = [i & 0xFFFFFFFF, i >> 32, low[1], high[1]]
    k0, k1 = low[0], high[0]
    for _ in range(10):
        h0, l0 = _mul_hi_lo(c[0], 0xD2511F53)
        h1, l1 = _mul_hi_lo(c[2], 0xCD9E8D57)
        c = [h1 ^ c[1] ^ k0, l1, h0 ^ c[3] ^ k1, l0]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return torch.stack(c, -1).flatten()[:n]


def _plain_dropout(s):
    x = s["x"]
    least = math.ceil(s["p"] * 2.0 ** 32)  # of the words that keep their element
    keep = (_plain_words(x.numel(), s["rng"]) >= least).view(x.shape)
    y = torch.where(keep, x.float() * (1.0 / (1.0 - s["p"])), 0.0)
    if s["r"] is not None:
        y += s["r"].float()
    return y.to(x.dtype)


# ---------------------------------------------------------------- the pass

def run(state):
    s = state
    if own:
        from rmsnorm_fp8_quantization_gb300 import ops
        if s["op"] == "dropout":
            if s["step"] == "bwd":
                return ops.dropout_bwd(s["x"], s["p"], s["rng"])
            return ops.dropout_fwd(s["x"], s["p"], s["rng"], residual=s["r"])
        kw = dict(causal=s["causal"], window=s["window"])
        if s["cu_q"] is not None:
            kw.update(cu_seqlens=s["cu_q"], max_q=s["max_q"])
            if s["k_max"]:
                kw.update(cu_seqlens_k=s["cu_k"], max_k=s["max_k"])
        if s["step"] == "bwd":
            out, lse = s["out"], s["lse"]
        else:
            out, lse = ops.attention_fwd(s["q"], s["k"], s["v"], **kw)
        dq, dk, dv = ops.attention_bwd(s["dout"], s["q"], s["k"], s["v"], out, lse, **kw)
        r = {"dq": dq, "dk": dk, "dv": dv}
        return r if s["step"] == "bwd" else {"out": out, "lse": lse, **r}
    if s["op"] == "dropout":
        return _plain_dropout(s)
    if s["step"] == "bwd":
        return _plain_backward(s, s["out"], s["lse"])
    out, lse = _plain_forward(s)
    return {"out": out, "lse": lse, **_plain_backward(s, out, lse)}


# ---------------------------------------------------------------- the definition in 64 bits

def _product_halves(a, b):
    """(high, low) 32 bits of a * b, both 32-bit numbers in int64, by 16-bit digits."""
    a1, a0, b1, b0 = a // 65536, a % 65536, b // 65536, b % 65536
    mid = a1 * b0 + (a0 * b0) // 65536
    mid2 = a0 * b1 + mid % 65536
    return a1 * b1 + mid // 65536 + mid2 // 65536, mid2 % 65536 * 65536 + a0 * b0 % 65536


def _exact_words(n, seed, offset):
    count = -(-n // 4)
    x = torch.arange(count, dtype=torch.int64, device="cuda")
    word = 2 ** 32
    x0, x1 = x % word, x // word
    x2, x3 = torch.full_like(x, offset % word), torch.full_like(x, offset // word % word)
    for r in range(10):
        key = ((seed % word + r * 0x9E3779B9) % word, (seed // word + r * 0xBB67AE85) % word)
        ha, la = _product_halves(x0, 0xD2511F53)
        hb, lb = _product_halves(x2, 0xCD9E8D57)
        x0, x1, x2, x3 = hb ^ x1 ^ key[0], lb, ha ^ x3 ^ key[1], la
    out = torch.empty(count, 4, dtype=torch.int64, device="cuda")
    for i, v in enumerate((x0, x1, x2, x3)):
        out[:, i] = v
    return out.reshape(-1)[:n]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "dropout":
        u = _exact_words(s["x"].numel(), *s["rng"].tolist()).double() / 2.0 ** 32
        y = s["x"].double() / (1.0 - case["p"])
        y[(u < case["p"]).view(y.shape)] = 0.0
        return y if s["r"] is None else y + s["r"].double()
    h, hk, d = case["heads"], case["kv_heads"], case["dim"]
    q, k, v, do = (s[n].reshape(-1, s[n].shape[-2], d) for n in ("q", "k", "v", "dout"))
    r = {"out": torch.zeros(q.shape, dtype=torch.float64, device="cuda"),
         "lse": torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device="cuda")}
    for n, x in (("dq", q), ("dk", k), ("dv", v)):
        r[n] = torch.zeros(x.shape, dtype=torch.float64, device="cuda")
    a = b = 0
    for nq, nk in zip(*_lengths(case)):
        back = (torch.arange(nk - nq, nk, device="cuda")[:, None]
                - torch.arange(nk, device="cuda"))  # how far key j lies behind query i
        drop = torch.zeros_like(back, dtype=torch.bool)
        if case["causal"]:
            drop |= back < 0
        if case["window"]:
            drop |= back >= case["window"]
        for n in range(h):
            g = n // (h // hk)
            qn, kn, vn, dn = q[a:a + nq, n].double(), k[b:b + nk, g].double(), \
                v[b:b + nk, g].double(), do[a:a + nq, n].double()
            z = qn @ kn.T / math.sqrt(d)
            z[drop] = -math.inf
            norm = torch.logsumexp(z, 1)
            some = norm > -math.inf
            w = torch.exp_(z.sub_(torch.where(some, norm, 0.0)[:, None]))
            r["lse"][a:a + nq, n] = norm
            r["out"][a:a + nq, n] = w @ vn
            r["dv"][b:b + nk, g] += w.T @ dn
            dw = dn @ vn.T
            dz = w.mul_(dw.sub_((w * dw).sum(1, keepdim=True)))
            r["dq"][a:a + nq, n] = dz @ kn / math.sqrt(d)
            r["dk"][b:b + nk, g] += dz.T @ qn / math.sqrt(d)
        a, b = a + nq, b + nk
    names = ("dq", "dk", "dv") if case["step"] == "bwd" else ("out", "lse", "dq", "dk", "dv")
    of = {"out": "q", "dq": "q", "dk": "k", "dv": "v"}
    return {n: r[n].view(s[of[n]].shape if n in of else s["q"].shape[:-1]) for n in names}
