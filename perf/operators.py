"""The attention-side operators' cases: rotary positions, the paged cache's append,
and the attention of a chunk of new tokens over that cache.

``run`` computes a case in plain torch operations (``own`` false) or through the
library's entry points (``own`` true); ``exact`` is the definition in 64 bits.

Lengths of a ragged batch follow from the case alone (spread evenly between the
smallest and the largest); values, page order and positions come from the seed.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32,
      "e4m3": torch.float8_e4m3fn}
SIZE = {"bf16": 2, "f16": 2, "f32": 4, "e4m3": 1}


# ---------------------------------------------------------------- cases

def _rope(name, **kw):
    c = dict(op="rope", direction="fwd", batch=1, seq=1, heads=32, kv_heads=8, dim=128, rotary=128,
             layout="half", dtype="bf16", packed=False, far=0, mscale=1.0)
    return {"name": name, **c, **kw}


def _append(name, **kw):
    c = dict(op="append", batch=1, q_min=1, q_max=1, kv_min=1, kv_max=1, heads=32, kv_heads=8,
             dim=128, rotary=128, layout="half", dtype="bf16", cache="bf16", page=16, mscale=1.0)
    return {"name": name, **c, **kw}


def _attend(name, **kw):
    c = dict(op="attend", batch=1, q_min=1, q_max=1, kv_min=1, kv_max=1, heads=32, kv_heads=8,
             dim=128, dtype="bf16", cache="bf16", page=16, causal=True, window=0, lse=False)
    return {"name": name, **c, **kw}


def listed():
    return [
        # one new token of each of 32 running sequences, deep in their contexts
        _rope("rope step", batch=32, far=131072),
        # a training batch
        _rope("rope train", batch=4, seq=4096),
        # its gradient, in a network that rotates half of each head in neighbouring pairs, keeps
        # fp32, and hands over views of one packed projection; odd lengths
        _rope("rope train bwd", direction="bwd", batch=3, seq=1021, heads=12, kv_heads=12, dim=96,
              rotary=48, layout="interleaved", dtype="f32", packed=True, mscale=1.25),
        # one new token of each of 64 running sequences
        _append("append step", batch=64, kv_min=1, kv_max=2000),
        # prompts of different lengths that enter together, some behind a shared prefix
        _append("append prompts", batch=12, q_min=37, q_max=1500, kv_min=300, kv_max=2100, page=64),
        # the same into an eight-bit cache, small heads
        _append("append prompts e4m3", batch=9, q_min=5, q_max=1111, kv_min=1111, kv_max=1700,
                heads=16, kv_heads=4, dim=64, rotary=32, layout="interleaved", dtype="f16",
                cache="e4m3", page=32, mscale=1.1),
        # a few short conversations, one token each: latency
        _attend("step few short", batch=4, kv_min=1, kv_max=700, heads=8, kv_heads=8, dim=64,
                dtype="f16", cache="f16"),
        # a full batch of one token each
        _attend("step batch", batch=64, kv_min=2000, kv_max=16000),
        # one long document in an eight-bit cache, one token
        _attend("step long e4m3", kv_min=262144, kv_max=262144, cache="e4m3", page=64),
        # a few tokens at once to be verified, under a sliding window
        _attend("verify window", batch=24, q_min=1, q_max=6, kv_min=100, kv_max=9000, heads=16,
                kv_heads=2, dim=64, dtype="f16", cache="f16", page=32, window=4096, lse=True),
        # chunks of prompts next to running sequences
        _attend("chunks mixed", batch=5, q_min=1, q_max=1500, kv_min=1500, kv_max=8000),
        # a whole prompt
        _attend("prompt", q_min=8192, q_max=8192, kv_min=8192, kv_max=8192, page=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cost(case):
    w = work(case)
    return max(w["bytes"] / 6.8e12, w["flops"] / 1.9e15)


def draw(rng):
    op = rng.choice(["rope", "append", "attend", "attend"])
    group = rng.choice([1, 2, 4, 5, 8])
    if op == "rope":
        kv = rng.choice([1, 2, 4, 8, 12])
        dim = rng.choice([64, 80, 96, 128, 256])
        tokens = _log(rng, 1, 16384)
        batch = _log(rng, 1, min(tokens, 64))
        c = _rope("", direction=rng.choice(["fwd", "bwd"]), batch=batch,
                  seq=max(1, tokens // batch), heads=kv * group, kv_heads=kv, dim=dim,
                  rotary=rng.choice([dim, dim // 2]), layout=rng.choice(["half", "interleaved"]),
                  dtype=rng.choice(["bf16", "bf16", "f16", "f32"]),
                  packed=rng.random() < 0.5, far=rng.choice([0, 4000, 1000000]),
                  mscale=rng.choice([1.0, 1.2]))
        most = _cost(listed()[1])
    else:
        kv = rng.choice([1, 2, 4, 8])
        dtype = rng.choice(["bf16", "bf16", "f16"])
        common = dict(heads=kv * group, kv_heads=kv, dtype=dtype,
                      cache=rng.choice([dtype, dtype, "e4m3"]), page=rng.choice([16, 32, 64, 128]))
        if op == "append":
            dim = rng.choice([64, 96, 128, 256])
            q_max = rng.choice([1, _log(rng, 1, 4000)])
            batch = _log(rng, 1, max(1, min(256, 16000 // q_max)))
            kv_max = q_max + _log(rng, 1, 4000)
            c = _append("", batch=batch, q_min=rng.randint(1, q_max), q_max=q_max,
                        kv_min=rng.randint(q_max, kv_max), kv_max=kv_max, dim=dim,
                        rotary=rng.choice([dim, dim // 2]),
                        layout=rng.choice(["half", "interleaved"]),
                        mscale=rng.choice([1.0, 1.2]), **common)
            most = _cost(listed()[4])
        else:
            kind = rng.choice(["step", "few", "chunks"])
            q_max = {"step": 1, "few": rng.randint(2, 16), "chunks": _log(rng, 17, 3000)}[kind]
            kv_max = q_max + _log(rng, 16, 100000 if kind != "chunks" else 6000)
            batch = _log(rng, 1, 64 if kind != "chunks" else 6)
            c = _attend("", batch=batch, q_min=rng.randint(1, q_max), q_max=q_max,
                        kv_min=rng.randint(max(q_max, kv_max // 4), kv_max), kv_max=kv_max,
                        dim=rng.choice([64, 128, 128, 80, 256]),
                        causal=rng.random() < 0.85, window=rng.choice([0, 0, 0, 1000]),
                        lse=rng.random() < 0.3, **common)
            most = _cost(listed()[7])
    del c["name"]
    small = {"rope": "seq"}.get(op, "batch")
    while _cost(c) > most and c[small] > 1:
        c[small] = max(1, c[small] * 3 // 4)
    if op == "attend":  # the plain form holds whole score matrices
        while c["batch"] * c["heads"] * c["q_max"] * c["kv_max"] > 2.2e9 and c["batch"] > 1:
            c["batch"] -= 1
        while _cost(c) > most or c["heads"] * c["q_max"] * c["kv_max"] > 2.2e9:
            c["kv_max"] = max(c["q_max"], c["kv_max"] * 3 // 4)
            c["kv_min"] = min(c["kv_min"], c["kv_max"])
            if c["kv_max"] == c["q_max"]:
                break
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
    """(new tokens, keys with them) of each sequence."""
    n = case["batch"]
    q = _spread(case["q_min"], case["q_max"], n, 7)
    kv = _spread(case["kv_min"], case["kv_max"], n, 3)
    return q, [max(a, b) for a, b in zip(q, kv)]


def _kept(case):
    """Kept (query, key) pairs of one head, and the keys that some query keeps."""
    pairs = keys = 0
    w = case["window"]
    for q, kv in zip(*_lengths(case)):
        off = kv - q
        first = kv
        for_all = 0
        if not case["causal"]:
            # query i keeps every key past off + i - w
            lows = range(off - w + 1, off - w + 1 + q) if w else ()
            for_all = q * kv - sum(max(0, x) for x in lows)
            first = max(0, off - w + 1) if w else 0
        else:
            full = q * off + q * (q + 1) // 2
            if w:
                # query i sees off + i + 1 keys, at most w of them
                m = min(q, max(0, w - off))  # queries that see no more than w
                for_all = m * off + m * (m + 1) // 2 + (q - m) * w
            else:
                for_all = full
            first = max(0, off - w + 1) if w else 0
        pairs += for_all
        keys += kv - first
    return pairs, keys


def work(case):
    e = SIZE[case["dtype"]]
    h, k, d = case["heads"], case["kv_heads"], case["dim"]
    if case["op"] == "rope":
        t = case["batch"] * case["seq"]
        return {"bytes": 2 * t * (h + k) * d * e + 8 * t + 4 * case["rotary"],
                "flops": 3 * t * (h + k) * case["rotary"]}
    q, kv = _lengths(case)
    t, n, c = sum(q), case["batch"], SIZE[case["cache"]]
    index = 4 * (2 * n + 1)
    if case["op"] == "append":
        pages = sum((b - 1) // case["page"] - (b - a) // case["page"] + 1 for a, b in zip(q, kv))
        return {"bytes": t * d * (2 * h * e + 2 * k * (e + c)) + index + 4 * pages + 4 * case["rotary"],
                "flops": 3 * t * (h + k) * case["rotary"]}
    pairs, keys = _kept(case)
    out = 2 * t * h * d * e + (4 * t * h if case["lse"] else 0)
    return {"bytes": out + 2 * keys * k * d * c + 4 * (keys // case["page"]) + index,
            "flops": 4 * pairs * h * d}


# ---------------------------------------------------------------- inputs

def _frequencies(rotary, base=500000.0, factor=8.0, original=8192):
    """Radians a position of each pair: a long context's, the slow pairs divided by ``factor``,
    the fast ones kept, a ramp between (by how often a pair turns within ``original``)."""
    i = torch.arange(rotary // 2, dtype=torch.float64)
    f = base ** (-2.0 * i / rotary)
    turns = original * f / (2 * math.pi)
    keep = ((turns - 1.0) / 31.0).clamp(0.0, 1.0)
    return (f * keep + f / factor * (1 - keep)).cuda()


def _normal(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * std).to(dtype)


def _heads(g, lead, heads, kv_heads, dim, dtype, packed, values):
    """q, k (and v) as tensors of their own, or as views of one projection's output."""
    if packed:
        x = _normal(g, (*lead, heads + 2 * kv_heads, dim), dtype)
        q, k, v = x.split([heads, kv_heads, kv_heads], dim=-2)
    else:
        q, k = _normal(g, (*lead, heads, dim), dtype), _normal(g, (*lead, kv_heads, dim), dtype)
        v = _normal(g, (*lead, kv_heads, dim), dtype) if values else None
    return q, k, v


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(1000003 * (seed + 1) + 17)
    dt, dev = DT[case["dtype"]], "cuda"
    s = dict(case)
    if case["op"] == "rope":
        b, n = case["batch"], case["seq"]
        s["q"], s["k"], _ = _heads(g, (b, n), case["heads"], case["kv_heads"], case["dim"], dt,
                                   case["packed"], False)
        start = torch.randint(0, case["far"] + 1, (b, 1), generator=g, device=dev)
        s["positions"] = start + torch.arange(n, device=dev)
        s["inv_freq"] = _frequencies(case["rotary"])
        return s
    q, kv = _lengths(case)
    page, k_heads, d = case["page"], case["kv_heads"], case["dim"]
    need = [-(-n // page) for n in kv]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    table = torch.full((case["batch"], max(need)), -1, dtype=torch.int32, device=dev)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    cu = [0]
    for n in q:
        cu.append(cu[-1] + n)
    s["cu_seqlens"] = torch.tensor(cu, dtype=torch.int32, device=dev)
    s["kv_lens"] = torch.tensor(kv, dtype=torch.int32, device=dev)
    s["block_table"] = table
    s["max_q"], s["max_kv"] = max(q), max(kv)
    cdt = DT[case["cache"]]
    shape = (pages, page, k_heads, d)
    gain = 24.0 if case["cache"] == "e4m3" else 1.0  # what the cache's values are multiplied by
    s["k_cache"] = _normal(g, shape, cdt, gain)
    s["v_cache"] = _normal(g, shape, cdt, gain)
    scale = torch.full((1,), gain, device=dev)
    s["k_scale"] = s["v_scale"] = scale if case["cache"] == "e4m3" else None
    s["k_scale_inv"] = s["v_scale_inv"] = 1.0 / scale if case["cache"] == "e4m3" else None
    if case["op"] == "append":
        s["q"], s["k"], s["v"] = _heads(g, (cu[-1],), case["heads"], k_heads, d, dt, True, True)
        s["inv_freq"] = _frequencies(case["rotary"])
    else:
        s["q"] = _normal(g, (cu[-1], case["heads"], d), dt)
    return s


# ---------------------------------------------------------------- plain forms

def _rotate(x, cos, sin, rotary, layout):
    """x [..., heads, dim] in 32 bits; cos, sin [..., 1, rotary / 2]."""
    y, rest = x[..., :rotary].float(), x[..., rotary:].float()
    if layout == "half":
        a, b = y[..., :rotary // 2], y[..., rotary // 2:]
        y = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    else:
        a, b = y[..., 0::2], y[..., 1::2]
        y = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    return torch.cat([y, rest], -1)


def _cos_sin(positions, inv_freq, mscale):
    """In 64 bits: the angles of far positions have no fraction left in 32."""
    angle = positions.double().unsqueeze(-1) * inv_freq
    return (mscale * angle.cos()).float().unsqueeze(-2), (mscale * angle.sin()).float().unsqueeze(-2)


def _plain_rope(s):
    cos, sin = _cos_sin(s["positions"], s["inv_freq"], s["mscale"])
    if s["direction"] == "bwd":
        sin = -sin
    return {n: _rotate(s[n], cos, sin, s["rotary"], s["layout"]).to(s[n].dtype) for n in ("q", "k")}


def _where(s):
    """Each new token's sequence, and its place among that sequence's keys."""
    cu = s["cu_seqlens"].long()
    t = torch.arange(s["q"].shape[0], device=cu.device)
    seq = (t[:, None] >= cu[None, 1:]).sum(1)
    q_len = cu[1:] - cu[:-1]
    return seq, t - cu[seq], (s["kv_lens"].long() - q_len)[seq]


def _store(x, scale, dtype):
    if scale is None:
        return x.to(dtype)
    return (x * scale).clamp(-448.0, 448.0).to(dtype)


def _plain_append(s):
    seq, i, before = _where(s)
    pos = before + i
    cos, sin = _cos_sin(pos, s["inv_freq"], s["mscale"])
    q = _rotate(s["q"], cos, sin, s["rotary"], s["layout"]).to(s["q"].dtype)
    k = _rotate(s["k"], cos, sin, s["rotary"], s["layout"])
    page = s["block_table"][seq, pos // s["page"]].long()
    slot = pos % s["page"]
    as_bytes = (lambda x: x.view(torch.uint8)) if s["cache"] == "e4m3" else (lambda x: x)
    as_bytes(s["k_cache"])[page, slot] = as_bytes(_store(k, s["k_scale"], s["k_cache"].dtype))
    as_bytes(s["v_cache"])[page, slot] = as_bytes(_store(s["v"].float(), s["v_scale"], s["v_cache"].dtype))
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_attend(s):
    heads, kv_heads, d = s["heads"], s["kv_heads"], s["dim"]
    group, n, mq = heads // kv_heads, s["batch"], s["max_q"]
    cu, kv = s["cu_seqlens"].long(), s["kv_lens"].long()
    q_len = cu[1:] - cu[:-1]
    dev = cu.device
    table = s["block_table"].clamp(min=0).long()
    length = table.shape[1] * s["page"]
    j = torch.arange(length, device=dev)
    here = (j < kv[:, None])[:, None, :, None]  # [n, 1, length, 1]

    def keys(cache, scale_inv):  # [n, kv_heads, length, d]
        x = cache[table].reshape(n, length, kv_heads, d).float().transpose(1, 2)
        x = torch.where(here, x, 0.0)
        return x if scale_inv is None else x * scale_inv

    i = torch.arange(mq, device=dev)
    rows = (cu[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][rows].float().view(n, mq, kv_heads, group, d).permute(0, 2, 1, 3, 4)
    q = q.reshape(n, kv_heads, mq * group, d)
    scores = (q @ keys(s["k_cache"], s["k_scale_inv"]).transpose(-1, -2)) * d ** -0.5
    at = ((kv - q_len)[:, None] + i)[:, :, None]  # each query's own place
    keep = (j < kv[:, None, None]).expand(n, mq, length)
    if s["causal"]:
        keep = keep & (j <= at)
    if s["window"]:
        keep = keep & (j > at - s["window"])
    scores = scores.view(n, kv_heads, mq, group, length)
    scores = scores.masked_fill_(~keep[:, None, :, None, :], -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = scores.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.view(n, kv_heads, mq * group, length) @ keys(s["v_cache"], s["v_scale_inv"]))
    o = o.view(n, kv_heads, mq, group, d) / torch.where(total == 0, 1.0, total)
    seq, at_row, _ = _where(s)
    out = {"out": o.permute(0, 2, 1, 3, 4).reshape(n, mq, heads, d)[seq, at_row].to(s["q"].dtype)}
    if s["lse"]:
        lse = (top + total.log()).squeeze(-1).permute(0, 2, 1, 3).reshape(n, mq, heads)
        out["lse"] = lse[seq, at_row]
    return out


# ---------------------------------------------------------------- the pass

def run(state):
    s = state
    if own:
        from rmsnorm_fp8_quantization_gb300 import ops
        if s["op"] == "rope":
            rope = ops.rope_fwd if s["direction"] == "fwd" else ops.rope_bwd
            q, k = rope(s["q"], s["k"], s["inv_freq"], s["positions"], layout=s["layout"],
                        mscale=s["mscale"])
            return {"q": q, "k": k}
        if s["op"] == "append":
            q = ops.paged_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["cu_seqlens"],
                                 s["kv_lens"], s["block_table"], q=s["q"], inv_freq=s["inv_freq"],
                                 layout=s["layout"], mscale=s["mscale"], k_scale=s["k_scale"],
                                 v_scale=s["v_scale"])
            return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
        out = ops.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["cu_seqlens"],
                                  s["kv_lens"], s["block_table"], max_q=s["max_q"],
                                  max_kv=s["max_kv"], causal=s["causal"], window=s["window"],
                                  k_scale_inv=s["k_scale_inv"], v_scale_inv=s["v_scale_inv"],
                                  return_lse=s["lse"])
        return {"out": out[0], "lse": out[1]} if s["lse"] else {"out": out}
    plain = {"rope": _plain_rope, "append": _plain_append, "attend": _plain_attend}[s["op"]]
    return plain(s)


# ---------------------------------------------------------------- the definition in 64 bits

def _turned(x, pos, inv_freq, case, sign=1.0):
    """Each pair as a complex number, times mscale * exp(i * angle)."""
    r, x = case["rotary"], x.double()
    by = torch.polar(torch.full_like(pos, case["mscale"], dtype=torch.float64).unsqueeze(-1).expand(*pos.shape, r // 2),
                     sign * pos.double().unsqueeze(-1) * inv_freq).unsqueeze(-2)
    if case["layout"] == "half":
        z = torch.complex(x[..., :r // 2], x[..., r // 2:r]) * by
        y = torch.cat([z.real, z.imag], -1)
    else:
        z = torch.view_as_complex(x[..., :r].reshape(*x.shape[:-1], r // 2, 2)) * by
        y = torch.view_as_real(z).reshape(*x.shape[:-1], r)
    return torch.cat([y, x[..., r:]], -1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        sign = -1.0 if case["direction"] == "bwd" else 1.0
        return {n: _turned(s[n], s["positions"], s["inv_freq"], case, sign) for n in ("q", "k")}
    q_lens, kv_lens = _lengths(case)
    table, page = s["block_table"].tolist(), case["page"]
    d, kv_heads = case["dim"], case["kv_heads"]
    if case["op"] == "append":
        pos = torch.cat([torch.arange(b - a, b) for a, b in zip(q_lens, kv_lens)]).cuda()
        slots = torch.tensor([table[i][p // page] * page + p % page
                              for i, (a, b) in enumerate(zip(q_lens, kv_lens))
                              for p in range(b - a, b)]).cuda()
        out = {"q": _turned(s["q"], pos, s["inv_freq"], case)}
        new = {"k": _turned(s["k"], pos, s["inv_freq"], case), "v": s["v"].double()}
        for n in ("k", "v"):
            flat = s[n + "_cache"].double().view(-1, kv_heads, d)
            scale = s[n + "_scale"]
            flat[slots] = new[n] if scale is None else (new[n] * scale.double()).clamp(-448.0, 448.0)
            out[n + "_cache"] = flat.view(s[n + "_cache"].shape)
        return out
    group = case["heads"] // kv_heads
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    row = 0
    for b, (a, n) in enumerate(zip(q_lens, kv_lens)):
        pages = torch.tensor(table[b][:-(-n // page)]).cuda()
        k = s["k_cache"].view(torch.uint8 if case["cache"] == "e4m3" else DT[case["cache"]])[pages]
        v = s["v_cache"].view(torch.uint8 if case["cache"] == "e4m3" else DT[case["cache"]])[pages]
        k, v = (x.view(DT[case["cache"]]).double().reshape(-1, kv_heads, d)[:n] for x in (k, v))
        if s["k_scale_inv"] is not None:
            k, v = k * s["k_scale_inv"].double(), v * s["v_scale_inv"].double()
        back = torch.arange(n - a, n, device="cuda")[:, None] - torch.arange(n, device="cuda")
        drop = torch.zeros_like(back, dtype=torch.bool)
        if case["causal"]:
            drop |= back < 0
        if case["window"]:
            drop |= back >= case["window"]
        for h in range(case["heads"]):
            z = (s["q"][row:row + a, h].double() / math.sqrt(d)) @ k[:, h // group].T
            z[drop] = -math.inf
            norm = torch.logsumexp(z, 1)
            some = norm > -math.inf
            lse[row:row + a, h] = norm
            weights = torch.exp(z - torch.where(some, norm, 0.0)[:, None])
            out[row:row + a, h] = weights @ v[:, h // group]
        row += a
    return {"out": out, "lse": lse} if case["lse"] else {"out": out}
