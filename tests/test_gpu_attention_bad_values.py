"""Infinities and NaN among the inputs of the attention over whole sequences: what the formulas make of the kept
pairs alone, NaN and infinities included, and in a bounded time."""
import dataclasses
import math

import pytest
import torch

from attention_train_cases import Case, flat, keep, make
from test_gpu_attention_train import F16, both, flags
from test_gpu_attention_train_values import places

pytestmark = pytest.mark.gpu
NAN, INF = math.nan, math.inf


def formulas(c, s, rounded):
    """{name: (value, allowed error)} in 64 bits, every sum over kept pairs alone; the errors are those of
    attention_train_cases, for sums of numbers.  delta is taken from the forward's ``rounded`` output, as the
    backward's definition has it: an infinite dout times an output next to 0 goes by its sign."""
    u = torch.finfo(c.dtype).eps / 2
    least = torch.finfo(c.dtype).smallest_normal * torch.finfo(c.dtype).eps
    f16 = c.dtype is F16
    scale = c.dim ** -0.5 if c.scale is None else c.scale
    q, k, v, do = (flat(s[n]).double() for n in ("q", "k", "v", "dout"))
    rounded = flat(rounded).double()
    r = {n: [torch.full_like(t, NAN), torch.zeros_like(t)] for n, t in (("out", q), ("dq", q), ("dk", k), ("dv", v))}
    group = c.heads // c.kv_heads
    a = b = c.lead
    for n, m in zip(c.q_lens, c.keys):
        qs, ks = slice(a, a + n), slice(b, b + m)
        on = keep(c, n, m, q.device)
        kept = lambda t: torch.where(on, t, 0.0)
        # sum over kept pairs of w_ij x_j (over: 1) or w_ij x_i (over: 0)
        total = lambda w, x, over: torch.where(on[..., None], w[..., None] * (x[None] if over else x[:, None]), 0.0).sum(over)
        size = lambda t: t.abs().nan_to_num(0.0, 0.0, 0.0)
        r["dk"][0][ks] = r["dv"][0][ks] = 0
        for h in range(c.heads if n and m else 0):
            g = h // group
            Q, K, V, D = q[qs, h], k[ks, g], v[ks, g], do[qs, h]
            z = scale * torch.einsum("id,jd->ijd", Q, K).sum(-1)
            lse = torch.logsumexp(z.masked_fill(~on, -INF), 1)
            lse[(on & (z.isnan() | (z == INF))).any(1)] = NAN   # (infinity less infinity, of the largest)
            p = kept(torch.exp(z - lse[:, None]))
            out = total(p, V, 1)
            dp = torch.einsum("id,jd->ijd", D, V).sum(-1)
            delta = (D * rounded[qs, h]).sum(1, keepdim=True)
            ds = kept(p * (dp - delta))
            e = 2.0 ** -18 * (1 + (scale * (size(Q) @ size(K).T)).amax(1, keepdim=True) + size(lse)[:, None])
            ps = size(p)
            out_err = (u + e) * (ps @ size(V)) + u * size(out) + least + (2.0 ** -34 * size(V).sum(0) if f16 else 0)
            E = (size(D) * out_err).sum(1, keepdim=True)
            off = 2.0 ** -20 * ((size(D) * size(out)).sum(1, keepdim=True) + size(D) @ size(V).T)
            ds_err = size(ds) * (u + e) + ps * (E + off)
            if f16:
                big = max(size(do[qs, g * group + x]).norm(dim=1).max() for x in range(group)) * size(V).norm(dim=1).max()
                ds_err = ds_err + 2.0 ** -39 * big * on
            r["out"][0][qs, h], r["out"][1][qs, h] = out, out_err
            dq = scale * total(ds, K, 1)
            r["dq"][0][qs, h] = dq
            r["dq"][1][qs, h] = scale * (ds_err @ size(K) + 2.0 ** -20 * (size(ds) @ size(K))) + u * size(dq) + least
            r["dk"][0][ks, g] += scale * total(ds, Q, 0)
            r["dk"][1][ks, g] += scale * (ds_err.T @ size(Q) + 2.0 ** -20 * (size(ds).T @ size(Q)))
            r["dv"][0][ks, g] += total(p, D, 0)
            r["dv"][1][ks, g] += ((u + e + 2.0 ** -20) * ps + (2.0 ** -37 * on if f16 else 0)).T @ size(D)
        for x in ("dk", "dv"):
            r[x][1][ks] += u * size(r[x][0][ks]) + least
        a, b = a + n, b + m
    return r


def alike(name, got, want):
    value, off = want
    got = got.double().reshape(value.shape)
    nan, inf = value.isnan(), value.isinf()
    assert torch.equal(got.isnan(), nan), (f"{name}: {int((got.isnan() & ~nan).sum())} NaN that do not belong there, "
                                           f"{int((nan & ~got.isnan()).sum())} missing")
    assert torch.equal(got[inf], value[inf]), f"{name}: infinities"
    rest = ~nan & ~inf
    excess = ((got - value).abs() - off)[rest]
    assert not (excess > 0).any(), f"{name}: {int((excess > 0).sum())} off, worst by {excess.max():.3g}"


CASES = {
    "causal": Case((300,), dim=32, uniform=True),
    "window": Case((400,), dim=64, window=40, heads=2, kv_heads=1),
    "packed": Case((70, 1, 0, 200, 129), dim=96, lead=3, trail=9),
    "cross": Case((300, 20), (150, 260), dim=128, heads=2),
    "not causal, window": Case((300,), dim=40, causal=False, window=60, heads=2, kv_heads=2),
    "shared steps": Case((1400,), uniform=True, kv_heads=1, dim=16),
    "heads in turn": Case((130,) * 40, uniform=True, heads=24, kv_heads=12, dim=16),
}
# (tensor, value, columns, every so many tokens)
BAD = {
    "dout nan": ("dout", NAN, slice(None), 97), "dout nan column": ("dout", NAN, slice(3, 4), 61),
    "dout inf": ("dout", INF, slice(None), 97), "dout inf column": ("dout", INF, slice(5, 6), 7),
    "dout -inf": ("dout", -INF, slice(2, 9), 41), "dout all inf": ("dout", INF, slice(None), 1),
    "v nan": ("v", NAN, slice(1, 3), 83), "v inf": ("v", INF, slice(0, 1), 90), "v -inf": ("v", -INF, slice(None), 111),
    "k nan": ("k", NAN, slice(4, 5), 119), "k inf": ("k", INF, slice(4, 5), 119), "q nan": ("q", NAN, slice(6, 7), 37),
    "q inf": ("q", INF, slice(6, 7), 37),
}


@pytest.mark.parametrize("dtype", [F16, torch.bfloat16], ids=["f16", "bf16"])
@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("name", CASES)
def test_kept_pairs_alone(gpu, name, bad, dtype):
    c = dataclasses.replace(CASES[name], dtype=dtype, q_std=0.25)
    s = make(c)
    tensor, value, columns, every = BAD[bad]
    # (not a sequence's first ones: queries that keep nothing but keys with a score of -inf are let alone)
    at = places(c, c.q_lens if tensor in ("q", "dout") else c.keys)[1]
    hit = (torch.arange(at.numel()) % every == every // 2) & (at >= 40)
    flat(s[tensor])[hit.to(s["q"].device), :, columns] = value
    flags()
    got = both(gpu, s)
    assert flags() == 0
    want = formulas(c, s, got["out"])
    inside = torch.zeros(flat(s["q"]).shape[0], dtype=torch.bool)
    inside[c.lead:inside.numel() - c.trail] = True
    for n in ("out", "dq", "dk", "dv"):
        g = flat(got[n])
        if n in ("out", "dq") or not c.k_lens:
            alike(n, g[inside], [x[inside] for x in want[n]])
        else:
            alike(n, g, want[n])


def quickest(call, times=3):
    """Seconds on the device of the quickest of a few calls."""
    best = INF
    for _ in range(times + 1):
        a, b = torch.cuda.Event(True), torch.cuda.Event(True)
        a.record()
        call()
        b.record()
        b.synchronize()
        best = min(best, a.elapsed_time(b) * 1e-3)
    return best


SPREAD = {
    "a NaN in a gradient": lambda s: s["dout"][0, 512].fill_(NAN),
    "an infinite column": lambda s: s["dout"][0, 512, :, 5].fill_(INF),
    "infinities all over": lambda s: s["dout"][:, ::7].fill_(INF),
    "gradients all NaN": lambda s: s["dout"].fill_(NAN),
    "gradients all infinite": lambda s: s["dout"].fill_(INF),
    "a NaN in the last query of the last head": lambda s: s["q"][0, -1, -1].fill_(NAN),
    "a NaN in the last queries, no gradient": lambda s: (s["q"][:, -1].fill_(NAN), s["dout"].zero_()),
    "a NaN in the last key": lambda s: s["k"][0, -1].fill_(NAN),
    "a NaN in a key": lambda s: s["k"][0, 512].fill_(NAN),
    "a NaN in a value": lambda s: s["v"][0, 512].fill_(NAN),
    "an infinite value": lambda s: s["v"][0, 512, :, 3].fill_(INF),
}


@pytest.mark.parametrize("kind", SPREAD)
@pytest.mark.parametrize("dtype", [F16, torch.bfloat16], ids=["f16", "bf16"])
def test_time_of_the_backward(gpu, kind, dtype):
    """2 x 1024 tokens, 32 / 8 heads of 128: 80 us without bad values.  With them at most every row of a tile is
    summed again, 32 rows a warp of up to 4 x 1024 pairs; at 200 ns a pair of a warp's 30 ms (measured: up to
    13; as it was, up to 156)."""
    c = Case((1024, 1024), uniform=True, heads=32, kv_heads=8, dim=128, dtype=dtype)
    s = make(c)
    SPREAD[kind](s)
    out, lse = gpu.attention_fwd(s["q"], s["k"], s["v"])
    assert quickest(lambda: gpu.attention_bwd(s["dout"], s["q"], s["k"], s["v"], out, lse)) < 0.03


@pytest.mark.parametrize("kind", ["first token", "a token", "infinite, a column", "infinite all over", "all"])
@pytest.mark.parametrize("dtype", [F16, torch.bfloat16], ids=["f16", "bf16"])
def test_time_of_the_forward(gpu, kind, dtype):
    """2 x 1024 tokens, 32 / 8 heads of 128: 31 us without bad values.  With them at most the rows of one tile are
    summed again (measured: up to 5.5 ms; as it was, 80)."""
    c = Case((1024, 1024), uniform=True, heads=32, kv_heads=8, dim=128, dtype=dtype)
    s = make(c)
    v = s["v"]
    {"first token": lambda: v[0, 0].fill_(NAN), "a token": lambda: v[0, 530].fill_(NAN),
     "infinite, a column": lambda: v[0, 530, :, 3].fill_(INF), "infinite all over": lambda: v[:, ::7].fill_(INF),
     "all": lambda: v.fill_(NAN)}[kind]()
    assert quickest(lambda: gpu.attention_fwd(s["q"], s["k"], v)) < 0.03


@pytest.mark.parametrize("fp8", [False, True], ids=["two bytes", "E4M3"])
@pytest.mark.parametrize("bad", [(NAN, slice(None)), (NAN, slice(3, 4)), (INF, slice(5, 40)), (-INF, slice(70, 71))],
                         ids=["nan", "nan column", "inf", "-inf column"])
@pytest.mark.parametrize("c", [Case((600,), (777,), heads=8, kv_heads=2, dim=128),
                               Case((60,), (9000,), heads=8, kv_heads=1, dim=128, dtype=F16),
                               Case((3,), (900,), heads=8, kv_heads=1, dim=96)],
                         ids=["prompt", "keys in parts", "few rows"])
def test_paged_kept_pairs_alone(gpu, c, bad, fp8):
    """The same over a paged cache: what a row keeps decides, in tiles and parts of keys that it drops some of."""
    s = make(dataclasses.replace(c, q_std=0.25))
    n, m, page = c.q_lens[0], c.keys[0], 64
    pages = -(-m // page)
    value, columns = bad
    # one that some rows drop, one that all keep
    s["v"][m - n // 2 - 1, :, columns] = value
    s["v"][m // 3, :, slice(columns.start or 0, (columns.start or 0) + 2)] = value
    kind = torch.float8_e4m3fn if fp8 else c.dtype
    k, v = (s[t].to(kind) for t in ("k", "v"))
    if fp8:
        v = torch.where(s["v"].isfinite(), s["v"], NAN).to(kind)   # E4M3 has no infinities
    s.update(k=k.to(c.dtype), v=v.to(c.dtype))
    table = torch.randperm(pages, generator=torch.Generator().manual_seed(1)).int().cuda()[None]
    caches = []
    for t in (k, v):
        room = torch.zeros(pages * page, *t.shape[1:], device="cuda").to(kind)
        room[:m] = t
        cache = torch.empty(pages, page, *t.shape[1:], device="cuda").to(kind)
        cache.view(torch.uint8)[table[0].long()] = room.view(pages, page, *t.shape[1:]).view(torch.uint8)
        caches.append(cache)
    one = torch.ones(1, device="cuda")
    kw = dict(k_scale_inv=one, v_scale_inv=one) if fp8 else {}
    out = gpu.paged_attention(s["q"], *caches, torch.tensor([0, n], dtype=torch.int32, device="cuda"),
                              torch.tensor([m], dtype=torch.int32, device="cuda"), table, max_q=n, max_kv=m, **kw)
    value, off = formulas(c, s, out)["out"]
    alike("out", out, (value, off))
    assert not value.isfinite().all() and value.isfinite().any()
