"""Cases of the attention over whole sequences, and its definition with its gradients in 64
bits, each value next to how far a kernel with 32-bit sums and 16-bit probabilities may be off.

u is half a step of the tensors' type (finfo.eps / 2).  With scores z_ij (natural units), their
probabilities p, dp_ij = dout_i.v_j and ds = p (dp - delta):

* a score or a row's logarithm is off by 2^-20 of what it sums (32-bit sums of exact products,
  taken as if every addition lost 2^-24 and up to 2^4 of them lined up), so a probability by
  e_ij = 2^-18 (1 + scale sum |q k| + |lse_i|) relative;
* out: the probabilities' rounding and e_ij weighed by p |v|, and its own rounding:
      (u + e) sum_j p |v| + u |out|;
* delta, from the rounded out: E_i = sum |dout| (u |out| + (u + e) sum_j p |v|) and 2^-20 of
  sum |dout out|; dp: 2^-20 sum |dout v|;
* ds: |ds| (u + e) + p (E + 2^-20 (sum |dout out| + sum |dout v|)), f16 besides 2^-39 of the
  sequence's largest |dout| |v|;
* dq, dk: those weighed by scale |k|, scale |q|, 2^-20 of the sum, and u of the result;
* dv: (u + e) p weighed by |dout| (f16 besides 2^-37 a pair), and u of the result.
Results below a type's smallest normal number: a step of those, finfo.smallest_normal * eps.
"""
from __future__ import annotations

import dataclasses
import math

import torch


@dataclasses.dataclass(frozen=True)
class Case:
    q_lens: tuple
    k_lens: tuple = ()           # (): the queries' own tokens
    heads: int = 4
    kv_heads: int = 2
    dim: int = 64
    dtype: torch.dtype = torch.bfloat16
    causal: bool = True
    window: int = 0
    scale: float | None = None
    uniform: bool = False        # [batch, seq, heads, dim], no cu_seqlens
    packed: bool = False         # q, k and v are views of one tensor
    lead: int = 0                # rows before the first sequence
    trail: int = 0               # and behind the last
    q_std: float = 1.0
    dout_std: float = 1.0
    seed: int = 0

    @property
    def keys(self):
        return self.k_lens or self.q_lens


def make(c: Case, device="cuda"):
    """Inputs of a case: q, k, v, dout, and the call's other arguments in ``kw``."""
    g = torch.Generator().manual_seed(c.seed + 7)
    h, hk, d = c.heads, c.kv_heads, c.dim
    r = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std).to(c.dtype).to(device)
    tq, tk = (sum(n) + c.lead + c.trail for n in (c.q_lens, c.keys))
    if c.uniform:
        b, n, m = len(c.q_lens), c.q_lens[0], c.keys[0]
        q_lead, k_lead = (b, n), (b, m)
        assert set(c.q_lens) == {n} and set(c.keys) == {m}
    else:
        q_lead, k_lead = (tq,), (tk,)
    if c.packed:
        q, k, v = r(*q_lead, h + 2 * hk, d).split([h, hk, hk], dim=-2)
    else:
        q, k, v = r(*q_lead, h, d, std=c.q_std), r(*k_lead, hk, d), r(*k_lead, hk, d)
    kw = dict(causal=c.causal, window=c.window)
    if c.scale is not None:
        kw["scale"] = c.scale
    if not c.uniform:
        cu = lambda lens: torch.tensor([c.lead, *lens]).cumsum(0).to(torch.int32).to(device)
        kw.update(cu_seqlens=cu(c.q_lens), max_q=max(c.q_lens))
        if c.k_lens:
            kw.update(cu_seqlens_k=cu(c.k_lens), max_k=max(c.k_lens))
    return dict(q=q, k=k, v=v, dout=r(*q_lead, h, d, std=c.dout_std), kw=kw)


def keep(c: Case, n, m, device="cpu"):
    """[n, m]: which keys a sequence's queries keep."""
    at = torch.arange(n, device=device)[:, None] + (m - n)
    j = torch.arange(m, device=device)
    k = torch.ones(n, m, dtype=torch.bool, device=device)
    if c.causal:
        k &= j <= at
    if c.window:
        k &= j > at - c.window
    return k


def flat(t):
    return t.reshape(-1, *t.shape[-2:])


def define(c: Case, s):
    """{name: (value, allowed error)} of out, lse, dq, dk, dv as [tokens, heads(, dim)]; rows
    outside the sequences are NaN."""
    dev = s["q"].device
    u = torch.finfo(c.dtype).eps / 2
    least = torch.finfo(c.dtype).smallest_normal * torch.finfo(c.dtype).eps
    f16 = c.dtype is torch.float16
    scale = c.dim ** -0.5 if c.scale is None else c.scale
    group = c.heads // c.kv_heads
    q, k, v, do = (flat(s[n]).double() for n in ("q", "k", "v", "dout"))
    new = lambda t, *dims: (torch.full(dims or t.shape, math.nan, dtype=torch.float64, device=dev),
                            torch.full(dims or t.shape, math.nan, dtype=torch.float64, device=dev))
    r = {"out": new(q), "lse": new(q, *q.shape[:2]), "dq": new(q), "dk": new(k), "dv": new(v)}
    a = b = c.lead
    for n, m in zip(c.q_lens, c.keys):
        qs, ks = slice(a, a + n), slice(b, b + m)
        for x in ("dk", "dv"):
            r[x][0][ks] = r[x][1][ks] = 0
        for h in range(c.heads):
            g = h // group
            Q, K, V, D = q[qs, h], k[ks, g], v[ks, g], do[qs, h]
            z = scale * (Q @ K.T)
            z = z.masked_fill(~keep(c, n, m, dev), -math.inf)
            lse = torch.logsumexp(z, 1) if m else torch.full((n,), -math.inf, device=dev).double()
            some = lse > -math.inf
            norm = torch.where(some, lse, 0.0)
            p = torch.exp(z - norm[:, None])
            out = p @ V
            size = scale * (Q.abs() @ K.abs().T)
            top = torch.where(p > 0, size, 0.0).amax(1) if m else torch.zeros(n, device=dev).double()
            e = 2.0 ** -18 * (1 + top + norm.abs())[:, None]
            weighed = p @ V.abs()
            r["lse"][0][qs, h] = lse
            r["lse"][1][qs, h] = 2.0 ** -20 * (1 + top + norm.abs())
            r["out"][0][qs, h] = out
            out_err = (u + e) * weighed + u * out.abs() + least + (2.0 ** -34 * V.abs().sum(0) if f16 else 0)
            r["out"][1][qs, h] = out_err
            dp = D @ V.T
            delta = (D * out).sum(1, keepdim=True)
            ds = p * (dp - delta)
            E = (D.abs() * out_err).sum(1, keepdim=True)
            off = 2.0 ** -20 * ((D * out).abs().sum(1, keepdim=True) + D.abs() @ V.abs().T)
            ds_err = ds.abs() * (u + e) + p * (E + off)
            if f16 and n and m:
                big = D.norm(dim=1).max() * V.norm(dim=1).max()
                # (the scale goes by every head of the group, and every one's is no larger than)
                big = torch.stack([do[qs, g * group + x].norm(dim=1).max() for x in range(group)]).max() \
                    * V.norm(dim=1).max()
                ds_err = ds_err + 2.0 ** -39 * big * (p > 0)
            dq = scale * (ds @ K)
            r["dq"][0][qs, h] = dq
            r["dq"][1][qs, h] = scale * (ds_err @ K.abs() + 2.0 ** -20 * (ds.abs() @ K.abs())) \
                + u * dq.abs() + least
            dk, dv = scale * (ds.T @ Q), p.T @ D
            r["dk"][0][ks, g] += dk
            r["dk"][1][ks, g] += scale * (ds_err.T @ Q.abs() + 2.0 ** -20 * (ds.abs().T @ Q.abs()))
            r["dv"][0][ks, g] += dv
            r["dv"][1][ks, g] += ((u + e + 2.0 ** -20) * p + (2.0 ** -37 * (p > 0) if f16 else 0)).T @ D.abs()
        for x in ("dk", "dv"):
            r[x][1][ks] += u * r[x][0][ks].abs() + least
        a, b = a + n, b + m
    return r


def check(name, got, want):
    """got within the allowed error of the value where that is a number, and nowhere NaN there."""
    value, off = want
    got = got.double().reshape(value.shape)
    inside = ~value.isnan()
    assert not got[inside].isnan().any(), f"{name}: NaN"
    same = (got == value) | ~inside              # infinities of empty rows
    excess = ((got - value).abs() - off).masked_fill(same, -1.0)
    worst = excess.max().item() if excess.numel() else -1.0
    assert worst <= 0, (f"{name}: {int((excess > 0).sum())} of {inside.sum()} off, worst by "
                        f"{worst:.3g} at {torch.nonzero(excess == excess.max())[0].tolist()}: "
                        f"{got[excess == excess.max()][0]:.6g} for {value[excess == excess.max()][0]:.6g}, "
                        f"allowed {off[excess == excess.max()][0]:.3g}")
