"""Batches for the paged cache's tests: packed tokens, lengths, pages in mixed
order, and NaN wherever the operators must not look (slots behind a sequence's
end, pages of no sequence, pages before a window)."""
from __future__ import annotations

import dataclasses

import numpy as np
import torch

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


@dataclasses.dataclass(frozen=True)
class Batch:
    q_lens: tuple
    kv_lens: tuple
    heads: int = 4
    kv_heads: int = 2
    dim: int = 64
    page: int = 16
    dtype: str = "bf16"
    fp8: bool = False
    causal: bool = True
    window: int = 0
    pad: int = 0            # padding rows behind the last sequence
    heads_first: bool = False  # cache [pages, heads, page, dim]
    seed: int = 0

    def __str__(self):
        f = (f"q{'.'.join(map(str, self.q_lens))[:24]}-kv{'.'.join(map(str, self.kv_lens))[:24]}-"
             f"h{self.heads}.{self.kv_heads}-d{self.dim}-p{self.page}-{self.dtype}")
        for name in ("fp8", "heads_first"):
            f += "-" + name if getattr(self, name) else ""
        return (f + ("" if self.causal else "-full") + (f"-w{self.window}" if self.window else "")
                + (f"-pad{self.pad}" if self.pad else ""))


def values(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g) * std).to(dtype)


def make(c: Batch, device="cuda"):
    """dict of tensors on ``device`` and, under "cpu", what the oracle reads."""
    g = torch.Generator().manual_seed(1234 + c.seed)
    dt = DT[c.dtype]
    n = len(c.q_lens)
    cu = np.concatenate([[0], np.cumsum(c.q_lens)]).tolist()
    tokens = cu[-1] + c.pad
    need = [-(-kv // c.page) for kv in c.kv_lens]
    pages = sum(need) + 2
    order = torch.randperm(pages, generator=g).tolist()
    table = torch.full((n, max(need + [1]) + 1), -1, dtype=torch.int32)
    at = 0
    for b in range(n):
        table[b, :need[b]] = torch.tensor(order[at:at + need[b]], dtype=torch.int32)
        at += need[b]
    shape = (pages, c.page, c.kv_heads, c.dim)
    cdt = torch.float8_e4m3fn if c.fp8 else dt
    gain = 24.0 if c.fp8 else 1.0
    bad = float("nan")
    caches = []
    for _ in range(2):
        x = values(g, shape, torch.float32, gain)
        live = torch.zeros(pages, c.page, dtype=torch.bool)
        for b in range(n):
            first = 0
            if c.window:
                first = max(0, c.kv_lens[b] - c.q_lens[b] - c.window + 1)
            for t in range(first, c.kv_lens[b]):
                live[table[b, t // c.page], t % c.page] = True
        x[~live] = bad
        caches.append(x.to(cdt))
    if c.window:  # pages wholly before every row's window are gone from the table
        for b in range(n):
            first = max(0, c.kv_lens[b] - c.q_lens[b] - c.window + 1)
            table[b, :first // c.page] = -1
    q = values(g, (tokens, c.heads, c.dim), dt)
    k = values(g, (tokens, c.kv_heads, c.dim), dt)
    v = values(g, (tokens, c.kv_heads, c.dim), dt)

    def place(x):
        if not c.heads_first:
            return x.to(device)
        return x.permute(0, 2, 1, 3).contiguous().to(device).permute(0, 2, 1, 3)

    s = dict(q=q.to(device), k=k.to(device), v=v.to(device), k_cache=place(caches[0]),
             v_cache=place(caches[1]), cu=torch.tensor(cu, dtype=torch.int32, device=device),
             kv_lens=torch.tensor(c.kv_lens, dtype=torch.int32, device=device),
             table=table.to(device), max_q=max(c.q_lens), max_kv=max(c.kv_lens))
    if c.fp8:
        s["scale"] = torch.full((1,), gain, device=device)
        s["scale_inv"] = torch.full((1,), 1.0 / gain, device=device)
    else:
        s["scale"] = s["scale_inv"] = None
    s["cpu"] = dict(q=q.double().numpy(), k=k.double().numpy(), v=v.double().numpy(),
                    k_cache=caches[0].double().numpy(), v_cache=caches[1].double().numpy(), cu=cu,
                    kv_lens=list(c.kv_lens), table=table.numpy(),
                    inv=float(s["scale_inv"].double()) if c.fp8 else 1.0)
    return s


def score_size(cpu, scale):
    """Per (token, head): largest sum_d |scale q_d k_d| over the cache's finite keys, bounded by
    norms of absolute values (what a score's fp32 summation error is relative to)."""
    k = np.nan_to_num(np.abs(cpu["k_cache"])) * cpu["inv"]
    top = k.max(axis=(0, 1))                                   # [kv_heads, d]
    g = cpu["q"].shape[1] // top.shape[0]
    return scale * (np.abs(cpu["q"]) * np.repeat(top, g, axis=0)[None]).sum(-1)
