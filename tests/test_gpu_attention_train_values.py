"""Attention over whole sequences and its backward pass where rows differ in size by powers of two: between
tiles of 128 rows, between sequences, and from row to row.  Against the definition in 64 bits."""
import dataclasses

import pytest
import torch

from attention_train_cases import Case, check, define, make
from test_gpu_attention_train import F16, both, flags

pytestmark = pytest.mark.gpu

CASES = {
    "one sequence": Case((256,), causal=False, q_std=4.0),
    "causal": Case((512,), dim=128, uniform=True, q_std=4.0),
    "packed": Case((300, 1, 0, 129, 257), (260, 5, 3, 511, 128), heads=6, kv_heads=3, dim=96, causal=False,
                   lead=2, trail=7),
    "window": Case((700,), dim=72, window=200, heads=3, kv_heads=1),
    # few CTAs of many steps: shared among several
    "shared steps": Case((1500,), uniform=True, kv_heads=1, dim=128),
    # many CTAs of few steps: several heads of a tile in one
    "heads in turn": Case((257,) * 20, uniform=True, heads=16, kv_heads=16, causal=False),
    "heads in turn, ragged": Case(tuple(3 + 37 * i % 290 for i in range(60)), heads=16, kv_heads=16, dim=40),
}
DTYPES = pytest.mark.parametrize("dtype", [F16, torch.bfloat16], ids=["f16", "bf16"])


def sized(c, s, name, exponents):
    """s with the rows of tensor ``name`` times 2^exponents[token]."""
    t = s[name]
    f = torch.exp2(exponents.double()).to(t.device)
    return dict(s, **{name: (t.double() * f.view(*t.shape[:-2], 1, 1)).to(t.dtype)})


def places(c, lens):
    """(sequence, place in it) of every token; outside the sequences -1."""
    seq = torch.full((c.lead + sum(lens) + c.trail,), -1)
    at = seq.clone()
    n = c.lead
    for b, m in enumerate(lens):
        seq[n:n + m], at[n:n + m] = b, torch.arange(m)
        n += m
    return seq, at


def held(gpu, c, s):
    flags()
    got, want = both(gpu, s), define(c, s)
    assert flags() == 0
    for n in got:
        check(n, got[n], want[n])


@DTYPES
@pytest.mark.parametrize("tensor, small", [("v", 0), ("v", 1), ("dout", 0), ("k", 1), ("q", 0)])
@pytest.mark.parametrize("name", CASES)
def test_tiles_of_different_size(gpu, name, tensor, small, dtype):
    """Every other tile of a sequence 2^-12 of the rest: a row's delta is a mean over all keys, so next to
    small values of its own tile it is as large as the largest of the sequence."""
    c = dataclasses.replace(CASES[name], dtype=dtype)
    _, at = places(c, c.q_lens if tensor in ("q", "dout") else c.keys)
    held(gpu, c, sized(c, make(c), tensor, torch.where(at // 128 % 2 == small, -12, 0)))


@DTYPES
@pytest.mark.parametrize("name", CASES)
def test_rows_of_different_size(gpu, name, dtype):
    c = dataclasses.replace(CASES[name], dtype=dtype)
    s = make(c)
    g = torch.Generator().manual_seed(3)
    for n, lens in (("q", c.q_lens), ("dout", c.q_lens), ("k", c.keys), ("v", c.keys)):
        s = sized(c, s, n, torch.randint(-12, 3, (places(c, lens)[0].numel(),), generator=g))
    held(gpu, c, s)


@DTYPES
@pytest.mark.parametrize("name", ["packed", "heads in turn", "heads in turn, ragged"])
def test_sequences_of_different_size(gpu, name, dtype):
    c = dataclasses.replace(CASES[name], dtype=dtype)
    s = make(c)
    for n, lens in (("v", c.keys), ("dout", c.q_lens)):
        s = sized(c, s, n, -6 * (places(c, lens)[0] % 3))
    held(gpu, c, s)


@pytest.mark.parametrize("dim", [64, 128])
def test_rounding_of_small_ds(gpu, dim):
    """f16 ds that lie where the type ends, all rounded the same way: off by at most 2^-39 of the largest
    |dout| |v| each, as documented.  Query 0 sets that (1) and has no part in dk (q_0 = 0); every other
    one's ds is 9/8 2^-38 of either sign (p = 2^-7, dout 2^-24, v 9/8 2^-7, delta 0)."""
    n = 128
    c = Case((n,), uniform=True, heads=1, kv_heads=1, dim=dim, dtype=F16, causal=False, scale=2.0 ** 10)
    q, k, v, dout = (torch.zeros(1, n, 1, dim, dtype=F16, device="cuda") for _ in range(4))
    q[0, 1:, 0, 1] = 2.0 ** 10
    dout[0, :, 0, 0] = 2.0 ** -24
    dout[0, 0, 0, 0] = 1.0
    v[0, 0::2, 0, 0], v[0, 1::2, 0, 0] = 1.125 * 2.0 ** -7, -1.125 * 2.0 ** -7
    v[0, 0, 0, 0], v[0, 1, 0, 0] = 1.0, -1.0
    s = dict(q=q, k=k, v=v, dout=dout, kw=dict(causal=False, scale=c.scale))
    held(gpu, c, s)
    dk = define(c, s)["dk"][0][:, 0, 1]
    assert abs(dk[2].item() / (127 * 2.0 ** 20 * 1.125 * 2.0 ** -38) - 1) < 1e-6
