"""The attention's gradients against differences of its definition in 64 bits, one element at a time, so that each
is held to its own allowed error (sums along a direction add the errors of every element up)."""
import pytest
import torch

from attention_train_cases import Case, define, flat, make
from test_gpu_attention_train import F16, both

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("c", [Case((40,), dim=32, heads=2, kv_heads=1, dtype=F16, uniform=True),
                               Case((7, 0, 30), (20, 5, 33), dim=16, heads=4, kv_heads=2, causal=False),
                               Case((50,), (30,), dim=24, heads=3, kv_heads=3, window=9)],
                         ids=["causal", "cross", "fewer keys, window"])
def test_single_elements(gpu, c):
    s = make(c)
    got, want = both(gpu, s), define(c, s)
    d64 = {n: s[n].double() for n in ("q", "k", "v", "dout")}
    g = torch.Generator().manual_seed(6)

    def loss(t):
        out = define(c, dict(t, kw=None))["out"][0]
        return (out * flat(t["dout"])).nansum()

    for n in ("q", "k", "v"):
        size = flat(s[n]).shape
        for _ in range(12):
            at = tuple(torch.randint(m, (1,), generator=g).item() for m in size)
            h = 2.0 ** -14
            f = []
            for sign in (2, 1, -1, -2):
                t = d64[n].clone()
                flat(t)[at] += sign * h
                f.append(loss(dict(d64, **{n: t})))
            # (8 (f(h) - f(-h)) - (f(2h) - f(-2h))) / 12 h: off by h^4 f5 / 30, with h^4 2^-56; f5 of a softmax of
            # arguments of size a few stays below 2^20, and 64-bit sums' 2^-46 over h is 2^-32: 2^-30 together
            slope = ((8 * (f[1] - f[2]) - (f[0] - f[3])) / (12 * h)).item()
            mine = flat(got["d" + n]).double()[at].item()
            off = want["d" + n][1][at].item()
            assert abs(mine - slope) <= off + 2.0 ** -30, (n, at, mine, slope, off)
            assert abs(slope - want["d" + n][0][at].item()) <= 2.0 ** -30
