"""Frequencies above one radian a position, at far positions."""
from decimal import Decimal, getcontext
from fractions import Fraction

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

PI = Fraction(Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803482534"))


def exact_angles(positions, freq):
    """Reduced angles from exact rational arithmetic, [positions, pairs]."""
    getcontext().prec = 60
    out = np.zeros((len(positions), len(freq)))
    for i, p in enumerate(positions):
        for j, f in enumerate(freq):
            turns = Fraction(f) * p / (2 * PI)
            out[i, j] = float((turns - round(turns)) * 2 * PI)
    return out


@pytest.mark.parametrize("backward", [False, True], ids=["fwd", "bwd"])
def test_large_frequencies_at_far_positions(gpu, backward):
    """Tolerance: test_gpu_rope's, of whose 3 * 2^-23 (|a| + |b|) the roundings named there take
    2.5, and for the angle 2^-64 (1 + |f| / 4) of a turn for each position.  Pairs that this
    leaves no eight bits are left out."""
    freq = [1.0, 3.9, -4.1, 100.0 / 3, 1e4 / 7, -3e9 / 11, 1e12 / 13, 2.0 ** 49 * 1.337, 2.0 ** -40, 0.0]
    pos = [0, 1, -1, 5, 4097, 131072, 2 ** 31 + 7, -2 ** 33, 2 ** 40 - 3]
    d = 2 * len(freq)
    g = torch.Generator().manual_seed(5)
    q = torch.randn(1, len(pos), 3, d, generator=g)
    f = torch.tensor(freq, dtype=torch.float64)
    fn = gpu.rope_bwd if backward else gpu.rope_fwd
    got, _ = fn(q.cuda(), None, f.cuda(), torch.tensor(pos).cuda())
    a = exact_angles(pos, freq)[:, None, :]                       # [positions, heads, pairs]
    c, s = np.cos(a), np.sin(a) * (-1 if backward else 1)
    x, y = q.double().numpy()[0], got.cpu().double().numpy()[0]
    lo, hi = x[..., :d // 2], x[..., d // 2:]
    off = (2 * np.pi * 2.0 ** -64
           * np.outer(np.abs(np.array(pos, float)), 1 + np.abs(freq) / 4.0))[:, None, :]
    lim = (np.abs(lo) + np.abs(hi)) * (3 * 2.0 ** -23 + off)
    held = np.broadcast_to(off < 2.0 ** -8, lim.shape)
    for err in (y[..., :d // 2] - (lo * c - hi * s), y[..., d // 2:] - (lo * s + hi * c)):
        assert (np.abs(err)[held] <= lim[held]).all(), (np.abs(err)[held] / lim[held]).max()
    assert held.mean() > 0.8
