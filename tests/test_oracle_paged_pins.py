"""Pins of the float64 oracle for rotary positions and the paged cache against
forms written apart from it: complex multiplication, closed forms, torch's
float64 softmax on the gathered keys."""
import math

import numpy as np
import pytest
import torch

from oracle import paged as P
from paged_cases import Batch, make


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotation_is_complex_multiplication(layout):
    g = np.random.default_rng(0)
    x = g.standard_normal((5, 3, 12))
    f = 100.0 ** (-np.arange(4) / 4)
    pos = np.array([0, 1, 17, -3, 900])
    y = P.rotate(x, pos, f, layout, 1.5)
    z = x[..., :4] + 1j * x[..., 4:8] if layout == "half" else x[..., 0:8:2] + 1j * x[..., 1:8:2]
    w = 1.5 * z * np.exp(1j * pos[:, None] * f)[:, None]
    got = y[..., :4] + 1j * y[..., 4:8] if layout == "half" else y[..., 0:8:2] + 1j * y[..., 1:8:2]
    assert np.allclose(got, w, rtol=0, atol=1e-12)
    assert np.array_equal(y[..., 8:], x[..., 8:])
    back = P.rotate(y / 1.5 ** 2, pos, f, layout, 1.5, backward=True)
    assert np.allclose(back[..., :8], x[..., :8], rtol=0, atol=1e-12)


def test_angles_of_far_positions():
    """pos * f modulo 2 pi in exact integer arithmetic (f = 2^-20: a binary fraction)."""
    from fractions import Fraction
    pi = Fraction(314159265358979323846264338327950288419716939937510, 10 ** 50)
    for pos in (1, 12345678901, 2 ** 40 - 1, -2 ** 35):
        a = Fraction(pos, 2 ** 20)
        a -= round(a / (2 * pi)) * 2 * pi
        got = P.angles(np.array([pos]), np.array([2.0 ** -20]))[0, 0]
        d = abs(got - float(a))
        assert min(d, abs(d - 2 * math.pi)) < 1e-12


def test_scores_depend_on_distance_only():
    g = np.random.default_rng(1)
    q, k = g.standard_normal((1, 1, 8)), g.standard_normal((1, 1, 8))
    f = 10.0 ** (-np.arange(4) / 4)
    dots = [float((P.rotate(q, np.array([a]), f) * P.rotate(k, np.array([b]), f)).sum())
            for a, b in ((9, 4), (1009, 1004), (5, 0))]
    assert np.allclose(dots, dots[0], atol=1e-11)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("window", [0, 7])
def test_paged_attention_against_torch(causal, window):
    c = Batch((3, 1, 5), (20, 4, 33), heads=4, kv_heads=2, dim=16, page=4, dtype="f16",
              causal=causal, window=window)
    s = make(c, "cpu")["cpu"]
    out, lse, mag = P.paged_attend(s["q"], s["k_cache"], s["v_cache"], s["cu"], s["kv_lens"],
                                   s["table"], 0.25, causal, window)
    for b in range(3):
        kv, n = c.kv_lens[b], c.q_lens[b]
        first = max(0, kv - n - window + 1) if window else 0
        idx = [(s["table"][b][t // 4], t % 4) for t in range(first, kv)]
        k = torch.tensor(np.stack([s["k_cache"][p, j] for p, j in idx]))
        v = torch.tensor(np.stack([s["v_cache"][p, j] for p, j in idx]))
        q = torch.tensor(s["q"][s["cu"][b]:s["cu"][b + 1]])
        k, v = k.repeat_interleave(2, 1), v.repeat_interleave(2, 1)
        z = torch.einsum("qhd,khd->hqk", q, k) * 0.25
        j = torch.arange(first, kv)
        t = torch.arange(kv - n, kv)[:, None]
        keep = (j <= t) if causal else torch.ones(n, kv - first, dtype=torch.bool)
        if window:
            keep = keep & (j > t - window)
        z = z.masked_fill(~keep, -math.inf)
        o = torch.einsum("hqk,khd->qhd", torch.softmax(z, -1), v)
        rows = slice(s["cu"][b], s["cu"][b + 1])
        assert np.allclose(out[rows], o.numpy(), atol=1e-12)
        assert np.allclose(lse[rows], torch.logsumexp(z, -1).T.numpy(), atol=1e-12)
        assert (mag[rows] >= np.abs(out[rows]) - 1e-12).all()


def test_rows_that_keep_nothing():
    q, k, v = np.ones((3, 4)), np.ones((2, 4)), np.ones((2, 4))
    out, lse, _ = P.attend(q, k, v, -1, 1.0)
    assert np.array_equal(out[0], np.zeros(4)) and lse[0] == -np.inf
    assert np.allclose(out[1:], 1.0) and np.allclose(lse[1:], [4.0, 4.0 + math.log(2)])


def test_a_dropped_key_never_enters():
    v = np.array([[1.0], [np.nan], [np.inf]])
    k = np.array([[0.0], [np.nan], [0.0]])
    out, lse, _ = P.attend(np.zeros((1, 1)), k, v, 0, 1.0)
    assert out[0, 0] == 1.0 and lse[0] == 0.0
