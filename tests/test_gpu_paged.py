"""GPU parity of the paged cache's append and of the attention over it, against
the float64 oracle.  Every batch has NaN in all slots and pages that the
operators must not look at.

Append: the keys' rotation within the rotary tests' bound, values and
unrotated keys bit-exact, E4M3 codes within one step of the exact value's code
and nearly all equal; everything else in the caches untouched.

Attention tolerance, per element, from the arithmetic alone.  With p the
softmax weights, A = sum_j p_j |v_j| and S the largest sum_d |scale q_d k_d|:
  * the stored rounding: eps(t) / 2 of the result;
  * the probabilities' rounding before the product with the values: eps / 2 of
    the value type (bf16 2^-8, f16 2^-11), so A times that;
  * the scores: products exact, d / 16 + 2 steps of fp32 accumulation that may
    truncate, 2^-23 each, then the scale's and the subtraction's roundings:
    dS = (d / 16 + 6) 2^-23 S absolute, which enters p and the sum: 2 dS A;
  * ex2 (2^-22 relative, twice) and the sums over n keys, n / 16 + 16
    accumulations of 2^-23 each, rescalings among them: A (n / 16 + 24) 2^-23.
lse: dS + (|lse| + n / 16 + 24) 2^-23."""
import dataclasses

import numpy as np
import pytest
import torch

from oracle import paged as P
from paged_cases import DT, Batch, make, score_size

pytestmark = pytest.mark.gpu


def attend(gpu, c, s, **kw):
    a = dict(max_q=s["max_q"], max_kv=s["max_kv"], causal=c.causal, window=c.window,
             k_scale_inv=s["scale_inv"], v_scale_inv=s["scale_inv"], return_lse=True)
    a.update(kw)
    return gpu.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["cu"], s["kv_lens"],
                               s["table"], **a)


def device_flags(clear=True):
    from rmsnorm_fp8_quantization_gb300 import gbnorm as G
    st, f = G.gbn_device_error(clear)
    assert st == G.GBN_OK
    return f


def check_attention(c, s, out, lse, scale=None):
    cpu = s["cpu"]
    scale = c.dim ** -0.5 if scale is None else scale
    n = cpu["cu"][-1]
    ref, rl, mag = P.paged_attend(cpu["q"], cpu["k_cache"], cpu["v_cache"], cpu["cu"],
                                  cpu["kv_lens"], cpu["table"], scale, c.causal, c.window,
                                  cpu["inv"], cpu["inv"])
    ds = (c.dim / 16 + 6) * 2.0 ** -23 * score_size(cpu, scale)
    dt = DT[c.dtype]
    vt = torch.float16 if c.fp8 else dt
    keys = max(c.kv_lens)
    half = torch.finfo(dt).eps / 2
    rel = torch.finfo(vt).eps / 2 + 2 * ds[..., None] + (keys / 16 + 24) * 2.0 ** -23
    inner = mag * rel
    lim = half * (np.abs(ref) + inner) + inner + (2.0 ** -25 if c.dtype == "f16" else 0.0)
    g = out.double().cpu().numpy()
    err = np.abs(g - ref)[:n]
    bad = ~(err <= lim[:n])
    assert not bad.any(), (int(bad.sum()), bad.size, np.argwhere(bad)[:4].tolist(),
                           err[bad][:4], lim[:n][bad][:4])
    if lse is not None:
        gl = lse.double().cpu().numpy()[:n]
        empty = np.isinf(rl[:n])
        assert np.array_equal(np.isneginf(gl), empty)
        diff = np.abs(np.where(empty, 0, gl) - np.where(empty, 0, rl[:n]))
        ll = ds[:n] + (np.abs(np.where(empty, 0, rl[:n])) + keys / 16 + 24) * 2.0 ** -23
        assert (diff <= ll).all(), (diff.max(), ll.min())


def B(q, kv, **kw):
    return Batch(tuple(q), tuple(kv), **kw)


STEP = [
    B([1], [1]),
    B([1, 1, 1], [1, 17, 300]),
    B([1] * 5, [64, 65, 63, 128, 1000], heads=8, kv_heads=1, dim=128, dtype="f16"),
    B([1, 1], [257, 4097], heads=8, kv_heads=8, dim=128, page=64),
    B([1, 1, 1], [5, 700, 90], dim=128, fp8=True),
    B([1, 1, 1], [5, 700, 90], fp8=True, dtype="f16", page=32),
    B([1, 1], [300, 31], dim=256, heads=6, kv_heads=3),
    B([1, 1], [300, 31], dim=256, fp8=True),
    B([1, 1, 1], [33, 450, 2], dim=80, page=1),
    B([1, 1], [129, 450], dim=48, page=8, fp8=True, heads=5, kv_heads=1),
    B([1, 0, 1], [40, 77, 0], dtype="f16"),              # no new token; no key at all
    B([1, 1], [200, 3000], page=1024, heads_first=True, dim=128),
    B([1, 1, 1], [100, 900, 5000], window=100, dim=128),
    B([1, 1], [513, 100], heads=40, kv_heads=1, dim=64),  # 40 rows: three row tiles
    B([1] * 33, list(range(1, 34)), heads=2, kv_heads=2, page=4),
]
FEW = [
    B([3, 1, 6], [3, 50, 700], heads=8, kv_heads=2, dim=128),
    B([4, 2, 5], [600, 333, 5], heads=16, kv_heads=2, dtype="f16", window=64, page=32),
    B([7, 8], [7, 1000], heads=4, kv_heads=1, fp8=True, dim=128),
    B([5, 3], [2, 3], heads=4, kv_heads=2),               # more tokens than keys: rows keep nothing
    B([9, 16], [100, 257], causal=False, dim=96),
    B([9, 16], [100, 257], causal=False, window=20),
    B([16, 1, 15], [16, 1, 400], heads=4, kv_heads=4, dim=256, fp8=True, dtype="f16"),
    B([13, 2], [65, 2000], heads=10, kv_heads=2, dim=80, pad=3),
    B([2, 2], [128, 640], window=1, dim=64),
    B([2, 3], [30000, 8], heads=2, kv_heads=1, dtype="f16", window=2 ** 31 - 1),
]
CHUNK = [
    B([130], [130], heads=4, kv_heads=1, dim=128),
    B([257, 1, 64], [257, 900, 500], heads=8, kv_heads=2, dim=128, page=64),
    B([200, 31], [200, 300], heads=2, kv_heads=2, dtype="f16"),
    B([150, 90], [500, 90], heads=5, kv_heads=1, dim=80, page=128),
    B([129, 300], [129, 700], heads=4, kv_heads=2, dim=128, window=130),
    B([129, 60], [200, 260], heads=4, kv_heads=2, dim=128, causal=False),
    B([200, 100], [150, 100], heads=4, kv_heads=2, dim=64, pad=5),   # rows that keep nothing
    B([300, 40], [300, 512], heads=4, kv_heads=1, dim=128, fp8=True),
    B([140, 260], [400, 260], heads=2, kv_heads=1, dim=64, fp8=True, dtype="f16", page=32),
    B([100, 33], [300, 33], heads=4, kv_heads=2, dim=256),
    B([70, 33], [300, 33], heads=4, kv_heads=2, dim=192, fp8=True),
    B([100, 200], [333, 200], heads=4, kv_heads=2, dim=128, page=2),
    B([128, 129, 127], [128, 256, 384], heads=1, kv_heads=1, dim=64, page=256, heads_first=True),
    B([200, 90], [200, 301], heads=4, kv_heads=2, dim=48),
    B([200, 90], [200, 301], heads=4, kv_heads=2, dim=96, fp8=True),
    B([200, 90], [200, 301], heads=4, kv_heads=2, dim=16, fp8=True, page=8),
    B([90], [1300], heads=16, kv_heads=2, dim=128, window=200, page=64),
]


@pytest.mark.parametrize("c", STEP + FEW + CHUNK, ids=str)
def test_attention(gpu, c):
    s = make(c)
    device_flags()
    out, lse = attend(gpu, c, s)
    torch.cuda.synchronize()
    assert device_flags() == 0
    check_attention(c, s, out, lse)


def spread(n, longest, **kw):
    """n sequences of one new token, from ``longest`` keys down to one."""
    return B([1] * n, [max(1, longest - i * longest // n) for i in range(n)], **kw)


# Key ranges split over as many CTAs as there is room for at once: eights, sixes, fours, threes,
# twos, one; a second kernel beyond; around the sizes where the split begins and where 33 rows
# and more change kernels.
ROUND = [
    spread(4, 1030, heads=16, kv_heads=8, dim=128),
    spread(5, 900, heads=8, kv_heads=8, dim=128, dtype="f16"),
    spread(9, 700, heads=16, kv_heads=8, dim=128, fp8=True),
    spread(12, 641, heads=8, kv_heads=8, dim=112, page=8),
    spread(16, 300, heads=8, kv_heads=8, dim=128),
    spread(24, 280, heads=16, kv_heads=8, dim=128, fp8=True, page=4),
    spread(14, 520, heads=8, kv_heads=8, dim=64),
    spread(7, 1200, heads=8, kv_heads=8, dim=64, fp8=True, dtype="f16", page=1),
    spread(2, 5000, heads=8, kv_heads=8, dim=32),
    spread(2, 1100, heads=8, kv_heads=4, dim=256),
    B([1, 1, 1], [256, 257, 255], heads=4, kv_heads=2, dim=128),
    B([1, 0, 1, 1], [257, 70, 0, 384], heads=4, kv_heads=2, dim=64, pad=2),
    B([4, 4, 1], [700, 4, 260], heads=8, kv_heads=2, dim=128, window=300),
    B([9, 1], [512, 300], heads=8, kv_heads=2, dim=128),
    B([9, 1, 9], [513, 300, 3], heads=8, kv_heads=2, dim=128, pad=1),
    B([9, 5], [600, 513], heads=8, kv_heads=2, dim=80, fp8=True),
    B([9, 5], [600, 513], heads=8, kv_heads=2, dim=64),
    B([16, 2], [700, 900], heads=8, kv_heads=2, dim=96, window=500, page=64),
    B([33, 33], [1500, 40], heads=2, kv_heads=2, dim=128, dtype="f16", causal=False),
]


@pytest.mark.parametrize("c", ROUND, ids=str)
def test_attention_in_one_round_and_around_the_choices(gpu, c):
    s = make(c)
    device_flags()
    out, lse = attend(gpu, c, s)
    again, _ = attend(gpu, c, s)
    torch.cuda.synchronize()
    assert device_flags() == 0
    n = s["cpu"]["cu"][-1]
    assert torch.equal(out[:n], again[:n])
    check_attention(c, s, out, lse)


@pytest.mark.parametrize("c", [B([9, 12], [700, 600], heads=8, kv_heads=2, dim=128, window=400),
                               B([40, 70], [300, 70], heads=4, kv_heads=1, dim=80)], ids=str)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")], ids=["nan", "inf"])
def test_a_bad_value_that_some_rows_drop(gpu, c, bad):
    """One value element of one key of the first sequence is bad: rows that keep it get a bad
    element there, rows that drop it (and every other column) are as they were."""
    s = make(c)
    clean, lse0 = attend(gpu, c, s)
    # Half of the rows come before the key; the window leaves it to half of the rows.
    key, col = 280 if c.window == 0 else 295, 5
    page = s["table"][0, key // c.page].item()
    s["v_cache"][page, key % c.page, 0, col] = bad
    out, lse = attend(gpu, c, s)
    torch.cuda.synchronize()
    assert torch.equal(lse, lse0)
    q0, off = c.q_lens[0], c.kv_lens[0] - c.q_lens[0]
    kept = torch.tensor([key <= off + i and (c.window == 0 or key > off + i - c.window)
                         for i in range(q0)])
    heads = c.heads // c.kv_heads
    hit = torch.zeros(out.shape, dtype=torch.bool)
    hit[:q0, :heads, col] = kept[:, None]
    assert not torch.isfinite(out.cpu()[hit]).any()
    same = torch.ones(out.shape, dtype=torch.bool)
    same[:q0, :heads, :] = False
    assert torch.equal(out.cpu()[same], clean.cpu()[same])
    # Rows that drop it: recomputed where the products of whole tiles met it.
    rest = ~hit & ~same
    a, b = out.cpu()[rest].double(), clean.cpu()[rest].double()
    assert torch.isfinite(a).all()
    # Both are within the tolerance of the header of the exact value, A and the result at most
    # the largest value.
    ds = ((c.dim / 16 + 6) * 2.0 ** -23 * score_size(s["cpu"], c.dim ** -0.5)).max()
    top = np.nan_to_num(np.abs(s["cpu"]["v_cache"])).max()
    half = torch.finfo(DT[c.dtype]).eps / 2
    rel = half + 2 * ds + (max(c.kv_lens) / 16 + 24) * 2.0 ** -23
    assert kept.any() and not kept.all()
    assert ((a - b).abs() <= 2 * (half * (1 + rel) + rel) * top).all()


@pytest.mark.parametrize("c", [STEP[2], FEW[0], CHUNK[1], CHUNK[7]], ids=str)
def test_attention_repeats_bit_for_bit_and_without_lse(gpu, c):
    s = make(c)
    a, la = attend(gpu, c, s)
    b, lb = attend(gpu, c, s)
    o = attend(gpu, c, s, return_lse=False)
    assert torch.equal(a, b) and torch.equal(a, o) and torch.equal(la, lb)


@pytest.mark.parametrize("c", [STEP[3], FEW[0], CHUNK[0], CHUNK[3]], ids=str)
def test_attention_loose_bounds_and_scale(gpu, c):
    """max_q and max_kv may be any upper bounds; another scale."""
    s = make(c)
    out, lse = attend(gpu, c, s, max_q=s["max_q"] + 300, max_kv=None, scale=0.3)
    check_attention(c, s, out, lse, 0.3)


@pytest.mark.parametrize("c", [B([3, 1], [40, 700], pad=4, dim=128),
                               B([200, 9], [300, 900], pad=6, dim=128),
                               B([200, 9], [300, 900], pad=6, dim=128, fp8=True)], ids=str)
def test_padding_rows_and_guard_bands_are_left_alone(gpu, c):
    s = make(c)
    t, n = s["q"].shape[0], s["cpu"]["cu"][-1]
    buf = torch.full((t + 4, c.heads + 1, c.dim + 8), 7.0, dtype=DT[c.dtype], device="cuda")
    lbuf = torch.full((t + 4, c.heads), 7.0, device="cuda")
    out, lse = buf[2:2 + t, :c.heads, :c.dim], lbuf[2:2 + t]
    attend(gpu, c, s, out=out, lse=lse)
    torch.cuda.synchronize()
    check_attention(c, s, out, lse)
    assert torch.all(out[n:] == 7) and torch.all(lse[n:] == 7)
    assert torch.all(buf[:2] == 7) and torch.all(buf[2 + t:] == 7)
    assert torch.all(buf[:, c.heads:] == 7) and torch.all(buf[..., c.dim:] == 7)
    assert torch.all(lbuf[:2] == 7) and torch.all(lbuf[2 + t:] == 7)


@pytest.mark.parametrize("c", [B([2, 1], [300, 40], dim=128), B([150, 3], [300, 40], dim=128),
                               B([150, 3], [300, 40], dim=128, fp8=True)], ids=str)
def test_bad_pages_and_lengths_are_flagged(gpu, c):
    """A page outside the cache, a length beyond the table: nothing out of range
    is touched, the flag is set, other sequences are right."""
    from rmsnorm_fp8_quantization_gb300 import gbnorm as G
    s = make(c)
    good = s["table"].clone()
    for bad in (-1, 10 ** 6):
        s["table"][1, 0] = bad
        device_flags()
        out, lse = attend(gpu, c, s)
        torch.cuda.synchronize()
        assert device_flags() == G.GBN_DEVICE_ERR_BAD_INDEX
        n = c.q_lens[0]
        s["table"].copy_(good)
        ok, ol = attend(gpu, c, s)
        assert torch.equal(out[:n], ok[:n]) and torch.equal(lse[:n], ol[:n])
    s["kv_lens"][1] = 10 ** 7
    attend(gpu, c, s, max_kv=None)
    assert device_flags() == G.GBN_DEVICE_ERR_BAD_INDEX
    assert device_flags() == 0


@pytest.mark.parametrize("c", [
    B([6, 5], [70, 300], heads=4, kv_heads=2, dim=64),
    B([6, 5], [70, 3000], heads=8, kv_heads=1, dim=128, dtype="f16", window=60),
    B([6, 5], [70, 300], heads=4, kv_heads=2, dim=128, fp8=True),
    B([150, 90], [150, 700], heads=4, kv_heads=2, dim=128),
    B([150, 90], [150, 700], heads=4, kv_heads=1, dim=64, fp8=True, window=100),
    B([40, 50], [40, 130], heads=2, kv_heads=1, dim=256),
], ids=str)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")], ids=["nan", "inf"])
def test_what_stands_in_a_dropped_key_does_not_enter(gpu, c, bad):
    """Keys and values that some rows of a tile keep and others drop, not finite:
    the rows that drop them are as if they were not there."""
    s = make(c)
    if c.fp8 and bad == float("inf"):
        bad = float("nan")  # E4M3 has no infinity
    cpu = s["cpu"]
    poisoned = [c.kv_lens[0] - 2, c.kv_lens[1] - 3]
    for name in ("k_cache", "v_cache"):
        host = s[name].float().cpu()
        for b, t in enumerate(poisoned):
            host[cpu["table"][b][t // c.page], t % c.page, :, 3:9] = bad
        s[name].copy_(host.to(s[name].dtype))
        cpu[name] = s[name].float().cpu().double().numpy()
    out, lse = attend(gpu, c, s)
    torch.cuda.synchronize()
    first = []  # rows before the poisoned position, per sequence
    for b in range(2):
        off = c.kv_lens[b] - c.q_lens[b]
        first += [cpu["cu"][b] + i for i in range(c.q_lens[b])
                  if off + i < poisoned[b] or (c.window and off + i - c.window >= poisoned[b])]
    rows = torch.tensor(first)
    assert torch.isfinite(out[rows.cuda()].float()).all()
    # against the oracle: only those rows (the others are not finite on both sides)
    with np.errstate(invalid="ignore", over="ignore"):
        ref, rl, mag = P.paged_attend(cpu["q"], cpu["k_cache"], cpu["v_cache"], cpu["cu"],
                                      cpu["kv_lens"], cpu["table"], c.dim ** -0.5, c.causal,
                                      c.window, cpu["inv"], cpu["inv"])
    clean = {**cpu, "k_cache": np.where(np.isfinite(cpu["k_cache"]), cpu["k_cache"], 0)}
    ds = (c.dim / 16 + 6) * 2.0 ** -23 * score_size(clean, c.dim ** -0.5)
    dt = DT[c.dtype]
    half = torch.finfo(dt).eps / 2
    rel = (torch.finfo(torch.float16 if c.fp8 else dt).eps / 2 + 2 * ds[..., None]
           + (max(c.kv_lens) / 16 + 24) * 2.0 ** -23)
    inner = mag * rel
    lim = half * (np.abs(ref) + inner) + inner + (2.0 ** -25 if c.dtype == "f16" else 0.0)
    err = np.abs(out.double().cpu().numpy() - ref)
    r = rows.numpy()
    assert (err[r] <= lim[r]).all(), (np.nanmax(err[r] / lim[r]))
    others = [i for i in range(cpu["cu"][-1]) if i not in set(first)]
    assert torch.isnan(out[torch.tensor(others).cuda()].float()).any(-1).all()


def test_attention_graph_with_lengths_that_change(gpu):
    """One captured call follows the lengths and the table on the device."""
    c = B([1, 1, 1], [900, 40, 300], dim=128, heads=8, kv_heads=2)
    s = make(c)
    ws = gpu.paged_attention_workspace(s["q"], s["k_cache"], s["table"], max_q=1)
    out = torch.empty_like(s["q"])
    graph = torch.cuda.CUDAGraph()
    attend(gpu, c, s, max_kv=None, out=out, workspace=ws, return_lse=False)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        attend(gpu, c, s, max_kv=None, out=out, workspace=ws, return_lse=False)
    for lens in ([900, 40, 300], [5, 40, 1], [64, 7, 299]):
        s["kv_lens"].copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        c2 = dataclasses.replace(c, kv_lens=tuple(lens))
        s["cpu"]["kv_lens"] = lens
        check_attention(c2, s, out, None)


def test_two_streams_with_their_own_workspaces(gpu):
    c = B([1, 1], [4000, 3000], dim=128, heads=8, kv_heads=2)
    a, b = make(c), make(dataclasses.replace(c, seed=1))
    ra, rb = (attend(gpu, c, s)[0] for s in (a, b))
    outs, streams = [], [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, st in ((a, streams[0]), (b, streams[1])):
            with torch.cuda.stream(st):
                outs.append((attend(gpu, c, s)[0], ra if s is a else rb))
    torch.cuda.synchronize()
    for o, r in outs:
        assert torch.equal(o, r)


@pytest.mark.parametrize("c", [B([2, 1], [40, 33], heads=16, kv_heads=8, dim=128),
                               B([100, 30], [100, 90], heads=16, kv_heads=8, dim=128),
                               B([2, 1], [40, 33], heads=16, kv_heads=8, dim=128, fp8=True),
                               B([100, 30], [100, 90], heads=16, kv_heads=8, dim=128, fp8=True),
                               B([2, 1], [40, 33], heads=16, kv_heads=8, dim=128, page=2)], ids=str)
def test_caches_beyond_two_to_the_31_elements(gpu, c):
    """Pages whose element (and byte) offsets do not fit 32 bits, written by the
    append and read by the attention."""
    s = make(c)
    used = s["k_cache"].shape[0]
    pages = (1 << 32) // (c.page * c.kv_heads * c.dim) + used + 5  # over 2^32 elements
    big = {}
    for n in ("k_cache", "v_cache"):
        big[n] = torch.empty(pages, *s[n].shape[1:], dtype=s[n].dtype, device="cuda")
        big[n][pages - used:].view(torch.uint8).copy_(s[n].view(torch.uint8))
    s["table"] = torch.where(s["table"] >= 0, s["table"] + (pages - used), -1).int()
    out, lse = attend(gpu, c, {**s, **big})
    torch.cuda.synchronize()
    check_attention(c, s, out, lse)
    f = gpu.rope_frequencies(c.dim)
    before = s["k_cache"].cpu().clone(), s["v_cache"].cpu().clone()
    qo = gpu.paged_append(s["k"], s["v"], big["k_cache"], big["v_cache"], s["cu"], s["kv_lens"],
                          s["table"], q=s["q"], inv_freq=f, k_scale=s["scale"], v_scale=s["scale"])
    torch.cuda.synchronize()
    tail = {n: big[n][pages - used:].clone() for n in big}
    del big
    check_append(c, {**s, **tail}, before, qo, f.cpu().numpy(), "half", 1.0)


@pytest.mark.parametrize("c", [B([1, 2], [300, 77], dim=128), B([100, 40], [300, 77], dim=64),
                               B([100, 1], [300, 77], dim=128, fp8=True)], ids=str)
def test_keys_and_values_in_one_tensor_and_strided_queries(gpu, c):
    """[pages, 2, page, heads, dim] caches, q as a view of a packed projection, the
    table as a view of a wider one, other values around all of them."""
    s = make(c)
    one = torch.stack([s["k_cache"], s["v_cache"]], 1)
    kc, vc = one[:, 0], one[:, 1]
    wide = torch.randn(s["q"].shape[0], c.heads + 3, c.dim, device="cuda").to(s["q"].dtype)
    wide[:, 1:1 + c.heads] = s["q"]
    table = torch.full((s["table"].shape[0], s["table"].shape[1] + 4), 10 ** 9, dtype=torch.int32,
                       device="cuda")
    table[:, :-4] = s["table"]
    v = {**s, "k_cache": kc, "v_cache": vc, "q": wide[:, 1:1 + c.heads], "table": table[:, :-4]}
    out, lse = attend(gpu, c, v)
    ref, rl = attend(gpu, c, s)
    assert torch.equal(out, ref) and torch.equal(lse, rl)
    f = gpu.rope_frequencies(c.dim)
    before = s["k_cache"].cpu().clone(), s["v_cache"].cpu().clone()
    qo = gpu.paged_append(s["k"], s["v"], kc, vc, s["cu"], s["kv_lens"], table[:, :-4], q=v["q"],
                          inv_freq=f, k_scale=s["scale"], v_scale=s["scale"])
    check_append(c, {**s, "k_cache": kc, "v_cache": vc}, before, qo, f.cpu().numpy(), "half", 1.0)


def test_attention_refuses_q_as_its_output(gpu):
    c = B([1], [20])
    s = make(c)
    with pytest.raises(ValueError):
        attend(gpu, c, s, out=s["q"])


def test_more_sequences_than_are_taken_by_length(gpu):
    n = 300
    c = B([9 + i % 3 for i in range(n)], [9 + i % 3 + (i * 37) % 80 for i in range(n)], heads=8,
          kv_heads=1, dim=64)
    s = make(c)
    out, lse = attend(gpu, c, s)
    torch.cuda.synchronize()
    check_attention(c, s, out, lse)


@pytest.mark.parametrize("q,kv", [((3, 1), (90, 700)), ((150, 70), (150, 700))])
def test_e4m3_scales_of_any_sign_and_large_queries(gpu, q, kv):
    """A negative k_scale_inv turns the scores' sign, 0 makes them equal; bf16
    queries far beyond f16's range, with a scale to match, change nothing."""
    c = B(q, kv, heads=8, kv_heads=2, dim=128, fp8=True)
    s = make(c)
    plus, lp = attend(gpu, c, s)
    s["q"].neg_()
    minus, lm = gpu.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["cu"], s["kv_lens"],
                                    s["table"], max_q=s["max_q"], k_scale_inv=-s["scale_inv"],
                                    v_scale_inv=s["scale_inv"], return_lse=True)
    assert torch.equal(plus, minus) and torch.equal(lp, lm)
    s["q"].neg_()
    for e in (90, -90):
        big = s["q"] * 2.0 ** e
        out = gpu.paged_attention(big, s["k_cache"], s["v_cache"], s["cu"], s["kv_lens"],
                                  s["table"], max_q=s["max_q"], k_scale_inv=s["scale_inv"],
                                  v_scale_inv=s["scale_inv"], scale=c.dim ** -0.5 * 2.0 ** -e)
        # the same bits but for roundings of the (power-of-two scaled) score factor
        assert torch.equal(out, plus)
    zero = torch.zeros(1, device="cuda")
    out, lse = gpu.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["cu"], s["kv_lens"],
                                   s["table"], max_q=s["max_q"], k_scale_inv=zero,
                                   v_scale_inv=s["scale_inv"], return_lse=True)
    s["cpu"]["q"] = s["cpu"]["q"] * 0
    check_attention(c, s, out, lse)


def test_stream_argument_while_the_current_stream_is_busy(gpu):
    """A call on another stream than the current one, its workspace and outputs
    allocated by the call, while the current stream reuses freed memory."""
    c = B([1, 1], [9000, 7000], dim=128, heads=8, kv_heads=2)
    s = make(c)
    ref, rl = attend(gpu, c, s)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for handle in (side, side.cuda_stream):
        outs = []
        for _ in range(30):
            outs.append(attend(gpu, c, s, stream=handle))
            junk = [torch.full((1 << 20,), 3.0, device="cuda") for _ in range(4)]
            del junk
        torch.cuda.synchronize()
        for o, l in outs:
            assert torch.equal(o, ref) and torch.equal(l, rl)
    q, k = torch.randn(2, 5, 4, 64, device="cuda"), torch.randn(2, 5, 2, 64, device="cuda")
    f = gpu.rope_frequencies(64)
    want = gpu.rope_fwd(q, k, f)
    torch.cuda.synchronize()
    got = gpu.rope_fwd(q, k, f, stream=side)
    side.synchronize()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


# ---------------------------------------------------------------- append

def check_append(c, s, before, q_out, f, layout, mscale):
    cpu = s["cpu"]
    dt = DT[c.dtype]
    n = cpu["cu"][-1]
    r = 2 * len(f)
    pos = np.zeros(n, dtype=np.int64)
    where = list(P.slots(cpu["cu"], cpu["kv_lens"], cpu["table"], c.page))
    for row, t, _, _ in where:
        pos[row] = t
    from test_gpu_rope import check
    if q_out is not None:
        ref = P.rotate(cpu["q"][:n], pos, f, layout, mscale)
        check(q_out[:n], cpu["q"][:n], ref, mscale, r, layout, dt, "q")
    kr = P.rotate(cpu["k"][:n], pos, f, layout, mscale)
    rows = [w[0] for w in where]
    pg = torch.tensor([w[2] for w in where])
    sl = torch.tensor([w[3] for w in where])
    kc, vc = s["k_cache"].cpu(), s["v_cache"].cpu()
    raw = (lambda x: x.view(torch.uint8)) if c.fp8 else (lambda x: x.view(torch.int16))
    if not c.fp8:
        check(kc[pg, sl], cpu["k"][rows], kr[rows], mscale, r, layout, dt, "k")
        if r < c.dim:
            assert torch.equal(raw(kc[pg, sl])[..., r:], raw(s["k"].cpu()[rows])[..., r:])
        assert torch.equal(raw(vc[pg, sl]), raw(s["v"].cpu()[rows]))
    else:
        gain = float(s["scale"])
        for got, want in ((kc, kr[rows] * gain), (vc, cpu["v"][rows] * gain)):
            want = np.clip(want, -448, 448)
            code = torch.from_numpy(want).float().to(torch.float8_e4m3fn)
            mine = got.view(torch.uint8)[pg, sl].view(torch.float8_e4m3fn)
            differ = mine.view(torch.uint8) != code.view(torch.uint8)
            # one step at most, and only where fp32 evaluation crosses a border
            err = (mine.double() - torch.from_numpy(want)).abs()
            lim = np.maximum(np.abs(want) * 2.0 ** -4, 2.0 ** -10) * (1 + 2.0 ** -10)
            assert (err.numpy() <= lim).all()
            assert int(differ.sum()) <= 1e-3 * differ.numel() + 2
    keep = torch.ones(kc.shape[:2], dtype=torch.bool)
    keep[pg, sl] = False
    for got, was in zip((kc, vc), before):
        assert torch.equal(raw(got.contiguous())[keep], raw(was.contiguous())[keep])


APPEND = [
    (B([1], [1]), 64, "half", 1.0),
    (B([1, 1, 1], [1, 17, 300], dim=128, heads=8), 128, "half", 1.2),
    (B([1] * 40, list(range(1, 41)), heads=2), 64, "interleaved", 1.0),
    (B([3, 0, 5], [3, 20, 700], dtype="f16", page=32, pad=3), 32, "half", 1.0),
    (B([100, 31], [100, 300], dim=128, page=64), 128, "half", 1.0),
    (B([100, 31], [100, 300], dim=96, page=64, fp8=True), 48, "interleaved", 1.1),
    (B([1, 1], [10, 300], fp8=True, dtype="f16"), 64, "half", 1.0),
    (B([10, 3], [10, 30], dim=80, heads_first=True, page=8), 40, "half", 1.0),
    (B([10, 3], [10, 30], dim=40, fp8=True, page=1), 20, "half", 1.0),
    (B([10, 3], [10, 30], dim=33, heads=2, kv_heads=1, page=4), 6, "interleaved", 1.0),
    (B([10, 3], [10, 30], dim=64), 0, "half", 1.0),
    (B([700, 1, 900], [700, 50, 1000], heads=8, kv_heads=8, page=128), 64, "half", 1.0),
]


@pytest.mark.parametrize("a", APPEND, ids=lambda a: f"{a[0]}-r{a[1]}-{a[2]}")
def test_append(gpu, a):
    c, r, layout, ms = a
    s = make(c)
    f = gpu.rope_frequencies(r, 10000.0, device="cpu") if r else torch.zeros(0, dtype=torch.float64)
    before = s["k_cache"].cpu().clone(), s["v_cache"].cpu().clone()
    device_flags()
    q_out = torch.full_like(s["q"], 7.0)
    got = gpu.paged_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["cu"], s["kv_lens"],
                           s["table"], q=s["q"], inv_freq=f.cuda() if r else None, layout=layout,
                           mscale=ms, k_scale=s["scale"], v_scale=s["scale"], q_out=q_out)
    torch.cuda.synchronize()
    assert got is q_out and device_flags() == 0
    assert torch.all(q_out[s["cpu"]["cu"][-1]:] == 7)
    check_append(c, s, before, q_out, f.numpy(), layout, ms)


def test_append_many_sequences(gpu):
    """More sequences than one probe round of the search covers, empty ones among them."""
    n = 3000
    q = [(i * 7) % 3 for i in range(n)]
    c = B(q, [a + 2 for a in q], heads=1, kv_heads=1, page=4)
    s = make(c)
    before = s["k_cache"].cpu().clone(), s["v_cache"].cpu().clone()
    f = gpu.rope_frequencies(64)
    qo = gpu.paged_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["cu"], s["kv_lens"],
                          s["table"], q=s["q"], inv_freq=f)
    check_append(c, s, before, qo, f.cpu().numpy(), "half", 1.0)


def test_append_views_of_a_packed_projection_and_saturation(gpu):
    c = B([6, 2], [9, 70], heads=4, kv_heads=2, dim=64, fp8=True)
    s = make(c)
    x = torch.cat([s["q"], s["k"] * 1000, s["v"]], 1)
    x[3, 5, 7] = float("nan")
    q, k, v = x.split([4, 2, 2], 1)
    one = torch.ones(1, device="cuda")
    gpu.paged_append(k, v, s["k_cache"].view(torch.uint8), s["v_cache"], s["cu"], s["kv_lens"],
                     s["table"], k_scale=one, v_scale=one)
    for row, _, pg, sl in P.slots(s["cpu"]["cu"], s["cpu"]["kv_lens"], s["cpu"]["table"], c.page):
        for src, dst in ((k, s["k_cache"]), (v, s["v_cache"])):
            want = src[row].float().clamp(-448, 448).to(torch.float8_e4m3fn)
            assert torch.equal(dst[pg, sl].view(torch.uint8), want.view(torch.uint8))


def test_append_bad_pages_and_lengths(gpu):
    from rmsnorm_fp8_quantization_gb300 import gbnorm as G
    c = B([2, 3], [20, 40])
    s = make(c)
    f = gpu.rope_frequencies(64)
    before = s["k_cache"].clone().view(torch.int16)

    def call():
        device_flags()
        gpu.paged_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["cu"], s["kv_lens"],
                         s["table"], inv_freq=f)
        return device_flags()

    page = s["table"][1, 2].clone()
    for bad in (-1, 10 ** 6):
        s["table"][1, 2] = bad     # positions 37, 38, 39
        assert call() == G.GBN_DEVICE_ERR_BAD_INDEX
        after = s["k_cache"].view(torch.int16)
        changed = (after != before).flatten(1).any(1).nonzero().flatten().tolist()
        assert changed == [int(s["table"][0, 1])]
    s["table"][1, 2] = page
    s["kv_lens"][1] = 2            # token before position 0
    assert call() == G.GBN_DEVICE_ERR_BAD_INDEX
    s["kv_lens"][1] = 10 ** 6      # beyond the table
    assert call() == G.GBN_DEVICE_ERR_BAD_INDEX
    s["kv_lens"][1] = 40
    assert call() == 0


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_prompt_then_steps_match_one_pass(gpu, fp8):
    """A prompt in two chunks and then single tokens, each appended and attended
    to, against the oracle on the whole sequence (read back from the cache): the
    way a server uses the three operators."""
    hq, hk, d, page = 8, 2, 128, 16
    lens = (70, 45)
    total = tuple(n + 4 for n in lens)
    g = torch.Generator().manual_seed(3)
    seqs = [tuple(torch.randn(n, h, d, generator=g).bfloat16().cuda() for h in (hq, hk, hk))
            for n in total]
    need = [-(-n // page) for n in total]
    table = torch.full((2, max(need)), -1, dtype=torch.int32)
    order = torch.randperm(sum(need), generator=g).int()
    table[0, :need[0]], table[1, :need[1]] = order[:need[0]], order[need[0]:]
    table = table.cuda()
    cdt = torch.float8_e4m3fn if fp8 else torch.bfloat16
    kc = torch.zeros(sum(need), page, hk, d, dtype=cdt, device="cuda")
    vc = torch.zeros_like(kc)
    sc = torch.full((1,), 16.0, device="cuda") if fp8 else None
    inv = 1.0 / sc if fp8 else None
    f = gpu.rope_frequencies(d, 10000.0)
    done, got = [0, 0], [[], []]
    rotated = [[], []]
    chunks = [(50, 45), (20, 0), (1, 1), (1, 1), (1, 1), (1, 1)]
    for ch in chunks:
        q, k, v = (torch.cat([seqs[b][i][done[b]:done[b] + ch[b]] for b in (0, 1)]) for i in (0, 1, 2))
        done = [done[b] + ch[b] for b in (0, 1)]
        cu = torch.tensor([0, ch[0], ch[0] + ch[1]], dtype=torch.int32, device="cuda")
        kv = torch.tensor(done, dtype=torch.int32, device="cuda")
        qr = gpu.paged_append(k, v, kc, vc, cu, kv, table, q=q, inv_freq=f, k_scale=sc, v_scale=sc)
        o = gpu.paged_attention(qr, kc, vc, cu, kv, table, max_q=max(ch), k_scale_inv=inv,
                                v_scale_inv=inv)
        for b, (lo, hi) in enumerate(((0, ch[0]), (ch[0], ch[0] + ch[1]))):
            got[b].append(o[lo:hi])
            rotated[b].append(qr[lo:hi])
    for b in (0, 1):
        c = B([total[b]], [total[b]], heads=hq, kv_heads=hk, dim=d, fp8=fp8)
        s = {"cpu": dict(q=torch.cat(rotated[b]).double().cpu().numpy(),
                         k_cache=kc.double().cpu().numpy(), v_cache=vc.double().cpu().numpy(),
                         cu=[0, total[b]], kv_lens=[total[b]], table=table[b:b + 1].cpu().numpy(),
                         inv=1.0 / 16 if fp8 else 1.0)}
        check_attention(c, s, torch.cat(got[b]), None)
