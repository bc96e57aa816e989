"""Attention over whole sequences and its backward pass against the definition in 64 bits."""
import pytest
import torch

from attention_train_cases import Case, check, define, flat, make

pytestmark = pytest.mark.gpu
F16 = torch.float16


def flags():
    from rmsnorm_fp8_quantization_gb300 import gbnorm as G
    st, v = G.gbn_device_error(True)
    assert st == G.GBN_OK
    return v


def both(gpu, s):
    out, lse = gpu.attention_fwd(s["q"], s["k"], s["v"], **s["kw"])
    dq, dk, dv = gpu.attention_bwd(s["dout"], s["q"], s["k"], s["v"], out, lse, **s["kw"])
    return dict(out=out, lse=lse, dq=dq, dk=dk, dv=dv)


CASES = {
    # one token; a tile; one more; several
    "one token": Case((1,), uniform=True),
    "uniform 128": Case((128, 128), uniform=True),
    "uniform 129": Case((129, 129), uniform=True, dim=128),
    "uniform 385 f16": Case((385,), uniform=True, dtype=F16),
    "packed projection": Case((200, 200), uniform=True, packed=True, dim=128, heads=8),
    "own keys a head": Case((260, 260), uniform=True, heads=3, kv_heads=3),
    "one kv head": Case((300,), uniform=True, heads=5, kv_heads=1, dim=96),
    "not causal": Case((130, 130), uniform=True, causal=False, dim=128),
    "window": Case((700,), uniform=True, window=100, dim=128),
    "window of one": Case((300,), uniform=True, window=1),
    "window, not causal": Case((400,), uniform=True, window=150, causal=False, dtype=F16),
    "window wider than all": Case((150,), uniform=True, window=2 ** 31 - 1),
    # ragged: lengths of zero and one among them, padding around
    "ragged": Case((1, 0, 57, 128, 300, 0, 2, 511), packed=True, dim=128),
    "ragged f16": Case((1, 0, 57, 128, 300, 0, 2, 511), heads=8, kv_heads=8, dtype=F16, lead=5, trail=9),
    "padded": Case((33, 257), lead=3, trail=200, dim=80),
    "all empty": Case((0, 0), trail=4),
    # queries and keys of their own
    "cross": Case((3, 140, 1, 0, 65), (211, 1, 300, 7, 128), causal=False, dim=96),
    "cross, no keys": Case((3, 140), (0, 20), causal=False),
    "more keys, causal": Case((5, 130), (400, 131), dim=128),
    "fewer keys, causal": Case((300, 129, 10), (100, 1, 0), dim=128),   # rows that keep nothing
    "fewer keys, window": Case((400,), (150,), window=20, dtype=F16),
    "few queries, many keys": Case((2, 1), (3000, 2500), causal=False, dim=128),
    "many queries, few keys": Case((2000,), (3,), causal=False, heads=8, kv_heads=1),
    # head sizes
    "dim 8": Case((140,), uniform=True, dim=8),
    "dim 16 f16": Case((140,), uniform=True, dim=16, dtype=F16),
    "dim 40": Case((200,), uniform=True, dim=40, packed=True),
    "dim 72": Case((200,), uniform=True, dim=72, packed=True, dtype=F16),
    "dim 120": Case((200,), uniform=True, dim=120),
    # values: large scores, small and large gradients
    "large scores": Case((300,), uniform=True, dim=128, q_std=20.0),
    "small gradients f16": Case((700,), uniform=True, dtype=F16, dout_std=1e-4, causal=False),
    "large gradients f16": Case((300,), uniform=True, dtype=F16, dout_std=3000.0, dim=128),
    "small gradients": Case((300,), uniform=True, dout_std=1e-20, dim=128),
    "scale": Case((150,), uniform=True, scale=0.3),
    # few CTAs of many steps: shared among several, added up afterwards
    "shared steps": Case((1500,), uniform=True, heads=4, kv_heads=1, dim=128),
    "shared steps, ragged f16": Case((900, 1, 0, 333), heads=6, kv_heads=1, dim=96, dtype=F16, lead=3, trail=5),
    "shared steps of dq": Case((100,), (4100,), causal=False, heads=1, kv_heads=1, dim=72),
    "shared steps, window": Case((3000,), uniform=True, heads=8, kv_heads=1, window=900),
    # many CTAs of few steps: several heads of a tile in one, an odd number of them, lengths that differ
    "heads in turn": Case((130,) * 40, uniform=True, heads=24, kv_heads=12),
    "heads in turn, dim 128": Case((129,) * 40, uniform=True, heads=24, kv_heads=12, dim=128, dtype=F16),
    "odd heads in turn": Case((200,) * 60, uniform=True, heads=9, kv_heads=9, dim=96, causal=False),
    "heads in turn, window": Case((700,) * 16, uniform=True, heads=16, kv_heads=4, dim=72, window=100),
    "heads in turn, ragged": Case(tuple(3 + 37 * i % 200 for i in range(100)), heads=16, kv_heads=16,
                                  dim=40, dtype=F16, lead=2, trail=9),
    "heads in turn, cross": Case((1, 140, 0) * 50, (300, 5, 64) * 50, heads=12, kv_heads=12, dim=128, causal=False),
    "long": Case((2500,), uniform=True, heads=2, kv_heads=1, dim=128),
    "long f16, not causal": Case((2500,), uniform=True, heads=2, kv_heads=1, dtype=F16, causal=False),
}


@pytest.mark.parametrize("name", CASES)
def test_against_definition(gpu, name):
    c = CASES[name]
    s = make(c)
    flags()
    got = both(gpu, s)
    torch.cuda.synchronize()
    assert flags() == 0
    want = define(c, s)
    for n in got:
        check(n, got[n], want[n])


def test_padding_rows_stay(gpu):
    c = Case((40, 0, 130), (50, 3, 131), lead=4, trail=37, causal=False, dim=128)
    s = make(c)
    for n in ("q", "dout"):     # what stands there does not matter
        s[n][:4], s[n][-37:] = float("nan"), float("inf")
    for n in ("k", "v"):
        s[n][:4], s[n][-37:] = float("inf"), float("nan")
    marks = {n: torch.full_like(s[k], 7.5) for n, k in (("out", "q"), ("dq", "q"), ("dk", "k"), ("dv", "v"))}
    out, lse = gpu.attention_fwd(s["q"], s["k"], s["v"], out=marks["out"], **s["kw"])
    lse[:4] = lse[-37:] = float("nan")
    gpu.attention_bwd(s["dout"], s["q"], s["k"], s["v"], out, lse, dq=marks["dq"], dk=marks["dk"],
                      dv=marks["dv"], **s["kw"])
    want = define(c, s)
    for n, t in marks.items():
        assert (t[:4] == 7.5).all() and (t[-37:] == 7.5).all(), n
        check(n, t, want[n])


def test_neighbours_do_not_matter(gpu):
    """A sequence's results next to sequences of infinities and NaN are those of it alone."""
    c = Case((70, 133, 200), dim=64)
    s = make(c)
    alone = {n: s[n][70:203].clone() for n in ("q", "k", "v", "dout")}
    for n in ("q", "k", "v", "dout"):
        s[n][:70] = float("nan")
        s[n][203:] = float("inf")
    got = both(gpu, s)
    c1 = Case((133,), dim=64)
    cu = torch.tensor([0, 133], dtype=torch.int32, device="cuda")
    one = both(gpu, dict(alone, kw=dict(cu_seqlens=cu, max_q=133)))
    want = define(c1, dict(alone))
    for n in got:
        check(n, got[n][70:203], want[n])
        assert torch.equal(got[n][70:203], one[n]), n


@pytest.mark.parametrize("batches", [1, 20, 200, 700])
def test_lengths_beyond_the_bounds_are_flagged(gpu, batches):
    """Bounds of 0 and of too little, in both passes; lengths of 0 fit a bound of 0."""
    from rmsnorm_fp8_quantization_gb300 import gbnorm as G
    c = Case((3,) * batches, dim=16)
    s = make(c)
    out, lse = gpu.attention_fwd(s["q"], s["k"], s["v"], **s["kw"])
    flags()
    for cu, bound, bad in ((s["kw"]["cu_seqlens"], 0, True), (s["kw"]["cu_seqlens"], 2, True),
                           (s["kw"]["cu_seqlens"], 3, False), (torch.zeros_like(s["kw"]["cu_seqlens"]), 0, False)):
        want = G.GBN_DEVICE_ERR_BAD_INDEX if bad else 0
        o, l = gpu.attention_fwd(s["q"], s["k"], s["v"], cu_seqlens=cu, max_q=bound)
        assert flags() == want, ("forward", bound)
        gpu.attention_bwd(s["dout"], s["q"], s["k"], s["v"], out, lse, cu_seqlens=cu, max_q=bound)
        assert flags() == want, ("backward", bound)


def test_given_outputs_and_strides(gpu):
    """Outputs that are views of one tensor, a gradient whose tokens lie apart."""
    c = Case((150, 20), dim=80, heads=6, kv_heads=3)
    s = make(c)
    room = torch.zeros(170, 12, 88, device="cuda", dtype=c.dtype)
    dq, dk, dv = (t[..., :80] for t in room.split([6, 3, 3], dim=1))
    wide = torch.zeros(170, 3, 6, 80, device="cuda", dtype=c.dtype)
    wide[:, 1] = s["dout"]
    out, lse = gpu.attention_fwd(s["q"], s["k"], s["v"], **s["kw"])
    r = gpu.attention_bwd(wide[:, 1], s["q"], s["k"], s["v"], out, lse, dq=dq, dk=dk, dv=dv,
                          workspace=gpu.attention_bwd_workspace(s["q"], s["k"], **s["kw"]),
                          **s["kw"])
    assert r[0] is dq and r[1] is dk and r[2] is dv
    assert (room[..., 80:] == 0).all()
    want = define(c, s)
    for n, t in (("dq", dq), ("dk", dk), ("dv", dv)):
        check(n, t, want[n])


@pytest.mark.parametrize("c", [Case((3, 140, 1), (211, 1, 300), causal=False, dim=96, scale=0.07),
                               Case((1500,), (1400,), heads=8, kv_heads=1, dim=128, scale=0.2, dtype=F16),
                               Case((130, 130), uniform=True, window=40, scale=0.3)],
                         ids=["cross", "cross, shared steps", "uniform"])
def test_workspace_of_the_callers(gpu, c):
    """Keys of their own and a scale: the workspace takes what the call takes, and its size is the call's."""
    s = make(c)
    out, lse = gpu.attention_fwd(s["q"], s["k"], s["v"], **s["kw"])
    w = gpu.attention_bwd_workspace(s["q"], s["k"], **s["kw"])
    want = gpu.attention_bwd(s["dout"], s["q"], s["k"], s["v"], out, lse, **s["kw"])
    for _ in range(2):
        got = gpu.attention_bwd(s["dout"], s["q"], s["k"], s["v"], out, lse, workspace=w, **s["kw"])
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    with pytest.raises(RuntimeError, match="WORKSPACE|workspace"):
        gpu.attention_bwd(s["dout"], s["q"], s["k"], s["v"], out, lse, workspace=w[:-1], **s["kw"])


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("c", [Case((600,), dim=128, heads=8, kv_heads=4, window=20, lead=2),
                               Case((130, 600), dim=64, dtype=F16, window=20),
                               Case((2600,), dim=64, heads=8, kv_heads=1, window=700),
                               Case((130,) * 60 + (600,), dim=128, heads=16, kv_heads=16, window=20)],
                         ids=lambda c: f"{len(c.q_lens)} sequences of {c.dim}")
def test_bad_values_in_pairs_that_are_not_kept(gpu, c, bad):
    """A token's keys and values, and another's query and gradient, of no use: the rows that have no
    kept pair with them come out as if they were 0, whatever else their tiles hold."""
    s = make(c)
    last = c.lead + sum(c.q_lens)
    first = last - c.q_lens[-1]
    m, i = (last - 5, first + 3) if c.window > 100 else (first + 300, first + 200)
    clean = {n: t.clone() for n, t in s.items() if n != "kw"}
    for n, at in (("k", m), ("v", m), ("q", i), ("dout", i)):
        s[n][at] = bad
        clean[n][at] = 0
    got, want = both(gpu, s), define(c, dict(clean, kw=s["kw"]))
    tokens = torch.arange(s["q"].shape[0], device="cuda")
    w = c.window - 1
    # query m .. m + w keeps key m; those keep keys m - w .. m + w; query i keeps keys i - w .. i
    q_out = ((tokens >= m) & (tokens <= m + w)) | (tokens == i)
    k_out = ((tokens >= m - w) & (tokens <= m + w)) | ((tokens >= i - w) & (tokens <= i))
    for n, t in got.items():
        out = k_out if n in ("dk", "dv") else q_out
        value, off = (x.clone() for x in want[n])
        value[out] = float("nan")
        assert not value.isnan().all()
        check(n, t, (value, off))
    assert got["dq"][i].isnan().any() and got["dk"][m].isnan().any()


@pytest.mark.parametrize("dim", [64, 128])
def test_one_bad_column(gpu, dim):
    """A NaN in one column of a gradient: dv's column of the keys that keep it, dq's row and dk's rows; the
    other columns of dv, and everything of rows that have no part in it, are numbers, and right."""
    c = Case((600,), dim=dim, heads=2, kv_heads=1, window=50)
    s = make(c)
    i = 300
    clean = dict(s, dout=s["dout"].clone())
    s["dout"][i, 1, 5] = float("nan")
    clean["dout"][i, 1] = 0
    out, lse = gpu.attention_fwd(s["q"], s["k"], s["v"], **s["kw"])
    dq, dk, dv = gpu.attention_bwd(s["dout"], s["q"], s["k"], s["v"], out, lse, **s["kw"])
    hit = torch.zeros(600, dtype=torch.bool, device="cuda")
    hit[i - 49:i + 1] = True
    assert dv[hit, 0, 5].isnan().all() and not dv[hit, 0, :5].isnan().any() and not dv[hit, 0, 6:].isnan().any()
    assert dk[hit].isnan().all() and dq[i, 1].isnan().all()
    want = define(c, clean)
    for n, t, out_ in (("dq", dq, (slice(i, i + 1), slice(1, 2))), ("dk", dk, (hit,)), ("dv", dv, (hit,))):
        value, off = (x.clone() for x in want[n])
        value[out_] = float("nan")
        check(n, t, (value, off))


@pytest.mark.parametrize("window", [0, 50])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_an_overflowed_gradient(gpu, dtype, window):
    """An infinity in a gradient, as a loss scale that is too large leaves: no gradient of a row that has a
    part in it is finite (in dv: of its column), and every other one is right."""
    c = Case((600,), heads=2, kv_heads=1, window=window, dtype=dtype)
    s = make(c)
    i = 300
    clean = dict(s, dout=s["dout"].clone())
    s["dout"][i, 1, 5] = float("inf")
    clean["dout"][i, 1] = 0
    out, lse = gpu.attention_fwd(s["q"], s["k"], s["v"], **s["kw"])
    dq, dk, dv = gpu.attention_bwd(s["dout"], s["q"], s["k"], s["v"], out, lse, **s["kw"])
    first = i - window + 1 if window else 0
    hit = torch.zeros(600, dtype=torch.bool, device="cuda")
    hit[first:i + 1] = True
    assert not dk[hit].isfinite().any() and not dq[i, 1].isfinite().any()
    assert not dv[hit, 0, 5].isfinite().any() and dv[hit, 0, :5].isfinite().all() and dv[hit, 0, 6:].isfinite().all()
    want = define(c, clean)
    for n, t, where in (("dq", dq, (slice(i, i + 1), slice(1, 2))), ("dk", dk, (hit,)), ("dv", dv, (hit,))):
        value, off = (x.clone() for x in want[n])
        value[where] = t[where].to(value.dtype) * float("nan")
        t = t.clone()
        t[where] = float("nan")
        check(n, t, (value, off))


def test_heads_outside_tokens(gpu):
    """Tensors that are stored [heads, tokens, dim]."""
    c = Case((150, 20), dim=128, heads=6, kv_heads=3)
    s = make(c)
    t = {n: s[n].transpose(0, 1).contiguous().transpose(0, 1) for n in ("q", "k", "v", "dout")}
    assert t["q"].stride() == (128, 170 * 128, 1)
    a, b = both(gpu, s), both(gpu, dict(t, kw=s["kw"]))
    for n in a:
        assert torch.equal(a[n], b[n]), n


def test_deterministic(gpu):
    c = Case((700, 300, 1), heads=8, kv_heads=2, dim=128)
    s = make(c)
    a = both(gpu, s)
    for _ in range(5):
        b = both(gpu, s)
        for n in a:
            assert torch.equal(a[n], b[n]), n


def test_another_stream(gpu):
    c = Case((300, 40), dim=64, dtype=F16)
    s = make(c)
    a = both(gpu, s)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, lse = gpu.attention_fwd(s["q"], s["k"], s["v"], stream=side, **s["kw"])
    r = gpu.attention_bwd(s["dout"], s["q"], s["k"], s["v"], out, lse, stream=side, **s["kw"])
    side.synchronize()
    for n, t in zip(("out", "lse", "dq", "dk", "dv"), (out, lse, *r)):
        assert torch.equal(t, a[n]), n


def test_against_differences(gpu):
    """The gradients against differences of the forward (in 64 bits, by the definition) along
    random directions: what the formulas say is what the function does."""
    c = Case((90,), dim=32, heads=2, kv_heads=1, dtype=F16, uniform=True)
    s = make(c)
    got = both(gpu, s)
    g = torch.Generator().manual_seed(5)
    d64 = {n: s[n].double() for n in ("q", "k", "v", "dout")}
    for n in ("q", "k", "v"):
        way = torch.randn(s[n].shape, generator=g).cuda().double()
        h = 1e-5
        f = []
        for sign in (1, -1):
            t = dict(d64, **{n: d64[n] + sign * h * way})
            f.append((define(c, dict(t, kw=None))["out"][0] * flat(d64["dout"])).sum())
        slope = ((f[0] - f[1]) / (2 * h)).item()
        want = define(c, s)["d" + n]
        mine = (flat(got["d" + n]).double() * flat(way)).sum().item()
        # 2^-30: the difference's own error (h^2 and 1e-16 / h, times the sums)
        assert abs(mine - slope) <= (want[1] * flat(way).abs()).sum().item() + 2.0 ** -20 * abs(slope)


def test_tensors_beyond_32_bits(gpu):
    """The last of 2400 sequences, past 2^31 elements of every tensor, gives what it gives alone."""
    b, n, h, d = 2400, 128, 64, 128
    if torch.cuda.mem_get_info()[0] < 10 * b * n * h * d * 2:
        pytest.skip("needs 50 GB")
    x = [torch.empty(b, n, h, d, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    for t in x:
        t[:-2].zero_()
        t[-2:].normal_()
    q, k, v, dout = x
    out, lse = gpu.attention_fwd(q, k, v)
    grads = gpu.attention_bwd(dout, q, k, v, out, lse)
    q, k, v, dout = (t[-1:].clone() for t in x)
    o1, l1 = gpu.attention_fwd(q, k, v)
    assert torch.equal(out[-1:], o1) and torch.equal(lse[-1:], l1)
    for a, c in zip(grads, gpu.attention_bwd(dout, q, k, v, o1, l1)):
        assert torch.equal(a[-1:], c)
