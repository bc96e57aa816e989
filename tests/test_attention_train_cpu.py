"""Attention over whole sequences and dropout without a GPU: refusals of the C entry points and
of the Python wrappers, and the autograd functions' plumbing with a stand-in for the library."""
import types

import pytest
import torch


@pytest.fixture(scope="module")
def ops():
    from rmsnorm_fp8_quantization_gb300 import _build
    _build.build()
    from rmsnorm_fp8_quantization_gb300 import ops as o
    return o


FAKE = 0x10000  # never dereferenced: every call below fails validation first
SIZES = dict(tokens=6, keys=6, batches=2, q_heads=4, kv_heads=2, head_dim=64, max_q=3, max_k=3,
             window=0, q_strides=(256, 64), k_strides=(128, 64), v_strides=(128, 64),
             out_strides=(256, 64), causal=True, scale=0.125, stream=0)
FWD = dict(q=FAKE, k=FAKE, v=FAKE, cu_q=FAKE, cu_k=FAKE, out=FAKE, lse=FAKE)
BWD = dict(q=FAKE, k=FAKE, v=FAKE, out=FAKE, dout=FAKE, lse=FAKE, cu_q=FAKE, cu_k=FAKE, dq=FAKE,
           dk=FAKE, dv=FAKE, workspace=FAKE, workspace_bytes=1 << 30)


def _fwd(G, **kw):
    return G.gbn_attention_fwd(**{**dict.fromkeys(FWD), **SIZES, "dtype": G.GBN_BF16, **kw})


def _bwd(G, **kw):
    a = dict(dout_strides=(256, 64), dq_strides=(256, 64), dk_strides=(128, 64), dv_strides=(128, 64))
    return G.gbn_attention_bwd(**{**dict.fromkeys(BWD), **SIZES, **a, "workspace_bytes": 0,
                                  "dtype": G.GBN_BF16, **kw})


def test_attention_refusals(ops):
    G = ops.G
    for call, have in ((_fwd, FWD), (_bwd, BWD)):
        assert call(G, cu_q=FAKE, cu_k=FAKE) == G.GBN_ERR_NULL
        needed = [n for n in have if not n.startswith(("cu_", "workspace"))
                  and not (call is _fwd and n == "lse")]
        for n in needed:
            assert call(G, **{**have, n: None}) == G.GBN_ERR_NULL, n
        for dt in (G.GBN_F32, G.GBN_E4M3, 9):
            assert call(G, **have, dtype=dt) == G.GBN_ERR_DTYPE
        for bad in (dict(head_dim=0), dict(head_dim=12), dict(head_dim=136), dict(head_dim=-8),
                    dict(q_heads=5), dict(q_heads=0), dict(kv_heads=0), dict(kv_heads=-2), dict(max_q=-1),
                    dict(max_k=-1), dict(max_k=(1 << 30) + 1), dict(window=-1), dict(window=1 << 31),
                    dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")),
                    dict(scale=3e38), dict(tokens=1 << 30), dict(tokens=-1), dict(keys=-1),
                    dict(keys=1 << 31), dict(batches=-1), dict(batches=(1 << 20) + 1),
                    dict(q_heads=65536 * 2)):
            assert call(G, **{**have, **bad}) == G.GBN_ERR_SHAPE, bad
        # no offsets: sequences of exactly max_q and max_k
        assert call(G, **{**have, "cu_q": None, "tokens": 7}) == G.GBN_ERR_SHAPE
        assert call(G, **{**have, "cu_k": None, "keys": 5}) == G.GBN_ERR_SHAPE
        for bad in (dict(k_strides=(0, 64)), dict(v_strides=(128, -64)), dict(k_strides=(1 << 39, 64))):
            assert call(G, **{**have, **bad}) == G.GBN_ERR_SHAPE, bad
        names = ["q", "k", "v", "out"] + (["dout", "dq", "dk", "dv"] if call is _bwd else [])
        for n in names:
            assert call(G, **{**have, n: FAKE + 8}) == G.GBN_ERR_ALIGNMENT, n
            for st in ((252, 64), (256, 60)):
                assert call(G, **{**have, n + "_strides": st}) == G.GBN_ERR_ALIGNMENT, (n, st)
        # nothing to do
        assert call(G, tokens=0, keys=0, cu_q=FAKE, cu_k=FAKE) == G.GBN_OK
        assert call(G, batches=0, cu_q=FAKE, cu_k=FAKE) == G.GBN_OK
    for bad in (dict(q_strides=(0, 64)), dict(dout_strides=(256, 0))):
        assert _bwd(G, **{**BWD, **bad}) == G.GBN_ERR_SHAPE
    for bad in (dict(workspace=None), dict(workspace=FAKE + 4), dict(workspace_bytes=100)):
        assert _bwd(G, **{**BWD, **bad}) == G.GBN_ERR_WORKSPACE


def test_workspace_size(ops):
    G = ops.G
    size = lambda *a: G.gbn_attention_bwd_workspace_size(*a)
    ok = (8192, 8192, 2, 32, 8, 128, 4096, 4096, 0, True)
    st, n = size(*ok, G.GBN_BF16)
    assert st == G.GBN_OK and n >= 2 * 32 * 8192 * 4
    assert size(*ok, G.GBN_F16)[1] > n             # the rows' norms
    st, few = size(4096, 4096, 1, 4, 1, 128, 4096, 4096, 0, True, G.GBN_BF16)
    assert few > 2 * 4 * 4096 * 4 + 2 * 2 * 4096 * 128 * 4   # parts of dk and dv
    assert size(0, 0, 0, 1, 1, 8, 0, 0, 0, False, G.GBN_BF16)[0] == G.GBN_OK
    assert size(*ok, G.GBN_F32)[0] == G.GBN_ERR_DTYPE
    for i, v in ((0, -1), (1, 1 << 31), (2, -1), (3, 0), (4, 5), (5, 100), (6, -1), (7, -1), (8, -1)):
        assert size(*ok[:i], v, *ok[i + 1:], G.GBN_BF16)[0] == G.GBN_ERR_SHAPE, i


def test_dropout_refusals(ops):
    G = ops.G
    for call in (lambda **a: G.gbn_dropout_fwd(a["x"], a["r"], a["out"], a["rng"], a["n"], a["p"], a["dt"], 0),
                 lambda **a: G.gbn_dropout_bwd(a["x"], a["out"], a["rng"], a["n"], a["p"], a["dt"], 0)):
        ok = dict(x=FAKE, r=None, out=FAKE, rng=FAKE, n=5, p=0.5, dt=G.GBN_F32)
        for n in ("x", "out", "rng"):
            assert call(**{**ok, n: None}) == G.GBN_ERR_NULL, n
        for dt in (G.GBN_E4M3, G.GBN_E8M0, -1):
            assert call(**{**ok, "dt": dt}) == G.GBN_ERR_DTYPE
        for bad in (dict(n=-1), dict(n=(1 << 40) + 1), dict(p=-1e-9), dict(p=1.0000001), dict(p=float("nan"))):
            assert call(**{**ok, **bad}) == G.GBN_ERR_SHAPE, bad
        for bad in (dict(x=FAKE + 2), dict(out=FAKE + 1), dict(rng=FAKE + 4)):
            assert call(**{**ok, **bad}) == G.GBN_ERR_ALIGNMENT, bad
        assert call(**{**ok, "n": 0, "x": None, "out": None}) == G.GBN_OK
    assert G.gbn_dropout_fwd(FAKE, FAKE + 2, FAKE, FAKE, 5, 0.5, G.GBN_F32, 0) == G.GBN_ERR_ALIGNMENT


def test_attention_wrapper_refusals(ops):
    b = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32)
    q, k = b(2, 3, 4, 16), b(2, 5, 2, 16)
    p, r = b(6, 4, 16), b(6, 2, 16)
    cu = i32(0, 2, 6)
    for match, a, kw in (
            ("dtype", (q.float(), k, k), {}), ("dtype", (q, k.half(), k), {}),
            ("expected \\[batch", (q[0, 0], k, k), {}), ("cu_seqlens", (p, r, r), {}),
            ("cu_seqlens", (q, k, k), dict(cu_seqlens=cu)), ("differ", (q, k, b(2, 4, 2, 16)), {}),
            ("head_dim", (q, b(2, 5, 2, 24), b(2, 5, 2, 24)), {}),
            ("sequences", (q, b(3, 5, 2, 16), b(3, 5, 2, 16)), {}),
            ("go with cu_seqlens", (q, k, k), dict(max_q=3)),
            ("max_q", (p, r, r), dict(cu_seqlens=cu)),
            ("dtype", (p, r, r), dict(cu_seqlens=cu.long(), max_q=4)),
            ("needs max_k", (p, r, r), dict(cu_seqlens=cu, max_q=4, cu_seqlens_k=cu)),
            ("entries", (p, r, r), dict(cu_seqlens=cu, max_q=4, cu_seqlens_k=cu[:2], max_k=4)),
            ("goes with", (p, r, r), dict(cu_seqlens=cu, max_q=4, max_k=4)),
            ("tokens", (p, b(7, 2, 16), b(7, 2, 16)), dict(cu_seqlens=cu, max_q=4)),
            ("at least one", (p, r, r), dict(cu_seqlens=i32(), max_q=4)),
            ("contiguous", (p, r, r), dict(cu_seqlens=i32(0, 0, 2, 2, 6, 6)[::2], max_q=4)),
            ("contiguous", (q.transpose(2, 3).contiguous().transpose(2, 3), k, k), {}),
            ("one run", (b(2, 2, 3, 4, 16)[:, 0], k, k), {}),
            ("dimensions", (q, r, r), {}), ("CUDA", (q, k, k), {}),
            ("CUDA", (p, r, r), dict(cu_seqlens=cu, max_q=4))):
        with pytest.raises(ValueError, match=match):
            ops.attention_fwd(*a, **kw)
        with pytest.raises(ValueError, match=match):
            ops.attention_bwd(a[0], *a, a[0], torch.zeros(1), **kw)


def test_dropout_wrapper_refusals(ops):
    x, rng = torch.zeros(4, 6), torch.tensor([1, 2])
    for match, a, kw in (
            ("dtype", (x.double(), 0.1, rng), {}), ("dtype", (x, 0.1, rng.int()), {}),
            ("rng", (x, 0.1, torch.tensor([1, 2, 3])), {}), ("dimensions", (x, 0.1, rng[None]), {}),
            ("contiguous", (x.T, 0.1, rng), {}), ("shape", (x, 0.1, rng), dict(residual=x[:3])),
            ("dtype", (x, 0.1, rng), dict(residual=x.half())), ("CUDA", (x, 0.1, rng), {}),
            ("shape", (x, 0.1, rng), dict(out=x[:2])),
            ("contiguous", (x, 0.1, rng), dict(residual=torch.zeros(6, 4).T))):
        with pytest.raises(ValueError, match=match):
            ops.dropout_fwd(*a, **kw)


@pytest.fixture
def fake(monkeypatch, ops):
    """autograd over a stand-in that records its calls."""
    from rmsnorm_fp8_quantization_gb300 import autograd as A
    calls = []

    def attention_fwd(q, k, v, *, cu_seqlens, cu_seqlens_k, out, **kw):
        calls.append(("fwd", q, k, v, out, kw))
        out = torch.empty(q.shape) if out is None else out
        return out, torch.zeros(q.shape[:-1])

    def attention_bwd(dout, q, k, v, out, lse, *, cu_seqlens, cu_seqlens_k, dq, dk, dv, **kw):
        calls.append(("bwd", dout, dq, kw))
        return tuple(torch.ones(t.shape) if d is None else d for t, d in ((q, dq), (k, dk), (v, dv)))

    def dropout_fwd(x, p, rng, *, residual):
        calls.append(("fwd", rng))
        return x * 1.0

    def dropout_bwd(dout, p, rng):
        calls.append(("bwd", rng.tolist(), dout.is_contiguous()))
        return dout * 2

    monkeypatch.setattr(A, "ops", types.SimpleNamespace(
        attention_fwd=attention_fwd, attention_bwd=attention_bwd, dropout_fwd=dropout_fwd,
        dropout_bwd=dropout_bwd))
    return A, calls


def test_strides_that_the_kernels_do_not_take_are_copied(fake):
    A, calls = fake
    x = torch.randn(2, 3, 8, 16, requires_grad=True)
    q, k, v = x.split([4, 2, 2], 2)
    A.attention(q, k, v).sum().backward()     # the gradient of a sum is expanded
    _, a, b, c, out, kw = calls[0]
    assert a.data_ptr() == q.data_ptr() and a.stride() == q.stride() and out is None
    assert calls[1][1].stride() == (192, 64, 16, 1)
    assert x.grad.shape == x.shape and (x.grad == 1).all()
    odd = torch.randn(2, 3, 4, 17)[..., :16]
    A.attention(odd, odd[:, :, :2], odd[:, :, :2], causal=False)
    assert calls[2][1].is_contiguous() and torch.equal(calls[2][1], odd) and not calls[2][5]["causal"]
    apart = torch.randn(2, 2, 3, 4, 16)[:, 0]
    A.attention(apart, apart, apart)
    assert calls[3][1].is_contiguous()


def test_padding_gets_zeros(fake):
    A, calls = fake
    q = torch.randn(9, 2, 16, requires_grad=True)
    y = A.attention(q, q, q, cu_seqlens=torch.tensor([0, 4]), max_q=4)
    assert (calls[0][4] == 0).all() and (y == 0).all()
    y.sum().backward()
    assert (q.grad == 0).all()


def test_dropout_keeps_its_own_numbers(fake):
    """rng may be advanced in place before the backward; the residual's gradient is the output's."""
    A, calls = fake
    x, r = torch.randn(4, 6, requires_grad=True), torch.randn(4, 6, requires_grad=True)
    rng = torch.tensor([7, 0])
    y = A.dropout(x, 0.5, rng, r)
    rng[1] += 1
    g = torch.randn(4, 6)
    y.backward(g)
    assert calls[1] == ("bwd", [7, 0], True)
    assert torch.equal(x.grad, 2 * g) and torch.equal(r.grad, g)
    y = A.dropout(x.detach(), 0.5, rng, r)
    y.sum().backward()                         # nothing to draw for the residual alone
    assert len(calls) == 3


def test_workspace_wrapper_refusals(ops):
    b = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32)
    q, k, cu, cu_k = b(6, 4, 16), b(9, 2, 16), i32(0, 2, 6), i32(0, 4, 9)
    for match, a, kw in (
            ("needs max_q", (q, k), dict(cu_seqlens=cu)),
            ("needs max_k", (q, k), dict(cu_seqlens=cu, max_q=4, cu_seqlens_k=cu_k)),
            ("entries", (q, k), dict(cu_seqlens=cu, max_q=4, cu_seqlens_k=i32(0, 9), max_k=9)),
            ("tokens", (q, k), dict(cu_seqlens=cu, max_q=4)),
            ("cu_seqlens", (q, k), {}),
            ("head_dim", (q, b(6, 2, 24)), dict(cu_seqlens=cu, max_q=4)),
            ("dtype", (q.float(), k.float()), dict(cu_seqlens=cu, max_q=4))):
        with pytest.raises(ValueError, match=match):
            ops.attention_bwd_workspace(*a, **kw)
    # what attention_bwd takes is taken, up to the tensors' device
    for kw in (dict(cu_seqlens=cu, max_q=4, cu_seqlens_k=cu_k, max_k=5, scale=0.3, causal=False, window=3),
               dict(cu_seqlens=cu, max_q=4, max_k=5)):
        with pytest.raises(ValueError, match="CUDA tensors"):
            ops.attention_bwd_workspace(q, k, **kw)


def test_numbers_that_require_a_gradient(ops):
    """A learnable scale (or p) would come out without a gradient: refused, as a rotation's frequencies are."""
    from rmsnorm_fp8_quantization_gb300 import autograd as A
    q, k = torch.zeros(2, 3, 4, 16, dtype=torch.bfloat16), torch.zeros(2, 5, 2, 16, dtype=torch.bfloat16)
    x, rng = torch.zeros(8), torch.zeros(2, dtype=torch.int64)
    number = torch.nn.Parameter(torch.tensor(0.5))
    with pytest.raises(ValueError, match="scale requires a gradient"):
        A.attention(q, k, k, scale=number)
    with pytest.raises(ValueError, match="p requires a gradient"):
        A.dropout(x, number, rng)
    for call in (lambda: A.attention(q, k, k, scale=number.detach()), lambda: A.dropout(x, number.detach(), rng)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):
        A.attention(q, k, k, scale=number)
