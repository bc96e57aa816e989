"""Rotary positions and the paged cache without a GPU: refusals of the C entry
points and of the Python wrappers, what the wrappers hand to the library, the
frequencies' scalings, and the autograd function's plumbing."""
import math

import numpy as np
import pytest
import torch

from oracle import paged as P


@pytest.fixture(scope="module")
def ops():
    from rmsnorm_fp8_quantization_gb300 import _build
    _build.build()
    from rmsnorm_fp8_quantization_gb300 import ops as o
    return o


FAKE = 0x10000  # never dereferenced: every call below fails validation first


def test_rope_refusals(ops):
    G = ops.G
    for fn, q, k, qo, ko in (("gbn_rope_fwd", "q", "k", "q_out", "k_out"),
                             ("gbn_rope_bwd", "dq", "dk", "dq_out", "dk_out")):
        def call(**kw):
            ren = {"q": q, "k": k, "q_out": qo, "k_out": ko}
            base = {ren[n]: None for n in ren}
            base.update({ren.get(n, n): v for n, v in kw.items()})
            a = dict(positions=None, inv_freq=None, batches=2, seq=3, q_heads=4, k_heads=2,
                     head_dim=64, rotary_dim=64, q_strides=(768, 256, 64), k_strides=(384, 128, 64),
                     q_out_strides=(768, 256, 64), k_out_strides=(384, 128, 64), position_stride=0,
                     position_bytes=8, dtype=G.GBN_BF16, layout=G.GBN_ROPE_HALF, mscale=1.0,
                     stream=0)
            a.update(base)
            return getattr(G, fn)(**a)
        assert call() == G.GBN_ERR_NULL
        assert call(q=FAKE, q_out=FAKE, k=FAKE, k_out=FAKE) == G.GBN_ERR_NULL  # inv_freq
        assert call(q=FAKE, q_out=FAKE, inv_freq=FAKE) == G.GBN_ERR_NULL       # k
        assert call(dtype=G.GBN_E4M3) == G.GBN_ERR_DTYPE
        assert call(position_bytes=2) == G.GBN_ERR_DTYPE
        assert call(layout=2) == G.GBN_ERR_ENUM
        for bad in (dict(head_dim=0), dict(head_dim=1025), dict(rotary_dim=63), dict(rotary_dim=66),
                    dict(rotary_dim=-2), dict(batches=-1), dict(seq=-1), dict(q_heads=-1),
                    dict(k_heads=5000), dict(batches=1 << 40, seq=1 << 40)):
            assert call(**bad) == G.GBN_ERR_SHAPE, bad
        assert call(seq=0) == G.GBN_OK and call(batches=0) == G.GBN_OK
        assert call(q_heads=0, k_heads=0) == G.GBN_OK


def _append(G, **kw):
    a = dict(q=None, k=None, v=None, q_out=None, k_cache=None, v_cache=None, inv_freq=None,
             k_scale=None, v_scale=None, cu_seqlens=None, kv_lens=None, block_table=None, tokens=5,
             batches=2, q_heads=4, kv_heads=2, head_dim=64, rotary_dim=64, num_pages=8,
             page_size=16, table_pages=4, table_stride=4, q_strides=(256, 64),
             k_strides=(128, 64), v_strides=(128, 64), q_out_strides=(256, 64),
             k_cache_strides=(2048, 128, 64), v_cache_strides=(2048, 128, 64), dtype=G.GBN_BF16,
             cache_dtype=G.GBN_BF16, layout=G.GBN_ROPE_HALF, mscale=1.0, stream=0)
    a.update(kw)
    return G.gbn_paged_append(**a)


def test_append_refusals(ops):
    G = ops.G
    have = dict(k=FAKE, v=FAKE, k_cache=FAKE, v_cache=FAKE, cu_seqlens=FAKE, kv_lens=FAKE,
                block_table=FAKE, inv_freq=FAKE, q=FAKE, q_out=FAKE)
    assert _append(G) == G.GBN_ERR_NULL
    for n in have:
        assert _append(G, **{**have, n: None}) == G.GBN_ERR_NULL, n
    assert _append(G, **have, cache_dtype=G.GBN_E4M3) == G.GBN_ERR_NULL  # scales
    assert _append(G, dtype=G.GBN_F32, cache_dtype=G.GBN_F32) == G.GBN_ERR_DTYPE
    assert _append(G, cache_dtype=G.GBN_F16) == G.GBN_ERR_DTYPE
    assert _append(G, layout=-1) == G.GBN_ERR_ENUM
    for bad in (dict(page_size=0), dict(page_size=24), dict(page_size=1 << 17), dict(kv_heads=0),
                dict(q_heads=-1), dict(head_dim=0), dict(rotary_dim=65), dict(rotary_dim=128),
                dict(tokens=-1), dict(batches=-1), dict(batches=(1 << 20) + 1), dict(num_pages=-1),
                dict(num_pages=1 << 31), dict(table_pages=-1), dict(table_stride=-1),
                dict(tokens=1 << 31)):
        assert _append(G, **bad) == G.GBN_ERR_SHAPE, bad
    assert _append(G, tokens=0) == G.GBN_OK and _append(G, batches=0) == G.GBN_OK


def _attend(G, **kw):
    a = dict(q=None, k_cache=None, v_cache=None, cu_seqlens=None, kv_lens=None, block_table=None,
             k_scale_inv=None, v_scale_inv=None, out=None, lse=None, workspace=None,
             workspace_bytes=0, tokens=5, batches=2, q_heads=4, kv_heads=2, head_dim=64,
             num_pages=8, page_size=16, table_pages=4, table_stride=4, max_q=3, max_kv=64,
             q_strides=(256, 64), out_strides=(256, 64), k_cache_strides=(2048, 128, 64),
             v_cache_strides=(2048, 128, 64), dtype=G.GBN_BF16, cache_dtype=G.GBN_BF16,
             causal=True, window=0, scale=0.125, stream=0)
    a.update(kw)
    return G.gbn_paged_attention(**a)


HAVE = dict(q=FAKE, k_cache=FAKE, v_cache=FAKE, cu_seqlens=FAKE, kv_lens=FAKE, block_table=FAKE,
            out=FAKE)


def test_attention_refusals(ops):
    G = ops.G
    assert _attend(G) == G.GBN_ERR_NULL
    for n in HAVE:
        assert _attend(G, **{**HAVE, n: None}) == G.GBN_ERR_NULL, n
    assert _attend(G, **HAVE, cache_dtype=G.GBN_E4M3) == G.GBN_ERR_NULL
    assert _attend(G, dtype=G.GBN_F32, cache_dtype=G.GBN_F32) == G.GBN_ERR_DTYPE
    assert _attend(G, cache_dtype=G.GBN_F16) == G.GBN_ERR_DTYPE
    for bad in (dict(page_size=48), dict(head_dim=72), dict(head_dim=272), dict(head_dim=8),
                dict(q_heads=5), dict(q_heads=1), dict(kv_heads=0), dict(max_q=-1),
                dict(max_kv=-1), dict(max_kv=(1 << 30) + 1), dict(window=-1), dict(window=1 << 31),
                dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
                dict(scale=float("inf")), dict(tokens=1 << 30), dict(num_pages=-1)):
        assert _attend(G, **bad) == G.GBN_ERR_SHAPE, bad
    for bad in (dict(k_cache_strides=(0, 128, 64)), dict(v_cache_strides=(2048, 128, -64)),
                dict(k_cache_strides=(1 << 40, 128, 64))):   # not what a tensor map takes
        assert _attend(G, **{**HAVE, **bad}) == G.GBN_ERR_SHAPE, bad
    for bad in (dict(q=FAKE + 8), dict(out=FAKE + 2), dict(k_cache=FAKE + 4),
                dict(q_strides=(252, 64)), dict(out_strides=(256, 68)),
                dict(k_cache_strides=(2048, 132, 64)), dict(v_cache_strides=(2050, 128, 64))):
        assert _attend(G, **{**HAVE, **bad}) == G.GBN_ERR_ALIGNMENT, bad
    assert _attend(G, tokens=0) == G.GBN_OK and _attend(G, batches=0) == G.GBN_OK
    assert _attend(G, max_q=0) == G.GBN_OK


def test_attention_workspace_query_refusals(ops):
    G = ops.G
    q = lambda *a: G.gbn_paged_attention_workspace_size(*a)[0]  # noqa: E731
    base = [5, 2, 4, 2, 64, 16, 4, 3, 64, 0, True, G.GBN_BF16, G.GBN_BF16]
    for at, bad in ((4, 72), (5, 3), (7, -1), (9, -1), (2, 5)):
        a = list(base)
        a[at] = bad
        assert q(*a) == G.GBN_ERR_SHAPE
    a = list(base)
    a[-1] = G.GBN_F32
    assert q(*a) == G.GBN_ERR_DTYPE
    a = list(base)
    a[0] = 0
    assert G.gbn_paged_attention_workspace_size(*a) == (G.GBN_OK, 0)


def _paged(**kw):
    a = dict(q=torch.zeros(5, 4, 64).bfloat16(), k=torch.zeros(5, 2, 64).bfloat16(),
             v=torch.zeros(5, 2, 64).bfloat16(), k_cache=torch.zeros(8, 16, 2, 64).bfloat16(),
             v_cache=torch.zeros(8, 16, 2, 64).bfloat16(),
             cu=torch.zeros(3, dtype=torch.int32), kv=torch.zeros(2, dtype=torch.int32),
             table=torch.zeros(2, 4, dtype=torch.int32))
    a.update(kw)
    return a


@pytest.mark.parametrize("bad", [
    dict(k_cache=torch.zeros(8, 16, 2, 64).half()),
    dict(v_cache=torch.zeros(8, 16, 2, 64).half()),
    dict(k_cache=torch.zeros(8, 16, 2, 80).bfloat16()),
    dict(v_cache=torch.zeros(7, 16, 2, 64).bfloat16()),
    dict(k_cache=torch.zeros(8, 16, 64).bfloat16(), v_cache=torch.zeros(8, 16, 64).bfloat16()),
    dict(k_cache=torch.zeros(8, 16, 64, 2).bfloat16().transpose(2, 3)),
    dict(cu=torch.zeros(3, dtype=torch.int64)), dict(cu=torch.zeros(4, dtype=torch.int32)),
    dict(kv=torch.zeros(3, dtype=torch.int32)), dict(table=torch.zeros(3, 4, dtype=torch.int32)),
    dict(table=torch.zeros(4, 2, dtype=torch.int32).T),
    dict(cu=torch.zeros(6, dtype=torch.int32)[::2]),
    dict(table=torch.zeros(2, dtype=torch.int32)),
    dict(k_cache=torch.zeros(8, 16, 2, 64, dtype=torch.uint8),
         v_cache=torch.zeros(8, 16, 2, 64, dtype=torch.uint8)),          # no scales
])
def test_wrappers_refuse_before_any_call(ops, bad):
    a = _paged(**bad)
    with pytest.raises(ValueError):
        ops.paged_attention(a["q"], a["k_cache"], a["v_cache"], a["cu"], a["kv"], a["table"],
                            max_q=1)
    with pytest.raises(ValueError):
        ops.paged_append(a["k"], a["v"], a["k_cache"], a["v_cache"], a["cu"], a["kv"], a["table"])


def test_wrappers_refuse_their_own_arguments(ops):
    a = _paged()
    args = (a["k_cache"], a["v_cache"], a["cu"], a["kv"], a["table"])
    for kw in (dict(out=a["q"][:4]), dict(lse=torch.zeros(5, 3)), dict(lse=torch.zeros(4, 5).T),
               dict(out=a["q"].half())):
        with pytest.raises(ValueError):
            ops.paged_attention(a["q"], *args, max_q=1, **kw)
    with pytest.raises(ValueError):   # fp32
        ops.paged_attention(a["q"].float(), *args, max_q=1)
    for kw in (dict(v=a["v"][:4]), dict(q=a["q"][:4]), dict(q_out=a["q"]),
               dict(inv_freq=torch.zeros(32)), dict(k=a["q"], v=a["q"]),
               dict(q=a["q"], q_out=a["q"].half()),
               dict(inv_freq=torch.zeros(64, dtype=torch.float64)[::2])):
        k, v = kw.pop("k", a["k"]), kw.pop("v", a["v"])
        with pytest.raises(ValueError):
            ops.paged_append(k, v, *args, **kw)
    with pytest.raises(ValueError):   # not on a GPU
        ops.paged_append(a["k"], a["v"], *args)
    with pytest.raises(ValueError):
        ops.paged_attention(a["q"], *args, max_q=1)


def test_rope_wrapper_refusals(ops):
    q, k = torch.zeros(2, 3, 4, 64), torch.zeros(2, 3, 2, 64)
    f = torch.zeros(32, dtype=torch.float64)
    for args, kw in (((None, None, f), {}), ((q[0], None, f), {}), ((q, k.half(), f), {}),
                     ((q, k[:1], f), {}), ((q, k, f.float()), {}),
                     ((q, k, f, torch.zeros(3)), {}),
                     ((q, k, f, torch.zeros(4, dtype=torch.int64)), {}),
                     ((q, k, f, torch.zeros(3, 2, dtype=torch.int64).T), {}),
                     ((q, k, f), dict(q_out=q[:1])), ((q, k, f), dict(k_out=k.half())),
                     ((torch.zeros(2, 3, 64, 4).transpose(2, 3), None, f), {}),
                     ((q.double(), None, f), {}), ((q, k, f), {})):  # the last: not on a GPU
        with pytest.raises(ValueError):
            ops.rope_fwd(*args, **kw)


def test_frequencies(ops):
    f = ops.rope_frequencies(8, 10000.0, device="cpu")
    assert f.dtype == torch.float64
    assert torch.allclose(f, torch.tensor([1.0, 0.1, 0.01, 0.001], dtype=torch.float64), rtol=1e-14)
    assert torch.equal(ops.rope_frequencies(8, scaling="linear", factor=4.0, device="cpu"), f / 4)
    n = ops.rope_frequencies(8, scaling="ntk", factor=4.0, device="cpu")
    assert n[0] == 1.0 and abs(float(n[3] / f[3]) - 0.25) < 1e-12
    y = ops.rope_frequencies(64, scaling="yarn", factor=4.0, original_length=4096, device="cpu")
    p = ops.rope_frequencies(64, device="cpu")
    turns = 4096 * p / (2 * math.pi)
    assert torch.equal(y[turns > 40], p[turns > 40])
    assert torch.allclose(y[turns < 0.5], p[turns < 0.5] / 4, rtol=1e-14)
    assert ((y <= p) & (y >= p / 4)).all() and (y[1:] < y[:-1]).all()
    assert ops.rope_mscale(1.0) == 1.0 and abs(ops.rope_mscale(math.e) - 1.1) < 1e-15
    for bad in (dict(rotary_dim=7), dict(rotary_dim=0), dict(rotary_dim=8, base=0.0),
                dict(rotary_dim=8, factor=0.5), dict(rotary_dim=8, scaling="other"),
                dict(rotary_dim=8, scaling="yarn", factor=2.0)):
        with pytest.raises(ValueError):
            ops.rope_frequencies(device="cpu", **bad)


def test_autograd_plumbing(ops, monkeypatch):
    """The backward is one transposed rotation of both gradients (oracle-backed stand-ins),
    against float64 autograd of the same formula."""
    from rmsnorm_fp8_quantization_gb300 import autograd as A
    calls = []

    class Fake:
        @staticmethod
        def _go(q, k, f, pos, layout, mscale, backward):
            calls.append((backward, q is None, k is None))
            return tuple(None if t is None else torch.from_numpy(
                P.rotate(t.detach().numpy(), pos.numpy(), f.numpy(), layout, mscale, backward))
                for t in (q, k))

        def rope_fwd(self, q, k, f, pos, *, layout, mscale):
            return self._go(q, k, f, pos, layout, mscale, False)

        def rope_bwd(self, q, k, f, pos, *, layout, mscale):
            return self._go(q, k, f, pos, layout, mscale, True)

    monkeypatch.setattr(A, "ops", Fake())
    g = torch.Generator().manual_seed(0)
    q = torch.randn(2, 3, 4, 8, generator=g, dtype=torch.float64).requires_grad_()
    k = torch.randn(2, 3, 2, 8, generator=g, dtype=torch.float64).requires_grad_()
    f = ops.rope_frequencies(6, device="cpu")
    pos = torch.tensor([[1, 2, 3], [9, 10, 11]])
    wq, wk = torch.randn_like(q), torch.randn_like(k)

    def plain(x):
        a = pos[..., None, None] * f
        c, s = 1.2 * a.cos(), 1.2 * a.sin()
        lo, hi = x[..., :3], x[..., 3:6]
        return torch.cat([lo * c - hi * s, lo * s + hi * c, x[..., 6:]], -1)

    (plain(q) * wq).sum().backward()
    (plain(k) * wk).sum().backward()
    want = q.grad.clone(), k.grad.clone()
    q.grad = k.grad = None
    qo, ko = A.rope(q, k, f, pos, "half", 1.2)
    ((qo * wq).sum() + (ko * wk).sum()).backward()
    assert torch.allclose(q.grad, want[0]) and torch.allclose(k.grad, want[1])
    assert calls == [(False, False, False), (True, False, False)]
    q.grad = None
    A.rope(q, k, f, pos)[0].sum().backward()
    assert calls[-1] == (True, False, True)
    out, none = A.rope(q, None, f, pos)
    assert none is None
    with pytest.raises(RuntimeError):   # no second derivative
        h, = torch.autograd.grad((out * out).sum(), q, create_graph=True)
        h.sum().backward()
    assert np.isfinite(want[0].numpy()).all()
