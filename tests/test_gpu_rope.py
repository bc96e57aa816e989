"""GPU parity of the rotary positions, forward and backward, against the
float64 oracle: both pair layouts, whole and partial rotation, every vector
width (16 bytes, 8 bytes, single elements), strided views, far positions,
shared and per-sequence positions, in place; the frequencies' scalings; the
autograd function.

Tolerance, per element of a pair (a, b) and from the arithmetic alone: the
stored rounding, eps(t) / 2 of the result (fp32: its own 2^-24 is in the
second term; f16: plus half its smallest step, 2^-25), plus m (|a| + |b|)
times 3 * 2^-23: the angle's reduced argument is off by 2^-24 relative, cos
and sin by an ulp (2^-24), the product with m by 2^-24, each product and the
sum by 2^-24."""
import numpy as np
import pytest
import torch

from oracle import paged as P
from paged_cases import DT

pytestmark = pytest.mark.gpu


def check(got, x, ref, mscale, rotary, layout, dtype, name=""):
    g = got.detach().cpu().double().numpy()
    pair = np.abs(x).astype(np.float64)
    r = rotary
    t = np.zeros_like(pair)
    lo = slice(0, r // 2) if layout == "half" else slice(0, r, 2)
    hi = slice(r // 2, r) if layout == "half" else slice(1, r, 2)
    t[..., lo] = t[..., hi] = mscale * (pair[..., lo] + pair[..., hi])
    half = 0.0 if dtype == torch.float32 else torch.finfo(dtype).eps / 2
    tiny = 2.0 ** -25 if dtype == torch.float16 else 0.0
    err = np.abs(g - ref)
    lim = half * (np.abs(ref) + 3 * 2.0 ** -23 * t) + 3 * 2.0 ** -23 * t + tiny
    bad = ~(err <= lim)
    assert not bad.any(), (name, int(bad.sum()), bad.size, err[bad][:4], lim[bad][:4])


CASES = [
    # batch, seq, heads, kv_heads, dim, rotary, layout, dtype, mscale
    (1, 1, 1, 1, 64, 64, "half", "bf16", 1.0),
    (2, 7, 8, 2, 128, 128, "half", "bf16", 1.0),
    (3, 33, 5, 1, 80, 40, "half", "f16", 1.3),          # 8-byte vectors
    (2, 5, 4, 4, 80, 40, "interleaved", "bf16", 1.0),
    (1, 19, 6, 3, 96, 48, "interleaved", "f32", 0.7),
    (2, 9, 3, 3, 96, 96, "half", "f32", 1.0),
    (1, 11, 2, 1, 33, 6, "half", "f32", 1.0),           # odd head: single elements
    (1, 11, 2, 1, 33, 6, "interleaved", "bf16", 1.0),
    (2, 3, 2, 2, 50, 50, "half", "f16", 1.0),           # rotary / 2 odd
    (1, 4, 64, 8, 256, 256, "interleaved", "bf16", 1.0),
    (1, 3, 3, 1, 1024, 1024, "half", "bf16", 1.0),      # the widest head
    (5, 700, 12, 4, 64, 32, "half", "bf16", 1.1),       # whole tokens per CTA
    (4, 1, 128, 8, 128, 128, "half", "f16", 1.0),       # heads split over CTAs
    (1, 2, 700, 1, 64, 64, "half", "bf16", 1.0),
    (2, 6, 4, 2, 64, 0, "half", "bf16", 1.0),           # nothing turns: a copy
]


def run_case(gpu, c, backward, packed):
    b, s, h, hk, d, r, layout, dtype, ms = c
    g = torch.Generator().manual_seed(b * 1000 + s)
    dt = DT[dtype]
    if packed:
        x = torch.randn(b, s, h + hk + 1, d, generator=g).to(dt)
        q, k = x[:, :, :h], x[:, :, h:h + hk]
    else:
        q, k = (torch.randn(b, s, n, d, generator=g).to(dt) for n in (h, hk))
    pos = torch.randint(0, 1 << 20, (b, s), generator=g)
    f = gpu.rope_frequencies(r, 10000.0, device="cpu") if r else torch.zeros(0, dtype=torch.float64)
    if packed:
        xc = x.cuda()
        qc, kc = xc[:, :, :h], xc[:, :, h:h + hk]
    else:
        qc, kc = q.cuda(), k.cuda()
    fn = gpu.rope_bwd if backward else gpu.rope_fwd
    qo, ko = fn(qc, kc, f.cuda(), pos.cuda(), layout=layout, mscale=ms)
    torch.cuda.synchronize()
    for name, t, o in (("q", q, qo), ("k", k, ko)):
        ref = P.rotate(t.double().numpy(), pos.numpy(), f.numpy(), layout, ms, backward)
        check(o, t.double().numpy(), ref, ms, r, layout, dt, name)


@pytest.mark.parametrize("backward", [False, True], ids=["fwd", "bwd"])
@pytest.mark.parametrize("c", CASES, ids=lambda c: "-".join(map(str, c)))
def test_rope(gpu, c, backward):
    run_case(gpu, c, backward, packed=False)


@pytest.mark.parametrize("c", [CASES[1], CASES[2], CASES[4], CASES[6]],
                         ids=lambda c: "-".join(map(str, c)))
def test_rope_of_packed_projection_views(gpu, c):
    run_case(gpu, c, False, packed=True)


def test_positions_far_negative_shared_and_default(gpu):
    """Positions up to 2^40 and below zero lose nothing: the angle is reduced
    exactly.  (The oracle's 64-bit significands cover 2^40 * 2^-64 of a turn.)"""
    g = torch.Generator().manual_seed(5)
    b, s, d = 2, 6, 64
    q = torch.randn(b, s, 3, d, generator=g)
    f = gpu.rope_frequencies(d, 500000.0, device="cpu")
    far = torch.tensor([[0, 1, -1, 2 ** 31 + 7, 2 ** 40 - 3, -2 ** 33], [5, 4, 3, 2, 1, 0]])
    for pos in (far, far[:1], far[0], far[1].int(), None):
        qo, none = gpu.rope_fwd(q.cuda(), None, f.cuda(), None if pos is None else pos.cuda())
        assert none is None
        p = np.arange(s) if pos is None else pos.numpy()
        p = np.broadcast_to(p, (b, s))
        ref = P.rotate(q.double().numpy(), p, f.numpy())
        check(qo, q.double().numpy(), ref, 1.0, d, "half", torch.float32, str(pos))


def test_strides_of_heads_before_positions_and_given_outputs(gpu):
    """[batch, heads, seq, dim] storage, outputs with strides of their own, and
    guard bands around them."""
    g = torch.Generator().manual_seed(6)
    b, s, h, d = 2, 9, 4, 64
    store = torch.randn(b, h, s, d, generator=g).bfloat16().cuda()
    q = store.permute(0, 2, 1, 3)
    f = gpu.rope_frequencies(d)
    out = torch.full((b, s + 2, h, d + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    view = out[:, 1:-1, :, :d]
    gpu.rope_fwd(q, None, f, q_out=view)
    ref, _ = gpu.rope_fwd(q.contiguous(), None, f)
    assert torch.equal(view, ref)
    assert torch.all(out[:, 0] == 7) and torch.all(out[:, -1] == 7)
    assert torch.all(out[..., d:] == 7)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("d,r", [(64, 64), (64, 32), (33, 6)])
def test_in_place(gpu, layout, d, r):
    g = torch.Generator().manual_seed(7)
    q = torch.randn(3, 50, 6, d, generator=g).half().cuda()
    k = torch.randn(3, 50, 2, d, generator=g).half().cuda()
    f = gpu.rope_frequencies(r)
    a, b = gpu.rope_fwd(q, k, f, layout=layout)
    gpu.rope_fwd(q, k, f, layout=layout, q_out=q, k_out=k)
    assert torch.equal(a, q) and torch.equal(b, k)


def test_backward_is_the_transpose(gpu):
    """<rope(x), y> = <x, rope_bwd(y)>, and a finite difference of a linear map
    is the map: fp32, relative to the norms, with the per-element bound summed."""
    g = torch.Generator().manual_seed(8)
    x = torch.randn(2, 31, 4, 96, generator=g).cuda()
    y = torch.randn(2, 31, 4, 96, generator=g).cuda()
    f = gpu.rope_frequencies(48)
    for layout in ("half", "interleaved"):
        fx, _ = gpu.rope_fwd(x, None, f, layout=layout, mscale=1.2)
        by, _ = gpu.rope_bwd(y, None, f, layout=layout, mscale=1.2)
        a, b = (fx.double() * y.double()).sum(), (x.double() * by.double()).sum()
        # every element of fx and by is off by at most 3 * 2^-23 * 1.2 (|a| + |b|)
        lim = 2 * 2 * 1.2 * 3 * 2.0 ** -23 * (x.double().norm() * y.double().norm())
        assert abs(float(a - b)) <= float(lim)
        e = torch.zeros_like(x)
        e[1, 17, 2, 5] = 1.0
        d, _ = gpu.rope_fwd(x + e, None, f, layout=layout, mscale=1.2)
        m, _ = gpu.rope_fwd(e, None, f, layout=layout, mscale=1.2)
        assert torch.allclose(d - fx, m, atol=6 * 2.0 ** -22 * 8, rtol=0)


def test_autograd(gpu):
    from rmsnorm_fp8_quantization_gb300 import autograd as A
    g = torch.Generator().manual_seed(9)
    q = torch.randn(2, 12, 4, 64, generator=g).bfloat16().cuda().requires_grad_()
    k = torch.randn(2, 12, 2, 64, generator=g).bfloat16().cuda().requires_grad_()
    f = gpu.rope_frequencies(64)
    pos = torch.arange(12, device="cuda") + 100
    wq, wk = torch.randn_like(q), torch.randn_like(k)
    qo, ko = A.rope(q, k, f, pos, "interleaved", 1.1)
    ((qo * wq).sum() + (ko * wk).sum()).backward()
    rq, rk = gpu.rope_bwd(wq, wk, f, pos, layout="interleaved", mscale=1.1)
    assert torch.equal(q.grad, rq) and torch.equal(k.grad, rk)
    # only one output used; expanded gradient
    q.grad = k.grad = None
    A.rope(q, k, f, pos)[0].sum().backward()
    rq, _ = gpu.rope_bwd(torch.ones_like(q), None, f, pos)
    assert torch.equal(q.grad, rq) and k.grad is None
    q.grad = None
    out, none = A.rope(q, None, f)
    assert none is None
    out.backward(wq.transpose(1, 2).contiguous().transpose(1, 2))
    assert torch.equal(q.grad, gpu.rope_bwd(wq, None, f)[0])


def test_graph_capture_and_other_stream(gpu):
    g = torch.Generator().manual_seed(10)
    q = torch.randn(2, 40, 4, 64, generator=g).bfloat16().cuda()
    f = gpu.rope_frequencies(64)
    ref, _ = gpu.rope_fwd(q, None, f)
    out = torch.zeros_like(q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    gpu.rope_fwd(q, None, f, q_out=out, stream=s)
    s.synchronize()
    assert torch.equal(out, ref)
    out.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gpu.rope_fwd(q, None, f, q_out=out)
    q.mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, gpu.rope_fwd(q, None, f)[0])


def test_empty(gpu):
    f = gpu.rope_frequencies(64)
    for shape in ((0, 5, 4, 64), (2, 0, 4, 64)):
        q, k = gpu.rope_fwd(torch.empty(shape, device="cuda"), None, f)
        assert q.shape == shape and k is None
