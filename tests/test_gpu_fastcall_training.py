"""The host-side shortcut of the attention over whole sequences and the dropout: bit for bit
what the wrappers' own way gives, and every unusual call left to it."""
import pytest
import torch

from attention_train_cases import Case, make
from test_gpu_fastcall import both, same  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("c", [Case((40, 40), uniform=True, packed=True), Case((40, 3, 0), dim=80),
                               Case((1,), uniform=True), Case((70, 20), (30, 140), causal=False, scale=0.2),
                               Case((5, 5), (9, 9), uniform=True, window=3, dtype=torch.float16)], ids=str)
def test_attention(gpu, both, c):  # noqa: F811
    s = make(c)
    same(*both(lambda: gpu.attention_fwd(s["q"], s["k"], s["v"], **s["kw"])))
    o, lse = gpu.attention_fwd(s["q"], s["k"], s["v"], **s["kw"])
    same(*both(lambda: gpu.attention_bwd(s["dout"], s["q"], s["k"], s["v"], o, lse, **s["kw"])))


def test_a_batch_of_single_tokens(gpu, both):  # noqa: F811
    """[batch, 1, heads, dim] views, whose token stride is the batch's."""
    x = torch.randn(9, 6, 8, 64, device="cuda").bfloat16()
    q, k, v = x[:, 2:3, :4], x[:, 2:3, 4:6], x[:, 2:3, 6:]
    same(*both(lambda: gpu.attention_fwd(q, k, v)))
    assert torch.equal(gpu.attention_fwd(q, k, v)[0], v.repeat_interleave(2, 2))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_dropout(gpu, both, dtype):  # noqa: F811
    x, r = (torch.randn(33, 47, device="cuda").to(dtype) for _ in range(2))
    rng = torch.tensor([3, 4], device="cuda")
    same(*both(lambda: gpu.dropout_fwd(x, 0.3, rng)))
    same(*both(lambda: gpu.dropout_fwd(x, 0.3, rng, residual=r)))
    same(*both(lambda: gpu.dropout_bwd(x, 0.3, rng)))


def test_unusual_calls_are_left_alone(gpu):
    fast = gpu._fast
    c = Case((20, 30))
    s = make(c)
    q, k, v, cu = s["q"], s["k"], s["v"], s["kw"]["cu_seqlens"]
    rest = (cu, None, 30, None, None, True, 0)
    assert fast.attention_fwd(q, k, v, *rest) is not None
    for a in ((q.float(), k, v, *rest), (q, k.half(), v, *rest), (q, k, v[:, :, :32], *rest),
              (q, k, v[:40], *rest), (q.cpu(), k, v, *rest), (q[None], k[None], v[None], *rest),
              (q, k, v, cu.long(), *rest[1:]), (q, k, v, cu[::2], *rest[1:]), (q, k, v, None, *rest[1:]),
              (q, k, v, cu, None, None, *rest[3:]), (q, k, v, cu, cu, 30, None, *rest[4:]),
              (q, k, v, cu, None, 30, 30, *rest[4:]), (q, k[:40], v[:40], *rest),
              (q, k, v, *rest[:4], torch.tensor(0.1), True, 0), (q, k, v, *rest[:5], 1, 0),
              (q, k, v, *rest[:6], 0.0), (q.transpose(1, 2), k.transpose(1, 2), v.transpose(1, 2), *rest)):
        assert fast.attention_fwd(*a) is None
    o, lse = gpu.attention_fwd(q, k, v, **s["kw"])
    d = s["dout"]
    assert fast.attention_bwd(d, o, lse, q, k, v, *rest) is not None
    for a in ((d.half(), o, lse), (d, o[:, :2], lse), (d, o, lse.double()), (d, o, lse.T.contiguous().T),
              (d.cpu(), o, lse), (d.transpose(0, 1).contiguous().transpose(0, 1)[:, :, ::2], o, lse)):
        assert fast.attention_bwd(*a, q, k, v, *rest) is None
    b = torch.randn(2, 2, 5, 4, 64, device="cuda").bfloat16()[:, 0]   # sequences apart: no run of rows
    none = (None,) * 5 + (True, 0)
    assert fast.attention_fwd(b, b, b, *none) is None
    with pytest.raises(ValueError, match="one run of tokens"):
        gpu.attention_fwd(b, b, b)
    x, rng = torch.randn(6, 8, device="cuda"), torch.tensor([1, 2], device="cuda")
    assert fast.dropout(0, x, 0.5, rng, None) is not None
    for a in ((x.double(), 0.5, rng, None), (x, 1, rng, None), (x.T, 0.5, rng, None), (x, 0.5, rng.int(), None),
              (x, 0.5, rng[:1], None), (x, 0.5, rng.cpu(), None), (x, 0.5, rng, x.half()),
              (x, 0.5, rng, x[:3])):
        assert fast.dropout(0, *a) is None
    from rmsnorm_fp8_quantization_gb300.gbnorm import GbnError
    for f in (lambda: gpu.dropout_fwd(x, 1.5, rng), lambda: gpu.dropout_fwd(x, float("nan"), rng),
              lambda: gpu.attention_fwd(q, k, v, cu_seqlens=cu, max_q=30, window=-1),
              lambda: gpu.attention_fwd(q, k, v, cu_seqlens=cu, max_q=30, scale=0.0)):
        with pytest.raises(GbnError):
            f()
