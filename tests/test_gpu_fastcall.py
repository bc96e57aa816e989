"""The wrappers' host-side shortcut (csrc/fastcall.cpp): it is there on a GPU machine,
gives what the wrappers' own way gives bit for bit, and leaves every unusual call
to it."""
import pytest
import torch

from paged_cases import Batch, make

pytestmark = pytest.mark.gpu


@pytest.fixture
def both(gpu, monkeypatch):
    """call(f): its result through the shortcut, and without it."""
    assert gpu._fast is not None, "fastcall.cpp was not built"

    def run(f):
        a = f()
        with monkeypatch.context() as m:
            m.setattr(gpu, "_fast", None)
            b = f()
        return a, b
    return run


def same(a, b):
    a, b = (x if isinstance(x, tuple) else (x,) for x in (a, b))
    for x, y in zip(a, b):
        assert x.shape == y.shape and x.stride() == y.stride() and x.dtype == y.dtype
        assert torch.equal(x, y)


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_rope(gpu, both, packed, dtype):
    x = torch.randn(3, 7, 9, 64, device="cuda").to(dtype)
    q, k = (x[:, :, :6], x[:, :, 6:8]) if packed else (x[:, :, :6].contiguous(),
                                                       x[:, :, 6:8].contiguous())
    f, pos = gpu.rope_frequencies(32), torch.arange(21, device="cuda").view(3, 7)
    for fn in (gpu.rope_fwd, gpu.rope_bwd):
        same(*both(lambda: fn(q, k, f, pos, layout="interleaved", mscale=1.5)))


@pytest.mark.parametrize("c", [Batch((1, 1), (300, 20)), Batch((5, 90), (700, 90), dim=128),
                               Batch((1, 3), (300, 20), fp8=True)], ids=str)
def test_paged(gpu, both, c):
    s = make(c)
    f = gpu.rope_frequencies(c.dim)
    same(*both(lambda: gpu.paged_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["cu"],
                                        s["kv_lens"], s["table"], q=s["q"], inv_freq=f,
                                        k_scale=s["scale"], v_scale=s["scale"])))
    for lse in (False, True):
        same(*both(lambda: gpu.paged_attention(
            s["q"], s["k_cache"], s["v_cache"], s["cu"], s["kv_lens"], s["table"],
            max_q=s["max_q"], k_scale_inv=s["scale_inv"], v_scale_inv=s["scale_inv"],
            return_lse=lse)))


def test_unusual_calls_are_left_alone(gpu, both):
    fast = gpu._fast
    s = make(Batch((1, 1), (30, 20)))
    f, pos = gpu.rope_frequencies(64), torch.arange(5, device="cuda")
    q, k = torch.randn(2, 5, 4, 64, device="cuda"), torch.randn(2, 5, 2, 64, device="cuda")
    pos2 = pos.expand(2, 5)
    for a in ((q, None, f, pos2.contiguous()), (q, k, f, None), (q, k, f, pos), (q, k, f, pos2),
              (q, k.half(), f, pos2.contiguous()), (q.cpu(), k, f, pos2.contiguous()),
              (q, k, f.float(), pos2.contiguous()), (q.double(), k.double(), f, pos2.contiguous()),
              (q, k[:, :4], f, pos2.contiguous())):
        assert fast.rope(0, *a, 0, 1.0) is None
    # torch counts a Parameter as a plain tensor: the same results both ways
    same(*both(lambda: gpu.rope_fwd(torch.nn.Parameter(q), k, f, pos2.contiguous())))
    assert fast.rope(0, q, k, f, pos2.contiguous(), 0, torch.tensor(1.0)) is None
    args = (s["k_cache"], s["v_cache"], s["cu"], s["kv_lens"], s["table"])
    ok = (1, None, None, True, 0, None, None, False)
    assert fast.attention(s["q"], *args, *ok) is not None
    for a in ((s["q"].float(), *args), (s["q"], s["k_cache"].half(), *args[1:]),
              (s["q"], *args[:2], s["cu"].long(), *args[3:]), (s["q"], *args[:4], s["table"].T),
              (s["q"][..., :32], *args)):
        assert fast.attention(*a, *ok) is None
    assert fast.attention(s["q"], *args, 1.0, *ok[1:]) is None
    # a refusal of the library comes out as its error
    from rmsnorm_fp8_quantization_gb300.gbnorm import GbnError
    with pytest.raises(GbnError):
        gpu.paged_attention(s["q"], *args, max_q=1, scale=-1.0)
    with pytest.raises(GbnError):
        gpu.paged_attention(s["q"], *args, max_q=1, window=-3)
