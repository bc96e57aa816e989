"""The attention side in captured graphs: an append whose lengths and pages change
between replays, a step of append and attention, and the rotation's forward and
backward with autograd."""
import dataclasses

import pytest
import torch

from paged_cases import Batch, make
from test_gpu_paged import attend, check_append, check_attention, device_flags

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp8", [False, True], ids=["two-byte", "e4m3"])
@pytest.mark.parametrize("n", [3, 40])
def test_append_follows_lengths_and_tables_on_the_device(gpu, n, fp8):
    c = Batch((1,) * n, (50,) * n, heads=4, kv_heads=2, dim=64, fp8=fp8)
    s = make(c)
    f = gpu.rope_frequencies(c.dim)
    q_out = torch.empty_like(s["q"])

    def call():
        gpu.paged_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["cu"], s["kv_lens"],
                         s["table"], q=s["q"], inv_freq=f, k_scale=s["scale"], v_scale=s["scale"],
                         q_out=q_out)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    device_flags()
    for seed, lens in ((1, [50] * n), (2, [1 + i % 50 for i in range(n)]), (3, [17] * n)):
        c2 = dataclasses.replace(c, kv_lens=tuple(lens), seed=seed)
        other = make(c2)
        wide = torch.full_like(s["table"], -1)
        wide[:, :other["table"].shape[1]] = other["table"]
        s["table"].copy_(wide)
        for name in ("q", "k", "v", "kv_lens"):
            s[name].copy_(other[name])
        before = s["k_cache"].cpu().clone(), s["v_cache"].cpu().clone()
        graph.replay()
        torch.cuda.synchronize()
        assert device_flags() == 0
        t = {**s, "cpu": {**other["cpu"], "table": wide.cpu().numpy()}}
        check_append(c2, t, before, q_out, f.cpu().numpy(), "half", 1.0)


def test_a_step_of_append_and_attention(gpu):
    """Both in one graph, replayed along the sequences: each replay one key longer."""
    c = Batch((1, 1, 1), (290, 40, 1), heads=8, kv_heads=2, dim=128)
    s = make(dataclasses.replace(c, kv_lens=(300, 50, 11)))   # pages for what is to come
    s["kv_lens"].copy_(torch.tensor(c.kv_lens, dtype=torch.int32))
    f = gpu.rope_frequencies(c.dim)
    room = gpu.paged_attention_workspace(s["q"], s["k_cache"], s["table"], max_q=1)
    q, out = torch.empty_like(s["q"]), torch.empty_like(s["q"])
    one = torch.ones_like(s["kv_lens"])

    def step():
        gpu.paged_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["cu"], s["kv_lens"],
                         s["table"], q=s["q"], inv_freq=f, q_out=q)
        attend(gpu, c, {**s, "q": q}, max_kv=None, out=out, workspace=room, return_lse=False)
        s["kv_lens"].add_(one)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    g = torch.Generator().manual_seed(3)
    for i in range(1, 8):
        for name in ("q", "k", "v"):
            s[name].copy_(torch.randn(s[name].shape, generator=g))
        graph.replay()
        torch.cuda.synchronize()
        lens = [n + i for n in c.kv_lens]
        assert s["kv_lens"].tolist() == [n + 1 for n in lens]
        cpu = {**s["cpu"], "q": q.double().cpu().numpy(), "kv_lens": lens,
               "k_cache": s["k_cache"].double().cpu().numpy(),
               "v_cache": s["v_cache"].double().cpu().numpy()}
        check_attention(dataclasses.replace(c, kv_lens=tuple(lens)), {"cpu": cpu}, out, None)


def test_rotation_with_its_gradients(gpu):
    from rmsnorm_fp8_quantization_gb300 import autograd as A
    f = gpu.rope_frequencies(64)
    pos = torch.arange(12, device="cuda").expand(2, 12).contiguous()
    q, k = (torch.randn(2, 12, h, 64, device="cuda").bfloat16() for h in (4, 2))
    w = torch.randn_like(q), torch.randn_like(k)

    def go():
        a, b = q.detach().requires_grad_(), k.detach().requires_grad_()
        x, y = A.rope(a, b, f, pos)
        return x, y, *torch.autograd.grad((x, y), (a, b), w)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        go()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = go()
    for t in (q, k, *w):
        t.copy_(torch.randn_like(t))
    pos.add_(100)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, go()):
        assert torch.equal(a, b)
