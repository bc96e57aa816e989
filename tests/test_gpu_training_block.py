"""The training-side operators together: a block's step (norm, projection, rotation, attention,
projection, dropout into the residual stream) with its gradients, eager and captured, each
operator held to its definition on what it was given."""
import pytest
import torch

from attention_train_cases import Case, check, define, flat
from test_gpu_dropout import check as check_dropout, kept

pytestmark = pytest.mark.gpu
HEADS, KV, DIM, HIDDEN = 6, 2, 64, 384


class Block:
    def __init__(self, gpu, q_lens, dtype=torch.bfloat16, uniform=True, seed=0):
        from rmsnorm_fp8_quantization_gb300 import autograd
        self.A, self.ops = autograd, gpu
        g = torch.Generator().manual_seed(seed)
        r = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std).to(dtype).cuda().requires_grad_()
        self.case = Case(q_lens, heads=HEADS, kv_heads=KV, dim=DIM, dtype=dtype, uniform=uniform)
        self.lead = (len(q_lens), q_lens[0]) if uniform else (sum(q_lens),)
        self.x = r(*self.lead, HIDDEN)
        self.gamma = r(HIDDEN)
        self.w1, self.w2 = r(HIDDEN, (HEADS + 2 * KV) * DIM, std=0.05), r(HEADS * DIM, HIDDEN, std=0.05)
        self.freq = gpu.rope_frequencies(DIM)
        self.rng = torch.tensor([11, 5], dtype=torch.int64, device="cuda")
        self.kw = {}
        if not uniform:
            cu = torch.tensor([0, *q_lens]).cumsum(0).to(torch.int32).cuda()
            self.kw = dict(cu_seqlens=cu, max_q=max(q_lens))
            self.pos = torch.cat([torch.arange(n) for n in q_lens])[None].cuda()
        self.grad = r(*self.lead, HIDDEN).detach()

    def leaves(self):
        return self.x, self.gamma, self.w1, self.w2

    def forward(self, leaves=None):
        """The block's output, and what passes between its operators."""
        x, gamma, w1, w2 = self.leaves() if leaves is None else leaves
        h, res = self.A.rms_norm_with_residual(x, gamma)
        q, k, v = (h @ w1).view(*self.lead, HEADS + 2 * KV, DIM).split([HEADS, KV, KV], -2)
        if self.kw:
            q, k = (t[0] for t in self.A.rope(q[None], k[None], self.freq, self.pos))
        else:
            q, k = self.A.rope(q, k, self.freq)
        o = self.A.attention(q, k, v, **self.kw)
        y = o.flatten(-2) @ w2
        out = self.A.dropout(y, 0.25, self.rng, res)
        return out, dict(q=q, k=k, v=v, o=o, y=y, res=res)


def held(block, mid, out):
    """Each operator's results and gradients against its definition on its own inputs."""
    s = dict(q=mid["q"].detach(), k=mid["k"].detach(), v=mid["v"].detach(), dout=mid["o"].grad, kw=block.kw)
    want = define(block.case, s)
    check("out", mid["o"].detach(), want["out"])
    for n in ("q", "k", "v"):
        check("d" + n, mid[n].grad, want["d" + n])
    n = mid["y"].numel()
    keep = kept(n, 0.25, 11, 5)
    check_dropout(out.detach(), mid["y"].detach(), 0.25, keep, mid["res"].detach())
    check_dropout(mid["y"].grad, block.grad, 0.25, keep)


@pytest.mark.parametrize("q_lens,uniform,dtype", [((200, 200), True, torch.bfloat16),
                                                  ((1, 130, 0, 77), False, torch.bfloat16),
                                                  ((129,), True, torch.float16)], ids=str)
def test_step(gpu, q_lens, uniform, dtype):
    b = Block(gpu, q_lens, dtype, uniform)
    out, mid = b.forward()
    for t in mid.values():
        t.retain_grad()
    out.backward(b.grad)
    torch.cuda.synchronize()
    held(b, mid, out)
    for t in b.leaves():
        assert t.grad is not None and t.grad.isfinite().all() and (t.grad != 0).any()
    # the residual stream's gradient reaches x beside the norm's
    assert torch.equal(mid["res"].grad, b.grad)


def test_captured_step(gpu):
    """Forward and backward in one graph, with an eager graph of the block alive, replayed on other
    values and other masks."""
    b = Block(gpu, (150, 150))
    leaves = [t.detach().clone() for t in b.leaves()]   # (the replays write them)

    def step():
        mine = [t.detach().requires_grad_() for t in leaves]
        out, mid = b.forward(mine)
        return out, mid["o"], *torch.autograd.grad(out, mine, b.grad)

    alive = b.forward()[0]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
        b.rng[1] += 1                            # the next replay draws another mask
    last = None
    for i in range(3):
        for t in leaves[:1] + [b.grad]:
            t.copy_(torch.randn_like(t))
        offset = b.rng[1].item()
        graph.replay()
        torch.cuda.synchronize()
        assert b.rng[1].item() == offset + 1
        b.rng[1] = offset
        want = step()
        b.rng[1] = offset + 1
        for x, y in zip(got, want):
            assert torch.equal(x, y)
        assert last is None or not torch.equal(last, got[0])
        last = got[0].clone()
    alive.sum().backward()
    assert all(t.grad.isfinite().all() for t in b.leaves())


def test_two_graphs_with_workspaces_of_their_own(gpu):
    """Backward passes captured on two streams and replayed at once."""
    from attention_train_cases import make
    calls = []
    for i, c in enumerate((Case((700,), uniform=True, dim=128, heads=4, kv_heads=1),
                           Case((300, 300), uniform=True, dtype=torch.float16, seed=3))):
        s = make(c)
        o, lse = gpu.attention_fwd(s["q"], s["k"], s["v"])
        g = {n: torch.empty(s[n[1]].shape, dtype=c.dtype, device="cuda") for n in ("dq", "dk", "dv")}
        kw = dict(g, workspace=gpu.attention_bwd_workspace(s["q"], s["k"]))
        gpu.attention_bwd(s["dout"], s["q"], s["k"], s["v"], o, lse, **kw)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            gpu.attention_bwd(s["dout"], s["q"], s["k"], s["v"], o, lse, **kw)
        calls.append((c, s, g, graph, torch.cuda.Stream(), o, lse, kw))   # (all that a graph uses)
    for _, _, _, graph, stream, *_ in calls * 3:
        with torch.cuda.stream(stream):
            graph.replay()
    torch.cuda.synchronize()
    for c, s, g, *_ in calls:
        want = define(c, s)
        for n, t in g.items():
            check(n, t, want[n])


def test_padding_gets_no_gradient(gpu):
    b = Block(gpu, (40, 3), uniform=False)
    cu = torch.tensor([2, 30, 41], dtype=torch.int32, device="cuda")     # rows 0, 1, 41, 42: nobody's
    b.kw = dict(cu_seqlens=cu, max_q=28)
    out, mid = b.forward()
    for t in mid.values():
        t.retain_grad()
    out.backward(b.grad)
    for n in ("q", "k", "v"):
        g = mid[n].grad
        assert (g[:2] == 0).all() and (g[41:] == 0).all() and (g[2:41] != 0).any(), n
    assert (mid["o"][:2] == 0).all() and (mid["o"][41:] == 0).all()


def test_lengths_that_do_not_fit_are_flagged(gpu):
    from attention_train_cases import make
    from rmsnorm_fp8_quantization_gb300 import gbnorm as G
    c = Case((40, 30, 20))
    s = make(c)
    q, k, v, d = s["q"], s["k"], s["v"], s["dout"]
    flag = lambda: (torch.cuda.synchronize(), G.gbn_device_error(True))[1][1]
    out, lse = gpu.attention_fwd(q, k, v, **s["kw"])
    flag()
    # beyond the tensor, longer than max_q, descending
    for cu, mq in (([0, 40, 70, 95], 40), ([0, 40, 70, 90], 39), ([0, 60, 40, 90], 60), ([-3, 40, 70, 90], 43)):
        kw = dict(cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"), max_q=mq)
        gpu.attention_fwd(q, k, v, **kw)
        assert flag() == G.GBN_DEVICE_ERR_BAD_INDEX, cu
        gpu.attention_bwd(d, q, k, v, out, lse, **kw)
        assert flag() == G.GBN_DEVICE_ERR_BAD_INDEX, cu
    both = gpu.attention_fwd(q, k, v, **s["kw"]), gpu.attention_bwd(d, q, k, v, out, lse, **s["kw"])
    assert flag() == 0
    want = define(c, s)
    check("out", both[0][0], want["out"])
    check("dq", both[1][0], want["dq"])


@pytest.mark.parametrize("many", [300, 1000])
def test_more_sequences_than_are_taken_by_length(gpu, many):
    lens = tuple((7 * i) % 40 for i in range(many))
    c = Case(lens, heads=2, kv_heads=1, lead=3, trail=70)
    from attention_train_cases import make
    from test_gpu_attention_train import both
    s = make(c)
    got, want = both(gpu, s), define(c, s)
    for n in got:
        check(n, got[n], want[n])


def test_no_keys_and_no_queries_at_all(gpu):
    q, k = torch.randn(2, 5, 4, 64, device="cuda").half(), torch.empty(2, 0, 2, 64, device="cuda").half()
    out, lse = gpu.attention_fwd(q, k, k, causal=False)
    assert (out == 0).all() and (lse == -float("inf")).all()
    dq, dk, dv = gpu.attention_bwd(q, q, k, k, out, lse, causal=False)
    assert (dq == 0).all() and dk.numel() == dv.numel() == 0
    q, k = q[:, :0], torch.randn(2, 5, 2, 64, device="cuda").half()
    out, lse = gpu.attention_fwd(q, k, k, causal=False)
    dq, dk, dv = gpu.attention_bwd(q, q, k, k, out, lse, causal=False)
    assert out.numel() == dq.numel() == 0 and (dk == 0).all() and (dv == 0).all()
