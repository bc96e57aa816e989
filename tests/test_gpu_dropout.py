"""Dropout with the residual's addition: the mask bit by bit, values within one rounding."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float16, torch.float32]


def draw(i, seed, offset):
    """The four words of Philox 4x32-10 of each counter (i, offset) under seed, one after another."""
    m = np.uint64(0xFFFFFFFF)
    half = lambda x: (np.uint64(x % 2 ** 32), np.uint64(x // 2 ** 32 % 2 ** 32))
    c = [i & m, i >> np.uint64(32), *(np.full_like(i, x) for x in half(offset))]
    k = [int(x) for x in half(seed)]
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), b & m,
             (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), a & m]
        k = [(k[0] + 0x9E3779B9) % 2 ** 32, (k[1] + 0xBB67AE85) % 2 ** 32]
    return np.stack(c, -1).reshape(-1)


def words(n, seed, offset):
    return draw(np.arange((n + 3) // 4, dtype=np.uint64), seed, offset)[:n]


def kept(n, p, seed, offset):
    return torch.from_numpy(words(n, seed % 2 ** 64, offset % 2 ** 64) >= np.uint64(math.ceil(p * 2 ** 32)))


def rng(seed=5, offset=0):
    return torch.tensor([seed, offset], dtype=torch.int64, device="cuda")


def check(got, x, p, keep, residual=None):
    """One rounding of the result, and 32-bit ones (the factor, the product, the sum) before it."""
    x64 = x.double().cpu()
    y = torch.where(keep.view(x.shape), x64 / (1 - p) if p < 1 else x64, 0.0)
    size = y.abs()
    if residual is not None:
        y = y + residual.double().cpu()
        size = size + residual.double().cpu().abs()
    f = torch.finfo(x.dtype)
    off = f.eps / 2 * y.abs() + 2.0 ** -22 * size + f.smallest_normal * f.eps
    assert ((got.double().cpu() - y).abs() <= off).all()
    if residual is None:
        assert (got.cpu()[~keep.view(x.shape)] == 0).all()


def test_known_answers():
    """The generator's published vectors."""
    assert [hex(w) for w in words(4, 0, 0)] == ["0x6627e8d5", "0xe169c58d", "0xbc57ac4c", "0x9b00dbd8"]


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("shape", [(1,), (3,), (7, 9), (64, 1024), (33, 257), (5, 4001), (513, 16), (2, 3, 5, 8)],
                         ids=str)
@pytest.mark.parametrize("add", [False, True], ids=["alone", "residual"])
def test_forward_and_backward(gpu, shape, dtype, add):
    g = torch.Generator().manual_seed(1)
    x, r, d = (torch.randn(*shape, generator=g).to(dtype).cuda() for _ in range(3))
    k = kept(x.numel(), 0.3, 5, 2 ** 40 + 3)
    r = r if add else None
    check(gpu.dropout_fwd(x, 0.3, rng(5, 2 ** 40 + 3), residual=r), x, 0.3, k, r)
    check(gpu.dropout_bwd(d, 0.3, rng(5, 2 ** 40 + 3)), d, 0.3, k)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("p", [0.0, 1e-30, 2.0 ** -32, 0.5, 0.9, 1 - 2.0 ** -32, 1 - 2.0 ** -40, 1.0])
def test_probabilities(gpu, p, dtype):
    x = torch.full((8200,), 0.5, dtype=dtype, device="cuda")
    r = torch.full_like(x, 3.0)
    got = gpu.dropout_fwd(x, p, rng(-77, -1), residual=r)
    if p < 1 - 2.0 ** -32:
        check(got, x, p, kept(8200, p, -77, -1), r)
    else:
        k = kept(8200, p, -77, -1)
        assert (got.cpu()[~k] == 3.0).all() and (p < 1 or not k.any())


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("skip", [1, 3])
def test_unaligned(gpu, dtype, skip):
    """The scalar path draws the same mask."""
    n = 5000
    base = [torch.randn(n + 16, device="cuda").to(dtype) for _ in range(3)]
    x, r, out = (t[skip:skip + n] for t in base)
    want = gpu.dropout_fwd(x.clone(), 0.4, rng(), residual=r.clone())
    guard = base[2].clone()
    gpu.dropout_fwd(x, 0.4, rng(), residual=r, out=out)
    assert torch.equal(out, want)
    assert torch.equal(base[2][:skip], guard[:skip]) and torch.equal(base[2][skip + n:], guard[skip + n:])


@pytest.mark.parametrize("p", [0.5, 1.0])
def test_dropped_values_have_no_part(gpu, p):
    k = kept(4096, p, 5, 0)
    x = torch.where(k.cuda(), 1.0, float("nan")).bfloat16()
    x[~k.cuda() & (torch.arange(4096, device="cuda") % 2 == 0)] = float("inf")
    got = gpu.dropout_fwd(x, p, rng(), residual=torch.ones_like(x))
    assert torch.equal(got.cpu(), torch.where(k, 1 + 1 / (1 - p) if p < 1 else 1.0, 1.0).bfloat16())


def test_in_place(gpu):
    x, r = (torch.randn(1000, 33, device="cuda") for _ in range(2))
    want = gpu.dropout_fwd(x, 0.2, rng(), residual=r)
    a, b = x.clone(), r.clone()
    assert gpu.dropout_fwd(a, 0.2, rng(), residual=r, out=a) is a and torch.equal(a, want)
    assert torch.equal(gpu.dropout_fwd(x, 0.2, rng(), residual=b, out=b), want)
    d = x.clone()
    assert torch.equal(gpu.dropout_bwd(d, 0.2, rng(), out=d), gpu.dropout_bwd(x, 0.2, rng()))


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("p", [0.0, 0.3, 1.0])
def test_in_place_of_many_blocks(gpu, p, dtype):
    """Whatever block runs first, each element is read before it is written."""
    g = torch.Generator().manual_seed(2)
    x, r = (torch.randn(3001, 1021, generator=g).to(dtype).cuda() for _ in range(2))
    for residual in (None, r):
        want = gpu.dropout_fwd(x, p, rng(8, 1), residual=residual)
        for _ in range(3):
            a = x.clone()
            assert torch.equal(gpu.dropout_fwd(a, p, rng(8, 1), residual=residual, out=a), want)
    for _ in range(3):
        b = r.clone()
        assert torch.equal(gpu.dropout_fwd(x, p, rng(8, 1), residual=b, out=b), want)


def test_counter_beyond_32_bits(gpu):
    """Elements past 2^34: the counter's high half."""
    n = 2 ** 34 + 4096 + 5
    if torch.cuda.mem_get_info()[0] < 4.5 * n:
        pytest.skip("needs 77 GB")
    x = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    out = gpu.dropout_fwd(x, 0.5, rng(9, 1), out=x)
    i = np.arange(2 ** 32, 2 ** 32 + 1026, dtype=np.uint64)
    tail = out[2 ** 34:].cpu()
    keep = draw(i, 9, 1)[: tail.numel()] >= 2 ** 31
    assert torch.equal(tail != 0, torch.from_numpy(keep))
    head = out[: 4096].cpu()
    assert torch.equal(head != 0, kept(4096, 0.5, 9, 1))


def test_offsets_and_seeds_differ(gpu):
    x = torch.ones(4096, device="cuda")
    masks = [gpu.dropout_fwd(x, 0.5, rng(s, o)) != 0 for s, o in ((1, 0), (1, 1), (2, 0), (1, 2 ** 32), (2 ** 32, 0))]
    for i, a in enumerate(masks):
        for b in masks[:i]:
            # equal bits of independent masks: 2048 +- 32 (one deviation); 10 of them
            assert abs((a == b).sum().item() - 2048) < 320


def test_share_of_dropped(gpu):
    n = 1 << 22
    got = gpu.dropout_fwd(torch.ones(n, device="cuda"), 0.1, rng(123, 4))
    # mean 0.1, deviation sqrt(0.09 / n): 8 of them
    assert abs((got == 0).double().mean().item() - 0.1) < 8 * math.sqrt(0.09 / n)
