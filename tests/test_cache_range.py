"""Attention over the cache where numbers of one call lie far apart: bfloat16 channels of any magnitude beside one another,
infinities and NaN in the open block.  The bound is that of the attention's other tests (test_kvcache.py): each output
against the sum of the magnitudes that go into it, so a small channel has to be as exact beside a large one as alone."""
import pytest
import torch

import huffman_decode_canonical_b200 as entro
from test_kvcache import HALF_STEP, Case, _check_attention

pytestmark = pytest.mark.gpu
BF16, FP16 = torch.bfloat16, torch.float16


def _spread(dim, low, high, g):
    """Powers of two from 2^low to 2^high, in any order."""
    return 2.0 ** torch.linspace(low, high, dim)[torch.randperm(dim, generator=g)].round()


@pytest.mark.parametrize("dim,page,n", [(64, 16, 13), (96, 64, 50), (128, 128, 127), (128, 16, 1)])
def test_channels_of_the_open_block(dim, page, n):
    """Keys whose channels span 2^120 (queries the inverse, so that all of them count) and values whose channels do."""
    c = Case(1, 2, dim, page, BF16, width=1, seed=20)
    k, v = c.tokens(n), c.tokens(n)
    by, of = _spread(dim, -60, 60, c.g), _spread(dim, -20, 100, c.g)
    c.append([n], packed=((k * by).to(BF16), (v * of).to(BF16)))
    _check_attention(c, 8, q=(torch.randn(1, 8, dim, generator=c.g) / by).to(BF16))


@pytest.mark.parametrize("dim", [64, 96, 128])
def test_a_large_number_of_the_open_block(dim):
    """One token's number 2^100 times the others', in a channel of its own; its token gets hardly any weight, or much."""
    for sign in (-1.0, 1.0):
        c = Case(1, 1, dim, 32, BF16, width=3, seed=21)
        k, v = c.tokens(75), c.tokens(75)
        k[:, 0, 1] = 0
        k[70, 0, 1] = 3 * sign
        v[70, 0, 7] = 2.0 ** 100
        c.append([75], packed=(k, v))
        q = torch.randn(1, 4, dim, generator=c.g)
        q[:, :, 1] = 4
        _check_attention(c, 4, q=q.to(BF16))


@pytest.mark.parametrize("dim,page,kv,group", [(64, 16, 2, 4), (96, 32, 1, 3), (128, 64, 2, 8), (128, 16, 1, 12)])
def test_channels_of_the_query(dim, page, kv, group):
    """Queries with a channel 2^60 times the others where the keys hold 0, or channels that span 2^200: coded and open blocks."""
    c = Case(3, kv, dim, page, BF16, width=-(-300 // page), seed=22)
    n = [300, 2 * page, page + 5]
    k, v = c.tokens(sum(n)), c.tokens(sum(n))
    k[..., 5] = 0
    c.append(n, packed=(k, v))
    q = torch.randn(3, kv * group, dim, generator=c.g)
    q[:, ::2, 5] = 2.0 ** 60
    q[1, 1] *= _spread(dim, -120, 0, c.g)
    q[2, 0, 5] = 2.0 ** 31  # the last that one factor fits, and the first that it does not
    q[2, 1, 5] = 2.0 ** 33
    _check_attention(c, kv * group, q=q.to(BF16))
    q = torch.randn(3, kv * group, dim, generator=c.g)
    q[0] = 0
    q[1, :, :] = 0
    q[1, 0, 9], q[1, 0, 10] = 2.0 ** -133, 2.0 ** -100  # the smallest number, beside another and alone
    q[1, 1, 9] = 2.0 ** -133
    _check_attention(c, kv * group, q=q.to(BF16))


def _expect(q, k, v, keep):
    """(o, sum p |v|, largest sum of the scores' magnitudes) over the tokens that are kept, 64 bits: q [heads, dim]"""
    g = q.shape[0] // k.shape[1]
    o, mag, big = (torch.zeros(q.shape, dtype=torch.float64) for _ in range(3))
    for h in range(q.shape[0]):
        a, b, w = q[h].double(), k[keep, h // g].double(), v[keep, h // g].double()
        p = torch.softmax(b @ a * q.shape[1] ** -0.5, 0)
        o[h], mag[h], big[h] = p @ w, p @ w.abs(), (b.abs() @ a.abs()).max() * q.shape[1] ** -0.5
    return o, mag, big


def _near(got, want, rows=slice(None), channels=slice(None)):
    o, mag, big = (t[rows][:, channels] for t in want)
    x = got.cpu().double()[rows][:, channels]
    bound = mag * (2.0 ** -11 + 2.0 ** -18 + 2 * 16 * 2.0 ** -23 * big) + o.abs() * HALF_STEP[got.dtype] + 2.0 ** -25
    assert bool(((x - o).abs() <= bound).all()), float(((x - o).abs() / bound).max())


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("dim", [64, 96, 128])
def test_infinities_in_the_open_block(dim, value, dtype):
    g = torch.Generator().manual_seed(23)
    n, page, at = 29, 32, 17
    q = torch.randn(4, dim, generator=g).to(dtype)
    q[:, 3] = 1
    k, v = (torch.randn(n, 2, dim, generator=g).to(dtype) for _ in range(2))
    everyone, others = torch.ones(n, dtype=torch.bool), torch.arange(n) != at
    table, lens = torch.zeros((1, 1), dtype=torch.int32, device="cuda"), torch.tensor([n], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")

    def attend(k, v):
        cache = entro.KVCache.empty(1, 2, dim, page, dtype=dtype)
        cache.append(k.cuda(), v.cuda(), cu, table, lens)
        return cache.attend(q[None].cuda(), table, lens)[0]

    # a value: its channel of its key head's queries has it, and no other output changes
    w = v.clone()
    w[at, 0, 5] = value
    got, want = attend(k, w), _expect(q, k, v, everyone)
    rest = torch.arange(dim) != 5
    _near(got, want, channels=rest)
    _near(got, want, rows=slice(2, 4))
    x = got[:2, 5].cpu().double()
    assert bool(torch.isnan(x).all()) if value != value else bool((x == value).all())
    # a key that scores -inf counts nothing; +inf and NaN leave no softmax
    w = k.clone()
    w[at, 0, 3] = value
    got = attend(w, v)
    _near(got, want, rows=slice(2, 4))
    if value == float("-inf"):
        _near(got, _expect(q, k, v, others), rows=slice(0, 2))
    else:
        assert bool(torch.isnan(got[:2]).all())
