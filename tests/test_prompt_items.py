"""Prompt attention in calls of more blocks than there are SMs: a CTA that is done with a block of 256 queries goes on with
the next one that has not started, and everything it keeps between them (barriers' phases, TMEM buffers, the ring of key and
value tiles, marks of values to be taken one by one) goes on too.  Every call here has several blocks for each SM, of unlike
shapes one after the other, and is compared with the 64-bit softmax under the bound of test_prompt.py."""
import numpy as np
import pytest
import torch

import huffman_decode_canonical_b200 as entro
from test_prompt import HALF_STEP, _cu, _gen, _inputs, _reference

pytestmark = pytest.mark.gpu

MIXED = [1, 44, 129, 0, 257, 900, 0, 300, 600, 2, 255, 256, 513, 31]


def _check(q, k, v, queries, keys, per_sm=2.0, repeats=3):
    """Against the definition, in 64 bits on the GPU; the same bits every time."""
    heads, sms = q.shape[1], torch.cuda.get_device_properties(0).multi_processor_count
    blocks = sum(-(-n // 256) for n in queries) * heads
    assert blocks >= per_sm * sms and (sum(keys) // len(keys) < 1024 or blocks > sms)  # (else a cluster shares keys: one block each)
    cu, cu_k = _cu(queries).cuda(), _cu(keys).cuda()
    q, k, v = (t.cuda() for t in (q, k, v))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = entro.attention_prompt(q, k, v, cu, None if queries == keys else cu_k, status=status)
    for _ in range(repeats):
        again = entro.attention_prompt(q, k, v, cu, None if queries == keys else cu_k)
        assert torch.equal(got.view(torch.int16), again.view(torch.int16))
    assert int(status) == 0
    with torch.device("cuda"):
        o, mag, big = _reference(q, k, v, cu.cpu(), cu_k.cpu(), q.shape[2] ** -0.5)
    h = HALF_STEP[q.dtype]
    bound = mag * (h + 2.0 ** -18 + 2 * 16 * 2.0 ** -23 * big + (k.shape[0] / 16 + 64) * 2.0 ** -23) + o.abs() * h + 2.0 ** -25
    x, nan, inf = got.double(), torch.isnan(o), torch.isinf(o)
    assert torch.equal(torch.isnan(x), nan) and torch.equal(x[inf], o[inf])
    ok = ~nan & ~inf
    assert bool(((x - o).abs() <= bound)[ok].all()), float(((x - o).abs() / bound)[ok].max())
    return got


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dim", [64, 96, 128])
def test_mixed_lengths(dim, dtype):
    q, k, v = _inputs(_gen(41, dim), sum(MIXED), sum(MIXED), 32, 8, dim, dtype)
    _check(q, k, v, MIXED, MIXED)


@pytest.mark.parametrize("dim", [64, 96, 128])
def test_continued_and_cut_off(dim):
    """Blocks that see no key, and ones whose first or second half does not, between ordinary ones."""
    queries = [300, 40, 0, 513, 200, 7, 256, 900, 130, 384, 1]
    keys = [20, 500, 9, 513, 0, 300, 100, 640, 2, 129, 700]
    q, k, v = _inputs(_gen(42, dim), sum(queries), sum(keys), 32, 8, dim, torch.bfloat16)
    got, at = _check(q, k, v, queries, keys), 0
    for n, m in zip(queries, keys):
        assert bool((got[at:at + max(0, n - m)] == 0).all())
        at += n


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dim", [64, 96, 128])
def test_blocks_taken_row_by_row_between_others(dim, dtype):
    """Infinities and NaN among the values of some sequences and key heads: consecutive blocks differ in whether they are
    taken again row by row."""
    lengths = [70, 129, 300, 0, 257, 44, 200, 31, 513]
    q, k, v = _inputs(_gen(43, dim), sum(lengths), sum(lengths), 32, 4, dim, dtype)
    ends = np.cumsum([0] + lengths)
    for b, head, at, value in ((0, 1, 69, "nan"), (1, 0, 128, "inf"), (2, 3, 40, "-inf"), (2, 2, 299, "inf"), (4, 1, 256, "nan"), (6, 0, 0, "inf"), (8, 2, 300, "-inf")):
        v[ends[b] + at, head, 3] = float(value)
    got = _check(q, k, v, lengths, lengths)
    assert bool(torch.isfinite(got[:, :, 4:]).all())


def test_many_short_prompts():
    g = _gen(44)
    lengths = torch.randint(0, 60, (300,), generator=g).tolist()
    q, k, v = _inputs(g, sum(lengths), sum(lengths), 8, 2, 64, torch.float16)
    _check(q, k, v, lengths, lengths)


@pytest.mark.parametrize("heads,kv", [(32, 1), (35, 5)])
def test_head_layouts(heads, kv):
    lengths = [700, 3, 256, 90, 400, 257, 128, 129]
    q, k, v = _inputs(_gen(45, heads), sum(lengths), sum(lengths), heads, kv, 128, torch.bfloat16)
    _check(q, k, v, lengths, lengths)


def test_one_long_prompt():
    q, k, v = _inputs(_gen(46), 5000, 5000, 16, 4, 128, torch.bfloat16)
    _check(q, k, v, [5000], [5000])


def test_sharp_scores():
    """Row maxima that rise block by block: outputs rescaled in some blocks and not in others."""
    lengths = [900, 129, 600, 44, 513, 257, 300, 700]
    q, k, v = _inputs(_gen(47), sum(lengths), sum(lengths), 32, 8, 96, torch.bfloat16)
    ramp = torch.linspace(0.05, 4, sum(lengths))[torch.randperm(sum(lengths), generator=_gen(48))]
    _check(q.abs(), (k.abs() * ramp[:, None, None]).to(k.dtype), v, lengths, lengths)


def test_captured_and_on_two_streams():
    q, k, v = (t.cuda() for t in _inputs(_gen(49), sum(MIXED), sum(MIXED), 32, 8, 64, torch.bfloat16))
    cu = _cu(MIXED).cuda()
    want = entro.attention_prompt(q, k, v, cu)
    held_cu, graph = torch.zeros_like(cu), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = entro.attention_prompt(q, k, v, held_cu)
    for _ in range(3):
        held_cu.copy_(cu)
        graph.replay()
        assert torch.equal(y, want)
        held_cu.copy_(cu.flip(0).sub(cu[-1]).neg())  # the lengths in the other order
        graph.replay()
        assert torch.equal(y, entro.attention_prompt(q, k, v, held_cu))
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    torch.cuda.synchronize()
    for _ in range(10):
        for s in streams:
            got.append(entro.attention_prompt(q, k, v, cu, stream=s))
    torch.cuda.synchronize()
    assert all(torch.equal(g, want) for g in got)
