"""Offsets and lengths at the ends of 32 bits.  They are read on the device: what the calls do not allow is reported in the
status word, its sequence is skipped, and the others are right.  Differences of such numbers do not fit 32 bits."""
import pytest
import torch

import huffman_decode_canonical_b200 as entro

gpu = pytest.mark.gpu
LOW, HIGH = -2 ** 31, 2 ** 31 - 1


def _ints(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def _cache():
    """Two sequences of 40 and 20 tokens in pages of 16: (cache, table, slots, their tokens)"""
    g = torch.Generator().manual_seed(3)
    cache = entro.KVCache.empty(8, 2, 64, 16, slots=3)
    x = torch.randn(60, 2, 64, generator=g).to(torch.bfloat16).cuda()
    table = torch.tensor([[5, 1, 7], [2, 0, 3]], dtype=torch.int32, device="cuda")
    slots = _ints(2, 0)
    cache.append(x, -x, _ints(0, 40, 60), table, _ints(40, 20), slots=slots)
    return cache, table, slots, x


@gpu
@pytest.mark.parametrize("cu,right", [((-5, 35, 55), [1]), ((LOW, 35, 55), [1]), ((LOW, LOW, 20), []), ((0, 40, HIGH), [0]), ((0, 40, 61), [0]),
                                      ((0, 40, 30), [0]), ((0, 40, LOW), [0]), ((1, LOW, 20), []), ((HIGH, HIGH, HIGH), []), ((LOW, HIGH, 60), []),
                                      ((20, 60, 59), [0])])
def test_read(cu, right):
    cache, table, slots, _ = _cache()
    want = [cache.read(table, _ints(0, 40, 60), 60, slots=slots)[i] for i in range(2)]
    out, status = [torch.full_like(w, 7.0) for w in want], _status()
    cache.read(table, _ints(*cu), 60, slots=slots, out=tuple(out), status=status)
    assert int(status) == entro.E_INVAL
    at, n = (0, 40), (40, 20)
    for got, w in zip(out, want):
        left = torch.ones(60, dtype=torch.bool)
        for b in right:
            length = cu[b + 1] - cu[b]
            assert length == n[b]
            assert torch.equal(got[cu[b]:cu[b + 1]], w[at[b]:at[b] + n[b]])
            left[cu[b]:cu[b + 1]] = False
        assert bool((got.cpu()[left] == 7).all())


@gpu
@pytest.mark.parametrize("cu,lens", [((0, 3, 5), (LOW, 22)), ((0, 3, 5), (LOW + 2, 22)), ((0, 3, 5), (2, 22)), ((1, LOW, 2), (43, 22)), ((1, LOW, 2), (HIGH, HIGH)),
                                     ((LOW, 3, 5), (43, 22)), ((0, HIGH, 5), (HIGH, 22)), ((0, 3, 5), (HIGH, 22)), ((0, 6, 5), (46, 22))])
def test_append(cu, lens):
    cache, table, slots, _ = _cache()
    held = [t.clone() for t in cache._buffers]
    status, x = _status(), torch.ones(5, 2, 64, dtype=torch.bfloat16, device="cuda")
    cache.append(x, x, _ints(*cu), table, _ints(*lens), slots=slots, status=status)
    assert int(status) == entro.E_INVAL
    second = cu[1] == 3 and lens[1] == 22  # sequence 1's arguments are right: two more tokens after its 20, in slot 0
    for i, (now, was) in enumerate(zip(cache._buffers, held)):
        if i >= 4 and second:  # the tails
            assert bool((now[0, :, 4:6] == 1).all())
            now, was = now.clone(), was.clone()
            now[0, :, 4:6] = was[0, :, 4:6] = 0
        # (the rest may hold NaN: compared as whole numbers)
        assert torch.equal(now.view(torch.int8), was.view(torch.int8))


@gpu
@pytest.mark.parametrize("cu,right", [((1, LOW, 100), []), ((40, LOW + 3, 100), []), ((LOW, 40, 100), [1]), ((0, 40, LOW), [0]), ((0, HIGH, LOW), []), ((LOW, LOW, LOW), [])])
@pytest.mark.parametrize("of", ["queries", "keys", "both"])
def test_prompt(cu, right, of):
    g = torch.Generator().manual_seed(4)
    q, k = (torch.randn(100, h, 64, generator=g).to(torch.bfloat16).cuda() for h in (4, 2))
    good, bad = _ints(0, 40, 100), _ints(*cu)
    want = entro.attention_prompt(q, k, k, good)
    out, status = torch.full_like(q, 7.0), _status()
    entro.attention_prompt(q, k, k, bad if of != "keys" else good, None if of == "both" else bad if of == "keys" else good, out=out, status=status)
    assert int(status) == entro.E_INVAL
    left = torch.ones(100, dtype=torch.bool)
    for b in right:
        at = slice(40 * b, 40 + 60 * b)
        assert torch.equal(out[at], want[at])
        left[at] = False
    assert bool((out.cpu()[left] == 7).all())
