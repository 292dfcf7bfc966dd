"""Visible keys that all score -infinity leave no softmax: the output is NaN, as by the formula, and not the 0 of a query
that sees no key.  Where only some of a query's keys score so, they count nothing."""
import pytest
import torch

import huffman_decode_canonical_b200 as entro
from test_prompt import HALF_STEP, _check, _cu, _gen, _inputs

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dim", [64, 96, 128])
@pytest.mark.parametrize("queries,keys", [([70, 200], [70, 200]), ([5, 40], [300, 20]), ([3], [4400]), ([200], [4100])])
def test_prompt(queries, keys, dim, dtype):
    g = _gen(31, queries[0], dim)
    q, k, v = _inputs(g, sum(queries), sum(keys), 4, 2, dim, dtype)
    k[..., 0] = -1
    q[2, 1, 0] = q[-1, 2, 0] = INF
    got = _check(q, k, v, _cu(queries), _cu(keys))
    assert bool(torch.isnan(got[2, 1]).all()) and int(torch.isnan(got).any(2).sum()) == 2
    # in the first sequence only the last key has a score; with an infinity among its values, its rows are taken one by one
    q, k, v = _inputs(g, sum(queries), sum(keys), 4, 2, dim, dtype)
    q[..., 0] = 1
    k[:keys[0] - 1, :, 0] = -INF
    got = _check(q, k, v, _cu(queries), _cu(keys))
    seen = queries[0] - 1  # the first sequence's last query sees its last key
    assert bool(torch.isfinite(got[seen]).all()) and bool(torch.isnan(got[:seen]).all())
    v[keys[0] - 1, 0, 3] = INF
    again = _check(q, k, v, _cu(queries), _cu(keys))
    assert bool(torch.isnan(again[:seen]).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("lengths", [[3, 1, 0, 16], [37, 64, 100, 5], [5000, 90, 16, 17]])
def test_cache(lengths, dtype):
    g = _gen(32, lengths[0])
    batch, dim, page = len(lengths), 64, 16
    width = max(lengths) // page
    table = torch.arange(batch * width, dtype=torch.int32, device="cuda").view(batch, width)
    lens, cu = torch.tensor(lengths, dtype=torch.int32, device="cuda"), _cu(lengths).cuda()
    q, k, v = (x.cuda() for x in _inputs(g, batch, sum(lengths), 4, 2, dim, dtype))
    k[..., 0] = -1

    def attend(q, k):
        cache = entro.KVCache.empty(batch * width, 2, dim, page, slots=batch, dtype=dtype)
        cache.append(k, v, cu, table, lens)
        return cache.attend(q, table, lens)

    plain = attend(q, k)
    w = q.clone()
    w[0, 1, 0] = w[-1, 3, 0] = INF
    w[2, 2, 0] = INF
    got = attend(w, k)
    for b, h in ((0, 1), (batch - 1, 3), (2, 2)):
        assert bool(torch.isnan(got[b, h]).all() if lengths[b] else (got[b, h] == 0).all())
        got[b, h] = plain[b, h]
    # The other heads' sums may be taken from another reference: on each side the weights are off by 2^-11 of themselves, the
    # sums by less than 2^-17, the output by half a step, all of at most the largest value.
    near = 2 * (HALF_STEP[dtype] + 2.0 ** -11 + 2.0 ** -17) * float(v.abs().max())
    assert float((got.float() - plain.float()).abs().max()) <= near
    # keys of the open block that all score -infinity: the coded ones have it all, and where there are none nothing has
    at = 0
    for n in lengths:
        k[at + n // page * page:at + n, :, 0] = -INF
        at += n
    q[..., 0] = 1
    got = attend(q, k)
    lens -= lens % page
    full = torch.cat([torch.arange(a, a + n // page * page) for a, n in zip(_cu(lengths).tolist(), lengths)]).cuda()
    cu, k, v = _cu(lens.tolist()).cuda(), k[full], v[full]
    alone = attend(q, k)
    for b, n in enumerate(lengths):
        if n and n < page:
            assert bool(torch.isnan(got[b]).all())
        else:  # (the same sums, cut elsewhere)
            assert float((got[b].float() - alone[b].float()).abs().max()) <= near
