"""Infinities and NaN among values that only some rows see: they reach the rows that see them, as by the formula, change no
other output by a bit, and a long context does not make the call give up its waits."""
import pytest
import torch

import huffman_decode_canonical_b200 as entro
from test_prompt import _check, _cu, _gen, _inputs

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dim", [64, 96, 128])
@pytest.mark.parametrize("queries,keys", [([300, 90, 257], [300, 90, 257]), ([130, 5], [500, 40]), ([200], [150]), ([40], [4096]), ([260], [2300])])
def test_values_of_every_kind(queries, keys, dim, dtype):
    g = _gen(61, queries[0], dim)
    q, k, v = _inputs(g, sum(queries), sum(keys), 4, 2, dim, dtype)
    plain = entro.attention_prompt(q.cuda(), k.cuda(), v.cuda(), _cu(queries).cuda(), _cu(keys).cuda()).cpu()
    q[..., 1] = 1
    at = keys[0] - 1
    for back, head, channel, value in ((0, 0, 3, INF), (0, 1, 5, NAN), (1, 0, 3, INF), (2, 0, 4, -INF), (5, 0, 4, INF), (9, 0, 6, -INF), (20, 1, 7, -INF)):
        v[at - back, head, channel] = value
    _check(q, k, v, _cu(queries), _cu(keys))
    # a key that scores -infinity has weight 0: 0 times its infinity is NaN
    k[at - 3, 0, 1] = -INF
    v[at - 3, 0, 9], v[at - 3, 0, 10] = INF, 2.0
    got = _check(q, k, v, _cu(queries), _cu(keys)).cpu()
    last = queries[0] - 1
    assert bool(torch.isnan(got[last, :2, 9]).all()) and bool(torch.isfinite(got[last, :2, 10:]).all())
    # and without any of them: the outputs that they do not reach have the same bits
    q, k, v = _inputs(_gen(61, queries[0], dim), sum(queries), sum(keys), 4, 2, dim, dtype)
    v[at, 0, 3] = v[at - 1, 0, 3] = INF
    got = entro.attention_prompt(q.cuda(), k.cuda(), v.cuda(), _cu(queries).cuda(), _cu(keys).cuda()).cpu()
    rest = torch.arange(dim) != 3
    assert torch.equal(got[..., rest], plain[..., rest]) and torch.equal(got[:, 2:], plain[:, 2:])
    assert bool((got[last, :2, 3] == INF).all())


@pytest.mark.parametrize("queries,keys,heads,kv", [(300, 200000, 8, 1), (4096, 150000, 16, 2), (1, 260000, 4, 4)])
def test_long_contexts(queries, keys, heads, kv):
    """(Rows taken one by one over all their keys would take longer than the waits of the warps beside them.)"""
    dim, g = 64, torch.Generator(device="cuda").manual_seed(62)
    q, k, v = (torch.randn(t, h, dim, generator=g, device="cuda").to(torch.bfloat16) for t, h in ((queries, heads), (keys, kv), (keys, kv)))
    cu, cu_k, status = _cu([queries]).cuda(), _cu([keys]).cuda(), torch.zeros(1, dtype=torch.int32, device="cuda")
    plain = entro.attention_prompt(q, k, v, cu, cu_k, status=status)
    at = keys - 1 - queries // 3
    v[at, 0, 3] = INF
    v[keys - 1, 0, 5] = NAN
    got, first, group = entro.attention_prompt(q, k, v, cu, cu_k, status=status), queries - 1 - queries // 3, heads // kv
    assert int(status) == 0
    assert bool((got[first:, :group, 3] == INF).all()) and bool(torch.isnan(got[-1, :group, 5]).all())
    got[first:, :group, 3] = plain[first:, :group, 3]
    got[-1, :group, 5] = plain[-1, :group, 5]
    assert torch.equal(got, plain)
