"""Long appends, in which a CTA takes four key heads one after the other: contents compared exactly, with numbers of key
heads that four does not divide, sequences that begin inside an open block and end inside another, and a page that does not
exist."""
import numpy as np
import pytest
import torch

import huffman_decode_canonical_b200 as entro
from test_kvcache import Case

pytestmark = pytest.mark.gpu

# from this many (block, key head) pairs on a CTA takes four heads
FOUR_HEADS = 8192


def _pairs(counts, kv, page):
    tokens, batch = sum(counts), len(counts)
    return min(tokens, (tokens + batch * (page - 2)) // page + batch) * kv


SHAPES = [(64, 16, 5), (96, 16, 6), (128, 32, 20), (64, 16, 2), (64, 64, 33)]


def _counts(page, kv):
    blocks = FOUR_HEADS // kv + 40
    return [page * (blocks // 4) + 5, 1, page * (blocks // 2), 0, page * (blocks // 4) + page - 1]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dim,page,kv", SHAPES)
def test_contents(dim, page, kv, dtype):
    counts = _counts(page, kv)
    c = Case(5, kv, dim, page, dtype, width=max(counts) // page + 3, seed=51)
    c.append([3, page - 1, 0, page, page + 7])  # open blocks, a full one, nothing
    c.check_contents()
    assert _pairs(counts, kv, page) >= FOUR_HEADS
    c.append(counts)
    c.check_contents()
    c.append([page - 1, 1, 2, 0, 1])
    c.check_contents()
    cu = torch.tensor([0] + list(np.cumsum(c.lens.numpy())), dtype=torch.int32).cuda()
    for i, got in enumerate(c.cache.read(c.table, cu, int(c.lens.sum()), slots=c.slots, status=c.status)):
        want = []
        for b in range(c.batch):
            q, s, open_tokens = c.expect(b, i)
            want += [(q.float() * s[..., None, None]).to(dtype).transpose(1, 2).flatten(0, 1), open_tokens]
        assert torch.equal(got.cpu(), torch.cat(want))
    assert int(c.status) == 0


@pytest.mark.parametrize("dim,page,kv", SHAPES[:3])
def test_a_page_that_does_not_exist(dim, page, kv):
    counts = _counts(page, kv)
    c = Case(5, kv, dim, page, torch.bfloat16, width=max(counts) // page + 3, seed=52)
    c.append([3, page - 1, 0, page, page + 7])
    good, at = c.table, (2, 17)
    c.table = good.clone()
    c.table[at] = c.pages
    c.append(counts)
    assert int(c.status) == entro.E_INVAL
    left = int(good[at])
    assert bool((c.cache.k_codes[left] == 99).all()) and bool((c.cache.v_codes[left] == 99).all())
    assert bool(torch.isnan(c.cache.k_scale[left]).all()) and bool(torch.isnan(c.cache.v_scale[left]).all())
    # the block by itself, once its page is there: then everything is as it should be
    c.table = good
    c.status.zero_()
    x = [c.held[2][i][at[1] * page:(at[1] + 1) * page].cuda() for i in range(2)]
    cu, lens = torch.tensor([0, page], dtype=torch.int32, device="cuda"), torch.tensor([(at[1] + 1) * page], dtype=torch.int32, device="cuda")
    c.cache.append(x[0], x[1], cu, good[2:3], lens, slots=c.slots[2:3], status=c.status)
    c.check_contents()
