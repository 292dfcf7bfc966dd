"""The 8-bit key/value cache: what append writes (exactly), what read gives back (exactly), and the attention of single
tokens over it against a 64-bit softmax over the values that the cache stands for.

Bound for the attention, for each output with o = sum p v: the weights are rounded to fp16 (half a step: 2^-11 of each, so
2^-11 sum p |v| in all); their exponents come from 32-bit scores, whose sums of head_dim products are off by a few 2^-23 of
the sum of the products' magnitudes (taken as 16 x 2^-23, which covers a rounding per MMA and the scales'), which moves a
weight by that much of itself, twice (numerator and sum); the rest of the 32-bit arithmetic by less than 2^-18 of
sum p |v|; the output is rounded by half a step of its type."""
import ctypes

import numpy as np
import pytest
import torch

import huffman_decode_canonical_b200 as entro

gpu = pytest.mark.gpu
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def _gen(*key):
    g = torch.Generator()
    g.manual_seed(hash(key) % (1 << 40))
    return g


class Case:
    """A cache and the plain record of what its sequences hold."""

    def __init__(self, batch, kv, dim, page, dtype, width, seed=0, fill=0):
        self.g = _gen(batch, kv, dim, page, width, seed)
        self.pages = batch * width + 3
        self.cache = entro.KVCache.empty(self.pages, kv, dim, page, slots=batch + 2, dtype=dtype)
        for t in (self.cache.k_codes, self.cache.v_codes):
            t.fill_(99)
        for t in (self.cache.k_scale, self.cache.v_scale, self.cache.k_tail, self.cache.v_tail):
            t.fill_(float("nan"))
        order = torch.randperm(self.pages, generator=self.g)[:batch * width].to(torch.int32)
        self.table = order.view(batch, width).cuda()
        self.slots = torch.randperm(batch + 2, generator=self.g)[:batch].to(torch.int32).cuda()
        self.lens = torch.zeros(batch, dtype=torch.int32)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.batch, self.kv, self.dim, self.page, self.dtype = batch, kv, dim, page, dtype
        self.held = [[torch.zeros(0, kv, dim, dtype=dtype) for _ in range(2)] for _ in range(batch)]

    def tokens(self, n):
        x = torch.randn(n, self.kv, self.dim, generator=self.g) * torch.exp(torch.randn(1, self.kv, 1, generator=self.g))
        return x.to(self.dtype)

    def append(self, counts, packed=None):
        k, v = packed if packed is not None else (self.tokens(sum(counts)), self.tokens(sum(counts)))
        cu = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32)
        for b, n in enumerate(counts):
            for i, x in enumerate((k, v)):
                self.held[b][i] = torch.cat([self.held[b][i], x[cu[b]:cu[b + 1]]])
        self.lens += torch.tensor(counts, dtype=torch.int32)
        self.cache.append(k.cuda(), v.cuda(), cu.cuda(), self.table, self.lens.cuda(), slots=self.slots, status=self.status)

    def expect(self, b, i):
        """(codes, scale, open tokens) by definition"""
        x = self.held[b][i]
        full = x.shape[0] // self.page
        blocks = x[:full * self.page].view(full, self.page, self.kv, self.dim).transpose(1, 2)
        a = blocks.float().abs().amax((2, 3), keepdim=True)
        q = torch.where(a > 0, torch.round(blocks.double() * 127 / a.double()), torch.zeros(1, dtype=torch.float64))
        return q, (a / 127)[..., 0, 0], x[full * self.page:]

    def check_contents(self):
        table, slots = self.table.cpu(), self.slots.cpu()
        used = set()
        for b in range(self.batch):
            for i, (codes, scale, tail) in enumerate(((self.cache.k_codes, self.cache.k_scale, self.cache.k_tail),
                                                      (self.cache.v_codes, self.cache.v_scale, self.cache.v_tail))):
                q, s, open_tokens = self.expect(b, i)
                at = table[b, :q.shape[0]].long()
                used.update(at.tolist())
                assert torch.equal(codes.cpu()[at].double(), q)
                assert torch.equal(scale.cpu()[at], s)
                assert torch.equal(tail.cpu()[slots[b].long(), :, :open_tokens.shape[0]], open_tokens.transpose(0, 1))
        free = [p for p in range(self.pages) if p not in used]
        assert bool((self.cache.k_codes.cpu()[free] == 99).all()) and bool(torch.isnan(self.cache.v_scale.cpu()[free]).all())
        assert int(self.status) == 0

    def values(self, b, i):
        """[token, head, channel] in 64 bits: what the cache stands for"""
        q, s, open_tokens = self.expect(b, i)
        coded = (q * s.double()[..., None, None]).transpose(1, 2).flatten(0, 1)
        return torch.cat([coded, open_tokens.double()])


def _attention(c, q, scale):
    """(o, sum p |v|, largest sum of the scores' magnitudes) of q [batch, heads, dim], in 64 bits"""
    o, mag = torch.zeros(q.shape, dtype=torch.float64), torch.zeros(q.shape, dtype=torch.float64)
    big = torch.zeros(q.shape[:2] + (1,), dtype=torch.float64)
    for b in range(c.batch):
        k, v = c.values(b, 0), c.values(b, 1)
        if not k.shape[0]:
            continue
        g = q.shape[1] // c.kv
        qq = q[b].double().view(c.kv, g, c.dim)
        p = torch.softmax(torch.einsum("hgd,thd->hgt", qq, k) * scale, 2)
        o[b] = torch.einsum("hgt,thd->hgd", p, v).flatten(0, 1)
        mag[b] = torch.einsum("hgt,thd->hgd", p, v.abs()).flatten(0, 1)
        big[b] = (torch.einsum("hgd,thd->hgt", qq.abs(), k.abs()) * scale).amax(2).flatten()[:, None]
    return o, mag, big


def _check_attention(c, heads, scale=None, q=None):
    q = torch.randn(c.batch, heads, c.dim, generator=c.g).to(c.dtype) if q is None else q
    got = c.cache.attend(q.cuda(), c.table, c.lens.cuda(), slots=c.slots, scale=scale, status=c.status)
    o, mag, big = _attention(c, q, c.dim ** -0.5 if scale is None else scale)
    bound = mag * (2.0 ** -11 + 2.0 ** -18 + 2 * 16 * 2.0 ** -23 * big) + o.abs() * HALF_STEP[c.dtype] + 2.0 ** -25
    err = (got.cpu().double() - o).abs()
    assert bool((err <= bound).all()), (float((err / bound).max()), (err > bound).nonzero()[:4])
    assert int(c.status) == 0
    again = c.cache.attend(q.cuda(), c.table, c.lens.cuda(), slots=c.slots, scale=scale)
    assert torch.equal(got, again)
    return got


# ------------------------------------------------------------------ refusals (no GPU needed)

def _buffers(pages=2, kv=2, page=16, dim=64, slots=1, dtype=torch.bfloat16):
    return ([torch.zeros(pages, kv, page, dim, dtype=torch.int8) for _ in range(2)] + [torch.zeros(pages, kv) for _ in range(2)]
            + [torch.zeros(slots, kv, page, dim, dtype=dtype) for _ in range(2)])


def test_refusals_of_the_binding():
    for kw in (dict(page=48), dict(dim=80), dict(dtype=torch.float32), dict(pages=0), dict(slots=0)):
        with pytest.raises(ValueError):
            entro.KVCache(*_buffers(**kw))
    for i in range(6):
        for change in (lambda t: t.double(), lambda t: t[..., :-1], lambda t: t.transpose(0, 1)):
            b = _buffers(kv=3)
            b[i] = change(b[i])
            with pytest.raises(ValueError):
                entro.KVCache(*b)
    with pytest.raises(ValueError, match="CUDA"):
        entro.KVCache(*_buffers())


def test_refusals_of_the_library():
    lib, p = entro.lib(), 4096  # any address: argument errors come before it is used

    def cache(**kw):
        f = dict(k_codes=p, v_codes=p, k_scale=p, v_scale=p, k_tail=p, v_tail=p, pages=4, slots=4, kv_heads=2, page_tokens=16, head_dim=64,
                 type=entro.BF16)
        f.update(kw)
        return entro._KVCache(*[f[n] for n, _ in entro._KVCache._fields_])

    def append(c=None, k=p, ks=128, kh=64, v=p, tokens=4, cu=p, table=p, stride=8, width=8, lens=p, slots=p, batch=2):
        return lib.entro_kv_append(c if c is not None else ctypes.byref(cache()), k, ks, kh, v, 128, 64, tokens, cu, table, stride, width, lens, slots, batch, None, None)

    def read(c=None, k=p, ks=128, v=p, tokens=4, cu=p, table=p, stride=8, width=8, slots=p, batch=2):
        return lib.entro_kv_read(c if c is not None else ctypes.byref(cache()), k, ks, 64, v, 128, 64, tokens, cu, table, stride, width, slots, batch, None, None)

    def attend(c=None, q=p, qs=256, heads=4, table=p, stride=8, width=8, lens=p, slots=p, batch=2, scale=0.1, out=p, work=p, nbytes=1 << 40):
        return lib.entro_kv_attend(c if c is not None else ctypes.byref(cache()), q, qs, 64, heads, table, stride, width, lens, slots, batch, scale, out, 256, 64,
                                   work, nbytes, None, None)

    for kw in (dict(k_codes=None), dict(v_scale=None), dict(k_tail=p + 8), dict(pages=0), dict(slots=0), dict(kv_heads=0), dict(kv_heads=65536),
               dict(page_tokens=8), dict(page_tokens=48), dict(head_dim=32), dict(type=entro.F32)):
        for call in (append, read, attend):
            assert call(c=ctypes.byref(cache(**kw))) == entro.E_INVAL, kw
    for call in (append, read, attend):
        for kw in (dict(stride=7), dict(width=-1), dict(batch=-1), dict(table=None), dict(slots=None, batch=5)):
            assert call(**kw) == entro.E_INVAL, (call, kw)
    for kw in (dict(k=None), dict(k=p + 2), dict(ks=100), dict(kh=12), dict(v=None), dict(tokens=-1), dict(cu=None), dict(lens=None)):
        assert append(**kw) == entro.E_INVAL, kw
    for kw in (dict(k=None), dict(ks=4), dict(v=None), dict(tokens=-1), dict(cu=None)):
        assert read(**kw) == entro.E_INVAL, kw
    for kw in (dict(q=None), dict(q=p + 8), dict(qs=12), dict(heads=3), dict(heads=0), dict(lens=None), dict(scale=0.0), dict(scale=-1.0),
               dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=3e38), dict(out=None), dict(work=None), dict(work=p + 4)):
        assert attend(**kw) == entro.E_INVAL, kw
    assert append(tokens=0, k=None) == entro.OK and read(batch=0, k=None) == entro.OK and attend(batch=0, q=None) == entro.OK


# ------------------------------------------------------------------ append and read

@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dim,page,kv", [(64, 16, 1), (64, 128, 3), (96, 32, 2), (96, 16, 5), (128, 64, 8), (128, 128, 2)])
def test_append_and_read_exact(dim, page, kv, dtype):
    """Prompts, chunks that end inside blocks, single tokens, and sequences that get nothing."""
    c = Case(5, kv, dim, page, dtype, width=5, seed=1)
    steps = [[0, 1, page, page - 1, 2 * page + 3], [0, 1, 1, 1, 1], [3, page - 2, 2 * page, 1, 0], [1] * 5, [page + 1, 0, 5, 3 * page - 1, page]]
    for counts in steps:
        c.append(counts)
        c.check_contents()
        cu = torch.tensor([0] + list(np.cumsum(c.lens.numpy())), dtype=torch.int32).cuda()
        total = int(c.lens.sum())
        out = [torch.full((total + 3, kv, dim), 7.0, dtype=dtype, device="cuda") for _ in range(2)]
        c.cache.read(c.table, cu, total + 3, slots=c.slots, out=out, status=c.status)
        for i, got in enumerate(out):
            want = []
            for b in range(c.batch):
                q, s, open_tokens = c.expect(b, i)
                want += [(q.float() * s[..., None, None]).to(dtype).transpose(1, 2).flatten(0, 1), open_tokens]
            assert torch.equal(got[:total].cpu(), torch.cat(want))
            assert bool((got[total:] == 7).all())  # tokens of no sequence
        assert int(c.status) == 0


@gpu
def test_contents_do_not_depend_on_the_chunks():
    whole, pieces = (Case(2, 2, 64, 32, torch.bfloat16, width=8, seed=2) for _ in range(2))
    n = [200, 131]
    k, v = whole.tokens(sum(n)), whole.tokens(sum(n))
    whole.append(n, packed=(k, v))
    done = [0, 0]
    for counts in ([1, 40], [70, 1], [100, 90], [29, 0]):
        part = [torch.cat([x[:200][done[0]:done[0] + counts[0]], x[200:][done[1]:done[1] + counts[1]]]) for x in (k, v)]
        pieces.append(counts, packed=part)
        done = [a + b for a, b in zip(done, counts)]
    assert done == n
    whole.check_contents()
    pieces.check_contents()
    for name in ("k_codes", "v_codes", "k_scale", "v_scale"):
        a, b = (getattr(x.cache, name)[x.table.long()[0, :6]] for x in (whole, pieces))
        assert torch.equal(a, b)


@gpu
def test_append_extremes():
    """Blocks of zeros, of the type's largest and smallest numbers, and with an infinity or NaN in one head."""
    for dtype in (torch.bfloat16, torch.float16):
        f = torch.finfo(dtype)
        c = Case(1, 2, 64, 16, dtype, width=6)
        k = torch.zeros(96, 2, 64, dtype=dtype)
        k[16:32] = f.max
        k[20] = -f.max
        k[32:48] = f.smallest_normal * f.eps
        k[50, 1, 3] = float("inf")
        k[66, 0, 5] = float("nan")
        k[80:] = torch.randn(16, 2, 64, generator=c.g).to(dtype)
        c.append([96], packed=(k, k.clone()))
        scale, codes = c.cache.k_scale.cpu()[c.table.cpu().long()[0]], c.cache.k_codes.cpu()[c.table.cpu().long()[0]]
        assert bool((codes[0] == 0).all()) and bool((scale[0] == 0).all())
        assert int(codes[1].max()) == 127 and int(codes[1].min()) == -127
        assert bool((codes[2] == 127).all())
        assert bool(torch.isnan(scale[3, 1])) and bool((scale[3, 0] == 0)) and bool((codes[3] == 0).all())
        assert bool(torch.isnan(scale[4, 0])) and bool((scale[4, 1] == 0))
        got, _ = c.cache.read(c.table, torch.tensor([0, 96], dtype=torch.int32).cuda(), 96, slots=c.slots)
        got = got.cpu()
        assert bool((got[:16] == 0).all()) and bool((got[16:32].float().abs() == f.max).all())
        assert bool(torch.isnan(got[48:64, 1]).all()) and not bool(torch.isnan(got[48:64, 0]).any())


@gpu
def test_strided_tokens():
    """Keys, values and queries as they lie in one projection's output, outputs inside a larger buffer, a table's slice."""
    c = Case(3, 2, 64, 16, torch.bfloat16, width=4, seed=3)
    qkv = torch.randn(30, 8, 64, generator=c.g).to(torch.bfloat16)
    wide = torch.full((3, 9), -5, dtype=torch.int32, device="cuda")
    wide[:, 2:6] = c.table
    c.table = wide[:, 2:6]
    cu = torch.tensor([0, 13, 13, 30], dtype=torch.int32).cuda()
    x = qkv.cuda()
    c.lens += torch.tensor([13, 0, 17], dtype=torch.int32)
    c.cache.append(x[:, 4:6], x[:, 6:8], cu, c.table, c.lens.cuda(), slots=c.slots, status=c.status)
    for b, (lo, hi) in enumerate(((0, 13), (13, 13), (13, 30))):
        c.held[b] = [qkv[lo:hi, 4:6], qkv[lo:hi, 6:8]]
    c.check_contents()
    big = torch.full((3, 6, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    q = x[:3, :4]
    got = c.cache.attend(q, c.table, c.lens.cuda(), slots=c.slots, out=big[:, 1:5])
    want = c.cache.attend(q.contiguous(), c.table.contiguous(), c.lens.cuda(), slots=c.slots)
    assert torch.equal(got, want) and bool((big[:, 0] == 7).all()) and bool((big[:, 5] == 7).all())
    assert bool((got[1] == 0).all())


# ------------------------------------------------------------------ attention

@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dim,page,kv,group", [(64, 16, 1, 1), (64, 64, 2, 5), (64, 128, 1, 32), (96, 16, 3, 1), (96, 32, 2, 8), (96, 128, 1, 9),
                                               (128, 64, 8, 4), (128, 16, 2, 16), (128, 128, 4, 1)])
def test_attend(dim, page, kv, group, dtype):
    c = Case(7, kv, dim, page, dtype, width=-(-700 // page), seed=4)
    c.append([0, 1, page - 1, page, 65, 333, 640])
    _check_attention(c, kv * group)
    c.append([1, 16, 1, 1, 0, 1, 3])
    _check_attention(c, kv * group, scale=0.3)


@gpu
@pytest.mark.parametrize("batch,longest", [(1, 5000), (1, 37), (3, 20000), (200, 90)])
def test_attend_splits(batch, longest):
    """One sequence over all SMs, uneven ones, and more sequences than CTAs have shares."""
    c = Case(batch, 2, 64, 16, torch.bfloat16, width=-(-longest // 16), seed=batch)
    c.append([max(1, longest * (b + 1) ** 2 // batch ** 2) for b in range(batch)])
    _check_attention(c, 8)


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_attend_sharp_and_large(dtype):
    """Scores far apart (one token takes all), values and keys near the type's limits, queries tiny and large."""
    c = Case(2, 1, 128, 32, dtype, width=12, seed=5)
    n = [300, 45]
    k, v = c.tokens(345), c.tokens(345)
    k[100] *= 30
    k[320] *= 30
    v[7] *= 1000
    c.append(n, packed=(k, v))
    q = torch.randn(2, 4, 128, generator=c.g)
    q[:, 1] *= 2.0 ** -20 if dtype == torch.float16 else 2.0 ** -60
    q[:, 2] *= 100
    q[:, 3] = 0
    _check_attention(c, 4, q=q.to(dtype))
    if dtype == torch.bfloat16:
        c = Case(1, 1, 64, 16, dtype, width=4, seed=6)
        k, v = c.tokens(41), c.tokens(41)
        c.append([41], packed=((k.float() * 2.0 ** 60).to(dtype), (v.float() * 2.0 ** 100).to(dtype)))
        _check_attention(c, 2, q=(torch.randn(1, 2, 64, generator=c.g) * 2.0 ** -60).to(dtype))


@gpu
def test_attend_keeps_what_is_not_cached_out():
    """Everything around the sequences' tokens is NaN: unused pages, the rest of the tails, other slots."""
    for page in (16, 64):
        c = Case(3, 2, 64, page, torch.bfloat16, width=5, seed=7)
        c.append([1, page + 5, 3 * page])
        assert bool(torch.isnan(c.cache.k_tail).any()) and bool(torch.isnan(c.cache.v_scale).any())
        assert not bool(torch.isnan(_check_attention(c, 4)).any())


@gpu
def test_attend_nan_stays_in_its_head():
    c = Case(2, 2, 64, 16, torch.bfloat16, width=4, seed=8)
    k, v = c.tokens(70), c.tokens(70)
    k[3, 1, 5] = float("nan")   # a coded block of sequence 0, key head 1
    v[69, 0, 2] = float("inf")  # the open block of sequence 1, key head 0
    c.append([35, 35], packed=(k, v))
    q = torch.randn(2, 4, 64, generator=c.g).to(torch.bfloat16)
    got = c.cache.attend(q.cuda(), c.table, c.lens.cuda(), slots=c.slots).cpu()
    assert bool(torch.isnan(got[0, 2:]).all()) and bool(torch.isfinite(got[0, :2]).all())
    assert bool(torch.isfinite(got[1, 2:]).all()) and bool(torch.isinf(got[1, :2, 2]).all())
    assert bool(torch.isfinite(got[1, :2, 3:]).all())
    q[0, 0, 0] = float("nan")
    got = c.cache.attend(q.cuda(), c.table, c.lens.cuda(), slots=c.slots).cpu()
    assert bool(torch.isnan(got[0, 0]).all()) and bool(torch.isfinite(got[0, 1]).all())


@gpu
def test_shared_pages():
    """Two sequences that share their first pages and one that is in the batch twice (reading only)."""
    c = Case(2, 2, 64, 16, torch.float16, width=4, seed=9)
    c.append([40, 33])
    table = c.table[[0, 0, 1]].contiguous()
    lens = torch.tensor([40, 32, 33], dtype=torch.int32).cuda()
    slots = c.slots[[0, 1, 1]].contiguous()  # the second holds two full blocks: its slot is not read
    q = torch.randn(1, 4, 64, generator=c.g).to(torch.float16).cuda().repeat(3, 1, 1)
    got = c.cache.attend(q, table, lens, slots=slots)
    one = c.cache.attend(q[:2].contiguous(), c.table, torch.tensor([32, 33], dtype=torch.int32).cuda(), slots=c.slots)
    assert float((got[1:] - one).abs().max()) < 4e-3  # another split of the work: other roundings


@gpu
def test_bad_indices_are_reported():
    def fresh():
        c = Case(2, 1, 64, 16, torch.bfloat16, width=3, seed=10)
        c.append([40, 20])
        torch.cuda.synchronize()
        return c, torch.randn(2, 2, 64, generator=c.g).to(torch.bfloat16).cuda()

    for bad in (-1, 9, 1 << 30):
        c, q = fresh()
        good = c.cache.attend(q, c.table, c.lens.cuda(), slots=c.slots)
        c.table[0, 1] = bad
        got = c.cache.attend(q, c.table, c.lens.cuda(), slots=c.slots, status=c.status)
        assert int(c.status) == entro.E_INVAL and bool(torch.isfinite(got).all())
        assert torch.equal(got[1], good[1])
        c.status.zero_()
        c.cache.read(c.table, torch.tensor([0, 40, 60], dtype=torch.int32).cuda(), 60, slots=c.slots, status=c.status)
        assert int(c.status) == entro.E_INVAL
        c.status.zero_()
        before = c.cache.k_codes.clone()
        x = torch.ones(24, 1, 64, dtype=torch.bfloat16, device="cuda")
        c.cache.append(x, x, torch.tensor([0, 24, 24], dtype=torch.int32).cuda(), torch.full_like(c.table, bad), torch.tensor([64, 20], dtype=torch.int32).cuda(),
                       slots=c.slots, status=c.status)
        assert int(c.status) == entro.E_INVAL and torch.equal(before, c.cache.k_codes)
    for lens in ([40, -3], [40, 64], [1 << 30, 20]):
        c, q = fresh()
        got = c.cache.attend(q, c.table, torch.tensor(lens, dtype=torch.int32).cuda(), slots=c.slots, status=c.status)
        torch.cuda.synchronize()
        assert int(c.status) == entro.E_INVAL
    for slots in ([-1, 0], [1 << 30, 0]):
        c, q = fresh()
        got = c.cache.attend(q, c.table, c.lens.cuda(), slots=torch.tensor(slots, dtype=torch.int32).cuda(), status=c.status)
        assert int(c.status) == entro.E_INVAL
        c.status.zero_()
        x = torch.ones(3, 1, 64, dtype=torch.bfloat16, device="cuda")
        c.cache.append(x, x, torch.tensor([0, 3, 3], dtype=torch.int32).cuda(), c.table, torch.tensor([43, 20], dtype=torch.int32).cuda(),
                       slots=torch.tensor(slots, dtype=torch.int32).cuda(), status=c.status)
        assert int(c.status) == entro.E_INVAL
    # packed tokens that the offsets do not describe
    for cu in ([0, 5, 3], [-1, 2, 4], [0, 2, 99]):
        c, q = fresh()
        before = [t.clone() for t in (c.cache.k_codes, c.cache.v_codes)]
        x = torch.ones(4, 1, 64, dtype=torch.bfloat16, device="cuda")
        c.cache.append(x, x, torch.tensor(cu, dtype=torch.int32).cuda(), c.table, torch.tensor([42, 22], dtype=torch.int32).cuda(), slots=c.slots, status=c.status)
        assert int(c.status) == entro.E_INVAL
        assert torch.equal(before[0], c.cache.k_codes) and torch.equal(before[1], c.cache.v_codes)


@gpu
def test_outputs_whose_rows_share_elements_are_refused():
    c = Case(2, 2, 64, 16, torch.bfloat16, width=3)
    c.append([5, 6])
    q, x = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(11, 2, 64, dtype=torch.bfloat16, device="cuda")
    cu = torch.tensor([0, 5, 11], dtype=torch.int32).cuda()
    for out in (q[:1].expand(2, 4, 64), q[:, :1].expand(2, 4, 64)):
        with pytest.raises(ValueError, match="share"):
            c.cache.attend(q, c.table, c.lens.cuda(), slots=c.slots, out=out)
    for out in ((x, x[:1].expand(11, 2, 64)), (x[:, :1].expand(11, 2, 64), x)):
        with pytest.raises(ValueError, match="share"):
            c.cache.read(c.table, cu, 11, slots=c.slots, out=out)
    with pytest.raises(ValueError, match="two tensors"):
        c.cache.read(c.table, cu, 11, slots=c.slots, out=(x, x))


@gpu
def test_the_buffers_cannot_be_exchanged():
    # the library holds the addresses of those that it was made of
    c = Case(1, 2, 64, 16, torch.bfloat16, width=3)
    for name in ("k_codes", "v_codes", "k_scale", "v_scale", "k_tail", "v_tail"):
        with pytest.raises(AttributeError):
            setattr(c.cache, name, getattr(c.cache, name).clone())


@gpu
def test_refusals_on_the_gpu():
    c = Case(2, 2, 64, 16, torch.bfloat16, width=3)
    c.append([5, 6])
    q, lens = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device="cuda"), c.lens.cuda()
    cu = torch.tensor([0, 1, 2], dtype=torch.int32).cuda()
    x = torch.zeros(2, 2, 64, dtype=torch.bfloat16, device="cuda")
    for bad in (q.half(), q[:, :3], q[:1], q[0], q[..., :32], torch.zeros(2, 4, 68, dtype=torch.bfloat16, device="cuda")[..., 4:], q.cpu()):
        with pytest.raises(ValueError):
            c.cache.attend(bad, c.table, lens, slots=c.slots)
    for kw in (dict(lens=lens.long()), dict(lens=lens[:1]), dict(page_table=c.table.long()), dict(page_table=c.table.t()), dict(slots=c.slots[:1]),
               dict(scale=0.0), dict(scale=float("inf")), dict(out=q[:1])):
        with pytest.raises(ValueError):
            c.cache.attend(**{**dict(q=q, page_table=c.table, lens=lens, slots=c.slots), **kw})
    for kw in (dict(k=x.half()), dict(v=x[:1]), dict(k=x[:, :1]), dict(cu_seqlens=cu[:2]), dict(lens=lens.cpu())):
        with pytest.raises(ValueError):
            c.cache.append(**{**dict(k=x, v=x, cu_seqlens=cu, page_table=c.table, lens=lens, slots=c.slots), **kw})
    with pytest.raises(ValueError):
        c.cache.read(c.table, cu, 2, slots=c.slots, out=(x[:1], x))
    with pytest.raises(ValueError):
        c.cache.attend(torch.zeros(9, 4, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(9, 3, dtype=torch.int32, device="cuda"),
                       torch.zeros(9, dtype=torch.int32, device="cuda"))  # more sequences than slots
    with pytest.raises(ValueError, match="gradient"):
        c.cache.attend(q.clone().requires_grad_(), c.table, lens, slots=c.slots)
    for status in (torch.zeros(1, dtype=torch.int64, device="cuda"), torch.zeros(0, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32)):
        for call in (lambda: c.cache.attend(q, c.table, lens, slots=c.slots, status=status), lambda: c.cache.read(c.table, cu, 2, slots=c.slots, status=status),
                     lambda: c.cache.append(x, x, cu, c.table, lens, slots=c.slots, status=status)):
            with pytest.raises(ValueError):
                call()


@gpu
def test_no_pages():
    """Sequences shorter than a block need no page: a table without columns."""
    c = Case(2, 2, 64, 16, torch.bfloat16, width=1, seed=13)
    c.table = torch.zeros((2, 0), dtype=torch.int32, device="cuda")
    c.append([7, 15])
    _check_attention(c, 4)
    got, _ = c.cache.read(c.table, torch.tensor([0, 7, 22], dtype=torch.int32).cuda(), 22, slots=c.slots, status=c.status)
    assert int(c.status) == 0 and torch.equal(got.cpu(), torch.cat([c.held[0][0], c.held[1][0]]))
    x = torch.ones(2, 2, 64, dtype=torch.bfloat16, device="cuda")  # the second block fills up: there is no page for it
    c.cache.append(x, x, torch.tensor([0, 1, 2], dtype=torch.int32).cuda(), c.table, torch.tensor([8, 16], dtype=torch.int32).cuda(), slots=c.slots, status=c.status)
    assert int(c.status) == entro.E_INVAL


@gpu
def test_given_outputs_and_streams_agree_with_the_usual_call():
    """The calls that go another way in the binding (an output or a stream given) give the same bits."""
    c = Case(3, 2, 96, 32, torch.float16, width=5, seed=14)
    c.append([40, 0, 130])
    q = torch.randn(3, 8, 96, generator=c.g).to(torch.float16).cuda()
    lens, cu = c.lens.cuda(), torch.tensor([0, 40, 40, 170], dtype=torch.int32).cuda()
    want = c.cache.attend(q, c.table, lens, slots=c.slots)
    assert torch.equal(c.cache.attend(q, c.table, lens, slots=c.slots, out=torch.empty_like(q)), want)
    assert torch.equal(c.cache.attend(q, c.table, lens, slots=c.slots, stream=torch.cuda.current_stream()), want)
    k, v = c.cache.read(c.table, cu, 170, slots=c.slots)
    for a, b in zip((k, v), c.cache.read(c.table, cu, 170, slots=c.slots, out=(torch.empty_like(k), torch.empty_like(v)))):
        assert torch.equal(a, b)
    other = entro.KVCache(*(t.clone() for t in (c.cache.k_codes, c.cache.v_codes, c.cache.k_scale, c.cache.v_scale, c.cache.k_tail, c.cache.v_tail)))
    x, y, one = c.tokens(3).cuda(), c.tokens(3).cuda(), torch.arange(4, dtype=torch.int32, device="cuda")
    c.cache.append(x, y, one, c.table, lens + 1, slots=c.slots)
    other.append(x, y, one, c.table, lens + 1, slots=c.slots, stream=torch.cuda.current_stream())
    for name in ("k_codes", "v_codes", "k_scale", "v_scale", "k_tail", "v_tail"):
        a, b = getattr(c.cache, name), getattr(other, name)
        assert torch.equal(torch.nan_to_num(a.float()), torch.nan_to_num(b.float()))


@gpu
def test_streams_and_graphs():
    """Another stream; a step (append and attend) captured once and replayed over growing sequences."""
    c = Case(3, 2, 64, 16, torch.bfloat16, width=6, seed=11)
    c.append([10, 33, 47])
    q = torch.randn(3, 8, 64, generator=c.g).to(torch.bfloat16).cuda()
    want = c.cache.attend(q, c.table, c.lens.cuda(), slots=c.slots)
    lens = c.lens.cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = c.cache.attend(q, c.table, lens, slots=c.slots, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    held_k, held_v = (torch.zeros(3, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    cu = torch.arange(4, dtype=torch.int32, device="cuda")
    graph, other = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lens.add_(1)
        c.cache.append(held_k, held_v, cu, c.table, lens, slots=c.slots)
        y = c.cache.attend(q, c.table, lens, slots=c.slots)
    with torch.cuda.graph(other, pool=graph.pool()):
        z = c.cache.attend(q, c.table, lens, slots=c.slots)
    for step in range(20):
        k, v = c.tokens(3), c.tokens(3)
        held_k.copy_(k)
        held_v.copy_(v)
        graph.replay()
        got = y.clone()
        for b in range(3):
            for i, x in enumerate((k, v)):
                c.held[b][i] = torch.cat([c.held[b][i], x[b:b + 1]])
        c.lens += 1
        assert torch.equal(lens.cpu(), c.lens)
        o, mag, big = _attention(c, q.cpu(), 0.125)
        bound = mag * (2.0 ** -11 + 2.0 ** -18 + 2 * 16 * 2.0 ** -23 * big) + o.abs() * HALF_STEP[c.dtype] + 2.0 ** -25
        assert bool(((got.cpu().double() - o).abs() <= bound).all()), step
        other.replay()
        assert torch.equal(z, got)
    c.check_contents()


@gpu
def test_long_cache_offsets():
    """Pages beyond 2^31 bytes of a pool."""
    kv, dim, page = 8, 128, 128
    pages = (1 << 31) // (kv * dim * page) + 40  # 2 GB of codes is 16384 pages
    c = Case(1, kv, dim, page, torch.bfloat16, width=3, seed=12)
    big = entro.KVCache.empty(pages, kv, dim, page, slots=3, dtype=torch.bfloat16)
    c.cache, c.pages = big, pages
    c.table = torch.tensor([[pages - 1, 5, pages - 30]], dtype=torch.int32).cuda()
    c.append([300])
    _check_attention(c, 32)
    got, _ = big.read(c.table, torch.tensor([0, 300], dtype=torch.int32).cuda(), 300, slots=c.slots)
    q, s, tail = c.expect(0, 0)
    want = torch.cat([(q.float() * s[..., None, None]).to(torch.bfloat16).transpose(1, 2).flatten(0, 1), tail])
    assert torch.equal(got.cpu(), want)
