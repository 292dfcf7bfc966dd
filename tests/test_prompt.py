"""Causal attention over packed prompts against a 64-bit softmax.

Bound for an output o = sum p v: the weights are rounded to the type (half a step h of each: h sum p |v|); scores come from
32-bit sums of head_dim products, off by a few 2^-23 of the sum of the products' magnitudes (16 x 2^-23: a rounding per MMA
and the scale's), which moves a weight by that much of itself, in numerator and sum; the 32-bit sums over the keys take a
rounding per 16 keys and 64 more; the rest is below 2^-18 of sum p |v|; the output is rounded by h |o|."""
import pathlib
import subprocess
import sys

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


def _inputs(g, tokens, keys, heads, kv, dim, dtype):
    return [torch.randn(t, h, dim, generator=g).to(dtype) for t, h in ((tokens, heads), (keys, kv), (keys, kv))]


def _cu(lengths):
    return torch.tensor([0] + list(np.cumsum(lengths)), dtype=torch.int32)


def _reference(q, k, v, cu, cu_k, scale):
    """(o, bound's parts) in 64 bits; hidden keys are left out, whatever they hold"""
    heads, kv = q.shape[1], k.shape[1]
    o, mag = torch.zeros(q.shape, dtype=torch.float64), torch.zeros(q.shape, dtype=torch.float64)
    big = torch.zeros(q.shape[:2] + (1,), dtype=torch.float64)
    for b in range(len(cu) - 1):
        a, e, c, d = int(cu[b]), int(cu[b + 1]), int(cu_k[b]), int(cu_k[b + 1])
        if e == a or d == c:
            continue
        qq = q[a:e].double().view(e - a, kv, heads // kv, -1)
        kk, vv = k[c:d].double(), v[c:d].double()
        seen = torch.arange(d - c) <= (torch.arange(e - a) + (d - c) - (e - a))[:, None]
        s = torch.einsum("ihgd,jhd->hgij", qq, kk) * scale
        p = torch.softmax(s.masked_fill(~seen, float("-inf")), 3)
        p = torch.where(seen, p, torch.zeros(1, dtype=torch.float64))  # (a row that sees nothing is all NaN)
        def put(vals):
            return torch.einsum("hgij,jhd->ihgd", p, vals).reshape(e - a, heads, -1)
        if torch.isfinite(vv).all():
            o[a:e], mag[a:e] = put(vv), put(vv.abs())
        else:  # row by row over what is seen
            for i in range(e - a):
                n = max(0, i + (d - c) - (e - a) + 1)
                w = p[:, :, i, :n]
                o[a + i] = torch.einsum("hgj,jhd->hgd", w, vv[:n]).reshape(heads, -1)
                mag[a + i] = torch.einsum("hgj,jhd->hgd", w, vv[:n].abs()).reshape(heads, -1)
        m = torch.einsum("ihgd,jhd->hgij", qq.abs(), kk.abs()) * scale
        big[a:e] = torch.where(seen, m, torch.zeros(1, dtype=torch.float64)).amax(3).permute(2, 0, 1).reshape(e - a, heads, 1)
    return o, mag, big


def _check(q, k, v, cu, cu_k=None, scale=None, got=None):
    dtype = q.dtype
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dev = [t.cuda() for t in (q, k, v)]
    if got is None:
        got = entro.attention_prompt(*dev, cu.cuda(), None if cu_k is None else cu_k.cuda(), scale=scale, status=status)
        assert int(status) == 0
    o, mag, big = _reference(q, k, v, cu, cu if cu_k is None else cu_k, q.shape[2] ** -0.5 if scale is None else scale)
    h, keys = HALF_STEP[dtype], k.shape[0]
    bound = mag * (h + 2.0 ** -18 + 2 * 16 * 2.0 ** -23 * big + (keys / 16 + 64) * 2.0 ** -23) + o.abs() * h + 2.0 ** -25
    end = int(cu[-1])
    x, o, bound = got.cpu().double()[:end], o[:end], bound[:end]
    nan = torch.isnan(o)
    assert torch.equal(torch.isnan(x), nan)
    inf = torch.isinf(o)
    assert torch.equal(x[inf], o[inf])
    err, ok = (x - o).abs(), ~nan & ~inf
    assert bool((err <= bound)[ok].all()), (float((err / bound)[ok].max()), (err > bound).nonzero()[:4])
    return got


# ------------------------------------------------------------------ refusals (no GPU needed)

def test_refusals_of_the_binding():
    q, k, cu = torch.zeros(6, 4, 64, dtype=torch.bfloat16), torch.zeros(6, 2, 64, dtype=torch.bfloat16), torch.tensor([0, 6], dtype=torch.int32)
    wide = torch.zeros(6, 4, 72, dtype=torch.bfloat16)
    for bad in (dict(q=q.float()), dict(q=q[0]), dict(q=q[..., :32]), dict(q=q[:, :3]), dict(q=wide[..., 4:68]), dict(k=k.half()), dict(v=k[:5]),
                dict(k=k[:5], v=k[:5]), dict(k=k[:, :1].expand(6, 2, 64)), dict(v=k[:1].expand(6, 2, 64)), dict(cu_seqlens=cu.long()), dict(cu_seqlens=cu[None]),
                dict(cu_seqlens=cu[:0]), dict(cu_keys=torch.tensor([0, 3, 6], dtype=torch.int32)), dict(out=q[:5]), dict(out=k), dict(scale=0.0), dict(scale=-1.0),
                dict(scale=float("nan"))):
        with pytest.raises(ValueError):
            entro.attention_prompt(**{**dict(q=q, k=k, v=k, cu_seqlens=cu), **bad})
    with pytest.raises(ValueError, match="CUDA"):
        entro.attention_prompt(q, k, k, cu)


@pytest.mark.parametrize("size,stride", [((6, 4, 64), (256, 0, 1)), ((6, 4, 64), (0, 64, 1)), ((6, 4, 64), (192, 64, 1)), ((6, 4, 64), (64, 64, 1)),
                                         ((6, 4, 64), (56, 448, 1)), ((6, 4, 64), (64, 320, 1))])
def test_outputs_whose_rows_share_elements_are_refused(size, stride):
    q, cu = torch.zeros(6, 4, 64, dtype=torch.bfloat16), torch.tensor([0, 6], dtype=torch.int32)
    out = torch.as_strided(torch.zeros(4096, dtype=torch.bfloat16), size, stride)
    with pytest.raises(ValueError, match="share"):
        entro.attention_prompt(q, q, q, cu, out=out)
    p = 4096
    assert entro.lib().entro_attention_prompt(entro.BF16, 64, p, 256, 64, 4, 6, p, 256, 64, p, 256, 64, 4, 6, p, None, 1, 0.1, p, stride[0], stride[1],
                                              None, None) == entro.E_INVAL


@pytest.mark.parametrize("stride", [(256, 64, 1), (64, 384, 1), (264, 64, 1), (64, 392, 1), (512, 128, 1)])
def test_outputs_with_separate_rows_are_taken(stride):
    # as far as the refusal of CPU tensors
    q, cu = torch.zeros(6, 4, 64, dtype=torch.bfloat16), torch.tensor([0, 6], dtype=torch.int32)
    out = torch.zeros(4096, dtype=torch.bfloat16).as_strided((6, 4, 64), stride)
    with pytest.raises(ValueError, match="CUDA"):
        entro.attention_prompt(q, q, q, cu, out=out)


def test_refusals_of_the_library():
    lib, p = entro.lib(), 4096  # any address: argument errors come before it is used
    good = dict(type=entro.BF16, dim=64, q=p, qt=256, qh=64, heads=4, tokens=8, k=p, kt=128, kh=64, v=p, vt=128, vh=64, kv=2, keys=8, cu=p, cuk=None,
                batch=1, scale=0.1, out=p, ot=256, oh=64)

    def call(**kw):
        return lib.entro_attention_prompt(*{**good, **kw}.values(), None, None)

    for kw in (dict(type=entro.F32), dict(dim=80), dict(heads=3), dict(kv=0), dict(tokens=-1), dict(keys=-1), dict(batch=-1), dict(scale=0.0),
               dict(scale=float("inf")), dict(q=None), dict(k=None), dict(v=None), dict(out=None), dict(cu=None), dict(q=p + 2), dict(k=p + 8), dict(qt=100),
               dict(kh=4), dict(vt=0), dict(kt=-128), dict(ot=4), dict(out=p + 2), dict(keys=9)):
        assert call(**kw) == entro.E_INVAL, kw
    assert call(tokens=2 ** 31 - 1, keys=2 ** 31 - 1) == entro.E_LIMIT
    assert call(tokens=0, keys=0, q=None) == entro.OK and call(batch=0, q=None) == entro.OK


# ------------------------------------------------------------------ values

@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dim,heads,kv", [(64, 2, 2), (96, 3, 1), (128, 4, 2)])
@pytest.mark.parametrize("lengths", [[1], [2, 1, 1, 3], [127], [128], [129], [255, 256, 257], [0, 5, 0, 0, 300, 0], [1000, 17, 640]])
def test_packed_prompts(lengths, dim, heads, kv, dtype):
    g = _gen(sum(lengths), len(lengths), dim)
    q, k, v = _inputs(g, sum(lengths), sum(lengths), heads, kv, dim, dtype)
    a = _check(q, k, v, _cu(lengths))
    again = entro.attention_prompt(q.cuda(), k.cuda(), v.cuda(), _cu(lengths).cuda())
    assert torch.equal(a, again)


@gpu
@pytest.mark.parametrize("dim", [64, 96, 128])
@pytest.mark.parametrize("queries,keys", [([1], [1000]), ([1, 1, 5], [128, 129, 5]), ([100], [700]), ([300, 2, 130], [301, 400, 1000]), ([256], [383]), ([200], [326]),
                                          ([5, 300, 140, 3], [2, 40, 139, 0])])
def test_continued_prompts(queries, keys, dim):
    """Queries behind a context, and ones that see less than themselves: the first of them see nothing and get 0."""
    g = _gen(sum(queries), sum(keys), dim)
    q, k, v = _inputs(g, sum(queries), sum(keys), 4, 2, dim, torch.bfloat16)
    got = _check(q, k, v, _cu(queries), _cu(keys)).cpu()
    at = 0
    for n, m in zip(queries, keys):
        assert bool((got[at:at + max(0, n - m)] == 0).all())
        at += n


@gpu
@pytest.mark.parametrize("heads,kv", [(32, 1), (5, 5), (24, 3)])
def test_head_layouts(heads, kv):
    g = _gen(heads, kv)
    q, k, v = _inputs(g, 333, 333, heads, kv, 64, torch.float16)
    _check(q, k, v, _cu([200, 133]), scale=0.25)


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_growing_and_sharp_scores(dtype):
    """The row maximum rises again and again over the key tiles (and falls), by a little and by far; one key takes all."""
    g = _gen(7)
    n = 1500
    q, k, v = _inputs(g, n, n, 3, 1, 64, dtype)
    q = q.abs() + 0.1
    ramp = torch.linspace(0.02, 6, n)[:, None, None]
    _check(q.to(dtype), (k.abs() * ramp).to(dtype), v, _cu([n]))
    _check(q.to(dtype), (k.abs() * ramp.flip(0)).to(dtype), v, _cu([n]))
    _check(q.to(dtype), (k.abs() * torch.where(torch.arange(n)[:, None, None] % 300 == 299, 20.0, 0.1)).to(dtype), v, _cu([n]))
    _check((q * 0).to(dtype), k, v, _cu([n]))


@gpu
def test_long_prompt():
    g = _gen(8)
    q, k, v = _inputs(g, 6000, 6000, 2, 1, 128, torch.bfloat16)
    _check(q, k, v, _cu([6000]))


# ------------------------------------------------------------------ layouts

@gpu
@pytest.mark.parametrize("dim", [64, 96, 128])
def test_slices_of_a_projection(dim):
    """q, k and v as one projection's output holds them, the output inside a larger buffer; transposed heads."""
    g = _gen(9, dim)
    heads, kv, n = 4, 2, 300
    qkv = torch.randn(n, heads + 2 * kv, dim, generator=g).to(torch.bfloat16).cuda()
    q, k, v = qkv[:, :heads], qkv[:, heads:heads + kv], qkv[:, heads + kv:]
    cu = _cu([170, 130])
    big = torch.full((n, heads + 2, dim), 7.0, dtype=torch.bfloat16, device="cuda")
    got = entro.attention_prompt(q, k, v, cu.cuda(), out=big[:, 1:-1])
    _check(q.cpu(), k.cpu(), v.cpu(), cu, got=got)
    assert bool((big[:, 0] == 7).all()) and bool((big[:, -1] == 7).all())
    by_head = [t.transpose(0, 1).contiguous().transpose(0, 1) for t in (q, k, v)]
    assert torch.equal(entro.attention_prompt(*by_head, cu.cuda()), got)
    one = entro.attention_prompt(q[:, :2], k[:, :1], v[:, :1], cu.cuda())
    assert torch.equal(one, got[:, :2])


@gpu
def test_rows_of_no_sequence():
    """Padding before, between and behind the sequences: left as it is, and its NaN reach nobody."""
    g = _gen(10)
    q, k, v = _inputs(g, 500, 500, 4, 4, 64, torch.bfloat16)
    cu = torch.tensor([0, 60, 400], dtype=torch.int32)
    for t in (q, k, v):
        t[400:] = float("nan")
    out = torch.full((500, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    got = entro.attention_prompt(q.cuda(), k.cuda(), v.cuda(), cu.cuda(), out=out)
    assert bool((got[400:] == 7).all())
    assert not bool(torch.isnan(got).any())
    _check(q[:400], k[:400], v[:400], cu, got=got[:400])


# Few queries over many keys: a cluster of CTAs shares a block's keys (from 1024 keys a sequence on, up to eight CTAs).
@gpu
@pytest.mark.parametrize("dim", [64, 96, 128])
@pytest.mark.parametrize("queries,keys", [([1], [1024]), ([1], [4096]), ([2], [4097]), ([40], [5003]), ([128], [2048]), ([129], [3001]), ([300], [4500]),
                                          ([256], [4160]), ([130, 0, 7], [2100, 5000, 3000]), ([1500], [1500]), ([1300], [1200]), ([3, 5], [8, 9000])])
def test_keys_shared_by_a_cluster(queries, keys, dim):
    g = _gen(21, len(queries), keys[0], dim)
    q, k, v = _inputs(g, sum(queries), sum(keys), 2, 1, dim, torch.float16 if sum(queries) % 2 else torch.bfloat16)
    got = _check(q, k, v, _cu(queries), _cu(keys))
    for _ in range(3):
        assert torch.equal(got, entro.attention_prompt(q.cuda(), k.cuda(), v.cuda(), _cu(queries).cuda(), _cu(keys).cuda()))


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_sharp_scores_in_shared_keys(dtype):
    # the largest score lies in one part, by far; each part in turn
    g = _gen(22)
    q, k, v = _inputs(g, 70, 4200, 4, 2, 128, dtype)
    for at in (0, 600, 1100, 2047, 2048, 3000, 3600, 4100):
        w = k.clone()
        w[at] = 8 * q[35, 0]
        _check(q, w, v, _cu([70]), _cu([4200]))


@gpu
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_hidden_values_in_shared_keys(value):
    g = _gen(23)
    q, k, v = _inputs(g, 300, 4400, 2, 1, 96, torch.bfloat16)
    plain = _check(q, k, v, _cu([300]), _cu([4400]))
    for at in (4100, 4101, 4228, 4399):
        w = v.clone()
        w[at, 0, 3] = value
        got = _check(q, k, w, _cu([300]), _cu([4400]))
        assert bool(torch.isfinite(got[:at - 4100]).all()) and bool(torch.isfinite(got[:, :, 4:]).all())
        w = k.clone()
        w[at, 0, 3] = value
        got = entro.attention_prompt(q.cuda(), w.cuda(), v.cuda(), _cu([300]).cuda(), _cu([4400]).cuda())
        assert torch.equal(got[:at - 4100], plain[:at - 4100])
    # bad offsets: reported, and the other sequence's rows are right
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full_like(q, 7).cuda()
    cu, cu_k = torch.tensor([0, 100, 301], dtype=torch.int32), torch.tensor([0, 4100, 4400], dtype=torch.int32)
    entro.attention_prompt(q.cuda(), k.cuda(), v.cuda(), cu.cuda(), cu_k.cuda(), out=out, status=status)
    assert int(status) == entro.E_INVAL and bool((out[100:] == 7).all())
    _check(q[:100], k[:4100], v[:4100], _cu([100]), _cu([4100]), got=out[:100])


_FIRST_CALL = """
import torch, huffman_decode_canonical_b200 as entro
g = torch.Generator(device="cuda").manual_seed(1)
q, k, v = (torch.randn(t, h, 64, generator=g, device="cuda").half() for t, h in ((40, 4), (5000, 2), (5000, 2)))
cu, cu_k = torch.tensor([0, 40], dtype=torch.int32, device="cuda"), torch.tensor([0, 5000], dtype=torch.int32, device="cuda")
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    y = entro.attention_prompt(q, k, v, cu, cu_k)
graph.replay()
first = y.clone()
cu_k[1] = 3000  # the table of a replay is the one of its time
graph.replay()
torch.cuda.synchronize()
assert torch.equal(first, entro.attention_prompt(q, k, v, cu, torch.tensor([0, 5000], dtype=torch.int32, device="cuda")))
seen = entro.attention_prompt(q, k[:3000], v[:3000], cu, cu_k).double()
assert (y.double() - seen).abs().max() <= 2.0 ** -9
a, b, outs = torch.cuda.Stream(), torch.cuda.Stream(), []
torch.cuda.synchronize()
for _ in range(20):
    for s in (a, b):
        outs.append(entro.attention_prompt(q, k, v, cu, cu_k, stream=s))
torch.cuda.synchronize()
assert all(torch.equal(o, y) for o in outs)
print("good")
"""


@gpu
def test_shared_keys_captured_first_and_on_two_streams():
    """A process whose first call is captured; then two streams at once.  Between the two cuts of the same sums: each side's
    weights are rounded to fp16 (2^-11 of sum p |v|, which is near 0.8 and below 1) and its output (below 2^-2: 2^-14);
    2 (2^-11 + 2^-14) is below 2^-9, with room for the 32-bit sums."""
    done = subprocess.run([sys.executable, "-c", _FIRST_CALL], cwd=pathlib.Path(__file__).resolve().parents[1], capture_output=True, text=True, timeout=120)
    assert done.returncode == 0 and done.stdout.strip() == "good", done.stderr[-2000:]


@gpu
def test_wait_gives_up_with_shared_keys():
    g = _gen(24)
    q, k, v = _inputs(g, 50, 5000, 2, 1, 64, torch.bfloat16)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    entro.test_stall_tables(16)
    try:
        entro.attention_prompt(q.cuda(), k.cuda(), v.cuda(), _cu([50]).cuda(), _cu([5000]).cuda(), status=status)
        torch.cuda.synchronize()
    finally:
        entro.test_stall_tables(0)
    assert int(status) == entro.E_TIMEOUT
    _check(q, k, v, _cu([50]), _cu([5000]))


@gpu
def test_batch_does_not_matter():
    g = _gen(11)
    lengths = [300, 31, 700]
    q, k, v = (t.cuda() for t in _inputs(g, sum(lengths), sum(lengths), 2, 2, 128, torch.float16))
    got = entro.attention_prompt(q, k, v, _cu(lengths).cuda())
    at = 0
    for n in lengths:
        alone = entro.attention_prompt(*(t[at:at + n].contiguous() for t in (q, k, v)), _cu([n]).cuda())
        assert torch.equal(alone, got[at:at + n])
        at += n


# ------------------------------------------------------------------ what the mask hides

@gpu
@pytest.mark.parametrize("dim", [64, 96, 128])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_hidden_values_do_not_count(dim, value):
    """Infinities and NaN in values: rows before them are untouched, rows from them on have them, other sequences not."""
    g = _gen(12, dim)
    lengths, heads, kv = [200, 90, 300], 2, 1
    q, k, v = _inputs(g, sum(lengths), sum(lengths), heads, kv, dim, torch.bfloat16)
    plain = entro.attention_prompt(q.cuda(), k.cuda(), v.cuda(), _cu(lengths).cuda())
    for at in (0, 150, 199, 200, 289, 290, 589):
        w = v.clone()
        w[at, 0, 3] = value
        got = _check(q, k, w, _cu(lengths))
        first = sum(lengths[:next(i for i in range(1, 4) if at < sum(lengths[:i])) - 1])
        assert torch.equal(got[:first], plain[:first])
        assert bool(torch.isfinite(got[first:at]).all())
        assert bool(torch.isfinite(got[at:, :, 4:]).all())


@gpu
def test_hidden_keys_do_not_count():
    g = _gen(13)
    lengths = [130, 260]
    q, k, v = _inputs(g, 390, 390, 2, 2, 64, torch.float16)
    plain = entro.attention_prompt(q.cuda(), k.cuda(), v.cuda(), _cu(lengths).cuda())
    for at in (129, 130, 300, 389):
        w = k.clone()
        w[at, 1] = float("nan")
        got = entro.attention_prompt(q.cuda(), w.cuda(), v.cuda(), _cu(lengths).cuda())
        end = 130 if at < 130 else 390
        keep = torch.ones(390, 2, dtype=torch.bool)
        keep[at:end, 1] = False
        assert torch.equal(got.cpu()[keep], plain.cpu()[keep])
        assert bool(torch.isnan(got.cpu()[at:end, 1]).all())
    q[50, 0, 0] = float("nan")
    got = entro.attention_prompt(q.cuda(), k.cuda(), v.cuda(), _cu(lengths).cuda()).cpu()
    assert bool(torch.isnan(got[50, 0]).all()) and int(torch.isnan(got).any(2).sum()) == 1


# ------------------------------------------------------------------ calls

@gpu
def test_bad_offsets_are_reported():
    g = _gen(14)
    q, k, v = (t.cuda() for t in _inputs(g, 100, 100, 2, 2, 64, torch.bfloat16))
    for cu, whole in (([0, 40, 30, 100], [0, 2]), ([-5, 40, 100], [1]), ([0, 40, 101], [0]), ([0, 2 ** 31 - 1, 100], []), ([7, 7, 2 ** 31 - 1], [])):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = torch.full((100, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        entro.attention_prompt(q, k, v, torch.tensor(cu, dtype=torch.int32).cuda(), out=out, status=status)
        assert int(status) == entro.E_INVAL
        touched = torch.zeros(100, dtype=torch.bool)
        for b in whole:
            touched[cu[b]:cu[b + 1]] = True
        assert bool((out.cpu()[~touched] == 7).all()) and not bool((out.cpu()[touched] == 7).all(2).any())


@gpu
def test_empty_calls():
    e = torch.zeros(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    assert entro.attention_prompt(e, e, e, torch.zeros(1, dtype=torch.int32, device="cuda")).shape == (0, 2, 64)
    q = torch.ones(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    got = entro.attention_prompt(q, e, e, _cu([3]).cuda(), _cu([0]).cuda())
    assert bool((got == 0).all())


@gpu
def test_streams_and_graphs():
    g = _gen(15)
    lengths = [150, 450]
    q, k, v = (t.cuda() for t in _inputs(g, 600, 600, 4, 2, 96, torch.bfloat16))
    cu = _cu(lengths).cuda()
    want = entro.attention_prompt(q, k, v, cu)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = entro.attention_prompt(q, k, v, cu, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    held, held_cu = torch.zeros_like(q), torch.zeros_like(cu)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = entro.attention_prompt(held, k, v, held_cu)
    held.copy_(q)
    held_cu.copy_(cu)  # lengths are read at replay
    graph.replay()
    assert torch.equal(y, want)
    held_cu.copy_(_cu([600, 0]))
    graph.replay()
    assert torch.equal(y, entro.attention_prompt(q, k, v, _cu([600, 0]).cuda()))


@gpu
def test_wait_gives_up():
    """The bounded waits: bytes that never arrive end in a status, and the next call is right."""
    g = _gen(16)
    q, k, v = _inputs(g, 100, 100, 2, 2, 64, torch.bfloat16)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    entro.test_stall_tables(16)
    try:
        entro.attention_prompt(q.cuda(), k.cuda(), v.cuda(), _cu([100]).cuda(), status=status)
        torch.cuda.synchronize()
    finally:
        entro.test_stall_tables(0)
    assert int(status) == entro.E_TIMEOUT
    _check(q, k, v, _cu([100]))


@gpu
def test_gradients_are_refused():
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="gradient"):
        entro.attention_prompt(q.clone().requires_grad_(), q, q, _cu([4]).cuda())
