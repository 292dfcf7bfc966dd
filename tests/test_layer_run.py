"""One decoder layer from coded weights, as it would be served: prompts in two parts (products of quantized tokens,
attention over the packed prompts, the cache written and read back for the second part), then single tokens (fused
GEMVs, append, attention over the cache).

Every stage is checked against the same stage in 64 bits on the same inputs (the run's own), so each keeps its own bound:
half a step of the output's type against the sum of the magnitudes that go into it, and for the attentions the same again
for their rounded weights.  The single tokens' reference takes codes times scale from the cache itself: the reader rounds
them to 16 bits, which moves a score by up to 2^-8 of its products' magnitudes, so its values are not what the attention
over the cache sees."""
import numpy as np
import pytest
import torch

import oracle
import workloads

import huffman_decode_canonical_b200 as entro

pytestmark = pytest.mark.gpu

HEADS, KV, DIM, HIDDEN = 8, 2, 64, 512


def _layer(bits, fmt, chunk):
    """Coded projections and their dequantized weights."""
    out = {}
    for i, (name, rows, cols) in enumerate((("q", HEADS * DIM, HIDDEN), ("k", KV * DIM, HIDDEN), ("v", KV * DIM, HIDDEN), ("o", HIDDEN, HEADS * DIM))):
        w = workloads.small_tensor("t4" if bits == 8 else "laplace", rows, cols, seed=20 + i) * 3
        q, scale, zero, _ = oracle.quantize(w, bits, oracle.MODE_ASYM)
        dt = entro.upload(entro.Blob.encode(w, bits=bits, quant_mode=entro.QUANT_ASYM, fmt=fmt, lanes=32, chunk_symbols=chunk))
        out[name] = dt, (q.reshape(rows, cols).astype(np.float64) - zero) * float(scale)
    return out


def _near(got, want, magnitude, steps=2):
    h = 2.0 ** -8
    err = np.abs(got.double().cpu().numpy() - want)
    assert (err <= steps * h * magnitude + 1e-6).all(), float((err / (h * magnitude + 1e-6)).max())


def _product(layer, name, xq):
    dt, w = layer[name]
    y = dt.matmul(xq)
    x = xq.codes.cpu().numpy().astype(np.float64) * xq.scale.cpu().numpy().astype(np.float64)[:, None]
    _near(y, x @ w.T, np.abs(x @ w.T), 1)
    return y


def _attention(q, k, v):
    """Causal attention of one sequence, its last query at its last key; values and magnitudes, 64 bits."""
    n, m, g = q.shape[0], k.shape[0], HEADS // KV
    o, mag = np.zeros(q.shape), np.zeros(q.shape)
    for h in range(HEADS):
        s = q[:, h] @ k[:, h // g].T / DIM ** 0.5
        s = np.where(np.arange(m) <= np.arange(n)[:, None] + m - n, s, -np.inf)
        p = np.exp(s - s.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
        o[:, h], mag[:, h] = p @ v[:, h // g], p @ np.abs(v[:, h // g])
    return o, mag


def _held(codes, scale, tail, table, length, slot):
    """A sequence's cached tokens in 64 bits: full blocks as codes times scale, then the open block."""
    page = codes.shape[2]
    at = table[:length // page].long()
    full = (codes[at].double() * scale[at].double()[..., None, None]).transpose(1, 2).flatten(0, 1)
    return torch.cat([full, tail[slot].double().transpose(0, 1)[:length % page]]).cpu().numpy()


def _np(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("bits,fmt,chunk", [(8, entro.FORMAT_ROWS, 4096), (4, entro.FORMAT_ROWS_CO, 8192)])
def test_layer(bits, fmt, chunk):
    layer = _layer(bits, fmt, chunk)
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    batch, page = 3, 16
    cache = entro.KVCache.empty(batch * 20, KV, DIM, page, slots=batch)
    table = torch.randperm(batch * 20, generator=torch.Generator().manual_seed(1)).to(torch.int32).view(batch, 20).cuda()
    lens = torch.zeros(batch, dtype=torch.int32, device="cuda")

    def cu(lengths):
        return torch.tensor([0] + list(np.cumsum(lengths)), dtype=torch.int32).cuda()

    # the prompts, in two parts
    for part, lengths in enumerate(([70, 5, 131], [40, 90, 1])):
        x = torch.randn(sum(lengths), HIDDEN, generator=g, device="cuda").to(torch.bfloat16)
        xq = entro.quantize_tokens(x)  # shared by three projections
        q, k, v = (_product(layer, n, xq).view(sum(lengths), -1, DIM) for n in "qkv")
        lens += torch.tensor(lengths, dtype=torch.int32, device="cuda")
        cache.append(k, v, cu(lengths), table, lens, status=status)
        if part == 0:
            keys, values, cu_keys = k, v, None
        else:
            held = lens.tolist()
            cu_keys = cu(held)
            keys, values = cache.read(table, cu_keys, sum(held), status=status)
        o = entro.attention_prompt(q, keys, values, cu(lengths), cu_keys, status=status)
        ends, kends = cu(lengths).tolist(), (cu(lengths) if cu_keys is None else cu_keys).tolist()
        for b in range(batch):
            want, mag = _attention(_np(q[ends[b]:ends[b + 1]]), _np(keys[kends[b]:kends[b + 1]]), _np(values[kends[b]:kends[b + 1]]))
            _near(o[ends[b]:ends[b + 1]], want, mag)
        y = _product(layer, "o", entro.quantize_tokens(o.view(sum(lengths), -1)))
        assert y.shape == (sum(lengths), HIDDEN) and int(status) == 0

    # single tokens
    one = cu([1] * batch)
    for _ in range(20):
        x = torch.randn(batch, HIDDEN, generator=g, device="cuda").to(torch.bfloat16)
        q, k, v = (layer[n][0].decode_gemv(x, status=status).to(torch.bfloat16).view(batch, -1, DIM) for n in "qkv")
        lens += 1
        cache.append(k, v, one, table, lens, status=status)
        o = cache.attend(q, table, lens, status=status)
        held = lens.tolist()
        for b in range(batch):
            keys = _held(cache.k_codes, cache.k_scale, cache.k_tail, table[b], held[b], b)
            values = _held(cache.v_codes, cache.v_scale, cache.v_tail, table[b], held[b], b)
            want, mag = _attention(_np(q[b:b + 1]), keys, values)
            _near(o[b:b + 1], want, mag)
        y = layer["o"][0].decode_gemv(o.view(batch, -1), status=status)
        assert bool(torch.isfinite(y).all()) and int(status) == 0


def test_two_streams_at_once():
    """Each operator on two streams side by side, over and over: the same bits as alone."""
    g = torch.Generator(device="cuda")
    g.manual_seed(9)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)

    w = torch.randint(0, 256, (1000, 768), generator=g, device="cuda", dtype=torch.uint8)
    xs, q, k = [normal(n, 768) for n in (20, 100, 700)], normal(900, 8, 64), normal(900, 2, 64)
    cu = torch.tensor([0, 300, 900], dtype=torch.int32, device="cuda")
    cache = entro.KVCache.empty(40, 2, 64, 16, slots=2)
    table, lens = torch.arange(38, dtype=torch.int32, device="cuda").view(2, 19), torch.tensor([300, 290], dtype=torch.int32, device="cuda")
    cache.append(k[:590], k[10:600], torch.tensor([0, 300, 590], dtype=torch.int32, device="cuda"), table, lens)
    work = [lambda x=x: entro.matmul_i8(entro.quantize_tokens(x), w, 0.01, 100) for x in xs]
    work += [lambda: entro.attention_prompt(q, k, k, cu), lambda: cache.attend(q[:2], table, lens)]
    want = [f() for f in work]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for turn in range(30):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                n = (turn + 2 * i) % len(work)
                got.append((n, work[n]()))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[n]) for n, y in got)
