"""The operators around the coded weights between decode launches that overlap (programmatic dependent launch): every call
gives the bits that it gives with overlap off, in a run that mixes them as a served model does."""
import pytest
import torch

import huffman_decode_canonical_b200 as entro
import workloads

pytestmark = pytest.mark.gpu

HEADS, KV, DIM, BATCH = 8, 2, 64, 12


@pytest.fixture
def overlap_off():
    previous = entro.set_overlap(False)
    yield
    entro.set_overlap(previous)


def _weights():
    out = []
    for i, (kind, bits, rows, cols, chunk, fmt) in enumerate((("laplace", 4, 4096, 512, 8192, entro.FORMAT_LANES), ("t4", 8, 768, 512, 6144, entro.FORMAT_LANES),
                                                             ("laplace", 4, 512, 512, 8192, entro.FORMAT_ROWS), ("t4", 8, 512, 4096, 4096, entro.FORMAT_ROWS))):
        w = workloads.small_tensor(kind, rows, cols, seed=60 + i)
        out.append(entro.upload(entro.Blob.encode(w, bits=bits, quant_mode=entro.QUANT_ASYM, chunk_symbols=chunk, fmt=fmt, lanes=32)))
    return out


def _run(weights, x, status):
    """Prompts, then single tokens: all that was computed, in order."""
    up, qkv, o, down = weights
    res = []

    def keep(t):
        res.append(t.clone())
        return t

    page, each = 16, x.shape[0] // BATCH
    cache = entro.KVCache.empty(BATCH * 8, KV, DIM, page, slots=BATCH)
    table = torch.arange(BATCH * 8, dtype=torch.int32, device="cuda").view(BATCH, 8)
    cu = torch.arange(BATCH + 1, dtype=torch.int32, device="cuda")
    lens = torch.full((BATCH,), each, dtype=torch.int32, device="cuda")
    h = keep(qkv.matmul(x, status=status)).view(-1, HEADS + 2 * KV, DIM)  # decode, quantize, product
    q, k, v = h[:, :HEADS], h[:, HEADS:HEADS + KV], h[:, HEADS + KV:]
    cache.append(k, v, cu * each, table, lens, status=status)
    a = keep(entro.attention_prompt(q, k, v, cu * each, status=status))
    codes = up.decode_codes(status=status)  # a decode launch right behind, and a product of what it writes
    wide = torch.empty((up.rows, up.cols), dtype=torch.uint8, device="cuda")
    entro._check(entro.lib().entro_unpack_codes(codes.data_ptr(), 4, up.rows, up.cols, wide.data_ptr(), up.cols, torch.cuda.current_stream().cuda_stream), "unpack")
    xq = entro.quantize_tokens(a.view(-1, HEADS * DIM))
    big = keep(entro.matmul_i8(xq, wide, up.info["scale"], up.info["zero"], status=status))
    x = keep(down.matmul(big, status=status))
    for _ in range(20):
        t = x[:BATCH].contiguous()
        h = keep(qkv.decode_gemv(t, status=status)).to(torch.bfloat16).view(BATCH, HEADS + 2 * KV, DIM)
        lens += 1
        cache.append(h[:, HEADS:HEADS + KV], h[:, HEADS + KV:], cu, table, lens, status=status)
        a = keep(cache.attend(h[:, :HEADS], table, lens, status=status))
        y = keep(o.decode_gemv(a.view(BATCH, -1), status=status))  # a fused GEMV on what the operator before it writes
        z = keep(entro.matmul_i8(entro.quantize_tokens(y.to(torch.bfloat16)), wide, 0.01, 7, status=status))
        x = keep(down.decode_gemv(torch.tanh(z), status=status)).to(torch.bfloat16)
    return res


def test_operators_between_overlapping_decodes(overlap_off):
    weights, g = _weights(), torch.Generator(device="cuda").manual_seed(6)
    x = torch.randn(BATCH * 20, 512, generator=g, device="cuda").to(torch.bfloat16)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = _run(weights, x, status)
    torch.cuda.synchronize()
    entro.set_overlap(True)
    for _ in range(5):
        got = _run(weights, x, status)
        torch.cuda.synchronize()
        assert int(status) == 0 and len(got) == len(want)
        for i, (a, b) in enumerate(zip(got, want)):
            assert torch.equal(a, b), i
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = _run(weights, x, status)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert int(status) == 0
        for i, (a, b) in enumerate(zip(got, want)):
            assert torch.equal(a, b), i
