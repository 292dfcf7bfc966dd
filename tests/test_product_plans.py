"""The 8-bit product's two kernels where a call keeps them busy: CTA pairs that walk several tiles each (both accumulators,
the ring of copies carried on from tile to tile), and clusters that share a tile's columns in every split.  Each test first
asks which kernel its sizes go to (`test_product_plan`), so that a later change of the cost model cannot empty it.

Products are compared with exact sums (64-bit floats hold them: below 2^53) under the bound of test_product.py."""
import pytest
import torch

import huffman_decode_canonical_b200 as entro
from test_product import _close, _rng, _tokens

gpu = pytest.mark.gpu

# (tokens, rows, cols), at least three tiles for each of 74 pairs; remainders in all three, fewer and more steps than the ring has
WIDE = [(4100, 5000, 136), (2100, 9000, 1100), (8200, 1800, 392), (515, 30001, 640)]
# (tokens, rows, cols), split, tile
NARROW = [((24, 2048, 2048), 8, 32), ((17, 1000, 8000), 8, 32), ((80, 2000, 4096), 8, 80), ((144, 2047, 16384), 8, 144), ((250, 1000, 16384), 8, 256),
          ((40, 4000, 4096), 4, 48), ((128, 4090, 14336), 4, 128), ((24, 8192, 4096), 2, 32), ((16, 8200, 5000), 2, 16), ((24, 14300, 4096), 1, 32),
          ((5, 14336, 4112), 1, 16)]


def _sms():
    return torch.cuda.get_device_properties(0).multi_processor_count if torch.cuda.is_available() else 148


def _wide(tokens, rows, cols):
    plan, pairs = entro.test_product_plan(tokens, rows, cols, _sms()), _sms() // 2
    return plan["wide"] == 1 and plan["row_tiles"] * plan["token_tiles"] >= 3 * pairs


def _narrow(tokens, rows, cols, split, tile):
    plan = entro.test_product_plan(tokens, rows, cols, _sms())
    return plan["wide"] == 0 and plan["split"] == split and plan["tile_tokens"] == tile


def test_plans():
    for case in WIDE:
        assert _wide(*case), case
    for case, split, tile in NARROW:
        assert _narrow(*case, split, tile), (case, entro.test_product_plan(*case, _sms()))
    for bad in ((0, 1, 1), (1, 0, 1), (1, 1, 0), (1, 1, 65537), (2 ** 24 + 1, 1, 1), (1, 2 ** 30 + 1, 1)):
        with pytest.raises(entro.EntroError):
            entro.test_product_plan(*bad)
    with pytest.raises(entro.EntroError):
        entro.test_product_plan(1, 1, 1, 1)


def _inputs(tokens, rows, cols, weights="u8"):
    rng = _rng(tokens, rows, cols, 5)
    g = torch.Generator(device="cuda").manual_seed(tokens + rows)
    low, high, dtype = (0, 256, torch.uint8) if weights == "u8" else (-128, 128, torch.int8)
    w = torch.randint(low, high, (rows, (cols + 15) // 16 * 16), generator=g, device="cuda", dtype=torch.int16).to(dtype)[:, :cols]
    scale = torch.exp(torch.randn(rows, generator=g, device="cuda")) * 1e-3
    zero = torch.randint(low, high, (rows,), generator=g, device="cuda", dtype=torch.int32)
    return _tokens(rng, tokens, cols, torch.bfloat16).cuda(), w, scale, zero


def _expect(xq, w, scale, zero):
    x, out = xq.codes.double(), []
    for part, s, z in zip(w.split(2048), scale.split(2048), zero.split(2048)):
        out.append(x @ (part.double() - z[:, None].double()).t() * xq.scale.double()[:, None] * s.double())
    return torch.cat(out, 1).cpu().numpy()


@gpu
@pytest.mark.parametrize("weights", ["u8", "s8"])
@pytest.mark.parametrize("tokens,rows,cols", WIDE)
def test_pairs_with_several_tiles(tokens, rows, cols, weights):
    assert _wide(tokens, rows, cols)
    x, w, scale, zero = _inputs(tokens, rows, cols, weights)
    xq, status = entro.quantize_tokens(x), torch.zeros(1, dtype=torch.int32, device="cuda")
    want = _expect(xq, w, scale, zero)
    for dtype in (torch.float32, torch.bfloat16):
        y = entro.matmul_i8(xq, w, scale, zero, out_dtype=dtype, status=status)
        _close(y, want)
        for _ in range(3):
            assert torch.equal(y, entro.matmul_i8(xq, w, scale, zero, out_dtype=dtype))
    assert int(status) == 0
    # an output inside a larger buffer: nothing around it changes
    big = torch.full((tokens + 2, rows + 7), 7.0, device="cuda")
    out = entro.matmul_i8(xq, w, scale, zero, out=big[1:-1, 3:3 + rows])
    _close(out, want)
    out.fill_(7.0)
    assert bool((big == 7.0).all())


@gpu
@pytest.mark.parametrize("weights", ["u8", "s8"])
@pytest.mark.parametrize("case,split,tile", NARROW)
def test_clusters_that_share_columns(case, split, tile, weights):
    assert _narrow(*case, split, tile)
    tokens, rows, cols = case
    x, w, scale, zero = _inputs(*case, weights)
    xq, status = entro.quantize_tokens(x), torch.zeros(1, dtype=torch.int32, device="cuda")
    want = _expect(xq, w, scale, zero)
    for dtype in (torch.float32, torch.float16, torch.bfloat16):
        y = entro.matmul_i8(xq, w, scale, zero, out_dtype=dtype, status=status)
        _close(y, want)
        for _ in range(3):
            assert torch.equal(y, entro.matmul_i8(xq, w, scale, zero, out_dtype=dtype))
    assert int(status) == 0
    big = torch.full((tokens + 2, rows + 7), 7.0, device="cuda")
    out = entro.matmul_i8(xq, w, scale, zero, out=big[1:-1, 3:3 + rows])
    _close(out, want)
    out.fill_(7.0)
    assert bool((big == 7.0).all())
    # zero points outside the codes' range: differences in 64 bits
    far = zero + (1 << 24)
    _close(entro.matmul_i8(xq, w, scale, far, out_dtype=torch.float32), _expect(xq, w, scale, far))


def _replayed(case):
    x, w, scale, zero = _inputs(*case)
    want = entro.matmul_i8(entro.quantize_tokens(x), w, scale, zero)
    held, graph = torch.zeros_like(x), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = entro.matmul_i8(entro.quantize_tokens(held), w, scale, zero)
    for _ in range(3):
        held.copy_(x)
        graph.replay()
        assert torch.equal(y, want)
        held.zero_()
        graph.replay()
        assert not y.any()


@gpu
@pytest.mark.parametrize("i", [0, 5, 7, 9])
def test_clusters_captured(i):
    assert _narrow(*NARROW[i][0], *NARROW[i][1:])
    _replayed(NARROW[i][0])


@gpu
def test_pairs_captured():
    assert _wide(*WIDE[1])
    _replayed(WIDE[1])


@gpu
def test_two_streams_at_once():
    """Both kernels in every split side by side on two streams: the same bits as alone."""
    cases = [NARROW[i][0] for i in (0, 5, 7, 9)] + [WIDE[0], WIDE[3]]
    work = []
    for case in cases:
        x, w, scale, zero = _inputs(*case)
        work.append(lambda x=x, w=w, scale=scale, zero=zero: entro.matmul_i8(entro.quantize_tokens(x), w, scale, zero))
    want = [f() for f in work]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for turn in range(24):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                n = (turn + 3 * i) % len(work)
                got.append((n, work[n]()))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[n]) for n, y in got)


@gpu
@pytest.mark.parametrize("case", [NARROW[0][0], NARROW[5][0], NARROW[9][0], WIDE[0]])
def test_waits_give_up(case):
    """Bytes that never arrive end in a status, across a cluster's barriers too, and the next call is right."""
    x, w, scale, zero = _inputs(*case)
    xq, status = entro.quantize_tokens(x), torch.zeros(1, dtype=torch.int32, device="cuda")
    want = entro.matmul_i8(xq, w, scale, zero)
    torch.cuda.synchronize()
    entro.test_stall_tables(16)
    try:
        entro.matmul_i8(xq, w, scale, zero, status=status)
        torch.cuda.synchronize()
    finally:
        entro.test_stall_tables(0)
    assert int(status) == entro.E_TIMEOUT
    status.zero_()
    assert torch.equal(entro.matmul_i8(xq, w, scale, zero, status=status), want) and int(status) == 0
