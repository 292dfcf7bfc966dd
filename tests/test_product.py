"""Products of quantized tokens and 8-bit codes (quantize_tokens, matmul_i8, DeviceTensor.matmul).

Codes are compared exactly: 127 x / max|x| is a quotient of short whole numbers, so its 64-bit quotient rounds to the
same whole number as the true one.  Products are compared with the exact integer sums times the scales in 64 bits: three
32-bit roundings (the sum, the product of the scales, their product) of at most 2^-24 each, and half a step of the output
type."""
import numpy as np
import pytest
import torch

import oracle
import workloads

import huffman_decode_canonical_b200 as entro

gpu = pytest.mark.gpu


def _rng(*key):
    return np.random.default_rng([17, *key])


def _tokens(rng, tokens, cols, dtype):
    x = torch.from_numpy(rng.standard_normal((tokens, cols)).astype(np.float32) * np.exp(rng.uniform(-3, 3, (tokens, 1)).astype(np.float32)))
    return x.to(dtype)


def _codes64(x):
    """(codes, scale) by definition, in 64 bits"""
    x = x.double()
    a = x.abs().amax(1, keepdim=True)
    ok = torch.isfinite(x).all(1, keepdim=True)
    q = torch.where(ok & (a > 0), torch.round(x * 127 / a), torch.zeros_like(x))
    return q, torch.where(ok, a / 127, torch.full_like(a, float("nan")))[:, 0]


def _expect(xq, w, w_scale, w_zero):
    """The product's definition on the tokens' codes, exactly in 64-bit whole numbers, then 64-bit scales"""
    c = w.cpu().numpy().astype(np.int64)
    if w_zero is not None:
        c = c - (w_zero.cpu().numpy().astype(np.int64)[:, None] if torch.is_tensor(w_zero) else w_zero)
    # 64-bit floats hold these sums exactly (below 2^53)
    acc = xq.codes.cpu().numpy().astype(np.float64) @ c.T.astype(np.float64)
    ws = w_scale.cpu().numpy().astype(np.float64) if torch.is_tensor(w_scale) else float(np.float32(w_scale))
    return acc * xq.scale.cpu().numpy().astype(np.float64)[:, None] * ws


def _close(y, want):
    half = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}[y.dtype]
    got, bound = y.cpu().double().numpy(), np.abs(want) * (3.01 * 2.0 ** -24 + half)
    if y.dtype == torch.float16:
        bound = bound + 2.0 ** -25  # half a step of its smallest numbers
    assert np.array_equal(np.isnan(got), np.isnan(want))
    bad = np.abs(got - want) > bound
    assert not bad[~np.isnan(want)].any(), (np.argwhere(bad)[:5], got[bad][:5], want[bad][:5])


# ------------------------------------------------------------------ refusals (no GPU needed)

def test_refusals_of_the_binding():
    x = torch.zeros(4, 32, dtype=torch.bfloat16)
    for bad in (x.float(), x[0], x.t(), x[:, :0]):
        with pytest.raises(ValueError):
            entro.quantize_tokens(bad)
    with pytest.raises(ValueError, match="CUDA"):
        entro.quantize_tokens(x)
    q = entro.QuantTokens(torch.zeros(4, 32, dtype=torch.int8), torch.zeros(4), torch.zeros(4, dtype=torch.int32))
    w = torch.zeros(8, 32, dtype=torch.uint8)
    for bad_w in (w.float(), w[0], w.t(), w[:, :31]):
        with pytest.raises(ValueError):
            entro.matmul_i8(q, bad_w, 1.0)
    for scale in (torch.ones(7), torch.ones(8, dtype=torch.float64), torch.ones(16)[::2]):
        with pytest.raises(ValueError):
            entro.matmul_i8(q, w, scale)
    for zero in (torch.ones(8), torch.ones(7, dtype=torch.int32), 2 ** 31):
        with pytest.raises(ValueError):
            entro.matmul_i8(q, w, 1.0, zero)
    with pytest.raises(ValueError):
        entro.matmul_i8(q._replace(scale=torch.zeros(3)), w, 1.0)
    with pytest.raises(ValueError):
        entro.matmul_i8(q._replace(sum=torch.zeros(4)), w, 1.0)
    with pytest.raises(ValueError, match="CUDA"):
        entro.matmul_i8(q, w, 1.0)


def test_refusals_of_the_library():
    lib, p = entro.lib(), 4096  # any address: argument errors come before it is used
    quant = dict(x=p, type=entro.BF16, tokens=4, cols=32, ldx=32, q=p, ldq=32, scale=p, sum=p)

    def quantize(**kw):
        a = {**quant, **kw}
        return lib.entro_quantize_tokens(a["x"], a["type"], a["tokens"], a["cols"], a["ldx"], a["q"], a["ldq"], a["scale"], a["sum"], None)

    for kw in (dict(x=None), dict(q=None), dict(scale=None), dict(sum=None), dict(type=entro.F32), dict(tokens=-1), dict(cols=0),
               dict(ldx=31), dict(ldq=16), dict(ldq=40), dict(q=p + 8), dict(x=p + 1)):
        assert quantize(**kw) == entro.E_INVAL, kw
    assert quantize(cols=65537, ldx=65537, ldq=65552) == entro.E_LIMIT
    assert quantize(tokens=2 ** 24 + 1) == entro.E_LIMIT
    assert quantize(tokens=0, x=None) == entro.OK

    prod = dict(q=p, ldq=32, xs=p, xz=p, tokens=4, w=p, wt=entro.U8, ldw=32, rows=8, cols=32, ws=p, wz=None, y=p, yt=entro.F32, ldy=8)

    def product(**kw):
        a = {**prod, **kw}
        return lib.entro_matmul_i8(a["q"], a["ldq"], a["xs"], a["xz"], a["tokens"], a["w"], a["wt"], a["ldw"], a["rows"], a["cols"], a["ws"],
                                   1.0, a["wz"], 0, a["y"], a["yt"], a["ldy"], None, None)

    for kw in (dict(q=None), dict(xs=None), dict(xz=None), dict(w=None), dict(y=None), dict(wt=entro.BF16), dict(yt=entro.S8),
               dict(ldq=31), dict(ldq=40), dict(ldw=16), dict(ldw=40), dict(ldy=7), dict(tokens=-1), dict(rows=-1), dict(cols=0),
               dict(q=p + 1), dict(w=p + 8), dict(y=p + 2)):
        assert product(**kw) == entro.E_INVAL, kw
    assert product(cols=65537, ldq=65552, ldw=65552) == entro.E_LIMIT
    assert product(tokens=0, y=None) == entro.OK and product(rows=0, y=None) == entro.OK

    def unpack(codes=p, bits=4, rows=4, cols=24, out=2 * p, ld=32):
        return lib.entro_unpack_codes(codes, bits, rows, cols, out, ld, None)

    for kw in (dict(codes=None), dict(out=None), dict(bits=2), dict(rows=-1), dict(ld=16), dict(ld=40), dict(codes=p + 1), dict(out=p)):
        assert unpack(**kw) == entro.E_INVAL, kw
    assert unpack(rows=0) == entro.OK


# ------------------------------------------------------------------ tokens to codes

@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("tokens,cols", [(1, 1), (3, 7), (5, 16), (2, 2047), (4, 2048), (3, 4100), (2, 16384), (2, 16400), (300, 264)])
def test_quantize_exact(dtype, tokens, cols):
    x = _tokens(_rng(tokens, cols), tokens, cols, dtype)
    if tokens > 2:
        x[1] = 0
        # many exact ties: 127 x / 254 with odd x
        x[2] = torch.from_numpy(_rng(cols).integers(-254, 255, cols).astype(np.float32)).to(dtype)
        x[2, 0] = 254 if dtype == torch.bfloat16 else 508
    got = entro.quantize_tokens(x.cuda())
    q, scale = _codes64(x)
    assert torch.equal(got.codes.cpu().double(), q)
    assert torch.equal(got.sum.cpu().double(), q.sum(1))
    assert torch.equal(got.scale.cpu(), (x.float().abs().amax(1) / 127))
    assert got.codes.stride(0) % 16 == 0


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("cols", [8192, 8193, 12001, 16385, 28672, 32768, 32769, 65536])
def test_quantize_long_rows(dtype, cols):
    for tokens in (1, 5):
        x = _tokens(_rng(tokens, cols, 1), tokens, cols, dtype)
        x[0, -1] = 2 * x[0].abs().max()  # the last column decides
        got = entro.quantize_tokens(x.cuda())
        q, scale = _codes64(x)
        assert torch.equal(got.codes.cpu().double(), q) and torch.equal(got.sum.cpu().double(), q.sum(1))
        assert torch.equal(got.scale.cpu(), x.float().abs().amax(1) / 127)
    y = torch.zeros(3, cols + 1, dtype=dtype)  # rows that do not begin on 16 bytes
    y[:, 1:] = _tokens(_rng(3, cols, 2), 3, cols, dtype)
    assert torch.equal(entro.quantize_tokens(y.cuda()[:, 1:]).codes.cpu().double(), _codes64(y[:, 1:])[0])


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_quantize_every_ratio(dtype):
    """Each significand of x against each of the largest value: every quotient that can tie."""
    bits = 128 if dtype == torch.bfloat16 else 1024
    n = bits if bits == 128 else 64
    tops = torch.from_numpy(_rng(bits).permutation(bits)[:n].astype(np.float32)) + bits
    sig = torch.arange(bits, 2 * bits, dtype=torch.float32)
    x = torch.cat([sig * 2.0 ** -e for e in range(0, 10)])[None].repeat(n, 1)
    x = torch.minimum(x, tops[:, None])
    x[:, 0] = tops
    x = (x * 2.0 ** -12).to(dtype)
    got = entro.quantize_tokens(x.cuda())
    q, _ = _codes64(x)
    assert torch.equal(got.codes.cpu().double(), q)


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_quantize_extremes(dtype):
    f = torch.finfo(dtype)
    tiny = f.smallest_normal * f.eps  # the smallest number of the type
    rows = [[f.max, -f.max, 1.0, f.max / 2], [tiny, -tiny, 0.0, tiny], [f.smallest_normal, tiny, 0.0, -f.smallest_normal / 2],
            [float("inf"), 1.0, 2.0, 3.0], [float("nan"), 1.0, 2.0, 3.0], [1.0, float("-inf"), 0.0, float("nan")], [0.0, -0.0, 0.0, 0.0]]
    x = torch.tensor(rows, dtype=torch.float64).to(dtype)
    got = entro.quantize_tokens(x.cuda())
    q, scale = _codes64(x)
    assert torch.equal(got.codes.cpu().double(), q)
    assert torch.equal(torch.isnan(got.scale.cpu()), torch.isnan(scale))
    ok = ~torch.isnan(scale)
    assert torch.equal(got.scale.cpu()[ok], scale[ok].float())


@gpu
def test_quantize_strides():
    wide = _tokens(_rng(5), 40, 300, torch.bfloat16).cuda()
    for x in (wide[:, 3:260], wide[::3, 8:208], wide[:0], wide[5:6, :1]):
        got = entro.quantize_tokens(x)
        q, _ = _codes64(x.cpu())
        assert torch.equal(got.codes.cpu().double(), q)


# ------------------------------------------------------------------ the product

SHAPES = [(1, 1, 1), (1, 128, 128), (3, 5, 40), (16, 128, 256), (17, 129, 200), (24, 2048, 2048), (33, 100, 1000), (64, 1024, 4096),
          (100, 300, 129), (128, 64, 512), (200, 257, 640), (256, 512, 384), (257, 256, 128), (300, 700, 1000), (515, 1000, 500),
          (1000, 300, 2056), (700, 5000, 136), (2100, 129, 64)]


@gpu
@pytest.mark.parametrize("weights", ["u8", "s8"])
@pytest.mark.parametrize("tokens,rows,cols", SHAPES)
def test_product(tokens, rows, cols, weights):
    rng = _rng(tokens, rows, cols)
    x = _tokens(rng, tokens, cols, torch.bfloat16).cuda()
    pitch = (cols + 15) // 16 * 16
    low, high = (0, 256) if weights == "u8" else (-128, 128)
    w = torch.from_numpy(rng.integers(low, high, (rows, pitch)).astype(np.uint8 if weights == "u8" else np.int8)).cuda()[:, :cols]
    xq = entro.quantize_tokens(x)
    scale = torch.from_numpy(np.exp(rng.standard_normal(rows)).astype(np.float32)).cuda()
    zero = torch.from_numpy(rng.integers(low, high, rows).astype(np.int32)).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for i, dtype in enumerate((torch.float32, torch.bfloat16, torch.float16)):
        ws, wz = (scale * 1e-4, zero) if i != 1 else (0.0123, 100 if i else None)
        y = entro.matmul_i8(xq, w, ws, wz, out_dtype=dtype, status=status)
        _close(y, _expect(xq, w, ws, wz))
        assert torch.equal(y, entro.matmul_i8(xq, w, ws, wz, out_dtype=dtype))
    assert int(status) == 0


@gpu
@pytest.mark.parametrize("tokens", [5, 300])
def test_product_largest_sums(tokens):
    """All products of one sign: the integer sums reach their largest values; zero points outside the codes' range."""
    cols = 65536
    x = torch.ones(tokens, cols, dtype=torch.bfloat16, device="cuda")
    x[1] = -1
    xq = entro.quantize_tokens(x)
    assert int(xq.codes.abs().min()) == 127
    w = torch.full((130, cols), 255, dtype=torch.uint8, device="cuda")
    w[0] = 0
    for zero in (0, 255, -256, 256, 1 << 24, -(1 << 24), -2 ** 31):
        y = entro.matmul_i8(xq, w, 1.0, zero, out_dtype=torch.float32)
        _close(y, _expect(xq, w, 1.0, zero))
    zero = torch.zeros(130, dtype=torch.int32, device="cuda")
    zero[7], zero[129] = 1 << 30, -300
    _close(entro.matmul_i8(xq, w, 1.0, zero, out_dtype=torch.float32), _expect(xq, w, 1.0, zero))


@gpu
def test_product_writes_its_rows_only():
    """An output inside a larger buffer: nothing around it changes; rows with NaN scale stay on their own rows."""
    for tokens, rows in ((20, 130), (300, 300)):
        rng = _rng(tokens, rows)
        x = _tokens(rng, tokens, 96, torch.bfloat16)
        x[3, 5] = float("nan")
        xq = entro.quantize_tokens(x.cuda())
        w = torch.from_numpy(rng.integers(0, 256, (rows, 96)).astype(np.uint8)).cuda()
        big = torch.full((tokens + 2, rows + 7), 7.0, device="cuda")
        out = big[1:-1, 3:3 + rows]
        assert entro.matmul_i8(xq, w, 0.5, 7, out=out) is out
        _close(out, _expect(xq, w, 0.5, 7))
        big[1:-1, 3:3 + rows] = 7.0
        assert bool((big == 7.0).all())


@gpu
def test_product_empty_and_refused():
    x = entro.quantize_tokens(torch.ones(4, 32, dtype=torch.bfloat16, device="cuda"))
    w = torch.ones(8, 32, dtype=torch.uint8, device="cuda")
    none = entro.quantize_tokens(torch.ones(0, 32, dtype=torch.bfloat16, device="cuda"))
    assert entro.matmul_i8(none, w, 1.0).shape == (0, 8)
    assert entro.matmul_i8(x, w[:0], 1.0).shape == (4, 0)
    with pytest.raises(ValueError):
        entro.matmul_i8(x, torch.ones(8, 40, dtype=torch.uint8, device="cuda")[:, 4:36], 1.0)
    with pytest.raises(ValueError):
        entro.matmul_i8(x, w, 1.0, out=torch.empty(4, 9, device="cuda"))
    with pytest.raises(ValueError):
        entro.matmul_i8(x, w, 1.0, out=torch.empty(4, 8, device="cuda", dtype=torch.float64))
    with pytest.raises(ValueError):
        entro.matmul_i8(x, w, torch.ones(8))  # on the host
    with pytest.raises(ValueError, match="gradient"):
        entro.matmul_i8(x, w, torch.ones(8, device="cuda", requires_grad=True))
    with torch.no_grad():
        entro.matmul_i8(x, w, torch.ones(8, device="cuda", requires_grad=True))
    with pytest.raises(ValueError):
        entro.matmul_i8(x, w, 1.0, status=torch.zeros(1, dtype=torch.int64, device="cuda"))
    with pytest.raises(entro.EntroError):
        entro.quantize_tokens(torch.ones(1, 32, dtype=torch.bfloat16, device="cuda").expand(3, 32))
    # scalars of other kinds, and an output that is given, go another way in the binding: the same bits
    want = entro.matmul_i8(x, w, 0.5, 3)
    assert torch.equal(entro.matmul_i8(x, w, np.float32(0.5), np.int64(3)), want)
    assert torch.equal(entro.matmul_i8(x, w, 0.5, 3, out=torch.empty_like(want)), want)
    assert torch.equal(entro.matmul_i8(x, w, torch.full((8,), 0.5, device="cuda"), torch.full((8,), 3, dtype=torch.int32, device="cuda")), want)


@gpu
def test_product_streams_and_graphs():
    """On another stream than the current one, and captured: the replay takes the inputs' new values."""
    rng = _rng(3)
    w = torch.from_numpy(rng.integers(-128, 128, (700, 512)).astype(np.int8)).cuda()
    for tokens in (40, 600):
        x = _tokens(rng, tokens, 512, torch.float16).cuda()
        want = entro.matmul_i8(entro.quantize_tokens(x), w, 0.01)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        got = entro.matmul_i8(entro.quantize_tokens(x, stream=side), w, 0.01, stream=side)
        side.synchronize()
        assert torch.equal(got, want)
        held = torch.zeros_like(x)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = entro.matmul_i8(entro.quantize_tokens(held), w, 0.01)
        for _ in range(2):
            held.copy_(x)
            graph.replay()
            assert torch.equal(y, want)
            held.zero_()
            graph.replay()
            assert not y.any()


@gpu
def test_product_wait_gives_up():
    """The bounded wait: bytes that never arrive end in a status, and the next call is right."""
    x = entro.quantize_tokens(torch.ones(20, 256, dtype=torch.bfloat16, device="cuda"))
    big = entro.quantize_tokens(torch.ones(300, 256, dtype=torch.bfloat16, device="cuda"))
    w = torch.ones(600, 256, dtype=torch.uint8, device="cuda")
    for q in (x, big):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        entro.test_stall_tables(16)
        try:
            entro.matmul_i8(q, w, 1.0, status=status)
            torch.cuda.synchronize()
        finally:
            entro.test_stall_tables(0)
        assert int(status) == entro.E_TIMEOUT
        status.zero_()
        _close(entro.matmul_i8(q, w, 1.0, out_dtype=torch.float32, status=status), _expect(q, w, 1.0, None))
        assert int(status) == 0


# ------------------------------------------------------------------ coded tensors

@gpu
@pytest.mark.parametrize("kind,bits,fmt,lanes,chunk,rows,cols", [
    ("t4", 8, entro.FORMAT_ROWS, 32, 4096, 200, 256), ("shifted", 8, entro.FORMAT_ROWS, 32, 4096, 70, 1000),
    ("positive", 8, entro.FORMAT_LANES, 32, 8192, 30, 72), ("laplace", 4, entro.FORMAT_ROWS, 32, 8192, 130, 512),
    ("laplace", 4, entro.FORMAT_LANES, 32, 8192, 33, 75), ("laplace", 4, entro.FORMAT_ROWS_CO, 32, 8192, 100, 1000),
    ("t4", 8, entro.FORMAT_SINGLE, 0, 4096, 64, 33), ("constant", 8, entro.FORMAT_ROWS, 32, 256, 5, 80)])
def test_coded_tensor_times_a_prompt(kind, bits, fmt, lanes, chunk, rows, cols):
    w = workloads.small_tensor(kind, rows, cols, seed=4)
    q, scale, zero, _ = oracle.quantize(w, bits, oracle.MODE_ASYM)
    dt = entro.upload(entro.Blob.encode(w, bits=bits, quant_mode=entro.QUANT_ASYM, fmt=fmt, chunk_symbols=chunk, lanes=lanes))
    codes = torch.from_numpy(q.reshape(rows, cols).astype(np.uint8))
    for tokens in (1, 20, 300):
        x = _tokens(_rng(tokens), tokens, cols, torch.bfloat16).cuda()
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        y = dt.matmul(x, out_dtype=torch.float32, status=status)
        assert int(status) == 0
        xq = entro.quantize_tokens(x)
        _close(y, _expect(xq, codes, float(scale), int(zero)))
        assert torch.equal(dt.matmul(xq, out_dtype=torch.float32), y)
