"""The operators around the coded weights, as measured: their cases, inputs and plain forms.

  linear   a prompt's activations times decoded codes: tokens quantized to 8 bits, an 8-bit integer product with a
           scale for each token and channel
  prompt   causal attention over packed prompts with grouped heads
  cache    keys and values appended to an 8-bit paged cache (a scale for each block of tokens and head) and read back
  attend   one new token's attention over that cache

Head layouts and widths are those of the model-shaped workloads (32 heads of 64, 96 and 128, 8 key heads of 128;
projections of 2048, 4096, 8192 and 14336).
"""
import math
import random

import torch

own = False  # True: run() calls the framework, False: the plain form in elementary torch operations

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # a few dozen sequences generate at once: one token each through a 2048-wide projection, just past the batch of
        # the fused GEMV; the latency of a small call counts
        dict(name="linear 24 tokens", op="linear", tokens=24, rows=2048, cols=2048, weights="u8", dtype="bf16", out="fp32"),
        # a chunk of a prompt (an odd number of tokens) through a gate or up projection
        dict(name="linear 515 tokens", op="linear", tokens=515, rows=14336, cols=4096, weights="u8", dtype="bf16", out="bf16"),
        # a packed batch of prompts through a down projection, symmetric codes
        dict(name="linear 8192 tokens", op="linear", tokens=8192, rows=4096, cols=14336, weights="s8", dtype="fp16", out="fp16"),
        # sixteen short questions packed together
        dict(name="prompt short pack", op="prompt", seqs=16, tokens=700, context=0, heads=32, kv_heads=32, dim=64, dtype="bf16"),
        # mail-sized prompts of uneven lengths
        dict(name="prompt ragged", op="prompt", seqs=5, tokens=6011, context=0, heads=32, kv_heads=32, dim=96, dtype="fp16"),
        # the next chunk of a long document behind its earlier part
        dict(name="prompt chunk", op="prompt", seqs=1, tokens=1000, context=5003, heads=32, kv_heads=8, dim=128, dtype="bf16"),
        # one long document
        dict(name="prompt long", op="prompt", seqs=1, tokens=8192, context=0, heads=32, kv_heads=8, dim=128, dtype="bf16"),
        # a token each of a few short chats, whose context is read back
        dict(name="cache tokens", op="cache", seqs=8, context=300, new=1, kv_heads=8, dim=128, page=64, dtype="bf16"),
        # whole prompts written, and read back for the next chunk
        dict(name="cache prompts", op="cache", seqs=6, context=0, new=8100, kv_heads=32, dim=96, page=32, dtype="fp16"),
        # one chat of ordinary length: one sequence has to fill the GPU
        dict(name="attend one", op="attend", seqs=1, most=1000, heads=32, kv_heads=8, dim=128, page=64, dtype="bf16"),
        # a serving batch with a key head for each head
        dict(name="attend batch", op="attend", seqs=48, most=2500, heads=32, kv_heads=32, dim=96, page=16, dtype="fp16"),
        # long documents, uneven
        dict(name="attend long", op="attend", seqs=48, most=32768, heads=32, kv_heads=8, dim=128, page=64, dtype="bf16"),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["linear", "prompt", "cache", "attend"])
    if op == "linear":
        rows, cols = _log(rng, 256, 14336), 8 * _log(rng, 32, 1792)
        tokens = min(_log(rng, 17, 8192), max(17, 8192 * 4096 * 14336 // (rows * cols)))
        return dict(op=op, tokens=tokens, rows=rows, cols=cols, weights=rng.choice(["u8", "s8"]), dtype=rng.choice(["bf16", "fp16"]), out=rng.choice(["bf16", "fp16", "fp32"]))
    dim = rng.choice([64, 96, 128])
    kv, group = rng.choice([(32, 1), (20, 1), (8, 4), (8, 1), (4, 8), (1, 16), (2, 5)])
    dtype = rng.choice(["bf16", "fp16"])
    page = rng.choice([16, 32, 64, 128])
    if op == "prompt":
        tokens = _log(rng, 40, 8192)
        seqs = min(tokens, _log(rng, 1, 32))
        context = _log(rng, 1, 4000) if tokens <= 3000 and rng.random() < 0.3 else 0
        return dict(op=op, seqs=seqs, tokens=tokens, context=context if seqs <= 4 else 0, heads=kv * group, kv_heads=kv, dim=dim, dtype=dtype)
    if op == "cache":
        if rng.random() < 0.5:
            return dict(op=op, seqs=_log(rng, 1, 64), context=_log(rng, 16, 2000), new=1, kv_heads=kv, dim=dim, page=page, dtype=dtype)
        return dict(op=op, seqs=_log(rng, 1, 6), context=0, new=_log(rng, 20, 8000), kv_heads=kv, dim=dim, page=page, dtype=dtype)
    return dict(op=op, seqs=_log(rng, 1, 48), most=_log(rng, 32, 32768 if kv <= 8 else 4000), heads=kv * group, kv_heads=kv, dim=dim, page=page, dtype=dtype)


def _uneven(case, n, low, high):
    """n whole numbers in [low, high], the largest equal to high: lengths that depend on the case alone."""
    r = random.Random("%s %d %d %d" % (case["op"], n, low, high))
    v = [r.randint(low, high) for _ in range(n)]
    v[r.randrange(n)] = high
    return v


def _lengths(case):
    """(tokens in the batch's sequences before the call, new tokens of each)"""
    n = case["seqs"]
    if case["op"] == "prompt":
        cuts = random.Random("cuts %d %d" % (n, case["tokens"])).sample(range(1, case["tokens"]), n - 1)
        edges = [0] + sorted(cuts) + [case["tokens"]]
        return [case["context"]] * n, [b - a for a, b in zip(edges, edges[1:])]
    if case["op"] == "cache":
        if case["new"] == 1:
            return _uneven(case, n, case["context"] // 4, case["context"]), [1] * n
        return [0] * n, _uneven(case, n, (case["new"] + 1) // 2, case["new"])
    return _uneven(case, n, case["most"] // 4, case["most"]), [0] * n


def work(case):
    if case["op"] == "linear":
        t, n, k = case["tokens"], case["rows"], case["cols"]
        out = 4 if case["out"] == "fp32" else 2
        return {"bytes": t * k * 2 + n * k + t * n * out + n * (8 if case["weights"] == "u8" else 4), "flops": 2 * t * n * k}
    before, new = _lengths(case)
    d, kv = case["dim"], case["kv_heads"]
    if case["op"] == "prompt":
        pairs = sum(n * b + n * (n + 1) // 2 for b, n in zip(before, new))
        rows, keys = sum(new), sum(new) + sum(before)
        return {"bytes": 2 * d * (2 * rows * case["heads"] + 2 * keys * kv), "flops": 4 * d * case["heads"] * pairs}
    p, total = case["page"], [b + n for b, n in zip(before, new)]
    token, code, scale = 2 * 2 * d * kv, 2 * d * kv, 2 * 4 * kv  # keys and values together
    if case["op"] == "cache":
        moved = 0
        for b, n, t in zip(before, new, total):
            filled = t // p - b // p
            moved += n * token + filled * (p * code + scale) + (t % p if filled else n) * token  # new tokens, to blocks and tail
            moved += b % p * token if filled else 0                                             # earlier tokens of the block that fills up
            moved += t // p * (p * code + scale) + t % p * token + t * token                    # read back
        return {"bytes": moved, "flops": 4 * d * kv * sum(new)}
    held = sum(t // p * (p * code + scale) + t % p * token for t in total)
    return {"bytes": held + 2 * 2 * d * case["heads"] * case["seqs"], "flops": 4 * d * case["heads"] * sum(total)}


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _ends(lengths):
    v = [0]
    for n in lengths:
        v.append(v[-1] + n)
    return v


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    dtype = DTYPES[case["dtype"]]
    s = dict(case=case, op=case["op"])
    if case["op"] == "linear":
        t, n, k = case["tokens"], case["rows"], case["cols"]
        x = normal(t, k) * torch.exp(0.5 * normal(1, k))  # some channels are larger than others
        x[1::97] = 0                                      # padding tokens
        pitch = (k + 15) // 16 * 16
        w = normal(n, pitch) * 24
        if case["weights"] == "u8":
            s.update(w=(w + 119).round_().clamp_(0, 255).to(torch.uint8)[:, :k], w_zero=(119 + 2 * normal(n)).round().to(torch.int32))
        else:
            s.update(w=w.round_().clamp_(-127, 127).to(torch.int8)[:, :k], w_zero=None)
        s.update(x=x.to(dtype), w_scale=1e-3 * torch.exp(0.3 * normal(n)), out=DTYPES[case["out"]])
        return s
    before, new = _lengths(case)
    total = [b + n for b, n in zip(before, new)]
    d, kv = case["dim"], case["kv_heads"]
    if case["op"] == "prompt":
        h = case["heads"]
        if case["context"] == 0:  # one projection's output, as it comes
            qkv = normal(sum(new), h + 2 * kv, d).to(dtype)
            q, k, v = qkv[:, :h], qkv[:, h:h + kv], qkv[:, h + kv:]
        else:
            q, k, v = (normal(r, m, d).to(dtype) for r, m in ((sum(new), h), (sum(total), kv), (sum(total), kv)))
        s.update(q=q, k=k, v=v, cu=_ints(_ends(new)), cu_keys=_ints(_ends(total)) if case["context"] else None, longest=max(new), longest_keys=max(total))
        return s
    p, n = case["page"], case["seqs"]
    blocks = max(-(-t // p) for t in total)
    pages = n * blocks + 1
    order = torch.randperm(pages - 1, generator=g, device="cuda").to(torch.int32) + 1  # page 0 is nobody's
    codes = [torch.empty((pages, kv, p, d), dtype=torch.int8, device="cuda") for _ in range(2)]
    for c in codes:
        for part in c.split(max(1, (1 << 28) // (kv * p * d))):
            part.copy_((normal(*part.shape) * 33).round_().clamp_(-127, 127))
    s.update(k_codes=codes[0], v_codes=codes[1], table=order.view(n, blocks), lens=_ints(total),
             slots=torch.randperm(n, generator=g, device="cuda").to(torch.int32))
    for name in ("k", "v"):
        s[name + "_scale"] = torch.exp(0.2 * normal(pages, kv)) / 33
        s[name + "_tail"] = normal(n, kv, p, d).to(dtype)
    if case["op"] == "cache":
        s.update(k=normal(sum(new), kv, d).to(dtype), v=normal(sum(new), kv, d).to(dtype), cu=_ints(_ends(new)), cu_all=_ints(_ends(total)), tokens=sum(total))
    else:
        s.update(q=normal(n, case["heads"], d).to(dtype))
    return s


def _cache(s):
    """The cache that a user's program keeps."""
    if "cache" not in s:
        import huffman_decode_canonical_b200 as entro
        s["cache"] = entro.KVCache(s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"], s["k_tail"], s["v_tail"])
    return s["cache"]


def run(s):
    op = s["op"]
    if own:
        import huffman_decode_canonical_b200 as entro
        if op == "linear":
            return entro.matmul_i8(entro.quantize_tokens(s["x"]), s["w"], s["w_scale"], s["w_zero"], out_dtype=s["out"])
        if op == "prompt":
            return entro.attention_prompt(s["q"], s["k"], s["v"], s["cu"], s["cu_keys"])
        if op == "cache":
            _cache(s).append(s["k"], s["v"], s["cu"], s["table"], s["lens"], slots=s["slots"])
            return s["cache"].read(s["table"], s["cu_all"], s["tokens"], slots=s["slots"])
        return _cache(s).attend(s["q"], s["table"], s["lens"], slots=s["slots"])
    return {"linear": _linear, "prompt": _prompt, "cache": _write_and_read, "attend": _attend}[op](s)


# ------------------------------------------------------------------ plain forms, 32 bits

def _codes(x, amax):
    """The nearest whole numbers to 127 x / amax, ties to even, as 32-bit floats; 0 where amax is 0."""
    return torch.where(amax > 0, (x * 127 / amax).round(), torch.zeros_like(x))


def _linear(s):
    x = s["x"].float()
    amax = x.abs().amax(1, keepdim=True)
    w = s["w"].float()
    if s["w_zero"] is not None:
        w = w - s["w_zero"].float()[:, None]
    return (_codes(x, amax) @ w.t() * (amax / 127 * s["w_scale"])).to(s["out"])


def _where_of(cu, tokens):
    """(sequence, position) of each of `tokens` packed tokens"""
    t = torch.arange(tokens, device="cuda", dtype=torch.int32)
    b = torch.searchsorted(cu, t, right=True) - 1
    return b, (t - cu[b]).long()


def _prompt(s):
    q, k, v, cu = s["q"].float(), s["k"].float(), s["v"].float(), s["cu"]
    cu_k = cu if s["cu_keys"] is None else s["cu_keys"]
    n, h, kv, d = cu.numel() - 1, q.shape[1], k.shape[1], q.shape[2]
    qlen, klen = cu.diff(), cu_k.diff()
    i, j = (torch.arange(m, device="cuda") for m in (s["longest"], s["longest_keys"]))
    qp = q[(cu[:-1, None] + i).clamp(max=q.shape[0] - 1)].view(n, -1, kv, h // kv, d)
    kp, vp = (a[(cu_k[:-1, None] + j).clamp(max=k.shape[0] - 1)] for a in (k, v))
    scores = torch.matmul(qp.permute(0, 2, 3, 1, 4), kp.permute(0, 2, 3, 1)[:, :, None]).mul_(1 / math.sqrt(d))  # [n, kv, group, query, key]
    seen = j <= i[:, None] + (klen - qlen)[:, None, None]
    scores.masked_fill_(~seen[:, None, None], -math.inf)
    scores.sub_(scores.amax(-1, keepdim=True)).exp_()
    o = torch.matmul(scores, vp.permute(0, 2, 1, 3)[:, :, None]) / scores.sum(-1, keepdim=True)
    b, at = _where_of(cu, q.shape[0])
    return o.permute(0, 3, 1, 2, 4)[b, at].reshape(q.shape).to(s["q"].dtype)


def _write(s, new, codes, scale, tail, cu, table, lens, slots):
    """The new tokens of one of keys and values into its blocks: full blocks as codes, the last one's tokens into the tail."""
    n, p, d = lens.numel(), codes.shape[2], codes.shape[3]
    start = lens - cu.diff()
    first, last = start // p, (lens - 1) // p
    blocks = table.shape[1]
    b, at = _where_of(cu, new.shape[0])
    at = at + start[b]
    rows = torch.zeros((n, blocks, p) + new.shape[1:], device="cuda")
    rows[torch.arange(n, device="cuda"), first] = tail[slots].float().transpose(1, 2)
    rows[b, at // p, at % p] = new.float()
    rows = rows.transpose(2, 3)  # [sequence, block, head, token, channel]
    j = torch.arange(blocks, device="cuda")
    full = (j >= first[:, None]) & ((j + 1) * p <= lens[:, None])
    amax = rows.abs().amax((3, 4), keepdim=True)
    page = torch.where(full, table.long(), 0)  # what is not full goes to the page that is nobody's
    codes[page] = _codes(rows, amax).to(torch.int8)
    scale[page] = amax[..., 0, 0] / 127
    open_block = rows[torch.arange(n, device="cuda"), last].to(tail.dtype)
    tail[slots] = torch.where((lens % p != 0)[:, None, None, None], open_block, tail[slots])


def _read(codes, scale, tail, table, lens, slots, b, at):
    p = codes.shape[2]
    page, off = table[b, at // p].long(), at % p
    held = codes[page, :, off].float() * scale[page][..., None]
    return torch.where((at >= lens[b] // p * p)[:, None, None], tail[slots[b].long(), :, off].float(), held).to(tail.dtype)


def _write_and_read(s):
    slots, lens = s["slots"].long(), s["lens"].long()
    b, at = _where_of(s["cu_all"], s["tokens"])
    out = []
    for name in ("k", "v"):
        held = s[name + "_codes"], s[name + "_scale"], s[name + "_tail"]
        _write(s, s[name], *held, s["cu"], s["table"], lens, slots)
        out.append(_read(*held, s["table"], lens, slots, b, at))
    return tuple(out)


def _attend(s):
    q, table, lens = s["q"].float(), s["table"].long(), s["lens"].long()
    n, h, d = q.shape
    kv, p = s["k_codes"].shape[1:3]
    full = lens // p * p
    j = torch.arange(table.shape[1] * p, device="cuda")
    i = torch.arange(p, device="cuda")
    seen = torch.cat([j < full[:, None], i < (lens - full)[:, None]], 1)[:, None, None]
    slots = s["slots"].long()

    def values(name):  # [sequence, head, token, channel]
        held = (s[name + "_codes"][table].float() * s[name + "_scale"][table][..., None, None]).transpose(1, 2).reshape(n, kv, -1, d)
        return torch.cat([held, s[name + "_tail"][slots].float()], 2)

    scores = torch.matmul(q.view(n, kv, h // kv, d), values("k").transpose(2, 3)) / math.sqrt(d)
    scores = scores.masked_fill(~seen, -math.inf)
    e = (scores - scores.amax(-1, keepdim=True)).exp()
    return (torch.matmul(e, values("v")) / e.sum(-1, keepdim=True)).view(q.shape).to(s["q"].dtype)


# ------------------------------------------------------------------ from the definitions, 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "linear":
        x, w = s["x"].double(), s["w"].double()
        if s["w_zero"] is not None:
            w -= s["w_zero"].double().unsqueeze(1)
        most = x.abs().max(dim=1, keepdim=True).values
        q = torch.round(x * 127 / most.clamp_min(1e-300))
        return (q @ w.T) * most / 127 * s["w_scale"].double()
    before, new = _lengths(case)
    total = [b + n for b, n in zip(before, new)]
    if case["op"] == "prompt":
        out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
        group = case["heads"] // case["kv_heads"]
        for a, m, c, t in zip(_ends(new), new, _ends(total), total):
            hidden = torch.ones((m, t), dtype=torch.bool, device="cuda").triu(t - m + 1)
            for h in range(case["heads"]):
                q, k, v = s["q"][a:a + m, h].double(), s["k"][c:c + t, h // group].double(), s["v"][c:c + t, h // group].double()
                out[a:a + m, h] = torch.softmax((q @ k.T / case["dim"] ** 0.5).masked_fill_(hidden, -math.inf), 1) @ v
        return out
    p, table, slots = case["page"], s["table"].tolist(), s["slots"].tolist()

    def context(name, b, t):
        """[token, head, channel] of sequence b before the call, whose blocks up to t // p are coded"""
        at = torch.tensor(table[b][:t // p], dtype=torch.long, device="cuda")
        coded = (s[name + "_codes"][at].double() * s[name + "_scale"][at].double()[:, :, None, None]).permute(0, 2, 1, 3).flatten(0, 1)
        return torch.cat([coded, s[name + "_tail"][slots[b]].double().transpose(0, 1)[:t % p]])

    if case["op"] == "cache":
        out = []
        for name in ("k", "v"):
            rows = []
            for b, (a, m) in enumerate(zip(_ends(new), new)):
                whole = torch.cat([context(name, b, before[b]), s[name][a:a + m].double()])
                lo, hi = before[b] // p * p, total[b] // p * p
                if hi > lo:
                    block = whole[lo:hi].view((hi - lo) // p, p, *whole.shape[1:])
                    most = block.abs().amax((1, 3), keepdim=True).clamp_min(1e-300)
                    whole[lo:hi] = (torch.round(block * 127 / most) * most / 127).flatten(0, 1)
                rows.append(whole)
            out.append(torch.cat(rows))
        return tuple(out)
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    for b, t in enumerate(total):
        k, v = context("k", b, t), context("v", b, t)
        q = s["q"][b].double().view(case["kv_heads"], -1, case["dim"])
        w = torch.softmax(torch.einsum("hgd,thd->hgt", q, k) / case["dim"] ** 0.5, 2)
        out[b] = torch.einsum("hgt,thd->hgd", w, v).flatten(0, 1)
    return out
