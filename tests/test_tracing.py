"""A trace (torch.jit.trace) cannot hold the operators: their results would be constants of it, so they refuse."""
import pytest
import torch

import huffman_decode_canonical_b200 as entro

pytestmark = [pytest.mark.gpu, pytest.mark.filterwarnings("ignore::DeprecationWarning")]


def test_traces_are_refused():
    q, x = torch.ones(3, 4, 64, dtype=torch.bfloat16, device="cuda"), torch.ones(3, 32, dtype=torch.bfloat16, device="cuda")
    w, xq = torch.ones(8, 32, dtype=torch.uint8, device="cuda"), entro.quantize_tokens(x)
    cu, lens = torch.arange(4, dtype=torch.int32, device="cuda"), torch.ones(3, dtype=torch.int32, device="cuda")
    table, cache = torch.zeros((3, 1), dtype=torch.int32, device="cuda"), entro.KVCache.empty(1, 4, 64, 16, slots=3)
    calls = [(lambda t: entro.quantize_tokens(t).codes, x), (lambda t: entro.matmul_i8(xq._replace(codes=t), w, 1.0), xq.codes),
             (lambda t: entro.attention_prompt(t, t, t, cu), q), (lambda t: cache.append(t, t, cu, table, lens), q),
             (lambda t: cache.read(table, t, 3)[0], cu), (lambda t: cache.attend(t, table, lens), q)]
    for call, t in calls:
        call(t)
        with pytest.raises(ValueError, match="traced"):
            torch.jit.trace(call, (t,), check_trace=False)
        call(t)
