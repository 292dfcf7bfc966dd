"""Forward-mode derivatives: the operators have none, so a dual tensor is refused where its tangent would be lost."""
import pytest
import torch
import torch.autograd.forward_ad as fwd

import huffman_decode_canonical_b200 as entro

pytestmark = pytest.mark.gpu


def _calls():
    """(name, call, its tensors that may carry a tangent)"""
    q, k = torch.ones(3, 4, 64, dtype=torch.bfloat16, device="cuda"), torch.ones(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    x, w = torch.ones(3, 32, dtype=torch.bfloat16, device="cuda"), torch.ones(8, 32, dtype=torch.uint8, device="cuda")
    scale, cu, lens = torch.ones(8, device="cuda"), torch.arange(4, dtype=torch.int32, device="cuda"), torch.ones(3, dtype=torch.int32, device="cuda")
    table = torch.zeros((3, 1), dtype=torch.int32, device="cuda")
    xq, cache = entro.quantize_tokens(x), entro.KVCache.empty(1, 2, 64, 16, slots=3)
    return [("quantize_tokens", lambda x: entro.quantize_tokens(x), dict(x=x)),
            ("matmul_i8", lambda s, t: entro.matmul_i8(xq._replace(scale=t), w, s), dict(s=scale, t=xq.scale)),
            ("attention_prompt", lambda q, k, v: entro.attention_prompt(q, k, v, cu), dict(q=q, k=k, v=k.clone())),
            ("append", lambda k, v: cache.append(k, v, cu, table, lens), dict(k=k, v=k.clone())),
            ("attend", lambda q: cache.attend(q, table, lens), dict(q=q)),
            ("attend with an output", lambda q, out: cache.attend(q, table, lens, out=out), dict(q=q, out=torch.empty_like(q)))]


@pytest.mark.parametrize("i", range(6))
def test_dual_tensors_are_refused(i):
    name, call, tensors = _calls()[i]
    call(**tensors)
    with fwd.dual_level():
        call(**tensors)  # no tangent: as ever
        for n, t in tensors.items():
            dual = fwd.make_dual(t, torch.ones_like(t))
            with pytest.raises(ValueError, match="dual"):
                call(**{**tensors, n: dual})
            with torch.no_grad(), pytest.raises(ValueError, match="dual"):  # (does not switch forward mode off)
                call(**{**tensors, n: dual})
            call(**{**tensors, n: fwd.unpack_dual(dual).primal})
    call(**tensors)
