"""The last run of a lanes-format tensor whose size is no multiple of 8: its few codes may all come with the lookup that
completes the run before, and must reach the output all the same."""
import numpy as np
import pytest
import torch

import oracle
import workloads

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lanes", [32, 64])
@pytest.mark.parametrize("kind,bits", [("laplace", 4), ("skew", 4), ("two_values", 4), ("skew", 8), ("t4", 8)])
def test_partial_last_run(kind, bits, lanes):
    import huffman_decode_canonical_b200 as entro
    for n in list(range(2401, 2417)) + [2475, 2 * 8192 + 1, 2 * 8192 + 8 * lanes + 3]:
        w = workloads.small_tensor(kind, 1, n, seed=4)
        q, scale, zero, _ = oracle.quantize(w, bits, oracle.MODE_ASYM)
        dt = entro.upload(entro.Blob.encode(w, bits=bits, quant_mode=entro.QUANT_ASYM, fmt=entro.FORMAT_LANES, chunk_symbols=8192,
                                            lanes=lanes))
        got = dt.decode_codes().cpu().numpy()
        if bits == 4:
            got = np.stack([got & 15, got >> 4], 1).reshape(-1)
        assert np.array_equal(got[:n], q.reshape(-1)[:n]), n
        want = oracle.dequant_bf16(q, scale, zero)
        assert np.array_equal(dt.decode_dequant_bf16().cpu().view(torch.int16).numpy().view(np.uint16).reshape(-1), want.reshape(-1)), n
