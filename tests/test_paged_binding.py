"""What the binding of the paged operators passes on (no GPU needed: the calls are recorded)."""
import ctypes as C

import pytest
import torch

import prefill_decode_layer_gb300 as pdl
from prefill_decode_layer_gb300 import ds4g


@pytest.mark.parametrize("window,passed", [(0, 0), (-1, 0), (1, 1), (2 ** 31 - 1, 2 ** 31 - 1), (2 ** 31, 2 ** 31 - 1),
                                           (2 ** 32 + 5, 2 ** 31 - 1), (2 ** 63, 2 ** 31 - 1), (5 - 2 ** 32, 0)])
def test_windows_beyond_32_bits(monkeypatch, window, passed):
    """A window wider than any sequence is that, not its low 32 bits."""
    args = []
    monkeypatch.setattr(ds4g, "_call", lambda name, index, stream, *a: args.extend(a))
    k, q = torch.zeros(4, 8, 2, 64), torch.zeros(3, 4, 64)
    batch = pdl.PagedBatch(torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32))
    pdl.paged_attention(pdl.PagedKV(k, k.clone()), batch, q, q.clone(), torch.zeros(16, dtype=torch.uint8), window=window)
    got = C.c_int(args[-3]).value   # window, workspace, its bytes
    assert max(got, 0) == passed


@pytest.mark.parametrize("most,passed", [(1, 1), (128, 128), (2 ** 31 - 1, 2 ** 31 - 1), (2 ** 32 + 1, 2 ** 31 - 1), (0, 0),
                                         (1 - 2 ** 32, 0)])
def test_counts_beyond_32_bits(most, passed):
    batch = pdl.PagedBatch(torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32),
                           torch.zeros(4, dtype=torch.int32), max_new=most)
    assert max(batch.struct.max_new, 0) == passed
