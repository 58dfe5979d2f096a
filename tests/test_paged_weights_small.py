"""Accumulated weights that are subnormal numbers (GPU): adding nothing to a weight leaves its bits, whichever way the
keys' sums reach the cache."""

import pytest
import torch

import exact_memory_efficient_b200 as m
from tests._paged import Batch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,counts,lens,H,Hkv,D,page", [
    (torch.bfloat16, [1, 1], [300, 77], 8, 2, 128, 16), (torch.bfloat16, [1] * 20, [130] * 20, 4, 4, 64, 16),
    (torch.bfloat16, [40, 90], [500, 90], 4, 2, 64, 16), (torch.bfloat16, [900, 3], [900, 700], 4, 1, 128, 64),
    (torch.float32, [1, 30], [77, 300], 4, 2, 64, 16),
])
def test_adding_nothing_keeps_subnormal_weights(dtype, counts, lens, H, Hkv, D, page):
    """With lse = 300 every probability is below e^-250 and so 0 in fp32."""
    bt = Batch(counts, lens, H, Hkv, D, page, dtype, seed=61)
    bits = torch.randint(1, 1 << 23, bt.weights.shape, generator=torch.Generator().manual_seed(62), dtype=torch.int32)
    w = bits.view(torch.float32).cuda()
    q, kc, cu, kv, tab = bt.gpu("q", "k_cache", "cu", "kv_len", "table")
    m.attention_paged_weights(q, torch.full((bt.T, H), 300.0, device="cuda"), kc, w, cu, kv, tab, bt.max_q, bt.max_kv)
    assert m.mea_last_device_error() == m.MEA_OK
    assert torch.equal(w.cpu().view(torch.int32), bits)
