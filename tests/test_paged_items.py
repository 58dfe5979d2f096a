"""Attention items of one query tile followed by items of two, in one CTA (GPU): the order in which the MMA
issuer of csrc/paged_tc.cu waits for a slot's epilogue and lets it finish its next item."""

import pytest
import torch

import exact_memory_efficient_b200 as m
from tests._paged import Batch
from tests.test_paged_attn import check, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("counts,lens,H,D,page,repeats", [
    ([300, 270, 384], [300, 270, 384], 160, 64, 16, 200),   # from one head's last tile to the next head's first pair
    ([300, 300], [300, 300], 160, 128, 16, 200),
    ([400, 129, 1], [400, 129, 50], 160, 128, 64, 200),
    ([257, 60, 300], [257, 60, 290], 160, 64, 32, 50),       # rows that see no key among them
])
def test_two_tiles_after_one(counts, lens, H, D, page, repeats):
    """Many heads over H_kv = H: every CTA takes several heads, and n mod 256 in 1..128 ends each of them with a
    single query tile.  The first key tile of the next head is all that its first query tile sees."""
    bt = Batch(counts, lens, H, H, D, page, torch.bfloat16, seed=31)
    want = run(bt)
    check(bt, want)
    q, kc, vc, cu, kv, tab = bt.gpu("q", "k_cache", "v_cache", "cu", "kv_len", "table")
    for _ in range(repeats):
        o, lse = m.attention_paged(q, kc, vc, cu, kv, tab, bt.max_q, bt.max_kv, bt.scale)
    assert m.mea_last_device_error() == m.MEA_OK
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
