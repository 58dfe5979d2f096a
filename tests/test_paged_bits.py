"""Equal bits for equal inputs of bf16 attention over a paged cache (GPU), whatever lies in the rows and the shared memory
around: a query tile's spare rows must not move the reference maximum of its rows."""

import pytest
import torch

import exact_memory_efficient_b200 as m
from tests._paged import Batch
from tests.test_paged_attn import check, run

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def leave_in_shared_memory(x):
    """Full query tiles of the value x (and keys of x) through every SM."""
    bt = Batch([256] * 8, [256] * 8, 32, 32, 128, 64, BF, seed=40)
    q, kc, vc, cu, kv, tab = bt.gpu("q", "k_cache", "v_cache", "cu", "kv_len", "table")
    g = torch.Generator(device="cuda").manual_seed(41)
    q = (torch.randn(q.shape, generator=g, device="cuda") * x).to(BF)
    m.attention_paged(q, kc, vc, cu, kv, tab, 256, 256)


def rising(counts, lens, H, Hkv, D, page, **kw):
    """Scores whose maximum rises a little along the keys, so that a rescale out of turn changes a row's bits."""
    bt = Batch(counts, lens, H, Hkv, D, page, BF, seed=42, **kw)
    for b, L in enumerate(lens):
        j = torch.arange(L)
        p, f = bt.table[b, j // page].long(), j % page
        bt.k_cache[p, :, f] = (bt.k_cache[p, :, f].float() * torch.linspace(0.3, 1.0, L)[:, None, None]).to(BF)
    return bt


# Sizes that give every CTA several key tiles of an item: the first tile of a part has no reference to move.
@pytest.mark.parametrize("counts,lens,H,Hkv,D,page", [
    ([1] * 8, [4000, 3000, 2500, 3999, 4001, 700, 2000, 3333], 32, 8, 128, 16),   # decode, 4 rows of a tile
    ([1] * 4, [5000] * 4, 24, 8, 64, 64),
    ([200, 190], [2000, 2500], 24, 8, 128, 16),         # chunks, 126 rows of 128
    ([70, 51], [3000, 2800], 40, 8, 64, 32), ([43, 20], [3000, 2777], 24, 8, 128, 64),
])
def test_bits_do_not_depend_on_what_ran_before(counts, lens, H, Hkv, D, page):
    bt = rising(counts, lens, H, Hkv, D, page)
    outs = []
    for x in (0.0, 1.0, 30.0, 300.0, 0.0):
        leave_in_shared_memory(x)
        outs.append(run(bt))
    check(bt, outs[0])
    for o, lse in outs[1:]:
        assert torch.equal(o, outs[0][0]) and torch.equal(lse, outs[0][1])


@pytest.mark.parametrize("counts,lens,H,Hkv,D,page,max_q", [
    ([1], [24000], 32, 8, 128, 16, 4), ([2, 1], [17000, 9000], 32, 16, 64, 32, 8), ([30], [9000], 48, 16, 128, 16, None),
    ([50], [9000], 16, 16, 128, 64, None),
])
def test_bits_do_not_depend_on_rows_of_others(counts, lens, H, Hkv, D, page, max_q):
    """Rows outside every sequence, which a tile's copy brings in with a sequence's last tokens."""
    bt = rising(counts, lens, H, Hkv, D, page, front=3, behind=200)
    used = list(bt.used_rows)
    outs = []
    for x in (0.0, 3.0, 100.0, float("nan"), float("inf")):
        keep = bt.q[used].clone()
        bt.q = torch.randn(bt.q.shape, generator=torch.Generator().manual_seed(43)).mul(x).to(BF)
        bt.q[used] = keep
        o, lse = run(bt, max_q=max_q)
        outs.append((o[used], lse[used]))
    assert m.mea_last_device_error() == m.MEA_OK
    for o, lse in outs[1:]:
        assert torch.equal(o, outs[0][0]) and torch.equal(lse, outs[0][1])


def test_bits_do_not_depend_on_the_sequence_behind():
    """The next sequence's tokens share the last query tile."""
    bt = rising([40, 300], [9000, 300], 48, 16, 128, 16)
    want = run(bt)[0][:40]
    bt.q[40:] *= 50
    assert torch.equal(run(bt)[0][:40], want)
