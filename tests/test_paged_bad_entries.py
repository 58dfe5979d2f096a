"""Page table entries out of range in append and accumulated weights (GPU): what they cost stays with their sequence.  The
page that reads of a bad entry go to (page 0) belongs to another sequence here."""

import pytest
import torch

import exact_memory_efficient_b200 as m
from tests._paged import Batch

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def batch(dtype, counts, lens, page, seed):
    """Sequence 0 owns page 0; sequence 1 will get the bad entries."""
    bt = Batch(counts, lens, 4, 2, 64, page, dtype, seed=seed, spare=5)
    was = int(bt.table[0, 0])
    swap = {0: was, was: 0}
    bt.table = bt.table.clone().apply_(lambda p: swap.get(p, p))
    assert bt.table[0, 0] == 0 and (bt.table[1:] != 0).all()
    return bt


def bad_tables(bt):
    """Tables whose sequence 1 has entries out of range, among the old keys' and among the new ones'."""
    has = -(-bt.lens[1] // bt.page)
    for value in (-1, 10**9, -2**31, bt.pages):
        for first in (0, has // 2, has - 1):
            t = bt.table.clone()
            t[1, first:] = value
            yield t


def others(bt):
    """Pages that are not sequence 1's."""
    keep = torch.ones(bt.pages, dtype=torch.bool)
    keep[bt.table[1][bt.table[1] >= 0].long()] = False
    return keep.cuda()


CASES = [(BF, [1, 1, 1], [40, 300, 70], 16), (BF, [30, 40, 1], [200, 90, 33], 16), (BF, [3, 2, 9], [20, 2, 500], 128),
         (BF, [600, 500, 1], [700, 900, 33], 32), (F32, [1, 1, 1], [40, 300, 70], 16), (F32, [30, 40, 1], [200, 90, 33], 64)]


@pytest.mark.parametrize("dtype,counts,lens,page", CASES)
@pytest.mark.parametrize("rotated", [False, True])
def test_append_writes_no_page_of_others(dtype, counts, lens, page, rotated):
    bt = batch(dtype, counts, lens, page, seed=51)
    q, k, v, cu, kv = bt.gpu("q", "k", "v", "cu", "kv_len")
    freq = m.mea_rope_frequencies(32).cuda() if rotated else None

    def run(table):
        kc, vc, w = bt.gpu("k_cache", "v_cache", "weights")
        return m.paged_append(q, k, v, kc, vc, w, cu, kv, table.cuda(), None, freq), kc, vc, w

    want, keep = run(bt.table), others(bt)
    assert m.mea_last_device_error() == m.MEA_OK
    rows = torch.ones(bt.T, dtype=torch.bool)
    rows[int(bt.cu[1]):int(bt.cu[2])] = False
    for table in bad_tables(bt):
        got = run(table)
        assert m.mea_last_device_error() == m.MEA_ERR_PAGE
        assert torch.equal(got[0][rows.cuda()], want[0][rows.cuda()])
        for x, y in zip(got[1:], want[1:]):
            assert torch.equal(x[keep], y[keep])


@pytest.mark.parametrize("dtype,counts,lens,page", CASES)
def test_weights_are_added_to_no_page_of_others(dtype, counts, lens, page):
    bt = batch(dtype, counts, lens, page, seed=52)
    q, kc, vc, cu, kv = bt.gpu("q", "k_cache", "v_cache", "cu", "kv_len")
    _, lse = m.attention_paged(q, kc, vc, cu, kv, bt.table.cuda(), bt.max_q, bt.max_kv)

    def run(table):
        w = bt.weights.cuda()
        m.attention_paged_weights(q, lse, kc, w, cu, kv, table.cuda(), bt.max_q, bt.max_kv)
        return w

    want, keep = run(bt.table), others(bt)
    assert m.mea_last_device_error() == m.MEA_OK
    for table in bad_tables(bt):
        got = run(table)
        assert m.mea_last_device_error() == m.MEA_ERR_PAGE
        assert torch.equal(got[keep], want[keep])


def test_a_length_above_the_pages_that_a_sequence_has():
    """kv_len a page too long, with -1 behind: the new token has no slot and is written nowhere."""
    bt = batch(BF, [1, 1, 1], [40, 300, 70], 16, seed=53)
    bt.kv_len[1] = 320
    bt.table[1, 300 // 16 + 1:] = -1
    bt.table = torch.nn.functional.pad(bt.table, (0, 3), value=-1)
    q, k, v, kc, vc, w, cu, kv, tab = bt.gpu("q", "k", "v", "k_cache", "v_cache", "weights", "cu", "kv_len", "table")
    kv[1] = 310
    m.paged_append(None, k, v, kc, vc, w, cu, kv, tab)
    assert m.mea_last_device_error() == m.MEA_ERR_PAGE
    page0 = bt.table[0, 0]
    for x, old in ((kc, bt.k_cache), (vc, bt.v_cache), (w, bt.weights)):
        assert torch.equal(x[page0].cpu(), old[page0])
