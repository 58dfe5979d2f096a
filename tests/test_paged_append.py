"""mea_paged_append against the fp64 definition (GPU)."""

import numpy as np
import pytest
import torch

import exact_memory_efficient_b200 as m
from oracle import paged
from tests._paged import Batch, f64, rope_bound

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def run(bt, pos, freq, interleaved=False, mscale=1.0, q=None, k=None, v=None, weights=True):
    kc, vc, w, cu, kv, tab = bt.gpu("k_cache", "v_cache", "weights", "cu", "kv_len", "table")
    q, k, v = (bt.q.cuda() if q is None else q), (bt.k.cuda() if k is None else k), (bt.v.cuda() if v is None else v)
    qo = torch.full((bt.T, bt.H, bt.D), 7.0, dtype=bt.dtype, device="cuda")
    m.mea_paged_append(q, qo, k, v, kc, vc, w if weights else None, cu, kv, tab, None if pos is None else pos.cuda(),
                       None if freq is None else freq.cuda(), int(interleaved), mscale)
    assert m.mea_last_device_error() == m.MEA_OK
    return qo, kc, vc, w


def check(bt, pos, freq, interleaved, mscale, got):
    fr = None if freq is None else freq.numpy()
    args = (bt.cu.numpy(), bt.kv_len.numpy(), bt.table.numpy(), None if pos is None else pos.numpy(), fr)
    wq, wk, wv, ww = paged.append(*bt.np("q", "k", "v", "k_cache", "v_cache", "weights"), *args,
                                  interleaved=interleaved, mscale=mscale)
    qo, kc, vc, w = (f64(t) for t in got)
    assert np.array_equal(vc, wv) and np.array_equal(w, ww)
    rows = list(bt.used_rows)
    others = [t for t in range(bt.T) if t not in bt.used_rows]
    assert (qo[others] == 7.0).all()
    if freq is None:
        assert np.array_equal(kc, wk) and np.array_equal(qo[rows], wq[rows])
        return
    tol = rope_bound(f64(bt.q), fr, interleaved, mscale, bt.dtype, wq)
    assert (np.abs(qo - wq) <= tol)[rows].all()
    # slots that were written; all others keep their bits
    new = np.zeros(kc.shape[0:1] + kc.shape[2:3], dtype=bool)
    for b, (n, L) in enumerate(zip(bt.counts, bt.lens)):
        for i in range(n):
            if L - n + i < 0:
                continue
            p, f = bt.table[b, (L - n + i) // bt.page], (L - n + i) % bt.page
            new[p, f] = True
            kb = f64(bt.k[int(bt.cu[b]) + i])
            t = rope_bound(kb, fr, interleaved, mscale, bt.dtype, wk[p, :, f])
            assert (np.abs(kc[p, :, f] - wk[p, :, f]) <= t).all()
    old = f64(bt.k_cache)
    keep = ~np.broadcast_to(new[:, None, :, None], kc.shape)
    assert np.array_equal(kc[keep], old[keep])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype,counts,lens,H,Hkv,D,page,rot", [
    (BF, [1], [1], 1, 1, 64, 16, 64), (BF, [1, 1, 1], [17, 16, 900], 8, 2, 128, 16, 128),
    (BF, [33, 0, 5], [33, 40, 300], 6, 3, 64, 32, 32), (BF, [7, 300], [4, 301], 5, 5, 128, 256, 96),
    (F32, [3, 20], [64, 21], 4, 1, 96, 64, 48), (F32, [1, 2], [0, 129], 2, 2, 32, 128, 32),
    (BF, [700, 200], [5000, 200], 24, 8, 128, 64, 64),
])
def test_append(dtype, counts, lens, H, Hkv, D, page, rot, interleaved):
    bt = Batch(counts, lens, H, Hkv, D, page, dtype, seed=len(lens), front=2, behind=3)
    pos = torch.randint(0, 100000, (bt.T,), generator=torch.Generator().manual_seed(5), dtype=torch.int32)
    freq = m.mea_rope_frequencies(rot)
    check(bt, pos, freq, interleaved, 1.1, run(bt, pos, freq, interleaved, 1.1))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_append_without_rotation_and_with_slots_as_positions(dtype):
    bt = Batch([3, 18, 1], [20, 18, 65], 4, 2, 64, 16, dtype, seed=9, behind=1)
    check(bt, None, None, False, 1.0, run(bt, None, None))
    freq = m.mea_rope_frequencies(64)
    check(bt, None, freq, False, 1.0, run(bt, None, freq))


def test_append_of_slices_of_a_projection():
    """q, k and v as views of one projection's rows, and with a stride beyond them."""
    bt = Batch([4, 9], [12, 90], 4, 2, 64, 16, BF, seed=11)
    freq = m.mea_rope_frequencies(64)
    row = torch.cat([bt.q.flatten(1), bt.k.flatten(1), bt.v.flatten(1), torch.zeros(bt.T, 24, dtype=BF)], 1).cuda()
    q, k, v, _ = row.split([256, 128, 128, 24], 1)
    got = run(bt, None, freq, q=q.view(-1, 4, 64), k=k.view(-1, 2, 64), v=v.view(-1, 2, 64))
    check(bt, None, freq, False, 1.0, got)


def test_append_in_place_and_keys_only():
    bt = Batch([4, 9], [12, 90], 4, 2, 128, 16, BF, seed=12)
    freq = m.mea_rope_frequencies(128)
    want = run(bt, None, freq)
    kc, vc, w, cu, kv, tab, q, k, v = bt.gpu("k_cache", "v_cache", "weights", "cu", "kv_len", "table", "q", "k", "v")
    m.mea_paged_append(q, q, k, v, kc, vc, w, cu, kv, tab, None, freq.cuda())
    assert torch.equal(q, want[0]) and torch.equal(kc, want[1])
    kc2, vc2 = bt.k_cache.cuda(), bt.v_cache.cuda()
    assert m.paged_append(None, k, v, kc2, vc2, None, cu, kv, tab, None, freq.cuda()) is None
    assert torch.equal(kc2, want[1]) and torch.equal(vc2, want[2])


def test_bad_pages_lengths_and_offsets_are_reported():
    """Entries out of range cost no access outside the buffers, and are reported."""
    bt = Batch([4, 9], [12, 90], 4, 2, 64, 16, BF, seed=13)
    kc, vc, w, cu, kv, tab, q, k, v = bt.gpu("k_cache", "v_cache", "weights", "cu", "kv_len", "table", "q", "k", "v")
    call = lambda **x: m.paged_append(*{**dict(q=q, k=k, v=v, kc=kc, vc=vc, w=w, cu=cu, kv=kv, tab=tab), **x}.values())  # noqa: E731
    bad = tab.clone()
    bad[1, 5] = 10**9
    for x in (dict(tab=bad), dict(tab=torch.full_like(tab, -7)), dict(kv=kv + 2**30), dict(kv=kv - 2**30),
              dict(cu=cu + 2**30), dict(cu=cu.flip(0).contiguous() + 5)):
        call(**x)
        st = m.mea_last_device_error()
        assert st in (m.MEA_ERR_PAGE, m.MEA_OK)
        # offsets behind T reach no row at all: nothing to report
        assert st == m.MEA_ERR_PAGE or "cu" in x
    call()
    assert m.mea_last_device_error() == m.MEA_OK
