"""mea_paged_evict against the definition (GPU): everything is moved bits and whole numbers, so exact."""

import math

import numpy as np
import pytest
import torch

import exact_memory_efficient_b200 as m
from oracle import paged
from tests._paged import Batch

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def dst_of(bt, n_keep):
    per = [-(-min(x, n_keep) // bt.page) for x in bt.lens]
    t = torch.full((len(per), max([1, -(-min(n_keep, bt.max_pages * bt.page) // bt.page)])), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(per):
        t[b, :n] = bt.free[at:at + n]
        at += n
    assert at <= len(bt.free)
    return t


def check(bt, n_keep, n_recent, in_place=False):
    dst = bt.table if in_place else dst_of(bt, n_keep)
    kc, vc, w, kv, tab = bt.gpu("k_cache", "v_cache", "weights", "kv_len", "table")
    kept, n = m.paged_evict(kc, vc, w, tab, kv, tab if in_place else dst.cuda(), n_keep, n_recent)
    assert m.mea_last_device_error() == m.MEA_OK
    bits = torch.int16 if bt.dtype == BF else torch.int32
    ints = lambda t, b: t.cpu().view(b).numpy()  # noqa: E731
    wk, wv, ww, wkept, wn = paged.evict(ints(bt.k_cache, bits), ints(bt.v_cache, bits), bt.weights.numpy(),
                                        bt.table.numpy(), bt.kv_len.numpy(), dst.numpy(), n_keep, n_recent)
    assert np.array_equal(kept.cpu().numpy(), wkept) and np.array_equal(n.cpu().numpy(), wn)
    assert np.array_equal(ints(kc, bits), wk) and np.array_equal(ints(vc, bits), wv)
    assert np.array_equal(ints(w, torch.int32), ww.view(np.int32))


CASES = [
    # dtype, lens, Hkv, D, page, n_keep, n_recent
    (BF, [20], 1, 64, 16, 8, 2), (BF, [1, 2, 3], 2, 128, 16, 2, 0), (BF, [500, 64, 65, 0], 3, 64, 32, 64, 16),
    (BF, [3000, 1999], 2, 128, 64, 1000, 128), (BF, [300], 4, 64, 256, 299, 299), (BF, [1025], 1, 128, 128, 1024, 0),
    (F32, [90, 40], 2, 32, 16, 33, 7), (F32, [700], 2, 96, 16, 300, 1), (F32, [130, 5000], 1, 128, 64, 129, 0),
]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("dtype,lens,Hkv,D,page,n_keep,n_recent", CASES)
def test_evict(dtype, lens, Hkv, D, page, n_keep, n_recent, in_place):
    bt = Batch([0] * len(lens), lens, Hkv, Hkv, D, page, dtype, seed=sum(lens), spare=200)
    check(bt, n_keep, n_recent, in_place)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("kind", ["equal", "zeros", "steps", "special", "negative", "low bits", "tiny"])
def test_evict_ties_and_special_weights(kind, in_place):
    bt = Batch([0, 0], [1500, 700], 2, 2, 64, 16, BF, seed=5, spare=100)
    g = torch.Generator().manual_seed(1)
    w = bt.weights
    if kind == "equal":
        w.fill_(0.25)
    elif kind == "zeros":
        w.copy_(torch.where(torch.rand(w.shape, generator=g) < 0.5, 0.0, -0.0))
    elif kind == "steps":
        w.copy_(torch.randint(0, 4, w.shape, generator=g).float())
    elif kind == "special":
        pick = torch.randint(0, 6, w.shape, generator=g)
        w.copy_(torch.tensor([math.nan, math.inf, -math.inf, 0.0, 1.0, -1.0])[pick])
    elif kind == "negative":
        w.mul_(-1)
    elif kind == "low bits":
        w.copy_((torch.randint(0, 300, w.shape, generator=g).int() + 0x3f800000).view(torch.float32))
    else:
        w.copy_(torch.randint(0, 5000, w.shape, generator=g).int().view(torch.float32))   # subnormal
    check(bt, 400, 30, in_place)


def test_evict_more_keys_than_shared_memory_holds():
    bt = Batch([0], [60001], 1, 1, 64, 64, BF, seed=6, spare=500)
    check(bt, 20000, 100)
    check(bt, 20000, 100, in_place=True)


def test_evict_twice_and_lengths_in_place():
    """kv_len_out may be kv_len; a second eviction takes the first one's result."""
    bt = Batch([0, 0], [400, 90], 2, 2, 64, 16, BF, seed=7)
    kc, vc, w, kv, tab = bt.gpu("k_cache", "v_cache", "weights", "kv_len", "table")
    k, v, ww, n = *(x.numpy() for x in (bt.k_cache.view(torch.int16), bt.v_cache.view(torch.int16), bt.weights)), bt.kv_len.numpy()
    for keep, recent in ((200, 20), (77, 5)):
        idx = torch.empty(2, 2, keep, dtype=torch.int32, device="cuda")
        m.mea_paged_evict(kc, vc, w, tab, kv, tab, kv, idx, recent)
        k, v, ww, kept, n = paged.evict(k, v, ww, bt.table.numpy(), n, bt.table.numpy(), keep, recent)
        assert np.array_equal(idx.cpu().numpy(), kept) and np.array_equal(kv.cpu().numpy(), n)
    assert np.array_equal(kc.cpu().view(torch.int16).numpy(), k) and np.array_equal(w.cpu().numpy(), ww)


def test_evict_graph_replay_and_without_lengths():
    bt = Batch([0, 0], [400, 90], 2, 2, 64, 16, BF, seed=8)
    kc, vc, w, kv, tab = bt.gpu("k_cache", "v_cache", "weights", "kv_len", "table")
    dst = dst_of_spare = torch.arange(bt.pages, bt.pages + 2 * 13, dtype=torch.int32).view(2, 13).cuda()
    grow = lambda t: torch.cat([t, torch.zeros(26, *t.shape[1:], dtype=t.dtype, device="cuda")])  # noqa: E731
    kc, vc, w = grow(kc), grow(vc), grow(w)
    idx = torch.empty(2, 2, 200, dtype=torch.int32, device="cuda")
    call = lambda: m.mea_paged_evict(kc, vc, w, tab, kv, dst_of_spare, None, idx, 20)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    kv -= 31
    w[:bt.pages] = torch.rand(bt.pages, 2, 16, device="cuda")
    before = [t.clone() for t in (kc, vc, w)]
    graph.replay()
    want = paged.evict(*(t.cpu().float().numpy() for t in before), bt.table.numpy(), kv.cpu().numpy(), dst.cpu().numpy(), 200, 20)
    assert np.array_equal(idx.cpu().numpy(), want[3])
    for got, ref in zip((kc, vc, w), want):
        assert np.array_equal(got.cpu().float().numpy(), ref)


def test_evict_bad_tables_are_reported():
    bt = Batch([0, 0], [400, 90], 2, 2, 64, 16, BF, seed=9, spare=60)
    kc, vc, w, kv, tab = bt.gpu("k_cache", "v_cache", "weights", "kv_len", "table")
    dst = dst_of(bt, 100).cuda()
    for x in (dict(tab=torch.full_like(tab, 10**9)), dict(tab=torch.full_like(tab, -3)), dict(kv=kv + 2**30),
              dict(kv=kv - 2**30), dict(dst=torch.full_like(dst, -1)), dict(dst=torch.full_like(dst, 10**9))):
        y = {**dict(tab=tab, kv=kv, dst=dst), **x}
        m.paged_evict(kc, vc, w, y["tab"], y["kv"], y["dst"], 100, 10)
        assert m.mea_last_device_error() == m.MEA_ERR_PAGE
    # a copy of the page table is not "in place": nothing is written over what is read
    before = [t.clone() for t in (kc, vc, w)]
    m.paged_evict(kc, vc, w, tab, kv, tab.clone(), 100, 10)
    assert m.mea_last_device_error() == m.MEA_ERR_PAGE
    assert all(torch.equal(x, y) for x, y in zip(before, (kc, vc, w)))
    m.paged_evict(kc, vc, w, tab, kv, dst, 100, 10)
    assert m.mea_last_device_error() == m.MEA_OK


def test_evict_many_sequences():
    g = torch.Generator().manual_seed(3)
    lens = torch.randint(0, 120, (700,), generator=g).tolist()
    bt = Batch([0] * 700, lens, 2, 2, 64, 16, BF, seed=10, spare=3000)
    check(bt, 40, 8)
    check(bt, 40, 8, in_place=True)


def test_evict_more_candidates_than_shared_memory_holds():
    """One CTA per head (75 of them) and more candidates than it can keep: the passes read the weights again."""
    heads, L, page, keep = 75, 50001, 256, 30000
    n = -(-L // page)
    k = torch.zeros(n, heads, page, 64, dtype=BF, device="cuda")
    w = torch.rand(n, heads, page, generator=torch.Generator().manual_seed(4))
    w[:, 3] = (w[:, 3] * 4).floor()          # many ties
    k[..., 0] = w.cuda().to(BF)              # a key that tells which one it was
    order = torch.randperm(n, generator=torch.Generator().manual_seed(5)).int()
    table = order.cuda()[None]
    kept, length = m.paged_evict(k, k.clone(), w.clone().cuda(), table, torch.tensor([L], dtype=torch.int32).cuda(), table,
                                 keep, 100)
    assert length.item() == keep and m.mea_last_device_error() == m.MEA_OK
    flat = w[order.long()].permute(1, 0, 2).reshape(heads, -1)[:, :L - 100]
    best = torch.sort(flat, dim=1, descending=True, stable=True)[1][:, :keep - 100].sort(1)[0]
    want = torch.cat([best, torch.arange(L - 100, L).expand(heads, -1)], 1)
    assert torch.equal(kept[0].cpu().long(), want)
    moved = k[order.cuda().long()].permute(1, 0, 2, 3).reshape(heads, -1, 64)[:, :keep, 0].cpu()
    full = w[order.long()].permute(1, 0, 2).reshape(heads, -1).to(BF)
    assert torch.equal(moved, full.gather(1, want))
