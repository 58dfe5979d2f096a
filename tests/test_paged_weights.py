"""mea_attn_paged_weights against the fp64 definition (GPU)."""

import math

import numpy as np
import pytest
import torch

import exact_memory_efficient_b200 as m
from oracle import paged
from tests._paged import Batch, f64, weight_bound

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def exact_lse(bt):
    """The fp32 lse that the call gets: the exact one, rounded (rows outside every sequence NaN)."""
    return torch.from_numpy(paged.attention_paged(*bt.np("q", "k_cache", "v_cache"), bt.cu.numpy(), bt.kv_len.numpy(),
                                                  bt.table.numpy(), bt.scale)[1]).float()


def check(bt, lse, got):
    assert m.mea_last_device_error() == m.MEA_OK
    q, kc, w = bt.np("q", "k_cache", "weights")
    want = paged.paged_weights(q, f64(lse), kc, w, bt.cu.numpy(), bt.kv_len.numpy(), bt.table.numpy(), bt.scale)
    err = np.abs(f64(got) - want)
    tol = weight_bound(bt, q, f64(lse), want)
    assert (err <= tol).all(), (err / tol).max()
    untouched = want == w
    assert np.array_equal(f64(got)[untouched], w[untouched])


def run(bt, lse, q=None, max_q=None, max_kv=None):
    kc, w, cu, kv, tab = bt.gpu("k_cache", "weights", "cu", "kv_len", "table")
    mq, mk = bt.max_q if max_q is None else max_q, bt.max_kv if max_kv is None else max_kv
    n = m.mea_attn_paged_weights_workspace_size(bt.T, len(bt.lens), bt.H, bt.Hkv, bt.D, mq, mk, bt.dtype)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda") if n else None    # garbage: NaN
    m.mea_attn_paged_weights(bt.q.cuda() if q is None else q, lse.cuda(), kc, w, cu, kv, tab, mq, mk, bt.scale, ws)
    return w


@pytest.mark.parametrize("dtype,counts,lens,H,Hkv,D,page", [
    (BF, [1], [1], 1, 1, 64, 16), (BF, [1, 1, 1], [17, 128, 900], 8, 2, 128, 16), (BF, [1, 1], [129, 3000], 5, 1, 64, 64),
    (BF, [40, 1, 0], [100, 257, 30], 6, 3, 64, 32), (BF, [128], [128], 2, 2, 128, 128), (BF, [200], [500], 4, 4, 128, 256),
    (BF, [130, 33], [130, 400], 8, 1, 64, 16), (BF, [300], [700], 7, 1, 128, 16), (BF, [65], [66], 14, 2, 128, 64),
    (F32, [1], [1], 2, 1, 32, 16), (F32, [1, 1], [900, 64], 8, 8, 64, 64), (F32, [30, 5], [77, 300], 6, 2, 96, 16),
    (F32, [70], [70], 4, 1, 128, 32),
])
def test_weights(dtype, counts, lens, H, Hkv, D, page):
    bt = Batch(counts, lens, H, Hkv, D, page, dtype, seed=sum(lens), front=1, behind=2)
    lse = exact_lse(bt)
    check(bt, lse, run(bt, lse))


@pytest.mark.parametrize("counts,lens,H,Hkv,D,page", [
    ([1500], [1500], 2, 1, 64, 16), ([2000], [2040], 4, 1, 128, 64), ([1] * 33, [i * 37 % 300 for i in range(33)], 4, 2, 128, 16),
    ([i % 3 for i in range(610)], [i * 13 % 60 for i in range(610)], 2, 1, 64, 16),
])
def test_many_parts_and_many_sequences(counts, lens, H, Hkv, D, page):
    """An item's units spread over tens of SMs; batches beyond a warp's and a block's threads."""
    bt = Batch(counts, lens, H, Hkv, D, page, BF, seed=22)
    lse = exact_lse(bt)
    check(bt, lse, run(bt, lse))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_that_see_nothing_add_nothing(dtype):
    bt = Batch([5, 40, 1], [2, 17, 0], 4, 2, 64, 16, dtype, seed=3)
    lse = exact_lse(bt)
    assert torch.isneginf(lse).any()
    check(bt, lse, run(bt, lse))


@pytest.mark.parametrize("garbage", [math.nan, math.inf])
@pytest.mark.parametrize("dtype,page", [(BF, 16), (BF, 32), (BF, 128), (BF, 256), (F32, 32), (F32, 256)])
def test_garbage_behind_the_sequences(dtype, page, garbage):
    bt = Batch([1, 70, 3], [65, 130, 40], 4, 2, 128, page, dtype, seed=4, garbage=garbage, front=1, behind=2)
    bt.q[0] = garbage
    bt.q[-2:] = garbage
    lse = exact_lse(bt)
    check(bt, lse, run(bt, lse))


def test_strided_rows_loose_bounds_and_bits():
    bt = Batch([90, 7], [95, 800], 8, 2, 64, 16, BF, seed=5)
    lse = exact_lse(bt)
    want = run(bt, lse)
    row = torch.cat([bt.q.flatten(1), torch.full((bt.T, 40), math.nan, dtype=BF)], 1).cuda()
    assert torch.equal(want, run(bt, lse, q=row[:, :512].view(-1, 8, 64)))
    for max_q, max_kv in ((0, 0), (1, 1), (1, 10**6), (10**6, 1)):
        check(bt, lse, run(bt, lse, max_q=max_q, max_kv=max_kv))


def test_sums_of_a_call_are_its_rows():
    """Every row's probabilities sum to one: with the library's own lse, the weights of a call sum to the
    rows it has, to the error of the exponentials (2^-21 relative and the lse bound, both below 1e-4)."""
    bt = Batch([100, 1, 20], [1000, 512, 20], 8, 2, 64, 16, BF, seed=6)
    q, kc, vc, cu, kv, tab = bt.gpu("q", "k_cache", "v_cache", "cu", "kv_len", "table")
    _, lse = m.attention_paged(q, kc, vc, cu, kv, tab, bt.max_q, bt.max_kv)
    w = torch.zeros(bt.pages, 2, 16, device="cuda")
    m.attention_paged_weights(q, lse, kc, w, cu, kv, tab, bt.max_q, bt.max_kv)
    assert abs(float(w.double().sum()) / (121 * 8) - 1) < 1e-4


def test_graph_replay_and_bad_tables():
    bt = Batch([1, 60], [300, 90], 4, 2, 64, 16, BF, seed=7)
    lse = exact_lse(bt)
    want = run(bt, lse)
    q, kc, w, cu, kv, tab, l2 = *bt.gpu("q", "k_cache", "weights", "cu", "kv_len", "table"), lse.cuda()
    call = lambda tab=tab, kv=kv, cu=cu: m.attention_paged_weights(q, l2, kc, w, cu, kv, tab, 60, 300)  # noqa: E731
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        call()
    w.copy_(bt.weights)
    graph.replay()
    assert torch.equal(w, want)
    for x in (dict(tab=torch.full_like(tab, 10**9)), dict(tab=torch.full_like(tab, -7)), dict(kv=kv + 2**30),
              dict(kv=kv - 2**30), dict(cu=cu + 2**30), dict(cu=cu.flip(0).contiguous() + 5)):
        call(**x)
        st = m.mea_last_device_error()
        assert st == m.MEA_ERR_PAGE or ("cu" in x and st == m.MEA_OK)


def test_many_sequences():
    g = torch.Generator().manual_seed(14)
    lens = torch.randint(1, 70, (900,), generator=g).tolist()
    lens[417] = 2000
    counts = [min(n, int(c)) for n, c in zip(lens, torch.randint(0, 4, (900,), generator=g))]
    counts[417] = 300
    for c in (counts, [1] * 900):
        bt = Batch(c, lens, 4, 2, 64, 16, BF, seed=15)
        lse = exact_lse(bt)
        check(bt, lse, run(bt, lse))


@pytest.mark.parametrize("dtype,G,D", [(BF, 128, 64), (BF, 130, 64), (BF, 43, 128), (F32, 20, 32)])
def test_large_groups(dtype, G, D):
    bt = Batch([1, 3], [200, 131], 2 * G, 2, D, 32, dtype, seed=17)
    lse = exact_lse(bt)
    check(bt, lse, run(bt, lse))


@pytest.mark.parametrize("scale", [0.0, -0.125])
def test_scale_of_zero_and_below(scale):
    for counts, lens in (([1, 1], [300, 45]), ([140, 3], [150, 45])):
        bt = Batch(counts, lens, 4, 2, 64, 16, BF, seed=18)
        bt.scale = scale
        lse = exact_lse(bt)
        got = run(bt, lse)
        q, kc, w = bt.np("q", "k_cache", "weights")
        want = paged.paged_weights(q, f64(lse), kc, w, bt.cu.numpy(), bt.kv_len.numpy(), bt.table.numpy(), scale)
        bt.scale = abs(scale)      # the bound takes magnitudes, against the exact lse of either sign
        tol = weight_bound(bt, q if scale >= 0 else -q, f64(lse), want)
        assert (np.abs(f64(got) - want) <= tol).all()


def test_bits_do_not_depend_on_the_run():
    bt = Batch([900, 1], [1500, 3000], 8, 2, 128, 64, BF, seed=19)
    lse = torch.zeros(bt.T, 8)
    a = run(bt, lse)
    for _ in range(3):
        assert torch.equal(a, run(bt, lse))
