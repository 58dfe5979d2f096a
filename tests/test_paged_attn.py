"""mea_attn_paged against the fp64 definition (GPU): every type and head dim, ragged chunks, decode, rows
that see nothing, garbage behind the sequences, page sizes, strides, graphs, streams, bad tables."""

import math

import numpy as np
import pytest
import torch

import exact_memory_efficient_b200 as m
from oracle import paged
from tests._paged import Batch, f64
from tests._parity import BF16_O, F32_O_MAX_ABS, assert_close, lse_tolerance

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def run(bt, q=None, max_q=None, max_kv=None, stream=None):
    kc, vc, cu, kv, tab = bt.gpu("k_cache", "v_cache", "cu", "kv_len", "table")
    q = bt.q.cuda() if q is None else q
    o = torch.full((bt.T, bt.H, bt.D), 7.0, dtype=bt.dtype, device="cuda")
    lse = torch.full((bt.T, bt.H), 7.0, device="cuda")
    mq, mk = bt.max_q if max_q is None else max_q, bt.max_kv if max_kv is None else max_kv
    n = m.mea_attn_paged_workspace_size(bt.T, len(bt.lens), bt.H, bt.Hkv, bt.D, mq, mk, bt.dtype)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda") if n else None    # garbage: NaN
    m.mea_attn_paged(q, kc, vc, o, lse, cu, kv, tab, mq, mk, bt.scale, ws, stream)
    return o, lse


def check(bt, got):
    assert m.mea_last_device_error() == m.MEA_OK
    o, lse = (f64(t) for t in got)
    q, kc, vc = bt.np("q", "k_cache", "v_cache")
    ro, rl = paged.attention_paged(q, kc, vc, bt.cu.numpy(), bt.kv_len.numpy(), bt.table.numpy(), bt.scale)
    rows = np.zeros(bt.T, dtype=bool)
    rows[list(bt.used_rows)] = True
    assert (o[~rows] == 7.0).all() and (lse[~rows] == 7.0).all()
    empty = np.isneginf(rl)
    assert np.array_equal(np.isneginf(lse)[rows], empty[rows])
    assert (o[rows][empty[rows]] == 0).all()
    if rows.any():
        if bt.dtype == BF:
            assert_close(o[rows], ro[rows], *BF16_O, what="O")
        else:
            assert_close(o[rows], ro[rows], F32_O_MAX_ABS, what="O")
    for b, n in enumerate(bt.counts):
        c = int(bt.cu[b])
        if n == 0 or bt.lens[b] == 0:
            continue
        k = bt.gathered_k(b)
        for h in range(bt.H):
            e = ~empty[c:c + n, h]
            tol = lse_tolerance(q[c:c + n, h], k[:, h // (bt.H // bt.Hkv)], bt.scale, rl[c:c + n, h])
            assert (np.abs(lse[c:c + n, h][e] - rl[c:c + n, h][e]) <= tol[e]).all()


SHAPES = [
    # counts, lens, H, Hkv, D, page
    ([1], [1], 1, 1, 64, 16), ([1], [1], 8, 2, 128, 16), ([1, 1, 1, 1], [1, 15, 16, 17], 4, 4, 128, 16),
    ([1] * 5, [63, 64, 65, 500, 129], 8, 2, 64, 32), ([1, 1], [3000, 5], 32, 8, 128, 16), ([1], [4097], 6, 1, 128, 64),
    ([1, 1], [700, 1300], 15, 3, 64, 128), ([2, 3], [200, 77], 8, 8, 128, 16), ([4], [127], 12, 4, 64, 256),
    # chunks
    ([128], [128], 2, 2, 64, 64), ([129], [129], 2, 2, 128, 16), ([100, 1, 57], [100, 300, 257], 4, 1, 128, 32),
    ([31, 33, 32], [600, 33, 129], 8, 2, 64, 16), ([256], [1000], 3, 3, 128, 128), ([300], [301], 5, 1, 64, 256),
    ([17, 0, 40, 0], [900, 12, 40, 0], 16, 2, 128, 64), ([65, 64], [65, 1999], 14, 2, 128, 16), ([50], [700], 7, 1, 64, 16),
    ([385, 130], [385, 513], 2, 1, 128, 32),
]


@pytest.mark.parametrize("counts,lens,H,Hkv,D,page", SHAPES)
def test_attention_bf16(counts, lens, H, Hkv, D, page):
    bt = Batch(counts, lens, H, Hkv, D, page, BF, seed=sum(lens) + H)
    check(bt, run(bt))


@pytest.mark.parametrize("counts,lens,H,Hkv,D,page", [
    ([1], [1], 2, 1, 32, 16), ([1, 1], [3000, 77], 8, 8, 64, 64), ([1], [2500], 6, 3, 96, 16), ([1, 1], [64, 65], 8, 1, 128, 32),
    ([5, 40], [70, 40], 4, 2, 64, 16), ([33], [900], 5, 1, 128, 128), ([9, 1, 20], [9, 300, 64], 2, 2, 32, 256),
    ([17], [161], 3, 1, 96, 16),
])
def test_attention_f32(counts, lens, H, Hkv, D, page):
    bt = Batch(counts, lens, H, Hkv, D, page, F32, seed=sum(lens) + H)
    check(bt, run(bt))


@pytest.mark.parametrize("counts,lens,H,Hkv,D,page", [
    ([1], [19000], 4, 1, 128, 64), ([70], [19000], 2, 1, 64, 16), ([3, 1], [9500, 9400], 5, 1, 64, 128),
    ([1] * 33, [i * 37 % 300 for i in range(33)], 4, 2, 128, 16),
    ([i % 3 for i in range(330)], [i * 13 % 60 for i in range(330)], 2, 1, 64, 16),
])
def test_many_parts_and_many_sequences(counts, lens, H, Hkv, D, page):
    """An item cut into about as many parts as there are SMs; batches beyond a warp's and a block's threads."""
    bt = Batch(counts, lens, H, Hkv, D, page, BF, seed=21)
    check(bt, run(bt))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("counts,lens", [([4, 1, 3], [2, 0, 50]), ([40, 300], [0, 170]), ([1, 1], [0, 3])])
def test_rows_that_see_no_key(dtype, counts, lens):
    """kv_len below the number of new tokens: the first rows have no key."""
    bt = Batch(counts, lens, 4, 2, 64, 16, dtype, seed=1, max_pages=12)
    check(bt, run(bt))


@pytest.mark.parametrize("garbage", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("dtype,page", [(BF, 16), (BF, 32), (BF, 128), (BF, 256), (F32, 32), (F32, 256)])
def test_garbage_behind_the_sequences(dtype, page, garbage):
    """Free pages and the slots behind a sequence's last key may hold anything; rows outside every sequence too."""
    for counts, lens in (([1, 1, 1, 1], [17, 65, 300, 200]), ([130, 5, 60, 260], [131, 77, 60, 330])):
        bt = Batch(counts, lens, 4, 2, 128, page, dtype, seed=2, garbage=garbage, front=1, behind=2)
        bt.q[0] = garbage
        bt.q[-2:] = garbage
        check(bt, run(bt))


@pytest.mark.parametrize("mult", [8.0, 40.0])
def test_large_scores(mult):
    """Scores up to about a thousand (a spread softmax and a nearly one-hot one): nothing overflows."""
    for counts, lens in (([1, 1], [900, 2000]), ([150], [400])):
        bt = Batch(counts, lens, 4, 2, 64, 16, F32, seed=3, mult=mult ** 0.5)
        o, lse = (f64(t) for t in run(bt))
        q, kc, vc = bt.np("q", "k_cache", "v_cache")
        ro, rl = paged.attention_paged(q, kc, vc, bt.cu.numpy(), bt.kv_len.numpy(), bt.table.numpy(), bt.scale)
        # a score s has an error of at most 64 u sum |q k| scale, which moves o by that much relative
        assert np.abs(lse - rl).max() < 1e-4 + 64 * 2.0**-24 * np.abs(rl).max() * 8
        assert np.abs(o - ro).max() < 64 * 2.0**-24 * np.abs(rl).max() * 8 * 4 + 1e-5


@pytest.mark.parametrize("counts,lens", [([1, 1], [2000, 700]), ([200], [1500])])
def test_rising_scores(counts, lens):
    """Scores that grow along the keys move the running maximum again and again."""
    bt = Batch(counts, lens, 4, 2, 128, 16, BF, seed=4)
    bt.q = torch.full_like(bt.q, 0.25)
    for b, L in enumerate(lens):
        j = torch.arange(L)
        ramp = torch.linspace(-1, 1, L) * 4
        bt.k_cache[bt.table[b, j // 16].long(), :, j % 16] = ramp[:, None, None].expand(-1, 2, 128).to(BF)
    bt.scale = 1.0
    check(bt, run(bt))


def test_strided_rows_and_loose_bounds():
    """q as a slice of a projection; max_q and max_kv only choose the launch: any value is right."""
    for counts, lens in (([1, 1, 1], [600, 33, 1]), ([90, 7], [95, 800])):
        bt = Batch(counts, lens, 8, 2, 64, 16, BF, seed=5)
        row = torch.cat([bt.q.flatten(1), torch.full((bt.T, 40), math.nan, dtype=BF)], 1).cuda()
        q = row[:, :512].view(-1, 8, 64)
        check(bt, run(bt, q=q))
        for max_q, max_kv in ((0, 0), (1, 1), (1, 10**6), (10**6, 1), (10**6, 10**6), (2, 64)):
            check(bt, run(bt, max_q=max_q, max_kv=max_kv))


def test_shared_prefix_pages():
    """Two sequences that read the same first pages."""
    bt = Batch([1, 30], [100, 130], 4, 2, 64, 16, BF, seed=6)
    bt.table[1, :4] = bt.table[0, :4]
    check(bt, run(bt))


def test_deterministic_and_two_streams():
    bt = Batch([1, 200, 1], [3000, 900, 77], 8, 2, 128, 16, BF, seed=7)
    want = run(bt)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    q, kc, vc, cu, kv, tab = bt.gpu("q", "k_cache", "v_cache", "cu", "kv_len", "table")
    torch.cuda.synchronize()
    outs = []
    for _ in range(4):   # two calls at once, each with a workspace of its own
        for s in (s1, s2):
            outs.append(m.attention_paged(q, kc, vc, cu, kv, tab, bt.max_q, bt.max_kv, bt.scale, stream=s))
    torch.cuda.synchronize()
    for o, lse in outs:
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    assert m.mea_last_device_error() == m.MEA_OK


@pytest.mark.parametrize("first,second", [(([1, 1, 1], [700, 100, 20]), ([1, 1, 1], [90, 701, 400])),
                                          (([60, 1, 40], [700, 100, 40]), ([1, 99, 1], [300, 99, 650]))])
def test_graph_replay_with_other_lengths(first, second):
    """A captured call replayed with other lengths, offsets, tables and values in the same buffers."""
    a = Batch(*first, 8, 2, 128, 16, BF, seed=8, max_pages=64, spare=100)
    b = Batch(*second, 8, 2, 128, 16, BF, seed=9, max_pages=64, spare=100)
    pages = max(a.pages, b.pages)
    grow = lambda t: torch.cat([t, torch.zeros(pages - t.shape[0], *t.shape[1:], dtype=t.dtype)])  # noqa: E731
    for bt in (a, b):
        bt.k_cache, bt.v_cache = grow(bt.k_cache), grow(bt.v_cache)
    assert a.T == b.T
    q, kc, vc, cu, kv, tab = a.gpu("q", "k_cache", "v_cache", "cu", "kv_len", "table")
    o, lse = torch.empty_like(q), torch.empty(a.T, 8, device="cuda")
    n = m.mea_attn_paged_workspace_size(a.T, 3, 8, 2, 128, 99, 1024)
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    call = lambda: m.mea_attn_paged(q, kc, vc, o, lse, cu, kv, tab, 99, 1024, a.scale, ws)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for bt in (b, a):
        for dst, src in ((q, bt.q), (kc, bt.k_cache), (vc, bt.v_cache), (cu, bt.cu), (kv, bt.kv_len), (tab, bt.table)):
            dst.copy_(src.cuda())
        graph.replay()
        check(bt, (o, lse))


def test_workspace_errors():
    bt = Batch([1], [4000], 8, 8, 128, 16, BF)
    q, kc, vc, cu, kv, tab = bt.gpu("q", "k_cache", "v_cache", "cu", "kv_len", "table")
    o, lse = torch.empty_like(q), torch.empty(1, 8, device="cuda")
    n = m.mea_attn_paged_workspace_size(1, 1, 8, 8, 128, 1, 4000)
    assert n > 0
    for ws, status in ((None, m.MEA_ERR_WORKSPACE), (torch.empty(n - 16, dtype=torch.uint8, device="cuda"), m.MEA_ERR_WORKSPACE),
                       (torch.empty(n + 16, dtype=torch.uint8, device="cuda")[8:], m.MEA_ERR_MISALIGNED)):
        with pytest.raises(m.MeaError) as e:
            m.mea_attn_paged(q, kc, vc, o, lse, cu, kv, tab, 1, 4000, 1.0, ws)
        assert e.value.status == status
    with pytest.raises(m.MeaError) as e:
        m.mea_attn_paged(q, kc, vc, o, lse, cu, kv, tab.long(), 1, 4000, 1.0, None)
    assert e.value.status == m.MEA_ERR_INVALID_ARG


def test_bad_tables_are_reported():
    """Pages, lengths and offsets out of range cost no access outside the buffers, and are reported."""
    for dtype in (BF, F32):
        bt = Batch([4, 90], [12, 290], 4, 2, 64, 16, dtype, seed=13)
        q, kc, vc, cu, kv, tab = bt.gpu("q", "k_cache", "v_cache", "cu", "kv_len", "table")
        bad = tab.clone()
        bad[1, 5] = 10**9
        call = lambda cu=cu, kv=kv, tab=tab: m.attention_paged(q, kc, vc, cu, kv, tab, 90, 290)  # noqa: E731
        for x in (dict(tab=bad), dict(tab=torch.full_like(tab, -7)), dict(kv=kv + 2**30), dict(kv=kv - 2**30),
                  dict(cu=cu + 2**30), dict(cu=cu.flip(0).contiguous() + 5)):
            call(**x)
            st = m.mea_last_device_error()
            assert st == m.MEA_ERR_PAGE or ("cu" in x and st == m.MEA_OK)
        check(bt, run(bt))


def test_many_sequences():
    """More sequences than a CTA has threads, most of them short, some without new tokens."""
    g = torch.Generator().manual_seed(14)
    lens = torch.randint(1, 70, (900,), generator=g).tolist()
    lens[417] = 2000
    counts = [min(n, int(c)) for n, c in zip(lens, torch.randint(0, 4, (900,), generator=g))]
    counts[417] = 300
    bt = Batch(counts, lens, 4, 2, 64, 16, BF, seed=15)
    check(bt, run(bt))
    bt = Batch([1] * 900, lens, 4, 2, 64, 16, BF, seed=16)
    check(bt, run(bt))


@pytest.mark.parametrize("dtype,G,D", [(BF, 128, 64), (BF, 130, 64), (BF, 43, 128), (F32, 20, 32)])
def test_large_groups(dtype, G, D):
    """Groups up to a whole query tile, and beyond one (the CUDA-core kernel takes those)."""
    bt = Batch([1, 3], [200, 131], 2 * G, 2, D, 32, dtype, seed=17)
    check(bt, run(bt))


@pytest.mark.parametrize("scale", [0.0, -0.125, -3.0])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_scale_of_zero_and_below(dtype, scale):
    for counts, lens in (([1, 1], [300, 45]), ([140, 3], [150, 45])):
        bt = Batch(counts, lens, 4, 2, 64, 16, dtype, seed=18)
        bt.scale = scale
        check(bt, run(bt))


def test_nothing_to_do():
    bt = Batch([2], [20], 4, 2, 64, 16, BF)
    q, kc, vc, cu, kv, tab = bt.gpu("q", "k_cache", "v_cache", "cu", "kv_len", "table")
    o, lse = m.attention_paged(q[:0], kc, vc, cu * 0, kv, tab, 0, 20)
    assert o.shape == (0, 4, 64) and lse.shape == (0, 4)
    o, lse = m.attention_paged(q, kc, vc, cu[:1].contiguous(), kv[:0], tab[:0], 0, 0)     # no sequences
    assert o.shape == q.shape


def test_one_row_with_any_stride():
    """A single row's token stride means nothing."""
    bt = Batch([1], [77], 4, 2, 64, 16, BF, seed=19)
    q = torch.as_strided(bt.q.cuda(), (1, 4, 64), (1, 64, 1))
    check(bt, run(bt, q=q))


@pytest.mark.parametrize("dtype,D", [(BF, 128), (F32, 64)])
def test_offsets_beyond_32_bits(dtype, D):
    """A cache of more than 2^32 elements whose sequences lie at its end: append, attention, weights, eviction."""
    counts, lens, H, Hkv, page = [1, 70], [300, 90], 4, 2, 256
    bt = Batch(counts, lens, H, Hkv, D, page, dtype, seed=20, spare=4)
    pages = (1 << 32) // (Hkv * page * D) + 40
    shift = pages - bt.pages
    big = []
    for t in (bt.k_cache, bt.v_cache):
        x = torch.empty(pages, Hkv, page, D, dtype=dtype, device="cuda")
        x[shift:] = t.cuda()
        big.append(x)
    assert big[0].numel() > 1 << 32
    w = torch.zeros(pages, Hkv, page, device="cuda")
    w[shift:] = bt.weights.cuda()
    table = torch.where(bt.table >= 0, bt.table + shift, bt.table).int()
    q, k, v, cu, kv = bt.gpu("q", "k", "v", "cu", "kv_len")
    m.paged_append(None, k, v, *big, w, cu, kv, table.cuda())
    o, lse = m.attention_paged(q, *big, cu, kv, table.cuda(), 70, 300, bt.scale)
    m.attention_paged_weights(q, lse, big[0], w, cu, kv, table.cuda(), 70, 300, bt.scale)
    _, kc, vc, wa = paged.append(None, *bt.np("k", "v", "k_cache", "v_cache", "weights"), bt.cu.numpy(),
                                 bt.kv_len.numpy(), bt.table.numpy())
    bt.k_cache, bt.v_cache = torch.from_numpy(kc).to(dtype), torch.from_numpy(vc).to(dtype)
    check(bt, (o, lse))
    want = paged.paged_weights(bt.np("q")[0], f64(lse), kc, wa, bt.cu.numpy(), bt.kv_len.numpy(), bt.table.numpy(),
                               bt.scale)
    assert np.abs(f64(w[shift:]) - want).max() < 1e-3
    before = [x[shift:].cpu().float().numpy() for x in (*big, w)]
    pages = table.cuda()          # in place: the same tensor twice, a copy of it is refused
    kept, n = m.paged_evict(*big, w, pages, kv, pages, 64, 16)
    assert m.mea_last_device_error() == 0
    ref = paged.evict(*before, bt.table.numpy(), bt.kv_len.numpy(), bt.table.numpy(), 64, 16)
    assert np.array_equal(kept.cpu().numpy(), ref[3]) and n.tolist() == [64, 64]
    for x, r in zip((*big, w), ref):
        assert np.array_equal(x[shift:].cpu().float().numpy(), r)
    assert m.mea_last_device_error() == m.MEA_OK
