"""PagedCache: the page list on the CPU with the fp64 definitions as compute steps, and whole serving runs
(append, attention, weights, eviction together) on the GPU against the same definitions."""

import numpy as np
import pytest
import torch

from exact_memory_efficient_b200.paged import PagedCache
from oracle import paged
from tests._parity import BF16_O, F32_O_MAX_ABS, assert_close
from tests._paged import f64


class OracleOps:
    """The definitions over the cache's own (CPU, fp64) tensors."""

    def append(self, q, k, v, c, cu, kv_len, table, positions):
        q, kc, vc, w = paged.append(f64(q), f64(k), f64(v), f64(c.k), f64(c.v), None if c.weights is None else f64(c.weights),
                                    cu.numpy(), kv_len.numpy(), table.numpy(), positions.numpy(),
                                    None if c.freq is None else c.freq.numpy(), c.interleaved, c.mscale)
        for dst, src in ((c.k, kc), (c.v, vc), (c.weights, w)):
            if dst is not None:
                dst.copy_(torch.from_numpy(src))
        return torch.from_numpy(q)

    def attend(self, q, c, cu, kv_len, table, max_q, max_kv, scale):
        o, lse = paged.attention_paged(f64(q), f64(c.k), f64(c.v), cu.numpy(), kv_len.numpy(), table.numpy(), scale)
        return torch.from_numpy(o), torch.from_numpy(lse)

    def weigh(self, q, lse, c, cu, kv_len, table, max_q, max_kv, scale):
        w = paged.paged_weights(f64(q), f64(lse), f64(c.k), f64(c.weights), cu.numpy(), kv_len.numpy(), table.numpy(), scale)
        c.weights.copy_(torch.from_numpy(w))

    def evict(self, c, table, kv_len, n_keep, n_recent):
        k, v, w, kept, _ = paged.evict(f64(c.k), f64(c.v), f64(c.weights), table.numpy(), kv_len.numpy(), table.numpy(),
                                       n_keep, n_recent)
        for dst, src in ((c.k, k), (c.v, v), (c.weights, w)):
            dst.copy_(torch.from_numpy(src))
        return torch.from_numpy(kept)


def cpu_cache(**kw):
    return PagedCache(**{**dict(num_pages=12, H_kv=2, D=32, page_size=16, dtype=torch.float64, device="cpu",
                                freq=torch.tensor([1.0, 0.1], dtype=torch.float64), ops=OracleOps()), **kw})


def tokens(g, n, H=4, Hkv=2, D=32, dtype=torch.float64):
    return tuple(torch.randn(n, h, D, generator=g).to(dtype) for h in (H, Hkv, Hkv))


def test_pages_are_taken_and_returned():
    c, g = cpu_cache(), torch.Generator().manual_seed(1)
    a, b = c.add(), c.add()
    c.step(*tokens(g, 17 + 3), [a, b], [17, 3])
    assert (c.length(a), c.length(b), c.free_pages) == (17, 3, 9)
    assert len(set(c.pages(a) + c.pages(b))) == 3
    c.step(*tokens(g, 13), [b], [13])               # fills b's page, needs no other
    assert c.free_pages == 9
    c.step(*tokens(g, 1), [b], [1])
    assert c.free_pages == 8
    kept = c.evict([a], 16, 2)
    assert c.length(a) == 16 and c.free_pages == 9 and kept.shape == (1, 2, 16)
    c.remove(a)
    assert c.free_pages == 10
    with pytest.raises(KeyError):
        c.step(*tokens(g, 1), [a], [1])
    d = c.add()
    assert d not in (a, b) and c.length(d) == 0


def test_refusals_change_nothing():
    c, g = cpu_cache(), torch.Generator().manual_seed(2)
    a, b = c.add(), c.add()
    c.step(*tokens(g, 5), [a], [5])
    state = (c.length(a), c.length(b), c.free_pages)
    for error, fn in ((MemoryError, lambda: c.step(*tokens(g, 300), [a], [300])),
                      (ValueError, lambda: c.step(*tokens(g, 4), [a, a], [2, 2])),
                      (ValueError, lambda: c.step(*tokens(g, 4), [a], [3])),
                      (ValueError, lambda: c.step(*tokens(g, 4), [a], [5, -1])),
                      (ValueError, lambda: c.evict([a], 0, 0)), (ValueError, lambda: c.evict([a], 4, 5)),
                      (KeyError, lambda: c.evict([77], 4, 1)),
                      (ValueError, lambda: cpu_cache(bounded=False).evict([], 4, 1))):
        with pytest.raises(error):
            fn()
        assert (c.length(a), c.length(b), c.free_pages) == state


def test_a_failing_step_leaves_the_page_list():
    class Fails(OracleOps):
        def attend(self, *args):
            raise RuntimeError("launch")

    c, g = cpu_cache(ops=Fails()), torch.Generator().manual_seed(7)
    a, b = c.add(), c.add()
    for _ in range(3):
        with pytest.raises(RuntimeError):
            c.step(*tokens(g, 50), [a, b], [33, 17])
        assert (c.length(a), c.length(b), c.free_pages, c.pages(a)) == (0, 0, 12, [])
    c.ops = OracleOps()
    c.step(*tokens(g, 50), [a, b], [33, 17])
    assert len(set(c.pages(a) + c.pages(b))) == 5 and c.free_pages == 7
    c.step(*tokens(g, 0), [b], [0])      # nothing new: nothing changes
    assert c.free_pages == 7


def test_positions_run_on_after_an_eviction():
    """The rotation of the token after an eviction is that of its place in the sequence, not of its slot."""
    c, g = cpu_cache(), torch.Generator().manual_seed(3)
    a = c.add()
    c.step(*tokens(g, 20), [a], [20])
    c.evict([a], 6, 3)
    q, k, v = tokens(g, 1)
    c.step(q, k, v, [a], [1])
    page, off = c.pages(a)[0], 6
    want = paged.rope(f64(k[0])[:, None], [20], c.freq.numpy())[:, 0]
    assert np.abs(f64(c.k[page, :, off]) - want).max() < 1e-12


def test_cache_without_an_eviction_is_causal_attention():
    """Chunks of any size through the cache give the attention of the whole sequence."""
    import oracle
    c, g = cpu_cache(freq=None), torch.Generator().manual_seed(4)
    a = c.add()
    q, k, v = tokens(g, 40)
    outs = [c.step(q[i:j], k[i:j], v[i:j], [a], [j - i])[0] for i, j in ((0, 17), (17, 18), (18, 40))]
    o = f64(torch.cat(outs))
    for t in (0, 5, 16, 17, 18, 39):
        qh = f64(q[t])[None, :, None]
        kh, vh = (f64(x[:t + 1]).transpose(1, 0, 2)[None] for x in (k, v))
        ro, _ = oracle.attention_forward_gqa(qh, kh, vh, 1 / np.sqrt(32))
        assert np.abs(o[t] - ro[0, :, 0]).max() < 1e-12


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,H,Hkv,D,page", [(torch.bfloat16, 8, 2, 128, 16), (torch.bfloat16, 3, 3, 64, 64),
                                                (torch.float32, 4, 2, 64, 32)])
def test_serving_run(dtype, H, Hkv, D, page):
    """Prompts, decode steps, an eviction, more steps, a removal: after every call the cache's tensors are
    read back and the call is repeated by the definitions on them, so that each call is held to its own bounds."""
    import exact_memory_efficient_b200 as m
    freq = m.mea_rope_frequencies(D // 2)
    c = PagedCache(num_pages=1500 // page, H_kv=Hkv, D=D, page_size=page, dtype=dtype, freq=freq)
    g = torch.Generator().manual_seed(5)
    ids = [c.add() for _ in range(3)]

    def step(seqs, counts):
        q, k, v = tokens(g, sum(counts), H, Hkv, D, dtype)
        o, lse = c.step(q.cuda(), k.cuda(), v.cuda(), seqs, counts)
        assert m.mea_last_device_error() == m.MEA_OK
        cu = np.concatenate([[0], np.cumsum(counts)])
        lens = np.array([c.length(s) for s in seqs])
        width = max(len(c.pages(s)) for s in seqs)
        table = np.array([c.pages(s) + [-1] * (width - len(c.pages(s))) for s in seqs])
        pos = np.concatenate([np.arange(c._pos[s] - n, c._pos[s]) for s, n in zip(seqs, counts)])
        # the reference takes the cache as the append left it, and q turned and rounded as it was
        qr = torch.from_numpy(paged.rope(f64(q).transpose(1, 0, 2), pos, freq.numpy())).to(dtype).transpose(0, 1)
        ro, rl = paged.attention_paged(f64(qr), f64(c.k), f64(c.v), cu, lens, table, 1 / np.sqrt(D))
        assert_close(f64(o), ro, *(BF16_O if dtype == torch.bfloat16 else (F32_O_MAX_ABS,)), what="o")
        # q is rounded from fp32 products here and there: a value may fall on the other
        # side of a tie, one bf16 step of q times a key's value and the scale, < 2^-7 * 9 * D^-1/2
        assert np.abs(f64(lse) - rl).max() < (2e-2 if dtype == torch.bfloat16 else 1e-4)

    step(ids, [200, 77, 1])
    for _ in range(3):
        step(ids, [1, 1, 1])
    step([ids[2], ids[0]], [130, 2])
    total = sum(c.weights[p].double().sum() for s in ids for p in c.pages(s))
    # every row so far spread a probability of 1 per query head over the cache
    assert abs(float(total) / (H * (278 + 9 + 132)) - 1) < 1e-4
    lens = [c.length(s) for s in ids]
    before = [t.cpu() for t in (c.k, c.v, c.weights)]
    tables = [c.pages(s) for s in ids]
    kept = c.evict(ids, 100, 20)
    width = max(len(t) for t in tables)
    tab = np.array([t + [-1] * (width - len(t)) for t in tables])
    bits = torch.int16 if dtype == torch.bfloat16 else torch.int32
    rk, rv, rw, rkept, _ = paged.evict(before[0].view(bits).numpy(), before[1].view(bits).numpy(), before[2].numpy(), tab,
                                       np.array(lens), tab, 100, 20)
    assert np.array_equal(kept.cpu().numpy(), rkept) and np.array_equal(c.k.cpu().view(bits).numpy(), rk)
    assert np.array_equal(c.v.cpu().view(bits).numpy(), rv) and np.array_equal(c.weights.cpu().numpy(), rw)
    assert [c.length(s) for s in ids] == [min(x, 100) for x in lens]
    step(ids, [1, 40, 1])
    c.remove(ids[1])
    step([ids[0], ids[2]], [64, 1])
    assert c.free_pages == 1500 // page - len(c.pages(ids[0])) - len(c.pages(ids[2]))
