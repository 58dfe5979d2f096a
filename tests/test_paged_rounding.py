"""Roundings of bf16 attention over a paged cache (GPU): what decode keeps of a probability."""

import numpy as np
import pytest
import torch

import exact_memory_efficient_b200 as m
from oracle import paged
from tests._paged import Batch, f64
from tests.test_paged_attn import run

BF = torch.bfloat16


def two_heavy_keys(lens, H, Hkv, D, page, places, counts=None):
    """Two keys per sequence and key/value head carry everything, with the probabilities 1 and x of about 0.7 before
    they are divided by their sum; the values -x rounded to bf16, and 1.  The output is what the rounding of x leaves: with
    x itself in bf16 it would be 0.  All other keys score 60 below: e^-60 of their values is far below the bound."""
    bt = Batch(counts or [1] * len(lens), lens, H, Hkv, D, page, BF, seed=17)
    bt.scale = 1.0
    bt.q.zero_()
    bt.q[..., 0] = 1.0
    g = torch.Generator().manual_seed(18)
    for b, (L, (i, j)) in enumerate(zip(lens, places)):
        at = torch.arange(L)
        p, f = bt.table[b, at // page].long(), at % page
        bt.k_cache[p, :, f] = 0.0
        bt.k_cache[p, :, f, 0] = -60.0
        low = (-0.3 - 0.1 * torch.rand(Hkv, generator=g)).to(BF)
        bt.k_cache[p[i], :, f[i], 0] = 0.0
        bt.k_cache[p[j], :, f[j], 0] = low
        x = torch.exp(low.double())
        bt.v_cache[p[i], :, f[i]] = -x.to(BF)[:, None].expand(Hkv, D)
        bt.v_cache[p[j], :, f[j]] = 1.0
    return bt


@pytest.mark.gpu
@pytest.mark.parametrize("lens,H,Hkv,D,page,places", [
    ([2, 40], 4, 4, 128, 16, [(0, 1), (3, 39)]),
    ([500, 77, 129], 8, 2, 128, 16, [(2, 499), (76, 0), (127, 128)]),
    ([3000], 16, 1, 64, 64, [(1, 2999)]), ([3000, 200], 8, 1, 64, 256, [(2900, 5), (150, 20)]),
    ([8000, 30], 4, 1, 128, 32, [(100, 7900), (1, 2)]),
])
def test_decode_keeps_more_than_bf16_of_a_probability(lens, H, Hkv, D, page, places):
    """Bound: a probability p is two bf16 terms.  The first leaves at most 2^-8 p (half a step), the second at most 2^-8
    of that: 2^-16 p.  Its exponential is off by 2^-22 and 3 u of the score (below 1: 2^-22), the two products' fp32 sum
    by 2^-23 of each and the merge of parts by a few u: 2^-19 in all.  So |o - exact| <= (2^-16 + 2^-19) sum |p v| / sum p,
    which is at most 1, and half a step of the result, 2^-8 |o|."""
    bt = two_heavy_keys(lens, H, Hkv, D, page, places)
    o, lse = run(bt)
    assert m.mea_last_device_error() == m.MEA_OK
    ro, _ = paged.attention_paged(*bt.np("q", "k_cache", "v_cache"), bt.cu.numpy(), bt.kv_len.numpy(), bt.table.numpy(), 1.0)
    tol = torch.finfo(BF).eps / 2 * np.abs(ro) + 2.0 ** -16 + 2.0 ** -19
    assert (np.abs(ro) > 4 * 2.0 ** -16).any()    # one term would give 0
    assert (np.abs(f64(o) - ro) <= tol).all(), (np.abs(f64(o) - ro) / tol).max()
