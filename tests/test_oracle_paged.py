"""Pins of the fp64 definitions in oracle/paged.py: closed forms, complex products, differences, and
agreement with the contiguous oracle (CPU)."""

import math

import numpy as np
import pytest

import oracle
from oracle import paged
from tests._paged import Batch, f64

import torch


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_is_a_product_of_complex_numbers(interleaved):
    rng = np.random.default_rng(1)
    x, pos, freq = rng.normal(size=(2, 5, 12)), np.array([0, 1, -3, 7, 100000]), np.array([1.0, 0.1, 0.03, 0.002])
    y = paged.rope(x, pos, freq, interleaved, 1.5)
    z = x[..., 0:8:2] + 1j * x[..., 1:8:2] if interleaved else x[..., :4] + 1j * x[..., 4:8]
    z = z * 1.5 * np.exp(1j * pos[:, None] * freq)
    got = y[..., 0:8:2] + 1j * y[..., 1:8:2] if interleaved else y[..., :4] + 1j * y[..., 4:8]
    assert np.abs(got - z).max() < 1e-12
    assert np.array_equal(y[..., 8:], x[..., 8:])


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_inverse_is_the_gradient(interleaved):
    """<dy, R x> = <R^T dy, x> for every x, and a central difference of the loss."""
    rng = np.random.default_rng(2)
    x, dy = rng.normal(size=(4, 8)), rng.normal(size=(4, 8))
    pos, freq = np.arange(4) * 5 + 2, np.array([0.9, 0.2, 0.01])
    dx = paged.rope(dy, pos, freq, interleaved, 0.8, inverse=True)
    if True:
        e, num = 1e-6, np.zeros_like(x)
        for i in np.ndindex(*x.shape):
            hi, lo = x.copy(), x.copy()
            hi[i] += e
            lo[i] -= e
            num[i] = ((paged.rope(hi, pos, freq, interleaved, 0.8) - paged.rope(lo, pos, freq, interleaved, 0.8))[:, :6]
                      * dy[:, :6]).sum() / (2 * e)
        assert np.abs(num[:, :6] - dx[:, :6]).max() < 1e-8
    assert np.array_equal(dx[:, 6:], dy[:, 6:])


def test_attention_over_pages_is_attention_over_the_gathered_keys():
    bt = Batch([1, 4, 0], [21, 40, 7], 6, 2, 64, 16, torch.float32, seed=3)
    q, kc, vc = bt.np("q", "k_cache", "v_cache")
    o, lse = paged.attention_paged(q, kc, vc, bt.cu.numpy(), bt.kv_len.numpy(), bt.table.numpy(), bt.scale)
    for b in range(3):
        p, f = paged.slots(bt.table.numpy()[b], bt.lens[b], 16)
        for i in range(bt.counts[b]):
            t, seen = int(bt.cu[b]) + i, bt.lens[b] - bt.counts[b] + i + 1
            k, v = (x[p, :, f][:seen].transpose(1, 0, 2)[None] for x in (kc, vc))
            ro, rl = oracle.attention_forward_gqa(q[t][None, :, None], k, v, bt.scale)
            assert np.abs(o[t] - ro[0, :, 0]).max() < 1e-12 and np.abs(lse[t] - rl[0, :, 0]).max() < 1e-12


def test_rows_without_a_key_and_without_a_sequence():
    bt = Batch([3], [2], 2, 1, 64, 16, torch.float32, front=1, behind=2)
    o, lse = paged.attention_paged(*bt.np("q", "k_cache", "v_cache"), bt.cu.numpy(), bt.kv_len.numpy(),
                                   bt.table.numpy(), bt.scale)
    assert (o[1] == 0).all() and (lse[1] == -math.inf).all()      # the first of three tokens has no slot
    assert np.isfinite(o[2:4]).all()
    assert np.isnan(o[[0, 4, 5]]).all()


def test_weights_of_a_call_sum_to_its_rows():
    bt = Batch([5, 2], [30, 9], 4, 2, 64, 16, torch.float32, seed=5)
    args = (bt.cu.numpy(), bt.kv_len.numpy(), bt.table.numpy(), bt.scale)
    q, kc, vc = bt.np("q", "k_cache", "v_cache")
    _, lse = paged.attention_paged(q, kc, vc, *args)
    w = paged.paged_weights(q, lse, kc, np.zeros(kc.shape[:3]), *args)
    assert abs(w.sum() - 7 * 4) < 1e-9      # every row's probabilities sum to 1
    w2 = paged.paged_weights(q, lse, kc, np.ones(kc.shape[:3]), *args)
    assert np.abs(w2 - 1 - w).max() < 1e-12


def test_append_puts_tokens_into_their_slots():
    bt = Batch([2, 1], [17, 5], 2, 2, 64, 16, torch.float32, seed=6)
    freq = paged_freq = np.array([1.0, 0.5])
    q, k, v, kc, vc, w = bt.np("q", "k", "v", "k_cache", "v_cache", "weights")
    qo, ko, vo, wo = paged.append(q, k, v, kc, vc, w, bt.cu.numpy(), bt.kv_len.numpy(), bt.table.numpy(),
                                  freq=paged_freq)
    page = bt.table.numpy()[0, 1]
    assert np.array_equal(vo[page, :, 0], v[1]) and (wo[page, :, 0] == 0).all()
    assert np.allclose(ko[page, :, 0], paged.rope(k[1][:, None], [16], freq)[:, 0])
    assert np.allclose(qo[0], paged.rope(q[0][:, None], [15], freq)[:, 0])
    changed = (ko != kc).any(axis=(1, 3)).sum()
    assert changed == 3      # three slots


def test_evict_keeps_heavy_and_recent_in_order():
    kc = np.arange(2 * 16, dtype=np.float64).reshape(2, 1, 16, 1)
    w = np.zeros((2, 1, 16))
    w[0, 0, :10] = [5, 1, 7, 7, 0, 7, 2, np.nan, 3, 9]
    k, v, ww, kept, n = paged.evict(kc, kc * 2, w, np.array([[0]]), np.array([10]), np.array([[1]]), 5, 2)
    assert kept.tolist() == [[[2, 3, 5, 8, 9]]] and n.tolist() == [5]
    assert k[1, 0, :5, 0].tolist() == [2, 3, 5, 8, 9] and v[1, 0, :5, 0].tolist() == [4, 6, 10, 16, 18]
    assert ww[1, 0, :5].tolist() == [7, 7, 7, 3, 9] and (k[1, 0, 5:] == kc[1, 0, 5:]).all()
    assert np.array_equal(k[0], kc[0])
    kept = paged.evict(kc, kc, w, np.array([[0]]), np.array([10]), np.array([[1]]), 4, 0)[3]
    assert kept.tolist() == [[[2, 3, 5, 9]]]      # of three sevens and a nine, all four


def test_f64_keeps_whole_numbers():
    assert f64(torch.tensor([3], dtype=torch.int32)).dtype == np.int32
