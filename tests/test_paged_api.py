"""Rotary positions and the paged cache: refusals of the C ABI and of the binding, and the host function
for the angles (CPU; no kernel is launched, fake device addresses are never dereferenced)."""

import ctypes
import math

import numpy as np
import pytest
import torch

import exact_memory_efficient_b200 as m

A = 0x10000
BF16, F32 = m.MEA_DTYPE_BF16, m.MEA_DTYPE_F32
INVALID, UNSUPPORTED, MISALIGNED = m.MEA_ERR_INVALID_ARG, m.MEA_ERR_UNSUPPORTED, m.MEA_ERR_MISALIGNED


@pytest.fixture(scope="module")
def lib():
    from exact_memory_efficient_b200 import build as b
    b.build()
    return m.load_library()


def rope(lib, x=A, y=A, pos=A, freq=A, B=1, H=2, N=8, D=64, rot=64, per=0, layout=0, mscale=1.0, inv=0, dtype=BF16):
    return lib.mea_rope(x, y, pos, freq, B, H, N, D, rot, per, layout, mscale, inv, dtype, None)


def append(lib, q=A, q_out=A + 16, k=A, v=A, kc=A, vc=A, w=A, cu=A, kv=A, table=A, pos=A, freq=A, T=4, B=2, H=4, Hkv=2,
           D=64, qs=256, ks=128, vs=128, pages=8, page=16, maxp=4, rot=64, layout=0, mscale=1.0, dtype=BF16):
    return lib.mea_paged_append(q, q_out, k, v, kc, vc, w, cu, kv, table, pos, freq, T, B, H, Hkv, D, qs, ks, vs, pages,
                                page, maxp, rot, layout, mscale, dtype, None)


def attend(lib, q=A, kc=A, vc=A, o=A, lse=A, cu=A, kv=A, table=A, T=4, B=2, H=4, Hkv=2, D=64, qs=256, pages=8, page=16,
           maxp=4, max_q=2, max_kv=64, scale=0.125, dtype=BF16, ws=None, ws_bytes=0):
    return lib.mea_attn_paged(q, kc, vc, o, lse, cu, kv, table, T, B, H, Hkv, D, qs, pages, page, maxp, max_q, max_kv,
                              scale, dtype, ws, ws_bytes, None)


def weigh(lib, q=A, lse=A, kc=A, w=A, cu=A, kv=A, table=A, T=4, B=2, H=4, Hkv=2, D=64, qs=256, pages=8, page=16,
          maxp=4, max_q=2, max_kv=64, scale=0.125, dtype=BF16):
    return lib.mea_attn_paged_weights(q, lse, kc, w, cu, kv, table, T, B, H, Hkv, D, qs, pages, page, maxp, max_q,
                                      max_kv, scale, dtype, None, 0, None)


def evict(lib, kc=A, vc=A, w=A, table=A, kv=A, dst=A + 64, out=A, idx=A, B=2, Hkv=2, D=64, pages=8, page=16, maxp=4,
          dmaxp=2, keep=32, recent=8, dtype=BF16):
    return lib.mea_paged_evict(kc, vc, w, table, kv, dst, out, idx, B, Hkv, D, pages, page, maxp, dmaxp, keep, recent,
                               dtype, None)


@pytest.mark.parametrize("status,args", [
    (INVALID, dict(x=None)), (INVALID, dict(freq=None)), (INVALID, dict(pos=None)), (INVALID, dict(B=-1)),
    (INVALID, dict(dtype=9)), (INVALID, dict(layout=2)), (INVALID, dict(rot=0)), (INVALID, dict(rot=80)),
    (INVALID, dict(mscale=math.inf)), (INVALID, dict(mscale=math.nan)), (UNSUPPORTED, dict(rot=24)),
    (UNSUPPORTED, dict(D=96)), (UNSUPPORTED, dict(D=40, dtype=F32, rot=16)), (MISALIGNED, dict(x=A + 8)),
    (MISALIGNED, dict(y=A + 2)), (MISALIGNED, dict(freq=A + 4)), (INVALID, dict(H=1 << 14, B=1 << 14, N=1 << 14)),
    (UNSUPPORTED, dict(B=4, N=1 << 30, H=1)),
    (0, dict(B=0, x=None)), (0, dict(H=0)), (0, dict(N=0, y=None)),
])
def test_rope_refusals(lib, status, args):
    assert rope(lib, **args) == status


COMMON = [
    (INVALID, dict(T=-1)), (INVALID, dict(B=-1)), (INVALID, dict(dtype=9)), (UNSUPPORTED, dict(D=96)),
    (INVALID, dict(Hkv=0)), (INVALID, dict(H=5)), (INVALID, dict(page=0)), (UNSUPPORTED, dict(page=8)),
    (UNSUPPORTED, dict(page=48)), (UNSUPPORTED, dict(page=512)), (INVALID, dict(maxp=1 << 28)),
    (INVALID, dict(pages=1 << 30, Hkv=2)), (INVALID, dict(pages=0)), (INVALID, dict(maxp=0)), (INVALID, dict(pages=-1)),
    (UNSUPPORTED, dict(B=70000)), (INVALID, dict(cu=None)), (INVALID, dict(kv=None)), (INVALID, dict(table=None)),
    (INVALID, dict(kc=None)), (MISALIGNED, dict(kc=A + 8)), (MISALIGNED, dict(table=A + 2)), (MISALIGNED, dict(q=A + 4)),
    (INVALID, dict(qs=255)), (MISALIGNED, dict(qs=260)), (INVALID, dict(T=1 << 30)), (0, dict(T=0, kc=None)),
    (0, dict(B=0, kv=None)),
]


@pytest.mark.parametrize("status,args", COMMON + [
    (INVALID, dict(q=None)), (INVALID, dict(q_out=None)), (INVALID, dict(k=None)), (INVALID, dict(vc=None)),
    (INVALID, dict(ks=127)), (MISALIGNED, dict(vs=132)), (INVALID, dict(rot=80)), (UNSUPPORTED, dict(rot=8)),
    (INVALID, dict(layout=-1)), (INVALID, dict(q_out=A, qs=512)), (MISALIGNED, dict(freq=A + 4)),
    (MISALIGNED, dict(pos=A + 1)), (MISALIGNED, dict(w=A + 2)), (INVALID, dict(mscale=math.nan)),
])
def test_append_refusals(lib, status, args):
    assert append(lib, **args) == status


@pytest.mark.parametrize("status,args", COMMON + [
    (INVALID, dict(q=None)), (INVALID, dict(o=None)), (INVALID, dict(lse=None)), (INVALID, dict(vc=None)),
    (MISALIGNED, dict(o=A + 2)), (MISALIGNED, dict(lse=A + 2)), (INVALID, dict(scale=math.nan)),
    (INVALID, dict(max_q=-1)), (INVALID, dict(max_kv=-1)),
])
def test_attention_refusals(lib, status, args):
    assert attend(lib, **args) == status


@pytest.mark.parametrize("status,args", COMMON + [
    (INVALID, dict(q=None)), (INVALID, dict(lse=None)), (INVALID, dict(w=None)), (MISALIGNED, dict(w=A + 1)),
    (INVALID, dict(scale=math.inf)), (INVALID, dict(max_q=-1)), (INVALID, dict(max_kv=-1)),
])
def test_weights_refusals(lib, status, args):
    assert weigh(lib, **args) == status


@pytest.mark.parametrize("status,args", [
    (INVALID, dict(kc=None)), (INVALID, dict(vc=None)), (INVALID, dict(w=None)), (INVALID, dict(table=None)),
    (INVALID, dict(kv=None)), (INVALID, dict(dst=None)), (INVALID, dict(idx=None)), (INVALID, dict(keep=0)),
    (INVALID, dict(recent=-1)), (INVALID, dict(recent=33)), (INVALID, dict(dmaxp=1)), (INVALID, dict(dst=A)),
    (INVALID, dict(B=-1)), (INVALID, dict(pages=0)), (UNSUPPORTED, dict(page=8)), (UNSUPPORTED, dict(B=40000)),
    (UNSUPPORTED, dict(D=32)), (MISALIGNED, dict(vc=A + 8)), (MISALIGNED, dict(out=A + 2)), (MISALIGNED, dict(idx=A + 1)),
    (0, dict(B=0, kc=None)),
])
def test_evict_refusals(lib, status, args):
    assert evict(lib, **args) == status


def test_workspace_size_refusals(lib):
    out = ctypes.c_size_t(7)
    check_sizes(lib.mea_attn_paged_workspace_size, out)
    check_sizes(lib.mea_attn_paged_weights_workspace_size, out)


def check_sizes(f, out):
    assert f(4, 2, 4, 2, 64, 2, 64, BF16, None) == INVALID
    assert f(4, 2, 5, 2, 64, 2, 64, BF16, ctypes.byref(out)) == INVALID
    assert f(4, 2, 4, 2, 96, 2, 64, BF16, ctypes.byref(out)) == UNSUPPORTED
    assert f(4, 2, 4, 2, 64, -1, 64, BF16, ctypes.byref(out)) == INVALID
    assert f(0, 2, 4, 2, 64, 0, 64, BF16, ctypes.byref(out)) == 0 and out.value == 0


def test_status_of_a_bad_page():
    assert m.mea_status_string(m.MEA_ERR_PAGE).startswith("MEA_ERR_PAGE")


def test_frequencies():
    f = m.mea_rope_frequencies(64, 10000.0).numpy()
    want = 10000.0 ** (-np.arange(32) / 32.0)
    assert f.dtype == np.float64 and np.abs(f / want - 1).max() < 1e-14
    g = m.mea_rope_frequencies(64, 10000.0, m.MEA_ROPE_SCALE_LINEAR, 4.0).numpy()
    assert np.abs(g * 4 / want - 1).max() < 1e-14
    # a scaled base: the first pair keeps its speed, the last slows down by the factor
    g = m.mea_rope_frequencies(64, 10000.0, m.MEA_ROPE_SCALE_BASE, 8.0).numpy()
    assert abs(g[0] - 1) < 1e-15 and abs(g[-1] * 8 / want[-1] - 1) < 1e-12
    assert (np.diff(want / g) > 0).all()
    # by parts: fast pairs as they are, slow ones divided, a mix between
    L, slow, fast = 4096.0, 1.0, 32.0
    g = m.mea_rope_frequencies(64, 10000.0, m.MEA_ROPE_SCALE_BY_PARTS, 16.0, L, slow, fast).numpy()
    turns = L * want / (2 * math.pi)
    mix = np.clip((turns - slow) / (fast - slow), 0, 1)
    assert np.abs(g / ((1 - mix) * want / 16 + mix * want) - 1).max() < 1e-13
    assert (g[turns > fast] == f[turns > fast]).all() and (mix == 0).any() and ((mix > 0) & (mix < 1)).any()


@pytest.mark.parametrize("args", [
    (63,), (0,), (64, 1.0), (64, math.nan), (64, 1e4, 7), (64, 1e4, 1, 0.5), (2, 1e4, 2, 4.0), (64, 1e4, 3, 4.0, 0.0),
    (64, 1e4, 3, 4.0, 4096.0, 32.0, 1.0),
])
def test_frequency_refusals(args):
    with pytest.raises(m.MeaError) as e:
        m.mea_rope_frequencies(*args)
    assert e.value.status == INVALID


def refused(fn, *args, **kw):
    with pytest.raises(m.MeaError) as e:
        fn(*args, **kw)
    assert e.value.status == INVALID, e.value


def test_binding_refuses_cpu_tensors_and_shapes():
    """Shapes, types and strides are checked before the device is; CPU tensors are refused."""
    bf, i32 = torch.bfloat16, torch.int32
    kc = torch.zeros(8, 2, 16, 64, dtype=bf)
    w = torch.zeros(8, 2, 16)
    cu, kv, tab = torch.zeros(3, dtype=i32), torch.zeros(2, dtype=i32), torch.zeros(2, 4, dtype=i32)
    q, k = torch.zeros(4, 4, 64, dtype=bf), torch.zeros(4, 2, 64, dtype=bf)
    lse, o = torch.zeros(4, 4), torch.zeros(4, 4, 64, dtype=bf)
    att = lambda **x: m.mea_attn_paged(**{**dict(q=q, k_cache=kc, v_cache=kc, o=o, lse=lse, cu_q=cu, kv_len=kv,  # noqa: E731
                                                 page_table=tab, max_q=2, max_kv=9, scale=1.0, workspace=None), **x})
    refused(att)                                             # on the CPU
    for bad in (dict(q=q.float()), dict(q=q[0]), dict(k_cache=kc[0]), dict(v_cache=kc[:4]), dict(o=o[:3]),
                dict(lse=lse.T.contiguous()[:2]), dict(cu_q=cu[:2]), dict(page_table=tab[:1]), dict(kv_len=tab),
                dict(q=q.transpose(1, 2).contiguous().transpose(1, 2)), dict(q=torch.zeros(4, 4, 32, dtype=bf))):
        refused(att, **bad)
    refused(m.attention_paged, q, kc, kc, cu, kv, tab, 2, 9)
    refused(m.mea_attn_paged_weights, q, lse, kc, w[:, :1], cu, kv, tab, 2, 9, 1.0)
    refused(m.mea_attn_paged_weights, q, lse[:2], kc, w, cu, kv, tab, 2, 9, 1.0)
    refused(m.mea_attn_paged_weights, q, lse, kc, w, cu, kv, tab, 2, 9, 1.0)
    app = lambda **x: m.mea_paged_append(**{**dict(q=q, q_out=o, k=k, v=k, k_cache=kc, v_cache=kc, weights=w, cu_q=cu,  # noqa: E731
                                                   kv_len=kv, page_table=tab), **x})
    for bad in (dict(), dict(q=None), dict(k=q), dict(v=k[:3]), dict(q_out=o[:2]), dict(positions=cu),
                dict(freq=torch.zeros(2, 2, dtype=torch.float64)), dict(weights=w[:3])):
        refused(app, **bad)
    idx = torch.zeros(2, 2, 8, dtype=i32)
    ev = lambda **x: m.mea_paged_evict(**{**dict(k_cache=kc, v_cache=kc, weights=w, page_table=tab, kv_len=kv,  # noqa: E731
                                                 dst_table=tab, kv_len_out=kv, keep_idx=idx, n_recent=2), **x})
    for bad in (dict(), dict(dst_table=tab[:1]), dict(keep_idx=idx[0]), dict(keep_idx=idx[:, :1]),
                dict(kv_len_out=cu), dict(v_cache=kc[:2])):
        refused(ev, **bad)
    refused(m.paged_evict, kc, kc, w, tab, kv, tab, 0, 0)
    x, pos, fr = torch.zeros(1, 2, 8, 64, dtype=bf), torch.zeros(8, dtype=i32), torch.zeros(8, dtype=torch.float64)
    for bad in ((x, x, pos, fr), (x, x[:, :1], pos, fr), (x, x, pos[:3], fr), (x[0], x[0], pos, fr), (x, x, pos, fr[None])):
        refused(m.mea_rope, *bad)


def test_binding_refuses_arguments_of_other_types(lib):
    x, pos, freq = torch.zeros(1, 2, 8, 64), torch.zeros(8, dtype=torch.int32), torch.zeros(32, dtype=torch.float64)
    q, kc = torch.zeros(4, 4, 64), torch.zeros(8, 2, 16, 64)
    cu, kv, table = (torch.zeros(n, dtype=torch.int32) for n in ((3,), (2,), (2, 4)))

    def refused(word, f, *args, **kw):
        with pytest.raises(m.MeaError) as e:
            f(*args, **kw)
        assert e.value.status == INVALID and word in str(e.value)

    refused("x must be a tensor", m.rope, x.numpy(), pos, freq)
    refused("freq must be a tensor", m.rope, x, pos, None)
    refused("inverse", m.rope, x, pos, freq, inverse=np.ones(2))
    refused("mscale", m.rope, x, pos, freq, mscale="1")
    refused("max_q", m.attention_paged, q, kc, kc, cu, kv, table, 1.5, 64)
    refused("max_q", m.attention_paged, q, kc, kc, cu, kv, table, 2**40, 64)
    refused("max_kv", m.attention_paged, q, kc, kc, cu, kv, table, 1, None)
    refused("n_keep", m.paged_evict, kc, kc, torch.zeros(8, 2, 16), table, kv, table, 0, 0)
