"""mea_rope against the fp64 definition (GPU)."""

import threading
from types import SimpleNamespace

import numpy as np
import pytest
import torch

import exact_memory_efficient_b200 as m
from oracle import paged
from tests._paged import f64, rope_bound

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def check(x, pos, freq, interleaved, mscale, inverse, y):
    p = pos.numpy() if pos.dim() == 2 else np.broadcast_to(pos.numpy(), (x.shape[0], x.shape[2]))
    for b in range(x.shape[0]):
        xb, got = f64(x[b]), f64(y[b])
        want = paged.rope(xb, p[b], freq.numpy(), interleaved, mscale, inverse)
        tol = rope_bound(xb, freq.numpy(), interleaved, mscale, x.dtype, want)
        assert (np.abs(got - want) <= tol).all(), (np.abs(got - want) - tol).max()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("dtype,B,H,N,D,rot,mscale", [
    (BF, 1, 1, 1, 64, 64, 1.0), (BF, 2, 3, 37, 128, 128, 1.0), (BF, 1, 5, 129, 128, 48, 1.25), (BF, 3, 17, 65, 64, 16, 1.0),
    (F32, 1, 2, 33, 32, 32, 1.0), (F32, 2, 4, 63, 96, 80, 0.7), (F32, 1, 9, 130, 128, 16, 1.0), (F32, 2, 1, 7, 64, 64, 1.0),
])
def test_rope(dtype, B, H, N, D, rot, mscale, inverse, interleaved):
    g = torch.Generator().manual_seed(N)
    x = torch.randn(B, H, N, D, generator=g).to(dtype)
    pos = torch.randint(0, 5000, (N,), generator=g, dtype=torch.int32)
    freq = m.mea_rope_frequencies(rot)
    y = m.rope(x.cuda(), pos.cuda(), freq.cuda(), interleaved, mscale, inverse)
    check(x, pos, freq, interleaved, mscale, inverse, y)


def test_positions_per_batch_far_and_negative():
    """Positions of a million and more: the angle is reduced in fp64."""
    x = torch.randn(3, 2, 50, 64, generator=torch.Generator().manual_seed(1))
    pos = torch.stack([torch.arange(50) - 25, torch.arange(50) * 40009 + 1000003, torch.full((50,), 2**31 - 1)]).int()
    freq = m.mea_rope_frequencies(64, 10000.0, m.MEA_ROPE_SCALE_BY_PARTS, 8.0, 4096.0)
    y = m.rope(x.cuda(), pos.cuda(), freq.cuda(), True)
    for b in range(2):
        check(x[b:b + 1], pos[b:b + 1], freq, True, 1.0, False, y[b:b + 1])
    # at 2^31 the fp64 angle itself is rounded by up to 2^-53 * 2^31 rad: 3e-7 with its products
    want = paged.rope(f64(x[2]), pos[2].numpy(), freq.numpy(), True)
    assert np.abs(f64(y[2]) - want).max() < 9 * 2.0**-24 * 10 + 3 * 4.8e-7 * 5


def test_in_place_equals_out_of_place_and_other_stream():
    x = torch.randn(2, 8, 300, 128, device="cuda").to(BF)
    pos = torch.arange(300, dtype=torch.int32, device="cuda")
    freq = m.mea_rope_frequencies(96).cuda()
    want = m.rope(x, pos, freq)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = m.rope(x, pos, freq, stream=s)
    s.synchronize()
    assert torch.equal(y, want)
    m.mea_rope(x, x, pos, freq)
    assert torch.equal(x, want)


def test_streams_of_the_binding():
    """None, a torch stream and its handle name the same stream; another device's and other objects are refused."""
    x = torch.randn(2, 8, 300, 128, device="cuda").to(BF)
    pos = torch.arange(300, dtype=torch.int32, device="cuda")
    freq = m.mea_rope_frequencies(96).cuda()
    want = m.rope(x, pos, freq)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = m.rope(x, pos, freq, stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(y, want)
    y = m.rope(x, pos, freq, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(y, want)
    for bad in (SimpleNamespace(cuda_stream=s.cuda_stream, device_index=1), object(), "0", 2.5):
        with pytest.raises(m.MeaError) as e:
            m.rope(x, pos, freq, stream=bad)
        assert e.value.status == m.MEA_ERR_INVALID_ARG and "stream" in str(e.value)


def test_calls_from_two_threads():
    xs = [torch.randn(2, 4, 200, 64, device="cuda") for _ in range(2)]
    pos = torch.arange(200, dtype=torch.int32, device="cuda")
    freq = m.mea_rope_frequencies(64).cuda()
    want = [m.rope(x, pos, freq) for x in xs]
    torch.cuda.synchronize()
    out = [None, None]

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(200):
                out[i] = m.rope(xs[i], pos, freq)
            torch.cuda.current_stream().synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


@pytest.mark.parametrize("interleaved", [False, True])
def test_inverse_is_the_gradient(interleaved):
    """<dy, rope(x)> has the gradient rope(dy, inverse) in x: against central differences of the library's
    own fp32 forward.  The map is linear, so the difference quotient with step 1 is exact up to the two
    roundings of each side: 20 u times the sum of the magnitudes."""
    g = torch.Generator().manual_seed(3)
    x, dy = (torch.randn(1, 1, 6, 32, generator=g).cuda() for _ in range(2))
    pos = torch.tensor([0, 3, 11, 500, 7, 1], dtype=torch.int32).cuda()
    freq = m.mea_rope_frequencies(16).cuda()
    dx = m.rope(dy, pos, freq, interleaved, 1.3, inverse=True)
    for n, d in ((1, 0), (1, 5), (3, 9), (3, 15), (4, 20), (5, 31)):
        hi, lo = x.clone(), x.clone()
        hi[0, 0, n, d] += 1
        lo[0, 0, n, d] -= 1
        num = ((m.rope(hi, pos, freq, interleaved, 1.3).double() - m.rope(lo, pos, freq, interleaved, 1.3).double())
               * dy.double()).sum() / 2
        assert abs(float(num) - float(dx[0, 0, n, d])) < 20 * 2.0**-24 * float((dy.abs() * (x.abs() + 1)).sum(-1)[0, 0, n])


def test_graph_replay_with_other_positions():
    x = torch.randn(1, 4, 64, 64, device="cuda").to(BF)
    pos = torch.arange(64, dtype=torch.int32, device="cuda")
    freq = m.mea_rope_frequencies(64).cuda()
    y = torch.empty_like(x)
    m.mea_rope(x, y, pos, freq)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.mea_rope(x, y, pos, freq)
    pos += 1000
    graph.replay()
    assert torch.equal(y, m.rope(x, pos, freq))


def test_training_pass_with_rotated_heads():
    """Rotation, grouped attention, its backward and the rotation's gradient, as a training step runs them,
    against the fp64 chain."""
    import oracle
    from tests._parity import BF16_GRAD, BF16_O, assert_close
    g = torch.Generator().manual_seed(4)
    q, k, v, do = (torch.randn(1, h, 200, 64, generator=g).to(BF) for h in (4, 2, 2, 4))
    pos, freq = torch.arange(200, dtype=torch.int32), m.mea_rope_frequencies(32)
    pc, fc = pos.cuda(), freq.cuda()
    qr, kr = m.rope(q.cuda(), pc, fc), m.rope(k.cuda(), pc, fc)
    o, lse = m.attention_forward(qr, kr, v.cuda(), 0.125)
    dqr, dkr, dv = m.attention_backward(qr, kr, v.cuda(), o, lse, do.cuda(), 0.125)
    dq, dk = m.rope(dqr, pc, fc, inverse=True), m.rope(dkr, pc, fc, inverse=True)
    assert m.mea_last_device_error() == m.MEA_OK
    # the reference takes the rotated, rounded q and k, as the attention does
    rq, rk, rv, ro, _ = oracle.attention_backward_gqa(f64(qr), f64(kr), f64(v), f64(do), 0.125)
    assert_close(f64(o), ro, *BF16_O, what="O")
    assert_close(f64(dq), paged.rope(rq, pos.numpy(), freq.numpy(), inverse=True), *BF16_GRAD, what="dq")
    assert_close(f64(dk), paged.rope(rk, pos.numpy(), freq.numpy(), inverse=True), *BF16_GRAD, what="dk")
    assert_close(f64(dv), rv, *BF16_GRAD, what="dv")
