"""The largest numbers that eviction takes."""

import pytest
import torch

import exact_memory_efficient_b200 as m
from tests.test_paged_api import INVALID, evict, lib  # noqa: F401  (lib: the fixture)

TOP = 2**31 - 1 - 65536      # B * H_kv * n_keep


@pytest.mark.parametrize("B,Hkv,keep", [(1, 1, 2**31 - 1), (1, 1, 2**31 - 8192), (1, 1, TOP + 1), (2, 1, TOP // 2 + 1),
                                        (2, 2, 2**29), (3, 5, 2**31 - 1)])
def test_too_many_kept_slots_are_refused(lib, B, Hkv, keep):  # noqa: F811
    """Slots are counted in 32 bits, and the kernels look up to a few thousand beyond the last one."""
    assert evict(lib, B=B, Hkv=Hkv, keep=keep, dmaxp=2**20, page=256, maxp=2**20) == INVALID


@pytest.mark.gpu
@pytest.mark.parametrize("in_place", [False, True])
def test_as_many_kept_slots_as_there_can_be(in_place):
    """An 8 GB list of slots for a sequence of 100 keys: all of them, then -1 to the end."""
    k = torch.randn(8, 1, 64, 64, device="cuda").to(torch.bfloat16)
    v, w = torch.randn_like(k), torch.rand(8, 1, 64, device="cuda")
    before = [t.clone() for t in (k, v, w)]
    n = torch.tensor([100], dtype=torch.int32, device="cuda")
    table = torch.tensor([[3, 1]], dtype=torch.int32, device="cuda")
    dst = table if in_place else torch.tensor([[5, 6]], dtype=torch.int32, device="cuda")
    kept, left = m.paged_evict(k, v, w, table, n, dst, TOP, 5)
    assert m.mea_last_device_error() == m.MEA_OK and left.item() == 100 and kept.shape == (1, 1, TOP)
    assert torch.equal(kept[0, 0, :100].cpu(), torch.arange(100, dtype=torch.int32))
    for part in kept[0, 0, 100:].split(1 << 28):
        assert int(part.max()) == -1 and int(part.min()) == -1
    for t, old in zip((k, v, w), before):
        if not in_place:
            old[5], old[6, :, :36] = old[3], old[1, :, :36]
        assert torch.equal(t, old)
