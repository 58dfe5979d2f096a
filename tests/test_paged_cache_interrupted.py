"""A serving step that is interrupted leaves the cache's page list as it was (CPU)."""

import pytest
import torch

from tests.test_paged_cache import OracleOps, cpu_cache, tokens


@pytest.mark.parametrize("step", ["append", "attend", "weigh"])
@pytest.mark.parametrize("error", [KeyboardInterrupt, SystemExit, RuntimeError])
def test_an_interrupted_step_leaves_the_page_list(step, error):
    class Stops(OracleOps):
        pass

    def stop(*args):
        raise error("here")

    c, g = cpu_cache(), torch.Generator().manual_seed(8)
    a, b = c.add(), c.add()
    c.step(*tokens(g, 20), [a, b], [17, 3])
    state = (c.length(a), c.length(b), c.free_pages, c.pages(a), c.pages(b), dict(c._pos))
    c.ops = Stops()
    setattr(c.ops, step, stop)
    with pytest.raises(error):
        c.step(*tokens(g, 50), [b, a], [33, 17])
    assert (c.length(a), c.length(b), c.free_pages, c.pages(a), c.pages(b), dict(c._pos)) == state
    c.ops = OracleOps()
    c.step(*tokens(g, 50), [b, a], [33, 17])
    assert len(set(c.pages(a) + c.pages(b))) == len(c.pages(a) + c.pages(b)) == 12 - c.free_pages
