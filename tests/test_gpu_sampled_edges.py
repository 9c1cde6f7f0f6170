"""GPU tests of accept_sampled at the edges of what its contract allows, against oracle/sampled.py (fp64)."""
import numpy as np
import pytest
import torch

from gpu_util import dev, host
from test_gpu_sampled import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kw", [dict(), dict(T=[0.7], k=[20], p=[0.9])])
def test_no_nodes_by_max_nodes(tv, kw):
    """max_nodes 0: no request has a node, whatever the offsets say, and neither a row nor the workspace is touched."""
    c = Case(50, [3, 5], 100, **kw)
    acc, best, path, bonus = c.run(tv, max_nodes=0, max_depth=2, ws=torch.empty(0, dtype=torch.uint8, device="cuda"))
    for t in (acc, best, path, bonus):
        assert bool((t == -1).all())


def test_nodes_beyond_max_nodes_are_left_out(tv):
    """The same as the requests without those nodes."""
    c = Case(51, [9, 4, 12], 300, T=[0.8], p=[0.95])
    got = c.run(tv, max_nodes=5)
    keep = np.concatenate([np.arange(a, min(a + 5, b)) for a, b in zip(c.off, c.off[1:])])
    for name in ("parent", "tok", "logits", "q", "drawn", "u"):
        setattr(c, name, getattr(c, name)[keep])
    c.off = np.array([0, 5, 9, 14], np.int32)
    for a, b in zip(got, c.run(tv)):
        assert np.array_equal(host(a), host(b))
    c.check(got, most=0.4)
