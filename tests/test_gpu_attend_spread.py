"""Values whose blocks' scales lie 2^100 apart, the most under which every weight counts:
slots of small values that outweigh those of large ones keep their share of the sum."""
import numpy as np
import pytest

from tests.gpu_support import log
from tests.kv8_support import World
from tests.test_gpu_attend import check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N,group,dim", [(1, 2, 64), (3, 4, 128), (20, 8, 128), (1, 1, 256)])
def test_scales_2_100_apart(N, group, dim):
    ps, slots = 16, 2000
    M = -(-(slots + N) // ps)
    w = World(seed=N + dim, P=M + 2, ps=ps, heads=1, dim=dim, rows=1, M=M)
    w.hold([slots], extra=N)
    w.o.scales[1] = np.where(w.rng.random(w.o.scales[1].shape) < 0.05, 177, 77)
    w.put()
    log(f"attend scales apart: N={N} group={group} dim={dim}")
    q = w.heads(1, N, group, dim, "bf16")
    check(w, q, "bf16", "apart")
