"""The factor on dot products: the range that is served, its ends, and what lies outside."""
import numpy as np
import pytest
import torch

from speculative_decoding_verification_pipeline_amd import sampler as SM
from tests.gpu_support import device, log
from tests.kv8_support import World, i32, np64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N,group", [(1, 2), (5, 4), (20, 8)])
def test_ends_of_the_range(N, group):
    """Keys of zeros, under the least scale of a block, and the least and largest factors:
    every slot that is seen weighs the same, and none that is not counts."""
    w = World(seed=N, P=20, ps=16, heads=1, dim=64, rows=2, M=5)
    w.hold([37, 0], extra=N)
    w.o.pool[0] = 0
    w.o.scales[0] = 67  # 2^-60
    w.o.scales[1] = 127
    w.put()
    q = w.heads(2, N, group, 64, "bf16")
    log(f"attend scales: N={N} group={group}")
    for scale in (2.0 ** -60, 1.0, 2.0 ** 60):
        got = np64(w.cache.attend(w.bt, 0, q, scale=scale))
        for b, at in enumerate((37, 0)):
            for n in range(N):
                v = w.o.read(1, b, 0, at + n + 1)[:, 0]
                # equal weights are exact; sums in binary32, the result to its type
                bound = 2.0 ** -8 * np.abs(v.mean(0)) + (at + N) * 2.0 ** -22 * np.abs(v).mean(0)
                assert np.all(np.abs(got[b, n] - v.mean(0)) <= bound), (scale, b, n)


def test_factors_outside_are_refused():
    """Outside, a factor times a block's scale is no binary32 number of its own."""
    w = World(rows=1)
    w.hold([3], extra=1)
    q = torch.zeros(1, 1, 4, 64, dtype=torch.bfloat16, device=device())
    for scale in (1e-40, 2.0 ** -61, 2.0 ** 61, 3.4e38):
        with pytest.raises(SM.SamplerError) as e:
            w.cache.attend(w.bt, 0, q, scale=scale)
        assert e.value.status == SM.SS_ERR_INVALID_ARG
