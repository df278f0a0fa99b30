"""Arguments of a write that nothing would use are refused, not dropped in silence."""
import pytest
import torch

from speculative_decoding_verification_pipeline_amd.rotary import Rotary
from tests.gpu_support import device
from tests.kv8_support import World, i32

pytestmark = pytest.mark.gpu


def test_write_refuses_what_it_would_not_use():
    w = World(rows=2)
    w.hold([3, 4], extra=4)
    k = torch.zeros(2, 4, 2, 64, dtype=torch.bfloat16, device=device())
    out = torch.full((2, 4, 4, 64), 5.0, dtype=torch.bfloat16, device=device())
    pos = i32([[0, 1, 2, 3]] * 2)
    before = w.planes()
    for bad in (dict(positions=pos), dict(out_queries=out), dict(out_queries=out, rotary=Rotary(64))):
        with pytest.raises(ValueError):
            w.cache.write(w.bt, 0, k, k, **bad)
    after = w.planes()
    assert all((a == b).all() for a, b in zip(before, after))
    assert w.cache.write(w.bt, 0, k, k, rotary=Rotary(64), positions=pos) is None
