"""Arguments that are no tensors, or of another rank, are refused as the others are."""
import pytest
import torch

from speculative_decoding_verification_pipeline_amd.rotary import Rotary
from tests.gpu_support import device
from tests.kv8_support import World, i32

pytestmark = pytest.mark.gpu


def test_read_and_rotate_refuse_what_is_no_tensor():
    w = World(rows=2)
    w.hold([3, 4])
    for bad in (dict(start=[0, 0]), dict(counts=[1, 1]), dict(start=3), dict(start=i32(0)),
                dict(start=i32([[0, 0]]).view(1, 2)), dict(start=torch.zeros(2, dtype=torch.int32))):
        with pytest.raises(ValueError):
            w.cache.read(w.bt, 0, 4, **bad)
    assert w.cache.read(w.bt, 0, 4, counts=i32([1]))[0].shape == (1, 4, 2, 64)
    r = Rotary(64)
    q = torch.zeros(2, 3, 64, dtype=torch.bfloat16, device=device())
    for keys in ([1.0], 2, q[0, 0], q.float(), q[None], q.cpu()):
        with pytest.raises(ValueError):
            r.rotate(q, i32([0, 1]), keys=keys)
