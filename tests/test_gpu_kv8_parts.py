"""Writing keys whose rotated part no 16 entries divide (half or a quarter of a head of 80),
against the definition on host arrays (oracle.kv8)."""
import random

import numpy as np
import pytest
import torch

from oracle import kv8 as K
from perf import more_operators
from speculative_decoding_verification_pipeline_amd.rotary import Rotary
from tests.gpu_support import device, log
from tests.kv8_support import HALF_STEP, World, i32, np64

pytestmark = pytest.mark.gpu

PARTS = [
    # head, rotated part, heads of the cache, page, block, layout
    (80, 40, 2, 32, 16, "hnd"),      # half a head: pairs in fours
    (80, 20, 3, 64, 64, "nhd"),      # a quarter: pairs in single entries
    (80, 10, 1, 16, 16, "padded"),   # five pairs
    (96, 24, 4, 48, 16, "nhd"),
    (144, 72, 2, 64, 32, "separate"),
    (16, 8, 8, 16, 16, "nhd"),
    (64, 2, 2, 32, 32, "nhd"),
    (256, 8, 2, 64, 64, "hnd"),      # 17 units a head in the largest block
]


@pytest.mark.parametrize("part", range(len(PARTS)))
@pytest.mark.parametrize("inter,tree,dtype", [(False, False, "bf16"), (True, True, "f16"),
                                              (False, True, "f16")])
def test_write_turned(part, inter, tree, dtype):
    """Bytes differ only where a value turned in binary64 lies on the border of two
    roundings. Queries turn along, in place too; what lies around them stays."""
    dim, rot, heads, ps, block, layout = PARTS[part]
    N = 40
    w = World(seed=part, rows=4, heads=heads, dim=dim, ps=ps, block=block, layout=layout,
              P=64, M=-(-(130 + N) // ps))
    w.hold([0, 50, 130, 7], extra=N)
    log(f"kv8 write turned: {PARTS[part]} interleaved={inter} tree={tree} {dtype}")
    r = Rotary(rot, scaling="parts", factor=8.0, original=1024, interleaved=inter)
    up = w.tree(4, N, lost=0.1) if tree else None
    counts = [40, 13, 0, 1]
    k, v = w.heads(4, N, heads, dim, dtype, 3.0), w.heads(4, N, heads, dim, dtype)
    qkv = w.heads(4, N, 39, dim, dtype)
    q = qkv[:, :, 1:38]
    pos = np.array(w.o.lens)[:, None] + (np.array([K.depths(u) for u in up]) if tree else np.arange(N))
    step = dict(counts=i32(counts), rotary=r)
    if tree:
        step["parents"] = i32(up)
    out = w.cache.write(w.bt, 0, k, v, queries=q, **step)
    w.o.write(0, K.turn(np64(k), pos, r.inv_freq, r.magnitude, inter), 4, counts=counts)
    w.o.write(1, np64(v), 4, counts=counts)
    pool, scales = w.planes()
    assert np.array_equal(scales, w.o.scales) and np.array_equal(pool[1], w.o.pool[1])
    assert np.mean(pool[0] != w.o.pool[0]) < 1e-5
    want = K.turn(np64(q), pos, r.inv_freq, r.magnitude, inter)
    for b in range(4):
        want[b, counts[b]:] = 0
    # four roundings to binary32 of up to |u| + |v| times the magnitude, and one to the type
    a = np.abs(np64(q)).max() * 2 * r.magnitude
    bound = HALF_STEP[dtype] * np.abs(want) * 1.001 + 4 * 2.0 ** -24 * a + (2.0 ** -25 if dtype == "f16" else 0)
    bound[..., rot:] = 0.0
    assert np.all(np.abs(np64(out) - want) <= bound)
    mine = qkv.clone()
    same = w.cache.write(w.bt, 0, k, v, queries=mine[:, :, 1:38], out_queries=mine[:, :, 1:38],
                         positions=i32(pos), counts=i32(counts), rotary=r)
    assert torch.equal(same, out)
    assert torch.equal(mine[:, :, 0], qkv[:, :, 0]) and torch.equal(mine[:, :, 38], qkv[:, :, 38])
    again, x = w.planes()
    assert np.array_equal(again, pool) and np.array_equal(x, scales)


def test_every_measured_part_is_served():
    """The heads and rotated parts of the cases that the measured calls draw."""
    rng = random.Random(5)
    drawn = [more_operators.draw(rng) for _ in range(600)]
    parts = {(c["dim"], c["rot"], c["interleaved"]) for c in drawn if c["op"] == "store"}
    assert (80, 40, False) in parts and (80, 40, True) in parts
    for dim, rot, inter in sorted(parts):
        log(f"kv8 write: {rot} of {dim} interleaved={inter}")
        w = World(seed=rot, rows=1, heads=2, dim=dim)
        w.hold([5], extra=3)
        k, v = w.heads(1, 3, 2, dim, "bf16"), w.heads(1, 3, 2, dim, "bf16")
        r = Rotary(rot, interleaved=inter)
        w.cache.write(w.bt, 0, k, v, rotary=r)
        w.o.write(0, K.turn(np64(k), 5 + np.arange(3)[None], r.inv_freq, 1.0, inter), 1)
        w.o.write(1, np64(v), 1)
        pool, scales = w.planes()
        assert np.array_equal(scales, w.o.scales)
        assert np.mean(pool != w.o.pool) < 1e-5
