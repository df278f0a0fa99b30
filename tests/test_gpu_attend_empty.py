"""Requests without tokens between others that have some, a workgroup each: all their rows
become 0 and -inf, whatever the output held."""
import numpy as np
import pytest
import torch

from tests.gpu_support import device, log
from tests.kv8_support import World, i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N,heads,group", [(1, 8, 2), (9, 7, 4), (40, 8, 4)])
@pytest.mark.parametrize("tree", [False, True])
def test_requests_without_tokens(N, heads, group, tree):
    B, ps = 300, 16
    M = -(-(20 + N) // ps)
    w = World(seed=N, P=B * M + 2, ps=ps, heads=heads, dim=64, rows=B, M=M)
    w.hold([int(x) for x in w.rng.integers(0, 21, B)], extra=N)
    log(f"attend empty requests: N={N} heads={heads} group={group} tree={tree}")
    q = w.heads(B, N, heads * group, 64, "bf16")
    up = i32(w.tree(B, N)) if tree else None
    full, lse_full = torch.empty_like(q), torch.empty(B, N, heads * group, device=device())
    w.cache.attend(w.bt, 0, q, parents=up, out=full, lse=lse_full)
    empty = w.rng.random(B) < 0.5
    for how in (dict(counts=i32(np.where(empty, 0, N))), dict(reserved=i32(~empty)),
                dict(lens=torch.where(i32(empty) > 0, -1, w.bt.lens))):
        out, lse = torch.full_like(q, 3.0), torch.full_like(lse_full, 3.0)
        w.cache.attend(w.bt, 0, q, parents=up, out=out, lse=lse, **how)
        mask = torch.from_numpy(empty).to(device())
        assert not out[mask].any() and bool((lse[mask] == -np.inf).all())
        assert torch.equal(out[~mask], full[~mask]) and torch.equal(lse[~mask], lse_full[~mask])
