"""Queries that are not finite over slots that lie on no page: what a token does not see
does not reach it, whatever its query holds."""
import numpy as np
import pytest
import torch

from tests.gpu_support import device, log
from tests.kv8_support import World, i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("N,group,tree", [
    (1, 2, False), (1, 2, True),   # a wave a row block
    (7, 4, False), (7, 4, True),
    (40, 8, False), (40, 8, True),  # keys and values shared by four waves
])
def test_rows_without_pages(N, group, tree, bad):
    """Rows that hold no page, as padding of a batch, and tokens all of whose slots lie on
    missing pages, get 0 and -inf; the others what they get without them."""
    heads, dim, ps = 2, 64, 16
    w = World(seed=N + group, P=40, ps=ps, heads=heads, dim=dim, rows=5, M=8)
    w.hold([60, 60, 0, 33, 70], extra=N)
    o = w.o
    for b in (1, 2):
        o.tables[b] = [-1] * 8
    o.tables[3] = [-1, -1] + o.tables[3][2:]  # tokens see slots 32 and on
    w.push()
    log(f"attend without pages: N={N} group={group} tree={tree} {bad}")
    q = w.heads(5, N, heads * group, dim, "bf16")
    up = i32(w.tree(5, N)) if tree else None
    clean = w.cache.attend(w.bt, 0, q, parents=up)
    q[1, :, :, 5] = bad
    q[2, 0] = bad
    lse = torch.zeros(5, N, heads * group, device=device())
    got = w.cache.attend(w.bt, 0, q, parents=up, lse=lse)
    assert not got[1:3].any() and bool((lse[1:3] == -np.inf).all())
    keep = [0, 3, 4]
    assert torch.equal(got[keep], clean[keep]) and bool(lse[keep].isfinite().all())
    # a token that sees a slot has what its query gives
    q[3, 0, 0] = float("nan")
    got = w.cache.attend(w.bt, 0, q, parents=up)
    assert bool(got[3, 0, 0].isnan().all()) and torch.equal(got[0], clean[0])


@pytest.mark.parametrize("group", [1, 40])
def test_first_tokens_of_a_prompt_on_missing_pages(group):
    """The step's first page is missing: its tokens there see nothing, those behind it do."""
    N, dim, ps = 50, 64, 16
    w = World(seed=group, P=20, ps=ps, heads=1, dim=dim, rows=2, M=5)
    w.hold([0, 0], extra=N)
    w.o.tables[0][0] = -1
    w.push()
    q = w.heads(2, N, group, dim, "f16")
    clean = w.cache.attend(w.bt, 0, q)
    q[0, :16] = float("nan")
    got = w.cache.attend(w.bt, 0, q)
    assert not got[0, :16].any()
    assert torch.equal(got, clean)
