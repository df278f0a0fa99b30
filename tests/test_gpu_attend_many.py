"""Long prompts, batches of prompts and large trees: blocks of 128 rows whose waves take 32
each, whole requests and cut ones, against the definition in binary64."""
import pytest

from tests.gpu_support import log
from tests.kv8_support import World
from tests.test_gpu_attend import check

pytestmark = pytest.mark.gpu

CASES = [
    # B, N, heads, group, dim, page, longest context, tree
    (64, 20, 4, 4, 128, 16, 90, True),     # one block of 80 rows, cut into shares over requests
    (64, 20, 4, 4, 128, 32, 90, False),
    (64, 20, 4, 4, 80, 16, 60, False),
    (64, 20, 4, 4, 96, 48, 60, True),
    (64, 20, 4, 4, 64, 16, 150, False),
    (16, 64, 8, 8, 128, 16, 200, True),    # four blocks of rows, cut
    (2, 260, 32, 4, 128, 64, 40, False),   # nine blocks of 32 heads: whole requests
]


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_blocks_of_128_rows(case, dtype):
    B, N, heads, group, dim, ps, most, tree = CASES[case]
    M = -(-(most + N) // ps)
    w = World(seed=case, P=B * M + 2, ps=ps, heads=heads, dim=dim, rows=B, M=M)
    lens = [int(x) for x in w.rng.integers(0, most + 1, B)]
    lens[0], lens[1] = most, 0
    w.hold(lens, extra=N)
    log(f"attend many rows: {CASES[case]} {dtype}")
    q = w.heads(B, N, heads * group, dim, dtype)
    step = {"parents": w.tree(B, N, lost=0.05)} if tree else {}
    step["counts"] = [N] + [int(x) for x in w.rng.integers(0, N + 1, B - 1)]
    check(w, q, dtype, "many rows", **step)
