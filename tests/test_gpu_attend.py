"""Attention over pages of 8-bit floats against the definition in binary64
(oracle.kv8.Pages8.attend), with bounds from the roundings that are made."""
import numpy as np
import pytest
import torch

from speculative_decoding_verification_pipeline_amd import sampler as SM
from speculative_decoding_verification_pipeline_amd.cache import PageCache
from tests.gpu_support import device, log
from tests.kv8_support import World, attention_bound, i32, np64

pytestmark = pytest.mark.gpu


def check(w, q, dtype, what, out=None, lse=None, **step):
    """One call against the definition."""
    host = {k: v for k, v in step.items() if v is not None}
    dev = {"lens" if k == "base" else k: i32(v) for k, v in host.items()}
    got_lse = torch.full(q.shape[:3], 7.0, device=device())
    got = w.cache.attend(w.bt, 0, q, lse=got_lse, out=out, **dev)
    scale = float(np.float32(q.shape[3] ** -0.5))
    want, lse, size, dots, least = w.o.attend(np64(q), scale, **host)
    slots = w.o.M * w.o.ps
    bound = attention_bound(dtype, want, size, dots, least, slots, q.shape[3])
    a = np64(got)
    with np.errstate(invalid="ignore"):
        fine = np.abs(a - want) <= bound
    if dtype == "f16":  # from 65520 on the nearest float16 is an infinity
        fine |= np.isinf(a) & (np.sign(a) == np.sign(want)) & (np.abs(want) + bound >= 65520)
    assert np.all(fine), (what, float(np.nanmax(np.abs(a - want) - bound)))
    seen = lse > -np.inf
    a = np64(got_lse)
    assert np.array_equal(a > -np.inf, seen), what
    rel = 2 * (q.shape[3] + 4) * 2.0 ** -23 * dots + 2.0 ** -15 + (slots + 8) * 2.0 ** -23
    assert np.all(np.abs(a[seen] - lse[seen]) <= rel[seen] + 2.0 ** -22 * np.abs(lse[seen])), what
    return got


SHAPES = [
    # heads, group, dim, page, block, layout
    (1, 1, 64, 16, 16, "nhd"),
    (2, 8, 128, 16, 16, "nhd"),
    (2, 3, 80, 32, 16, "hnd"),
    (1, 16, 16, 16, 16, "padded"),
    (1, 5, 256, 64, 32, "separate"),
    (3, 2, 96, 48, 16, "nhd"),
    (2, 4, 144, 64, 64, "hnd"),
    (1, 7, 128, 128, 64, "padded"),
]


@pytest.mark.parametrize("shape", range(len(SHAPES)))
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_single_tokens(shape, dtype):
    heads, group, dim, ps, block, layout = SHAPES[shape]
    lens = [0, 1, 14, 15, 16, 31, 33, 127, 128, 200]
    M = -(-201 // ps)
    w = World(seed=shape, P=10 * M + 2, ps=ps, heads=heads, dim=dim, block=block, rows=10, M=M,
              layout=layout)
    w.hold(lens, extra=1)
    log(f"attend single: {SHAPES[shape]} {dtype}")
    q = w.heads(10, 1, heads * group, dim, dtype)
    check(w, q, dtype, "single")
    check(w, q, dtype, "counts", counts=[1, 0, 2, 1, -1, 1, 1, 0, 1, 1], reserved=[1] * 5 + [0] + [1] * 4)


@pytest.mark.parametrize("shape", range(len(SHAPES)))
@pytest.mark.parametrize("N", [2, 13, 64])
def test_trees(shape, N):
    heads, group, dim, ps, block, layout = SHAPES[shape]
    M = -(-(130 + N) // ps)
    w = World(seed=shape + N, P=4 * M + 2, ps=ps, heads=heads, dim=dim, block=block, rows=4, M=M,
              layout=layout)
    w.hold([0, 5, 64, 130], extra=N)
    log(f"attend tree: {SHAPES[shape]} N={N}")
    dtype = "bf16" if shape % 2 else "f16"
    q = w.heads(4, N, heads * group, dim, dtype)
    check(w, q, dtype, "tree", parents=w.tree(4, N))
    check(w, q, dtype, "tree with lost nodes", parents=w.tree(4, N, lost=0.3), counts=[N, 1, N - 1, N])


@pytest.mark.parametrize("shape", range(len(SHAPES)))
@pytest.mark.parametrize("N", [3, 37, 150])
def test_prompts(shape, N):
    heads, group, dim, ps, block, layout = SHAPES[shape]
    M = -(-(70 + N) // ps)
    w = World(seed=shape + N, P=3 * M + 2, ps=ps, heads=heads, dim=dim, block=block, rows=3, M=M,
              layout=layout)
    w.hold([0, 70, 33], extra=N)
    log(f"attend prompt: {SHAPES[shape]} N={N}")
    dtype = "f16" if shape % 2 else "bf16"
    q = w.heads(3, N, heads * group, dim, dtype)
    check(w, q, dtype, "prompt", counts=[N, N - 1, N // 2])


@pytest.mark.parametrize("B,N,len_", [(1, 1, 9000), (2, 1, 5000), (3, 4, 2100), (70, 1, 300)])
def test_long_rows_are_cut(B, N, len_):
    """Rows cut into pieces and joined; uneven rows, one of them empty."""
    ps = 32
    M = -(-(len_ + N) // ps)
    w = World(seed=B, P=B * M + 2, ps=ps, heads=2, dim=64, rows=B, M=M)
    lens = [len_] + [int(x) for x in w.rng.integers(0, len_, B - 1)]
    if B > 2:
        lens[1] = 0
    w.hold(lens, extra=N)
    log(f"attend long: B={B} N={N} {len_}")
    q = w.heads(B, N, 4, 64, "bf16")
    a = check(w, q, "bf16", "long")
    # the same bits again: nothing depends on the order in which workgroups end
    for _ in range(3):
        assert torch.equal(a, w.cache.attend(w.bt, 0, q))


@pytest.mark.parametrize("B,N,heads,group,tree", [
    (300, 1, 4, 2, False),    # few rows, 16 of them a workgroup
    (257, 5, 4, 4, False),    # few rows, 32
    (300, 9, 7, 4, True),    # many rows, a block of 64 each
    (1, 140, 260, 1, False),  # more blocks of rows than shares
])
def test_whole_requests(B, N, heads, group, tree):
    """Requests enough that each is a workgroup's, uneven ones, empty ones among them."""
    ps = 16
    M = -(-(40 + N) // ps)
    w = World(seed=B + N, P=B * M + 2, ps=ps, heads=heads, dim=16, rows=B, M=M)
    lens = [int(x) for x in w.rng.integers(0, 41, B)]
    if B > 1:
        lens[0] = lens[B - 1] = 0
    w.hold(lens, extra=N)
    log(f"attend whole requests: B={B} N={N} heads={heads}")
    q = w.heads(B, N, heads * group, 16, "bf16")
    step = {"parents": w.tree(B, N)} if tree else {}
    if B > 1:
        step["counts"] = [N if b % 7 else 0 for b in range(B)]
    check(w, q, "bf16", "whole", **step)


def test_peaks_and_rising_scores():
    """A score that towers over the others, first, in the middle and last, and scores that
    rise slot by slot: the running reference moves."""
    w = World(seed=3, P=40, ps=32, heads=1, dim=64, rows=4, M=8)
    w.hold([200, 200, 200, 200], extra=1)
    o = w.o
    for b, at in enumerate([0, 97, 200, None]):
        for s in range(201):
            page = o.tables[b][s // 32]
            o.scales[0, page, :] = 120
            x = 0x70 if s == at else 0x20  # 128 and 0.125
            o.pool[0, page, s % 32] = 0x20 + s // 3 if at is None else x
    w.put()
    q = torch.ones(4, 1, 2, 64, dtype=torch.bfloat16, device=device())
    q[:, :, 1] = -4.0
    check(w, q, "bf16", "peaks")


def test_missing_pages_and_rows_behind_the_table():
    w = World(seed=5, P=40, ps=16, heads=2, dim=64, rows=5, M=6)
    w.hold([60, 60, 60, 90, 10], extra=8)
    o = w.o
    o.tables[0][1] = -1
    o.tables[1] = [-1] * 6            # a row without any page: nothing to see
    o.tables[2][0] = 1 << 24          # no such page
    w.push()
    q = w.heads(5, 8, 4, 64, "bf16")
    base = [60, 60, 60, 92, -1]       # the fourth row's step ends behind its table
    check(w, q, "bf16", "pages", base=base)
    check(w, q[:4].contiguous(), "bf16", "far", base=[97, 2 ** 31 - 1, 96, 0])


def test_what_a_token_does_not_see_does_not_reach_it():
    """Every byte that no token sees is a NaN, scales among it; then values that some see."""
    w = World(seed=6, P=16, ps=16, heads=2, dim=64, rows=3, M=5)
    N = 9
    w.hold([37, 0, 16], extra=N)
    o = w.o
    up = w.tree(3, N)
    up[0][4] = 9                       # seen by itself only, and it sees nothing
    q = w.heads(3, N, 4, 64, "f16")
    counts = [9, 5, 9]
    pool = np.full_like(o.pool, 0x7f)
    scales = np.where(np.indices(o.scales.shape).sum(0) % 2, 255, 0).astype(np.uint8)
    for b in range(3):
        for s in range(o.lens[b] + counts[b]):
            page = o.tables[b][s // 16]
            pool[:, page, s % 16] = o.pool[:, page, s % 16]
            scales[:, page] = o.scales[:, page]
    page, at = o.tables[0][(37 + 4) // 16], (37 + 4) % 16
    pool[:, page, at] = 0xff           # the lost node's own slot
    o.pool, o.scales = pool, scales
    w.put()
    for kw in (dict(parents=up, counts=counts), dict(counts=[4, 5, 9])):
        got = check(w, q, "f16", "unseen", **kw)
        assert not got.isnan().any()
    # one value, of node 3 of row 2: its row's entry in the tokens that see node 3
    page, at = o.tables[2][(16 + 3) // 16], (16 + 3) % 16
    pool[1, page, at, 1, 21] = 0x7f
    w.put()
    from oracle.kv8 import above
    got = w.cache.attend(w.bt, 0, q, parents=i32(up), counts=i32(counts)).isnan().cpu().numpy()
    want = np.zeros_like(got)
    want[2, above(up[2])[:, 3], 2:, 21] = True
    assert np.array_equal(got, want)
    got = w.cache.attend(w.bt, 0, q, counts=i32(counts)).isnan().cpu().numpy()
    want[:] = False
    want[2, 3:, 2:, 21] = True
    want[0, 4:] = True                 # without a tree, those behind it see the NaN of row 0
    assert np.array_equal(got, want)
    # and a key: the whole row of those that see it
    pool[1, page, at, 1, 21] = 0
    pool[0, page, at, 0, 5] = 0xff
    w.put()
    got = w.cache.attend(w.bt, 0, q, parents=i32(up), counts=i32(counts)).isnan().cpu().numpy()
    want[:] = False
    want[2, above(up[2])[:, 3], :2] = True
    assert np.array_equal(got, want)


def test_queries_that_are_not_finite_stay_in_their_rows():
    w = World(seed=8, P=20, ps=16, heads=1, dim=64, rows=2, M=8)
    w.hold([100, 3], extra=3)
    q = w.heads(2, 3, 4, 64, "bf16")
    clean = w.cache.attend(w.bt, 0, q)
    q[0, 1, 2, 5] = float("nan")
    q[1, 0, 0, 0] = float("inf")
    got = w.cache.attend(w.bt, 0, q)
    bad = got.isnan().any(-1)
    assert bool(bad[0, 1, 2]) and bool(bad[1, 0, 0]) and int(bad.sum()) == 2
    keep = ~bad
    assert torch.equal(got[keep], clean[keep])


def test_scales_far_apart():
    """Blocks of values 2^70 apart, weights that favour the small ones."""
    w = World(seed=10, P=12, ps=16, heads=1, dim=64, rows=1, M=8)
    w.hold([120], extra=1)
    w.o.scales[1] = w.rng.choice([92, 127, 162], w.o.scales[1].shape)
    w.put()
    check(w, w.heads(1, 1, 2, 64, "bf16", 3.0), "bf16", "far apart")


def test_strides_outputs_and_streams():
    w = World(seed=12, P=20, ps=16, heads=2, dim=64, rows=3, M=6, layers=2)
    w.hold([40, 7, 80], extra=5)
    qkv = w.heads(3, 6, 9, 64, "bf16")
    q = qkv[:, :5, 2:8]
    want = w.cache.attend(w.bt, 0, q.contiguous())
    big = torch.full((4, 7, 8, 80), 3.0, dtype=torch.bfloat16, device=device())
    out = big[:3, 1:6, 1:7, 8:72]
    assert w.cache.attend(w.bt, 0, q, out=out) is out
    assert torch.equal(out, want)
    big[:3, 1:6, 1:7, 8:72] = 3.0
    assert bool((big == 3.0).all())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = w.cache.attend(w.bt, 0, q, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    half = w.cache.attend(w.bt, 0, q, scale=0.03)
    assert not torch.equal(half, want)
    other = w.cache.attend(w.bt, 1, q)
    assert not torch.equal(other, want)
    assert w.cache.attend(w.bt, 0, q[:0]).shape == (0, 5, 6, 64)


def test_graphs_of_one_handle():
    """Two calls in two graphs of one handle, replayed one after the other with lengths
    changed in place: each replay equals the eager call."""
    w = World(seed=14, P=150, ps=32, heads=2, dim=64, rows=2, M=70)
    w.hold([1900, 30], extra=60)
    q1, q2 = w.heads(2, 1, 8, 64, "bf16"), w.heads(2, 8, 8, 64, "bf16")
    up = i32(w.tree(2, 8))
    o1, o2 = torch.empty_like(q1), torch.empty_like(q2)
    w.cache.attend(w.bt, 0, q1)
    graphs = []
    for call in (lambda: w.cache.attend(w.bt, 0, q1, out=o1),
                 lambda: w.cache.attend(w.bt, 0, q2, parents=up, out=o2)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        graphs.append(g)
    for lens in ([1900, 30], [5, 1000], [0, 0], [1950, 1]):
        w.bt.lens.copy_(i32(lens))
        q1.copy_(torch.randn(q1.shape).bfloat16())
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o1, w.cache.attend(w.bt, 0, q1))
        assert torch.equal(o2, w.cache.attend(w.bt, 0, q2, parents=up))


def test_two_handles_at_once():
    """Calls of two handles on two streams, each as alone."""
    ws = [World(seed=s, P=140, ps=32, heads=2, dim=64, rows=1, M=130) for s in (1, 2)]
    for w in ws:
        w.hold([4000], extra=1)
    qs = [w.heads(1, 1, 8, 64, "bf16") for w in ws]
    want = [w.cache.attend(w.bt, 0, q) for w, q in zip(ws, qs)]
    streams = [torch.cuda.Stream() for _ in ws]
    torch.cuda.synchronize()
    for _ in range(20):
        got = [w.cache.attend(w.bt, 0, q, stream=s) for w, q, s in zip(ws, qs, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_refusals():
    w = World(rows=2, heads=2)
    w.hold([3, 4], extra=4)
    q = torch.zeros(2, 4, 4, 64, dtype=torch.bfloat16, device=device())
    for bad in (dict(layer=1), dict(queries=q.float()), dict(queries=q[..., :32]), dict(queries=q[:, :, :3]),
                dict(queries=q[:, :0]), dict(out=q.half()), dict(out=q[:, :1].expand(2, 4, 4, 64)),
                dict(lse=torch.zeros(2, 4, 3, device=device())), dict(parents=i32([[0, 0]])),
                dict(lens=i32([0])), dict(queries=torch.zeros(2, 97, 4, 64, dtype=torch.bfloat16, device=device())),
                dict(queries=torch.zeros(2, 65, 4, 64, dtype=torch.bfloat16, device=device()),
                     parents=torch.zeros(2, 65, dtype=torch.int32, device=device())),
                dict(queries=torch.zeros(3, 4, 4, 64, dtype=torch.bfloat16, device=device()))):
        args = dict(layer=0, queries=q)
        args.update(bad)
        if "queries" in bad and bad["queries"].shape[0] == 3:
            w.bt.tables = w.bt.tables[:2]
            w.bt.lens = w.bt.lens[:2]
        with pytest.raises(ValueError):
            w.cache.attend(w.bt, **args)
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises(SM.SamplerError) as e:
            w.cache.attend(w.bt, 0, q, scale=scale)
        assert e.value.status == SM.SS_ERR_INVALID_ARG
    odd = torch.zeros(2 * 4 * 4 * 64 + 1, dtype=torch.bfloat16, device=device())[1:].view(2, 4, 4, 64)
    with pytest.raises(SM.SamplerError) as e:
        w.cache.attend(w.bt, 0, odd)
    assert e.value.status == SM.SS_ERR_UNSUPPORTED
    plain = PageCache(torch.zeros(2, 4, 16, 1, 16, dtype=torch.uint8, device=device()), 2, 2)
    with pytest.raises(ValueError):
        plain.attend(plain.new_tables(), 0, q)
