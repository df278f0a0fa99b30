"""Parity of ss_lmhead_quant_logits with the binary64 oracle.

Per logit the bound is oracle.quant.error_bound (every addition off by a step of
the largest partial sum), plus half a step of a bfloat16 output. Over a whole
result the roundings are independent: a group's g additions of partial sums that
grow as sqrt(k) 24 |x| leave sqrt(g) sqrt(g / 2) 24 2^-24 |x| at most, against
a result of sqrt(g) 4.6 |x|: (24 / 4.6) sqrt(g / 2) 2^-24 <= 2.5e-6 at g = 128,
so 1e-5 of the norm holds with room for the group sums."""
import numpy as np
import pytest
import torch

from oracle import quant as OQ
from speculative_decoding_verification_pipeline_amd import sampler as SM
from tests.gpu_support import device, log

pytestmark = pytest.mark.gpu


def make(B, V, K, group, zeros, scale, seed=0):
    g = torch.Generator().manual_seed(seed)
    ng = -(-K // group)
    x = torch.randn(B, K, generator=g).bfloat16()
    q = torch.randint(0, 256, (V, K // 2), generator=g, dtype=torch.uint8)
    s = (0.01 * torch.randn(V, ng, generator=g)).to(scale)  # either sign
    z = torch.randint(0, 256, (V, (ng + 1) // 2), generator=g, dtype=torch.uint8) if zeros else None
    return x, q, s, z


def expect(x, q, s, z, group):
    h, sc = x.float().numpy(), s.float().numpy()
    y = OQ.logits(h, q.numpy(), sc, None if z is None else z.numpy(), group)
    return y, OQ.error_bound(h, sc, group)


def call(sampler, x, q, s, z, group, **kw):
    d = device()
    return sampler.lmhead_quant_logits(x.to(d), q.to(d), s.to(d), group,
                                       zeros=None if z is None else z.to(d), **kw)


@pytest.mark.parametrize("B,V,K,group,zeros,scale,out", [
    (1, 1, 64, 32, False, "f16", "f32"),
    (1, 15, 64, 128, True, "bf16", "f32"),
    (2, 16, 128, 64, True, "f16", "bf16"),
    (1, 300, 448, 128, True, "f16", "f32"),
    (3, 129, 192, 32, True, "bf16", "f32"),
    (15, 127, 320, 64, False, "bf16", "f32"),
    (16, 513, 1024, 128, False, "f16", "f32"),
    (17, 200, 1088, 64, True, "f16", "f32"),
    (32, 257, 2048, 32, True, "f16", "bf16"),
    (33, 100, 1984, 128, True, "bf16", "f32"),
    (48, 1000, 512, 32, False, "f16", "f32"),
    (64, 777, 2112, 64, True, "bf16", "bf16"),
    (64, 5003, 1600, 128, True, "f16", "f32"),
    (7, 20011, 4160, 128, True, "f16", "f32"),
    (20, 33000, 256, 128, True, "f16", "f32"),
    (40, 70001, 192, 64, False, "f16", "f32"),
    (5, 130001, 128, 32, False, "f16", "f32"),
    # every choice of tiles, at sizes on both sides of its rule
    (64, 12288, 448, 64, True, "f16", "f32"),
    (36, 12289, 448, 128, True, "f16", "f32"),
    (40, 32768, 192, 32, True, "bf16", "f32"),
    (33, 40001, 256, 32, True, "f16", "f32"),
    (50, 40001, 192, 64, True, "f16", "f32"),
    (64, 65537, 320, 128, True, "f16", "f32"),
    (35, 65600, 576, 64, True, "f16", "bf16"),
    (17, 32768, 448, 64, False, "f16", "f32"),
    (31, 32769, 704, 32, True, "bf16", "f32"),
    (16, 32769, 1088, 64, True, "f16", "f32"),
    (2, 32767, 704, 128, True, "f16", "f32"),
    # one row: whole rows where the lanes are used, else the tiles
    (1, 301, 2048, 64, False, "f16", "f32"),
    (1, 18, 4096, 128, True, "bf16", "bf16"),
    (1, 5, 1664, 32, True, "f16", "f32"),
    (1, 37, 1600, 32, True, "f16", "f32"),
    (1, 33, 24576, 128, True, "f16", "f32"),
    (1, 3, 24640, 64, True, "f16", "f32"),
    (1, 1, 3776, 128, True, "f16", "f32"),
    (64, 16, 24640, 128, True, "f16", "f32"),
])
def test_matches_the_oracle(B, V, K, group, zeros, scale, out):
    log(f"quant: B={B} V={V} K={K} group={group} zeros={zeros} {scale} {out}")
    sc = torch.float16 if scale == "f16" else torch.bfloat16
    od = torch.float32 if out == "f32" else torch.bfloat16
    args = make(B, V, K, group, zeros, sc, seed=V + K)
    want, bound = expect(*args, group)
    s = SM.Sampler(B, V, hidden_size=K, device=0)
    got = call(s, *args, group, out_dtype=od)
    assert got.dtype == od and torch.equal(got, call(s, *args, group, out_dtype=od))
    got = got.double().cpu().numpy()
    half = 2.0 ** -8 if out == "bf16" else 0.0
    assert np.all(np.abs(got - want) <= bound + half * (np.abs(want) + bound))
    if out == "f32":
        assert np.linalg.norm(got - want) <= 1e-5 * np.linalg.norm(want)
    s.close()


@pytest.mark.parametrize("B,V,K,group", [
    (13, 32800, 1088, 128),   # one block left over, the last part shorter
    (8, 40000, 2048, 32),     # nearly half a round left over
    (16, 33500, 1600, 64),    # as many parts as stages
    (24, 32900, 1024, 128),
    (20, 67000, 768, 64),
    (64, 33500, 1024, 128),
    (64, 17000, 1024, 64),
    (33, 50000, 1088, 32),
    (50, 70000, 1280, 128),
    (33, 131100, 768, 128),   # behind two whole rounds
    (9, 32769, 128, 128),     # a single set: not cut
    # all row blocks cut, with K in two ranges inside each part
    (2, 1, 8192, 128),
    (16, 1000, 8192, 128),
    (3, 3001, 2112, 32),
    (24, 2999, 4160, 64),
    (40, 8192, 2048, 128),
    (64, 70, 24640, 32),
    (64, 1003, 3136, 64),
    (10, 20000, 2048, 64),    # one round and some blocks cut
    (64, 16384, 1024, 128),
    (1, 300, 4160, 128),      # one row that the tiles take
])
def test_left_over_row_blocks(B, V, K, group):
    """Row blocks behind a multiple of the CUs, or all of few, are cut along K between
    workgroups: eager, again, and in a graph replayed with other hidden states."""
    log(f"quant: left over, B={B} V={V} K={K} group={group}")
    x, q, sc, z = make(B, V, K, group, True, torch.float16, V + K)
    s = SM.Sampler(B, V, hidden_size=K, device=0)
    d = device()
    xd, qd, sd, zd = x.to(d), q.to(d), sc.to(d), z.to(d)
    out = torch.empty(B, V, device=d)

    def go(o=None):
        return s.lmhead_quant_logits(xd, qd, sd, group, zeros=zd, out=o)

    want, bound = expect(x, q, sc, z, group)
    go(out)
    got = out.double().cpu().numpy()
    assert np.all(np.abs(got - want) <= bound)
    assert np.linalg.norm(got - want) <= 1e-5 * np.linalg.norm(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go(out)
    for turn in range(4):
        if turn:
            xd.copy_(make(B, 1, K, group, False, torch.float16, turn)[0])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, go())
    xd.copy_(x)
    graph.replay()
    torch.cuda.synchronize()
    assert np.array_equal(out.double().cpu().numpy(), got)
    s.close()


@pytest.mark.parametrize("group", [32, 64, 128])
def test_every_weight_has_its_place(group):
    """One nonzero x per row: the logit is that weight times its scale, exactly
    (integers of at most 5 bits times scales of 2^-3 or 2^-2)."""
    B, V, K = 64, 48, 640
    g = torch.Generator().manual_seed(group)
    q = torch.randint(0, 256, (V, K // 2), generator=g, dtype=torch.uint8)
    ng = -(-K // group)
    sc = torch.where(torch.rand(V, ng, generator=g) < 0.5, 0.125, 0.25).half()
    z = torch.randint(0, 256, (V, (ng + 1) // 2), generator=g, dtype=torch.uint8)
    w = OQ.weights(q.numpy(), sc.float().numpy(), z.numpy(), group)
    s = SM.Sampler(B, V, hidden_size=K, device=0)
    for k0 in range(0, K, B):
        x = torch.zeros(B, K).bfloat16()
        x[torch.arange(B), k0 + torch.arange(B)] = 1.0
        got = call(s, x, q, sc, z, group).double().cpu().numpy()
        assert np.array_equal(got, w[:, k0:k0 + B].T)
    s.close()


@pytest.mark.parametrize("nibbles", [0x00, 0xFF, 0x88])
def test_constant_weights(nibbles):
    """Weights of 0, 15 and the default zero point (whose logits are exactly 0 for
    integer x: every sum is an integer below 2^24)."""
    B, V, K = 3, 70, 256
    g = torch.Generator().manual_seed(1)
    x = torch.randint(-8, 9, (B, K), generator=g).bfloat16()
    q = torch.full((V, K // 2), nibbles, dtype=torch.uint8)
    sc = torch.ones(V, 2).half()
    s = SM.Sampler(B, V, hidden_size=K, device=0)
    got = call(s, x, q, sc, None, 128).double().cpu().numpy()
    assert np.array_equal(got, (nibbles % 16 - 8.0) * x.double().numpy().sum(1)[:, None].repeat(V, 1))
    s.close()


def test_rows_are_independent_and_padding_stays():
    B, V, K = 19, 1003, 576
    x, q, sc, z = make(B, V, K, 64, True, torch.float16, 9)
    s = SM.Sampler(B, V, hidden_size=K, device=0)
    clean = call(s, x, q, sc, z, 64)
    x[4], x[11] = float("inf"), float("nan")
    buf = torch.full((B, V + 13), -5.0, device=device())
    out = call(s, x, q, sc, z, 64, out=buf[:, 3:V + 3])  # rows that start on any element
    rest = [b for b in range(B) if b not in (4, 11)]
    assert torch.equal(out[rest], clean[rest])
    assert bool((buf[:, :3] == -5).all()) and bool((buf[:, V + 3:] == -5).all())
    one = call(s, x[7:8], q, sc, z, 64)
    want, bound = expect(x[7:8], q, sc, z, 64)
    assert np.all(np.abs(one.double().cpu().numpy() - want) <= bound)
    s.close()


def test_captured_calls_replay():
    B, V, K = 6, 2000, 512
    x, q, sc, z = make(B, V, K, 128, True, torch.float16, 2)
    s = SM.Sampler(B, V, hidden_size=K, device=0)
    d = device()
    xd, qd, sd, zd = x.to(d), q.to(d), sc.to(d), z.to(d)
    out = torch.empty(B, V, device=d)
    s.lmhead_quant_logits(xd, qd, sd, 128, zeros=zd, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.lmhead_quant_logits(xd, qd, sd, 128, zeros=zd, out=out)
    for seed in range(3):
        xd.copy_(make(B, V, K, 128, True, torch.float16, 50 + seed)[0])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, s.lmhead_quant_logits(xd, qd, sd, 128, zeros=zd))
    s.close()


def test_weights_beyond_32_bit_offsets():
    """The last vocabulary rows of a weight of more than 2^32 bytes."""
    V, K, group = 131200, 65536, 128
    for B in (2, 40):
        log(f"quant: {V * K // 2} bytes of weights, B={B}")
        g = torch.Generator(device=device()).manual_seed(B)
        x = torch.randn(B, K, generator=g, device=device()).bfloat16()
        q = torch.randint(0, 256, (V, K // 2), generator=g, device=device(), dtype=torch.uint8)
        sc = (0.01 * torch.rand(V, K // group, generator=g, device=device())).half()
        z = torch.randint(0, 256, (V, K // group // 2), generator=g, device=device(), dtype=torch.uint8)
        s = SM.Sampler(B, V, hidden_size=K, device=0)
        got = s.lmhead_quant_logits(x, q, sc, group, zeros=z)
        for rows in (slice(0, 3), slice(V - 21, V)):
            want, bound = expect(x.cpu(), q[rows].cpu(), sc[rows].cpu(), z[rows].cpu(), group)
            assert np.all(np.abs(got[:, rows].double().cpu().numpy() - want) <= bound)
        s.close()


def test_refusals():
    B, V, K = 4, 100, 128
    x, q, sc, z = make(B, V, K, 32, True, torch.float16)
    d = device()
    x, q, sc, z = x.to(d), q.to(d), sc.to(d), z.to(d)
    s = SM.Sampler(B, V, hidden_size=K, device=0)
    good = dict(hidden=x, qweight=q, scales=sc, group=32, zeros=z)
    for change in ({"hidden": x.float()}, {"hidden": x[:, :64]}, {"hidden": x.t()},
                   {"qweight": q[:, :-1]}, {"qweight": q[:-1]}, {"qweight": q.char()},
                   {"scales": sc.float()}, {"scales": sc[:, :-1]}, {"group": 16}, {"group": 48},
                   {"group": 64}, {"zeros": z[:, :-1]}, {"zeros": z.int()},
                   {"out_dtype": torch.float16}, {"out": torch.empty(B, V - 1, device=d)},
                   {"out": torch.empty(V, B, device=d).t()}, {"qweight": q.cpu()}):
        with pytest.raises(ValueError):
            s.lmhead_quant_logits(**{**good, **change})
    with pytest.raises(SM.SamplerError):
        s.lmhead_quant_logits(**{**good, "hidden": torch.zeros(B + 1, K, device=d).bfloat16()})
    out = torch.empty(B, V, device=d)
    p = SM._ptr

    def raw(h=s.handle, x_=p(x), q_=p(q), s_=p(sc), sdt=2, g=32, n=B, o=p(out), odt=0, stride=V):
        return s.lib.ss_lmhead_quant_logits(h, x_, q_, s_, sdt, p(z), g, n, o, odt, stride, None)

    at = lambda t, k: SM.ctypes.c_void_p(t.data_ptr() + k)  # noqa: E731
    for c in (dict(x_=None), dict(q_=None), dict(s_=None), dict(o=None), dict(sdt=0), dict(odt=2),
              dict(n=0), dict(n=B + 1), dict(stride=V - 1), dict(s_=at(sc, 1)), dict(o=at(out, 2))):
        assert raw(**c) == SM.SS_ERR_INVALID_ARG, c
    for c in (dict(g=16), dict(g=256), dict(x_=at(x, 2)), dict(q_=at(q, 8))):
        assert raw(**c) == SM.SS_ERR_UNSUPPORTED, c
    plain = SM.Sampler(B, V, device=0)  # no hidden size
    assert raw(h=plain.handle) == SM.SS_ERR_INVALID_ARG
    plain.close()
    assert raw() == SM.SS_OK
    s.close()


def test_the_parts_take_no_workspace_of_their_own():
    """Partial sums lie in the scratch of whole rows, which the other calls use between
    them; only what ss_lmhead_sample needs (8 + 64 bytes per row and 128 vocabulary
    rows) and the counters come with a hidden size."""
    for V, B in ((128256, 64), (32000, 64)):
        with_head, without = (SM.Sampler(B, V, hidden_size=k, device=0) for k in (8192, 0))
        extra = with_head.workspace_bytes() - without.workspace_bytes()
        assert 0 < extra <= 64 * 72 * -(-V // 128) + (256 << 10)
        with_head.close()
        without.close()
    V, K = 3000, 1024
    for B in (1, 7, 30, 64):
        log(f"quant: shared scratch B={B}")
        x, q, sc, z = make(B, V, K, 64, True, torch.float16, B)
        s, fresh = SM.Sampler(B, V, hidden_size=K, device=0), SM.Sampler(B, V, device=0)
        want = call(s, x, q, sc, z, 64).clone()
        # rows whose filters keep more than the candidates: selected over their scratch
        p = SM.SamplingParams(temperature=torch.full((B,), 5.0, device=device()),
                              top_p=torch.full((B,), 0.999, device=device()), seed=5)
        wide = torch.randn(B, V, generator=torch.Generator().manual_seed(B)).to(device())
        tokens = fresh.sample(wide, p)
        for turn in range(3):
            assert torch.equal(call(s, x, q, sc, z, 64), want)
            assert torch.equal(s.sample(wide, p), tokens)
        s.close()
        fresh.close()
