"""Measured calls of three operators that stand around speculative verification.

* ``verify``: drafted tokens checked against probability rows with uniforms that
  the caller drew (Sampler.spec_verify_probs).
* ``cache``: the pages of a key/value cache around a verification step: reserving
  slots, forking with copy on write, compacting an accepted tree path, releasing
  and copying pages (PageCache).
* ``head``: LM-head logits from 4-bit weights with group scales
  (Sampler.lmhead_quant_logits).

``run`` computes the plain form with elementary torch operations, or calls the
framework where ``own`` is true.
"""
import torch

own = False

_F = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_BYTES = {"f32": 4, "bf16": 2, "f16": 2}


def listed():
    return [
        # one interactive request, a small vocabulary: latency
        {"name": "verify 1x4x32000 f32", "op": "verify", "B": 1, "G": 4, "V": 32000, "dtype": "f32",
         "rows": True, "ragged": False},
        # the library's own speculative batch: every request drafts 4 tokens
        {"name": "verify 32x4x128256 f32", "op": "verify", "B": 32, "G": 4, "V": 128256,
         "dtype": "f32", "rows": True, "ragged": False},
        # a serving batch of greedy drafts (one-hot, no draft rows), odd vocabulary, ragged drafts
        {"name": "verify 48x5x50257 greedy", "op": "verify", "B": 48, "G": 5, "V": 50257,
         "dtype": "f32", "rows": False, "ragged": True},
        # a large batch whose probabilities are kept in 16 bits, ragged drafts
        {"name": "verify 64x7x152064 bf16", "op": "verify", "B": 64, "G": 7, "V": 152064,
         "dtype": "bf16", "rows": True, "ragged": True},
        # requests end and others are admitted: pages freed and handed out, nothing copied
        {"name": "cache admit 32", "op": "cache", "kind": "admit", "B": 32, "layers": 1, "heads": 1,
         "dim": 64, "page": 16, "pages": 16384, "len": 4000, "N": 0, "layout": "nhd"},
        # the cache's part of one tree step of a few requests
        {"name": "cache step 4", "op": "cache", "kind": "step", "B": 4, "layers": 8, "heads": 2,
         "dim": 64, "page": 16, "pages": 512, "len": 900, "N": 16, "layout": "nhd"},
        # the same of a full batch: 32 layers of 8 heads of 128
        {"name": "cache step 64", "op": "cache", "kind": "step", "B": 64, "layers": 32, "heads": 8,
         "dim": 128, "page": 16, "pages": 768, "len": 100, "N": 16, "layout": "nhd"},
        # parallel samples of a few prompts: prefix shared, the partial page copied on write
        {"name": "cache fork 48", "op": "cache", "kind": "fork", "B": 48, "layers": 24, "heads": 4,
         "dim": 128, "page": 32, "pages": 256, "len": 300, "N": 4, "layout": "hnd"},
        # pages copied to others, as where a request is duplicated whole
        {"name": "cache copy 100", "op": "cache", "kind": "copy", "B": 100, "layers": 32, "heads": 8,
         "dim": 128, "page": 16, "pages": 256, "len": 0, "N": 0, "layout": "nhd"},
        # a draft model's head, one token
        {"name": "head 1x32000x2048", "op": "head", "B": 1, "V": 32000, "K": 2048, "group": 64,
         "zeros": False, "out": "f32", "scale": "f16"},
        # a small batch, odd vocabulary, a last group that is half full
        {"name": "head 13x50257x4160", "op": "head", "B": 13, "V": 50257, "K": 4160, "group": 128,
         "zeros": True, "out": "f32", "scale": "f16"},
        # the library's own LM-head shape at its largest batch
        {"name": "head 64x128256x8192", "op": "head", "B": 64, "V": 128256, "K": 8192, "group": 128,
         "zeros": True, "out": "bf16", "scale": "bf16"},
    ]


def _span(rng, lo, hi):
    """A whole number, even over the logarithm of [lo, hi]."""
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["verify", "cache", "head"])
    if op == "verify":
        return {"op": op, "B": _span(rng, 1, 64), "G": rng.randint(1, 7), "V": _span(rng, 1000, 152064),
                "dtype": rng.choice(["f32", "bf16", "f16"]) if rng.random() < 0.5 else "f32",
                "rows": rng.random() < 0.7, "ragged": rng.random() < 0.5}
    if op == "head":
        return {"op": op, "B": _span(rng, 1, 64), "V": _span(rng, 1000, 128256),
                "K": 64 * _span(rng, 4, 128), "group": rng.choice([32, 64, 128]),
                "zeros": rng.random() < 0.5, "out": rng.choice(["f32", "bf16"]),
                "scale": rng.choice(["f16", "bf16"])}
    kind = rng.choice(["admit", "step", "fork", "copy"])
    page = rng.choice([16, 32, 64])
    c = {"op": op, "kind": kind, "layers": _span(rng, 1, 32), "heads": rng.choice([1, 2, 4, 8]),
         "dim": rng.choice([64, 80, 128]), "page": page, "layout": rng.choice(["nhd", "hnd"])}
    if kind == "admit":
        n = _span(rng, 2, 64)
        c.update(B=n, layers=1, heads=1, len=_span(rng, 64, 4000), N=0)
        c["pages"] = 2 * n * (c["len"] // page + 2)
    elif kind == "step":
        n = _span(rng, 1, 64)
        c.update(B=n, len=rng.randint(1, 200), N=rng.randint(2, 32))
        c["pages"] = n * ((c["len"] * 3 // 2 + c["N"]) // page + 4)
    elif kind == "fork":
        n = _span(rng, 2, 48)
        c.update(B=n, len=rng.randint(1, 300), N=rng.randint(1, 4))
        c["pages"] = n * 3 + 4 * (c["len"] * 3 // 2 // page + 4)
    else:
        n = _span(rng, 1, 100)
        c.update(B=n, pages=2 * n + rng.randint(0, 50), len=0, N=0)
    while 2 * c["layers"] * c["pages"] * page * c["heads"] * c["dim"] > 2 * 32 * 768 * 16 * 1024:
        c["layers"] = max(1, c["layers"] // 2)
        if c["layers"] == 1:
            break
    return c


# --------------------------------------------------------------------------
# inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


_samplers = {}


def _sampler(**limits):
    """The sampler handle of a program with these limits on this device and stream
    (calls that overlap in time need handles of their own): made once, kept. Of more
    than four the one made first is let go; states that use it keep it."""
    from speculative_decoding_verification_pipeline_amd.sampler import Sampler
    device = torch.cuda.current_device()
    key = (device, torch.cuda.current_stream().cuda_stream, *sorted(limits.items()))
    if key not in _samplers:
        if len(_samplers) == 4:
            del _samplers[next(iter(_samplers))]
        _samplers[key] = Sampler(device=device, **limits)
    return _samplers[key]


def _prepare_verify(case, seed):
    """Zipf-like target rows, drafts from a noisy copy of the target."""
    B, G, V, dt = case["B"], case["G"], case["V"], _F[case["dtype"]]
    g = _gen(seed)
    rank = torch.arange(1, V + 1, device="cuda", dtype=torch.float32)
    base = -2.0 * torch.log(rank)
    perm = torch.rand(B, V, generator=g, device="cuda").argsort(1)
    x = base[perm][:, None] + 0.3 * torch.randn(B, G + 1, V, generator=g, device="cuda")
    y = x[:, :G] + 0.5 * torch.randn(B, G, V, generator=g, device="cuda")
    target, draft = torch.softmax(x, -1).to(dt), None
    if case["rows"]:
        draft = torch.softmax(y, -1).to(dt)
        y -= torch.empty_like(y).exponential_(generator=g).log_()  # Gumbel noise: drafts drawn from q
    tokens = y.argmax(-1).int()
    u = torch.rand(B, G + 1, generator=g, device="cuda")
    n = None
    if case["ragged"]:
        n = torch.randint(0, G + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    st = {"op": "verify", "target": target, "draft": draft, "tokens": tokens, "u": u, "n": n}
    if own:
        st["sampler"] = _sampler(max_batch=64, vocab_size=V, max_draft=7)
    return st


def _prepare_head(case, seed):
    B, V, K, grp = case["B"], case["V"], case["K"], case["group"]
    g = _gen(seed)
    ng = -(-K // grp)
    st = {"op": "head", "group": grp, "out": _F[case["out"]],
          "x": torch.randn(B, K, generator=g, device="cuda").bfloat16(),
          "q": torch.randint(0, 256, (V, K // 2), generator=g, device="cuda", dtype=torch.uint8),
          "s": (0.004 * (0.5 + torch.rand(V, ng, generator=g, device="cuda"))).to(_F[case["scale"]]),
          "z": None}
    if case["zeros"]:
        st["z"] = torch.randint(0, 256, (V, -(-ng // 2)), generator=g, device="cuda",
                                dtype=torch.uint8)
    if own:
        st["sampler"] = _sampler(max_batch=64, vocab_size=V, hidden_size=K)
    return st


def _prepare_cache(case, seed):
    """A pool with its block tables: rows hold pages in a shuffled order."""
    B, ps, P, kind = case["B"], case["page"], case["pages"], case["kind"]
    g = _gen(seed)
    shape = (2 * case["layers"], P, ps, case["heads"], case["dim"])
    if case["layout"] == "hnd":  # heads outside the slots of a page
        a, b, c, d, e = shape
        pool = torch.empty(a, b, d, c, e, device="cuda", dtype=torch.bfloat16)
        pool.normal_(generator=g)
        pool = pool.transpose(2, 3)
    else:
        pool = torch.empty(shape, device="cuda", dtype=torch.bfloat16)
        pool.normal_(generator=g)
    st = {"op": "cache", "kind": kind, "pool": pool, "page": ps}
    perm = torch.randperm(P, generator=g, device="cuda").int()
    if kind == "copy":
        st["src"], st["dst"] = perm[:B].contiguous(), perm[B:2 * B].contiguous()
    else:
        L, N = case["len"], case["N"]
        M = (L * 3 // 2 + N) // ps + 2
        lens = torch.randint(max(1, L // 2), L * 3 // 2 + 1, (B,), generator=g, device="cuda",
                             dtype=torch.int32)
        rows = torch.arange(B, device="cuda")
        if kind == "fork":  # the first N rows are prompts, the others samples of them
            roots = min(N, B - 1)
            lens[roots:] = 0
            st["src"] = torch.randint(0, roots, (B - roots,), generator=g, device="cuda",
                                      dtype=torch.int32)
            st["dst"] = rows[roots:].int()
            st["add"] = (rows >= roots).int()
        if kind == "admit":  # every other request ends; as many of other lengths are admitted
            st["rows"] = rows[::2].int()
            st["keep"] = torch.zeros_like(st["rows"])
            st["add"] = torch.where(rows % 2 == 0, lens, torch.ones_like(lens)).int()
            st["base"] = torch.where(rows % 2 == 0, torch.zeros_like(lens), lens).int()
        if kind == "step":
            st["N"] = N
            st["add"] = torch.full((B,), N, device="cuda", dtype=torch.int32)
            st["base"] = lens.clone()
            # accepted tree nodes: ascending, distinct, node 0 is the root
            pick = torch.rand(B, N - 1, generator=g, device="cuda").argsort(1).int() + 1
            st["acc"] = torch.randint(0, min(N, 6), (B,), generator=g, device="cuda",
                                      dtype=torch.int32)
            cols = torch.arange(N - 1, device="cuda")
            pick = torch.where(cols < st["acc"][:, None], pick, pick + N).sort(1).values
            nodes = torch.where(cols < st["acc"][:, None], pick, torch.full_like(pick, -1))
            st["nodes"] = torch.cat([nodes, torch.full((B, 1), -1, device="cuda")], 1).int().contiguous()
        held = (lens + ps - 1) // ps
        cols = torch.arange(M, device="cuda")
        used = cols[None, :] < held[:, None]
        at = (used.flatten().cumsum(0) - 1).reshape(B, M)
        st["tables"] = torch.where(used, perm[at.clamp(0, P - 1)], torch.full_like(perm[:1], -1)).contiguous()
        ref = torch.zeros(P, device="cuda", dtype=torch.int32)
        ref[perm] = (torch.arange(P, device="cuda") < used.sum()).int()
        st["ref"], st["lens"] = ref, lens
    if own:
        from speculative_decoding_verification_pipeline_amd.cache import BlockTables, PageCache
        if kind != "copy":
            st["bt"] = BlockTables(st["tables"], st["ref"], st["lens"])
        st["cache"] = PageCache(pool, max_batch=B, max_blocks=1 if kind == "copy" else M)
    return st


def prepare(case, seed):
    return {"verify": _prepare_verify, "cache": _prepare_cache, "head": _prepare_head}[case["op"]](case, seed)


# --------------------------------------------------------------------------
# the plain forms

def _plain_verify(st):
    p, q, d, u = st["target"], st["draft"], st["tokens"].long(), st["u"].double()
    B, G1, V = p.shape
    G = G1 - 1
    j = torch.arange(G, device=p.device)
    row = torch.arange(B, device=p.device)
    n = torch.full((B,), G, device=p.device) if st["n"] is None else st["n"].long()
    pd = p[:, :G].gather(2, d[:, :, None])[:, :, 0].double()
    qd = torch.ones_like(pd) if q is None else q.gather(2, d[:, :, None])[:, :, 0].double()
    stays = ((u[:, :G] * qd < pd) & (j < n[:, None])).long().cumprod(1)
    acc = stays.sum(1)
    rejected = acc < n
    last = acc.clamp(max=G - 1)
    full = p[row, acc].double()
    if q is None:
        hot = torch.arange(V, device=p.device) == d[row, last][:, None]
        r = torch.where(hot & rejected[:, None], 0.0, full)
    else:
        r = torch.where(rejected[:, None], full - q[row, last].double(), full).clamp(min=0)
    r = torch.where(r.sum(1, keepdim=True) > 0, r, full)
    cum = r.cumsum(1)
    final = (cum <= u[:, G:] * cum[:, -1:]).sum(1)
    k = torch.arange(G1, device=p.device)
    drafted = torch.cat([d, torch.zeros_like(d[:, :1])], 1)
    out = torch.where(k < acc[:, None], drafted, torch.full_like(drafted, -1))
    out = torch.where(k == acc[:, None], final[:, None], out)
    return out.int(), acc.int()


def _plain_head(st):
    q, s = st["q"], st["s"].float()
    V, K = q.shape[0], q.shape[1] * 2
    n = torch.stack([q & 15, q >> 4], -1).reshape(V, K)
    g = torch.arange(K, device=q.device) // st["group"]
    if st["z"] is None:
        w = n.float() - 8.0
    else:
        z = torch.stack([st["z"] & 15, st["z"] >> 4], -1).reshape(V, -1)
        w = n.float() - z[:, g].float()
    return (st["x"].float() @ (w * s[:, g]).t()).to(st["out"])


def _plain_reserve(st, lens, add):
    tab, ref, pool, ps = st["tables"], st["ref"], st["pool"], st["page"]
    M = tab.shape[1]
    lens, add = lens.long(), add.long()
    idx = torch.arange(M, device=tab.device)
    lo, hi = lens // ps, (lens + add + ps - 1) // ps
    page = tab.long()
    held = page >= 0
    shared = held & (ref[page.clamp(min=0)] > 1)
    takes = (idx >= lo[:, None]) & (idx < hi[:, None]) & (add > 0)[:, None] & (~held | shared)
    fits = (hi <= M) | (add == 0)
    takes &= fits[:, None]
    ok = fits & (takes.sum(1).cumsum(0) <= (ref == 0).sum())
    takes &= ok[:, None]
    free = torch.sort((ref != 0).int(), stable=True).indices  # free pages first, lowest first
    new = free[(takes.flatten().cumsum(0) - 1).clamp(min=0)].reshape(tab.shape)
    copied = takes & shared
    b, c = (copied & (idx == lo[:, None])).nonzero(as_tuple=True)
    fresh, old = new[b, c], page[b, c]
    slots = torch.arange(ps, device=tab.device)
    keep = (slots < (lens % ps)[b][:, None])[None, :, :, None, None]
    pool[:, fresh] = torch.where(keep, pool[:, old], pool[:, fresh])
    left = page[copied]
    ref.index_add_(0, left, torch.full_like(left, -1).int())
    ref[new[takes]] = 1
    tab.copy_(torch.where(takes, new, page))
    return ok.int()


def _plain_truncate(st, rows, keep):
    tab, ref, ps = st["tables"], st["ref"], st["page"]
    rows, keep = rows.long(), keep.long()
    page = tab[rows].long()
    gone = (torch.arange(tab.shape[1], device=tab.device) >= ((keep + ps - 1) // ps)[:, None]) & (page >= 0)
    left = page[gone]
    ref.index_add_(0, left, torch.full_like(left, -1).int())
    tab[rows] = torch.where(gone, -1, page).int()
    st["lens"][rows] = torch.minimum(st["lens"][rows], keep.int())


def _plain_fork(st):
    tab, ref, lens, ps = st["tables"], st["ref"], st["lens"], st["page"]
    src, dst = st["src"].long(), st["dst"].long()
    old = tab[dst].long()
    held = old[old >= 0]
    ref.index_add_(0, held, torch.full_like(held, -1).int())
    n = (lens[src].long() + ps - 1) // ps
    new = torch.where(torch.arange(tab.shape[1], device=tab.device) < n[:, None], tab[src].long(), -1)
    kept = new[new >= 0]
    ref.index_add_(0, kept, torch.ones_like(kept).int())
    tab[dst] = new.int()
    lens[dst] = lens[src]


def _plain_commit(st):
    tab, pool, ps, base = st["tables"].long(), st["pool"], st["page"], st["base"].long()
    acc, nodes = st["acc"].long(), st["nodes"].long()
    i = torch.arange(nodes.shape[1], device=tab.device)
    b, c = ((i < acc[:, None]) & (nodes != i + 1)).nonzero(as_tuple=True)
    src, dst = base[b] + nodes[b, c], base[b] + 1 + c
    sp, dp = tab[b, src // ps], tab[b, dst // ps]
    pool[:, dp, dst % ps] = pool[:, sp, src % ps]
    new = base + 1 + acc
    st["lens"].copy_(new)
    _plain_truncate(st, torch.arange(tab.shape[0], device=tab.device), new)


def _plain_cache(st):
    kind = st["kind"]
    if kind == "copy":
        st["pool"][:, st["dst"].long()] = st["pool"][:, st["src"].long()]
        return {"pool": st["pool"]}
    if kind == "admit":
        _plain_truncate(st, st["rows"], st["keep"])
        ok = _plain_reserve(st, st["base"], st["add"])
        return {"tables": st["tables"], "ref": st["ref"], "lens": st["lens"], "ok": ok}
    if kind == "fork":
        _plain_fork(st)
        ok = _plain_reserve(st, st["lens"], st["add"])
    else:
        ok = _plain_reserve(st, st["base"], st["add"])
        _plain_commit(st)
    return {"tables": st["tables"], "ref": st["ref"], "lens": st["lens"], "ok": ok, "pool": st["pool"]}


# --------------------------------------------------------------------------
# the framework's calls

def _own_cache(st):
    kind, cache = st["kind"], st["cache"]
    if kind == "copy":
        cache.copy_pages(st["src"], st["dst"])
        return {"pool": st["pool"]}
    bt = st["bt"]
    if kind == "admit":
        cache.truncate(bt, st["keep"], rows=st["rows"])
        ok = cache.reserve(bt, st["add"], lens=st["base"])
        return {"tables": st["tables"], "ref": st["ref"], "lens": st["lens"], "ok": ok}
    if kind == "fork":
        cache.fork(bt, st["src"], st["dst"])
        ok = cache.reserve(bt, st["add"])
    else:
        ok = cache.reserve(bt, st["add"], lens=st["base"])
        cache.commit(bt, st["acc"], nodes=st["nodes"], base=st["base"])
    return {"tables": st["tables"], "ref": st["ref"], "lens": st["lens"], "ok": ok, "pool": st["pool"]}


def run(state):
    op = state["op"]
    if own:
        if op == "verify":
            return state["sampler"].spec_verify_probs(state["target"], state["draft"], state["tokens"],
                                                      state["u"], draft_len=state["n"])
        if op == "head":
            return state["sampler"].lmhead_quant_logits(state["x"], state["q"], state["s"],
                                                        state["group"], zeros=state["z"],
                                                        out_dtype=state["out"])
        return _own_cache(state)
    return {"verify": _plain_verify, "head": _plain_head, "cache": _plain_cache}[op](state)


# --------------------------------------------------------------------------
# what a pass cannot do without

def _mean_accepted(case):
    """Accepted nodes per row: uniform on 0 .. min(N, 6) - 1."""
    return (min(case["N"], 6) - 1) / 2


def work(case):
    op, B = case["op"], case["B"]
    if op == "verify":
        G, V, es = case["G"], case["V"], _BYTES[case["dtype"]]
        rows = 2 if case["rows"] else 1  # the row drawn from, and the draft row it is held against
        return {"bytes": B * (rows * V * es + G * (2 * es + 4) + (G + 1) * 8), "flops": 4.0 * B * V}
    if op == "head":
        V, K, ng = case["V"], case["K"], -(-case["K"] // case["group"])
        b = V * K // 2 + 2 * V * ng + 2 * B * K + B * V * _BYTES[case["out"]]
        if case["zeros"]:
            b += V * ((ng + 1) // 2)
        return {"bytes": b, "flops": 2.0 * B * V * K}
    kind, ps = case["kind"], case["page"]
    slot = 2 * case["layers"] * case["heads"] * case["dim"] * 2  # bytes of a slot over all planes
    if kind == "copy":
        return {"bytes": 2 * B * ps * slot + 8 * B, "flops": 0}
    tables = 8 * B * (case["len"] // ps + 1) + 4 * case["pages"]
    if kind == "admit":
        return {"bytes": tables, "flops": 0}
    if kind == "fork":  # half a page on average
        return {"bytes": tables + (B - min(case["N"], B - 1)) * ps * slot, "flops": 0}
    return {"bytes": tables + int(2 * B * _mean_accepted(case) * slot), "flops": 0}


# --------------------------------------------------------------------------
# the definitions, in 64 bits

def _exact_verify(case, seed):
    st = _prepare_verify(case, seed)
    B, G = case["B"], case["G"]
    out = torch.full((B, G + 1), -1, dtype=torch.int32)
    num = torch.zeros(B, dtype=torch.int32)
    for b in range(B):
        n = G if st["n"] is None else int(st["n"][b])
        k, rest = 0, None
        while k < n:
            d = int(st["tokens"][b, k])
            p = st["target"][b, k].cpu().double()
            q = torch.zeros_like(p)
            if st["draft"] is None:
                q[d] = 1.0
            else:
                q = st["draft"][b, k].cpu().double()
            if not float(st["u"][b, k]) * float(q[d]) < float(p[d]):
                rest = torch.relu(p - q)
                break
            out[b, k] = d
            k += 1
        p = st["target"][b, k].cpu().double()
        rest = p if rest is None or float(rest.sum()) == 0 else rest
        mass = torch.cumsum(rest, 0)
        out[b, k] = int(torch.searchsorted(mass, float(st["u"][b, G]) * float(mass[-1]), right=True))
        num[b] = k
    return out, num


def _exact_head(case, seed):
    """Group by group: scale times (sum n x - zero sum x)."""
    st = _prepare_head(case, seed)
    V, K, grp = case["V"], case["K"], case["group"]
    y = torch.zeros(case["B"], V, dtype=torch.float64, device="cuda")
    for k0 in range(0, K, grp):
        k1, g = min(K, k0 + grp), k0 // grp
        q = st["q"][:, k0 // 2:k1 // 2].double()
        hi = torch.floor(q / 16)
        x = st["x"][:, k0:k1].double()
        dot = x[:, 0::2] @ (q - 16 * hi).t().contiguous() + x[:, 1::2] @ hi.t().contiguous()
        zero = 8.0
        if st["z"] is not None:
            zb = st["z"][:, g // 2].double()
            zh = torch.floor(zb / 16)
            zero = (zh if g % 2 else zb - 16 * zh)[None, :]
        y += st["s"][:, g].double()[None, :] * (dot - zero * x.sum(1, keepdim=True))
    return y


def _exact_cache(case, seed):
    """Page by page and row by row on host copies of the tables."""
    st = _prepare_cache(case, seed)
    pool, ps, kind = st["pool"].double(), case["page"], case["kind"]
    if kind == "copy":
        for s, d in zip(st["src"].tolist(), st["dst"].tolist()):
            pool[:, d] = pool[:, s].clone()
        return {"pool": pool}
    tab, ref, lens = st["tables"].tolist(), st["ref"].tolist(), st["lens"].tolist()

    def drop(b, keep):
        for i in range(-(-keep // ps), len(tab[b])):
            if tab[b][i] >= 0:
                ref[tab[b][i]] -= 1
                tab[b][i] = -1

    if kind == "admit":
        for b in st["rows"].tolist():
            drop(b, 0)
            lens[b] = 0
    if kind == "fork":
        for s, d in zip(st["src"].tolist(), st["dst"].tolist()):
            drop(d, 0)
            for i in range(-(-lens[s] // ps)):
                tab[d][i] = tab[s][i]
                ref[tab[s][i]] += 1
            lens[d] = lens[s]
    base = lens if kind == "fork" else st["base"].tolist()
    before, free, ok = list(ref), [i for i, r in enumerate(ref) if r == 0], []
    used = 0
    for b, add in enumerate(st["add"].tolist()):
        todo = []
        if add > 0:
            todo = [i for i in range(base[b] // ps, -(-(base[b] + add) // ps))
                    if tab[b][i] < 0 or before[tab[b][i]] > 1]
        ok.append(int(used + len(todo) <= len(free)))
        used += len(todo)
        for k, i in enumerate(todo if ok[-1] else []):
            new = free[used - len(todo) + k]
            old = tab[b][i]
            if old >= 0:
                ref[old] -= 1
                if i == base[b] // ps and base[b] % ps:
                    pool[:, new, :base[b] % ps] = pool[:, old, :base[b] % ps]
            ref[new] = 1
            tab[b][i] = new
    if kind == "step":
        nodes, acc = st["nodes"].tolist(), st["acc"].tolist()
        for b in range(case["B"]):
            for i in range(acc[b]):
                s, d = base[b] + nodes[b][i], base[b] + 1 + i
                pool[:, tab[b][d // ps], d % ps] = pool[:, tab[b][s // ps], s % ps].clone()
            lens[b] = base[b] + 1 + acc[b]
            drop(b, lens[b])
    got = {"tables": torch.tensor(tab, dtype=torch.int32), "ref": torch.tensor(ref, dtype=torch.int32),
           "lens": torch.tensor(lens, dtype=torch.int32), "ok": torch.tensor(ok, dtype=torch.int32)}
    return got if kind == "admit" else {**got, "pool": pool}


def exact(case, seed):
    return {"verify": _exact_verify, "cache": _exact_cache, "head": _exact_head}[case["op"]](case, seed)
