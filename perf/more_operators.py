"""What a decoding round needs beside the attention and the tree's experts, as measured cases.

Operators: the whole mixture-of-experts layer for a few tokens; sampling from logits with
temperature, top-k, top-p and min-p; the walk of a verified draft tree along its samples; and the
upkeep of the cache's pages (sequences that end, fork and grow; a pool that is compacted).

`run` computes a case in elementary torch operations, or (own = True) through the library's
entry points. `exact` computes it in 64 bits from the definitions.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"


# ----------------------------------------------------------------------------- cases

def listed():
    return [
        # one user, one token: a layer of a stack (pre-norm, residual); the experts' weights are all
        # the cost
        dict(name="few_1x2048", op="few", dtype="bf16", d=2048, E=128, k=8, f=768, R=1, norm=True,
             slots=False, std=0.02),
        # a small batch, or a short chain of drafted tokens: most tokens bring experts of their own
        dict(name="few_16x2048", op="few", dtype="bf16", d=2048, E=128, k=8, f=768, R=16, norm=True,
             slots=False, std=0.02),
        # wide experts of which a part is held in slots, peaked router: tokens share experts
        dict(name="few_4x2880_slots", op="few", dtype="bf16", d=2880, E=32, k=4, f=2880, R=4,
             norm=False, slots=True, std=0.1),
        # a small fp32 layer of odd sizes (a drafter's): latency counts
        dict(name="few_3x520_fp32", op="few", dtype="fp32", d=520, E=20, k=3, f=264, R=3, norm=False,
             slots=False, std=0.02),
        # one user's next token, the usual settings: latency counts
        dict(name="sample_1x151936", op="sample", dtype="bf16", R=1, V=151936, pad=0, T=0.7, k=50,
             p=0.95, m=0.0, mix=False, masked=0.0),
        # a server's batch, every request with settings of its own (greedy ones, flat ones, grammars
        # that mask most tokens), logits as wide as the padded head
        dict(name="sample_192x50257_mix", op="sample", dtype="fp32", R=192, V=50257, pad=47, T=1.0,
             k=0, p=1.0, m=0.0, mix=True, masked=0.25),
        # one draft tree: every node sampled, the samples followed through the tree
        dict(name="verify_1x65", op="verify", dtype="bf16", B=1, N=65, V=151936, pad=0, T=0.8, k=20,
             p=0.9, m=0.0, mix=False, masked=0.0, P=7),
        # a server's batch of draft trees without top-k, settings for each sequence
        dict(name="verify_16x65", op="verify", dtype="bf16", B=16, N=65, V=151936, pad=0, T=1.0, k=0,
             p=0.95, m=0.02, mix=False, masked=0.0, P=7),
        # a few samples of one prompt begin anew: their pages are given back, they fork the prompt's
        # sequence, everybody gets room for the next block
        dict(name="turnover_4of16", op="turnover", dtype="bf16", Hkv=4, dh=128, page=16,
             layout="nhd", B=16, F=4, ctx=2003, extra=65, spare=64),
        # the same on a busy server
        dict(name="turnover_128of512", op="turnover", dtype="bf16", Hkv=8, dh=64, page=64,
             layout="hnd", B=512, F=128, ctx=3001, extra=65, spare=700),
        # a small pool moved together
        dict(name="compact_1k", op="compact", dtype="bf16", Hkv=4, dh=128, page=16, layout="nhd",
             B=8, ctx=1500, used=0.8, n_pages=1000),
        # a large pool, half of it in use and scattered
        dict(name="compact_16k", op="compact", dtype="bf16", Hkv=4, dh=128, page=64, layout="hnd",
             B=200, ctx=3000, used=0.5, n_pages=16384),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["few", "few", "few", "sample", "sample", "sample", "verify", "turnover",
                     "compact"])
    if op == "few":
        dtype = "fp32" if rng.random() < 0.25 else "bf16"
        R, k = rng.randint(1, 16), rng.randint(1, 8)
        E = max(k, _log(rng, 4, 256))
        d, f = 8 * _log(rng, 16, 600), 8 * _log(rng, 8, 600)
        most = min(7.7e8, 6.0e9 * min(E, R * k) / E) / (12 if dtype == "fp32" else 6)
        while min(E, R * k) * d * f > most:
            d, f = max(128, d // 16 * 8), max(64, f // 16 * 8)
        return dict(op=op, dtype=dtype, d=d, E=E, k=k, f=f, R=R, norm=rng.random() < 0.5,
                    slots=rng.random() < 0.3, std=rng.choice([0.02, 0.1]))
    if op in ("sample", "verify"):
        case = dict(op=op, dtype=rng.choice(["bf16", "bf16", "fp32"]),
                    pad=rng.choice([0, 0, 7, 64]), T=rng.choice([0.0, 0.3, 0.7, 1.0, 1.6]),
                    k=rng.choice([0, 0, 1, 20, 50, 300, 2000]),
                    p=rng.choice([1.0, 0.95, 0.9, 0.5]), m=rng.choice([0.0, 0.0, 0.02, 0.1]),
                    mix=rng.random() < 0.4, masked=rng.choice([0.0, 0.0, 0.3]))
        case["V"] = _log(rng, 500, 260000)
        if op == "sample":
            case["R"] = _log(rng, 1, min(1024, 1e8 / case["V"]))
        else:
            case["N"] = _log(rng, 2, 130)
            case["B"] = _log(rng, 1, max(1, min(64, 1e8 / case["V"] / case["N"])))
            case["P"] = rng.choice([1, 4, 7, 9])
        return case
    Hkv, dh = rng.choice([(4, 128), (8, 64), (2, 64), (1, 80), (2, 96)])
    case = dict(op=op, dtype=rng.choice(["bf16", "bf16", "fp32"]), Hkv=Hkv, dh=dh,
                page=rng.choice([16, 16, 32, 64, 24, 7]), layout=rng.choice(["nhd", "hnd"]))
    token = Hkv * dh * (4 if case["dtype"] == "fp32" else 2)
    if op == "turnover":
        B = _log(rng, 2, 400)
        case.update(B=B, F=max(1, int(B * rng.uniform(0.05, 0.5))), extra=rng.choice([1, 9, 65]),
                    ctx=_log(rng, 1, min(6000, 1.6e9 / (B * token) + 1)))
        case["spare"] = case["F"] * (1 + case["extra"] // case["page"] + 1) + _log(rng, 1, 500)
    else:
        n = _log(rng, 8, min(16000, 1.0e9 / (case["page"] * token)))
        used = rng.uniform(0.1, 0.95)
        case.update(n_pages=n, used=used, B=max(1, _log(rng, 1, 200)))
        case["ctx"] = max(1, int(n * used * case["page"] / case["B"]))
    return case


# ----------------------------------------------------------------------------- inputs

def _dt(case):
    return torch.float32 if case["dtype"] == "fp32" else torch.bfloat16


def _randn(gen, dt, *shape, std=1.0):
    t = torch.empty(*shape, dtype=dt, device=DEV)
    for part in t.view(-1).split(1 << 29):
        part.copy_(torch.randn(part.shape, generator=gen, device=DEV) * std)
    return t


def _tree(r, N):
    """parent [N] (root -1) of a random draft tree, at most 8 deep; wide near the root, as
    drafted trees are."""
    parent = np.full(N, -1, np.int32)
    depth = np.zeros(N, np.int32)
    for i in range(1, N):
        p = int(i * r.random() ** 1.5)
        while depth[p] >= 8:
            p = int(parent[p])
        parent[i], depth[i] = p, depth[p] + 1
    return parent


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    r = np.random.default_rng([seed, 7])
    st = {"case": case}
    {"few": _prepare_few, "sample": _prepare_sample, "verify": _prepare_verify,
     "turnover": _prepare_turnover, "compact": _prepare_compact}[case["op"]](st, gen, r)
    return st


def _prepare_few(st, gen, r):
    case = st["case"]
    d, E, k, f, R, dt = case["d"], case["E"], case["k"], case["f"], case["R"], _dt(case)
    st["x"] = _randn(gen, dt, R, d)
    st["wr"] = _randn(gen, dt, E, d, std=case["std"])
    S = E + 2 if case["slots"] else E
    st["wg"] = _randn(gen, dt, S, f, d, std=0.02)
    st["wu"] = _randn(gen, dt, S, f, d, std=0.02)
    st["wd"] = _randn(gen, dt, S, d, f, std=0.02)
    st["slot"] = None
    if case["slots"]:  # a pool of expert slots, filled in the order the experts came
        st["slot"] = torch.from_numpy(r.permutation(S)[:E].astype(np.int32)).to(DEV)
    st["y"] = torch.empty_like(st["x"])
    if own:
        from expert_select_gb300 import moetree as M
        st["L"] = M.layer_desc(d, E, k, f, dt, slots=S)
        st["ws"] = M.few_workspace(st["L"], R, device=DEV)
        st["opts"] = M.run_opts(residual=case["norm"], norm_input=case["norm"])


def _logits(st, gen, r, R):
    """Logits as a model gives them: most tokens far below a few likely ones. `masked`: the share of
    rows in which a grammar leaves a few tokens."""
    case = st["case"]
    V = case["V"]
    x = torch.randn(R, V + case["pad"], generator=gen, device=DEV) * 2.5
    top = torch.from_numpy(r.integers(0, V, (R, 24))).to(DEV)
    up = 5 + 9 * torch.rand(R, 24, generator=gen, device=DEV)
    x.scatter_add_(1, top, up)
    if case["masked"]:
        rows = torch.from_numpy(r.random(R) < case["masked"]).to(DEV)
        lost = torch.rand(R, V + case["pad"], generator=gen, device=DEV) < 0.98
        lost[:, 0] = False
        x = x.masked_fill(lost & rows[:, None], -math.inf)
    st["wide"] = x.to(_dt(case))
    st["logits"] = st["wide"][:, :V]


def _settings(st, r, n):
    """Temperature, top-k, top-p and min-p of n requests (None: not asked for)."""
    case = st["case"]
    T, k, p, m = ([case[c]] * n for c in ("T", "k", "p", "m"))
    if case["mix"]:
        T = [float(v) for v in r.choice([0.0, 0.5, 0.8, 1.0, 1.3], n)]
        k = [int(v) for v in r.choice([0, 0, 1, 10, 40, 1000], n)]
        p = [float(v) for v in r.choice([1.0, 1.0, 0.95, 0.8], n)]
        m = [float(v) for v in r.choice([0.0, 0.0, 0.05], n)]
    f32 = dict(dtype=torch.float32, device=DEV)
    st["T"] = torch.tensor(T, **f32)
    st["k"] = torch.tensor(k, dtype=torch.int32, device=DEV) if any(k) else None
    st["p"] = torch.tensor(p, **f32) if min(p) < 1 else None
    st["m"] = torch.tensor(m, **f32) if any(m) else None


def _prepare_sample(st, gen, r):
    case = st["case"]
    R = case["R"]
    _logits(st, gen, r, R)
    _settings(st, r, R)
    st["group"] = 1
    st["u"] = torch.rand(R, generator=gen, device=DEV)
    st["token"] = torch.empty(R, dtype=torch.int32, device=DEV)
    st["logprob"] = torch.empty(R, dtype=torch.float32, device=DEV)


def _prepare_verify(st, gen, r):
    case = st["case"]
    B, N, P = case["B"], case["N"], case["P"]
    R = B * N
    _logits(st, gen, r, R)
    _settings(st, r, B)
    st["group"] = N
    st["u"] = torch.rand(R, generator=gen, device=DEV)
    parent = np.stack([_tree(r, N) for _ in range(B)])
    # a drafter proposes what is likely: a node's token is one of its parent's likeliest
    row = torch.from_numpy(np.maximum(parent, 0) + N * np.arange(B)[:, None]).to(DEV).reshape(-1)
    best = st["logits"].float().topk(min(4, case["V"]), -1).indices
    pick = torch.from_numpy(r.integers(0, best.shape[1], R)).to(DEV)
    st["draft"] = best[row].gather(1, pick[:, None])[:, 0].int()
    st["parent_h"] = parent
    st["parent"] = torch.from_numpy(parent.reshape(-1)).to(DEV)
    anc = np.zeros((B, N, N), bool)  # ancestors and self, the root left out
    for i in range(1, N):
        anc[np.arange(B), i] = anc[np.arange(B), parent[:, i]]
        anc[:, i, i] = True
    st["anc"] = torch.from_numpy(anc).to(DEV)
    i32 = dict(dtype=torch.int32, device=DEV)
    st["token"] = torch.empty(R, **i32)
    st["logprob"] = torch.empty(R, dtype=torch.float32, device=DEV)
    st["path"], st["next"] = torch.empty(B, P, **i32), torch.empty(B, P, **i32)
    st["acc"] = torch.empty(B, **i32)


def _pools(st, gen, n_pages):
    case = st["case"]
    p, h, d, dt = case["page"], case["Hkv"], case["dh"], _dt(case)
    for name in ("kp", "vp"):
        if case["layout"] == "nhd":
            st[name] = _randn(gen, dt, n_pages, p, h, d)
        else:
            st[name] = _randn(gen, dt, n_pages, h, p, d).permute(0, 2, 1, 3)


def _book(st, table, held, lens, ref):
    """What the pages' upkeep works on: page table, pages held by each sequence, tokens of each,
    and how many table entries hold each page."""
    case = st["case"]
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)  # noqa: E731
    st["table"], st["held"], st["lens"], st["ref"] = up(table), up(held), up(lens), up(ref)
    if own:
        from expert_select_gb300 import moetree as M
        st["book"] = M.page_book(st["table"], st["held"], st["lens"], st["ref"], case["page"])
        st["C"] = M.cache_desc(st["kp"], case["Hkv"], table.shape[1])
        st["ws"] = M.pages_workspace(st["book"])


def _prepare_turnover(st, gen, r):
    case = st["case"]
    B, F, ctx, page, extra = (case[c] for c in ("B", "F", "ctx", "page", "extra"))
    shape = np.random.default_rng([B, F, ctx, page])  # lengths belong to the case
    lens = shape.integers(max(1, ctx // 4), ctx + 1, B)
    dst = np.sort(shape.choice(B, F, replace=False))
    others = np.setdiff1d(np.arange(B), dst)
    src = shape.choice(others, F) if len(others) else np.zeros(0, int)
    if len(src) == 0:
        dst = dst[:0]
    lens[dst] = lens[src]
    held = -(-(lens + extra) // page)
    n_pages = int(held.sum()) + case["spare"]
    order = r.permutation(n_pages)
    table = np.full((B, int(held.max()) + 1), -1)
    ref = np.zeros(n_pages)
    at = 0
    for b, c in enumerate(held):
        table[b, :c] = order[at:at + c]
        ref[order[at:at + c]] = 1
        at += c
    _pools(st, gen, n_pages)
    st["src_h"], st["dst_h"] = src, dst
    st["src"] = torch.from_numpy(src.astype(np.int32)).to(DEV)
    st["dst"] = torch.from_numpy(dst.astype(np.int32)).to(DEV)
    st["moves"] = torch.full((len(dst), 3), -1, dtype=torch.int32, device=DEV)
    _book(st, table, held, lens, ref)


def _prepare_compact(st, gen, r):
    case = st["case"]
    B, ctx, page, n_pages = (case[c] for c in ("B", "ctx", "page", "n_pages"))
    shape = np.random.default_rng([B, ctx, page, n_pages])
    lens = shape.integers(max(1, ctx // 2), ctx + 1, B)
    held = -(-lens // page)
    while held.sum() > n_pages * case["used"]:
        lens = lens * 9 // 10
        held = -(-lens // page)
    order = r.permutation(n_pages)
    table = np.full((B, int(held.max()) + 1), -1)
    ref = np.zeros(n_pages)
    at = 0
    for b, c in enumerate(held):
        if b % 4 == 3:  # a quarter of the sequences share the first half of another's pages
            half = min(c, held[b - 1]) // 2
            table[b, :half] = table[b - 1, :half]
            table[b, half:c] = order[at:at + c - half]
            at += c - half
        else:
            table[b, :c] = order[at:at + c]
            at += c
        np.add.at(ref, table[b, :c], 1)
    _pools(st, gen, n_pages)
    _book(st, table, held, lens, ref)
    i32 = dict(dtype=torch.int32, device=DEV)
    st["table_out"], st["ref_out"] = torch.zeros_like(st["table"]), torch.zeros_like(st["ref"])
    st["moves"] = torch.full((n_pages // 2, 3), -1, **i32)
    st["counts"] = torch.zeros(2, **i32)


# ----------------------------------------------------------------------------- plain forms

def _plain_few(st):
    case = st["case"]
    x = st["x"]
    if case["norm"]:
        t = x.double()
        x = (t / torch.sqrt((t * t).mean(-1, keepdim=True) + 1e-6)).to(x.dtype)
    xf = x.float()
    logits = xf @ st["wr"].float().T
    top, idx = torch.sort(logits, dim=-1, descending=True, stable=True)
    top, idx = top[:, :case["k"]], idx[:, :case["k"]]
    e = torch.exp(top - top[:, :1])
    gates = e / e.sum(-1, keepdim=True)
    slot = idx if st["slot"] is None else st["slot"].long()[idx]
    g = (st["wg"][slot].float() @ xf[:, None, :, None])[..., 0]      # [R, k, f]
    u = (st["wu"][slot].float() @ xf[:, None, :, None])[..., 0]
    h = g / (1 + torch.exp(-g)) * u
    y = ((st["wd"][slot].float() @ h[..., None])[..., 0] * gates[..., None]).sum(1)
    if case["norm"]:
        y = y + st["x"].float()
    st["y"].copy_(y)
    return st["y"]


def _plain_sample(st):
    x = st["logits"].double()
    R, V = x.shape
    row = torch.arange(R, device=DEV) // st["group"]
    T = st["T"].double()[row, None]
    x = torch.where(torch.isnan(x), torch.full_like(x, -math.inf), x)
    val, idx = torch.sort(x, dim=-1, descending=True, stable=True)
    d = val - val[:, :1]
    pos = torch.arange(V, device=DEV)[None]
    s = torch.where(T > 0, d / T, torch.where(pos == 0, torch.zeros_like(d), -math.inf))
    w = torch.exp(s)
    if st["k"] is not None:
        k = st["k"].long()[row, None]
        w = torch.where((pos < k) | (k <= 0), w, torch.zeros_like(w))
    if st["p"] is not None:
        p = st["p"].double()[row, None]
        before = torch.cumsum(w, -1) - w
        w = torch.where((before < p * w.sum(-1, keepdim=True)) | (p >= 1), w, torch.zeros_like(w))
    if st["m"] is not None:
        w = torch.where(w >= st["m"].double()[row, None], w, torch.zeros_like(w))
    w = torch.zeros_like(w).scatter_(1, idx, w)                      # in the order of the tokens
    c = torch.cumsum(w, -1)
    t = (c <= st["u"].double()[:, None] * c[:, -1:]).sum(-1, keepdim=True)
    st["token"].copy_(t[:, 0])
    st["logprob"].copy_(torch.log(w.gather(1, t) / c[:, -1:])[:, 0])
    return st["token"], st["logprob"]


def _plain_verify(st):
    case = st["case"]
    B, N, P = case["B"], case["N"], case["P"]
    token, logprob = _plain_sample(st)
    token, draft, parent = (t.view(B, N) for t in (token, st["draft"], st["parent"]))
    match = draft == token.gather(1, parent.clamp_min(0).long())
    # of siblings with the same token the first counts
    same = (parent[:, :, None] == parent[:, None, :]) & (draft[:, :, None] == draft[:, None, :])
    match &= ~torch.tril(same, -1).any(-1)
    kept = ~(st["anc"] & ~match[:, None, :]).any(-1)                 # every node on its way matches
    at = torch.cumsum(kept, -1) - 1
    kept &= at < P
    node = torch.arange(N, device=DEV).expand(B, N).int()
    slot = torch.where(kept, at, torch.full_like(at, P))
    none = torch.full((B, P + 1), -1, dtype=torch.int32, device=DEV)
    st["path"].copy_(none.scatter(1, slot, node)[:, :P])
    st["next"].copy_(none.scatter(1, slot, token)[:, :P])
    st["acc"].copy_(kept.sum(-1))
    return token, logprob, st["path"], st["acc"], st["next"]


def _copy_tokens(st, src, dst, tokens):
    """The first `tokens` slots of pages src go to pages dst."""
    for pool in (st["kp"], st["vp"]):
        few = torch.arange(pool.shape[1], device=DEV)[None] < tokens[:, None]
        pool[dst] = torch.where(few[..., None, None], pool[src], pool[dst])


def _plain_turnover(st):
    page, extra = st["case"]["page"], st["case"]["extra"]
    table, held, lens, ref = st["table"], st["held"], st["lens"], st["ref"]
    src, dst = st["src"].long(), st["dst"].long()
    col = torch.arange(table.shape[1], device=DEV)[None]
    n_pages = ref.numel()

    def count(t, held, by):
        ref.index_add_(0, t[col < held[:, None]].long(),
                       torch.full_like(t[col < held[:, None]], by))

    count(table[dst], held[dst], -1)                                 # the ended ones give back
    held[dst] = 0
    lens[dst] = 0
    full, tail = lens[src] // page, lens[src] % page                 # forks share full pages
    count(table[src], full, 1)
    need = (tail > 0).int()
    free = torch.nonzero(ref == 0)[:, 0].int()
    new = free[(torch.cumsum(need, 0) - 1).clamp_min(0)]
    old = table[src].gather(1, full[:, None].long())[:, 0]
    table[dst] = torch.where(col < full[:, None], table[src], table[dst])
    at = col == full[:, None]
    table[dst] = torch.where(at & (need > 0)[:, None], new[:, None], table[dst])
    ref.index_add_(0, new[need > 0].long(), need[need > 0])
    held[dst] = full + need
    lens[dst] = lens[src]
    moves = torch.stack([old, new, tail], 1)
    st["moves"].copy_(torch.where(need[:, None] > 0, moves, torch.tensor([-1, -1, 0], device=DEV)))
    want = (lens + extra + page - 1) // page                         # room for the next block
    grow = (want - held).clamp_min(0)
    first = torch.cumsum(grow, 0) - grow
    free = torch.nonzero(ref == 0)[:, 0].int()
    here = (col >= held[:, None]) & (col < (held + grow)[:, None])
    nth = (first[:, None] + col - held[:, None]).clamp(0, free.numel() - 1)
    table.copy_(torch.where(here, free[nth], table))
    ref[free[:int(grow.sum())].long()] = 1
    held += grow
    some = need > 0
    _copy_tokens(st, old[some].long(), new[some].long(), tail[some])
    return table, held, lens, ref, st["moves"], st["kp"], st["vp"]


def _plain_compact(st):
    page, ref = st["case"]["page"], st["ref"]
    n = ref.numel()
    used = ref > 0
    n_used = used.sum()
    at = torch.arange(n, device=DEV)
    high = torch.nonzero(used & (at >= n_used))[:, 0]
    hole = torch.nonzero(~used & (at < n_used))[:, 0]
    to = at.int()
    to[high] = hole.int()
    col = torch.arange(st["table"].shape[1], device=DEV)[None]
    mine = col < st["held"][:, None]
    st["table_out"].copy_(torch.where(mine, to[st["table"].clamp_min(0).long()], st["table"]))
    st["ref_out"].copy_(ref)
    st["ref_out"][hole] = ref[high]
    st["ref_out"][high] = 0
    m = high.numel()
    st["moves"][:m] = torch.stack([high, hole, torch.full_like(high, page)], 1).int()
    st["counts"].copy_(torch.stack([torch.tensor(m, device=DEV), n_used]))
    _copy_tokens(st, high, hole, torch.full_like(high, page))
    return st["table_out"], st["ref_out"], st["moves"], st["counts"], st["kp"], st["vp"]


# ----------------------------------------------------------------------------- one pass

def run(st):
    case = st["case"]
    op = case["op"]
    if not own:
        return {"few": _plain_few, "sample": _plain_sample, "verify": _plain_verify,
                "turnover": _plain_turnover, "compact": _plain_compact}[op](st)
    from expert_select_gb300 import moetree as M
    if op == "few":
        M.moe_few_forward(st["L"], st["x"], st["wr"], st["wg"], st["wu"], st["wd"], st["slot"],
                          st["y"], st["ws"], opts=st["opts"])
        return st["y"]
    if op in ("sample", "verify"):
        M.moe_sample(st["logits"], st["u"], st["token"], temperature=st["T"], top_k=st["k"],
                     top_p=st["p"], min_p=st["m"], param_rows=st["group"], logprob=st["logprob"])
        if op == "sample":
            return st["token"], st["logprob"]
        B, N = case["B"], case["N"]
        M.moe_tree_accept(st["draft"], st["parent"], st["token"], B, N, st["path"], st["acc"],
                          st["next"])
        return st["token"].view(B, N), st["logprob"], st["path"], st["acc"], st["next"]
    if op == "turnover":
        M.moe_kv_free(st["book"], st["dst"], st["ws"])
        M.moe_kv_fork(st["book"], st["src"], st["dst"], st["moves"], st["ws"])
        M.moe_kv_reserve(st["book"], case["extra"], st["ws"])
        M.moe_kv_copy_pages(st["C"], st["kp"], st["vp"], st["moves"], ws=st["ws"])
        return (st["table"], st["held"], st["lens"], st["ref"], st["moves"], st["kp"], st["vp"])
    M.moe_kv_compact(st["book"], st["table_out"], st["ref_out"], st["moves"], st["counts"],
                     st["ws"])
    M.moe_kv_copy_pages(st["C"], st["kp"], st["vp"], st["moves"], count=st["counts"], ws=st["ws"])
    return st["table_out"], st["ref_out"], st["moves"], st["counts"], st["kp"], st["vp"]


# ----------------------------------------------------------------------------- floors

def work(case):
    """Bytes and operations of a pass."""
    e = 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "few":
        d, E, k, f, R = (case[c] for c in ("d", "E", "k", "f", "R"))
        # R tokens of k experts each, as many different ones as chance gives
        experts = E * (1 - (1 - k / E) ** R)
        return {"bytes": int((experts * 3 * f * d + E * d + 2 * R * d) * e),
                "flops": int(2 * R * d * (E + 3 * k * f))}
    if case["op"] in ("sample", "verify"):
        R = case["R"] if case["op"] == "sample" else case["B"] * case["N"]
        return {"bytes": R * (case["V"] * e + 12), "flops": 4 * R * case["V"]}
    token = case["Hkv"] * case["dh"] * e
    if case["op"] == "turnover":
        B, F, page = case["B"], case["F"], case["page"]
        cols = case["ctx"] * 5 // 8 // page
        pages = B * (cols + case["extra"] // page + 1) + case["spare"]
        return {"bytes": int(4 * F * page / 2 * token + 4 * pages + 16 * F * cols + 16 * B),
                "flops": pages}
    st = case["n_pages"]
    used = min(case["used"], case["B"] * case["ctx"] * 0.66 / case["page"] / st)
    moved = st * used * (1 - used)
    return {"bytes": int(4 * moved * case["page"] * token + 12 * moved + 8 * st * (1 + used)),
            "flops": st}


# ----------------------------------------------------------------------------- 64 bits

def _exact_few(st):
    case = st["case"]
    k = case["k"]
    x = st["x"].double()
    inp = x
    if case["norm"]:
        ms = torch.einsum("rd,rd->r", x, x) / case["d"]
        inp = (x * torch.rsqrt(ms + 1e-6)[:, None]).to(st["x"].dtype).double()
    score = torch.einsum("rd,ed->re", inp, st["wr"].double()).cpu().numpy()
    y = x.clone() if case["norm"] else torch.zeros_like(x)
    slot = None if st["slot"] is None else st["slot"].cpu().numpy()
    for r in range(case["R"]):
        best = sorted(range(case["E"]), key=lambda e: (-score[r, e], e))[:k]
        z = np.logaddexp.reduce(score[r, best])
        for e in best:
            s = e if slot is None else int(slot[e])
            a, b = st["wg"][s].double().mv(inp[r]), st["wu"][s].double().mv(inp[r])
            y[r] += math.exp(score[r, e] - z) * st["wd"][s].double().mv(a * torch.sigmoid(a) * b)
    return y


def _exact_sample(st):
    R, V = st["logits"].shape
    none = lambda t, v: [v] * R if t is None else t.cpu().numpy().astype(np.float64)  # noqa: E731
    T, K, Pp, Mp = none(st["T"], 1.0), none(st["k"], 0), none(st["p"], 1.0), none(st["m"], 0.0)
    us = st["u"].cpu().numpy().astype(np.float64)
    tokens, logs = [], []
    for r in range(R):
        i = r // st["group"]
        x = st["logits"][r].double()
        if T[i] <= 0:
            best = x.max()
            tokens.append(int((x == best).nonzero()[0]))
            logs.append(0.0)
            continue
        z = (x - x.max()) / T[i]
        order = torch.argsort(-z, stable=True)
        if K[i] > 0:
            order = order[:int(K[i])]
        share = torch.softmax(z[order], 0)
        if Pp[i] < 1:
            ahead = torch.cumsum(share, 0).roll(1)
            ahead[0] = 0
            order = order[:max(1, int((ahead < Pp[i]).sum()))]
        if Mp[i] > 0:
            order = order[z[order] >= math.log(Mp[i])]
        ids = order.sort().values
        share = torch.softmax(z[ids], 0)
        cdf = torch.cumsum(share, 0)
        n = torch.searchsorted(cdf, cdf[-1] * float(us[r]), right=True)
        n = min(int(n), ids.numel() - 1)
        tokens.append(int(ids[n]))
        logs.append(float(torch.log_softmax(z[ids], 0)[n]))
    return (torch.tensor(tokens, dtype=torch.int32, device=DEV),
            torch.tensor(logs, dtype=torch.float64, device=DEV))


def _exact_verify(st):
    case = st["case"]
    B, N, P = case["B"], case["N"], case["P"]
    token, logs = _exact_sample(st)
    token = token.view(B, N)
    got, draft = token.cpu().numpy(), st["draft"].view(B, N).cpu().numpy()
    path = np.full((B, P), -1, np.int32)
    nxt = np.full((B, P), -1, np.int32)
    acc = np.zeros(B, np.int32)
    for b in range(B):
        node = 0
        while node >= 0 and acc[b] < P:
            path[b, acc[b]], nxt[b, acc[b]] = node, got[b, node]
            acc[b] += 1
            node = next((c for c in range(node + 1, N) if st["parent_h"][b, c] == node and
                         draft[b, c] == got[b, node]), -1)
    up = lambda a: torch.from_numpy(a).to(DEV)  # noqa: E731
    return token, logs, up(path), up(acc), up(nxt)


def _exact_turnover(st):
    page, extra = st["case"]["page"], st["case"]["extra"]
    table, held, lens, ref = (st[n].cpu().numpy().copy() for n in ("table", "held", "lens", "ref"))
    kp, vp = st["kp"].clone(), st["vp"].clone()
    for b in st["dst_h"]:
        for j in range(held[b]):
            ref[table[b, j]] -= 1
        held[b] = lens[b] = 0
    moves = st["moves"].cpu().numpy().copy()
    for a, b in zip(st["src_h"], st["dst_h"]):
        for j in range(lens[a] // page):
            ref[table[a, j]] += 1
    for i, (a, b) in enumerate(zip(st["src_h"], st["dst_h"])):
        c, t = lens[a] // page, lens[a] % page
        table[b, :c] = table[a, :c]
        moves[i] = -1, -1, 0
        if t:
            new = int(np.flatnonzero(ref == 0)[0])
            ref[new] = 1
            table[b, c] = new
            old = int(table[a, c])
            kp[new, :t], vp[new, :t] = kp[old, :t], vp[old, :t]
            moves[i] = old, new, t
        held[b], lens[b] = c + (t > 0), lens[a]
    free = iter(np.flatnonzero(ref == 0))
    for b in range(len(lens)):
        while held[b] * page < lens[b] + extra:
            p = int(next(free))
            table[b, held[b]] = p
            ref[p] = 1
            held[b] += 1
    up = lambda a: torch.from_numpy(a).to(DEV)  # noqa: E731
    return up(table), up(held), up(lens), up(ref), up(moves), kp, vp


def _exact_compact(st):
    table, held, ref = (st[n].cpu().numpy().copy() for n in ("table", "held", "ref"))
    kp, vp = st["kp"].clone(), st["vp"].clone()
    moves = st["moves"].cpu().numpy().copy()
    n_used = int((ref > 0).sum())
    lo, m = 0, 0
    to = {}
    for p in range(n_used, len(ref)):
        if ref[p] > 0:
            while ref[lo] > 0:
                lo += 1
            to[p] = lo
            moves[m] = p, lo, st["case"]["page"]
            m += 1
            lo += 1
    for p, q in to.items():
        ref[q], ref[p] = ref[p], 0
        kp[q], vp[q] = kp[p], vp[p]
    for b in range(len(held)):
        table[b, :held[b]] = [to.get(int(p), int(p)) for p in table[b, :held[b]]]
    up = lambda a: torch.from_numpy(a).to(DEV)  # noqa: E731
    return (up(table), up(ref), up(moves), torch.tensor([m, n_used], dtype=torch.int32, device=DEV),
            kp, vp)


def exact(case, seed):
    """The definitions in 64 bits, one token, row or sequence after the other."""
    st = prepare(case, seed)
    return {"few": _exact_few, "sample": _exact_sample, "verify": _exact_verify,
            "turnover": _exact_turnover, "compact": _exact_compact}[case["op"]](st)
