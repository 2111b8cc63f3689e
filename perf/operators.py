"""The attention half of a decoder block run over verification blocks, as measured cases.

Operators: attention of new tokens over a paged key/value cache (draft trees, prompt chunks,
single tokens), the same with a sliding window and first tokens that stay visible, the write of
new keys and values into the cache's pages (with query/key norms and rotary positions), the move
of a tree's accepted path to the front of its block, and the norms before and after a block
fused with its gate and residual scale.

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
        # one user far into a long document, one token at a time: the whole cost is the cache
        dict(name="decode_1x131k", op="attention", kind="decode", dtype="bf16", H=32, Hkv=4,
             dh=128, page=64, layout="nhd", B=1, N=1, ctx=130941, ragged=False),
        # one user's draft tree of 65 nodes verified over an ordinary context: latency counts
        dict(name="tree65_1x4k", op="attention", kind="tree", dtype="bf16", H=32, Hkv=4, dh=128,
             page=16, layout="hnd", B=1, N=65, ctx=4003, ragged=False),
        # a server's batch of draft trees, every context of its own length
        dict(name="tree65_64x4k", op="attention", kind="tree", dtype="bf16", H=32, Hkv=4, dh=128,
             page=16, layout="nhd", B=64, N=65, ctx=8200, ragged=True),
        # chunked prompts: two users' next 4k tokens behind what is cached already
        dict(name="chunk4k_2x28k", op="attention", kind="chunk", dtype="bf16", H=32, Hkv=4,
             dh=128, page=64, layout="nhd", B=2, N=4096, ctx=28001, ragged=False),
        # a batch of single tokens in a layer with a 128-token window, four first tokens that
        # stay visible and a learned sink logit for each head
        dict(name="win128_decode_128x16k", op="window", kind="decode", dtype="bf16", H=64, Hkv=8,
             dh=64, page=32, layout="nhd", B=128, N=1, ctx=16300, ragged=True, window=128,
             sinks=4, logit=True),
        # fp32 trees, pages of an odd size that end inside every tile, a window that is shorter
        # than the context
        dict(name="win200_fp32_tree33_5x1k", op="window", kind="tree", dtype="fp32", H=16, Hkv=2,
             dh=64, page=7, layout="hnd", B=5, N=33, ctx=1021, ragged=True, window=200, sinks=3,
             logit=False),
        # a batch of single tokens written to the cache: latency counts
        dict(name="append_64x1", op="append", dtype="bf16", H=32, Hkv=4, dh=128, page=16,
             layout="nhd", B=64, N=1, ctx=2001, ragged=True, kind="decode", norm=True, rot=128),
        # two prompt chunks written to the cache, far positions
        dict(name="append_chunk_2x4k", op="append", dtype="bf16", H=64, Hkv=8, dh=64, page=64,
             layout="hnd", B=2, N=4096, ctx=60001, ragged=True, kind="chunk", norm=False, rot=64),
        # one tree's accepted path moved to the front of its block
        dict(name="commit_1x5", op="commit", dtype="bf16", H=32, Hkv=4, dh=128, page=16,
             layout="nhd", B=1, N=65, ctx=3001, ragged=False, kind="tree", P=5),
        # a server's batch of accepted paths
        dict(name="commit_256x6", op="commit", dtype="bf16", H=64, Hkv=8, dh=64, page=32,
             layout="hnd", B=256, N=65, ctx=1500, ragged=True, kind="tree", P=6),
        # one verification block of 65 rows between attention and experts
        dict(name="norm_65x2048", op="norm", dtype="bf16", R=65, d=2048, post=True, gate=0,
             scale=1.0),
        # a prompt chunk's rows, with a gate row for each sequence
        dict(name="norm_8192x2880", op="norm", dtype="bf16", R=8192, d=2880, post=True, gate=4096,
             scale=0.5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "window", "window", "append",
                     "commit", "norm"])
    dtype = "fp32" if rng.random() < 0.2 else "bf16"
    if op == "norm":
        d = 8 * _log(rng, 32, 768)
        R = _log(rng, 1, 12000)
        return dict(op="norm", dtype=dtype, R=R, d=d, post=rng.random() < 0.6,
                    gate=rng.choice([0, 0, R, max(1, R // 3)]), scale=rng.choice([1.0, 0.5, 0.22]))
    H, Hkv, dh = rng.choice([(32, 4, 128), (64, 8, 64), (8, 8, 128), (16, 2, 64), (40, 8, 128),
                             (28, 4, 128), (16, 1, 80), (6, 2, 96)])
    case = dict(op=op, dtype=dtype, H=H, Hkv=Hkv, dh=dh,
                page=rng.choice([16, 16, 32, 64, 128, 24, 20, 7]),
                layout=rng.choice(["nhd", "hnd"]), ragged=rng.random() < 0.6)
    kind = "tree" if op == "commit" else rng.choice(["decode", "tree", "chunk"])
    small = dtype == "fp32"
    if kind == "decode":
        B, N = _log(rng, 1, 128), 1
        ctx = _log(rng, 1, min(131000, (4000000 if not small else 200000) // (B * Hkv)))
    elif kind == "tree":
        B, N = _log(rng, 1, 64 if not small else 6), _log(rng, 2, 200)
        most = 8000 * 64 * 65 if not small else 2000 * 130
        ctx = _log(rng, 1, min(40000, max(2, most // (B * max(N, 65)) + 60)))
    else:
        B, N = rng.choice([1, 1, 2]), _log(rng, 16, 4000 if not small else 300)
        ctx = _log(rng, 1, 28000 if not small else 2000)
        if N * (ctx + N) * B * H * dh > 4096 * 30000 * 2 * 32 * 128:
            B = 1
    case.update(kind=kind, B=B, N=N, ctx=ctx)
    if op == "window":
        case.update(window=_log(rng, 1, 4096), sinks=rng.choice([0, 0, 1, 4, 130]),
                    logit=rng.random() < 0.5)
    if op == "append":
        case.update(norm=rng.random() < 0.5, rot=rng.choice([dh, dh, dh // 2]))
    if op == "commit":
        case["N"] = max(12, case["N"])
        case["P"] = rng.choice([1, 2, 4, 5, 6])
    return case


# ----------------------------------------------------------------------------- inputs

def _dt(case):
    return torch.float32 if case["dtype"] == "fp32" else torch.bfloat16


def _lens(case):
    """Committed tokens and new tokens of every sequence (host lists, as a scheduler has them).
    They belong to the case: output sizes follow them."""
    B, N, ctx = case["B"], case["N"], case["ctx"]
    r = np.random.default_rng([B, N, ctx])
    lens = [ctx] * B
    ns = [N] * B
    if case["ragged"]:
        lens = [int(v) for v in r.integers(max(1, ctx // 40), ctx + 1, B)]
        if case["kind"] == "chunk":
            ns = [int(v) for v in r.integers(max(1, N // 2), N + 1, B)]
    return lens, ns


def _tree(r, N):
    """parent [N] (root -1) and depth [N] of a random draft tree, at most 8 deep; wide near the
    root, as drafted trees are."""
    parent = np.full(N, -1, np.int32)
    depth = np.zeros(N, np.int32)
    for i in range(1, N):
        p = int(i * r.random() ** 1.5)
        while depth[p] >= 8:
            p = int(parent[p])
        parent[i], depth[i] = p, depth[p] + 1
    return parent, depth


def _randn(gen, dt, *shape):
    return torch.randn(*shape, generator=gen, device=DEV, dtype=torch.float32).to(dt)


def _pool(case, gen, n_pages):
    """A page pool [n_pages, page, Hkv, dh] (a view of one, for the head-major layout)."""
    p, h, d = case["page"], case["Hkv"], case["dh"]
    if case["layout"] == "nhd":
        return _randn(gen, _dt(case), n_pages, p, h, d)
    return _randn(gen, _dt(case), n_pages, h, p, d).permute(0, 2, 1, 3)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    r = np.random.default_rng([seed, 5])
    st = {"case": case}
    dt = _dt(case)
    if case["op"] == "norm":
        R, d = case["R"], case["d"]
        st["x"] = _randn(gen, dt, R, d) * 3
        st["branch"] = _randn(gen, dt, R, d)
        st["w_post"] = (1 + 0.2 * _randn(gen, torch.float32, d)).to(dt) if case["post"] else None
        st["w_pre"] = (1 + 0.2 * _randn(gen, torch.float32, d)).to(dt)
        g = case["gate"]
        st["gate"] = _randn(gen, dt, -(-R // g), d) if g else None
        st["h"], st["hn"] = torch.empty_like(st["x"]), torch.empty_like(st["x"])
        if own:
            from expert_select_gb300 import moetree as M
            st["L"] = M.layer_desc(d, 8, 1, 64, dt)
        return st

    B, N, H, Hkv, dh, page = (case[k] for k in ("B", "N", "H", "Hkv", "dh", "page"))
    lens, ns = _lens(case)
    rows = [0]
    for n in ns:
        rows.append(rows[-1] + n)
    R = rows[-1]
    need = [-(-(l + n) // page) for l, n in zip(lens, ns)]
    n_pages = sum(need) + 3
    max_pages = max(need) + 1
    order = torch.from_numpy(r.permutation(n_pages)).to(torch.int32)
    table = torch.zeros(B, max_pages, dtype=torch.int32)
    at = 0
    for b, c in enumerate(need):
        table[b, :c] = order[at:at + c]
        at += c
    st.update(lens=lens, ns=ns, rows=rows, table=table.to(DEV),
              cache_len=torch.tensor(lens, dtype=torch.int32, device=DEV),
              row_start=torch.tensor(rows, dtype=torch.int32, device=DEV)
              if ns != [N] * B else None)
    st["kp"], st["vp"] = _pool(case, gen, n_pages), _pool(case, gen, n_pages)
    st["parent"] = st["depth"] = None
    if case["kind"] == "tree":
        trees = [_tree(r, N) for _ in range(B)]
        st["parent_h"] = [t[0] for t in trees]
        st["parent"] = torch.from_numpy(np.concatenate([t[0] for t in trees])).to(DEV)
        st["depth"] = torch.from_numpy(np.concatenate([t[1] for t in trees])).to(DEV)
        # ancestors (and self) of each node: what the plain form masks with
        anc = np.zeros((B, N, N), bool)
        for b in range(B):
            for i in range(N):
                p = int(trees[b][0][i])
                if p >= 0:
                    anc[b, i] = anc[b, p]
                anc[b, i, i] = True
        st["anc"] = torch.from_numpy(anc).to(DEV)
    op = case["op"]
    if op in ("attention", "window"):
        st["q"] = _randn(gen, dt, R, H, dh) * 1.5
        st["out"] = torch.empty_like(st["q"])
        st["logit"] = _randn(gen, torch.float32, H) if case.get("logit") else None
    elif op == "append":
        # one projection's output holds q, k and v side by side
        qkv = _randn(gen, dt, R, H + 2 * Hkv, dh)
        st["q"], st["k"], st["v"] = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
        st["q_out"] = torch.empty(R, H, dh, dtype=dt, device=DEV)
        rot = case["rot"]
        st["inv_freq"] = torch.from_numpy(
            (150000.0 ** (-np.arange(0, rot, 2) / rot)).astype(np.float32)).to(DEV)
        st["wq"] = st["wk"] = None
        if case["norm"]:
            st["wq"] = (1 + 0.2 * _randn(gen, torch.float32, dh)).to(dt)
            st["wk"] = (1 + 0.2 * _randn(gen, torch.float32, dh)).to(dt)
    else:
        P = case["P"]
        # accepted paths: the root, then nodes behind the first P (so that a pass may repeat)
        path = np.zeros((B, P), np.int32)
        for b in range(B):
            path[b, 1:] = np.sort(r.choice(np.arange(P, N), P - 1, replace=False))
        acc = r.integers(1, P + 1, B).astype(np.int32) if case["ragged"] else np.full(B, P, np.int32)
        st["path_h"], st["acc_h"] = path, acc
        st["path"] = torch.from_numpy(path).to(DEV)
        st["acc"] = torch.from_numpy(acc).to(DEV)
        st["new_len"] = torch.empty(B, dtype=torch.int32, device=DEV)
    if own:
        from expert_select_gb300 import moetree as M
        st["C"] = M.cache_desc(st["kp"], H, max_pages, window=case.get("window", 0),
                               sink_tokens=case.get("sinks", 0))
        st["ws"] = M.attention_workspace(st["C"], B, N, device=DEV)
    return st


# ----------------------------------------------------------------------------- plain forms

def _gather(pool, table_row, n, page):
    """The first n cached slots of one sequence, [n, Hkv, dh], in 32 bits."""
    pages = table_row[:-(-n // page)].long()
    t = pool[pages]
    return t.reshape(-1, t.shape[2], t.shape[3])[:n].float()


def _plain_attention(st):
    case = st["case"]
    H, Hkv, dh, page = (case[k] for k in ("H", "Hkv", "dh", "page"))
    G, W, S = H // Hkv, case.get("window", 0), case.get("sinks", 0)
    scale = 1.0 / math.sqrt(dh)
    out = st["out"]
    for b in range(case["B"]):
        ln, n, r0 = st["lens"][b], st["ns"][b], st["rows"][b]
        L = ln + n
        # a window needs the first slots and those from the oldest query's window on
        lo = max(S, ln - W + 1) if W else 0
        k = _gather(st["kp"], st["table"][b], L, page)
        v = _gather(st["vp"], st["table"][b], L, page)
        slot = torch.arange(L, device=DEV)
        if W and lo > S:
            keep = (slot < S) | (slot >= lo)
            k, v, slot = k[keep], v[keep], slot[keep]
        k, v = k.permute(1, 2, 0), v.permute(1, 0, 2)       # [Hkv, dh, K], [Hkv, K, dh]
        if st["depth"] is not None:
            dep = st["depth"][r0:r0 + n].long()
        else:
            dep = torch.arange(n, device=DEV)
        kpos = torch.where(slot < ln, slot, ln + dep[(slot - ln).clamp_min(0)])
        step = max(1, min(n, (1 << 28) // max(1, H * slot.numel())))
        for i0 in range(0, n, step):
            i1 = min(n, i0 + step)
            q = st["q"][r0 + i0:r0 + i1].float()             # [m, H, dh]
            m = i1 - i0
            qg = q.reshape(m, Hkv, G, dh).permute(1, 0, 2, 3).reshape(Hkv, m * G, dh)
            s = torch.matmul(qg, k) * scale                  # [Hkv, m G, K]
            qpos = ln + dep[i0:i1]
            if st["parent"] is not None:
                a = st["anc"][b, i0:i1][:, (slot - ln).clamp_min(0)]
                see = (slot < ln)[None, :] | a
            else:
                see = slot[None, :] <= qpos[:, None]
            if W:
                see = see & ((qpos[:, None] - kpos[None, :] < W) | (kpos < S)[None, :])
            see = see[:, None, :].expand(m, G, -1).reshape(1, m * G, -1)
            s = torch.where(see, s, torch.full_like(s, -math.inf))
            mx = s.amax(-1, keepdim=True)
            if st["logit"] is not None:
                lg = st["logit"].reshape(Hkv, 1, G, 1).expand(Hkv, m, G, 1).reshape(Hkv, m * G, 1)
                mx = torch.maximum(mx, lg)
            p = torch.exp(s - mx)
            den = p.sum(-1, keepdim=True)
            if st["logit"] is not None:
                den = den + torch.exp(lg - mx)
            o = torch.matmul(p, v) / den
            out[r0 + i0:r0 + i1] = (o.reshape(Hkv, m, G, dh).permute(1, 0, 2, 3)
                                    .reshape(m, H, dh).to(out.dtype))
    return out


def _slots(st, page):
    """(page id, slot within it, position) of every new row."""
    case = st["case"]
    ln = torch.repeat_interleave(st["cache_len"].long(),
                                 torch.tensor(st["ns"], device=DEV), output_size=st["rows"][-1])
    seq = torch.repeat_interleave(torch.arange(case["B"], device=DEV),
                                  torch.tensor(st["ns"], device=DEV), output_size=st["rows"][-1])
    first = torch.tensor(st["rows"][:-1], device=DEV)[seq]
    node = torch.arange(st["rows"][-1], device=DEV) - first
    slot = ln + node
    pos = ln + (st["depth"].long() if st["depth"] is not None else node)
    return st["table"].long()[seq, slot // page], slot % page, pos


def _plain_append(st):
    case = st["case"]
    page, rot = case["page"], case["rot"]
    pg, off, pos = _slots(st, page)
    ang = pos.double()[:, None] * st["inv_freq"].double()[None, :]
    cos, sin = torch.cos(ang).float()[:, None, :], torch.sin(ang).float()[:, None, :]

    def turn(t, w):
        t = t.float()
        if w is not None:
            t = t / torch.sqrt((t * t).mean(-1, keepdim=True) + 1e-6) * w.float()
        a, b, rest = t[..., :rot // 2], t[..., rot // 2:rot], t[..., rot:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, rest], -1)

    st["q_out"].copy_(turn(st["q"], st["wq"]))
    st["kp"][pg, off] = turn(st["k"], st["wk"]).to(st["kp"].dtype)
    st["vp"][pg, off] = st["v"]
    return st["q_out"], st["kp"], st["vp"]


def _plain_commit(st):
    case = st["case"]
    page = case["page"]
    ln, path, acc = st["cache_len"].long(), st["path"].long(), st["acc"]
    j = torch.arange(case["P"], device=DEV)
    src, dst = ln[:, None] + path, ln[:, None] + j[None, :]
    dst = torch.where(j[None, :] < acc[:, None], dst, src)    # what is not accepted stays
    spg, dpg = torch.gather(st["table"].long(), 1, src // page), torch.gather(
        st["table"].long(), 1, dst // page)
    for pool in (st["kp"], st["vp"]):
        pool[dpg, dst % page] = pool[spg, src % page]
    st["new_len"].copy_(st["cache_len"] + acc)
    return st["kp"], st["vp"], st["new_len"]


def _plain_norm(st):
    case = st["case"]
    x, u = st["x"].float(), st["branch"].float()
    if st["w_post"] is not None:
        u = u / torch.sqrt((u * u).mean(-1, keepdim=True) + 1e-6) * st["w_post"].float()
    if st["gate"] is not None:
        u = u * st["gate"].float().repeat_interleave(case["gate"], 0)[:case["R"]]
    h = x + case["scale"] * u
    st["h"].copy_(h)
    st["hn"].copy_(h / torch.sqrt((h * h).mean(-1, keepdim=True) + 1e-6) * st["w_pre"].float())
    return st["h"], st["hn"]


# ----------------------------------------------------------------------------- one pass

def run(st):
    case = st["case"]
    op = case["op"]
    if not own:
        return {"attention": _plain_attention, "window": _plain_attention,
                "append": _plain_append, "commit": _plain_commit, "norm": _plain_norm}[op](st)
    from expert_select_gb300 import moetree as M
    if op in ("attention", "window"):
        M.moe_tree_attention(st["C"], st["q"], st["kp"], st["vp"], st["table"], st["cache_len"],
                             case["B"], case["N"], st["out"], st["ws"], parent=st["parent"],
                             row_start=st["row_start"], sink_logit=st["logit"])
        return st["out"]
    if op == "append":
        M.moe_kv_append(st["C"], st["q"], st["k"], st["v"], st["kp"], st["vp"], st["table"],
                        st["cache_len"], case["B"], case["N"], st["q_out"], st["ws"],
                        depth=st["depth"], row_start=st["row_start"], inv_freq=st["inv_freq"],
                        q_weight=st["wq"], k_weight=st["wk"], eps=1e-6)
        return st["q_out"], st["kp"], st["vp"]
    if op == "commit":
        M.moe_kv_commit(st["C"], st["kp"], st["vp"], st["table"], st["cache_len"], st["path"],
                        st["acc"], st["new_len"], st["ws"])
        return st["kp"], st["vp"], st["new_len"]
    M.moe_block_norm(st["L"], st["x"], st["branch"], st["h"], st["hn"], w_post=st["w_post"],
                     gate=st["gate"], gate_rows=case["gate"], scale=case["scale"],
                     w_pre=st["w_pre"], eps=1e-6)
    return st["h"], st["hn"]


# ----------------------------------------------------------------------------- floors

def work(case):
    """Bytes and operations of a pass."""
    e = 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "norm":
        R, d = case["R"], case["d"]
        vecs = 1 + bool(case["post"]) + (-(-R // case["gate"]) if case["gate"] else 0)
        return {"bytes": (4 * R + vecs) * d * e, "flops": 10 * R * d}
    H, Hkv, dh, B = case["H"], case["Hkv"], case["dh"], case["B"]
    lens, ns = _lens(case)
    R = sum(ns)
    if case["op"] == "append":
        return {"bytes": 2 * R * (H + 2 * Hkv) * dh * e, "flops": 6 * R * (H + Hkv) * dh}
    if case["op"] == "commit":
        P = case["P"]
        moved = (P - 1) if not case["ragged"] else (P - 1) / 2
        return {"bytes": int(4 * B * moved * Hkv * dh * e) + 8 * B, "flops": 0}
    W, S = case.get("window", 0), case.get("sinks", 0)
    pairs = slots = 0
    for ln, n in zip(lens, ns):
        if case["kind"] == "tree":
            per = ln if not W else min(ln, W + S)
            pairs += n * (per + min(6, n))
            slots += per + n
        elif not W:
            pairs += n * ln + n * (n + 1) // 2
            slots += ln + n
        else:
            i = np.arange(ln, ln + n, dtype=np.int64)
            lo = np.maximum(0, i - W + 1)
            pairs += int((i - lo + 1 + np.minimum(lo, S)).sum())
            slots += int(ln + n - lo[0] + min(lo[0], S))
    return {"bytes": 2 * R * H * dh * e + 2 * slots * Hkv * dh * e,
            "flops": int(4 * pairs * H * dh)}


# ----------------------------------------------------------------------------- 64 bits

def exact(case, seed):
    """The definitions in 64 bits, one sequence (attention: one kv head) after the other."""
    st = prepare(case, seed)
    d64 = torch.float64
    if case["op"] == "norm":
        R = case["R"]
        h = st["x"].to(d64).clone()
        br = st["branch"].to(d64)
        if st["w_post"] is not None:
            ms = torch.einsum("rd,rd->r", br, br) / case["d"]
            br = br * (st["w_post"].to(d64)[None] / torch.sqrt(ms + 1e-6)[:, None])
        if st["gate"] is not None:
            idx = torch.arange(R, device=DEV).div(case["gate"], rounding_mode="floor")
            br = br * st["gate"].to(d64)[idx]
        h += case["scale"] * br
        ms = torch.einsum("rd,rd->r", h, h) / case["d"]
        return h, h * (st["w_pre"].to(d64)[None] / torch.sqrt(ms + 1e-6)[:, None])

    page = case["page"]
    table = st["table"].cpu().numpy()

    def where(b, slots):
        slots = np.asarray(slots)
        return (torch.from_numpy(table[b][slots // page]).long().to(DEV),
                torch.from_numpy(slots % page).long().to(DEV))

    if case["op"] == "commit":
        kp, vp = st["kp"].to(d64), st["vp"].to(d64)
        for b in range(case["B"]):
            n = int(st["acc_h"][b])
            s = where(b, st["lens"][b] + st["path_h"][b][:n])
            t = where(b, st["lens"][b] + np.arange(n))
            for pool in (kp, vp):
                pool[t] = pool[s]
        return kp, vp, torch.tensor(st["lens"], device=DEV).int() + st["acc"]

    if case["op"] == "append":
        kp, vp = st["kp"].to(d64), st["vp"].to(d64)
        half = case["rot"] // 2
        freq = st["inv_freq"].cpu().numpy().astype(np.float64)
        outs = []
        for b in range(case["B"]):
            ln, n, r0 = st["lens"][b], st["ns"][b], st["rows"][b]
            dep = (st["depth"][r0:r0 + n].cpu().numpy() if st["depth"] is not None
                   else np.arange(n))
            z = np.exp(1j * ((ln + dep)[:, None] * freq[None]))
            z = torch.from_numpy(z).to(DEV)[:, None, :]

            def rotate(t, w):
                t = t[r0:r0 + n].to(d64)
                if w is not None:
                    t = t * torch.rsqrt(t.square().sum(-1, keepdim=True) / case["dh"] + 1e-6)
                    t = t * w.to(d64)
                c = torch.complex(t[..., :half].contiguous(), t[..., half:2 * half].contiguous())
                c = c * z
                return torch.cat([c.real, c.imag, t[..., 2 * half:]], -1)

            outs.append(rotate(st["q"], st["wq"]))
            to = where(b, ln + np.arange(n))
            kp[to] = rotate(st["k"], st["wk"])
            vp[to] = st["v"][r0:r0 + n].to(d64)
        return torch.cat(outs), kp, vp

    H, Hkv, dh = case["H"], case["Hkv"], case["dh"]
    G, W, S = H // Hkv, case.get("window", 0), case.get("sinks", 0)
    if work(case)["flops"] > 8e12:
        return None
    out = torch.zeros(st["rows"][-1], H, dh, dtype=d64, device=DEV)
    for b in range(case["B"]):
        ln, n, r0 = st["lens"][b], st["ns"][b], st["rows"][b]
        # (query node, slot) pairs that see one another, from the definition
        kpos = np.arange(ln + n)
        if case["kind"] == "tree":
            par = st["parent_h"][b]
            lvl = np.zeros(n, np.int64)
            tree = np.zeros((n, n), bool)
            for i in range(n):
                j = i
                while j >= 0:
                    tree[i, j] = True
                    j = int(par[j])
                lvl[i] = tree[i].sum() - 1
        else:
            lvl, tree = np.arange(n), None
        kpos[ln:] = ln + lvl
        first = 0
        if W:
            first = max(0, ln - W + 1)
        use = np.concatenate([np.arange(min(S, first)), np.arange(first, ln + n)])
        pg = where(b, use)
        kpos_u = torch.from_numpy(kpos[use]).to(DEV)
        old = torch.from_numpy(use < ln).to(DEV)
        for g in range(Hkv):
            k, v = st["kp"][pg[0], pg[1], g].to(d64), st["vp"][pg[0], pg[1], g].to(d64)
            for i0 in range(0, n, 1024):
                i1 = min(n, i0 + 1024)
                qp = torch.from_numpy(ln + lvl[i0:i1]).to(DEV)
                if tree is None:
                    ok = kpos_u[None] <= qp[:, None]
                else:
                    ok = torch.zeros(i1 - i0, len(use), dtype=torch.bool, device=DEV)
                    ok[:, old] = True
                    ok[:, len(use) - n:] = torch.from_numpy(tree[i0:i1]).to(DEV)
                if W:
                    ok &= (kpos_u[None] > qp[:, None] - W) | (kpos_u[None] < S)
                for j in range(G):
                    hd = g * G + j
                    s = (st["q"][r0 + i0:r0 + i1, hd].to(d64) / math.sqrt(dh)) @ k.T
                    s.masked_fill_(~ok, -math.inf)
                    if st["logit"] is not None:
                        s = torch.cat([s, st["logit"][hd].to(d64).expand(i1 - i0, 1)], 1)
                    p = torch.softmax(s, 1)[:, :len(use)]
                    out[r0 + i0:r0 + i1, hd] = p @ v
    return out
