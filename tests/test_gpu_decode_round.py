"""GPU tests of the decoding calls as they are used together: rounds of drafting, verification and
commits over pages that are reserved, forked, given back and compacted; captured and replayed; on
several streams."""
import numpy as np
import pytest
import torch

from expert_select_gb300 import moetree as M

pytestmark = pytest.mark.gpu
DEV = "cuda"
I32 = dict(dtype=torch.int32, device=DEV)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from expert_select_gb300 import build
    build.build()
    M.lib()


class Model:
    """One fp32 block (attention half, experts) between an embedding and a head, random weights."""

    d, H, Hkv, dh, E, k, f, V = 128, 8, 2, 32, 12, 3, 64, 300

    def __init__(self, seed):
        g = torch.Generator(device=DEV).manual_seed(seed)
        n = lambda *s, std=1.0: torch.randn(*s, generator=g, device=DEV) * std  # noqa: E731
        d, hq, hk = self.d, self.H * self.dh, self.Hkv * self.dh
        self.emb, self.head = n(self.V, d), n(self.V, d, std=0.3)
        self.wqkv, self.wo = n(hq + 2 * hk, d, std=d ** -0.5), n(d, hq, std=hq ** -0.5)
        self.wr = n(self.E, d, std=0.2)
        self.wg, self.wu = n(self.E, self.f, d, std=0.1), n(self.E, self.f, d, std=0.1)
        self.wd = n(self.E, d, self.f, std=0.2)
        self.inv_freq = (10000.0 ** (-torch.arange(0, self.dh, 2, device=DEV) / self.dh)).float()
        self.L = M.layer_desc(d, self.E, self.k, self.f, torch.float32)
        self.few_ws = M.few_workspace(self.L, 16)


class Engine:
    """Sequences over one layer's pages."""

    def __init__(self, model, B, n_pages=64, page=8, width=24):
        self.m, self.B, self.page = model, B, page
        shape = (n_pages, page, model.Hkv, model.dh)
        self.kp, self.vp = torch.randn(shape, device=DEV), torch.randn(shape, device=DEV)
        self.table = torch.full((B, width), -1, **I32)
        self.held, self.lens = torch.zeros(B, **I32), torch.zeros(B, **I32)
        self.ref = torch.zeros(n_pages, **I32)
        self.book = M.page_book(self.table, self.held, self.lens, self.ref, page)
        self.ws = M.pages_workspace(self.book)
        self.C = M.cache_desc(self.kp, model.H, width)
        self.aws = M.attention_workspace(self.C, B, 64)

    def step(self, tokens, parent=None, depth=None, n_new=None, rows=None):
        """Logits [R, V] of every new token of every sequence; their keys and values are in the cache.
        tokens [R], N = R / B rows a sequence, or rows[b] each."""
        m = self.m
        R = tokens.numel()
        N = R // self.B if rows is None else int(max(np.diff(rows)))
        start = None if rows is None else torch.tensor(rows, **I32)
        M.moe_kv_reserve(self.book, N, self.ws, n_new=n_new)
        x = m.emb[tokens.long()]
        xn = torch.empty_like(x)
        M.moe_block_norm(m.L, x, h=None, hn=xn)
        qkv = (xn @ m.wqkv.T).view(R, m.H + 2 * m.Hkv, m.dh)
        q, k, v = qkv[:, :m.H], qkv[:, m.H:m.H + m.Hkv], qkv[:, m.H + m.Hkv:]
        qr = torch.empty(R, m.H, m.dh, device=DEV)
        M.moe_kv_append(self.C, q, k, v, self.kp, self.vp, self.table, self.lens, self.B, N, qr,
                        self.aws, depth=depth, row_start=start, inv_freq=m.inv_freq)
        o = torch.empty_like(qr)
        M.moe_tree_attention(self.C, qr, self.kp, self.vp, self.table, self.lens, self.B, N, o,
                             self.aws, parent=parent, row_start=start)
        h = torch.empty_like(x)
        M.moe_block_norm(m.L, x, o.view(R, -1) @ m.wo.T, h=h)
        opts = M.run_opts(residual=True, norm_input=True)
        for r0 in range(0, R, 16):  # in groups, as the layer for a few tokens takes them
            part = h[r0:r0 + 16]
            M.moe_few_forward(m.L, part, m.wr, m.wg, m.wu, m.wd, None, part, m.few_ws, opts=opts)
        return h @ m.head.T

    def sample(self, logits, u, group=1, **kw):
        token = torch.empty(logits.shape[0], **I32)
        M.moe_sample(logits, u, token, param_rows=group, **kw)
        return token

    def checks(self):
        for ws in (self.ws, self.aws, self.m.few_ws):
            assert M.moe_workspace_check(ws) == 0


def _prompts(B, seed):
    r = np.random.default_rng(seed)
    ns = [int(v) for v in r.integers(3, 30, B)]
    toks = [r.integers(0, Model.V, n) for n in ns]
    return ns, torch.tensor(np.concatenate(toks), **I32)


def _prefill(e, seed):
    """The first sampled token of each sequence (greedy)."""
    ns, toks = _prompts(e.B, seed)
    rows = np.concatenate([[0], np.cumsum(ns)])
    lg = e.step(toks, n_new=torch.tensor(ns, **I32), rows=rows)
    e.lens += torch.tensor(ns, **I32)
    T = torch.zeros(e.B, device=DEV)
    return e.sample(lg[torch.from_numpy(rows[1:] - 1).to(DEV)].contiguous(),
                    torch.zeros(e.B, device=DEV), temperature=T)


def _plain(model, B, steps, seed):
    """Greedy decoding token by token."""
    e = Engine(model, B)
    tok = _prefill(e, seed)
    out = [tok]
    T, u = torch.zeros(B, device=DEV), torch.zeros(B, device=DEV)
    for _ in range(steps):
        lg = e.step(tok)
        e.lens += 1
        tok = e.sample(lg, u, temperature=T)
        out.append(tok)
    e.checks()
    return torch.stack(out, 1).cpu().numpy()


def _tree(r, N):
    parent = np.full(N, -1, np.int32)
    for i in range(1, N):
        parent[i] = int(i * r.random() ** 2)
    depth = np.zeros(N, np.int32)
    for i in range(1, N):
        depth[i] = depth[parent[i]] + 1
    return parent, depth


@pytest.mark.parametrize("compact", [False, True])
def test_drafted_rounds_give_the_tokens_of_plain_decoding(compact):
    """Drafts that are partly right are verified as trees; what is emitted is what greedy decoding token
    by token gives, whatever is accepted, also over a pool that is compacted on the way."""
    m, B, steps, N, P = Model(1), 3, 24, 14, 6
    want = _plain(m, B, steps + P, 5)
    r = np.random.default_rng(2)
    e = Engine(m, B)
    root = _prefill(e, 5)
    got = [[int(t)] for t in root.cpu()]
    T = torch.zeros(B, device=DEV)
    accepted = []
    for rnd in range(40):
        if min(map(len, got)) > steps:
            break
        trees = [_tree(r, N) for _ in range(B)]
        draft = r.integers(0, m.V, (B, N)).astype(np.int32)
        for b, (par, dep) in enumerate(trees):
            draft[b, 0] = got[b][-1]
            for i in range(1, N):  # the right token now and then, in one or several branches
                at = len(got[b]) - 1 + dep[i]
                if r.random() < 0.6 and at < want.shape[1]:
                    draft[b, i] = want[b, at]
        up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV).view(-1)  # noqa: E731
        parent, depth = up(np.stack([t[0] for t in trees])), up(np.stack([t[1] for t in trees]))
        tokens = up(draft)
        lg = e.step(tokens, parent=parent, depth=depth)
        s = e.sample(lg, torch.rand(B * N, device=DEV), group=N, temperature=T)
        path, acc, out = torch.empty(B, P, **I32), torch.empty(B, **I32), torch.empty(B, P, **I32)
        M.moe_tree_accept(tokens, parent, s, B, N, path, acc, out)
        M.moe_kv_commit(e.C, e.kp, e.vp, e.table, e.lens, path, acc, e.lens, e.aws)
        # pages behind the accepted tokens go back
        M.moe_kv_free(e.book, torch.arange(B, **I32), e.ws, keep=e.lens.clone())
        for b in range(B):
            n = int(acc[b])
            accepted.append(n)
            got[b] += out[b, :n].tolist()
        if compact and rnd % 3 == 1:
            moves, counts = torch.empty(e.ref.numel() // 2, 3, **I32), torch.empty(2, **I32)
            M.moe_kv_compact(e.book, e.table, e.ref, moves, counts, e.ws)
            M.moe_kv_copy_pages(e.C, e.kp, e.vp, moves, count=counts, ws=e.ws)
            used = int((e.ref > 0).sum())
            assert counts[1].item() == used and (e.ref[used:] == 0).all()
            dead = torch.full_like(e.kp[used:], float("nan"))  # nothing is left there
            e.kp[used:], e.vp[used:] = dead, dead
    e.checks()
    assert min(accepted) >= 1 and max(accepted) > 2
    for b in range(B):
        n = min(len(got[b]), want.shape[1])
        assert n > steps and got[b][:n] == want[b, :n].tolist()


def test_forks_go_their_own_ways():
    """Forks of a prompt's sequence: their pages are shared up to the last full one, and each goes on as
    if it had the prompt to itself."""
    m, page = Model(3), 8
    ns, toks = [21], torch.tensor(np.random.default_rng(0).integers(0, Model.V, 21), **I32)
    u = torch.rand(12, 4, generator=torch.Generator().manual_seed(3)).to(DEV)
    T, K = torch.full((4,), 0.9, device=DEV), torch.full((4,), 40, **I32)

    def alone(j):
        e = Engine(m, 1)
        lg = e.step(toks)
        e.lens += 21
        tok = e.sample(lg[-1:].contiguous(), u[0, j:j + 1], temperature=T[:1], top_k=K[:1])
        out = [int(tok)]
        for s in range(1, 12):
            lg = e.step(tok)
            e.lens += 1
            tok = e.sample(lg, u[s, j:j + 1], temperature=T[:1], top_k=K[:1])
            out.append(int(tok))
        return out

    e = Engine(m, 4)
    lg = e.step(toks, n_new=torch.tensor([21, 0, 0, 0], **I32), rows=[0, 21, 21, 21, 21])
    e.lens[0] += 21
    moves = torch.empty(3, 3, **I32)
    M.moe_kv_fork(e.book, torch.zeros(3, **I32), torch.tensor([1, 2, 3], **I32), moves, e.ws)
    M.moe_kv_copy_pages(e.C, e.kp, e.vp, moves, ws=e.ws)
    assert e.lens.tolist() == [21] * 4 and (e.table[:, :2] == e.table[0, :2]).all()
    assert (e.ref == 4).sum() == 21 // page and len(set(e.table[:, 2].tolist())) == 4
    tok = e.sample(lg[-1:].expand(4, -1).contiguous(), u[0], temperature=T, top_k=K)
    out = [tok]
    for s in range(1, 12):
        lg = e.step(tok)
        e.lens += 1
        tok = e.sample(lg, u[s], temperature=T, top_k=K)
        out.append(tok)
    e.checks()
    got = torch.stack(out, 1).tolist()
    assert got == [alone(j) for j in range(4)]
    M.moe_kv_free(e.book, torch.arange(4, **I32), e.ws)
    assert (e.ref == 0).all() and (e.held == 0).all()


def test_a_captured_round_is_replayed_with_other_inputs():
    m, B, N, P = Model(7), 2, 7, 4
    r = np.random.default_rng(7)
    parent, depth = (torch.from_numpy(np.concatenate([t] * B)).to(DEV) for t in _tree(r, N))

    def fresh():
        e = Engine(m, B)
        _prefill(e, 9)
        return e

    def state(e):
        return [t.clone() for t in (e.kp, e.vp, e.table, e.held, e.lens, e.ref)]

    def put(e, s):
        for t, v in zip((e.kp, e.vp, e.table, e.held, e.lens, e.ref), s):
            t.copy_(v)

    e = fresh()
    s0 = state(e)
    tokens, u = torch.zeros(B * N, **I32), torch.zeros(B * N, device=DEV)
    T, p = torch.full((B,), 1.1, device=DEV), torch.full((B,), 0.8, device=DEV)
    path, acc, out = torch.empty(B, P, **I32), torch.empty(B, **I32), torch.empty(B, P, **I32)
    moves, counts = torch.empty(e.ref.numel() // 2, 3, **I32), torch.empty(2, **I32)
    keep = torch.empty(B, **I32)
    both = torch.arange(B, **I32)

    def round_():
        lg = e.step(tokens, parent=parent, depth=depth)
        s = e.sample(lg, u, group=N, temperature=T, top_p=p)
        M.moe_tree_accept(tokens, parent, s, B, N, path, acc, out)
        M.moe_kv_commit(e.C, e.kp, e.vp, e.table, e.lens, path, acc, e.lens, e.aws)
        keep.copy_(e.lens)
        M.moe_kv_free(e.book, both, e.ws, keep=keep)
        M.moe_kv_compact(e.book, e.table, e.ref, moves, counts, e.ws)
        M.moe_kv_copy_pages(e.C, e.kp, e.vp, moves, count=counts, ws=e.ws)
        return lg

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        round_()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lg = round_()
    for i in range(4):
        tokens.copy_(torch.from_numpy(r.integers(0, m.V, B * N).astype(np.int32)))
        u.copy_(torch.from_numpy(r.random(B * N).astype(np.float32)))
        T.fill_(0.3 + 0.4 * i)
        p.fill_(1.0 - 0.2 * i)
        put(e, s0)
        want_lg = round_().clone()
        want = state(e) + [t.clone() for t in (path, acc, out, counts)]
        put(e, s0)
        g.replay()
        for a, b in zip([want_lg] + want, [lg] + state(e) + [path, acc, out, counts]):
            assert torch.equal(a, b)
    e.checks()


def test_calls_on_two_streams_at_once():
    """Each with a workspace of its own; the few-token launches are capped so that both have room."""
    dt, d, E, k, f = torch.bfloat16, 512, 32, 4, 256
    g = torch.Generator(device=DEV).manual_seed(1)
    n = lambda *s: (torch.randn(*s, generator=g, device=DEV) * 0.1).to(dt)  # noqa: E731
    wr, wg, wu, wd = n(E, d), n(E, f, d), n(E, f, d), n(E, d, f)
    L = M.layer_desc(d, E, k, f, dt)
    lanes = []
    for i in range(2):
        x = n(5 + 6 * i, d) * 10
        lg = n(70, 9001).float() * 30
        lanes.append(dict(s=torch.cuda.Stream(), x=x, y=torch.empty_like(x), ws=M.few_workspace(L, x.shape[0]),
                          lg=lg, u=torch.rand(70, generator=g, device=DEV), tok=torch.empty(70, **I32),
                          p=torch.full((70,), 0.9, device=DEV)))
    opts = M.run_opts(residual=True, norm_input=True, ffn_max_ctas=70)

    def calls(a, stream):
        M.moe_few_forward(L, a["x"], wr, wg, wu, wd, None, a["y"], a["ws"], opts=opts, stream=stream)
        M.moe_sample(a["lg"], a["u"], a["tok"], top_p=a["p"], stream=stream)

    want = []
    for a in lanes:
        calls(a, None)
        want.append((a["y"].clone(), a["tok"].clone()))
    torch.cuda.synchronize()
    for rep in range(20):
        for a in lanes:
            a["y"].zero_()
            a["tok"].zero_()
        torch.cuda.synchronize()
        for _ in range(3):
            for a in lanes:
                calls(a, a["s"])
        torch.cuda.synchronize()
        for a, (y, tok) in zip(lanes, want):
            assert torch.equal(a["y"], y) and torch.equal(a["tok"], tok)
            assert M.moe_workspace_check(a["ws"]) == 0
