"""GPU tests of what a decoding round needs beside the tree's layer and attention (moe_few_forward,
moe_sample, moe_tree_accept, the pages' calls) against plain 64-bit computations.

The layer's tolerance, per output element (u = half a step of the type: 2^-8 bf16, 2^-24 fp32; sums of
n fp32 terms t: (n + 32) 2^-24 sum |t|, the 32 for the fixed tree behind each lane's share):
  * gate and up products: eG, eU = (d + 32) 2^-24 sum |w| |x|;
  * activation h = silu(g) u, |silu'| <= 1.1: dh = 1.1 eG (|u| + eU) + (|silu g| + 1.1 eG) eU + r |h|,
    r = 2^-20 for exp, the divide and three products, and for bf16 2^-17 more (value and rest);
  * gates: scores off by eL = (d + 32) 2^-24 sum |w_r| |x|, so 2 max eL + 2^-20 relative;
  * output: sum |w_d| dh + ((k f + 64) 2^-24 + the gates') sum |w_d| |h|, and u |y|.
"""
import math

import numpy as np
import pytest
import torch

from expert_select_gb300 import moetree as M

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from expert_select_gb300 import build
    build.build()
    M.lib()


# --------------------------------------------------------------------- a few tokens

class Few:
    def __init__(self, seed, R, d, E, k, f, dtype, slots=False, std=0.02, same=False):
        g = torch.Generator().manual_seed(seed)
        n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        self.shape = (R, d, E, k, f)
        self.dtype = dtype
        self.x = n(R, d).to(dtype)
        if same:
            self.x[:] = self.x[:1]
        self.wr = (n(E, d) * std).to(dtype)
        S = E + 3 if slots else E
        self.wg, self.wu = (n(S, f, d) * 0.05).to(dtype), (n(S, f, d) * 0.05).to(dtype)
        self.wd = (n(S, d, f) * 0.05).to(dtype)
        self.slot = (torch.randperm(S, generator=g)[:E].int() if slots else None)
        self.L = M.layer_desc(d, E, k, f, dtype, slots=S)

    def upload(self):
        up = lambda t: None if t is None else t.to(DEV)  # noqa: E731
        self.dev = [up(t) for t in (self.x, self.wr, self.wg, self.wu, self.wd, self.slot)]
        R, d, E, k, f = self.shape
        self.logits = torch.empty(R, E, device=DEV)
        self.idx = torch.empty(R, k, dtype=torch.int32, device=DEV)
        self.gates = torch.empty(R, k, device=DEV)
        self.ws = M.few_workspace(self.L, R)
        self.y = torch.full((R, d), 7.0, dtype=self.dtype, device=DEV)
        return self

    def run(self, norm=False, residual=False, max_ctas=0, y=None):
        x, wr, wg, wu, wd, slot = self.dev
        M.moe_few_forward(self.L, x, wr, wg, wu, wd, slot, self.y if y is None else y, self.ws,
                          logits=self.logits, topk_idx=self.idx, gates=self.gates,
                          opts=M.run_opts(residual=residual, norm_input=norm,
                                          ffn_max_ctas=max_ctas))
        return self

    def check(self, norm=False, residual=False, y=None):
        R, d, E, k, f = self.shape
        assert M.moe_workspace_check(self.ws) == 0
        x = self.x.double()
        inp = x
        if norm:
            inp = (x / torch.sqrt((x * x).mean(1, keepdim=True) + 1e-6)).to(self.dtype).double()
        wr = self.wr.double()
        logits, eL = inp @ wr.T, (d + 32) * 2.0 ** -24 * (inp.abs() @ wr.abs().T)
        got = self.logits.cpu()
        assert ((got.double() - logits).abs() <= eL).all()
        top, idx = torch.sort(got, dim=1, descending=True, stable=True)
        assert torch.equal(self.idx.cpu().long(), idx[:, :k])
        gates = torch.softmax(logits.gather(1, idx[:, :k]), 1)
        egate = 2 * eL.amax(1, keepdim=True) + 2.0 ** -20
        assert ((self.gates.cpu().double() - gates).abs() <= egate * gates).all()
        out = (self.y if y is None else y).cpu().double()
        rel = 2.0 ** -20 + (2.0 ** -17 if self.dtype == torch.bfloat16 else 0)
        for r in range(R):
            want, tol = (x[r].clone() if residual else torch.zeros(d, dtype=torch.float64)), 0
            xr = inp[r]
            for j in range(k):
                e = int(idx[r, j])
                s = e if self.slot is None else int(self.slot[e])
                wg, wu, wd = (t[s].double() for t in (self.wg, self.wu, self.wd))
                g, u = wg @ xr, wu @ xr
                eG, eU = ((d + 32) * 2.0 ** -24 * (t.abs() @ xr.abs()) for t in (wg, wu))
                sl = g * torch.sigmoid(g)
                h = sl * u
                dh = 1.1 * eG * (u.abs() + eU) + (sl.abs() + 1.1 * eG) * eU + rel * h.abs()
                want = want + gates[r, j] * (wd @ h)
                tol = tol + gates[r, j] * (wd.abs() @ dh + ((k * f + 64) * 2.0 ** -24 + egate[r]) *
                                           (wd.abs() @ h.abs()))
            tol = tol * (1 + 2.0 ** -8) + U[self.dtype] * want.abs() + 1e-30
            bad = (out[r] - want).abs() > tol
            assert not bad.any(), (r, int(bad.sum()), float(((out[r] - want).abs() / tol).max()))


FEW = [
    # R, d, E, k, f, dtype, options
    (1, 2048, 128, 8, 768, "bf16", {}), (1, 256, 8, 2, 64, "bf16", {}),
    (8, 512, 32, 4, 128, "bf16", {}), (9, 512, 32, 4, 128, "bf16", {}),
    (16, 320, 64, 8, 96, "bf16", dict(slots=True)), (16, 320, 64, 8, 96, "bf16", dict(same=True)),
    (7, 72, 5, 5, 40, "bf16", {}), (3, 8, 1, 1, 8, "bf16", {}), (2, 2888, 6, 3, 1000, "bf16", {}),
    (16, 6144, 4, 2, 8, "bf16", {}), (12, 64, 256, 16, 24, "bf16", dict(std=0.5)),
    (5, 264, 200, 16, 16, "bf16", dict(same=True, slots=True)),
    (1, 256, 8, 2, 64, "fp32", {}), (16, 136, 20, 3, 72, "fp32", dict(slots=True)),
    (6, 8, 3, 3, 8, "fp32", {}), (16, 6144, 4, 2, 8, "fp32", {}), (4, 520, 40, 16, 264, "fp32", {}),
]


@pytest.mark.parametrize("case", FEW, ids=lambda c: "-".join(map(str, c[:6])) + "".join(c[6]))
@pytest.mark.parametrize("norm,residual", [(False, False), (True, True)], ids=["plain", "block"])
def test_few_tokens(case, norm, residual):
    R, d, E, k, f, dt, kw = case
    t = Few(R + d + E, R, d, E, k, f, torch.bfloat16 if dt == "bf16" else torch.float32, **kw)
    t.upload().run(norm, residual).check(norm, residual)
    # again, on the same workspace and another number of CTAs, over its own input
    first = t.y.clone()
    t.run(norm, residual)
    assert torch.equal(first, t.y)
    x = t.dev[0].clone()
    t.dev[0] = x
    t.run(norm, residual, max_ctas=37, y=x).check(norm, residual, y=x)


def test_few_agrees_with_the_tree_layer():
    t = Few(5, 6, 512, 32, 4, 128, torch.bfloat16).upload().run(True, True)
    x, wr, wg, wu, wd, _ = t.dev
    y = torch.empty_like(x)
    M.moe_tree_forward(t.L, M.select_params(M.MOE_ROUTE_NATURAL), x, wr, wg, wu, wd, None,
                       torch.zeros(6, dtype=torch.int32, device=DEV), 1, 6, None, y,
                       M.workspace(t.L, 1, 6), None, M.run_opts(residual=True, norm_input=True))
    # both round the output once, and the tree's layer its activations and experts' outputs too
    a, b, x = t.y.double(), y.double(), x.double()
    assert ((a - b).abs() <= 2.0 ** -8 * (a.abs() + b.abs()) + 2.0 ** -5 * (a - x).abs().amax()).all()


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_few_scales_of_the_norm(dt):
    """Rows whose squares leave fp32's range, tiny rows and zero rows."""
    t = Few(3, 5, 256, 8, 2, 64, dt)
    for r, by in enumerate((1e25, 1e-25, 0.0, 1e-3, 3e18)):
        t.x[r] = (t.x[r].double() * by).to(dt)
    t.upload().run(norm=True, residual=False).check(norm=True)


def test_few_bad_slots_and_other_experts_infinities():
    t = Few(11, 4, 128, 16, 2, 64, torch.bfloat16, slots=True).upload().run()
    base = t.y.clone()
    chosen = t.idx.cpu()
    # weights that only token 0 meets hold infinities: the other tokens keep their outputs
    only = [int(e) for e in chosen[0] if int(e) not in chosen[1:].flatten().tolist()]
    assert only
    s = int(t.slot[only[0]])
    keep = [t.dev[i][s].clone() for i in (2, 3, 4)]
    for i in (2, 3, 4):
        t.dev[i][s] = math.inf
    t.run()
    assert torch.equal(t.y[1:], base[1:])
    assert not torch.isfinite(t.y[0]).any()
    for i, w in zip((2, 3, 4), keep):
        t.dev[i][s] = w
    # a token that is not finite keeps to itself
    t.dev[0][2] = math.nan
    t.run()
    assert torch.equal(t.y[[0, 1, 3]], base[[0, 1, 3]]) and t.y[2].isnan().all()
    t.dev[0][2] = t.x[2].to(DEV)
    # an expert outside the pool is skipped and told
    t.dev[5][only[0]] = t.L.slots
    t.run()
    assert torch.equal(t.y[1:], base[1:]) and torch.isfinite(t.y).all()
    assert M.moe_workspace_check(t.ws) == 1 and M.moe_workspace_check(t.ws) == 0


# --------------------------------------------------------------------- sampling

def sample_ref(logits, u, T, k, p, m):
    """Token and log probability of one row (numpy float64 of the row's values)."""
    x = logits.astype(np.float64).copy()
    x[np.isnan(x)] = -np.inf
    V = len(x)
    if not (x > -np.inf).any():
        return -1, -math.inf
    if not T > 0:
        return int(np.argmax(x)), 0.0
    with np.errstate(invalid="ignore", over="ignore"):
        s = (x - x.max()) / T
    s[x == -np.inf] = -np.inf
    w = np.exp(s)  # (64 bits, not long double: values that differ by 1e-30 weigh the same)
    w[w < 2.0 ** -43] = 0
    order = np.argsort(-x, kind="stable")
    keep = np.zeros(V, bool)
    n = k if 0 < k < V else V
    keep[order[:n]] = True
    if p < 1:
        before = np.cumsum(w[order[:n]]) - w[order[:n]]
        out = before >= p * w[order[:n]].sum()
        out[0] = False
        keep[order[:n][out]] = False
    if m > 0:
        keep &= s >= math.log(min(m, 1.0))
    w = np.where(keep, w, 0)
    c = np.cumsum(w)
    u = 0.0 if not u > 0 else u
    t = int(np.searchsorted(c, u * c[-1], side="right")) if u < 1 else V
    last = int(np.flatnonzero(w > 0)[-1])
    t = min(t, last)
    return t, float(np.log(w[t] / c[-1]))


def sample_check(x, u, T=None, k=None, p=None, m=None, group=1, pad=0, shift=0):
    R, V = x.shape
    buf = torch.full((R * (V + pad) + shift + 16,), math.nan, dtype=x.dtype, device=DEV)
    rows = buf[shift:shift + R * (V + pad)].view(R, V + pad)[:, :V]
    rows.copy_(x)
    n = -(-R // group)
    put = lambda v, dt: None if v is None else torch.as_tensor(v, dtype=dt).expand(n).contiguous().to(DEV)  # noqa: E731
    Td, kd = put(T, torch.float32), put(k, torch.int32)
    pd, md = put(p, torch.float32), put(m, torch.float32)
    token = torch.full((R,), -9, dtype=torch.int32, device=DEV)
    lp = torch.empty(R, device=DEV)
    M.moe_sample(rows, u.to(DEV), token, temperature=Td, top_k=kd, top_p=pd, min_p=md,
                 param_rows=group, logprob=lp)
    got, lp = token.cpu().numpy(), lp.cpu().numpy()
    at = lambda t, i, v: v if t is None else t[i // group].item()  # noqa: E731
    xs = x.float().numpy()
    big = torch.finfo(x.dtype).max
    for r in range(R):
        t, l = sample_ref(np.minimum(xs[r], np.float32(big)), u[r].item(), at(Td, r, 1.0),
                          at(kd, r, 0), at(pd, r, 1.0), at(md, r, 0.0))
        assert got[r] == t, (r, got[r], t)
        # fp32 steps: the difference over T and the logarithm, each off by a few 2^-24 of itself
        assert lp[r] == l or abs(lp[r] - l) <= 2.0 ** -20 * (abs(l) + 2.0 ** -20), (r, lp[r], l)


def peaked(g, R, V, dt, sigma=2.5):
    x = torch.randn(R, V, generator=g) * sigma
    x.scatter_add_(1, torch.randint(0, V, (R, 16), generator=g), 5 + 9 * torch.rand(R, 16, generator=g))
    return x.to(dt)


SETTINGS = [dict(), dict(T=0.0), dict(T=0.7, k=50, p=0.95), dict(k=1), dict(p=0.9), dict(p=0.3, m=0.1),
            dict(T=1.5, k=700, p=0.99), dict(m=0.05), dict(k=5, m=1.0), dict(T=0.01), dict(T=300.0, p=0.5),
            dict(T=1.3, p=0.9999), dict(k=100000, p=0.97), dict(p=0.0), dict(p=1e-9, k=3)]


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [1, 2, 7, 33, 1000, 50257, 151936])
def test_sample_settings(V, dt):
    g = torch.Generator().manual_seed(V)
    R = 6 if V > 10000 else 24
    for i, kw in enumerate(SETTINGS):
        u = torch.rand(R, generator=g)
        sample_check(peaked(g, R, V, dt), u, pad=i % 5, shift=i % 4, **kw)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_sample_rows_beyond_shared_memory(dt):
    g = torch.Generator().manual_seed(3)
    for kw in (dict(), dict(p=0.9), dict(k=40, T=0.8)):
        sample_check(peaked(g, 2, 524288, dt), torch.rand(2, generator=g), shift=1, **kw)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_sample_many_rows_with_their_own_settings(dt):
    g = torch.Generator().manual_seed(8)
    R, V, N = 330, 4001, 3
    n = R // N
    pick = lambda vals: torch.tensor(vals)[torch.randint(0, len(vals), (n,), generator=g)]  # noqa: E731
    sample_check(peaked(g, R, V, dt), torch.rand(R, generator=g), T=pick([0.0, 0.5, 1.0, 2.0]),
                 k=pick([0, 1, 10, 900]), p=pick([1.0, 0.9, 0.5]), m=pick([0.0, 0.02, 0.3]), group=N)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [13, 4099, 70001])
def test_sample_ties_and_masks(V, dt):
    """Equal values across every cut, masked rows of each kind, and what is not a number."""
    g = torch.Generator().manual_seed(V)
    low = torch.finfo(dt).min
    rows = [torch.zeros(V), torch.full((V,), -3.0), torch.full((V,), low),
            torch.randint(0, 3, (V,), generator=g).float(),
            torch.randint(-2, 2, (V,), generator=g).float() * 0.25,
            torch.where(torch.rand(V, generator=g) < 0.9, -math.inf, 1.5),
            torch.where(torch.rand(V, generator=g) < 0.9, low, torch.randn(V, generator=g)),
            torch.where(torch.rand(V, generator=g) < 0.5, math.nan, torch.randn(V, generator=g)),
            torch.full((V,), -math.inf), torch.full((V,), math.nan),
            torch.where(torch.rand(V, generator=g) < 0.2, math.inf, torch.randn(V, generator=g)),
            torch.where(torch.arange(V) == V // 2, math.inf, -0.0),
            torch.where(torch.rand(V, generator=g) < 0.5, 0.0, -0.0),
            torch.randn(V, generator=g) * 1e-3, torch.randn(V, generator=g) * 1e-30,
            torch.randn(V, generator=g) * 200, torch.randn(V, generator=g) * 1e6,
            torch.arange(V).float() * 2.0 ** -20, 300 + torch.randn(V, generator=g)]
    x = torch.stack(rows).to(dt)
    R = len(rows)
    for kw in (dict(), dict(k=V // 3 + 1), dict(p=0.5), dict(p=0.35, k=max(1, V // 2)), dict(m=0.5),
               dict(T=0.0), dict(T=1e-20, p=0.7), dict(T=1e20, k=9), dict(T=0.5, k=3, p=0.6, m=0.2)):
        for u in (torch.rand(R, generator=g), torch.full((R,), 0.5), torch.zeros(R)):
            sample_check(x, u, **kw)


def test_sample_random_numbers_at_the_ends():
    g = torch.Generator().manual_seed(2)
    u = torch.tensor([0.0, -1.0, math.nan, 1.0 - 2.0 ** -24, 1.0, 7.0, 2.0 ** -30, math.inf])
    for dt in (torch.bfloat16, torch.float32):
        for kw in (dict(), dict(k=20, p=0.9)):
            sample_check(peaked(g, len(u), 2003, dt), u, **kw)


def test_sample_temperatures_at_the_ends():
    g = torch.Generator().manual_seed(4)
    T = torch.tensor([math.inf, 1e-45, 1e38, math.nan, -1.0, -0.0])
    x = torch.randn(6, 777, generator=g)
    ref = x.clone()
    # beyond 10^30 all tokens weigh the same, below 10^-30 only the largest ones count
    token = torch.empty(6, dtype=torch.int32, device=DEV)
    u = torch.rand(6, generator=g)
    M.moe_sample(x.to(DEV), u.to(DEV), token, temperature=T.to(DEV))
    for r in range(6):
        want = int(u[r].item() * 777) if r in (0, 2) else int(ref[r].argmax())
        assert token[r].item() == want


# --------------------------------------------------------------------- the walk

def accept_ref(token, parent, sampled, P):
    path, node = [], 0 if len(token) else -1
    while node >= 0 and len(path) < P:
        path.append(node)
        t = sampled[node]
        node = next((c for c in range(node + 1, len(token)) if
                     (parent[c] if parent is not None else c - 1) == node and token[c] == t and t >= 0), -1)
    return path


@pytest.mark.parametrize("P", [1, 3, 8])
@pytest.mark.parametrize("kind", ["tree", "chain", "junk"])
@pytest.mark.parametrize("ns", [(1,), (65, 65, 65, 65, 65), (3, 0, 40, 1, 129), (700, 5)])
def test_accept(ns, kind, P):
    r = np.random.default_rng(sum(ns) + P)
    R = sum(ns)
    vocab = 3
    token = r.integers(0, vocab, R).astype(np.int32)
    sampled = r.integers(-1 if kind == "junk" else 0, vocab, R).astype(np.int32)
    parent = np.concatenate([np.array([-1] + [r.integers(max(0, i - 6), i) for i in range(1, n)])[:n]
                             for n in ns]).astype(np.int32)
    if kind == "junk":
        parent[r.random(R) < 0.3] = r.integers(-5, 1000)
    rows = np.concatenate([[0], np.cumsum(ns)]).astype(np.int32)
    B, N = len(ns), max(ns)
    up = lambda a: torch.from_numpy(a).to(DEV)  # noqa: E731
    i32 = dict(dtype=torch.int32, device=DEV)
    path, out, acc = torch.full((B, P), 9, **i32), torch.full((B, P), 9, **i32), torch.full((B,), 9, **i32)
    uniform = len(set(ns)) == 1
    M.moe_tree_accept(up(token), None if kind == "chain" else up(parent), up(sampled), B, N, path, acc,
                      out, row_start=None if uniform else up(rows))
    for b, n in enumerate(ns):
        s = slice(rows[b], rows[b + 1])
        want = accept_ref(token[s], None if kind == "chain" else parent[s], sampled[s], P)
        fill = [-1] * (P - len(want))
        assert path[b].tolist() == want + fill
        assert out[b].tolist() == [int(sampled[s][j]) for j in want] + fill
        assert acc[b].item() == len(want)


def test_accept_ranges_that_do_not_fit():
    i32 = dict(dtype=torch.int32, device=DEV)
    token = torch.zeros(6, **i32)
    rows = torch.tensor([0, 4, -3, 2, 900], **i32)
    path, acc = torch.empty(4, 9, **i32), torch.empty(4, **i32)
    M.moe_tree_accept(token, None, token, 4, 3, path, acc, row_start=rows)
    # 4 rows cut to N = 3; a range that ends before its start; one that starts before row 0; 898 rows
    # cut to 3 of the 4 that there are behind row 2
    assert acc.tolist() == [3, 0, 0, 3]


# --------------------------------------------------------------------- pages

class Book:
    """A book and a plain model of it."""

    def __init__(self, seed, B, width, n_pages, page, used=0.5):
        r = self.r = np.random.default_rng(seed)
        self.B, self.width, self.n, self.page = B, width, n_pages, page
        self.table = np.full((B, width), -5, np.int32)
        self.held, self.len = np.zeros(B, np.int32), np.zeros(B, np.int32)
        self.ref = np.zeros(n_pages, np.int32)
        free = list(r.permutation(n_pages)[:int(n_pages * used)])
        for b in range(B):
            c = min(int(r.integers(0, width + 1)), len(free))
            self.table[b, :c] = [free.pop() for _ in range(c)]
            self.ref[self.table[b, :c]] = 1
            self.held[b] = c
            self.len[b] = r.integers(0, c * page + 1)
        self.flags = 0
        self.dev = [torch.from_numpy(a.copy()).to(DEV) for a in (self.table, self.held, self.len, self.ref)]
        self.K = M.page_book(*self.dev, page)
        self.ws = M.pages_workspace(self.K)
        self.ws[4096:] = 255  # scratch holds anything

    def same(self):
        for name, t, a in zip(("table", "held", "len", "ref"), self.dev,
                              (self.table, self.held, self.len, self.ref)):
            got = t.cpu().numpy()
            assert np.array_equal(got, a), (name, np.argwhere(got != a)[:5], got[got != a][:5], a[got != a][:5])
        assert M.moe_workspace_check(self.ws) == self.flags
        self.flags = 0

    def free_pages(self):
        return [int(p) for p in np.flatnonzero(self.ref <= 0)]

    def sane(self, b):
        return 0 <= self.held[b] <= self.width and 0 <= self.len[b] <= int(self.held[b]) * self.page

    def reserve(self, n_new):
        each = isinstance(n_new, np.ndarray)
        M.moe_kv_reserve(self.K, 0 if each else n_new, self.ws,
                         n_new=torch.from_numpy(n_new).to(DEV) if each else None)
        free, short = self.free_pages(), False
        for b in range(self.B):
            more = int(n_new[b]) if each else n_new
            want = -(-(int(self.len[b]) + more) // self.page)
            if not self.sane(b) or more < 0 or want > self.width:
                self.flags |= 8
                continue
            need = max(0, want - int(self.held[b]))
            if need and (short or need > len(free)):
                short = True
                self.flags |= 16
                continue
            for _ in range(need):
                self.table[b, self.held[b]] = free.pop(0)
                self.ref[self.table[b, self.held[b]]] = 1
                self.held[b] += 1

    def free(self, seqs, keep=None):
        put = lambda v: None if v is None else torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
        M.moe_kv_free(self.K, put(seqs), self.ws, keep=put(keep))
        for i, b in enumerate(seqs):
            left = 0 if keep is None else keep[i]
            if not 0 <= b < self.B or left < 0:
                self.flags |= 8
                continue
            for j in range(-(-left // self.page), min(int(self.held[b]), self.width)):
                p = self.table[b, j]
                if 0 <= p < self.n and self.ref[p] > 0:
                    self.ref[p] -= 1
                else:
                    self.flags |= 4
            self.held[b] = min(self.held[b], -(-left // self.page))
            self.len[b] = min(self.len[b], left)

    def fork(self, src, dst):
        put = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
        moves = torch.full((len(src), 3), 77, dtype=torch.int32, device=DEV)
        M.moe_kv_fork(self.K, put(src), put(dst), moves, self.ws)
        want = np.full((len(src), 3), -1, np.int32)
        want[:, 2] = 0
        free = self.free_pages()
        first = {}
        for i, b in enumerate(dst):
            first.setdefault(b, i)
        held = self.held.copy()
        for i, (a, b) in enumerate(zip(src, dst)):
            if not (0 <= a < self.B and 0 <= b < self.B) or first[b] != i or a in first or held[b] or \
                    not self.sane(a):
                self.flags |= 8
                continue
            full, tail = divmod(int(self.len[a]), self.page)
            if tail and not free:
                self.flags |= 16
                continue
            self.table[b, :full] = self.table[a, :full]
            np.add.at(self.ref, self.table[a, :full], 1)
            if tail:
                p = free.pop(0)
                self.table[b, full] = p
                self.ref[p] = 1
                want[i] = self.table[a, full], p, tail
            self.held[b], self.len[b] = full + (tail > 0), self.len[a]
        assert np.array_equal(moves.cpu().numpy(), want)
        return moves

    def compact(self, in_place):
        out = self.dev[0] if in_place else torch.full_like(self.dev[0], 99)
        ref = self.dev[3] if in_place else torch.full_like(self.dev[3], 99)
        moves = torch.full((self.n // 2, 3), 77, dtype=torch.int32, device=DEV)
        counts = torch.full((2,), 77, dtype=torch.int32, device=DEV)
        M.moe_kv_compact(self.K, out, ref, moves, counts, self.ws)
        used = self.ref > 0
        n_used = int(used.sum())
        high = [p for p in range(n_used, self.n) if used[p]]
        hole = [p for p in range(n_used) if not used[p]]
        to = {int(p): int(p) for p in np.flatnonzero(used)} | dict(zip(high, hole))
        for b in range(self.B):
            for j in range(min(int(self.held[b]), self.width)):
                self.table[b, j] = to[int(self.table[b, j])]
        self.ref[hole] = self.ref[high]
        self.ref[high] = 0
        m = len(high)
        want = np.array([[p, q, self.page] for p, q in zip(high, hole)], np.int32).reshape(m, 3)
        assert counts.tolist() == [m, n_used]
        got = moves.cpu().numpy()
        assert np.array_equal(got[:m], want) and (got[m:] == 77).all()
        if not in_place:
            self.dev[0].copy_(out)
            self.dev[3].copy_(ref)
        return moves, counts


@pytest.mark.parametrize("B,width,n,page", [(1, 1, 1, 1), (3, 4, 7, 16), (40, 9, 300, 7),
                                            (300, 40, 9001, 64), (1100, 6, 5000, 16), (5, 900, 40000, 3)])
def test_pages_through_many_calls(B, width, n, page):
    k = Book(B + n, B, width, n, page)
    r = k.r
    for step in range(8):
        some = [int(b) for b in r.integers(0, B, max(1, B // 4))]  # with repeats
        k.free(some, None if step % 2 else [int(v) for v in r.integers(0, width * page + 1, len(some))])
        k.same()
        dst = [b for b in dict.fromkeys(some) if k.held[b] == 0]
        src = [b for b in range(B) if b not in dst]
        if dst and src:
            k.fork([int(s) for s in r.choice(src, len(dst))], dst)
            k.same()
        k.reserve(int(r.integers(0, 3 * page)) if step % 3 else
                  r.integers(0, 2 * page, B).astype(np.int32))
        k.same()
        k.len[:] = [r.integers(0, h * page + 1) for h in k.held]
        k.dev[2].copy_(torch.from_numpy(k.len))
        if step % 2:
            k.compact(in_place=step % 4 == 1)
            k.same()


def test_pages_refusals_and_shortage():
    k = Book(1, 8, 6, 24, 4, used=0.4)
    k.free(list(range(8)))
    k.same()
    k.free([-1, 8, 3, 1 << 30], [4, 4, -2, 0])
    k.same()
    k.reserve(np.array([24, 25, 16, 3, 0, 9, 1, 24], np.int32))  # 6 + refused + 4 + 1 + 0 + 3 + 1 + 6
    k.same()
    k.len[:] = [23, 0, 16, 2, 0, 9, 1, 24]
    k.dev[2].copy_(torch.from_numpy(k.len))
    k.reserve(2)  # sequence 1, 2, 4 need one each, 5 has room, 0 and 7 would need a seventh page
    k.same()
    k.free([1, 4, 6])
    k.same()
    # a target twice, one that holds pages, one that is a source, one outside, its own copy
    k.fork([5, 3, 5, 1, 5, 2], [1, 1, 2, 6, 8, 2])
    k.same()
    k.free([1, 4, 6])
    k.same()
    k.reserve(np.array([0, 0, 0, 0, 0, 0, 23, 0], np.int32))
    k.same()
    k.len[6] = 23
    k.dev[2].copy_(torch.from_numpy(k.len))
    k.fork([6, 5, 2], [1, 4, 1])
    k.same()
    # a sequence whose numbers do not fit is left alone
    k.held[3] = -4
    k.len[5] = 1000
    for i, a in ((1, k.held), (2, k.len)):
        k.dev[i].copy_(torch.from_numpy(a))
    k.reserve(1)
    k.same()


def test_pages_of_nobody():
    """Table entries outside the pool and pages that nobody held."""
    k = Book(4, 4, 5, 50, 8)
    k.free([0, 1, 2, 3])
    k.reserve(np.array([40, 40, 0, 0], np.int32))
    k.table[0, 1], k.table[0, 3] = -2, 50
    k.dev[0].copy_(torch.from_numpy(k.table))
    lost = int(k.table[1, 2])
    k.ref[lost] = 0
    k.dev[3].copy_(torch.from_numpy(k.ref))
    k.free([0, 1])
    k.same()


def _pools(layout, n, page, heads, dh, dt, seed):
    g = torch.Generator().manual_seed(seed)
    shape = dict(nhd=(n, page, heads, dh), hnd=(n, heads, page, dh), wide=(n, page, heads, dh + 8),
                 both=(n, 2, page, heads, dh))[layout]
    out = []
    for _ in range(2):
        t = torch.randn(*shape, generator=g).to(dt).to(DEV)
        if layout == "hnd":
            t = t.permute(0, 2, 1, 3)
        elif layout == "wide":
            t = t[..., :dh]
        elif layout == "both":
            t = t[:, 1]
        out.append(t)
    return out


@pytest.mark.parametrize("layout", ["nhd", "hnd", "wide", "both"])
@pytest.mark.parametrize("page,heads,dh,dt", [(16, 4, 128, torch.bfloat16), (7, 3, 8, torch.bfloat16),
                                              (64, 8, 64, torch.float32), (1, 1, 72, torch.bfloat16)])
def test_copy_pages(layout, page, heads, dh, dt):
    n = 90
    kp, vp = _pools(layout, n, page, heads, dh, dt, page)
    r = np.random.default_rng(page)
    order = r.permutation(n)
    m = 40
    moves = np.stack([order[:m], order[m:2 * m], r.integers(0, page + 1, m)], 1).astype(np.int32)
    moves[3, 2] = page + 1                      # refused
    moves[4, 0], moves[5, 1] = n, -1            # refused
    moves[6, 2] = -1                            # nothing
    moves[7, 1] = moves[7, 0]                   # nothing
    moves[8, 2] = page
    want = [kp.clone(), vp.clone()]
    C = M.cache_desc(kp, heads, 4)
    count = torch.tensor([m - 5, 0], dtype=torch.int32, device=DEV)
    for s, d, t in moves[:m - 5]:
        if 0 <= s < n and 0 <= d < n and 0 < t <= page:
            for p in want:
                p[d, :t] = p[s, :t].clone()
    ws = torch.zeros(4096, dtype=torch.uint8, device=DEV)
    M.moe_kv_copy_pages(C, kp, vp, torch.from_numpy(moves).to(DEV), count=count, ws=ws)
    assert torch.equal(kp, want[0]) and torch.equal(vp, want[1])
    assert M.moe_workspace_check(ws) == 4
    count.fill_(1 << 30)  # more than the list has
    for s, d, t in moves:
        if 0 <= s < n and 0 <= d < n and 0 < t <= page:
            for p in want:
                p[d, :t] = p[s, :t].clone()
    M.moe_kv_copy_pages(C, kp, vp, torch.from_numpy(moves).to(DEV), count=count)
    assert torch.equal(kp, want[0]) and torch.equal(vp, want[1])
    count.fill_(-3)
    M.moe_kv_copy_pages(C, kp, vp, torch.from_numpy(moves).to(DEV), count=count)
    assert torch.equal(kp, want[0])


# ---------------------------------------------- where numbers do not fit, and sizes at the ends

@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("size", [1e20, 1.8422e19])
def test_few_activations_at_the_end_of_the_range(dt, size):
    """An activation beyond fp32 gives infinities of the signs of W_down's rows; one between bf16's and
    fp32's largest is held by its value and rest (both signs of it, so that y is finite)."""
    R, d, E, k, f = 3, 64, 4, 1, 32
    t = Few(19, R, d, E, k, f, dt)
    t.x = torch.ones(R, d, dtype=dt)
    t.wg[:, 3], t.wu[:, 3] = 0, 0
    t.wg[:, 3, 5] = t.wu[:, 3, 7] = size
    t.wd[t.wd == 0] = 1
    big = float(t.wg[0, 3, 5]) * float(t.wu[0, 3, 7])
    if size < 1e20:
        # the product at row 3 lies above bf16's largest value's upper half step, below fp32's
        t.wu[:, 3, 7] = 1.8446744073709552e19
        t.wg[:, 3, 5], t.wg[:, 3, 6] = 1.8374686479671624e19, 4e16  # 255 2^56, and a little
        big = (float(t.wg[0, 3, 5]) + float(t.wg[0, 3, 6])) * 2.0 ** 64
        assert 3.3961775e38 < big < 3.4028e38
        t.wd[:, :, 3] = t.wd[:, :, 3].sign() * 2.0 ** -20
    t.upload().run()
    y = t.y.cpu().double()
    for r in range(R):
        e = int(t.idx[r, 0])
        if size < 1e20:
            want = big * t.wd[e, :, 3].double()
            tol = (U[dt] + 2.0 ** -16) * want.abs()  # (what the other activations add is far below)
            assert ((y[r] - want).abs() <= tol).all()
        else:
            assert torch.equal(y[r], t.wd[e, :, 3].double().sign() * math.inf)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("ctas", [1, 2, 151])
def test_few_on_any_number_of_ctas(dt, ctas):
    t = Few(23, 11, 2888, 9, 3, 200, dt).upload().run(True, True, max_ctas=ctas)
    t.check(True, True)


def test_pages_of_sequences_whose_numbers_do_not_fit():
    """They are left as they are and told, whichever call meets them, also beside others of the list."""
    k = Book(31, 12, 5, 90, 8)
    k.free(list(range(12)))
    k.reserve(20)
    k.same()
    k.held[1], k.held[2], k.len[3], k.len[4] = -3, 6, 25, -1  # (three pages of 8 each)
    k.len[5:] = [24, 17, 16, 9, 1, 0, 8]
    for i, a in ((1, k.held), (2, k.len)):
        k.dev[i].copy_(torch.from_numpy(a))
    odd = [1, 2, 3, 4]
    saved = k.held[odd].copy(), k.len[odd].copy(), k.ref.copy()
    put = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    M.moe_kv_free(k.K, put(odd), k.ws)
    M.moe_kv_free(k.K, put(odd + odd), k.ws, keep=put([8, 8, 8, 8, 0, 30, 0, 5]))
    k.flags = 8
    k.same()
    # the same sequence many times, in any order: the smallest keep holds
    lists = [5, 6] * 40
    keeps = [int(v) for v in np.random.default_rng(3).integers(3, 25, 80)]
    k.free(lists, keeps)
    k.same()
    assert np.array_equal(saved[0], k.held[odd]) and np.array_equal(saved[1], k.len[odd])


def test_copy_pages_past_4_gb():
    n, page, heads, dh = 40000, 64, 8, 128  # 5.2 GB a pool
    kp = torch.empty(n, page, heads, dh, dtype=torch.bfloat16, device=DEV)
    vp = torch.empty(n, heads, page, dh, dtype=torch.bfloat16, device=DEV).permute(0, 2, 1, 3)
    for p in (kp, vp):
        C = M.cache_desc(p, heads, 4)
        p[n - 1].normal_()
        p[3].fill_(7)
        p[n - 2].fill_(5)
        want = p[n - 1].clone()
        M.moe_kv_copy_pages(C, p, p, torch.tensor([[n - 1, 3, 64], [n - 1, n - 2, 9]], dtype=torch.int32, device=DEV))
        assert torch.equal(p[3], want) and torch.equal(p[n - 1], want)
        assert torch.equal(p[n - 2, :9], want[:9]) and bool((p[n - 2, 9:] == 5).all())


@pytest.mark.parametrize("B,n,page", [(1500, 700, 5), (2300, 900, 16), (700, 256, 4), (700, 257, 4)])
def test_pages_of_many_sequences(B, n, page):
    """More forks than a thread block keeps, more sequences than it has threads, entries that are refused
    among them, and too few pages for the last."""
    k = Book(B, B, 30, 9 * B, page, used=0.2)
    r = k.r
    k.free(list(range(0, B, 2)))
    k.same()
    empty = [b for b in range(B) if k.held[b] == 0]
    full = [b for b in range(B) if k.held[b]]
    dst = [int(v) for v in r.choice(empty, n)]  # with repeats
    src = [int(v) for v in r.choice(full, n)]
    for i in r.integers(0, n, 12):
        src[i] = int(r.choice([-1, B, dst[0], 1 << 30]))
        dst[(i + 5) % n] = int(r.choice([-7, B, full[0]]))
    k.fork(src, dst)
    k.same()
    k.reserve(r.integers(0, 25 * page, B).astype(np.int32))  # more than there are
    k.same()
    k.reserve(1)
    k.same()
