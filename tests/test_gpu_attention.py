"""GPU tests of the attention half of the block (moe_tree_attention, moe_kv_append, moe_kv_commit,
moe_block_norm) against plain 64-bit computations.

Attention's tolerance, per output element, from the roundings it is allowed (u = half a step of
the type: 2^-8 bf16, 2^-24 fp32; A = sum_j p_j |v_j| with the exact p):
  * output rounding: u |out|;
  * bf16 only: the second product's p rounded to bf16, 2^-8 relative each: 2^-8 A;
  * scores: dh + 8 fp32 roundings of terms up to |q|.|k|, so e_s = (dh + 8) 2^-24 max_j |q|.|k_j|
    scale absolute, a relative 2 e_s in each p (numerator and denominator): 2 e_s A;
  * exp2 and the logit arithmetic: 2^-20 (1 + max |s|) A; sums over K slots: K 2^-24 A.
Nothing of the sequences' unused slots and pages may be read into a result: they hold NaN.
"""
import math

import numpy as np
import pytest
import torch

from expert_select_gb300 import moetree as M
from expert_select_gb300 import workload as W

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


class Block:
    """A block of new nodes over a paged cache, on the CPU, and its upload."""

    def __init__(self, seed, dtype=torch.bfloat16, H=8, Hkv=2, dh=64, page=16, layout="nhd",
                 lens=(37,), ns=(9,), kind="chain", window=0, sinks=0, logit=False, pad_rows=0,
                 depth_max=6, qscale=1.5, wide=0, spare=0):
        g = torch.Generator().manual_seed(seed)
        r = np.random.default_rng(seed)
        self.dtype, self.H, self.Hkv, self.dh, self.page = dtype, H, Hkv, dh, page
        self.lens, self.ns, self.window, self.sinks = list(lens), list(ns), window, sinks
        self.B, self.N = len(lens), max(ns)
        self.rows = np.concatenate([[0], np.cumsum(ns)]).astype(int)
        self.R = int(self.rows[-1]) + pad_rows
        self.ragged = pad_rows > 0 or len(set(ns)) > 1
        need = [-(-(l + n) // page) for l, n in zip(lens, ns)]
        self.n_pages, self.max_pages = sum(need) + 2, max(max(need), 1) + 1 + spare
        order = r.permutation(self.n_pages)
        self.table = np.full((self.B, self.max_pages), -7, np.int32)  # never read past the end
        at = 0
        for b, c in enumerate(need):
            self.table[b, :c] = order[at:at + c]
            at += c
        nan = float("nan")
        shape = (self.n_pages, page, Hkv, dh)
        self.k, self.v = torch.full(shape, nan).to(dtype), torch.full(shape, nan).to(dtype)
        for b in range(self.B):
            j = np.arange(lens[b] + ns[b])
            at_ = (torch.from_numpy(self.table[b, j // page].astype(np.int64)),
                   torch.from_numpy(j % page))
            self.k[at_] = torch.randn(len(j), Hkv, dh, generator=g).to(dtype)
            self.v[at_] = torch.randn(len(j), Hkv, dh, generator=g).to(dtype)
        self.q = (torch.randn(self.R, H, dh, generator=g) * qscale).to(dtype)
        self.layout, self.wide = layout, wide
        self.parent = None
        if kind != "chain":
            ps = []
            for n in ns:
                p = np.full(n, -1, np.int32)
                d = np.zeros(n, int)
                for i in range(1, n):
                    if kind == "deep":
                        p[i] = i - 1
                    elif kind == "forest":
                        p[i] = -1 if r.random() < 0.2 else r.integers(0, i)
                    else:
                        p[i] = r.integers(0, i)
                        while d[p[i]] >= depth_max:
                            p[i] = p[p[i]]
                        d[i] = d[p[i]] + 1
                ps.append(p)
            self.parent = np.concatenate(ps + [np.zeros(pad_rows, np.int32)]).astype(np.int32)
        self.logit = torch.randn(H, generator=g) * 2 if logit else None

    def upload(self):
        def pool(t):
            if self.layout == "hnd":
                return t.permute(0, 2, 1, 3).contiguous().to(DEV).permute(0, 2, 1, 3)
            return t.to(DEV)
        self.kd, self.vd = pool(self.k), pool(self.v)
        if self.wide:  # q as a part of wider rows
            buf = torch.zeros(self.R, self.H + self.wide, self.dh, dtype=self.dtype, device=DEV)
            buf[:, :self.H] = self.q.to(DEV)
            self.qd = buf[:, :self.H]
        else:
            self.qd = self.q.to(DEV)
        self.tabled = torch.from_numpy(self.table).to(DEV)
        self.lend = torch.tensor(self.lens, dtype=torch.int32, device=DEV)
        self.startd = (torch.from_numpy(self.rows.astype(np.int32)).to(DEV) if self.ragged
                       else None)
        self.parentd = None if self.parent is None else torch.from_numpy(self.parent).to(DEV)
        self.logitd = None if self.logit is None else self.logit.to(DEV)
        self.C = M.cache_desc(self.kd, self.H, self.max_pages, window=self.window,
                              sink_tokens=self.sinks)
        self.ws = M.attention_workspace(self.C, self.B, self.N)
        self.out = torch.full((self.R, self.H, self.dh), 7.25, dtype=self.dtype, device=DEV)
        self.lse = torch.full((self.R, self.H), 7.25, device=DEV)
        return self

    def attend(self):
        M.moe_tree_attention(self.C, self.qd, self.kd, self.vd, self.tabled, self.lend, self.B,
                             self.N, self.out, self.ws, parent=self.parentd,
                             row_start=self.startd, sink_logit=self.logitd, lse=self.lse)
        return self

    def visible(self, b):
        """[n, len + n] from the definition."""
        ln, n = self.lens[b], self.ns[b]
        see = np.zeros((n, ln + n), bool)
        depth = np.zeros(n, int)
        for i in range(n):
            if self.parent is None:
                see[i, :ln + i + 1] = True
                depth[i] = i
            else:
                p = self.parent[self.rows[b] + i]
                see[i, :ln] = True
                if 0 <= p < i:
                    see[i] |= see[p]
                    depth[i] = depth[p] + 1
                see[i, ln + i] = True
        if self.window:
            kpos = np.concatenate([np.arange(ln), ln + depth])
            qpos = (ln + depth)[:, None]
            see &= (qpos - kpos[None] < self.window) | (kpos < self.sinks)[None]
        return see

    def reference(self):
        """out, lse and the tolerance of out, in 64 bits; rows of no sequence are NaN."""
        f64 = torch.float64
        out = torch.full((self.R, self.H, self.dh), math.nan, dtype=f64)
        tol = torch.full_like(out, math.nan)
        lse = torch.full((self.R, self.H), math.nan, dtype=f64)
        scale, G, u = self.dh ** -0.5, self.H // self.Hkv, U[self.dtype]
        for b in range(self.B):
            ln, n, r0 = self.lens[b], self.ns[b], self.rows[b]
            if n == 0:
                continue
            L = ln + n
            idx = np.arange(L)
            pg = torch.from_numpy(self.table[b, idx // self.page].astype(np.int64))
            k = self.k[pg, torch.from_numpy(idx % self.page)].to(f64)
            v = self.v[pg, torch.from_numpy(idx % self.page)].to(f64)
            see = torch.from_numpy(self.visible(b))
            for h in range(self.H):
                q = self.q[r0:r0 + n, h].to(f64)
                s = (q @ k[:, h // G].T) * scale
                mag = ((q.abs() @ k[:, h // G].abs().T) * scale).masked_fill(~see, 0).amax(1)
                s = s.masked_fill(~see, -math.inf)
                top = s.abs().masked_fill(~see, 0).amax(1)
                z = s
                if self.logit is not None:
                    z = torch.cat([s, self.logit[h].to(f64).expand(n, 1)], 1)
                lse[r0:r0 + n, h] = torch.logsumexp(z, 1)
                p = torch.exp(s - lse[r0:r0 + n, h, None])
                vv = v[:, h // G]
                # a slot takes part only in rows that see it, whatever it holds
                o = torch.stack([p[i, see[i]] @ vv[see[i]] for i in range(n)])
                A = torch.stack([p[i, see[i]] @ vv[see[i]].abs() for i in range(n)])
                out[r0:r0 + n, h] = o
                rel = 2 * (self.dh + 8) * 2.0 ** -24 * mag + 2.0 ** -20 * (1 + top) + L * 2.0 ** -24
                if self.dtype == torch.bfloat16:
                    rel = rel + 2.0 ** -8
                tol[r0:r0 + n, h] = rel[:, None] * A + u * o.abs() + 1e-30
        return out, lse, tol

    def check(self):
        torch.cuda.synchronize()
        assert M.moe_workspace_check(self.ws) == 0
        out, lse, tol = self.reference()
        n = int(self.rows[-1])
        got, gl = self.out.double().cpu(), self.lse.double().cpu()
        err = (got[:n] - out[:n]).abs() - tol[:n]
        assert torch.isfinite(got[:n]).all()
        assert (err <= 0).all(), (err.max(), np.argwhere((err > 0).numpy())[:5])
        assert ((gl[:n] - lse[:n]).abs() <= 1e-4 + 1e-5 * lse[:n].abs()).all()
        # rows behind the last sequence are left as they were
        assert (got[n:] == 7.25).all() and (gl[n:] == 7.25).all()
        return self


BF, F32 = torch.bfloat16, torch.float32
CASES = [
    dict(),
    dict(lens=(0,), ns=(1,)),
    dict(lens=(1,), ns=(1,), page=1),
    dict(lens=(0, 5, 300), ns=(1, 1, 1), dh=128),
    dict(lens=(130,), ns=(1,), H=1, Hkv=1, dh=128),
    dict(lens=(127, 128, 129, 255), ns=(1, 1, 1, 1), dh=128, H=32, Hkv=4),
    dict(lens=(5000,), ns=(1,), dh=128, H=32, Hkv=4, page=64),
    dict(lens=(9001, 17), ns=(1, 1), dh=64, H=64, Hkv=8, page=32, layout="hnd"),
    dict(lens=(700,), ns=(65,), kind="tree", dh=128, H=32, Hkv=4),
    dict(lens=(0, 63, 2000), ns=(65, 65, 65), kind="tree", dh=128, H=16, Hkv=2, layout="hnd"),
    dict(lens=(250, 3), ns=(40, 17), kind="tree", H=8, Hkv=8, dh=128),
    dict(lens=(77,), ns=(300,), kind="deep", H=2, Hkv=2),
    dict(lens=(77,), ns=(200,), kind="forest", H=6, Hkv=2, page=24),
    dict(lens=(0,), ns=(257,), dh=128, H=4, Hkv=1),
    dict(lens=(1000, 0, 333), ns=(130, 260, 1), dh=128, H=8, Hkv=1, page=64),
    dict(lens=(500, 20, 90), ns=(0, 33, 0), pad_rows=5),
    dict(lens=(60, 20, 90), ns=(31, 0, 64), pad_rows=3, kind="tree", H=5, Hkv=1, dh=128),
    dict(lens=(513,), ns=(50,), H=7, Hkv=1, dh=128, page=7),
    dict(lens=(513, 100), ns=(50, 12), H=14, Hkv=2, dh=80, page=20, kind="tree"),
    dict(lens=(400,), ns=(20,), dh=8, H=4, Hkv=2, page=3),
    dict(lens=(400,), ns=(20,), dh=96, H=4, Hkv=2, page=128),
    dict(lens=(400,), ns=(20,), dh=136, H=4, Hkv=2, page=5),
    dict(lens=(300,), ns=(33,), dh=256, H=4, Hkv=2, kind="tree"),
    dict(lens=(400,), ns=(20,), dh=72, H=4, Hkv=2, page=200, wide=3),
    # windows, first tokens, sink logits
    dict(lens=(1000, 3, 130), ns=(1, 1, 1), window=128, sinks=4, logit=True, H=64, Hkv=8),
    dict(lens=(1000,), ns=(1,), window=1, dh=128),
    dict(lens=(1000,), ns=(1,), window=1, sinks=1, dh=128),
    dict(lens=(300,), ns=(300,), window=100, sinks=0, dh=128, H=4, Hkv=1),
    dict(lens=(700,), ns=(300,), window=100, sinks=130, dh=64, H=4, Hkv=1),
    dict(lens=(20,), ns=(30,), window=200, sinks=300, logit=True),
    dict(lens=(900, 50), ns=(65, 65), window=60, sinks=3, kind="tree", dh=128, H=16, Hkv=2),
    dict(lens=(40,), ns=(150,), window=30, sinks=2, kind="deep"),
    dict(lens=(40,), ns=(90,), window=3, sinks=41, kind="tree", logit=True),
    dict(lens=(0,), ns=(70,), window=2, sinks=1, kind="tree"),
    # few rows of several nodes
    dict(lens=(100, 0, 31), ns=(8, 8, 8), kind="tree", H=4, Hkv=2, dh=128),
    dict(lens=(100, 7), ns=(16, 3), H=2, Hkv=2, page=5),
    dict(lens=(300, 64), ns=(4, 4), H=8, Hkv=2, dh=80, window=37, sinks=2, kind="deep", logit=True),
    dict(lens=(20000,), ns=(2,), H=16, Hkv=2, dh=128, page=64),
]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(f"{k}{v}" for k, v in c.items())
                         .replace(" ", "") or "default")
def test_attention_matches_64_bits(case, dtype):
    Block(len(str(case)), dtype, **case).upload().attend().check()


# which kernel takes more than 16 rows of few blocks depends on the page table's capacity: the same
# blocks with a table of 2^17 more slots, and more blocks that are small enough for the other one
@pytest.mark.parametrize("case", [c for c in CASES if max(c.get("ns", (9,))) * c.get("H", 8)
                                  // c.get("Hkv", 2) > 16 and c.get("dh", 64) <= 128],
                         ids=lambda c: "-".join(f"{k}{v}" for k, v in c.items())
                         .replace(" ", "") or "default")
def test_wide_page_tables_match_64_bits(case):
    Block(len(str(case)), BF, spare=(1 << 17) // case.get("page", 16), **case).upload().attend() \
        .check()


@pytest.mark.parametrize("case", [
    dict(lens=(1500,), ns=(9,), kind="tree", dh=128, H=32, Hkv=4),
    dict(lens=(70,), ns=(16,), kind="tree", H=32, Hkv=4, page=8, layout="hnd"),
    dict(lens=(0,), ns=(128,), kind="deep", H=4, Hkv=2, dh=128),
    dict(lens=(33,), ns=(512,), H=1, Hkv=1, dh=128, page=64),
    dict(lens=(333,), ns=(70,), kind="forest", H=7, Hkv=1, dh=80, page=7),
    dict(lens=(333, 9, 61), ns=(20, 0, 11), kind="tree", H=3, Hkv=1, pad_rows=3, dh=128),
    dict(lens=(3000, 16), ns=(1, 16), H=16, Hkv=2, dh=128, page=64),
    dict(lens=(4000,), ns=(16,), H=32, Hkv=4, window=128, sinks=4, logit=True),
    dict(lens=(300, 90), ns=(24, 10), kind="tree", H=10, Hkv=2, window=3, sinks=2, dh=128),
    dict(lens=(25,), ns=(100,), kind="deep", H=4, Hkv=1, window=40, sinks=30, wide=2),
], ids=lambda c: "-".join(f"{k}{v}" for k, v in c.items()).replace(" ", ""))
@pytest.mark.parametrize("copies", [1, 12])
def test_blocks_of_some_rows_match_64_bits(case, copies):
    """One copy is few blocks of 16 rows, twelve are many."""
    many = {**case, "lens": case["lens"] * copies, "ns": case["ns"] * copies}
    Block(len(str(case)), BF, **many).upload().attend().check()


@pytest.mark.parametrize("dtype,n", [(BF, 1), (BF, 5), (F32, 2)])
def test_more_sequences_than_a_block_has_threads(dtype, n):
    r = np.random.default_rng(n)
    lens = tuple(int(v) for v in np.where(r.random(520) < 0.9, r.integers(0, 60, 520),
                                          r.integers(60, 900, 520)))
    Block(80 + n, dtype, lens=lens, ns=(n,) * 520, H=4, Hkv=1, page=8).upload().attend().check()


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_chunks_and_single_tokens_in_one_block(dtype):
    """A batch of a few prompt chunks among many single tokens and empty sequences."""
    r = np.random.default_rng(5)
    ns = [1] * 60
    ns[7], ns[31], ns[32], ns[59] = 300, 0, 77, 130
    lens = tuple(int(v) for v in r.integers(0, 400, 60))
    Block(90, dtype, lens=lens, ns=tuple(ns), H=8, Hkv=2, page=16, pad_rows=2).upload().attend() \
        .check()


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("kind,dh,ns", [("tree", 128, (70, 33)), ("chain", 64, (70, 33)),
                                        ("tree", 136, (70, 33)), ("tree", 128, (4, 3)),
                                        ("tree", 128, (9, 7)), ("chain", 64, (20, 21)),
                                        ("chain", 64, (3, 4)), ("chain", 256, (2, 3)),
                                        ("chain", 128, (1, 1))])
def test_masked_infinities_and_nan_take_no_part(dtype, kind, dh, ns):
    """A node's keys and values hold NaN and infinities: rows that do not see it are what they
    would be without it, rows that do see it are not finite."""
    blk = Block(5, dtype, lens=(200, 30), ns=ns, kind=kind, dh=dh, H=8, Hkv=2)
    blk.upload().attend().check()
    want = blk.out.clone()
    bad = {0: (ns[0] * 4 // 7, "v"), 1: (ns[1] * 20 // 33, "k")}
    for b, (m, which) in bad.items():
        j = blk.lens[b] + m
        t = (blk.vd if which == "v" else blk.kd)[int(blk.table[b, j // blk.page]), j % blk.page]
        t[0] = float("nan")
        t[1] = float("inf") if which == "v" else float("nan")
        if which == "v":
            t[1, ::2] = -float("inf")
    blk.attend()
    torch.cuda.synchronize()
    G = blk.H // blk.Hkv
    for b, (m, which) in bad.items():
        see = blk.visible(b)[:, blk.lens[b] + m]
        rows = torch.from_numpy(np.flatnonzero(~see) + blk.rows[b]).to(DEV)
        assert torch.equal(blk.out[rows], want[rows])
        hit = blk.out[torch.from_numpy(np.flatnonzero(see) + blk.rows[b]).to(DEV)].float()
        assert len(hit) and torch.isnan(hit[:, :G]).all()
        if which == "v":
            assert (hit[:, G:, 0::2] == -math.inf).all() and (hit[:, G:, 1::2] == math.inf).all()
        else:
            assert torch.isnan(hit).all()


@pytest.mark.parametrize("dtype,dh", [(BF, 128), (BF, 256), (F32, 64)])
def test_a_part_of_only_nan_scores_is_not_lost(dtype, dh):
    """A long item is cut between CTAs; the part that holds the last slots sees one key, of NaN:
    its running maximum never rises, and its sum is NaN."""
    for ln in (4096, 8192, 12352):  # whole tiles of committed slots before the node's own
        blk = Block(12, dtype, lens=(ln,), ns=(1,), dh=dh, H=4, Hkv=1, page=64).upload()
        blk.attend().check()
        blk.kd[int(blk.table[0, ln // 64]), ln % 64] = float("nan")
        blk.attend()
        assert torch.isnan(blk.out).all()


def test_nothing_visible_gives_zeros():
    """A window that ends before the page table does: rows whose own slot does not fit see
    nothing (and the check word says so)."""
    blk = Block(3, lens=(16,), ns=(2,), page=4, H=4, Hkv=1, window=1).upload()
    blk.lend[0] = blk.max_pages * blk.page - 1  # the second node's slot is past the table
    blk.tabled[:] = blk.tabled[0, 0]
    blk.kd[:] = 1
    blk.vd[:] = 2
    blk.attend()
    torch.cuda.synchronize()
    assert M.moe_workspace_check(blk.ws) == 8
    assert (blk.out[0] == 2).all() and (blk.out[1] == 0).all()
    assert torch.isinf(blk.lse[1]).all()


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_bad_pages_and_lengths_are_flagged_and_not_read(dtype):
    blk = Block(4, dtype, lens=(100, 50), ns=(5, 5), H=8, Hkv=2, dh=128).upload()
    blk.attend().check()
    # a page outside the pool: its slots are not seen
    t = blk.table.copy()
    for bad in (-1, blk.n_pages, 1 << 30):
        blk.tabled[0, 2] = bad
        blk.attend()
        torch.cuda.synchronize()
        assert M.moe_workspace_check(blk.ws) == 4
        assert M.moe_workspace_check(blk.ws) == 0
        keep = [j for j in range(105) if j // 16 != 2]
        idx = torch.tensor(keep)
        k = blk.k[torch.from_numpy(t[0][idx // 16].astype(int)), idx % 16].double()
        v = blk.v[torch.from_numpy(t[0][idx // 16].astype(int)), idx % 16].double()
        s = torch.einsum("hd,jd->hj", blk.q[4, :4].double(), k[:, 0]) * 128 ** -0.5
        want = torch.softmax(s, 1) @ v[:, 0]
        assert ((blk.out[4, :4].double().cpu() - want).abs() <= 0.02).all()
    blk.tabled.copy_(torch.from_numpy(t))
    for bad in (-3, 1 << 30):
        blk.lend[1] = bad
        blk.tabled[1] = blk.tabled[1, 0]
        blk.attend()
        torch.cuda.synchronize()
        assert M.moe_workspace_check(blk.ws) & 8
        assert torch.equal(blk.out[:5].isfinite().all(), torch.tensor(True, device=DEV))


def test_row_ranges_that_do_not_fit_are_cut():
    blk = Block(6, lens=(40, 50, 60), ns=(4, 9, 2), H=8, Hkv=2).upload()
    blk.attend().check()
    want = blk.out.clone()
    blk.startd.copy_(torch.tensor([0, 4, 13, 1000], dtype=torch.int32))  # past R
    blk.attend()
    torch.cuda.synchronize()
    assert M.moe_workspace_check(blk.ws) == 8
    assert torch.equal(blk.out[:13], want[:13])
    blk.startd.copy_(torch.tensor([0, 4, 3, 15], dtype=torch.int32))     # not ascending
    blk.attend()
    torch.cuda.synchronize()
    # the last sequence now has 9 (cut from 12) nodes in slots 60 .. 68, and the page of slots
    # 64 .. 79 is past the end of its table row's valid entries: bit 2 too
    assert M.moe_workspace_check(blk.ws) == 12
    assert torch.equal(blk.out[:3], want[:3])


def test_attention_repeats_bit_for_bit():
    blk = Block(7, lens=(3000, 10, 700), ns=(65, 65, 65), kind="tree", dh=128, H=16, Hkv=2).upload()
    blk.attend()
    first, lse = blk.out.clone(), blk.lse.clone()
    for _ in range(5):
        blk.attend()
        assert torch.equal(blk.out, first) and torch.equal(blk.lse, lse)


@pytest.mark.parametrize("dtype,dh,kind,ns", [(BF, 128, "chain", (1, 1)), (BF, 64, "tree", (33, 33)),
                                             (BF, 128, "chain", (140, 140)),
                                             (F32, 64, "tree", (9, 9))])
def test_attention_in_a_graph_follows_new_lengths_and_tables(dtype, dh, kind, ns):
    """A captured call is replayed after the lengths, the table and q have changed, on another
    stream than the capture's."""
    big = Block(9, dtype, lens=(2000, 700), ns=ns, kind=kind, dh=dh, H=16, Hkv=2, page=8).upload()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        big.attend()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        big.attend()
    big.out.zero_()
    g.replay()
    big.check()
    # other contents
    big.lens, big.lend[:] = [1300, 699], torch.tensor([1300, 699], dtype=torch.int32, device=DEV)
    perm = np.random.default_rng(0).permutation(big.n_pages)
    inv = np.argsort(perm)
    big.k, big.v = big.k[torch.from_numpy(perm)], big.v[torch.from_numpy(perm)]
    used = big.table >= 0
    big.table[used] = inv[big.table[used]]
    big.kd.copy_(big.k)
    big.vd.copy_(big.v)
    big.tabled.copy_(torch.from_numpy(big.table))
    big.q = torch.randn_like(big.q)
    big.qd.copy_(big.q)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        g.replay()
    torch.cuda.current_stream().wait_stream(side)
    big.check()


def test_attention_on_two_streams_at_once():
    """Calls that overlap in time, each with its own workspace, on streams given explicitly."""
    blocks = [Block(60 + i, **c).upload() for i, c in enumerate([
        dict(lens=(6000, 9000), ns=(65, 65), kind="tree", dh=128, H=16, Hkv=2),
        dict(lens=(12000,), ns=(300,), dh=64, H=8, Hkv=2),
        dict(lens=(20000, 3), ns=(1, 1), dh=128, H=16, Hkv=2)])]
    streams = [torch.cuda.Stream() for _ in blocks]
    torch.cuda.synchronize()
    for _ in range(4):
        for b, s in zip(blocks, streams):
            M.moe_tree_attention(b.C, b.qd, b.kd, b.vd, b.tabled, b.lend, b.B, b.N, b.out, b.ws,
                                 parent=b.parentd, row_start=b.startd, lse=b.lse, stream=s)
    for b in blocks:
        b.check()


@pytest.mark.parametrize("N", [1, 2, 16, 17, 65])
@pytest.mark.parametrize("spare", [0, 1 << 13])
def test_single_rows_do_not_depend_on_the_kernel(N, spare):
    """The same query node as the last of a chain of N: the kernels for few and for many rows give
    the same output up to the roundings of one of them each."""
    shape = dict(lens=(700,), ns=(N,), dh=128, H=8, Hkv=1, spare=spare)
    blk = Block(70, **shape).upload().attend().check()
    last = Block(70, **shape).upload()
    one = torch.empty(1, 8, 128, dtype=BF, device=DEV)
    M.moe_tree_attention(last.C, last.qd[N - 1:], last.kd, last.vd, last.tabled,
                         last.lend + (N - 1), 1, 1, one, last.ws)
    _, _, tol = blk.reference()
    diff = (one.double().cpu()[0] - blk.out.double().cpu()[N - 1]).abs()
    assert (diff <= 2 * tol[N - 1]).all()


def test_one_workspace_serves_blocks_of_any_shape():
    """Calls in a row on one stream, of other shapes and kernels, share a workspace that the
    largest of them sized."""
    blocks = [Block(20 + i, **c).upload() for i, c in enumerate([
        dict(lens=(4000,), ns=(65,), kind="tree", dh=128, H=32, Hkv=4),
        dict(lens=(3, 900), ns=(1, 1), dh=64),
        dict(lens=(300,), ns=(20,), dh=256),
        dict(lens=(2000, 5), ns=(1, 1), dh=128, H=32, Hkv=4)])]
    ws = max((b.ws for b in blocks), key=lambda w: w.numel())
    for _ in range(2):
        for b in blocks:
            b.ws = ws
            b.out.fill_(float("nan"))
            b.attend()
    for b in blocks:
        b.check()


def test_far_slots_of_a_large_pool():
    """Pages whose byte offsets pass 32 bits."""
    dh, page, Hkv = 128, 64, 4
    n_pages = (5 << 30) // (page * Hkv * dh * 2)  # 5 GiB a pool
    kd = torch.zeros(n_pages, page, Hkv, dh, dtype=BF, device=DEV)
    vd = torch.zeros_like(kd)
    blk = Block(11, lens=(500,), ns=(3,), dh=dh, H=8, Hkv=Hkv, page=page).upload()
    used = blk.table[0][blk.table[0] >= 0]
    far = [n_pages - 1 - 3 * i for i in range(len(used))]
    for u, f in zip(used, far):
        kd[f], vd[f] = blk.kd[int(u)], blk.vd[int(u)]
    blk.tabled[0, :len(far)] = torch.tensor(far, dtype=torch.int32)
    blk.kd, blk.vd = kd, vd
    blk.C = M.cache_desc(kd, blk.H, blk.max_pages)
    blk.attend().check()


# ------------------------------------------------------------------------------ append

def _angles(pos, freq):
    a = pos.astype(np.float64)[:, None] * freq.astype(np.float64)[None]
    return np.cos(a), np.sin(a)


APPEND = [
    dict(lens=(37, 0), ns=(9, 9), rot=64, norm=True),
    dict(lens=(1000000 - 20,), ns=(5,), rot=64, norm=False, page=4096),
    dict(lens=(5, 300, 8), ns=(1, 0, 130), rot=32, norm=True, pad_rows=4),
    dict(lens=(60,), ns=(65,), rot=128, norm=True, dh=128, H=32, Hkv=4, kind="tree"),
    dict(lens=(60,), ns=(3,), rot=0, norm=False, dh=8, H=4, Hkv=4, page=1),
    dict(lens=(60,), ns=(3,), rot=0, norm=True, dh=80, H=4, Hkv=2, page=7, layout="hnd"),
    dict(lens=(60,), ns=(7,), rot=256, norm=True, dh=256, H=3, Hkv=1, page=7, layout="hnd"),
    dict(lens=(60,), ns=(7,), rot=104, norm=True, dh=136, H=3, Hkv=1, scale=1.3),
    dict(lens=(60,), ns=(7,), rot=24, norm=True, dh=40, H=3, Hkv=3, scale=0.7),
    dict(lens=(9, 0, 40), ns=(1400, 0, 1301), rot=64, norm=True, pad_rows=3, H=4, Hkv=1),
    dict(lens=(70000, 131071), ns=(3, 3), rot=96, norm=False, dh=128, H=4, Hkv=1, page=256),
]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("case", APPEND, ids=range(len(APPEND)))
@pytest.mark.parametrize("only_cache", [False, True])
def test_append_matches_64_bits(case, dtype, only_cache):
    """Every written element within its roundings of the 64-bit value: norm (dh + 8 fp32
    roundings of a sum of squares, half of that relative in its root, 4 more) and the turn (two
    products and a sum of terms up to |x| + |y|, angles off by 2^-22) in fp32, then one rounding to
    the type. Nothing else of the pools changes."""
    case = dict(case)
    rot, norm, scale = case.pop("rot"), case.pop("norm"), case.pop("scale", 1.0)
    blk = Block(31 + rot, dtype, **{**dict(kind="chain"), **case})
    H, Hkv, dh, R = blk.H, blk.Hkv, blk.dh, blk.R
    blk.k = torch.full((blk.n_pages, blk.page, Hkv, dh), 3.0).to(dtype)
    blk.v = blk.k.clone()
    blk.wide = 0
    blk.upload()
    g = torch.Generator().manual_seed(rot)
    qkv = torch.randn(R, H + 2 * Hkv, dh, generator=g).to(dtype)
    dev = qkv.to(DEV)
    wq = (1 + 0.3 * torch.randn(dh, generator=g)).to(dtype) if norm else None
    wk = (1 + 0.3 * torch.randn(dh, generator=g)).to(dtype) if norm else None
    freq = (10000.0 ** (-np.arange(0, rot, 2) / max(rot, 1))).astype(np.float32)
    depth = None
    if blk.parent is not None:
        depth = np.zeros(R, np.int32)
        for i in range(R):
            depth[i] = depth[blk.parent[i]] + 1 if blk.parent[i] >= 0 else 0
    q_out = torch.full((R, H, dh), 7.25, dtype=dtype, device=DEV)
    M.moe_kv_append(blk.C, None if only_cache else dev[:, :H], dev[:, H:H + Hkv],
                    dev[:, H + Hkv:], blk.kd, blk.vd, blk.tabled, blk.lend, blk.B, blk.N,
                    None if only_cache else q_out, blk.ws,
                    depth=None if depth is None else torch.from_numpy(depth).to(DEV),
                    row_start=blk.startd, inv_freq=torch.from_numpy(freq).to(DEV) if rot else None,
                    rope_scale=scale, q_weight=None if wq is None else wq.to(DEV),
                    k_weight=None if wk is None else wk.to(DEV))
    torch.cuda.synchronize()
    assert M.moe_workspace_check(blk.ws) == 0
    u = U[dtype]
    want_k, want_v = blk.k.double(), blk.v.double()
    tol_k = torch.zeros_like(want_k)
    for b in range(blk.B):
        for i in range(blk.ns[b]):
            r = int(blk.rows[b]) + i
            pos = blk.lens[b] + (int(depth[r]) if depth is not None else i)
            c, s = (torch.from_numpy(t[0]) for t in _angles(np.array([pos]), freq))

            def turn(x, w):
                x = x.double()
                rel = 0.0
                if w is not None:
                    x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w.double()
                    rel = (dh / 2 + 8) * 2.0 ** -24
                x1, x2, rest = x[:, :rot // 2], x[:, rot // 2:rot], x[:, rot:]
                y = torch.cat([(x1 * c - x2 * s) * scale, (x2 * c + x1 * s) * scale, rest], 1)
                size = torch.cat([(x1.abs() + x2.abs()) * scale] * 2 + [rest.abs()], 1)
                return y, u * y.abs() + (rel + 2.0 ** -21) * size + 1e-30
            j = blk.lens[b] + i
            p, o = int(blk.table[b, j // blk.page]), j % blk.page
            want_k[p, o], tol_k[p, o] = turn(qkv[r, H:H + Hkv], wk)
            want_v[p, o] = qkv[r, H + Hkv:].double()
            if not only_cache:
                y, tol = turn(qkv[r, :H], wq)
                assert ((q_out[r].double().cpu() - y).abs() <= tol).all()
    assert ((blk.kd.double().cpu() - want_k).abs() <= tol_k).all()
    assert torch.equal(blk.vd.double().cpu(), want_v)
    if blk.R > blk.rows[-1]:
        assert (q_out[int(blk.rows[-1]):] == 7.25).all()


def test_append_in_place_and_bad_slots():
    blk = Block(40, lens=(30, 10), ns=(4, 4), H=8, Hkv=2).upload()
    freq = torch.tensor([1.0, 0.1, 0.01, 0.001], device=DEV)
    k, v = torch.randn(8, 2, 64).to(BF).to(DEV), torch.randn(8, 2, 64).to(BF).to(DEV)
    q1, q2 = blk.qd.clone(), blk.qd.clone()
    out = torch.empty_like(q1)
    args = (k, v, blk.kd, blk.vd, blk.tabled, blk.lend, 2, 4)
    M.moe_kv_append(blk.C, q1, *args, out, blk.ws, inv_freq=freq)
    M.moe_kv_append(blk.C, q2, *args, q2, blk.ws, inv_freq=freq)
    assert torch.equal(out, q2) and not torch.equal(q1, q2)
    assert M.moe_workspace_check(blk.ws) == 0
    # no valid page, or no slot: the rows are rotated, nothing is written, the word tells
    blk.kd.fill_(1)
    blk.vd.fill_(1)
    blk.tabled[0] = blk.n_pages
    blk.lend[1] = -5
    M.moe_kv_append(blk.C, blk.qd, *args, out, blk.ws, inv_freq=freq)
    assert M.moe_workspace_check(blk.ws) == 12
    assert (blk.kd == 1).all() and (blk.vd == 1).all()
    blk.lend[1] = blk.max_pages * blk.page - 2  # two of four rows fit
    blk.tabled[1] = 0
    M.moe_kv_append(blk.C, blk.qd, *args, out, blk.ws, inv_freq=freq)
    assert M.moe_workspace_check(blk.ws) == 12
    assert torch.equal(blk.kd[0, blk.page - 2:].isfinite().all(), torch.tensor(True, device=DEV))
    assert (blk.kd[0, :blk.page - 2] == 1).all() and (blk.kd[1:] == 1).all()


# ------------------------------------------------------------------------------ commit

@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("layout,page,dh", [("nhd", 16, 128), ("hnd", 3, 64), ("nhd", 1, 8)])
def test_commit_moves_accepted_paths(dtype, layout, page, dh):
    paths = [[0, 1, 2, 5], [0, 3, 11, 12], [4, 5, 6, 7], [0, 2, 4, 20], [9, 10, 30, 31]]
    acc = [4, 3, 4, 0, 1]
    blk = Block(50, dtype, lens=(10, 33, 0, 5, 64), ns=(40,) * 5, dh=dh, page=page, layout=layout,
                H=4, Hkv=2).upload()
    k, v = blk.kd.clone(), blk.vd.clone()
    for b in range(5):
        for j in range(acc[b]):
            s, d = blk.lens[b] + paths[b][j], blk.lens[b] + j
            src = (int(blk.table[b, s // page]), s % page)
            dst = (int(blk.table[b, d // page]), d % page)
            k[dst], v[dst] = blk.kd[src], blk.vd[src]
    new = torch.empty(5, dtype=torch.int32, device=DEV)
    M.moe_kv_commit(blk.C, blk.kd, blk.vd, blk.tabled, blk.lend,
                    torch.tensor(paths, dtype=torch.int32, device=DEV),
                    torch.tensor(acc, dtype=torch.int32, device=DEV), new, blk.ws)
    assert M.moe_workspace_check(blk.ws) == 0
    assert torch.equal(blk.kd.nan_to_num(9), k.nan_to_num(9))
    assert torch.equal(blk.vd.nan_to_num(9), v.nan_to_num(9))
    assert new.tolist() == [l + a for l, a in zip(blk.lens, acc)]


def test_commit_long_path_in_place_length_and_bad_paths():
    n = 300
    blk = Block(51, lens=(7,), ns=(n,), H=4, Hkv=1).upload()
    rng = np.random.default_rng(1)
    path = np.sort(rng.choice(n, 120, replace=False)).astype(np.int32)
    k = blk.kd.clone()
    for j, m in enumerate(path):
        k[int(blk.table[0, (7 + j) // 16]), (7 + j) % 16] = \
            blk.kd[int(blk.table[0, (7 + m) // 16]), (7 + int(m)) % 16]
    p = torch.from_numpy(path)[None].to(DEV)
    M.moe_kv_commit(blk.C, blk.kd, blk.vd, blk.tabled, blk.lend, p,
                    torch.tensor([120], dtype=torch.int32, device=DEV), blk.lend, blk.ws)
    assert torch.equal(blk.kd.nan_to_num(9), k.nan_to_num(9)) and blk.lend.tolist() == [127]
    assert M.moe_workspace_check(blk.ws) == 0
    for bad, kept, bits in (([0, 2, 2, 9], 2, 8), ([-1, 2, 3, 4], 0, 8), ([0, 4, 3, 9], 2, 8),
                            ([0, 4, 1 << 30, 1 << 30], 2, 8)):
        new = torch.zeros(1, dtype=torch.int32, device=DEV)
        blk.lend[0] = 7
        M.moe_kv_commit(blk.C, blk.kd, blk.vd, blk.tabled, blk.lend,
                        torch.tensor([bad], dtype=torch.int32, device=DEV),
                        torch.tensor([4], dtype=torch.int32, device=DEV), new, blk.ws)
        assert M.moe_workspace_check(blk.ws) == bits and new.tolist() == [7 + kept]
    # a page outside the pool ends the path; more accepted nodes than the path has are cut
    blk.tabled[0, 1] = blk.n_pages
    for acc, kept, bits in ((4, 1, 4), (9, 1, 12), (-2, 0, 8)):
        M.moe_kv_commit(blk.C, blk.kd, blk.vd, blk.tabled, blk.lend,
                        torch.tensor([[0, 20, 30, 40]], dtype=torch.int32, device=DEV),
                        torch.tensor([acc], dtype=torch.int32, device=DEV), new, blk.ws)
        assert M.moe_workspace_check(blk.ws) == bits and new.tolist() == [7 + kept]


# -------------------------------------------------------------------------- block norm

def _norm_ref(x, o, w_post, gate, gate_rows, scale, w_pre, eps):
    f64 = torch.float64
    h = x.to(f64)
    d = x.shape[1]
    if o is not None:
        t = o.to(f64)
        if w_post is not None:
            t = t / torch.sqrt((t * t).mean(1, keepdim=True) + eps) * w_post.to(f64)
        if gate is not None:
            t = t * gate.to(f64).repeat_interleave(gate_rows, 0)[:len(x)]
        size = h.abs() + (scale * t).abs()
        h = h + scale * t
    else:
        size = h.abs()
    rms = torch.sqrt((h * h).mean(1, keepdim=True) + eps)
    w = 1.0 if w_pre is None else w_pre.to(f64)
    # h in fp32: (d / 2 + 12) roundings relative to its terms; the second norm as much again
    rel = (d / 2 + 12) * 2.0 ** -24
    e_rms = torch.sqrt(((rel * size) ** 2).mean(1, keepdim=True))
    hn = h / rms * w
    return h, hn, rel * size, (rel * size / rms * (w.abs() if w_pre is not None else 1.0) +
                               hn.abs() * (e_rms / rms + rel))


NORMS = [(1, 8, True, 0, 1.0, True), (65, 2048, True, 0, 1.0, True),
         (37, 264, False, 37, 0.5, True), (300, 2880, True, 7, -2.0, False),
         (1300, 2880, True, 700, 0.5, True), (2000, 136, True, 0, 1.0, True),
         (1217, 4096, False, 1217, 1.5, False), (1500, 1032, True, 3, 1.0, True),
         (33, 6144, True, 1, 0.25, True), (5, 4104, False, 0, 1.0, False)]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("R,d,post,gate_rows,scale,pre", NORMS)
def test_block_norm_matches_64_bits(dtype, R, d, post, gate_rows, scale, pre):
    g = torch.Generator().manual_seed(R * 7 + d)
    rows = torch.exp(torch.randn(R, 1, generator=g) * 3)
    x, o = ((torch.randn(R, d, generator=g) * rows).to(dtype) for _ in range(2))
    wp = (1 + 0.2 * torch.randn(d, generator=g)).to(dtype) if post else None
    wn = (1 + 0.2 * torch.randn(d, generator=g)).to(dtype) if pre else None
    gate = torch.randn(-(-R // gate_rows), d, generator=g).to(dtype) if gate_rows else None
    L = M.layer_desc(d, 8, 1, 64, dtype)
    up = lambda t: None if t is None else t.to(DEV)
    h, hn = (torch.full((R, d), float("nan"), dtype=dtype, device=DEV) for _ in range(2))
    args = dict(w_post=up(wp), gate=up(gate), gate_rows=gate_rows, scale=scale, w_pre=up(wn))
    M.moe_block_norm(L, up(x), up(o), h, hn, **args)
    wh, whn, th, thn = _norm_ref(x, o, wp, gate, gate_rows, scale, wn, 1e-6)
    u = U[dtype]
    assert ((h.double().cpu() - wh).abs() <= th + u * wh.abs() + 1e-37).all()
    assert ((hn.double().cpu() - whn).abs() <= thn + u * whn.abs() + 1e-37).all()
    # the buffers that may be shared
    for hx, hnx in (("x", "o"), ("o", "x"), ("x", None)):
        buf = {"x": up(x), "o": up(o), None: None}
        a, b = buf[hx], buf[hnx]
        M.moe_block_norm(L, buf["x"], buf["o"], a, b, **args)
        assert torch.equal(a, h) and (b is None or torch.equal(b, hn))
    # without a branch: a norm with weights
    only = torch.empty_like(hn)
    M.moe_block_norm(L, up(x), None, None, only, w_pre=up(wn))
    wh, whn, th, thn = _norm_ref(x, None, None, None, 0, 1.0, wn, 1e-6)
    assert ((only.double().cpu() - whn).abs() <= thn + u * whn.abs() + 1e-37).all()


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("eps", [1e-6, 0.0])
@pytest.mark.parametrize("times", [1, 200])
def test_block_norm_rows_at_the_ends_of_the_range(dtype, eps, times):
    """Rows whose squares overflow or vanish in fp32, zero rows and a single large element; few
    rows and many (another kernel)."""
    d = 512
    L = M.layer_desc(d, 8, 1, 64, dtype)
    g = torch.Generator().manual_seed(3)
    x = torch.randn(7, d, generator=g)
    x[1] *= 1e30
    x[2] *= 1e-30
    x[3] = 0
    x[3, 5] = 3.0
    x[4] = 3e38
    x[5] *= 1e-18
    x[6, :] = 1e-20
    x[6, 3] = 1e25
    x = x.to(dtype).repeat(times, 1)
    hn, h2 = torch.empty_like(x, device=DEV), torch.empty_like(x, device=DEV)
    ones = torch.ones(d, dtype=dtype, device=DEV)
    M.moe_block_norm(L, x.to(DEV), None, None, hn, eps=eps)
    want = x.double() / torch.sqrt((x.double() ** 2).mean(1, keepdim=True) + eps)
    tol = (U[dtype] + (d / 2 + 12) * 2.0 ** -24) * want.abs() + 1e-37
    assert ((hn.double().cpu() - want).abs() <= tol).all()
    # the same rows as the branch of a zero residual
    M.moe_block_norm(L, torch.zeros_like(x, device=DEV), x.to(DEV), h2, None, w_post=ones, eps=eps)
    assert ((h2.double().cpu() - want).abs() <= tol).all()
    if eps:
        z = torch.zeros(2, d, dtype=dtype, device=DEV)
        out = torch.ones_like(z)
        M.moe_block_norm(L, z, None, None, out, eps=eps)
        assert (out == 0).all()


# ------------------------------------------------------------------------ used together

def test_a_verification_round_of_a_block():
    """Two rounds of a decoder block as an engine runs them: append, attend, norm and residual,
    the MoE layer, commit of an accepted path, and a second tree over the longer context. The
    attention output of the second round equals that of a cache into which the accepted tokens
    were written one by one."""
    shape = W.QWEN3_30B_A3B
    H, Hkv, dh, page, ctx = 16, 4, 128, 16, 90  # H dh = shape.d
    g = torch.Generator().manual_seed(77)
    t = W.eagle_tree(5)
    N = t.N
    parent = torch.from_numpy(t.parent.astype(np.int32)).to(DEV)
    depth = torch.from_numpy(t.depth.astype(np.int32)).to(DEV)
    pools = [torch.zeros(40, page, Hkv, dh, dtype=BF, device=DEV) for _ in range(4)]
    table = torch.randperm(40, generator=g).to(torch.int32)[None].to(DEV)
    C_ = M.cache_desc(pools[0], H, 40)
    ws = M.attention_workspace(C_, 1, ctx)
    freq = torch.from_numpy((1e4 ** (-np.arange(0, dh, 2) / dh)).astype(np.float32)).to(DEV)
    wq = (1 + 0.1 * torch.randn(dh, generator=g)).to(BF).to(DEV)

    def rows(n):
        return torch.randn(n, H + 2 * Hkv, dh, generator=g).to(BF).to(DEV)

    def append(kp, vp, qkv, ln, dep=None, n=None):
        q = torch.empty(len(qkv), H, dh, dtype=BF, device=DEV)
        M.moe_kv_append(C_, qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:], kp, vp, table, ln, 1,
                        len(qkv), q, ws, depth=dep, inv_freq=freq, q_weight=wq, k_weight=wq)
        return q
    zero = torch.zeros(1, dtype=torch.int32, device=DEV)
    prompt = rows(ctx)
    for i in (0, 2):
        append(pools[i], pools[i + 1], prompt, zero)
    ln = torch.tensor([ctx], dtype=torch.int32, device=DEV)
    tree1 = rows(N)
    q = append(pools[0], pools[1], tree1, ln, depth)
    o = torch.empty(N, H, dh, dtype=BF, device=DEV)
    M.moe_tree_attention(C_, q, pools[0], pools[1], table, ln, 1, N, o, ws, parent=parent)
    # norm and residual, then the MoE layer with its own residual
    L = M.layer_desc(shape.d, shape.E, shape.k, shape.f, "bf16")
    x = torch.randn(N, shape.d, generator=g).to(BF).to(DEV)
    h, hn = torch.empty_like(x), torch.empty_like(x)
    w = torch.ones(shape.d, dtype=BF, device=DEV)
    M.moe_block_norm(L, x, o.view(N, -1), h, hn, w_pre=w)
    wr = W.router_weight(1, shape, device=DEV)
    wg, wu, wd = W.expert_weights(2, shape, device=DEV)
    y = torch.empty_like(x)
    lws = M.workspace(L, 1, N)
    P = M.select_params(M.MOE_ROUTE_ACCEPT, W.C_EAGLE)
    M.moe_tree_forward(L, P, hn, wr, wg, wu, wd, None, depth, 1, N, None, y, lws)
    M.moe_block_norm(L, h, y, h, hn, w_pre=w)
    torch.cuda.synchronize()
    assert M.moe_workspace_check(lws) == 0 and torch.isfinite(hn.float()).all()
    # the deepest leaf's path is accepted
    leaf = int(np.argmax(t.depth))
    path = []
    while leaf >= 0:
        path.insert(0, leaf)
        leaf = int(t.parent[leaf])
    n = len(path)
    M.moe_kv_commit(C_, pools[0], pools[1], table, ln,
                    torch.tensor([path], dtype=torch.int32, device=DEV),
                    torch.tensor([n], dtype=torch.int32, device=DEV), ln, ws)
    append(pools[2], pools[3], tree1[path], torch.tensor([ctx], dtype=torch.int32, device=DEV))
    assert ln.tolist() == [ctx + n]
    tree2 = rows(N)
    outs = []
    for i in (0, 2):
        q = append(pools[i], pools[i + 1], tree2, ln, depth)
        o = torch.empty(N, H, dh, dtype=BF, device=DEV)
        M.moe_tree_attention(C_, q, pools[i], pools[i + 1], table, ln, 1, N, o, ws, parent=parent)
        outs.append(o)
    assert M.moe_workspace_check(ws) == 0
    assert torch.equal(outs[0], outs[1])
    assert torch.isfinite(outs[0].float()).all()
