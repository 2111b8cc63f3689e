"""GPU tests of the attention half's edges: pieces of one key tile, entries of the page table that no
row needs, rows that see nothing, paths that do not fit, values at the ends of the range."""
import numpy as np
import pytest
import torch

from expert_select_gb300 import moetree as M
from test_gpu_attention import BF, DEV, F32, Block

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from expert_select_gb300 import build
    build.build()
    M.lib()


@pytest.mark.parametrize("dh,page", [(128, 16), (64, 64)])
@pytest.mark.parametrize("B", [2048, 700])
def test_many_pieces_of_one_key_tile(B, dh, page):
    """Short sequences of several nodes, one key tile and at most 128 rows each: a CTA has a dozen
    such pieces in a row, in which the second slot has nothing to compute; some of two tiles lie
    between them."""
    r = np.random.default_rng(B)
    lens = tuple(int(v) for v in np.where(r.random(B) < 0.9, r.integers(0, 50, B),
                                          r.integers(60, 200, B)))
    blk = Block(B, BF, lens=lens, ns=(10,) * B, H=4, Hkv=2, dh=dh, page=page, kind="tree").upload()
    for _ in range(3):
        blk.attend()
    blk.check()


@pytest.mark.parametrize("path,room", [([-5, -3, 0], 1), ([3, 0, 1, 2], 3), ([7, -1, 0, 1, 2], 2)])
def test_a_bad_path_looks_up_no_slot_past_the_table(path, room):
    """Behind its first bad node a path ascends again from a low one: node path[j] has a slot in the
    table, slot len + j has none. The entry behind the row belongs to the next sequence, whose table
    is not to be looked at (its entries are outside the pool: bit 2 would tell)."""
    blk = Block(52, BF, lens=(40, 40), ns=(8, 8), H=4, Hkv=1, page=1).upload()
    cap = blk.max_pages
    blk.lend.copy_(torch.tensor([cap - room, 0], dtype=torch.int32))
    blk.tabled[0] = torch.arange(cap, dtype=torch.int32) % blk.n_pages
    blk.tabled[1] = -9
    k, v = blk.kd.clone(), blk.vd.clone()
    paths = torch.tensor([path, [0] * len(path)], dtype=torch.int32, device=DEV)
    new = torch.zeros(2, dtype=torch.int32, device=DEV)
    M.moe_kv_commit(blk.C, blk.kd, blk.vd, blk.tabled, blk.lend, paths,
                    torch.tensor([len(path), 0], dtype=torch.int32, device=DEV), new, blk.ws)
    assert M.moe_workspace_check(blk.ws) == 8
    kept = 1 if 0 <= path[0] < room else 0
    assert new.tolist() == [cap - room + kept, 0]
    if not kept:
        assert torch.equal(blk.kd.nan_to_num(9), k.nan_to_num(9))
        assert torch.equal(blk.vd.nan_to_num(9), v.nan_to_num(9))


@pytest.mark.parametrize("dh,ns,ln", [(128, 10, 300), (64, 12, 60), (128, 70, 200)])
def test_values_that_are_not_finite_in_many_pieces_in_a_row(dh, ns, ln):
    """Every third sequence has a node of infinite values: while a piece's output is formed, the
    warp that looks after V meets such values in a later one. Rows that do not see them are what they
    were, rows that do are infinite."""
    r = np.random.default_rng(dh + ns)
    B = 400
    lens = tuple(int(v) for v in r.integers(0, ln, B))
    blk = Block(53, BF, lens=lens, ns=(ns,) * B, H=4, Hkv=2, dh=dh, kind="tree").upload().attend()
    torch.cuda.synchronize()
    want = blk.out.clone()
    sees = torch.zeros(blk.R, dtype=torch.bool)
    for b in range(0, B, 3):
        m = ns // 2
        j = lens[b] + m
        blk.vd[int(blk.table[b, j // blk.page]), j % blk.page] = float("inf")
        sees[blk.rows[b]:blk.rows[b + 1]] = torch.from_numpy(blk.visible(b)[:, j])
    for _ in range(3):
        blk.out.fill_(7.25)
        blk.attend()
        assert torch.equal(blk.out[~sees.to(DEV)], want[~sees.to(DEV)])
        assert torch.isinf(blk.out[sees.to(DEV)]).all()
    assert M.moe_workspace_check(blk.ws) == 0


# shape, and which kernel it takes in bf16
WINDOWED = [
    dict(lens=(1000, 130, 77), ns=(1, 1, 1), H=16, Hkv=2, window=100, sinks=4),           # few rows
    dict(lens=(1000, 5), ns=(12, 12), H=8, Hkv=2, dh=128, window=50, kind="tree", page=5),  # few rows
    dict(lens=(900, 400), ns=(65, 65), H=16, Hkv=2, dh=128, window=128, sinks=4, kind="tree"),
    dict(lens=(900, 1200), ns=(65, 1), H=16, Hkv=2, dh=128, window=130, sinks=70, page=1),
    dict(lens=(3000,), ns=(300,), H=8, Hkv=1, window=200, page=32, layout="hnd"),
    dict(lens=(2000, 0), ns=(200, 150), H=8, Hkv=1, dh=80, window=70, sinks=9, page=7),
    dict(lens=(600, 64), ns=(30, 40), H=4, Hkv=2, dh=136, window=40, sinks=3, page=8),    # CUDA cores
]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("case", WINDOWED, ids=range(len(WINDOWED)))
@pytest.mark.parametrize("entry", [-1, 1 << 30])
def test_pages_older_than_every_window_need_no_entry(case, dtype, entry):
    """An engine with a window gives pages back that no row can see any more: their entries may hold
    anything, what is left in the pages too, and nothing is flagged."""
    blk = Block(54, dtype, **case).upload()
    gone = 0
    for b, ln in enumerate(blk.lens):
        for p in range(ln // blk.page):
            if p * blk.page >= blk.sinks and (p + 1) * blk.page - 1 <= ln - blk.window:
                pg = int(blk.table[b, p])
                blk.kd[pg] = float("nan")
                blk.vd[pg] = float("nan")
                blk.tabled[b, p] = entry
                gone += 1
    assert gone > 0
    blk.attend().check()


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("n", [1, 65])
@pytest.mark.parametrize("entry", [-1, -(1 << 31), (1 << 31) - 1])
def test_any_entry_outside_the_pool_is_flagged(dtype, n, entry):
    blk = Block(58, dtype, lens=(200,), ns=(n,), H=4, Hkv=1, dh=128).upload()
    blk.tabled[0, 3] = entry
    blk.attend()
    assert M.moe_workspace_check(blk.ws) == 4


@pytest.mark.parametrize("dtype,dh", [(BF, 64), (BF, 128), (BF, 136), (F32, 64)])
@pytest.mark.parametrize("N,over", [(1, 0), (40, 2), (300, 3), (300, 0)])
def test_rows_past_the_table_that_see_nothing_give_zeros(dtype, dh, N, over):
    """A sequence whose length leaves its block `over` slots of a table that ends with a key tile,
    under a window of 2: node i sees slots len + i - 1 and len + i as far as there are any. Rows of
    whole items see nothing."""
    blk = Block(55, dtype, lens=(16,), ns=(N,), page=64, H=4, Hkv=1, dh=dh, window=2).upload()
    blk.lend[0] = blk.max_pages * blk.page - over
    blk.tabled[:] = blk.tabled[0, 0]
    blk.kd[:] = 1
    blk.vd[:] = 2
    blk.attend()
    torch.cuda.synchronize()
    assert M.moe_workspace_check(blk.ws) == 8
    assert (blk.out[:over + 1] == 2).all() and torch.isfinite(blk.lse[:over + 1]).all()
    assert (blk.out[over + 1:] == 0).all() and (blk.lse[over + 1:] == -float("inf")).all()
    one = Block(55, dtype, lens=(16,), ns=(N,), page=64, H=4, Hkv=1, dh=dh, window=1).upload()
    one.lend[0] = one.max_pages * one.page
    one.attend()
    torch.cuda.synchronize()
    assert M.moe_workspace_check(one.ws) == 8
    assert (one.out == 0).all() and (one.lse == -float("inf")).all()


def test_a_single_row_of_a_projection_is_rotated_in_place():
    """q as the first heads of one row of a projection's output, and q_out the same memory."""
    blk = Block(59, BF, lens=(30,), ns=(1,), H=8, Hkv=2).upload()
    freq = torch.tensor([1.0, 0.1, 0.01, 0.001], device=DEV)
    qkv = torch.randn(1, 12, 64, device=DEV).to(BF)
    want, kept = torch.empty(1, 8, 64, dtype=BF, device=DEV), qkv.clone()
    for q_out in (want, qkv[:, :8]):
        M.moe_kv_append(blk.C, qkv[:, :8], qkv[:, 8:10], qkv[:, 10:], blk.kd, blk.vd, blk.tabled,
                        blk.lend, 1, 1, q_out, blk.ws, inv_freq=freq)
    assert torch.equal(qkv[:, :8], want) and not torch.equal(want, kept[:, :8])
    assert torch.equal(qkv[:, 8:], kept[:, 8:])


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("eps", [1e-6, 0.0])
@pytest.mark.parametrize("dh,rot", [(64, 64), (40, 24), (256, 0)])
def test_append_norms_at_the_ends_of_the_range(dtype, eps, dh, rot):
    """Heads whose squares overflow or vanish in fp32, and a single large element: x / rms(x) as the
    64-bit value within the roundings of a norm ((dh / 2 + 12) 2^-24) and of a turn by angle 0 (none:
    cos 0 = 1, sin 0 = 0), then one to the type. Zero heads stay zero where eps is not."""
    g = torch.Generator().manual_seed(dh)
    scales = [1.0, 1e30, 1e-30, 1e-18, 3e37, 1e19]
    x = torch.randn(1, 8, dh, generator=g)
    for i, s in enumerate(scales):
        x[0, i] *= s / x[0, i].abs().max()
    x[0, 6] = 1e-20
    x[0, 6, 3] = 1e25
    x[0, 7] = 0 if eps else 1
    x = x.to(dtype)
    blk = Block(56, dtype, lens=(0,), ns=(1,), H=8, Hkv=8, dh=dh).upload()
    w = torch.ones(dh, dtype=dtype, device=DEV)
    q_out = torch.empty(1, 8, dh, dtype=dtype, device=DEV)
    freq = torch.ones(rot // 2, device=DEV) if rot else None
    M.moe_kv_append(blk.C, x.to(DEV), x.to(DEV), x.to(DEV), blk.kd, blk.vd, blk.tabled, blk.lend, 1,
                    1, q_out, blk.ws, inv_freq=freq, q_weight=w, k_weight=w, eps=eps)
    assert M.moe_workspace_check(blk.ws) == 0
    d = x.double()
    want = d / torch.sqrt((d * d).mean(2, keepdim=True) + eps)
    u = 2.0 ** -8 if dtype == BF else 2.0 ** -24
    tol = (u + (dh / 2 + 12) * 2.0 ** -24) * want.abs() + 1e-37
    page = int(blk.table[0, 0])
    for got in (q_out[0], blk.kd[page, 0]):
        assert ((got.double().cpu() - want[0]).abs() <= tol[0]).all()
    assert torch.equal(blk.vd[page, 0].cpu(), x[0])


@pytest.mark.parametrize("top", [10 ** 6, 1 << 24])
def test_angles_of_far_positions(top):
    """Heads of ones and zeros, so that the written key is the angle's cosine and sine in fp32. They
    are off by 2^-24 (a sine or cosine right to a unit in the last place), 2^-25 (one more rounding)
    and by the angle's own error, 2^-45 of pos freq: 1 / (2 pi) as two fp32 values (2^-48) and its
    product with freq as two more (2^-47 and 2^-48), the same of the product with pos (2^-46), all
    of them at their worst."""
    dh, n = 256, 512
    r = np.random.default_rng(7)
    blk = Block(57, F32, lens=(0,), ns=(n,), H=1, Hkv=1, dh=dh, page=64).upload()
    pos = r.integers(0, top, n).astype(np.int32)
    pos[:3] = (0, 1, top - 1)
    freq = np.exp(-r.random(dh // 2) * np.log(1e6)).astype(np.float32)
    freq[:2] = (1.0, 0.7)
    k = torch.zeros(n, 1, dh, device=DEV)
    k[..., :dh // 2] = 1
    q = torch.empty(n, 1, dh, device=DEV)
    M.moe_kv_append(blk.C, k, k, k, blk.kd, blk.vd, blk.tabled, blk.lend, 1, n, q, blk.ws,
                    depth=torch.from_numpy(pos).to(DEV), inv_freq=torch.from_numpy(freq).to(DEV))
    assert M.moe_workspace_check(blk.ws) == 0
    # (pos has 24 bits and freq 24: their product is exact in 64 bits)
    a = pos.astype(np.float64)[:, None] * freq.astype(np.float64)[None]
    got = q[:, 0].double().cpu().numpy()
    tol = 2.0 ** -24 + 2.0 ** -25 + 2.0 ** -45 * np.abs(a)
    assert (np.abs(got[:, :dh // 2] - np.cos(a)) <= tol).all()
    assert (np.abs(got[:, dh // 2:] - np.sin(a)) <= tol).all()
