"""GPU tests of the decoding calls at values, sizes and paths where they can go wrong, against the same plain
64-bit computations as test_gpu_decode.py (its tolerances hold here too)."""
import numpy as np
import pytest
import torch

from expert_select_gb300 import moetree as M
from test_gpu_decode import Book, Few, peaked, sample_check

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from expert_select_gb300 import build
    build.build()
    M.lib()


# --------------------------------------------------------------------- sampling

@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [600, 4099, 70001])
def test_sample_min_p_at_zero(V, dt):
    """min-p's least value is 0.0 itself, in lists and where more is kept than a list holds."""
    g = torch.Generator().manual_seed(V)
    r = torch.rand(V, generator=g)
    n = torch.randn(V, generator=g)
    rows = [torch.zeros(V), torch.where(r < 0.5, 0.0, -0.0), torch.where(r < 0.9, 0.0, -n.abs()),
            torch.where(r < 0.9, -n.abs(), 0.0), torch.where(r < 0.95, 0.0, -1e-38),
            torch.where(torch.arange(V) == V // 3, 0.0, -n.abs() - 0.1)]
    x = torch.stack(rows).to(dt)
    for kw in (dict(m=1.0), dict(m=2.0), dict(m=1.0, k=300), dict(m=1.0, p=0.6), dict(m=1.0, k=550, p=0.7),
               dict(m=1.0, T=0.3), dict(m=0.999, p=0.8)):
        for u in (torch.rand(len(rows), generator=g), torch.zeros(len(rows))):
            sample_check(x, u, **kw)


@pytest.mark.parametrize("V", [700, 4099, 70001])
def test_sample_between_zero_and_the_smallest_values(V):
    """Zeros of both signs among denormals, cuts among them: keys beside zero's."""
    g = torch.Generator().manual_seed(V)
    tiny = lambda most: torch.randint(1, most, (V,), generator=g).int().view(torch.float32)  # noqa: E731
    r = torch.rand(V, generator=g)
    zero = torch.where(torch.rand(V, generator=g) < 0.5, 0.0, -0.0)
    rows = []
    for most in (8, 4096, 0x400000):
        rows += [torch.where(r < 0.3, zero, -tiny(most)), torch.where(r < 0.3, zero, tiny(most)),
                 torch.where(r < 0.2, zero, torch.where(r < 0.6, tiny(most), -tiny(most)))]
    # the largest 2^n - 1 steps above zero
    for n in (1, 3, 10, 13, 20):
        row = torch.where(r < 0.3, zero, -tiny(0x400000))
        row[V // 2] = torch.tensor((1 << n) - 1, dtype=torch.int32).view(torch.float32)
        rows.append(row)
    x = torch.stack(rows)
    for kw in (dict(k=V // 4 + 300), dict(k=V * 3 // 5 + 200), dict(k=V - 2), dict(p=0.55), dict(p=0.9),
               dict(p=0.7, k=V * 4 // 5), dict(T=1e-30, p=0.6), dict(T=1e-30, k=V * 2 // 3 + 90)):
        sample_check(x, torch.rand(len(rows), generator=g), **kw)


# --------------------------------------------------------------------- a few tokens

def _few(d, E, k, f, R, dt, wr, wg, wu, wd):
    up = lambda t: t.to(dt).to(DEV).contiguous()  # noqa: E731
    L = M.layer_desc(d, E, k, f, dt)
    return L, [up(t) for t in (wr, wg, wu, wd)], M.few_workspace(L, R)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_few_norm_rounds_each_element_once(dt):
    """The router is the identity, so the logits are the normed elements: each is the 64-bit one rounded once.
    Rows are those of many that have elements beside the middle of two values of the type. (The scale is good
    to 2^-45, so an element within 2^-44 of a middle may go either way.)"""
    d, R = 256, 16
    g = torch.Generator().manual_seed(12)
    x = (torch.randn(60000, d, generator=g) * (0.1 + 10 * torch.rand(60000, 1, generator=g))).to(dt)
    step = 2.0 ** (-8 if dt == torch.bfloat16 else -24)

    def normed(x):
        t = x.double()
        return t / torch.sqrt((t * t).mean(1, keepdim=True) + 1e-6)

    def off_middle(y):  # relative distance from the nearest middle
        m, e = torch.frexp(y)
        q = m.abs() / step  # in steps of the type, in [1 / 2, 1) / step
        return (q - torch.floor(q) - 0.5).abs() * step

    def rounded(y):  # (torch's conversion to bf16 rounds to fp32 first)
        m, e = torch.frexp(y)
        return torch.ldexp(torch.round(m / step) * step, e)
    near = (off_middle(normed(x)) < 2.0 ** (-22 if dt == torch.bfloat16 else -38)).any(1)
    x = x[near][:960]
    assert len(x) >= 320
    x = x[:len(x) // R * R]
    zero = torch.zeros(d, 8, d)
    L, w, ws = _few(d, d, 1, 8, R, dt, torch.eye(d), zero, zero, zero.transpose(1, 2))
    y, logits = torch.empty(R, d, dtype=dt, device=DEV), torch.empty(len(x), d, device=DEV)
    for r in range(0, len(x), R):
        M.moe_few_forward(L, x[r:r + R].to(DEV), *w, None, y, ws, logits=logits[r:r + R],
                          opts=M.run_opts(norm_input=True))
    want = normed(x)
    got = logits.cpu()
    bad = (got.double() != rounded(want)) & (off_middle(want) > 2.0 ** -44)
    assert not bad.any(), (int(bad.sum()), int(bad.any(1).sum()), len(x))
    # where it may go either way, one of the two
    assert ((got.double() - want).abs() <= (step / 2 + 2.0 ** -44) * 2 * want.abs()).all()


@pytest.mark.parametrize("R,d,E,k,f", [(16, 136, 3, 3, 72), (13, 520, 7, 7, 264), (9, 64, 2, 2, 24), (16, 8, 1, 1, 8),
                                       (12, 328, 5, 4, 1000), (10, 2048, 4, 4, 16)])
@pytest.mark.parametrize("ctas", [0, 3])
def test_few_fp32_experts_of_many_tokens(R, d, E, k, f, ctas):
    """9 to 16 tokens of an expert: more than a lane's sums take at a time, in both halves of the call."""
    t = Few(R + d, R, d, E, k, f, torch.float32).upload().run(True, True, max_ctas=ctas)
    counts = torch.bincount(t.idx.cpu().flatten().long(), minlength=E)
    assert counts.max() >= 9
    t.check(True, True)


@pytest.mark.parametrize("depth,R,d", [(10, 1, 512), (10, 2, 6144), (7, 3, 512), (7, 6, 6144), (5, 7, 512), (5, 8, 6144),
                                       (5, 16, 512), (5, 16, 3392), (4, 16, 3400), (5, 9, 6016), (4, 9, 6024)])
@pytest.mark.parametrize("f", [8, 264])
def test_few_rings_of_every_depth(depth, R, d, f):
    """bf16 layers on both sides of the sizes at which a warp's ring gets fewer entries: parts of a row that are
    shorter than the ring, and longer ones."""
    Few(R + d, R, d, 4, 2, f, torch.bfloat16).upload().run().check()


@pytest.mark.parametrize("dt,R,d", [(torch.bfloat16, 16, 3912), (torch.bfloat16, 13, 4808), (torch.float32, 16, 2984),
                                    (torch.float32, 9, 5320)])
def test_few_tokens_of_several_launches(dt, R, d):
    """One token more than fit a CTA's shared memory together."""
    t = Few(R + d, R, d, 4, 2, 16, dt).upload().run(True, True)
    t.check(True, True)
    x = t.dev[0].clone()
    t.dev[0] = x
    t.run(True, True, y=x).check(True, True, y=x)


# --------------------------------------------------------------------- rows too long for shared memory

def _many(row, R, u, **kw):
    """Tokens of R equal rows, row r at u[r]."""
    V = row.numel()
    x = row.to(DEV).expand(R, V).contiguous()
    token = torch.full((R,), -9, dtype=torch.int32, device=DEV)
    put = lambda n, dt: torch.full((R,), kw[n], dtype=dt, device=DEV) if n in kw else None  # noqa: E731
    M.moe_sample(x, u.to(DEV), token, temperature=put("T", torch.float32), top_k=put("k", torch.int32),
                 top_p=put("p", torch.float32))
    return token.cpu()


def test_sample_border_beside_a_sum_that_rounds_away():
    """Rows of one CTA each, summed block after block: 512 threads begin with a weight of 1 and three of 2^-24,
    and what follows, 2^-24 a block, is lost in fp32 (each a tie that goes to even), 258 2^-24 in all. top-p's
    limit is put so that the 257th of the equal tokens is kept only if the weight is known better than to that."""
    V, threads, blocks = 1 << 19, 512, 256
    octaves = torch.full((16, blocks, 32, 4), 26.0)  # by warp, turn, lane: a block of four
    octaves[:, 0, :, 1:] = 24.0
    octaves[:, 0, :, 0] = 0.0
    row = -octaves.reshape(V)
    T = torch.tensor(1.4426950408889634).item()  # an octave is a step of one in the logits
    heavy = torch.nonzero(row == 0).flatten()
    assert len(heavy) == threads
    z = threads * (1 + 258 * 2.0 ** -24)
    # the border of the 257th token (256 before it) lies between p z and p times what is left of z with an error of 2^-16
    p = torch.tensor(256 / z * (1 + 0.9 * 2.0 ** -24)).item()
    assert p * z > 256 * (1 + 2.0 ** -26) and p * threads * (1 + 2.0 ** -16) < 256 * (1 - 2.0 ** -26)
    R = 240
    u = (torch.arange(R) + 0.5) / R
    got = _many(row, R, u, T=T, p=p)
    assert torch.equal(got.long(), heavy[(u.double() * 257).long()])


@pytest.mark.parametrize("dt,V", [(torch.float32, 79000), (torch.float32, 151936), (torch.bfloat16, 330007)])
def test_sample_many_long_rows(dt, V):
    """Rows of one CTA each whose blocks' largest values do not fit shared memory, every row with settings of its
    own: lists of top-k, of min-p, of top-p of the whole row, and what no list holds."""
    g = torch.Generator().manual_seed(V)
    R = 232
    pick = lambda vals: torch.tensor(vals)[torch.randint(0, len(vals), (R,), generator=g)]  # noqa: E731
    x = peaked(g, R, V, dt)
    sample_check(x, torch.rand(R, generator=g), T=pick([0.0, 0.3, 0.7, 0.7, 1.0]), k=pick([0, 0, 1, 20, 250, 1000]),
                 p=pick([1.0, 0.95, 0.9, 0.5]), m=pick([0.0, 0.0, 0.02, 0.3]), shift=3, pad=1)
    # settings shared among rows: fewer rows take one CTA each
    R = 160
    sample_check(x[:R], torch.rand(R, generator=g), T=0.8, k=40, p=0.9, group=R)
    sample_check(x[:R], torch.rand(R, generator=g), T=0.6, p=0.9, m=0.001, group=R)


# --------------------------------------------------------------------- pages

@pytest.mark.parametrize("n", [2, 300])
def test_fork_of_a_target(n):
    """Of the entries (a, b), (b, c) the first is carried out and the second refused, in lists of both kinds."""
    k = Book(3, 900, 4, 5000, 8, used=0.0)
    k.reserve(np.array([11, 9] + [0] * 898, np.int32))
    k.len[:2] = 11, 9
    k.dev[2].copy_(torch.from_numpy(k.len))
    dst = list(range(2, 2 + n))
    k.fork([0, 2] + [0] * (n - 2), [2, 3] + dst[2:])
    assert k.flags & 8
    k.same()
    assert k.held[2] > 0 and k.held[3] == 0


def test_free_keeps_the_pages_of_keep():
    """Pages of ceil(keep / page_size) stay although the tokens need fewer; those behind go."""
    k = Book(4, 6, 12, 90, 16, used=0.0)
    k.reserve(np.array([5, 100, 16, 17, 0, 190], np.int32))
    k.len[:] = [5, 20, 16, 17, 0, 3]
    k.dev[2].copy_(torch.from_numpy(k.len))
    k.same()
    k.free([0, 1, 2, 3, 4, 5], [16, 33, 1000, 16, 7, 32])
    k.same()
    assert k.held.tolist() == [1, 3, 1, 1, 0, 2] and k.len.tolist() == [5, 20, 16, 16, 0, 3]
