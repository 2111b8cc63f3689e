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
