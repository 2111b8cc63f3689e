"""Outputs over inputs of the attention half's calls are refused, before any CUDA call, where rows are
taken in no order; and what is allowed stays allowed."""
import ctypes as C

import pytest
import torch

from expert_select_gb300 import build as B
from expert_select_gb300 import moetree as M
from test_attention_host import _desc

BASE, OK_UNTIL_CUDA = 0x10000000, (M.MOE_OK, M.MOE_ERR_CUDA)  # (no GPU, or a pointer never read)


@pytest.fixture(scope="module", autouse=True)
def built():
    B.build()


def _append(q=BASE, ldq=4096, k=BASE + (1 << 20), ldk=512, v=BASE + (2 << 20), ldv=512,
            q_out=BASE + (3 << 20), R=4):
    at = lambda p: None if p is None else C.c_void_p(p)
    f = C.c_void_p(BASE + (4 << 20))
    P = M.RopeParams(None, None, 1e-6, None, 0, 1.0)
    return M.lib().moe_kv_append(C.byref(_desc()), C.byref(P), at(q), ldq, at(k), ldk, at(v), ldv,
                                 f, f, f, f, None, None, 1, R, R, at(q_out), None, None)


ROW = 4096 * 2  # bytes of a row of q


@pytest.mark.parametrize("kw", [
    dict(q_out=BASE + ROW), dict(q_out=BASE - ROW), dict(q_out=BASE + 4 * ROW - 16),
    dict(q_out=BASE - 4 * ROW + 16),                       # q by some rows, or by 16 bytes
    dict(ldq=5120, q_out=BASE),                            # q itself, rows further apart
    dict(ldq=3 * 4096, q_out=BASE + ROW),                  # the gap between q's rows
    dict(q_out=BASE + (1 << 20)), dict(q_out=BASE + (1 << 20) + 3 * 1024),      # k
    dict(q_out=BASE + (2 << 20) - 4 * ROW + 16),                                # v
    dict(k=BASE + 512, q_out=BASE),                        # q itself, k inside it
    dict(k=BASE + 2 * 4096, ldk=5120, v=BASE + 2 * 4608, ldv=5120, ldq=5120, q_out=BASE + 2 * 5120),
], ids=range(11))
def test_append_refuses_queries_over_what_it_reads(kw):
    assert _append(**kw) == M.MOE_ERR_ARG


@pytest.mark.skipif(torch.cuda.is_available(), reason="the pointers are not a device's")
@pytest.mark.parametrize("kw", [
    dict(), dict(q_out=BASE), dict(q_out=BASE + 4 * ROW), dict(q_out=BASE - 4 * ROW),
    dict(q_out=BASE + (1 << 20) + 4 * 1024), dict(q=None, q_out=None),
    # one projection's rows, q_out behind them
    dict(k=BASE + 2 * 4096, ldk=5120, v=BASE + 2 * 4608, ldv=5120, ldq=5120,
         q_out=BASE + 4 * 2 * 5120),
    # a single row of a projection, in place
    dict(R=1, k=BASE + 2 * 4096, v=BASE + 2 * 4608, q_out=BASE),
], ids=range(8))
def test_append_takes_queries_beside_what_it_reads(kw):
    assert _append(**kw) in OK_UNTIL_CUDA


def test_a_single_row_has_no_stride():
    """The row of one token in a projection's output: the binding gives its width as its stride."""
    rows = torch.zeros(1, 40, 128, dtype=torch.bfloat16)
    assert M._rows("f", "q", rows[:, :32], torch.bfloat16, (1, 32, 128), -1) == 32 * 128
    assert M._rows("f", "q", torch.zeros(3, 40, 128)[:, :32], torch.float32, (3, 32, 128),
                   -1) == 40 * 128


def _norm(x=BASE, branch=BASE + (1 << 20), post=None, gate=None, rows=0, pre=None, R=4,
          h=BASE + (2 << 20), hn=BASE + (3 << 20), dtype="bf16"):
    at = lambda p: None if p is None else C.c_void_p(p)
    L = M.layer_desc(2048, 8, 1, 64, dtype)
    return M.lib().moe_block_norm(C.byref(L), at(x), at(branch), at(post), at(gate), rows, 1.0,
                                  at(pre), 1e-6, R, at(h), at(hn), None)


X, BR, HH, HN, D = BASE, BASE + (1 << 20), BASE + (2 << 20), BASE + (3 << 20), 4096  # D: a bf16 row


@pytest.mark.parametrize("kw", [
    dict(h=X + D), dict(h=X - D), dict(h=BR + 3 * D), dict(hn=X + D), dict(hn=BR - 3 * D),
    dict(h=None, branch=None, hn=X + D), dict(hn=HH + D), dict(hn=HH - 3 * D), dict(h=X, hn=X),
    dict(gate=HH, rows=4), dict(gate=HH + D, rows=1), dict(gate=HN + 3 * D, rows=4),
    dict(gate=HH - D, rows=2), dict(post=HH), dict(pre=HN + 2 * D), dict(pre=HH + 3 * D),
    dict(dtype="fp32", h=X + 7 * D),
], ids=range(17))
def test_block_norm_refuses_outputs_over_other_rows(kw):
    assert _norm(**kw) == M.MOE_ERR_ARG


@pytest.mark.skipif(torch.cuda.is_available(), reason="the pointers are not a device's")
@pytest.mark.parametrize("kw", [
    dict(), dict(h=X), dict(h=BR), dict(h=X, hn=BR), dict(h=BR, hn=X), dict(hn=X), dict(hn=BR),
    dict(hn=None), dict(branch=None, h=None, hn=X), dict(branch=None, h=X), dict(x=BR),
    dict(h=X + 4 * D), dict(h=X - 4 * D), dict(hn=HH + 4 * D), dict(hn=HH - 4 * D),
    dict(gate=HH, rows=1), dict(gate=HH - D, rows=4), dict(gate=HH - 2 * D, rows=3),
    dict(post=HH - D, pre=HN + 4 * D), dict(post=X, pre=X),
], ids=range(20))
def test_block_norm_takes_outputs_beside_or_row_for_row(kw):
    assert _norm(**kw) in OK_UNTIL_CUDA
