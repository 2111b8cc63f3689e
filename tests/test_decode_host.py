"""Checks of the decoding round's entry points that need no GPU: workspace sizes, and bad arguments
refused by the library (before any CUDA call) and by the binding."""
import ctypes as C

import pytest
import torch

from expert_select_gb300 import build as B
from expert_select_gb300 import moetree as M

F, ODD, NUL = C.c_void_p(0x100000), C.c_void_p(0x100008), None  # never dereferenced


@pytest.fixture(scope="module", autouse=True)
def built():
    B.build()


def _layer(**kw):
    base = dict(d=2048, E=128, k=8, f=768, dtype=M.MOE_DTYPE_BF16, slots=0)
    base.update(kw)
    return M.LayerDesc(*(base[n] for n in ("d", "E", "k", "f", "dtype", "slots")))


def test_few_workspace_bytes():
    a, b = M.moe_few_workspace_bytes(_layer(), 1), M.moe_few_workspace_bytes(_layer(), 16)
    assert 4096 < a < b and a % 256 == 0
    assert M.moe_few_workspace_bytes(_layer(), 0) == 0
    assert M.moe_few_workspace_bytes(_layer(), 17) == 0
    assert M.moe_few_workspace_bytes(_layer(d=2044), 1) == 0


def _few(L=None, x=F, wr=F, wg=F, wu=F, wd=F, R=1, y=C.c_void_p(0x900000), ws=F, opts=None):
    return M.lib().moe_few_forward(C.byref(L or _layer()), x, wr, wg, wu, wd, NUL, R, y, NUL, NUL,
                                   NUL, ws, None if opts is None else C.byref(opts), NUL)


def test_few_arguments_are_refused():
    for kw in (dict(x=NUL), dict(x=ODD), dict(wr=NUL), dict(wr=ODD), dict(wg=NUL), dict(wg=ODD),
               dict(wu=NUL), dict(wd=ODD), dict(y=NUL), dict(y=ODD), dict(ws=NUL), dict(ws=ODD),
               dict(R=-1), dict(L=_layer(k=0)), dict(L=_layer(E=300)), dict(L=_layer(f=12)),
               dict(y=C.c_void_p(0x100000 + 16)), dict(R=4, y=C.c_void_p(0x100000 + 3 * 4096)),
               dict(opts=M.RunOpts(ffn_max_ctas=-1)), dict(opts=M.RunOpts(ffn_begin=0x1000)),
               dict(opts=M.RunOpts(select_begin=0x1000))):
        assert _few(**kw) == M.MOE_ERR_ARG, kw
    assert _few(R=17) == M.MOE_ERR_UNSUPPORTED
    assert _few(R=0, x=NUL) == M.MOE_OK


def _sample(V=100, dtype=M.MOE_DTYPE_F32, rows=1, logits=F, ld=100, u=F, R=1, token=F):
    P = M.SampleParams(V, dtype, rows, None, None, None, None)
    return M.lib().moe_sample(C.byref(P), logits, ld, u, R, token, NUL, NUL)


def test_sample_arguments_are_refused():
    for kw in (dict(V=0), dict(dtype=2), dict(rows=0), dict(ld=99), dict(R=-1), dict(logits=NUL),
               dict(u=NUL), dict(token=NUL), dict(logits=C.c_void_p(0x100002))):
        assert _sample(**kw) == M.MOE_ERR_ARG, kw
    assert M.lib().moe_sample(NUL, F, 100, F, 1, F, NUL, NUL) == M.MOE_ERR_ARG
    assert _sample(V=(1 << 19) + 1, ld=1 << 20) == M.MOE_ERR_UNSUPPORTED
    assert _sample(R=0, logits=NUL) == M.MOE_OK


def test_accept_arguments_are_refused():
    def call(token=F, sampled=F, start=NUL, B_=2, N=3, R=6, P=4, path=F, acc=F):
        return M.lib().moe_tree_accept(token, F, sampled, start, B_, N, R, P, path, acc, NUL, NUL)
    for kw in (dict(B_=-1), dict(N=-1), dict(R=-1), dict(R=5), dict(P=0), dict(path=NUL),
               dict(acc=NUL), dict(token=NUL), dict(sampled=NUL)):
        assert call(**kw) == M.MOE_ERR_ARG, kw
    assert call(B_=0, R=0) == M.MOE_OK


def _book(**kw):
    base = dict(page_table=0x10000, held=0x20000, cache_len=0x30000, ref=0x40000, B=4, max_pages=8,
                n_pages=64, page_size=16)
    base.update(kw)
    return M.PageBook(**base)


BAD_BOOKS = [dict(page_table=0), dict(held=0), dict(cache_len=0), dict(ref=0), dict(B=0),
             dict(B=65537), dict(max_pages=0), dict(n_pages=0), dict(n_pages=(1 << 24) + 1),
             dict(page_size=0), dict(page_size=1 << 16, max_pages=1 << 15)]


@pytest.mark.parametrize("bad", BAD_BOOKS, ids=lambda d: "-".join(f"{k}={v}" for k, v in d.items()))
def test_bad_books_are_refused(bad):
    K, lib = C.byref(_book(**bad)), M.lib()
    assert lib.moe_pages_workspace_bytes(K) == 0
    assert lib.moe_kv_reserve(K, 1, NUL, F, NUL) == M.MOE_ERR_ARG
    assert lib.moe_kv_free(K, F, NUL, 1, F, NUL) == M.MOE_ERR_ARG
    assert lib.moe_kv_fork(K, F, F, 1, F, F, NUL) == M.MOE_ERR_ARG
    assert lib.moe_kv_compact(K, F, F, F, F, F, NUL) == M.MOE_ERR_ARG


def test_page_arguments_are_refused():
    K, lib = C.byref(_book()), M.lib()
    assert lib.moe_pages_workspace_bytes(K) > 4096
    assert lib.moe_kv_reserve(K, -1, NUL, F, NUL) == M.MOE_ERR_ARG
    for ws in (NUL, ODD):
        assert lib.moe_kv_reserve(K, 1, NUL, ws, NUL) == M.MOE_ERR_ARG
        assert lib.moe_kv_free(K, F, NUL, 1, ws, NUL) == M.MOE_ERR_ARG
        assert lib.moe_kv_fork(K, F, F, 1, F, ws, NUL) == M.MOE_ERR_ARG
        assert lib.moe_kv_compact(K, F, F, F, F, ws, NUL) == M.MOE_ERR_ARG
    assert lib.moe_kv_free(K, F, NUL, -1, F, NUL) == M.MOE_ERR_ARG
    assert lib.moe_kv_free(K, NUL, NUL, 1, F, NUL) == M.MOE_ERR_ARG
    assert lib.moe_kv_free(K, NUL, NUL, 0, F, NUL) == M.MOE_OK
    for args in ((NUL, F, 1, F), (F, NUL, 1, F), (F, F, 1, NUL), (F, F, -1, F), (F, F, 5, F)):
        assert lib.moe_kv_fork(K, *args, F, NUL) == M.MOE_ERR_ARG, args
    assert lib.moe_kv_fork(K, NUL, NUL, 0, NUL, F, NUL) == M.MOE_OK
    for args in ((NUL, F, F, F), (F, NUL, F, F), (F, F, NUL, F), (F, F, F, NUL)):
        assert lib.moe_kv_compact(K, *args, F, NUL) == M.MOE_ERR_ARG, args
    # outputs over other inputs, or an input shifted
    for table, ref in ((0x10004, 0x80000), (0x40000, 0x80000), (0x20000, 0x80000),
                       (0x80000, 0x40004), (0x80000, 0x10000), (0x80000, 0x20004),
                       (0x80000, 0x80010)):
        assert lib.moe_kv_compact(K, C.c_void_p(table), C.c_void_p(ref), F, F, F,
                                  NUL) == M.MOE_ERR_ARG, (table, ref)


def test_copy_arguments_are_refused():
    def call(n=1, k=F, v=F, moves=F, ws=NUL, **kw):
        base = dict(H=32, H_kv=4, dh=128, dtype=M.MOE_DTYPE_BF16, page_size=16, n_pages=100,
                    max_pages=10, stride_page=8192, stride_tok=512, stride_head=128, window=0,
                    sink_tokens=0, scale=0.1)
        base.update(kw)
        return M.lib().moe_kv_copy_pages(C.byref(M.CacheDesc(**base)), k, v, moves, n, NUL, ws, NUL)
    for kw in (dict(n=-1), dict(k=NUL), dict(v=ODD), dict(moves=NUL), dict(ws=ODD), dict(dh=12),
               dict(stride_tok=4)):
        assert call(**kw) == M.MOE_ERR_ARG, kw
    assert call(page_size=1 << 28, max_pages=1, H_kv=4, stride_page=1 << 36) == M.MOE_ERR_UNSUPPORTED
    assert call(n=0, k=NUL) == M.MOE_OK


def test_binding_refuses_other_tensors():
    i32 = torch.int32
    with pytest.raises(ValueError, match="logits are"):
        M.moe_sample(torch.zeros(2, 8, dtype=torch.float16), torch.zeros(2), torch.zeros(2, dtype=i32))
    with pytest.raises(ValueError, match="side by side"):
        M.moe_sample(torch.zeros(8, 2).T, torch.zeros(2), torch.zeros(2, dtype=i32))
    with pytest.raises(ValueError, match="u has shape"):
        M.moe_sample(torch.zeros(2, 8), torch.zeros(3), torch.zeros(2, dtype=i32))
    with pytest.raises(ValueError, match="temperature has shape"):
        M.moe_sample(torch.zeros(4, 8), torch.zeros(4), torch.zeros(4, dtype=i32),
                     temperature=torch.ones(4), param_rows=2)
    with pytest.raises(ValueError, match="param_rows"):
        M.moe_sample(torch.zeros(2, 8), torch.zeros(2), torch.zeros(2, dtype=i32), param_rows=0)
    with pytest.raises(ValueError, match="CUDA device"):
        M.moe_sample(torch.zeros(2, 8), torch.zeros(2), torch.zeros(2, dtype=i32))
    t = torch.zeros(3, 4, dtype=i32)
    K = M.page_book(t, t[:, 0].contiguous(), t[:, 1].contiguous(), torch.zeros(9, dtype=i32), 16)
    assert (K.B, K.max_pages, K.n_pages) == (3, 4, 9)
    ws = M.pages_workspace(K)
    with pytest.raises(ValueError, match="moves has shape"):
        M.moe_kv_fork(K, t[:2, 0].contiguous(), t[:2, 1].contiguous(), t, ws)
    with pytest.raises(ValueError, match="workspace"):
        M.moe_kv_reserve(K, 1, ws[:100])
    with pytest.raises(ValueError, match="needs a workspace"):
        M.moe_kv_reserve(K, 1, None)
    with pytest.raises(ValueError, match="int64"):
        M.page_book(t.long(), t[:, 0].contiguous(), t[:, 1].contiguous(), t[0], 16)
    L = M.layer_desc(64, 4, 2, 32, "fp32")
    x = torch.zeros(2, 64)
    w = torch.zeros(4, 32, 64)
    with pytest.raises(ValueError, match="W_down has shape"):
        M.moe_few_forward(L, x, torch.zeros(4, 64), w, w, w, None, x, None)
    with pytest.raises(ValueError, match="needs a workspace"):
        M.moe_few_forward(L, x, torch.zeros(4, 64), w, w, torch.zeros(4, 64, 32), None, x, None)
    with pytest.raises(ValueError, match="path has shape"):
        M.moe_tree_accept(t[0], None, t[0], 1, 4, t, t[0])
