"""Checks of the attention half's entry points that need no GPU: workspace sizes, and bad
arguments refused by the library (before any CUDA call) and by the binding."""
import ctypes as C

import pytest
import torch

from expert_select_gb300 import build as B
from expert_select_gb300 import moetree as M


@pytest.fixture(scope="module", autouse=True)
def built():
    B.build()


def _desc(**kw):
    base = dict(H=32, H_kv=4, dh=128, dtype=M.MOE_DTYPE_BF16, page_size=16, n_pages=100,
                max_pages=10, stride_page=8192, stride_tok=512, stride_head=128, window=0,
                sink_tokens=0, scale=0.1)
    base.update(kw)
    return M.CacheDesc(**base)


BAD_DESCS = [dict(H_kv=0), dict(H=30), dict(H=2), dict(dh=0), dict(dh=12), dict(dh=264),
             dict(dtype=2), dict(page_size=0), dict(n_pages=0), dict(max_pages=0),
             dict(page_size=1 << 16, max_pages=1 << 15), dict(stride_tok=120),
             dict(stride_head=132), dict(stride_page=0), dict(window=-1), dict(sink_tokens=-1),
             dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
             dict(scale=float("inf"))]


def test_workspace_bytes():
    a = M.moe_attention_workspace_bytes(_desc(), 1, 1)
    b = M.moe_attention_workspace_bytes(_desc(), 1, 65)
    assert 4096 < a <= b and a % 256 == 0
    assert M.moe_attention_workspace_bytes(_desc(), 0, 1) == 0
    assert M.moe_attention_workspace_bytes(_desc(), 1, 0) == 0
    assert M.moe_attention_workspace_bytes(_desc(), 1, 1 << 29) == 0


@pytest.mark.parametrize("bad", BAD_DESCS, ids=lambda d: "-".join(f"{k}={v}" for k, v in d.items()))
def test_bad_cache_descriptions_are_refused(bad):
    C_ = _desc(**bad)
    f, nul = C.c_void_p(0x100000), None  # never dereferenced: the description fails first
    lib = M.lib()
    assert M.moe_attention_workspace_bytes(C_, 1, 1) == 0
    assert lib.moe_tree_attention(C.byref(C_), f, 4096, f, f, f, f, nul, nul, nul, 1, 1, 1, f, nul,
                                  f, nul) == M.MOE_ERR_ARG
    P = M.RopeParams(None, None, 1e-6, None, 0, 1.0)
    assert lib.moe_kv_append(C.byref(C_), C.byref(P), f, 4096, f, 512, f, 512, f, f, f, f, nul,
                             nul, 1, 1, 1, f, nul, nul) == M.MOE_ERR_ARG
    assert lib.moe_kv_commit(C.byref(C_), f, f, f, f, f, f, 1, 1, f, nul, nul) == M.MOE_ERR_ARG


def test_attention_arguments_are_refused():
    lib, C_ = M.lib(), _desc()
    f, odd, nul = C.c_void_p(0x100000), C.c_void_p(0x100008), None

    def call(q=f, ldq=4096, k=f, v=f, table=f, lens=f, start=nul, B_=1, N=1, R=1, out=f, ws=f):
        return lib.moe_tree_attention(C.byref(C_), q, ldq, k, v, table, lens, start, nul, nul, B_,
                                      N, R, out, nul, ws, nul)
    for kw in (dict(q=nul), dict(q=odd), dict(ldq=4088), dict(ldq=4100), dict(k=nul), dict(k=odd),
               dict(v=odd), dict(table=nul), dict(lens=nul), dict(out=nul), dict(out=odd),
               dict(ws=nul), dict(ws=odd), dict(B_=-1), dict(N=-1), dict(R=-1), dict(R=2),
               dict(B_=2, N=3, R=5), dict(N=1 << 28, R=1 << 28)):
        assert call(**kw) == M.MOE_ERR_ARG, kw
    assert lib.moe_tree_attention(nul, f, 4096, f, f, f, f, nul, nul, nul, 1, 1, 1, f, nul, f,
                                  nul) == M.MOE_ERR_ARG
    # more (sequence, block of rows) pairs than are counted
    assert call(B_=1 << 25, N=1 << 12, R=8, start=f) == M.MOE_ERR_UNSUPPORTED
    # an output over its queries: the same rows, the last one's end, a wider row's gap
    base = 0x100000
    for kw in (dict(), dict(R=2, N=2, out=C.c_void_p(base + 8192 + 8176)),
               dict(R=2, N=2, ldq=3 * 4096, out=C.c_void_p(base + 8192)),
               dict(q=C.c_void_p(base + 8176))):
        assert call(**kw) == M.MOE_ERR_ARG, kw
    # nothing to do is fine
    assert call(B_=0, N=5, R=0, q=nul) == M.MOE_OK
    assert call(B_=3, N=0, R=0, q=nul) == M.MOE_OK


def test_append_and_commit_arguments_are_refused():
    lib, C_ = M.lib(), _desc()
    f, g, odd, nul = C.c_void_p(0x100000), C.c_void_p(0x200000), C.c_void_p(0x100008), None

    def append(P=M.RopeParams(None, None, 1e-6, None, 0, 1.0), q=f, ldq=4096, k=f, ldk=512, v=f,
               ldv=512, kp=f, vp=f, table=f, lens=f, q_out=g, ws=nul, R=1):
        return lib.moe_kv_append(C.byref(C_), C.byref(P) if P else nul, q, ldq, k, ldk, v, ldv, kp,
                                 vp, table, lens, nul, nul, 1, 1, R, q_out, ws, nul)
    rope = lambda **kw: M.RopeParams(**{**dict(q_weight=None, k_weight=None, eps=1e-6,
                                               inv_freq=0x100000, rot_dim=128, rope_scale=1.0),
                                        **kw})
    for kw in (dict(P=None), dict(q=nul), dict(q_out=nul), dict(q=odd), dict(ldq=4088),
               dict(q=f, q_out=f, ldq=5120), dict(k=nul), dict(ldk=504), dict(v=odd),
               dict(ldv=516), dict(kp=nul), dict(vp=odd), dict(table=nul), dict(lens=nul),
               dict(ws=odd), dict(R=2), dict(P=rope(rot_dim=0)), dict(P=rope(rot_dim=6)), dict(P=rope(rot_dim=12)),
               dict(P=rope(rot_dim=132)), dict(P=rope(rope_scale=float("inf"))),
               dict(P=rope(eps=-1.0)), dict(P=rope(eps=float("nan"))),
               dict(P=rope(q_weight=0x100008)), dict(P=rope(k_weight=0x100002))):
        assert append(**kw) == M.MOE_ERR_ARG, kw

    def commit(kp=f, vp=f, table=f, lens=f, path=f, acc=f, B_=1, P=1, new=f, ws=nul):
        return lib.moe_kv_commit(C.byref(C_), kp, vp, table, lens, path, acc, B_, P, new, ws, nul)
    for kw in (dict(kp=nul), dict(vp=odd), dict(table=nul), dict(lens=nul), dict(path=nul),
               dict(acc=nul), dict(B_=-1), dict(P=-1), dict(new=nul), dict(ws=odd)):
        assert commit(**kw) == M.MOE_ERR_ARG, kw
    assert commit(B_=0) == M.MOE_OK


def test_block_norm_arguments_are_refused():
    lib = M.lib()
    L = M.layer_desc(2048, 8, 1, 64, "bf16")
    f, g, odd, nul = C.c_void_p(0x100000), C.c_void_p(0x200000), C.c_void_p(0x100008), None

    def call(x=f, branch=f, post=nul, gate=nul, rows=0, scale=1.0, pre=nul, eps=1e-6, R=4, h=f,
             hn=g, L=L):
        return lib.moe_block_norm(C.byref(L), x, branch, post, gate, rows, scale, pre, eps, R, h,
                                  hn, nul)
    for kw in (dict(x=nul), dict(x=odd), dict(branch=odd), dict(post=odd), dict(pre=odd),
               dict(gate=odd, rows=1), dict(gate=f, rows=0), dict(h=nul), dict(h=nul, hn=nul),
               dict(hn=odd), dict(h=f, hn=f), dict(branch=nul, post=f), dict(branch=nul, gate=f,
                                                                             rows=1),
               dict(eps=-1e-6), dict(eps=float("nan")), dict(scale=float("nan")), dict(R=-1),
               dict(L=M.layer_desc(2047, 8, 1, 64, "bf16"))):
        assert call(**kw) == M.MOE_ERR_ARG, kw
    assert call(R=0, x=nul) == M.MOE_OK


def _host_pool(dtype=torch.bfloat16):
    return torch.zeros(6, 16, 4, 128, dtype=dtype)


def test_cache_desc_reads_strides_of_both_layouts():
    a = M.cache_desc(_host_pool(), 32, 10)
    assert (a.stride_page, a.stride_tok, a.stride_head) == (16 * 512, 512, 128)
    assert (a.n_pages, a.page_size, a.H_kv, a.dh, a.H) == (6, 16, 4, 128, 32)
    assert abs(a.scale - 128 ** -0.5) < 1e-7
    hm = torch.zeros(6, 4, 16, 128).permute(0, 2, 1, 3)
    b = M.cache_desc(hm, 4, 10, window=5, sink_tokens=2, scale=0.5)
    assert (b.stride_page, b.stride_tok, b.stride_head) == (4 * 16 * 128, 128, 16 * 128)
    assert (b.window, b.sink_tokens, b.scale, b.dtype) == (5, 2, 0.5, M.MOE_DTYPE_F32)
    one = M.cache_desc(torch.zeros(1, 1, 1, 8), 1, 1)
    assert min(one.stride_page, one.stride_tok, one.stride_head) >= 8
    with pytest.raises(ValueError):
        M.cache_desc(torch.zeros(2, 4, 2, 64, dtype=torch.float16), 4, 3)
    with pytest.raises(ValueError):
        M.cache_desc(torch.zeros(2, 4, 64, 2).transpose(2, 3), 4, 3)


@pytest.mark.parametrize("name,value", [
    ("q", torch.zeros(3, 32, 128)), ("q", torch.zeros(3, 31, 128, dtype=torch.bfloat16)),
    ("q", torch.zeros(3, 128, 32, dtype=torch.bfloat16).transpose(1, 2)),
    ("v", torch.zeros(6, 16, 4, 128)), ("v", torch.zeros(6, 4, 16, 128,
                                                         dtype=torch.bfloat16).transpose(1, 2)),
    ("table", torch.zeros(1, 10, dtype=torch.int64)), ("table", torch.zeros(1, 9,
                                                                            dtype=torch.int32)),
    ("lens", torch.zeros(2, dtype=torch.int32)), ("out", torch.zeros(3, 32, 128)),
    ("parent", torch.zeros(3, dtype=torch.int64)), ("parent", torch.zeros(2, dtype=torch.int32)),
    ("logit", torch.zeros(4)), ("lse", torch.zeros(3, 4)), ("ws", torch.zeros(64,
                                                                              dtype=torch.uint8)),
    ("ws", None),
])
def test_binding_refuses_wrong_tensors(name, value):
    t = dict(q=torch.zeros(3, 32, 128, dtype=torch.bfloat16), v=_host_pool(),
             table=torch.zeros(1, 10, dtype=torch.int32), lens=torch.zeros(1, dtype=torch.int32),
             out=torch.zeros(3, 32, 128, dtype=torch.bfloat16), parent=None, logit=None, lse=None,
             ws=torch.zeros(1 << 20, dtype=torch.uint8))
    t[name] = value
    k = _host_pool()
    with pytest.raises(ValueError):
        M.moe_tree_attention(M.cache_desc(k, 32, 10), t["q"], k, t["v"], t["table"], t["lens"], 1,
                             3, t["out"], t["ws"], parent=t["parent"], sink_logit=t["logit"],
                             lse=t["lse"])


def test_binding_refuses_wrong_norm_tensors():
    L = M.layer_desc(64, 8, 1, 64, "fp32")
    x, o = torch.zeros(5, 64), torch.zeros(5, 64)
    for kw in (dict(x=torch.zeros(5, 72)), dict(branch=torch.zeros(4, 64)),
               dict(h=o.bfloat16()), dict(w_pre=torch.zeros(5)),
               dict(gate=torch.zeros(2, 64), gate_rows=5), dict(gate=torch.zeros(2, 64)),
               dict(x=torch.zeros(64, 5).T)):
        args = dict(x=x, branch=o, h=o, hn=torch.zeros(5, 64))
        args.update(kw)
        with pytest.raises(ValueError):
            M.moe_block_norm(L, **args)
