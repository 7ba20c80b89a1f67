"""Refusals of the operators' C entry points and wrappers (no GPU needed).

Every call here returns before any CUDA call: its arguments are refused. The
pointers are addresses of host memory that nothing reads.
"""
import ctypes
import math

import pytest


@pytest.fixture(scope="module")
def mx():
    from muon_adamw_hybrid_grad_gb300 import build

    build.build()
    import muon_adamw_hybrid_grad_gb300 as m

    m.load_library()
    return m


BUF = ctypes.create_string_buffer(4096 + 256)
AT = (ctypes.addressof(BUF) + 255) // 256 * 256


def refused(mx, name, status, *args):
    lib = mx.load_library()
    got = getattr(lib, name)(*args)
    assert got == status, (got, lib.muon_adamw_last_error())
    assert lib.muon_adamw_last_error()


def embed_args(**kw):
    a = dict(weight=AT, wdt=0, ws=16, vocab=10, width=16, ids=AT, idb=8, n=4, scale=1.0, out=AT, odt=1, os=16)
    a.update(kw)
    return (a["weight"], a["wdt"], a["ws"], a["vocab"], a["width"], a["ids"], a["idb"], a["n"], a["scale"], a["out"],
            a["odt"], a["os"], None)


@pytest.mark.parametrize("kw,status", [
    ({"weight": None}, "ARG"), ({"ids": None}, "ARG"), ({"out": None}, "ARG"), ({"idb": 2}, "ARG"),
    ({"scale": math.nan}, "ARG"), ({"scale": math.inf}, "ARG"), ({"wdt": 2}, "DTYPE"), ({"odt": -1}, "DTYPE"),
    ({"vocab": 0}, "SHAPE"), ({"width": 0}, "SHAPE"), ({"width": 2 ** 20 + 1, "ws": 2 ** 21, "os": 2 ** 21}, "SHAPE"),
    ({"n": -1}, "SHAPE"), ({"ws": 15}, "SHAPE"), ({"os": 8}, "SHAPE"), ({"weight": AT + 2}, "ALIGN"),
    ({"out": AT + 1}, "ALIGN"), ({"ids": AT + 4}, "ALIGN")])
def test_embedding_refuses(mx, kw, status):
    refused(mx, "muon_adamw_embedding", getattr(mx, "MA_ERR_" + status), *embed_args(**kw))


def embed_back_args(**kw):
    a = dict(dout=AT, ddt=1, ds=16, ids=AT, idb=4, n=4, scale=1.0, grad=AT, gdt=0, gs=16, vocab=10, width=16, acc=0,
             ws=AT, wsb=1 << 20)
    a.update(kw)
    return (a["dout"], a["ddt"], a["ds"], a["ids"], a["idb"], a["n"], a["scale"], a["grad"], a["gdt"], a["gs"],
            a["vocab"], a["width"], a["acc"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,status", [
    ({"dout": None}, "ARG"), ({"grad": None}, "ARG"), ({"ids": None}, "ARG"), ({"acc": 2}, "ARG"), ({"ws": None}, "ARG"),
    ({"wsb": 100}, "ARG"), ({"ws": AT + 16}, "ALIGN"), ({"gdt": 3}, "DTYPE"), ({"ddt": 9}, "DTYPE"),
    ({"gs": 4}, "SHAPE"), ({"ds": 4}, "SHAPE"), ({"vocab": 2 ** 31}, "SHAPE"), ({"grad": AT + 2}, "ALIGN")])
def test_embedding_backward_refuses(mx, kw, status):
    refused(mx, "muon_adamw_embedding_backward", getattr(mx, "MA_ERR_" + status), *embed_back_args(**kw))


def test_embedding_backward_workspace(mx):
    lib, n = mx.load_library(), ctypes.c_int64()
    assert lib.muon_adamw_embedding_backward_workspace(1000, 50, 64, ctypes.byref(n)) == 0
    assert n.value >= 1000 * 16
    refused(mx, "muon_adamw_embedding_backward_workspace", mx.MA_ERR_ARG, 1000, 50, 64, None)
    refused(mx, "muon_adamw_embedding_backward_workspace", mx.MA_ERR_SHAPE, -1, 50, 64, ctypes.byref(n))


def qk(mx, **kw):
    a = dict(n_tokens=4, n_heads=2, n_kv_heads=1, head_dim=64, rot_dim=64, dtype=1, neighbours=0, position_bytes=4,
             reserved=0, eps=1e-6, q=AT, k=AT, q_token_stride=192, q_head_stride=64, k_token_stride=192,
             k_head_stride=64, q_weight=AT, k_weight=AT, cos_table=AT, sin_table=AT, table_rows=8, positions=AT)
    a.update(kw)
    return ctypes.byref(mx.QkNormRope(**a))


@pytest.mark.parametrize("kw,status", [
    ({"n_tokens": -1}, "SHAPE"), ({"n_heads": -1}, "SHAPE"), ({"n_heads": 0, "n_kv_heads": 0}, "SHAPE"),
    ({"head_dim": 60}, "SHAPE"), ({"head_dim": 264}, "SHAPE"), ({"rot_dim": 72}, "SHAPE"), ({"rot_dim": 80}, "SHAPE"),
    ({"rot_dim": -16}, "SHAPE"), ({"table_rows": 0}, "SHAPE"), ({"dtype": 2}, "DTYPE"), ({"neighbours": 2}, "ARG"),
    ({"position_bytes": 2}, "ARG"), ({"eps": -1.0}, "ARG"), ({"eps": math.nan}, "ARG"), ({"q": None}, "ARG"),
    ({"k": None}, "ARG"), ({"q_weight": None}, "ARG"), ({"cos_table": None}, "ARG"), ({"positions": None}, "ARG"),
    ({"q": AT + 8}, "ALIGN"), ({"q_token_stride": 196}, "ALIGN"), ({"k_head_stride": 65}, "ALIGN"),
    ({"k_weight": AT + 4}, "ALIGN"), ({"sin_table": AT + 8}, "ALIGN"), ({"positions": AT + 2}, "ALIGN")])
def test_qk_norm_rope_refuses(mx, kw, status):
    want = getattr(mx, "MA_ERR_" + status)
    refused(mx, "muon_adamw_qk_norm_rope", want, qk(mx, **kw), AT, AT, None)
    refused(mx, "muon_adamw_qk_norm_rope_backward", want, qk(mx, **kw), AT, 128, 64, AT, 64, 64, AT, AT, AT, AT, AT,
            1 << 30, None)


def test_qk_norm_rope_refuses_outputs(mx):
    for name in ("muon_adamw_qk_norm_rope",):
        refused(mx, name, mx.MA_ERR_ARG, None, AT, AT, None)
        refused(mx, name, mx.MA_ERR_ARG, qk(mx), None, AT, None)
        refused(mx, name, mx.MA_ERR_ALIGN, qk(mx), AT, AT + 4, None)
    name = "muon_adamw_qk_norm_rope_backward"
    ok = [qk(mx), AT, 128, 64, AT, 64, 64, AT, AT, AT, AT, AT, 1 << 30, None]
    for i, x, status in ((1, None, mx.MA_ERR_ARG), (1, AT + 2, mx.MA_ERR_ALIGN), (2, 130, mx.MA_ERR_ALIGN),
                         (4, None, mx.MA_ERR_ARG), (7, None, mx.MA_ERR_ARG), (8, AT + 8, mx.MA_ERR_ALIGN),
                         (9, None, mx.MA_ERR_ARG), (10, AT + 2, mx.MA_ERR_ALIGN)):
        bad = list(ok)
        bad[i] = x
        refused(mx, name, status, *bad)


def attn(mx, **kw):
    a = dict(n_tokens=4, n_heads=4, n_kv_heads=2, head_dim=64, sinks=1, window=2, scale=0.1, cu_seqlens=AT, n_seqs=1,
             reserved=0, q=AT, k=AT, v=AT, q_token_stride=256, q_head_stride=64, k_token_stride=128, k_head_stride=64,
             v_token_stride=128, v_head_stride=64)
    a.update(kw)
    return ctypes.byref(mx.WindowAttention(**a))


@pytest.mark.parametrize("kw,status", [
    ({"n_tokens": -1}, "SHAPE"), ({"n_heads": 0}, "SHAPE"), ({"n_kv_heads": 0}, "SHAPE"), ({"n_heads": 5}, "SHAPE"),
    ({"head_dim": 60}, "SHAPE"), ({"head_dim": 136}, "SHAPE"), ({"head_dim": 0}, "SHAPE"), ({"window": -1}, "ARG"),
    ({"sinks": -1}, "ARG"), ({"sinks": 129}, "ARG"), ({"scale": math.inf}, "ARG"), ({"n_seqs": 0}, "ARG"),
    ({"cu_seqlens": AT + 2}, "ALIGN"), ({"q": None}, "ARG"), ({"k": None}, "ARG"), ({"v": None}, "ARG"),
    ({"q": AT + 8}, "ALIGN"), ({"k_token_stride": 132}, "ALIGN"), ({"v_head_stride": 60}, "ALIGN")])
def test_window_attention_refuses(mx, kw, status):
    want = getattr(mx, "MA_ERR_" + status)
    refused(mx, "muon_adamw_window_attention", want, attn(mx, **kw), AT, AT, None)
    refused(mx, "muon_adamw_window_attention_backward", want, attn(mx, **kw), AT, 256, 64, AT, AT, AT, AT, AT, AT,
            1 << 30, None)


@pytest.mark.parametrize("kw,status", [
    ({"out_token_stride": 132, "out_head_stride": 64}, "ALIGN"), ({"out_token_stride": 256, "out_head_stride": 60}, "ALIGN"),
    ({"out_token_stride": 256, "out_head_stride": 56}, "SHAPE"), ({"out_token_stride": 56, "out_head_stride": 64}, "SHAPE")])
def test_window_attention_refuses_output_strides(mx, kw, status):
    refused(mx, "muon_adamw_window_attention_backward", getattr(mx, "MA_ERR_" + status), attn(mx, **kw), AT, 256, 64, AT,
            AT, AT, AT, AT, AT, 1 << 30, None)


def test_window_attention_refuses_outputs(mx):
    name = "muon_adamw_window_attention"
    refused(mx, name, mx.MA_ERR_ARG, None, AT, AT, None)
    refused(mx, name, mx.MA_ERR_ARG, attn(mx), None, AT, None)
    refused(mx, name, mx.MA_ERR_ARG, attn(mx), AT, None, None)
    refused(mx, name, mx.MA_ERR_ALIGN, attn(mx), AT + 8, AT, None)
    name = "muon_adamw_window_attention_backward"
    ok = [attn(mx), AT, 256, 64, AT, AT, AT, AT, AT, AT, 1 << 30, None]
    for i, x, status in ((1, None, mx.MA_ERR_ARG), (2, 100, mx.MA_ERR_ALIGN), (4, None, mx.MA_ERR_ARG),
                         (5, AT + 2, mx.MA_ERR_ALIGN), (6, None, mx.MA_ERR_ARG), (7, AT + 2, mx.MA_ERR_ALIGN),
                         (8, None, mx.MA_ERR_ARG), (9, None, mx.MA_ERR_ARG), (9, AT + 16, mx.MA_ERR_ALIGN),
                         (10, 8, mx.MA_ERR_ARG)):
        bad = list(ok)
        bad[i] = x
        refused(mx, name, status, *bad)


def test_wrappers_refuse_cpu_tensors(mx):
    torch = pytest.importorskip("torch")
    from muon_adamw_hybrid_grad_gb300 import ops

    w, ids = torch.zeros(4, 16), torch.zeros(3, dtype=torch.int64)
    x = torch.zeros(3, 2, 16, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        ops.embedding(w, ids)
    with pytest.raises(ValueError, match="CUDA"):
        ops.embedding_backward(torch.zeros(3, 16), ids, w)
    with pytest.raises(ValueError, match="CUDA"):
        ops.qk_norm_rope(x, x, w, w, w, w, ids)
    with pytest.raises(ValueError, match="CUDA"):
        ops.window_attention(x, x, x, window=1)
