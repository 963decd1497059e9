"""Refusals of the paged append and the dense attention, on the host before
any CUDA call (CPU only; addresses are never dereferenced)."""
import ctypes

import pytest
import torch

import block_sparse_attention_22_b200 as qsa
from dense_testlib import D, shape

P16 = 16                  # a fake, aligned address


def _pages(**kw):
    f = dict(k=P16, v=P16, table=P16, n_pages=100, page_tokens=64, n_rows=3, max_pages=10)
    f.update(kw)
    return qsa.qsa_pages_t(f["k"], f["v"], f["table"], f["n_pages"], f["page_tokens"], f["n_rows"], f["max_pages"])


def _append(cfg=None, pages=None, segs=((0, 8, 0, 0),), T=8, k=P16, ld_k=512, v=P16, ld_v=512, q=None, ld_q=0,
            q_out=None):
    cfg = cfg or qsa.make_config(shape())
    pages = pages or _pages()
    arr, n = qsa.make_segments(segs)
    return qsa.get_lib().qsa_append_kv(ctypes.byref(cfg), ctypes.byref(pages), arr, n, T, k, ld_k, v, ld_v, q, ld_q,
                                       q_out, None)


def _paged(cfg=None, pages=None, segs=((0, 8, 0, 0),), T=8, q=P16, o=P16, lse=None, ws=None, ws_bytes=0):
    cfg = cfg or qsa.make_config(shape())
    pages = pages or _pages()
    arr, n = qsa.make_segments(segs)
    return qsa.get_lib().qsa_paged_attn_fwd(ctypes.byref(cfg), ctypes.byref(pages), arr, n, T, q, o, lse, ws, ws_bytes,
                                            None)


def _prompt(cfg=None, segs=((0, 8, 0, 0),), T=8, q=P16, k=P16, v=P16, o=P16, lse=None, ws=None, ws_bytes=0):
    cfg = cfg or qsa.make_config(shape())
    arr, n = qsa.make_segments(segs)
    return qsa.get_lib().qsa_prompt_attn_fwd(ctypes.byref(cfg), arr, n, T, q, k, v, o, lse, ws, ws_bytes, None)


def _prompt_bwd(cfg=None, segs=((0, 8, 0, 0),), T=8, ws=P16, ws_bytes=1 << 30, **kw):
    a = dict(q=P16, k=P16, v=P16, o=P16, lse=P16, dout=P16, dq=P16, dk=P16, dv=P16)
    a.update(kw)
    cfg = cfg or qsa.make_config(shape())
    arr, n = qsa.make_segments(segs)
    return qsa.get_lib().qsa_prompt_attn_bwd(ctypes.byref(cfg), arr, n, T, a["q"], a["k"], a["v"], a["o"], a["lse"],
                                             a["dout"], a["dq"], a["dk"], a["dv"], ws, ws_bytes, None)


@pytest.mark.parametrize("call", [_append, _paged, _prompt, _prompt_bwd])
def test_configurations_are_checked(call):
    cfg = qsa.make_config(shape())
    cfg.head_dim = 128
    assert call(cfg=cfg) == qsa.QSA_ERR_UNSUPPORTED
    cfg = qsa.make_config(shape())
    cfg.dtype = 5
    assert call(cfg=cfg) == qsa.QSA_ERR_INVALID_ARG


@pytest.mark.parametrize("call", [_append, _paged])
@pytest.mark.parametrize("field,value,status", [
    ("k", None, qsa.QSA_ERR_INVALID_ARG), ("v", 24, qsa.QSA_ERR_INVALID_ARG), ("table", None, qsa.QSA_ERR_INVALID_ARG),
    ("table", 18, qsa.QSA_ERR_INVALID_ARG), ("n_pages", 0, qsa.QSA_ERR_INVALID_ARG),
    ("page_tokens", 0, qsa.QSA_ERR_INVALID_ARG), ("page_tokens", -16, qsa.QSA_ERR_INVALID_ARG),
    ("page_tokens", 24, qsa.QSA_ERR_UNSUPPORTED), ("n_rows", 0, qsa.QSA_ERR_INVALID_ARG),
    ("max_pages", 0, qsa.QSA_ERR_INVALID_ARG), ("n_pages", 1 << 30, qsa.QSA_ERR_UNSUPPORTED),
])
def test_page_tables_are_checked(call, field, value, status):
    assert call(pages=_pages(**{field: value})) == status


@pytest.mark.parametrize("call", [_append, _paged])
@pytest.mark.parametrize("seg", [(0, -1, 0, 0), (-1, 4, 0, 0), (4, 5, 0, 0), (0, 8, -1, 0), (0, 8, 633, 0),
                                 (0, 8, 0, 3), (0, 8, 0, -1), (0, 8, 2147483647, 0)])
def test_segments_are_checked(call, seg):
    assert call(segs=[seg]) == qsa.QSA_ERR_INVALID_ARG


@pytest.mark.parametrize("call", [_append, _paged, _prompt, _prompt_bwd])
def test_overlapping_segments_are_refused(call):
    for segs in ([(0, 4, 0, 0), (3, 4, 0, 1)], [(4, 4, 0, 0), (0, 5, 0, 1)], [(0, 8, 0, 0), (2, 1, 0, 1)],
                 [(0, 4, 0, 0), (0, 4, 0, 0)]):
        assert call(segs=segs) == qsa.QSA_ERR_INVALID_ARG, segs


@pytest.mark.parametrize("call", [_append, _paged, _prompt, _prompt_bwd])
def test_calls_without_tokens_do_nothing(call):
    assert call(segs=[], T=0) == qsa.QSA_OK
    assert call(segs=[(0, 0, 0, 0), (5, 0, 0, 1)]) == qsa.QSA_OK


def test_append_pointers_and_strides_are_checked():
    bad = qsa.QSA_ERR_INVALID_ARG
    assert _append(k=None) == bad and _append(v=None) == bad and _append(k=8) == bad and _append(v=24) == bad
    assert _append(ld_k=511) == bad and _append(ld_k=516) == bad and _append(ld_v=256) == bad
    assert _append(q=P16, ld_q=6144) == bad                       # q without q_out
    assert _append(q_out=P16) == bad
    assert _append(q=P16, ld_q=6143, q_out=32) == bad
    assert _append(q=P16, ld_q=6152, q_out=P16) == bad            # in place, but strided
    f32 = qsa.make_config(shape(dtype="f32"))
    assert _append(cfg=f32, ld_k=514) == bad


def test_attention_pointers_and_workspaces_are_checked():
    bad = qsa.QSA_ERR_INVALID_ARG
    assert _paged(q=None) == bad and _paged(o=None) == bad and _paged(q=8) == bad and _paged(lse=18) == bad
    assert _prompt(k=None) == bad and _prompt(v=8) == bad and _prompt(segs=[(0, 8, 4, 0)]) == bad
    for name in ("q", "k", "v", "o", "lse", "dout", "dq", "dk", "dv"):
        assert _prompt_bwd(**{name: None}) == bad, name
    assert _prompt_bwd(dk=8) == bad and _prompt_bwd(segs=[(0, 8, 1, 0)]) == bad
    assert _prompt_bwd(ws=None) == qsa.QSA_ERR_WORKSPACE and _prompt_bwd(ws_bytes=10) == qsa.QSA_ERR_WORKSPACE
    # one row over many keys is cut between CTAs: a workspace is needed
    long = dict(segs=[(0, 1, 600, 0)], pages=_pages())
    assert _paged(**long) == qsa.QSA_ERR_WORKSPACE
    assert _paged(**long, ws=P16, ws_bytes=16) == qsa.QSA_ERR_WORKSPACE
    assert _paged(**long, ws=24, ws_bytes=1 << 30) == bad


def test_workspace_sizes():
    cfg = qsa.make_config(shape())
    one = qsa.make_segments([(0, 1, 0, 0)])
    assert qsa.workspace_size(cfg, one, 1, qsa.QSA_OP_PAGED_ATTN) == 0           # one key: nothing to cut
    assert qsa.workspace_size(cfg, one, 5, qsa.QSA_OP_PROMPT_ATTN_BWD) >= 5 * 24 * 4
    none = qsa.make_segments([])
    for op in (qsa.QSA_OP_PAGED_ATTN, qsa.QSA_OP_PROMPT_ATTN, qsa.QSA_OP_PROMPT_ATTN_BWD):
        assert qsa.workspace_size(cfg, none, 0, op) == 0


def test_python_refuses_tensors_that_do_not_fit():
    cfg = qsa.make_config(shape())
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype)
    kp, table = z(4, 2, 16, D), z(1, 4, dtype=torch.int32)
    pages = qsa.make_pages(kp, z(4, 2, 16, D), table)
    with pytest.raises(ValueError):
        qsa.make_pages(kp, z(4, 2, 32, D), table)
    with pytest.raises(ValueError):
        qsa.make_pages(kp, z(4, 2, 16, D), table.long())
    with pytest.raises(ValueError):
        qsa.make_pages(z(2, 4, 16, D).transpose(0, 1), z(4, 2, 16, D), table)
    segs = qsa.make_segments([(0, 3, 0, 0)])
    q, k, o = z(3, 24, D), z(3, 2, D), z(3, 24, D)
    f32 = torch.float32
    for bad in (dict(q=z(2, 24, D)), dict(q=z(3, 16, D)), dict(q=q.float()), dict(lse=z(3, 24)), dict(o=z(3, 24, 512))):
        a = dict(q=q, o=o, lse=None)
        a.update(bad)
        with pytest.raises(ValueError):
            qsa.qsa_paged_attn_fwd(cfg, pages, segs, 3, **a)
    with pytest.raises(ValueError):
        qsa.qsa_paged_attn_fwd(cfg, pages, segs, 3, z(3, 48, D)[:, ::2], o)
    with pytest.raises(ValueError):
        qsa.qsa_prompt_attn_fwd(cfg, segs, 3, q, z(3, 24, D), k, o)
    with pytest.raises(ValueError):
        qsa.qsa_prompt_attn_bwd(cfg, segs, 3, q, k, k, o, z(3, 24, dtype=f32), q, q, k.float(), k)
    with pytest.raises(ValueError):
        qsa.qsa_append_kv(cfg, pages, segs, 3, z(3, 4, D)[:, ::2], k)
    with pytest.raises(ValueError):
        qsa.qsa_append_kv(cfg, pages, segs, 3, k, z(2, 2, D))
