"""Refusals of the paged append and the dense attention that were missing, and
calls that were refused without a reason, on the host (CPU only; addresses are
never dereferenced)."""
import ctypes

import pytest
import torch

import block_sparse_attention_22_b200 as qsa
from dense_testlib import D, shape


def _z(*s, dtype=torch.bfloat16):
    return torch.zeros(s, dtype=dtype)


def test_tensors_of_the_host_are_refused():
    """Shapes and dtypes fit, but the kernels would take the host's addresses."""
    cfg = qsa.make_config(shape())
    pages = qsa.make_pages(_z(4, 2, 16, D), _z(4, 2, 16, D), _z(1, 4, dtype=torch.int32))
    segs = qsa.make_segments([(0, 3, 0, 0)])
    q, o, k, v, g = _z(3, 24, D), _z(3, 24, D), _z(3, 2, D), _z(3, 2, D), _z(3, 24, D)
    lse, ws = _z(3, 24, dtype=torch.float32), _z(1 << 20, dtype=torch.uint8)
    for call in (lambda: qsa.qsa_append_kv(cfg, pages, segs, 3, k, v),
                 lambda: qsa.qsa_append_kv(cfg, pages, segs, 3, k, v, q, o),
                 lambda: qsa.qsa_paged_attn_fwd(cfg, pages, segs, 3, q, o, lse, ws),
                 lambda: qsa.qsa_prompt_attn_fwd(cfg, segs, 3, q, k, v, o, lse, ws),
                 lambda: qsa.qsa_prompt_attn_bwd(cfg, segs, 3, q, k, v, o, lse, g, _z(3, 24, D), _z(3, 2, D),
                                                 _z(3, 2, D), ws)):
        with pytest.raises(ValueError, match="not on a GPU"):
            call()


BASE = 1 << 40                # fake addresses, far from each other unless a test moves one; no call here may be valid


@pytest.mark.parametrize("dtype,row", [("bf16", 512), ("f32", 1024)])
def test_outputs_that_share_memory_with_another_array_are_refused(dtype, row):
    """Ranges of 8 tokens of 24 heads or 2 groups; `row` bytes of a head."""
    cfg = qsa.make_config(shape(dtype=dtype))
    lib, T = qsa.get_lib(), 8
    arr, n = qsa.make_segments([(0, T, 0, 0)])
    at = {name: BASE + (i << 32) for i, name in enumerate(("q", "k", "v", "o", "lse", "dout", "dq", "dk", "dv", "ws"))}
    q_end, kv_end = T * 24 * row, T * 2 * row

    def paged(**move):
        a = dict(at, **move)
        pages = qsa.qsa_pages_t(a["k"], a["v"], BASE - 4096, 4, 16, 1, 4)
        return lib.qsa_paged_attn_fwd(ctypes.byref(cfg), ctypes.byref(pages), arr, n, T, a["q"], a["o"], a["lse"],
                                      a["ws"], 1 << 31, None)

    def prompt(**move):
        a = dict(at, **move)
        return lib.qsa_prompt_attn_fwd(ctypes.byref(cfg), arr, n, T, a["q"], a["k"], a["v"], a["o"], a["lse"], a["ws"],
                                       1 << 31, None)

    def bwd(**move):
        a = dict(at, **move)
        return lib.qsa_prompt_attn_bwd(ctypes.byref(cfg), arr, n, T, *(a[x] for x in (
            "q", "k", "v", "o", "lse", "dout", "dq", "dk", "dv", "ws")), 1 << 31, None)

    bad = qsa.QSA_ERR_INVALID_ARG
    for call in (paged, prompt):
        assert call(o=at["q"]) == bad and call(o=at["q"] + q_end - 16) == bad and call(o=at["q"] - q_end + 16) == bad
        assert call(o=at["k"]) == bad and call(o=at["v"] + kv_end - 16) == bad
        assert call(lse=at["q"] + 64) == bad and call(lse=at["o"] + q_end - 4) == bad and call(lse=at["k"]) == bad
    assert paged(o=at["v"] + 4 * 2 * 16 * row - 16) == bad              # the last row of the last page
    for out, end in (("dq", q_end), ("dk", kv_end), ("dv", kv_end)):
        for other in ("q", "k", "v", "o", "lse", "dout", "dq", "dk", "dv"):
            if other != out:
                assert bwd(**{out: at[other]}) == bad and bwd(**{out: at[other] - end + 16}) == bad, (out, other)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("page,n_pages", [(16, (2 ** 31 - 256) // 32), (16, (2 ** 31 - 512 + 32) // 32), (2 ** 30 - 16, 1)])
def test_caches_whose_rows_leave_no_room_for_a_box_are_unsupported(dtype, page, n_pages):
    """Refused as what they are, not by the failure of a tensor map."""
    cfg = qsa.make_config(shape(dtype=dtype))
    arr, n = qsa.make_segments([(0, 8, 0, 0)])
    assert 2 ** 31 - 512 <= n_pages * 2 * page < 2 ** 31
    pages = qsa.qsa_pages_t(BASE, BASE << 1, BASE - 4096, n_pages, page, 1, 1)
    assert qsa.get_lib().qsa_paged_attn_fwd(ctypes.byref(cfg), ctypes.byref(pages), arr, n, 8, BASE + 4096, BASE + (1 << 30),
                                            None, None, 0, None) == qsa.QSA_ERR_UNSUPPORTED
    assert qsa.get_lib().qsa_append_kv(ctypes.byref(cfg), ctypes.byref(pages), arr, n, 8, BASE, 512, BASE, 512, None, 0, None,
                                       None) == qsa.QSA_ERR_UNSUPPORTED


def test_a_rotation_of_all_dims_is_not_held_to_the_indexers_limit():
    """idx_dim 128 in bf16: the indexer rotates at most 64 dims, the append any number
    of the head's.  Calls that are refused later, or do nothing, show what the
    configuration's check says."""
    sh = shape(rope_fraction=1.0)
    sh.idx_dim = 128
    cfg = qsa.make_config(sh)
    lib = qsa.get_lib()
    one, none = qsa.make_segments([(0, 8, 0, 0)]), qsa.make_segments([])
    pages = qsa.qsa_pages_t(BASE, BASE << 1, BASE - 4096, 4, 16, 1, 4)
    assert lib.qsa_append_kv(ctypes.byref(cfg), ctypes.byref(pages), *none, 0, BASE, 512, BASE, 512, None, 0, None,
                             None) == qsa.QSA_OK
    assert lib.qsa_paged_attn_fwd(ctypes.byref(cfg), ctypes.byref(pages), *none, 0, BASE, BASE, None, None, 0,
                                  None) == qsa.QSA_OK
    for op in (qsa.QSA_OP_PAGED_ATTN, qsa.QSA_OP_PROMPT_ATTN, qsa.QSA_OP_PROMPT_ATTN_BWD):
        assert qsa.workspace_size(cfg, one, 8, op) < 1 << 40
    assert qsa.workspace_size(cfg, one, 8, qsa.QSA_OP_FORWARD) == ctypes.c_size_t(-1).value
    assert lib.qsa_prompt_attn_fwd(ctypes.byref(cfg), *none, 0, BASE, BASE, BASE, BASE, None, None, 0,
                                   None) == qsa.QSA_OK
    assert lib.qsa_prompt_attn_bwd(ctypes.byref(cfg), *one, 8, *([BASE] * 9), None, 0, None) == qsa.QSA_ERR_WORKSPACE


def test_strides_of_dims_of_size_one_are_not_looked_at():
    """One group's [1, T, D] array seen as [T, 1, D], and one token cut from a longer row."""
    assert qsa._token_stride("append", "k", _z(1, 5, D).transpose(0, 1)) == D
    assert qsa._token_stride("append", "k", _z(1, 2 * D + 3)[:, :2 * D].view(1, 2, D)) == 2 * D
    assert qsa._token_stride("append", "k", _z(4, 2 * D + 8)[:, :2 * D].view(4, 2, D)) == 2 * D + 8
    for bad in (_z(5, 2, 2 * D)[..., ::2], _z(2, 5, D).transpose(0, 1), _z(5, 4, D)[:, ::2]):
        with pytest.raises(ValueError):
            qsa._token_stride("append", "k", bad)
