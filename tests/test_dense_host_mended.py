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
