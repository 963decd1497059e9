"""Calls of the paged append and the dense attention that once went wrong, or
could.  Bounds: dense_testlib."""
import math

import pytest
import torch

import block_sparse_attention_22_b200 as qsa
from dense_testlib import (D, F64, attend64, check_forward, fill_pages, make_table, score_error, shape, torch_dtype,
                           workspace)

pytestmark = pytest.mark.gpu
SCALE = 1.0 / math.sqrt(D)
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _need_cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _randn(gen, *size, dtype=BF):
    return torch.randn(size, generator=gen).to(dtype).cuda()


def _prompts(heads, groups, lens, seed=1, dtype="bf16"):
    sh = shape(heads, groups, dtype)
    gen = torch.Generator().manual_seed(seed)
    offs = [sum(lens[:i]) for i in range(len(lens))]
    x = dict(cfg=qsa.make_config(sh), T=sum(lens), lens=lens, offs=offs, dt=torch_dtype(sh),
             segs=qsa.make_segments([(o, n, 0, 0) for o, n in zip(offs, lens)]))
    for name, h in (("q", heads), ("dout", heads), ("k", groups), ("v", groups)):
        x[name] = _randn(gen, x["T"], h, D, dtype=x["dt"])
    return x


def _forward(x):
    o = torch.full_like(x["q"], 5.0)
    lse = torch.full(x["q"].shape[:2], 5.0, device="cuda")
    qsa.qsa_prompt_attn_fwd(x["cfg"], x["segs"], x["T"], x["q"], x["k"], x["v"], o, lse,
                            workspace(x["cfg"], x["segs"], x["T"], qsa.QSA_OP_PROMPT_ATTN))
    return o, lse


# ------------------------------------------------------------------ the lists of values that are not finite
@pytest.mark.parametrize("heads,groups,lens", [
    (8, 8, [256, 255, 129, 200, 1, 130, 2, 131] * 40),      # a head per group: up to 255 own keys a unit
    (12, 1, [21, 22, 43, 1, 2, 10, 64, 11] * 60),           # units of a token or two, of a chunk
    (4, 4, [128, 1, 1, 64, 127, 1] * 100),                  # single CTAs: lengths of at most 128
], ids=["256-row tiles", "few tokens", "single CTAs"])
def test_many_short_units_each_with_their_own_list(heads, groups, lens):
    """A CTA goes through several units of a chunk or two; the warp that checks
    their values neither falls behind nor runs over a list in use.  Values of
    some prompts' last tokens are infinite, so the lists differ."""
    x = _prompts(heads, groups, lens, seed=3)
    odd = range(0, len(lens), 7)
    for i in odd:
        x["v"][x["offs"][i] + lens[i] - 1, 0, i % D] = float("inf")
    first = _forward(x)
    for _ in range(5):
        for a, b in zip(_forward(x), first):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    qsa.qsa_device_status()
    o, lse = first
    hit = torch.zeros(o.shape, dtype=torch.bool, device="cuda")
    for i in odd:
        hit[x["offs"][i] + lens[i] - 1, :heads // groups, i % D] = True
    assert torch.equal(torch.isinf(o), hit) and bool(torch.isfinite(o[~hit].float()).all())
    for i in list(range(0, 14)) + list(range(len(lens) - 7, len(lens))):
        t = slice(x["offs"][i], x["offs"][i] + lens[i])
        v = torch.where(torch.isfinite(x["v"][t]), x["v"][t], 0)
        ref = list(attend64(x["q"][t], x["k"][t], v, 0, SCALE))
        ref[0] = torch.where(hit[t], 0.0, ref[0])
        check_forward(torch.where(hit[t], 0.0, o[t]), lse[t], ref, score_error(x["q"][t], x["k"][t], SCALE), BF, i)


@pytest.mark.parametrize("heads,groups", [(8, 8), (24, 2)])
def test_cut_chunks_without_own_keys_next_to_short_units(heads, groups):
    """Pieces that end before their unit's own keys have an empty list."""
    sh = shape(heads, groups)
    gen = torch.Generator().manual_seed(4)
    seqs = [(9000, 40), (5000, 300), (0, 130), (17, 2), (300, 5), (0, 20)]
    table, n_pages = make_table([c + n for c, n in seqs], 48, gen)
    kp, vp = (torch.full((n_pages, groups, 48, D), float("nan"), dtype=BF, device="cuda") for _ in range(2))
    offs, kv, segs, T = [], [], [], 0
    for i, (c, n) in enumerate(seqs):
        k, v = (_randn(gen, c + n, groups, D) for _ in range(2))
        fill_pages(kp, vp, table, 48, i, k, v)
        kv.append((k, v))
        segs.append((T, n, c, i))
        T += n
    q = _randn(gen, T, heads, D)
    cfg, segs_c, pages = qsa.make_config(sh), qsa.make_segments(segs), qsa.make_pages(kp, vp, table.cuda())
    o, lse = torch.empty_like(q), torch.empty((T, heads), device="cuda")
    for _ in range(3):
        qsa.qsa_paged_attn_fwd(cfg, pages, segs_c, T, q, o, lse, workspace(cfg, segs_c, T, qsa.QSA_OP_PAGED_ATTN))
    qsa.qsa_device_status()
    for (off, n, c, i), (k, v) in zip(segs, kv):
        t = slice(off, off + n)
        check_forward(o[t], lse[t], attend64(q[t], k, v, c, SCALE), score_error(q[t], k, SCALE), BF, i)


# ------------------------------------------------------------------ shared memory of a pair's other CTA
def test_rows_zeroed_by_either_cta_of_a_pair_are_zero_in_the_product():
    """Every prompt ends inside a chunk and is followed by NaN rows, which the
    softmax warps of both CTAs zero in their own halves of the operands before
    the leader's products read them: the same finite bits each time."""
    heads, groups, gap = 24, 2, 7
    lens = [130, 257, 300, 61, 1000, 129, 515]
    x = _prompts(heads, groups, [n + gap for n in lens], seed=5)
    segs = [(off, n, 0, 0) for off, n in zip(x["offs"], lens)]
    x["segs"] = qsa.make_segments(segs)
    used = torch.zeros(x["T"], dtype=torch.bool, device="cuda")
    for off, n, _, _ in segs:
        used[off:off + n] = True
    for name in ("q", "k", "v", "dout"):
        x[name][~used] = float("nan")
    runs = []
    for _ in range(20):
        o, lse = _forward(x)
        g = [torch.full_like(x[n], 5.0) for n in ("q", "k", "v")]
        qsa.qsa_prompt_attn_bwd(x["cfg"], x["segs"], x["T"], x["q"], x["k"], x["v"], o, lse, x["dout"], *g,
                                workspace(x["cfg"], x["segs"], x["T"], qsa.QSA_OP_PROMPT_ATTN_BWD))
        runs.append((o, lse, *g))
    qsa.qsa_device_status()
    for r in runs:
        for a, b in zip(r, runs[0]):
            assert torch.equal(a, b) and bool(torch.isfinite(a).all())
