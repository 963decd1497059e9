"""Calls of the paged append and the dense attention that once went wrong, or
could.  Bounds: dense_testlib."""
import math

import pytest
import torch

import block_sparse_attention_22_b200 as qsa
from dense_testlib import (D, F64, attend64, check_forward, fill_pages, make_table, rotate64, score_error, shape,
                           torch_dtype, workspace)

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


# ------------------------------------------------------------------ rows whose every score is -inf
def _paged_with_keys_at_minus_inf(dtype, seqs, page=16, seed=6):
    """Group 0's keys have -inf in dim 9, its queries something positive there."""
    sh = shape(24, 2, dtype)
    dt = torch_dtype(sh)
    gen = torch.Generator().manual_seed(seed)
    table, n_pages = make_table([c + n for c, n in seqs], page, gen)
    kp, vp = (torch.full((n_pages, 2, page, D), 5.0, dtype=dt, device="cuda") for _ in range(2))
    kv, segs, T = [], [], 0
    for i, (c, n) in enumerate(seqs):
        k, v = (_randn(gen, c + n, 2, D, dtype=dt) for _ in range(2))
        kv.append((k, v))
        segs.append((T, n, c, i))
        T += n
    q = _randn(gen, T, 24, D, dtype=dt)
    q[..., 9] = q[..., 9].abs() + 0.5
    x = dict(cfg=qsa.make_config(sh), T=T, q=q, kv=kv, segs_at=segs, segs=qsa.make_segments(segs), table=table, kp=kp,
             vp=vp, dt=dt, page=page)
    clean = _run_paged(x)
    for k, _ in kv:
        k[:, 0, 9] = -math.inf
    return x, clean


def _run_paged(x):
    for i, (k, v) in enumerate(x["kv"]):
        fill_pages(x["kp"], x["vp"], x["table"], x["page"], i, k, v)
    o, lse = torch.full_like(x["q"], 5.0), torch.full(x["q"].shape[:2], 5.0, device="cuda")
    qsa.qsa_paged_attn_fwd(x["cfg"], qsa.make_pages(x["kp"], x["vp"], x["table"].cuda()), x["segs"], x["T"], x["q"], o,
                           lse, workspace(x["cfg"], x["segs"], x["T"], qsa.QSA_OP_PAGED_ATTN))
    return o, lse


KINDS = [[(0, 1), (40, 1), (127, 1)], [(900, 1)] * 60, [(2000, 1)] * 8, [(20000, 1)], [(4000, 5)] * 3, [(0, 3), (30, 7)],
         [(1500, 300), (0, 200)], [(0, 20)]]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("seqs", KINDS, ids=["decode", "few pieces", "many pieces", "long", "short", "first", "chunks",
                                             "tile"])
def test_a_row_whose_every_score_is_minus_infinity_is_nan(dtype, seqs):
    """0 / 0 by the formula, with lse = -inf, whole or cut; the other group's heads
    keep their bits."""
    x, (clean, clean_lse) = _paged_with_keys_at_minus_inf(dtype, seqs)
    o, lse = _run_paged(x)
    qsa.qsa_device_status()
    assert bool(torch.isnan(o[:, :12]).all()) and bool((lse[:, :12] == -math.inf).all())
    assert torch.equal(o[:, 12:], clean[:, 12:]) and torch.equal(lse[:, 12:], clean_lse[:, 12:])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("seqs", KINDS[1:], ids=["few pieces", "many pieces", "long", "short", "first", "chunks", "tile"])
def test_one_finite_score_among_minus_infinities_takes_the_row(dtype, seqs):
    """Its weight is 1 in whichever piece it lies: o is that key's value, rounded once."""
    x, _ = _paged_with_keys_at_minus_inf(dtype, seqs)
    at = []
    for i, ((c, n), (k, _)) in enumerate(zip(seqs, x["kv"])):
        at.append(c * (i + 1) // len(seqs))               # visible to every row of the segment
        k[at[-1], 0, 9] = 0.0
    o, lse = _run_paged(x)
    for (off, n, c, i), j in zip(x["segs_at"], at):
        k, v = x["kv"][i]
        assert torch.equal(o[off:off + n, :12], v[j, :1].expand(n, 12, D))
        s = (x["q"][off:off + n, :12].to(F64) * k[j, 0].to(F64)).sum(-1) * SCALE
        e = score_error(x["q"], torch.where(torch.isfinite(k), k, 0), SCALE)
        assert bool(((lse[off:off + n, :12].to(F64) - s).abs() <= e + 2.0 ** -20 * (1 + s.abs())).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("seqs", [[(900, 1)] * 30, [(2000, 1)] * 4, [(3000, 5)] * 3, [(100, 200)]],
                         ids=["decode", "many pieces", "short", "chunks"])
def test_rows_without_a_key_stay_zero_beside_rows_at_minus_infinity(dtype, seqs):
    """All pages of the last sequence out of range: no key, o = 0.  All but one
    of the first one's: still keys, all at -inf, o = NaN."""
    x, _ = _paged_with_keys_at_minus_inf(dtype, seqs + [(700, 4)])
    c, n = seqs[0]
    good = x["table"]
    for i, (k, v) in enumerate(x["kv"]):
        fill_pages(x["kp"], x["vp"], good, x["page"], i, k, v)
    bad = good.clone()
    bad[0, :] = -1
    bad[0, c // 2 // 16] = good[0, c // 2 // 16]
    bad[len(seqs), :] = 1 << 30
    o, lse = torch.full_like(x["q"], 5.0), torch.full(x["q"].shape[:2], 5.0, device="cuda")
    qsa.qsa_paged_attn_fwd(x["cfg"], qsa.make_pages(x["kp"], x["vp"], bad.cuda()), x["segs"], x["T"], x["q"], o, lse,
                           workspace(x["cfg"], x["segs"], x["T"], qsa.QSA_OP_PAGED_ATTN))
    assert qsa.device_status() == qsa.QSA_ERR_BAD_INDEX
    assert bool(torch.isnan(o[:n, :12]).all()) and bool((lse[:, :12] == -math.inf).all())
    assert bool(torch.isfinite(o[:n, 12:]).all()) and bool(torch.isfinite(lse[:n, 12:]).all())
    assert bool((o[-4:] == 0).all()) and bool((lse[-4:] == -math.inf).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prompts_at_minus_infinity_and_their_gradient_are_nan_in_their_rows_alone(dtype):
    """Keys of the first 30 tokens of the second prompt at -inf in group 0: rows
    before token 30 have no other score; the rows after it do."""
    lens = [70, 333, 40]
    x = _prompts(24, 2, lens, seed=7, dtype=dtype)
    x["q"][..., 9] = x["q"][..., 9].abs() + 0.5
    clean = _forward(x)
    x["k"][70:100, 0, 9] = -math.inf
    o, lse = _forward(x)
    hit = torch.zeros(lse.shape, dtype=torch.bool, device="cuda")
    hit[70:100, :12] = True
    assert bool(torch.isnan(o[hit]).all()) and bool((lse[hit] == -math.inf).all())
    assert bool(torch.isfinite(o[~hit]).all()) and bool(torch.isfinite(lse[~hit]).all())
    for a, b in zip((o, lse), clean):
        assert torch.equal(a[:70], b[:70]) and torch.equal(a[403:], b[403:]) and torch.equal(a[:, 12:], b[:, 12:])
    t = slice(100, 403)
    ref = attend64(x["q"][t, :12], x["k"][t, :1], x["v"][t, :1], 0, SCALE)        # the keys with a weight
    check_forward(o[t, :12], lse[t, :12], ref, score_error(x["q"][t], x["k"][t], SCALE), x["dt"])
    g = [torch.full_like(x[n], 5.0) for n in ("q", "k", "v")]
    qsa.qsa_prompt_attn_bwd(x["cfg"], x["segs"], x["T"], x["q"], x["k"], x["v"], o, lse, x["dout"], *g,
                            workspace(x["cfg"], x["segs"], x["T"], qsa.QSA_OP_PROMPT_ATTN_BWD))
    qsa.qsa_device_status()
    assert bool(torch.isnan(g[0][hit]).all())
    assert bool(torch.isfinite(g[0][:, 12:]).all()) and bool(torch.isfinite(g[0][:70]).all())
    for a in g[1:]:
        assert bool(torch.isfinite(a[100:, 0]).all()) and bool(torch.isfinite(a[:, 1]).all())


# ------------------------------------------------------------------ delta of the first rows
@pytest.mark.parametrize("heads,groups", [(8, 8), (6, 2), (24, 2), (10, 5)])
@pytest.mark.parametrize("lens", [[129], [128, 300, 1], [600, 257]])
def test_gradients_of_the_first_rows_do_not_carry_the_rounding_of_o(heads, groups, lens):
    """Every value of a prompt is a permutation of one vector whose dims add up to 0,
    in eighths, and dout is 1 in all dims, so dP is 0 for every key, exactly: dS, dq
    and dk are 0, and what is left is delta's error.  From the row's own P and dP,
    for rows of at most 128 keys, there is none; from a rounded o it was 2^-9 of its
    parts.  Later rows have it still, and the rounding of P: delta is off by at most
    (2^-8 + 2^-8 + fp32) sum |v| of a key, which bounds their part of dk."""
    x = _prompts(heads, groups, lens, seed=8)
    gen = torch.Generator().manual_seed(9)
    half = torch.round(torch.randn(D // 2, generator=gen) * 8) / 8
    order = torch.argsort(torch.rand((x["T"], groups, D), generator=gen), dim=-1)
    x["v"] = torch.cat([half, -half]).to(BF)[order].cuda()
    x["dout"] = torch.ones_like(x["dout"])
    o, lse = _forward(x)
    g = [torch.full_like(x[n], 5.0) for n in ("q", "k", "v")]
    qsa.qsa_prompt_attn_bwd(x["cfg"], x["segs"], x["T"], x["q"], x["k"], x["v"], o, lse, x["dout"], *g,
                            workspace(x["cfg"], x["segs"], x["T"], qsa.QSA_OP_PROMPT_ATTN_BWD))
    qsa.qsa_device_status()
    hpg = heads // groups
    ddelta = 1.1 * 2.0 ** -7 * x["v"][0, 0].to(F64).abs().sum().item()
    for off, n in zip(x["offs"], lens):
        assert not g[0][off:off + min(n, 128)].any()
        if n <= 128:
            assert not g[1][off:off + n].any()
            continue
        t = slice(off, off + n)
        q, k = x["q"][t].to(F64), x["k"][t].to(F64)
        for grp in range(groups):
            tol = torch.zeros((n, D), dtype=F64, device="cuda")
            for h in range(grp * hpg, (grp + 1) * hpg):
                s = (q[:, h] @ k[:, grp].t()) * SCALE
                s.masked_fill_(torch.ones_like(s, dtype=torch.bool).triu(1), -math.inf)
                tol += SCALE * ddelta * (torch.softmax(s, 1)[128:].t() @ q[128:, h].abs())
            assert bool((g[1][t, grp].to(F64).abs() <= tol).all()), (grp, n)


# ------------------------------------------------------------------ rotations beyond the indexer's
@pytest.mark.parametrize("frac", [1.0, 0.6])
def test_append_rotates_more_dims_than_the_indexer_can(frac):
    """idx_dim 128 in bf16.  A rotated value: cos, sin and two products and a sum in
    fp32 (2^-24 each) of |a| + |b|, one rounding."""
    sh = shape(24, 2, "bf16", frac)
    sh.idx_dim = 128
    cfg, gen = qsa.make_config(sh), torch.Generator().manual_seed(12)
    kp, vp = (torch.zeros((3, 2, 16, D), dtype=BF, device="cuda") for _ in range(2))
    table = torch.tensor([[2, 0, 1]], dtype=torch.int32, device="cuda")
    k, v, q = _randn(gen, 40, 2, D), _randn(gen, 40, 2, D), _randn(gen, 40, 24, D)
    q_out, pos = torch.empty_like(q), torch.arange(40, device="cuda")
    qsa.qsa_append_kv(cfg, qsa.make_pages(kp, vp, table), qsa.make_segments([(0, 40, 0, 0)]), 40, k, v, q, q_out)
    qsa.qsa_device_status()
    pg = table[0].long()[pos // 16]
    for got, x in ((kp[pg, :, pos % 16], k), (q_out, q)):
        ref = rotate64(x, pos, frac)
        tol = 2.0 ** -8 * ref.abs() * 1.001 + 8 * 2.0 ** -24 * x.to(F64).abs().amax(dim=-1, keepdim=True)
        assert bool(((got.to(F64) - ref).abs() <= tol).all())
    assert torch.equal(vp[pg, :, pos % 16], v)


# ------------------------------------------------------------------ strides of dims of size 1
def test_append_of_one_group_or_one_token_takes_any_stride_of_the_dim_of_size_one():
    gen = torch.Generator().manual_seed(13)
    for groups, T, k, v in (
            (1, 5, _randn(gen, 1, 5, D).transpose(0, 1), _randn(gen, 1, 5, D).transpose(0, 1)),
            (2, 1, _randn(gen, 1, 2 * D + 3)[:, :2 * D].view(1, 2, D), _randn(gen, 1, 2 * D + 3)[:, :2 * D].view(1, 2, D))):
        cfg = qsa.make_config(shape(12 * groups, groups, "bf16", 0.0))
        kp, vp = (torch.zeros((1, groups, 16, D), dtype=BF, device="cuda") for _ in range(2))
        pages = qsa.make_pages(kp, vp, torch.zeros((1, 1), dtype=torch.int32, device="cuda"))
        qsa.qsa_append_kv(cfg, pages, qsa.make_segments([(0, T, 3, 0)]), T, k, v)
        assert torch.equal(kp[0, :, 3:3 + T], k.transpose(0, 1)) and torch.equal(vp[0, :, 3:3 + T], v.transpose(0, 1))
        assert not kp[0, :, :3].any() and not kp[0, :, 3 + T:].any()
