"""Paged append, dense paged attention and packed prompt attention with its
gradient, against plain 64-bit forms.  Bounds: dense_testlib."""
import math

import pytest
import torch

import block_sparse_attention_22_b200 as qsa
from dense_testlib import (D, F64, attend64, check_forward, fill_pages, gradients64, half_step, make_table, rotate64,
                           score_error, shape, torch_dtype, workspace)

pytestmark = pytest.mark.gpu
NAN = float("nan")
SCALE = 1.0 / math.sqrt(D)


@pytest.fixture(scope="module", autouse=True)
def _need_cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _randn(gen, *size, dtype):
    return torch.randn(size, generator=gen).to(dtype).cuda()


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("heads,groups,dtype,page,frac", [
    (24, 2, "bf16", 64, 0.25), (16, 4, "f32", 16, 0.25), (8, 8, "bf16", 48, 1.0), (12, 1, "bf16", 1024, 0.3),
    (6, 2, "f32", 32, 0.0), (24, 2, "bf16", 16, 0.01),
])
@pytest.mark.parametrize("seqs", [[(0, 1)], [(5, 3), (0, 0), (63, 2), (100, 1)], [(1048570, 6)], [(17, 300), (0, 65)]])
def test_append_matches_definition(heads, groups, dtype, page, frac, seqs):
    sh = shape(heads, groups, dtype, frac)
    dt = torch_dtype(sh)
    cfg = qsa.make_config(sh)
    gen = torch.Generator().manual_seed(3)
    T = sum(n for _, n in seqs) + 3                      # one unused row before, two behind
    offs, at = [], 1
    for _, n in seqs:
        offs.append(at)
        at += n
    table = torch.full((len(seqs), max((c + n + page - 1) // page for c, n in seqs) + 1), -1, dtype=torch.int32)
    free = list(torch.randperm(200, generator=gen).tolist())
    for i, (c, n) in enumerate(seqs):
        for p in range(c // page, (c + n + page - 1) // page):
            table[i, p] = free.pop()
    pool = 200 if page < 1024 else 200
    kp = torch.full((pool, groups, page, D), 7.0, dtype=dt, device="cuda")
    vp = torch.full_like(kp, -7.0)
    qkv = _randn(gen, T, (heads + 2 * groups) * D, dtype=dt)         # a fused projection's output
    q = qkv[:, :heads * D].view(T, heads, D)
    k = qkv[:, heads * D:(heads + groups) * D].view(T, groups, D)
    v = qkv[:, (heads + groups) * D:].view(T, groups, D)
    q_out = torch.full((T, heads, D), 3.0, dtype=dt, device="cuda")
    pages = qsa.make_pages(kp, vp, table.cuda())
    segs = qsa.make_segments([(off, n, c, i) for i, ((c, n), off) in enumerate(zip(seqs, offs))])
    ek, ev, eq = kp.to(F64), vp.to(F64), q_out.to(F64)
    qsa.qsa_append_kv(cfg, pages, segs, T, k, v, q, q_out)
    torch.cuda.synchronize()
    qsa.qsa_device_status()
    tk, tq = torch.zeros_like(ek), torch.zeros_like(eq)
    u = half_step(dt)
    # a rotated value: cos, sin rounded (2^-24 each), two products and a sum in
    # fp32 (2^-24 each) on |a| + |b|, then one rounding to the I/O dtype
    slack = 4 * 2.0 ** -24
    for i, ((c, n), off) in enumerate(zip(seqs, offs)):
        pos = torch.arange(c, c + n, device="cuda")
        pg = table[i].cuda().long()[pos // page]
        rk, rq = (rotate64(x[off:off + n], pos, frac) for x in (k, q))
        ek[pg, :, pos % page] = rk
        ev[pg, :, pos % page] = v[off:off + n].to(F64)
        eq[off:off + n] = rq
        mk, mq = (x[off:off + n].to(F64).abs().amax(dim=-1, keepdim=True) for x in (k, q))
        tk[pg, :, pos % page] = u * rk.abs() * 1.001 + 2 * slack * mk
        tq[off:off + n] = u * rq.abs() * 1.001 + 2 * slack * mq
    assert ((kp.to(F64) - ek).abs() <= tk).all()
    assert torch.equal(vp.to(F64), ev)
    assert ((q_out.to(F64) - eq).abs() <= tq).all()
    # in place, without strides, without q
    q2 = q.contiguous()
    kp2, vp2 = torch.full_like(kp, 7.0), torch.full_like(vp, -7.0)
    qsa.qsa_append_kv(cfg, qsa.make_pages(kp2, vp2, table.cuda()), segs, T, k.contiguous(), v.contiguous(), q2, q2)
    for off, n in zip(offs, [n for _, n in seqs]):
        assert torch.equal(q2[off:off + n], q_out[off:off + n])
    assert torch.equal(kp2, kp) and torch.equal(vp2, vp)
    kp2.fill_(7.0), vp2.fill_(-7.0)
    qsa.qsa_append_kv(cfg, qsa.make_pages(kp2, vp2, table.cuda()), segs, T, k, v)
    assert torch.equal(kp2, kp) and torch.equal(vp2, vp)


def test_append_skips_and_reports_bad_pages():
    sh = shape()
    cfg = qsa.make_config(sh)
    gen = torch.Generator().manual_seed(5)
    table = torch.tensor([[0, 9, 2]], dtype=torch.int32).cuda()       # 9 pages do not exist
    kp = torch.zeros((3, 2, 16, D), dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    k, v = (_randn(gen, 48, 2, D, dtype=torch.bfloat16) for _ in range(2))
    segs = qsa.make_segments([(0, 48, 0, 0)])
    qsa.qsa_append_kv(cfg, qsa.make_pages(kp, vp, table), segs, 48, k, v)
    assert qsa.device_status() == qsa.QSA_ERR_BAD_INDEX
    assert qsa.device_status() == qsa.QSA_OK
    assert torch.equal(vp[0], v[:16].transpose(0, 1)) and torch.equal(vp[2], v[32:].transpose(0, 1))
    assert not kp[1].any() and not vp[1].any()


# ------------------------------------------------------------------ paged attention
def _paged_case(sh, page, seqs, seed=1, spread=1.0, poison=NAN):
    """Random sequences in a poisoned page pool; token rows shuffled between
    the segments, with unused rows around them."""
    dt = torch_dtype(sh)
    gen = torch.Generator().manual_seed(seed)
    T = sum(n for _, n in seqs) + 2
    order = torch.randperm(len(seqs), generator=gen).tolist()
    offs, at = [0] * len(seqs), 1
    for i in order:
        offs[i] = at
        at += seqs[i][1]
    table, n_pages = make_table([c + n for c, n in seqs], page, gen)
    kp = torch.full((n_pages, sh.n_groups, page, D), poison, dtype=dt, device="cuda")
    vp = torch.full_like(kp, poison)
    q = _randn(gen, T, sh.n_heads, D, dtype=dt) * spread
    kv = []
    for i, (c, n) in enumerate(seqs):
        k = _randn(gen, c + n, sh.n_groups, D, dtype=dt)
        v = _randn(gen, c + n, sh.n_groups, D, dtype=dt)
        fill_pages(kp, vp, table, page, i, k, v)
        kv.append((k, v))
    segs = qsa.make_segments([(off, n, c, i) for i, ((c, n), off) in enumerate(zip(seqs, offs))])
    return dict(cfg=qsa.make_config(sh), q=q, kv=kv, T=T, offs=offs, segs=segs, seqs=seqs, dt=dt,
                pages=qsa.make_pages(kp, vp, table.cuda()), kp=kp, vp=vp, table=table)


def _run_paged(x, lse=True):
    o = torch.full((x["T"], x["q"].shape[1], D), 5.0, dtype=x["dt"], device="cuda")
    l = torch.full((x["T"], x["q"].shape[1]), 5.0, device="cuda") if lse else None
    ws = workspace(x["cfg"], x["segs"], x["T"], qsa.QSA_OP_PAGED_ATTN)
    qsa.qsa_paged_attn_fwd(x["cfg"], x["pages"], x["segs"], x["T"], x["q"], o, l, ws)
    torch.cuda.synchronize()
    return o, l


def _check_paged(x, o, l):
    used = torch.zeros(x["T"], dtype=torch.bool)
    for (c, n), off, (k, v) in zip(x["seqs"], x["offs"], x["kv"]):
        used[off:off + n] = True
        if n == 0:
            continue
        q = x["q"][off:off + n]
        check_forward(o[off:off + n], None if l is None else l[off:off + n], attend64(q, k, v, c, SCALE),
                      score_error(q, k, SCALE), x["dt"], (c, n))
    assert (o[~used] == 5.0).all() and (l is None or (l[~used] == 5.0).all())


@pytest.mark.parametrize("heads,groups", [(24, 2), (16, 2), (8, 8), (12, 1), (3, 1), (32, 2)])
@pytest.mark.parametrize("dtype,page", [("bf16", 64), ("f32", 16), ("bf16", 16), ("bf16", 48), ("bf16", 1024)])
@pytest.mark.parametrize("seqs", [
    [(0, 1)],                                            # a first token
    [(63, 1), (64, 1), (127, 1), (128, 1), (0, 1), (700, 1), (5, 0)],
    [(2999, 1)],                                         # one row, keys split over the GPU
    [(130, 4), (15, 7), (0, 2), (999, 5)],
    [(0, 129), (40, 300), (511, 33), (256, 64)],
], ids=["first", "decode", "long_decode", "few", "chunks"])
def test_paged_attention_matches_definition(heads, groups, dtype, page, seqs):
    x = _paged_case(shape(heads, groups, dtype), page, seqs)
    o, l = _run_paged(x)
    qsa.qsa_device_status()
    _check_paged(x, o, l)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_paged_attention_of_long_and_many_sequences(dtype):
    """A decode batch of more segments than one launch holds, next to chunks
    whose units fill whole rounds and a tail."""
    seqs = [((37 * i) % 1500, 1) for i in range(140)] + [(3000, 1200), (100, 900 if dtype == "bf16" else 100)]
    x = _paged_case(shape(24, 2, dtype), 32, seqs, seed=2)
    o, l = _run_paged(x)
    _check_paged(x, o, l)
    o2, l2 = _run_paged(x)
    assert torch.equal(o, o2) and torch.equal(l, l2)             # the same bits again
    o3, _ = _run_paged(x, lse=False)
    assert torch.equal(o, o3)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_paged_attention_with_rising_and_peaked_scores(dtype):
    """Maxima that keep rising along the keys (every chunk rescales) and rows
    that a single key takes over."""
    x = _paged_case(shape(24, 2, dtype), 64, [(1500, 40), (2000, 1), (0, 300)], seed=4)
    for i, (k, v) in enumerate(x["kv"]):
        up = torch.linspace(0, 3, k.shape[0], device="cuda")[:, None, None]
        direction = torch.ones(D, device="cuda")
        k.copy_((k.float() + up * direction).to(x["dt"]))
        k[k.shape[0] // 2] *= 3
        fill_pages(x["kp"], x["vp"], x["table"], 64, i, k, v)
    x["q"].copy_((x["q"].float() + 0.7).to(x["dt"]))
    o, l = _run_paged(x)
    _check_paged(x, o, l)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("value", [NAN, float("inf"), -float("inf")])
def test_later_keys_do_not_reach_earlier_rows(dtype, value):
    """Keys and values of a late token that are not finite: rows before it
    are those of the clean cache, bit for bit."""
    for seqs, at in [([(300, 60)], 330), ([(0, 200)], 100), ([(64, 5)], 67), ([(1, 2)], 2)]:
        x = _paged_case(shape(24, 2, dtype), 16, seqs, seed=6)
        clean, cl = _run_paged(x)
        k, v = x["kv"][0]
        k[at:], v[at:] = value, value
        fill_pages(x["kp"], x["vp"], x["table"], 16, 0, k, v)
        o, l = _run_paged(x)
        n = at - seqs[0][0]                              # rows of positions before `at`
        off = x["offs"][0]
        assert torch.equal(o[off:off + n], clean[off:off + n])
        assert torch.equal(l[off:off + n], cl[off:off + n])
        assert not torch.isfinite(o[off + n:off + seqs[0][1]].float()).all(dim=-1).any()   # later rows do see it


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_values_that_are_not_finite_stay_in_their_dims(dtype):
    """An infinite value in one dim of one key: the rows that attend it are
    infinite in that dim and right in the others."""
    x = _paged_case(shape(24, 2, dtype), 16, [(200, 50)], seed=7)
    k, v = x["kv"][0]
    v[220, 0, 17] = float("inf")
    fill_pages(x["kp"], x["vp"], x["table"], 16, 0, k, v)
    o, l = _run_paged(x)
    off = x["offs"][0]
    rows = o[off:off + 50].float()
    assert torch.isinf(rows[20:, :12, 17]).all() and torch.isfinite(rows[:20]).all()
    v2 = v.clone()
    v2[220, 0, 17] = 0
    x["kv"][0] = (k, v2)
    o[off + 20:off + 50, :12, 17] = 0
    ref = list(attend64(x["q"][off:off + 50], k, v2, 200, SCALE))
    ref[0][20:, :12, 17] = 0
    check_forward(o[off:off + 50], l[off:off + 50], ref, score_error(x["q"], k, SCALE), x["dt"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_paged_attention_skips_and_reports_bad_pages(dtype):
    """Pages out of range count for nothing; a row whose every key is gone is
    zero with lse -inf."""
    x = _paged_case(shape(24, 2, dtype), 16, [(150, 20), (40, 1), (30, 1)], seed=8)
    t = x["table"].clone()
    t[0, 3] = 1 << 20
    t[0, 4] = -1
    t[1, :] = -5
    x["pages"] = qsa.make_pages(x["kp"], x["vp"], t.cuda())
    o, l = _run_paged(x)
    assert qsa.device_status() == qsa.QSA_ERR_BAD_INDEX
    assert qsa.device_status() == qsa.QSA_OK
    off = x["offs"][1]
    assert (o[off] == 0).all() and (l[off] == -math.inf).all()
    k, v = x["kv"][0]
    keep = torch.cat([torch.arange(48), torch.arange(80, 170)]).cuda()      # rows 48..79 are gone
    off = x["offs"][0]
    q = x["q"][off:off + 20]
    check_forward(o[off:off + 20], l[off:off + 20], attend64(q, k[keep], v[keep], 150 - 32, SCALE),
                  score_error(q, k, SCALE), x["dt"])
    off = x["offs"][2]
    check_forward(o[off:off + 1], l[off:off + 1], attend64(x["q"][off:off + 1], *x["kv"][2], 30, SCALE),
                  score_error(q, k, SCALE), x["dt"])


def test_paged_attention_is_the_sparse_attention_with_every_block_kept():
    """Append into a slot cache (its pages are the slots), then the whole QSA
    forward with a budget that covers the context: the dense attention over
    the same cache gives the same result."""
    sh = shape()
    cfg = qsa.make_config(sh)
    gen = torch.Generator().manual_seed(9)
    n, cap = 1200, 2048
    kc, vc = (torch.full((2, 2, cap, D), NAN, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k_idx = _randn(gen, 2, cap, 64, dtype=torch.bfloat16)
    khat = torch.zeros((2, cap // 4, 64), dtype=torch.bfloat16, device="cuda")
    pages = qsa.make_pages(kc, vc, torch.arange(2, dtype=torch.int32, device="cuda")[:, None])
    qkv = _randn(gen, 2 * n, 28 * D, dtype=torch.bfloat16)
    q_raw, k, v = qkv.view(2 * n, 28, D).split([24, 2, 2], dim=1)
    q = torch.empty((2 * n, 24, D), dtype=torch.bfloat16, device="cuda")
    segs = qsa.make_segments([(0, n, 0, 0), (n, n, 0, 1)])
    qsa.qsa_append_kv(cfg, pages, segs, 2 * n, k, v, q_raw, q)
    q_idx = _randn(gen, 2 * n, 4, 64, dtype=torch.bfloat16)
    w = torch.rand((2 * n, 4), generator=gen).cuda()
    o, o2, o3 = (torch.empty_like(q) for _ in range(3))
    lse, lse2, lse3 = (torch.empty((2 * n, 24), device="cuda") for _ in range(3))
    cache = qsa.make_cache(k_idx, khat, kc, vc)
    qsa.qsa_forward(cfg, cache, segs, 2 * n, q, q_idx, w, o, lse,
                    workspace=workspace(cfg, segs, 2 * n, qsa.QSA_OP_FORWARD))
    qsa.qsa_paged_attn_fwd(cfg, pages, segs, 2 * n, q, o2, lse2, workspace(cfg, segs, 2 * n, qsa.QSA_OP_PAGED_ATTN))
    krot = torch.cat([kc[i, :, :n].transpose(0, 1) for i in range(2)]).contiguous()
    qsa.qsa_prompt_attn_fwd(cfg, segs, 2 * n, q, krot, v.contiguous(), o3, lse3,
                            workspace(cfg, segs, 2 * n, qsa.QSA_OP_PROMPT_ATTN))
    qsa.qsa_device_status()
    for i in range(2):
        t = slice(i * n, i * n + n)
        ref = attend64(q[t], kc[i, :, :n].transpose(0, 1), vc[i, :, :n].transpose(0, 1), 0, SCALE)
        e = score_error(q[t], krot, SCALE)
        for a, b in ((o, lse), (o2, lse2), (o3, lse3)):
            check_forward(a[t], b[t], ref, e, torch.bfloat16, i)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prefill_then_decode_over_the_paged_cache(dtype):
    """A prompt in two chunks, then single tokens, append and attention each
    step: every row equals the packed prompt's."""
    sh = shape(16, 2, dtype)
    dt = torch_dtype(sh)
    cfg = qsa.make_config(sh)
    gen = torch.Generator().manual_seed(10)
    n, page = 210, 48
    table, n_pages = make_table([n, n], page, gen)
    kp, vp = (torch.full((n_pages, 2, page, D), NAN, dtype=dt, device="cuda") for _ in range(2))
    pages = qsa.make_pages(kp, vp, table.cuda())
    q, k, v = (_randn(gen, 2 * n, h, D, dtype=dt) for h in (16, 2, 2))
    o, qr = torch.empty_like(q), torch.empty_like(q)
    lse = torch.empty((2 * n, 16), device="cuda")
    for a, b in [(0, 100), (100, 200)] + [(i, i + 1) for i in range(200, n)]:
        segs = qsa.make_segments([(a, b - a, a, 0), (n + a, b - a, a, 1)])
        qsa.qsa_append_kv(cfg, pages, segs, 2 * n, k, v, q, qr)
        qsa.qsa_paged_attn_fwd(cfg, pages, segs, 2 * n, qr, o, lse, workspace(cfg, segs, 2 * n, qsa.QSA_OP_PAGED_ATTN))
    qsa.qsa_device_status()
    pos = torch.arange(n, device="cuda")
    for i in range(2):
        t = slice(i * n, i * n + n)
        pg = table[i].cuda().long()[pos // page]
        ref = attend64(qr[t], kp[pg, :, pos % page], v[t], 0, SCALE)
        check_forward(o[t], lse[t], ref, score_error(qr[t], k, SCALE), dt, i)


# ------------------------------------------------------------------ packed prompts
def _prompt_case(sh, lens, seed=1, gap=1):
    dt = torch_dtype(sh)
    gen = torch.Generator().manual_seed(seed)
    T = sum(lens) + gap * (len(lens) + 1)
    offs, at = [], gap
    for n in lens:
        offs.append(at)
        at += n + gap
    q, dout = (_randn(gen, T, sh.n_heads, D, dtype=dt) for _ in range(2))
    k, v = (_randn(gen, T, sh.n_groups, D, dtype=dt) for _ in range(2))
    used = torch.zeros(T, dtype=torch.bool)
    for n, off in zip(lens, offs):
        used[off:off + n] = True
    for t in (q, k, v, dout):
        t[~used.cuda()] = NAN                            # rows of no prompt
    return dict(cfg=qsa.make_config(sh), q=q, k=k, v=v, dout=dout, T=T, offs=offs, lens=lens, dt=dt, used=used,
                segs=qsa.make_segments([(off, n, 0, 0) for n, off in zip(lens, offs)]))


def _run_prompt(x):
    o = torch.full_like(x["q"], 5.0)
    lse = torch.full((x["T"], o.shape[1]), 5.0, device="cuda")
    qsa.qsa_prompt_attn_fwd(x["cfg"], x["segs"], x["T"], x["q"], x["k"], x["v"], o, lse,
                            workspace(x["cfg"], x["segs"], x["T"], qsa.QSA_OP_PROMPT_ATTN))
    return o, lse


def _run_prompt_bwd(x, o, lse):
    g = [torch.full_like(x[n], 5.0) for n in ("q", "k", "v")]
    qsa.qsa_prompt_attn_bwd(x["cfg"], x["segs"], x["T"], x["q"], x["k"], x["v"], o, lse, x["dout"], *g,
                            workspace(x["cfg"], x["segs"], x["T"], qsa.QSA_OP_PROMPT_ATTN_BWD))
    torch.cuda.synchronize()
    return g


@pytest.mark.parametrize("heads,groups", [(24, 2), (16, 2), (8, 8), (12, 1), (3, 1)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [[1], [64, 1, 0, 65, 127], [130, 11, 300], [513], [10, 21, 22, 128, 256]])
def test_prompt_attention_and_gradient_match_definition(heads, groups, dtype, lens):
    x = _prompt_case(shape(heads, groups, dtype), lens)
    o, lse = _run_prompt(x)
    grads = _run_prompt_bwd(x, o, lse)
    qsa.qsa_device_status()
    for n, off in zip(lens, x["offs"]):
        if n == 0:
            continue
        t = slice(off, off + n)
        q, k, v = x["q"][t], x["k"][t], x["v"][t]
        check_forward(o[t], lse[t], attend64(q, k, v, 0, SCALE), score_error(q, k, SCALE), x["dt"], n)
        ref, tol = gradients64(q, k, v, x["dout"][t], SCALE)
        for name, got in zip(("dq", "dk", "dv"), grads):
            err = (got[t].to(F64) - ref[name]).abs()
            assert (err <= tol[name] + 1e-30).all(), (name, n, (err / (tol[name] + 1e-30)).max().item())
    for t in (o, lse, *grads):
        assert (t[~x["used"].cuda()] == 5.0).all()
    for a, b in zip(grads, _run_prompt_bwd(x, o, lse)):
        assert torch.equal(a, b)                         # the same bits again


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prompt_attention_of_more_prompts_than_a_launch_holds(dtype):
    lens = [(i * 13) % 70 for i in range(150)] + [700]
    x = _prompt_case(shape(6, 2, dtype), lens, seed=3, gap=0)
    o, lse = _run_prompt(x)
    grads = _run_prompt_bwd(x, o, lse)
    for n, off in zip(lens, x["offs"]):
        if n == 0:
            continue
        t = slice(off, off + n)
        q, k, v = x["q"][t], x["k"][t], x["v"][t]
        check_forward(o[t], lse[t], attend64(q, k, v, 0, SCALE), score_error(q, k, SCALE), x["dt"], n)
        ref, tol = gradients64(q, k, v, x["dout"][t], SCALE)
        for name, got in zip(("dq", "dk", "dv"), grads):
            err = (got[t].to(F64) - ref[name]).abs()
            assert (err <= tol[name] + 1e-30).all(), (name, n, (err / (tol[name] + 1e-30)).max().item())


def test_gradient_matches_differences():
    """Central differences of sum(dout . o) in fp32: the loss is a smooth
    function; a step h gives an error of h^2/6 times the third derivative
    (below 1e-3 of the gradient's scale at h = 2^-5) plus the loss's own fp32
    error 2^-24 * sum|dout . o| / h."""
    x = _prompt_case(shape(6, 2, "f32"), [40], seed=11, gap=0)
    o, lse = _run_prompt(x)
    grads = _run_prompt_bwd(x, o, lse)
    gen = torch.Generator().manual_seed(12)
    h = 2.0 ** -5
    for name, grad in zip(("q", "k", "v"), grads):
        base = x[name].clone()
        for _ in range(3):
            step = torch.randn(base.shape, generator=gen).cuda() / math.sqrt(base.numel()) * 4
            loss = []
            for sign in (1, -1):
                x[name] = (base + sign * h * step).contiguous()
                oo, _ = _run_prompt(x)
                loss.append((oo.to(F64) * x["dout"].to(F64)).sum().item())
            x[name] = base
            want = (grad.to(F64) * step.to(F64)).sum().item()
            got = (loss[0] - loss[1]) / (2 * h)
            size = grad.to(F64).norm().item() * step.to(F64).norm().item()
            noise = 2.0 ** -20 * (o.to(F64) * x["dout"].to(F64)).abs().sum().item() / h
            assert abs(got - want) <= 1e-3 * size + noise, (name, got, want, size, noise)
