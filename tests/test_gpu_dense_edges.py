"""Dense attention where its kernels meet an edge: decode lengths around the
tiles, caches beyond 32-bit offsets, values that are not finite in a gradient's
inputs, other streams, captured graphs.  Bounds: dense_testlib."""
import math

import pytest
import torch

import block_sparse_attention_22_b200 as qsa
from dense_testlib import (D, F64, attend64, check_forward, fill_pages, gradients64, make_table, score_error, shape,
                           torch_dtype, workspace)

pytestmark = pytest.mark.gpu
NAN = float("nan")
SCALE = 1.0 / math.sqrt(D)
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _need_cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _randn(gen, *size, dtype=BF):
    return torch.randn(size, generator=gen).to(dtype).cuda()


def _cache(heads, groups, page, seqs, seed=1, dtype="bf16", poison=NAN):
    sh = shape(heads, groups, dtype)
    dt = torch_dtype(sh)
    gen = torch.Generator().manual_seed(seed)
    table, n_pages = make_table([c + n for c, n in seqs], page, gen)
    kp = torch.full((n_pages, groups, page, D), poison, dtype=dt, device="cuda")
    vp = torch.full_like(kp, poison)
    kv, offs, at = [], [], 0
    for i, (c, n) in enumerate(seqs):
        k, v = (_randn(gen, c + n, groups, D, dtype=dt) for _ in range(2))
        fill_pages(kp, vp, table, page, i, k, v)
        kv.append((k, v))
        offs.append(at)
        at += n
    return dict(cfg=qsa.make_config(sh), dt=dt, seqs=seqs, offs=offs, T=at, kv=kv, kp=kp, vp=vp, table=table,
                q=_randn(gen, at, heads, D, dtype=dt), pages=qsa.make_pages(kp, vp, table.cuda()),
                segs=qsa.make_segments([(o, n, c, i) for i, ((c, n), o) in enumerate(zip(seqs, offs))]))


def _attend(x, ws=None, stream=None):
    o = torch.full_like(x["q"], 5.0)
    lse = torch.full(x["q"].shape[:2], 5.0, device="cuda")
    ws = workspace(x["cfg"], x["segs"], x["T"], qsa.QSA_OP_PAGED_ATTN) if ws is None else ws
    qsa.qsa_paged_attn_fwd(x["cfg"], x["pages"], x["segs"], x["T"], x["q"], o, lse, ws, stream)
    return o, lse


def _check(x, o, lse):
    for (c, n), off, (k, v) in zip(x["seqs"], x["offs"], x["kv"]):
        if n:
            q = x["q"][off:off + n]
            check_forward(o[off:off + n], lse[off:off + n], attend64(q, k, v, c, SCALE), score_error(q, k, SCALE),
                          x["dt"], (c, n))


@pytest.mark.parametrize("heads,groups", [(24, 2), (32, 2), (16, 1), (5, 5), (3, 1), (14, 2)])
@pytest.mark.parametrize("page", [16, 48, 256])
def test_decode_lengths_around_the_tiles(heads, groups, page):
    """Contexts that end inside, at and behind a warp's 16 keys, a chunk's 128 and a page."""
    lens = [1, 2, 15, 16, 17, 31, 33, 47, 48, 49, 127, 128, 129, 143, 144, 255, 256, 257, 1000, 2049]
    x = _cache(heads, groups, page, [(n - 1, 1) for n in lens])
    o, lse = _attend(x)
    qsa.qsa_device_status()
    _check(x, o, lse)
    o2, lse2 = _attend(x)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("heads,groups", [(24, 2), (32, 2), (14, 2), (8, 1), (4, 1), (5, 5)])
@pytest.mark.parametrize("page", [16, 48, 256])
def test_fp32_decode_lengths_around_the_tiles(heads, groups, page):
    lens = [1, 2, 3, 4, 5, 15, 16, 17, 18, 31, 33, 48, 49, 127, 128, 129, 131, 144, 255, 257, 1000, 4099]
    x = _cache(heads, groups, page, [(n - 1, 1) for n in lens], dtype="f32")
    o, lse = _attend(x)
    qsa.qsa_device_status()
    _check(x, o, lse)
    o2, lse2 = _attend(x)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_fp32_decode_rescales_and_skips_bad_pages():
    x = _cache(24, 2, 16, [(900, 1), (300, 1)], seed=14, dtype="f32")
    k, v = x["kv"][0]
    k.add_(torch.linspace(0, 3, k.shape[0], device="cuda")[:, None, None])
    fill_pages(x["kp"], x["vp"], x["table"], 16, 0, k, v)
    x["q"].add_(0.7)
    t = x["table"].clone()
    t[0, 5], t[0, 56], t[1, :] = -1, 1 << 30, -2          # 56 holds the row's own key
    x["pages"] = qsa.make_pages(x["kp"], x["vp"], t.cuda())
    o, lse = _attend(x)
    assert qsa.device_status() == qsa.QSA_ERR_BAD_INDEX
    keep = torch.tensor([j for j in range(901) if j // 16 not in (5, 56)]).cuda()
    q = x["q"][:1]
    check_forward(o[:1], lse[:1], attend64(q, k[keep], v[keep], 900, SCALE), score_error(q, k, SCALE), x["dt"])
    assert (o[1] == 0).all() and (lse[1] == -math.inf).all()


def test_decode_of_one_long_row_in_many_pieces():
    x = _cache(24, 2, 64, [(50000, 1)], seed=2)
    o, lse = _attend(x)
    _check(x, o, lse)


def test_decode_with_rising_scores_rescales():
    x = _cache(24, 2, 32, [(3000, 1), (700, 1)], seed=3)
    for i, (k, v) in enumerate(x["kv"]):
        k.add_(torch.linspace(0, 3, k.shape[0], device="cuda")[:, None, None].to(BF))
        fill_pages(x["kp"], x["vp"], x["table"], 32, i, k, v)
    x["q"].add_(0.7)
    o, lse = _attend(x)
    _check(x, o, lse)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("seqs", [[(2000, 1)] * 8, [(900, 1)] * 60, [(4000, 5)] * 3, [(1500, 300), (40, 70)]],
                         ids=["many pieces", "few pieces", "short", "chunks"])
def test_queries_and_keys_that_are_nan_show_in_their_rows_alone(seqs, dtype):
    """A row whose every score is NaN has no maximum in any piece, one with a NaN
    score among others has one: NaN by the formula both, whole or cut."""
    x = _cache(24, 2, 64, seqs, dtype=dtype)
    clean, clean_lse = _attend(x)
    last = [off + n - 1 for (c, n), off in zip(seqs, x["offs"])]
    hit = torch.zeros(clean_lse.shape, dtype=torch.bool, device="cuda")
    for i, (row, h) in enumerate(zip(last, [0, 5, 11, 12, 23] * len(seqs))):
        x["q"][row, h, (37 * i) % D] = NAN
        hit[row, h] = True
    c, n = seqs[-1]
    page = x["table"][len(seqs) - 1, c // 64]              # key c, of the first of these queries: all attend it
    x["kp"][page, 1, c % 64, 200] = NAN
    hit[x["offs"][-1]:, 12:] = True
    o, lse = _attend(x)
    assert torch.equal(torch.isnan(lse), hit)
    assert bool(torch.isnan(o[hit]).all())
    assert torch.equal(o[~hit], clean[~hit]) and torch.equal(lse[~hit], clean_lse[~hit])


def test_decode_skips_bad_pages_inside_a_sequence():
    x = _cache(24, 2, 16, [(400, 1), (300, 1), (20, 1)], seed=4)
    t = x["table"].clone()
    t[0, 2], t[0, 9], t[0, 25] = -1, 1 << 30, x["kp"].shape[0]       # the last one holds the row's own key
    t[1, :] = -2
    x["pages"] = qsa.make_pages(x["kp"], x["vp"], t.cuda())
    o, lse = _attend(x)
    assert qsa.device_status() == qsa.QSA_ERR_BAD_INDEX
    keep = torch.tensor([j for j in range(401) if j // 16 not in (2, 9, 25)]).cuda()
    k, v = x["kv"][0]
    q = x["q"][:1]
    check_forward(o[:1], lse[:1], attend64(q, k[keep], v[keep], 400, SCALE), score_error(q, k, SCALE), BF)
    assert (o[1] == 0).all() and (lse[1] == -math.inf).all()
    q, (k, v) = x["q"][2:], x["kv"][2]
    check_forward(o[2:], lse[2:], attend64(q, k, v, 20, SCALE), score_error(q, k, SCALE), BF)


def test_a_mixed_batch_is_its_parts():
    """Decode, few-token and chunk segments in one call (kernels that overlap)
    against calls of each alone, bit for bit where the kernel is the same."""
    seqs = [(900, 1), (100, 300), (33, 1), (512, 4), (0, 129), (2000, 1)]
    x = _cache(24, 2, 16, seqs, seed=5)
    o, lse = _attend(x)
    _check(x, o, lse)
    decode = [i for i, (_, n) in enumerate(seqs) if n == 1]
    y = dict(x, segs=qsa.make_segments([(x["offs"][i], 1, seqs[i][0], i) for i in decode]))
    o1, lse1 = _attend(y)
    for i in decode:
        assert torch.equal(o1[x["offs"][i]], o[x["offs"][i]]) and torch.equal(lse1[x["offs"][i]], lse[x["offs"][i]])
    assert (o1[1:301] == 5.0).all()


def test_caches_beyond_32_bit_offsets():
    """Pages whose elements lie behind 2^31 and bytes behind 2^32."""
    groups, page, n_pages = 2, 64, 72000                  # 72000 * 2 * 64 * 256 = 2.36e9 elements
    kp, vp = (torch.empty((n_pages, groups, page, D), dtype=BF, device="cuda") for _ in range(2))
    gen = torch.Generator().manual_seed(6)
    seqs = [(150, 1), (40, 150), (100, 3)]
    table = torch.full((3, 4), -1, dtype=torch.int32)
    ids = [n_pages - 1 - i for i in range(8)] + [0, 65535]
    x = dict(seqs=seqs, offs=[0, 1, 151], T=154, dt=BF, cfg=qsa.make_config(shape()), kv=[], q=_randn(gen, 154, 24, D))
    for i, (c, n) in enumerate(seqs):
        for p in range((c + n + page - 1) // page):
            table[i, p] = ids.pop(0)
        raw = _randn(gen, c + n, groups, D), _randn(gen, c + n, groups, D)
        pages = qsa.make_pages(kp, vp, table.cuda())
        qsa.qsa_append_kv(x["cfg"], pages, qsa.make_segments([(0, c + n, 0, i)]), c + n, *raw)
        pos = torch.arange(c + n, device="cuda")
        pg = table[i].cuda().long()[pos // page]
        x["kv"].append((kp[pg, :, pos % page], vp[pg, :, pos % page]))
        assert torch.equal(x["kv"][-1][1], raw[1])
    x["pages"] = qsa.make_pages(kp, vp, table.cuda())
    x["segs"] = qsa.make_segments([(o, n, c, i) for i, ((c, n), o) in enumerate(zip(seqs, x["offs"]))])
    o, lse = _attend(x)
    qsa.qsa_device_status()
    _check(x, o, lse)


# ------------------------------------------------------------------ gradient
def _prompts(heads, groups, lens, seed=1, dtype="bf16", gap=0):
    sh = shape(heads, groups, dtype)
    dt = torch_dtype(sh)
    gen = torch.Generator().manual_seed(seed)
    T = sum(lens) + gap * len(lens)
    offs, at = [], 0
    for n in lens:
        offs.append(at)
        at += n + gap
    x = dict(cfg=qsa.make_config(sh), T=T, lens=lens, offs=offs, dt=dt,
             segs=qsa.make_segments([(o, n, 0, 0) for o, n in zip(offs, lens)]))
    for name, h in (("q", heads), ("dout", heads), ("k", groups), ("v", groups)):
        x[name] = _randn(gen, T, h, D, dtype=dt)
    return x


def _train(x, stream=None):
    o = torch.full_like(x["q"], 5.0)
    lse = torch.full(x["q"].shape[:2], 5.0, device="cuda")
    qsa.qsa_prompt_attn_fwd(x["cfg"], x["segs"], x["T"], x["q"], x["k"], x["v"], o, lse,
                            workspace(x["cfg"], x["segs"], x["T"], qsa.QSA_OP_PROMPT_ATTN), stream)
    g = [torch.full_like(x[n], 5.0) for n in ("q", "k", "v")]
    qsa.qsa_prompt_attn_bwd(x["cfg"], x["segs"], x["T"], x["q"], x["k"], x["v"], o, lse, x["dout"], *g,
                            workspace(x["cfg"], x["segs"], x["T"], qsa.QSA_OP_PROMPT_ATTN_BWD), stream)
    return o, lse, g


def _check_grads(x, grads, i, rows=slice(None)):
    off, n = x["offs"][i], x["lens"][i]
    t = slice(off, off + n)
    ref, tol = gradients64(x["q"][t], x["k"][t], x["v"][t], x["dout"][t], SCALE)
    for name, got in zip(("dq", "dk", "dv"), grads):
        err = ((got[t].to(F64) - ref[name]).abs() / (tol[name] + 1e-30))[rows]
        assert (err <= 1).all(), (name, i, err.max().item())


@pytest.mark.parametrize("heads,groups", [(32, 2), (24, 2), (7, 1), (4, 4)])
@pytest.mark.parametrize("lens", [[1], [127, 1, 128, 129, 2], [255, 256, 257], [1300, 40]])
def test_gradient_around_the_tiles(heads, groups, lens):
    x = _prompts(heads, groups, lens)
    _, _, grads = _train(x)
    qsa.qsa_device_status()
    for i in range(len(lens)):
        _check_grads(x, grads, i)


@pytest.mark.parametrize("name,value", [("dout", NAN), ("dout", float("inf")), ("q", NAN), ("k", float("inf")),
                                        ("v", NAN), ("v", -float("inf"))])
def test_a_gradient_of_what_is_not_finite_stays_where_it_belongs(name, value):
    """One token of the second prompt is not finite: the other prompts are those
    of the clean inputs, bit for bit, and in its own prompt the tokens that no
    pair with it reaches still have the right gradient."""
    x = _prompts(24, 2, [200, 333, 70], seed=2)
    _, _, clean = _train(x)
    at = 150                                             # of the second prompt
    bad = dict(x)
    bad[name] = x[name].clone()
    bad[name][200 + at, 0, 3] = value                    # query head 0 or KV group 0
    _, _, grads = _train(bad)
    for a, b in zip(grads, clean):
        assert torch.equal(a[:200], b[:200]) and torch.equal(a[533:], b[533:])
    heads = slice(0, 1) if name in ("dout", "q") else slice(0, 12)
    assert not torch.isfinite(grads[0][200 + at, heads].float()).all()
    # group 1 does not see it; rows before the token do not attend it; keys behind it are not attended by it
    t = slice(200, 533)
    ref, tol = gradients64(x["q"][t], x["k"][t], x["v"][t], x["dout"][t], SCALE)
    dq, dk, dv = (g[t].to(F64) for g in grads)
    assert ((dq[:, 12:] - ref["dq"][:, 12:]).abs() <= tol["dq"][:, 12:] + 1e-30).all()
    assert ((dq[:at] - ref["dq"][:at]).abs() <= tol["dq"][:at] + 1e-30).all()
    assert ((dk[:, 1] - ref["dk"][:, 1]).abs() <= tol["dk"][:, 1] + 1e-30).all()
    if name in ("dout", "q"):
        assert ((dk[at + 1:, 0] - ref["dk"][at + 1:, 0]).abs() <= tol["dk"][at + 1:, 0] + 1e-30).all()
        assert ((dv[at + 1:, 0] - ref["dv"][at + 1:, 0]).abs() <= tol["dv"][at + 1:, 0] + 1e-30).all()


def test_rows_of_no_prompt_may_hold_anything():
    x = _prompts(24, 2, [130, 61, 300], seed=3, gap=5)
    for off, n in zip(x["offs"], x["lens"]):
        for name in ("q", "k", "v", "dout"):
            x[name][off + n:off + n + 5] = NAN
    o, lse, grads = _train(x)
    for i, (off, n) in enumerate(zip(x["offs"], x["lens"])):
        _check_grads(x, grads, i)
        for t in (o, lse, *grads):
            assert (t[off + n:off + n + 5] == 5.0).all()


# ------------------------------------------------------------------ streams and graphs
def test_two_calls_on_two_streams():
    a, b = _cache(24, 2, 64, [(5000, 1), (0, 300)], seed=7), _cache(24, 2, 64, [(300, 500), (9000, 1)], seed=8)
    ref = [_attend(x) for x in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    ws = [workspace(x["cfg"], x["segs"], x["T"], qsa.QSA_OP_PAGED_ATTN) for x in (a, b)]
    torch.cuda.synchronize()
    out = []
    for _ in range(5):
        for x, s, w in zip((a, b), streams, ws):
            with torch.cuda.stream(s):
                out.append(_attend(x, w))
    torch.cuda.synchronize()
    for i, (o, lse) in enumerate(out):
        assert torch.equal(o, ref[i % 2][0]) and torch.equal(lse, ref[i % 2][1])


def test_a_captured_step_replays_on_new_inputs():
    """Append, attention over the cache and a training step in one graph."""
    x = _cache(24, 2, 48, [(700, 1), (90, 260), (20, 3)], seed=9, poison=0.0)
    y = _prompts(24, 2, [300, 77], seed=10)
    gen = torch.Generator().manual_seed(11)
    k, v, q = _randn(gen, x["T"], 2, D), _randn(gen, x["T"], 2, D), _randn(gen, x["T"], 24, D)
    o, lse = torch.zeros_like(x["q"]), torch.zeros(x["q"].shape[:2], device="cuda")
    ws = workspace(x["cfg"], x["segs"], x["T"], qsa.QSA_OP_PAGED_ATTN)
    po, pl = torch.zeros_like(y["q"]), torch.zeros(y["q"].shape[:2], device="cuda")
    g = [torch.zeros_like(y[n]) for n in ("q", "k", "v")]
    wf = workspace(y["cfg"], y["segs"], y["T"], qsa.QSA_OP_PROMPT_ATTN)
    wb = workspace(y["cfg"], y["segs"], y["T"], qsa.QSA_OP_PROMPT_ATTN_BWD)

    def step():
        qsa.qsa_append_kv(x["cfg"], x["pages"], x["segs"], x["T"], k, v, q, x["q"])
        qsa.qsa_paged_attn_fwd(x["cfg"], x["pages"], x["segs"], x["T"], x["q"], o, lse, ws)
        qsa.qsa_prompt_attn_fwd(y["cfg"], y["segs"], y["T"], y["q"], y["k"], y["v"], po, pl, wf)
        qsa.qsa_prompt_attn_bwd(y["cfg"], y["segs"], y["T"], y["q"], y["k"], y["v"], po, pl, y["dout"], *g, wb)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (12, 13):
        gen = torch.Generator().manual_seed(seed)
        for t in (k, v, q, y["q"], y["k"], y["v"], y["dout"]):
            t.copy_(_randn(gen, *t.shape))
        for t in (o, lse, po, pl, *g):
            t.zero_()
        graph.replay()
        got = [t.clone() for t in (x["kp"], x["vp"], x["q"], o, lse, po, pl, *g)]
        for t in (o, lse, po, pl, *g):
            t.zero_()
        step()
        for a, b in zip(got, (x["kp"], x["vp"], x["q"], o, lse, po, pl, *g)):
            assert torch.equal(a, b)
    qsa.qsa_device_status()
