"""Performance cases of the dense attention operators around a paged KV cache.

Three operators, all over the layer geometry of the sparse path (24 query
heads, 2 KV groups, head dim 256, rotary base 1e7 on a quarter of the dims)
and its neighbours:

  append  keys and values of new tokens written to a paged cache, the keys
          (and the queries) rotated to their positions on the way
  paged   causal grouped-query attention of new tokens over a paged cache:
          single tokens, a few tokens, long chunks
  prompt  causal grouped-query attention over packed whole prompts, forward
          alone or with its gradient ("train")

`run` computes them in plain torch operations in 32 bits (`own` false) or
through the library's entry points (`own` true).
"""
import math
import types

import torch

own = False

D = 256                    # head dim of every case
ROPE_FRACTION = 0.25
ROPE_BASE = 1e7


# ------------------------------------------------------------------ cases
# A case: op, dtype, heads, groups, and for each sequence how many tokens are
# cached before the call ("ctx") and how many are new ("new"), written as
# "ctx+new" joined by commas ("ctx+new*n" repeats).  Prompt cases have ctx 0.
def listed():
    return [
        # one decode step of 8 sequences: the latency of a single-token append
        dict(name="append_decode_8", op="append", dtype="bf16", heads=24, groups=2, page=64, seqs="16383+1*8",
             with_q=True),
        # a prefill chunk of 4096 tokens over a cached prefix, queries rotated too
        dict(name="append_chunk_4k", op="append", dtype="bf16", heads=24, groups=2, page=64, seqs="12000+4096",
             with_q=True),
        # packed odd-length prompts in fp32, small pages, keys and values alone
        dict(name="append_prompts_f32", op="append", dtype="f32", heads=16, groups=4, page=16,
             seqs="0+4097,0+1,0+333,7+2050,100+15", with_q=False),
        # decode of 8 short sequences, small pages: launch latency counts
        dict(name="paged_decode_short", op="paged", dtype="bf16", heads=24, groups=2, page=16,
             seqs="511+1,1300+1,0+1,77+1,2047+1,640+1,128+1,1023+1"),
        # decode of 32 sequences of ragged length: a serving step, HBM bound
        dict(name="paged_decode_32", op="paged", dtype="bf16", heads=24, groups=2, page=64,
             seqs="32767+1*8,16000+1*8,49999+1*8,32001+1*8"),
        # one sequence at a long context: the keys of one query split over the GPU
        dict(name="paged_decode_256k", op="paged", dtype="bf16", heads=24, groups=2, page=128, seqs="262143+1"),
        # a 4096-token prefill chunk at the end of a 131072-token sequence
        dict(name="paged_chunk_128k", op="paged", dtype="bf16", heads=24, groups=2, page=64, seqs="126976+4096"),
        # a mixed step: decode, speculative decode, ragged chunks, pages of 48 tokens
        dict(name="paged_mixed", op="paged", dtype="bf16", heads=24, groups=2, page=48,
             seqs="5000+1*6,3001+5*3,2000+777,0+1301,1+255,9000+0"),
        # two whole prompts of 8192 tokens, forward
        dict(name="prompt_fwd_8k", op="prompt", dtype="bf16", heads=24, groups=2, train=False, seqs="0+8192*2"),
        # training step of two packed prompts of 8192 tokens
        dict(name="prompt_train_8k", op="prompt", dtype="bf16", heads=24, groups=2, train=True, seqs="0+8192*2"),
        # training step of packed documents of odd lengths, one of them a single token
        dict(name="prompt_train_ragged", op="prompt", dtype="bf16", heads=16, groups=2, train=True,
             seqs="0+1,0+977,0+130,0+3001,0+63,0+511,0+1500"),
        # the fp32 training step of a small model
        dict(name="prompt_train_f32", op="prompt", dtype="f32", heads=24, groups=2, train=True,
             seqs="0+256,0+700,0+33"),
    ]


def draw(rng):
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    heads, groups = rng.choice([(24, 2), (24, 2), (16, 2), (16, 4), (8, 8), (12, 1), (6, 2), (32, 2)])
    op = rng.choice(["append", "paged", "paged", "prompt"])
    case = dict(op=op, dtype="bf16" if rng.random() < 0.8 else "f32", heads=heads, groups=groups)
    f32 = case["dtype"] == "f32"
    if op != "prompt":
        case["page"] = rng.choice([16, 32, 48, 64, 96, 128, 256, 1024])
    if op == "append":
        case["with_q"] = rng.random() < 0.6
        n = log_int(1, 32)
        if rng.random() < 0.4:
            seqs = ["%d+1" % (log_int(1, 20000) - 1) for _ in range(n)]
        else:
            n = min(n, 6)
            seqs = ["%d+%d" % (log_int(1, 9000) - 1, log_int(1, 5000)) for _ in range(n)]
    elif op == "paged":
        kind = rng.choice(["decode", "few", "chunk", "mixed"])
        top = 8000 if f32 else 70000
        if kind == "decode":
            seqs = ["%d+1" % (log_int(1, top) - 1) for _ in range(log_int(1, 24))]
        elif kind == "few":
            seqs = ["%d+%d" % (log_int(1, top) - 1, rng.randint(2, 12)) for _ in range(log_int(1, 12))]
        elif kind == "chunk":
            seqs = ["%d+%d" % (log_int(1, top // 2) - 1, log_int(16, 500 if f32 else 3500))]
        else:
            seqs = ["%d+1" % (log_int(1, top // 4) - 1) for _ in range(rng.randint(1, 6))]
            seqs += ["%d+%d" % (log_int(1, top // 8) - 1, log_int(2, 300 if f32 else 1400))
                     for _ in range(rng.randint(1, 4))]
    else:
        case["train"] = rng.random() < 0.5
        n = rng.randint(1, 8)
        seqs = ["0+%d" % log_int(1, 900 if f32 else 5000) for _ in range(n)]
    case["seqs"] = ",".join(seqs)
    return case


def _seqs(case):
    out = []
    for part in case["seqs"].split(","):
        part, _, rep = part.partition("*")
        ctx, new = part.split("+")
        out += [(int(ctx), int(new))] * (int(rep) if rep else 1)
    return out


def work(case):
    """Bytes: inputs once, outputs once.  Flops: products over the unmasked pairs."""
    e = 2 if case["dtype"] == "bf16" else 4
    H, G = case["heads"], case["groups"]
    seqs = _seqs(case)
    T = sum(n for _, n in seqs)
    if case["op"] == "append":
        b = 2 * 2 * T * G * D * e + (2 * T * H * D * e if case["with_q"] else 0)
        return {"bytes": b, "flops": 3 * T * int(D * ROPE_FRACTION) * (G + (H if case["with_q"] else 0))}
    pairs = sum(n * c + n * (n + 1) // 2 for c, n in seqs)
    keys = sum(c + n for c, n in seqs if n > 0)
    b = 2 * T * H * D * e + 2 * keys * G * D * e + 4 * T * H
    f = 4 * D * H * pairs
    if case.get("train"):
        b += 2 * T * H * D * e + 2 * T * G * D * e
        f += 10 * D * H * pairs
    return {"bytes": b, "flops": f}


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(1000003 * seed + 17)
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    H, G = case["heads"], case["groups"]
    seqs = _seqs(case)
    T = sum(n for _, n in seqs)
    offs, at = [], 0
    for _, n in seqs:
        offs.append(at)
        at += n

    def randn(*shape):
        return torch.randn(shape, generator=gen, device="cuda", dtype=dt)

    s = dict(case=case, seqs=seqs, offs=offs, T=T, dt=dt, H=H, G=G, hpg=H // G, scale=1.0 / math.sqrt(D))
    if case["op"] == "append":
        # one fused projection holds q, k and v of a token, as a layer's output does
        qkv = randn(T, (H + 2 * G) * D)
        s["q"] = qkv[:, :H * D].view(T, H, D) if case["with_q"] else None
        s["k"] = qkv[:, H * D:(H + G) * D].view(T, G, D)
        s["v"] = qkv[:, (H + G) * D:].view(T, G, D)
        if case["with_q"]:
            s["q_out"] = torch.empty((T, H, D), device="cuda", dtype=dt)
    else:
        # queries share a direction that each sequence's first key answers (the
        # sink that attention keeps on the first token); the rest is N(0, 1)
        sink = randn(G, 1, D)
        s["q"] = randn(T, H, D).view(T, G, H // G, D).add_(sink, alpha=0.25).view(T, H, D)
    if case["op"] == "prompt":
        s["k"] = randn(T, G, D)
        s["v"] = randn(T, G, D)
        for (_, n), off in zip(seqs, offs):
            if n:
                s["k"][off].add_(sink[:, 0], alpha=0.25)
        s["o"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((T, H), device="cuda", dtype=torch.float32)
        if case["train"]:
            s["dout"] = randn(T, H, D)
            for n in ("q", "k", "v"):
                s["d" + n] = torch.empty_like(s[n])
    else:
        P = case["page"]
        need = [(c + n + P - 1) // P for c, n in seqs]
        if case["op"] == "append":
            # only the pages that receive tokens are real; a sequence's older pages are any pages
            first = [c // P if n else m for (c, n), m in zip(seqs, need)]
        else:
            first = [0] * len(seqs)
        n_pages = sum(m - f for m, f in zip(need, first)) + 3
        perm = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
        table = torch.zeros((len(seqs), max(1, max(need))), device="cuda", dtype=torch.int32)
        at = 0
        for i, (m, f) in enumerate(zip(need, first)):
            table[i, f:m] = perm[at:at + m - f]
            at += m - f
        s["table"] = table
        s["kp"] = randn(n_pages, G, P, D)
        s["vp"] = randn(n_pages, G, P, D)
        if case["op"] == "paged":
            for i, (c, n) in enumerate(seqs):
                if n:
                    s["kp"][table[i, 0].long(), :, 0] += 0.25 * sink[:, 0]
            s["o"] = torch.empty_like(s["q"])
            s["lse"] = torch.empty((T, H), device="cuda", dtype=torch.float32)
    if own:
        import block_sparse_attention_22_b200 as qsa
        shape = types.SimpleNamespace(r=4, budget_tokens=2048, n_heads=H, n_groups=G, head_dim=D, idx_heads=4,
                                      idx_dim=128, rope_fraction=ROPE_FRACTION, rope_base=ROPE_BASE,
                                      dtype=case["dtype"])
        s["qsa"] = qsa
        s["cfg"] = qsa.make_config(shape)
        s["segs"] = qsa.make_segments([(off, n, c, i) for i, ((c, n), off) in enumerate(zip(seqs, offs))])
        if case["op"] != "prompt":
            s["pages"] = qsa.make_pages(s["kp"], s["vp"], s["table"])

        def workspace(op):
            n = qsa.workspace_size(s["cfg"], s["segs"], T, op)
            return torch.empty(max(1, n), device="cuda", dtype=torch.uint8)

        if case["op"] == "paged":
            s["ws"] = workspace(qsa.QSA_OP_PAGED_ATTN)
        elif case["op"] == "prompt":
            s["ws"] = workspace(qsa.QSA_OP_PROMPT_ATTN)
            if case["train"]:
                s["ws_bwd"] = workspace(qsa.QSA_OP_PROMPT_ATTN_BWD)
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    op = s["case"]["op"]
    if own:
        qsa = s["qsa"]
        if op == "append":
            qsa.qsa_append_kv(s["cfg"], s["pages"], s["segs"], s["T"], s["k"], s["v"], s["q"], s.get("q_out"))
            return (s["kp"], s["vp"]) + ((s["q_out"],) if "q_out" in s else ())
        if op == "paged":
            qsa.qsa_paged_attn_fwd(s["cfg"], s["pages"], s["segs"], s["T"], s["q"], s["o"], s["lse"], s["ws"])
            return s["o"], s["lse"]
        qsa.qsa_prompt_attn_fwd(s["cfg"], s["segs"], s["T"], s["q"], s["k"], s["v"], s["o"], s["lse"], s["ws"])
        if not s["case"]["train"]:
            return s["o"], s["lse"]
        qsa.qsa_prompt_attn_bwd(s["cfg"], s["segs"], s["T"], s["q"], s["k"], s["v"], s["o"], s["lse"], s["dout"],
                                s["dq"], s["dk"], s["dv"], s["ws_bwd"])
        return s["o"], s["lse"], s["dq"], s["dk"], s["dv"]
    if op == "append":
        return _append(s)
    if op == "paged":
        return _paged(s)
    return _prompt(s)


def _rotate(x, pos):
    """x [n, heads, D] at positions pos [n]: fp64 angles, 32-bit products, one rounding."""
    rd = int(D * ROPE_FRACTION)
    half = rd // 2
    theta = ROPE_BASE ** (-2.0 * torch.arange(half, device=x.device, dtype=torch.float64) / rd)
    ang = pos.double()[:, None] * theta
    c, sn = ang.cos().float()[:, None], ang.sin().float()[:, None]
    y = x.float()
    a, b = y[..., :half], y[..., half:rd]
    return torch.cat([a * c - b * sn, b * c + a * sn, y[..., rd:]], dim=-1).to(x.dtype)


def _append(s):
    P = s["case"]["page"]
    for i, ((c, n), off) in enumerate(zip(s["seqs"], s["offs"])):
        if n == 0:
            continue
        pos = torch.arange(c, c + n, device="cuda")
        page = s["table"][i].long()[pos // P]
        s["kp"][page, :, pos % P] = _rotate(s["k"][off:off + n], pos)
        s["vp"][page, :, pos % P] = s["v"][off:off + n]
        if "q_out" in s:
            s["q_out"][off:off + n] = _rotate(s["q"][off:off + n], pos)
    return (s["kp"], s["vp"]) + ((s["q_out"],) if "q_out" in s else ())


def _probabilities(q, k, pos, scale):
    """exp(scores - max) over the keys at or before each row's position, with
    the sums and the log-sum-exp; q [rows, D], pos [rows], k [keys, D]."""
    sc = (q @ k.t()) * scale
    sc.masked_fill_(torch.arange(k.shape[0], device=k.device)[None, :] > pos[:, None], -math.inf)
    m = sc.amax(dim=1, keepdim=True)
    p = sc.sub_(m).exp_()
    total = p.sum(dim=1, keepdim=True)
    return p, total, (m + total.log())[:, 0]


def _row_chunk(hpg, keys):
    return max(1, (1 << 28) // max(1, keys * hpg))


def _attend(q, k, v, pos0, scale, o, lse):
    """o, lse of q [n, hpg, D] (fp32) at positions pos0.. over k, v [keys, D] (fp32)."""
    n, hpg, _ = q.shape
    step = _row_chunk(hpg, k.shape[0])
    for a in range(0, n, step):
        b = min(n, a + step)
        kk, vv = k[:pos0 + b], v[:pos0 + b]
        pos = torch.arange(pos0 + a, pos0 + b, device=q.device).repeat_interleave(hpg)
        p, total, l = _probabilities(q[a:b].reshape(-1, D), kk, pos, scale)
        o[a:b] = ((p @ vv) / total).view(b - a, hpg, D).to(o.dtype)
        lse[a:b] = l.view(b - a, hpg)


def _paged(s):
    P, hpg = s["case"]["page"], s["hpg"]
    for i, ((c, n), off) in enumerate(zip(s["seqs"], s["offs"])):
        if n == 0:
            continue
        L = c + n
        pages = s["table"][i, :(L + P - 1) // P].long()
        for g in range(s["G"]):
            k = s["kp"][pages, g].reshape(-1, D)[:L].float()
            v = s["vp"][pages, g].reshape(-1, D)[:L].float()
            h = slice(g * hpg, (g + 1) * hpg)
            _attend(s["q"][off:off + n, h].float(), k, v, c, s["scale"], s["o"][off:off + n, h],
                    s["lse"][off:off + n, h])
    return s["o"], s["lse"]


def _prompt(s):
    hpg, scale = s["hpg"], s["scale"]
    for (_, n), off in zip(s["seqs"], s["offs"]):
        if n == 0:
            continue
        for g in range(s["G"]):
            t, h = slice(off, off + n), slice(g * hpg, (g + 1) * hpg)
            q, k, v = s["q"][t, h].float(), s["k"][t, g].float(), s["v"][t, g].float()
            _attend(q, k, v, 0, scale, s["o"][t, h], s["lse"][t, h])
            if s["case"]["train"]:
                _gradients(s, t, h, g, q, k, v, s["dout"][t, h].float())
    if not s["case"]["train"]:
        return s["o"], s["lse"]
    return s["o"], s["lse"], s["dq"], s["dk"], s["dv"]


def _gradients(s, t, h, g, q, k, v, dout):
    n, hpg, _ = q.shape
    dk, dv = torch.zeros_like(k), torch.zeros_like(v)
    step = _row_chunk(hpg, n)
    for a in range(0, n, step):
        b = min(n, a + step)
        kk, vv = k[:b], v[:b]
        pos = torch.arange(a, b, device=q.device).repeat_interleave(hpg)
        qq, dd = q[a:b].reshape(-1, D), dout[a:b].reshape(-1, D)
        p, total, _ = _probabilities(qq, kk, pos, s["scale"])
        p = p.div_(total)
        dv[:b] += p.t() @ dd
        dp = dd @ vv.t()
        ds = dp.sub_((p * dp).sum(dim=1, keepdim=True)).mul_(p).mul_(s["scale"])
        dk[:b] += ds.t() @ qq
        s["dq"][t, h][a:b] = (ds @ kk).view(b - a, hpg, D).to(s["dt"])
    s["dk"][t, g] = dk.to(s["dt"])
    s["dv"][t, g] = dv.to(s["dt"])


# ------------------------------------------------------------------ definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    G, hpg = s["G"], s["hpg"]
    if case["op"] == "append":
        kp, vp = s["kp"].to(f64), s["vp"].to(f64)
        q_out = torch.zeros((s["T"], s["H"], D), device="cuda", dtype=f64)
        rd = int(D * ROPE_FRACTION)
        inv = torch.tensor([ROPE_BASE ** (-2.0 * i / rd) for i in range(rd // 2)], device="cuda", dtype=f64)
        for i, ((c, n), off) in enumerate(zip(s["seqs"], s["offs"])):
            # rotate-half as a complex product
            p = torch.arange(c, c + n, device="cuda")
            turn = torch.polar(torch.ones((n, 1, rd // 2), device="cuda", dtype=f64), (p.to(f64)[:, None] * inv)[:, None])

            def turned(x):
                x = x.to(f64).clone()
                z = torch.complex(x[..., :rd // 2].contiguous(), x[..., rd // 2:rd].contiguous()) * turn
                x[..., :rd // 2] = z.real
                x[..., rd // 2:rd] = z.imag
                return x

            pg = s["table"][i].long()[torch.div(p, case["page"], rounding_mode="floor")]
            r = p % case["page"]
            k = turned(s["k"][off:off + n])
            for g in range(G):
                kp[pg, g, r] = k[:, g]
                vp[pg, g, r] = s["v"][off:off + n, g].to(f64)
            if "q_out" in s:
                q_out[off:off + n] = turned(s["q"][off:off + n])
        return (kp, vp) + ((q_out,) if "q_out" in s else ())
    train = bool(case.get("train"))
    o = torch.zeros((s["T"], s["H"], D), device="cuda", dtype=f64)
    lse = torch.zeros((s["T"], s["H"]), device="cuda", dtype=f64)
    grads = [torch.zeros(s[n].shape, device="cuda", dtype=f64) for n in ("q", "k", "v")] if train else []
    for i, ((c, n), off) in enumerate(zip(s["seqs"], s["offs"])):
        if n == 0:
            continue
        L = c + n
        for g in range(G):
            if case["op"] == "paged":
                j = torch.arange(L, device="cuda")
                row = s["table"][i].long()[j // case["page"]]
                k = s["kp"][row, g, j % case["page"]].to(f64)
                v = s["vp"][row, g, j % case["page"]].to(f64)
            else:
                k, v = s["k"][off:off + n, g].to(f64), s["v"][off:off + n, g].to(f64)
            step = max(1, (1 << 27) // L)
            for h in range(g * hpg, (g + 1) * hpg):
                for a in range(0, n, step):
                    b = min(n, a + step)
                    q = s["q"][off + a:off + b, h].to(f64)
                    z = torch.einsum("td,jd->tj", q * s["scale"], k)
                    seen = torch.ones((b - a, L), device="cuda", dtype=torch.bool).tril_(c + a)
                    z = torch.where(seen, z, torch.full((), -math.inf, device="cuda", dtype=f64))
                    lz = torch.logsumexp(z, dim=1)
                    w = torch.exp(z - lz[:, None])
                    out = torch.einsum("tj,jd->td", w, v)
                    o[off + a:off + b, h] = out
                    lse[off + a:off + b, h] = lz
                    if train:
                        dy = s["dout"][off + a:off + b, h].to(f64)
                        dz = w * (torch.einsum("td,jd->tj", dy, v) - (dy * out).sum(1, keepdim=True))
                        grads[0][off + a:off + b, h] = s["scale"] * torch.einsum("tj,jd->td", dz, k)
                        grads[1][off:off + n, g] += s["scale"] * torch.einsum("tj,td->jd", dz, q)
                        grads[2][off:off + n, g] += torch.einsum("tj,td->jd", w, dy)
    return (o, lse, *grads)
