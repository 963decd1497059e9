"""Plain 64-bit forms of the paged append and the dense attention, and the
error bounds that the arithmetic of the kernels allows.

Bounds (u = half a step of the I/O dtype, 2^-8 for bf16, 2^-24 for fp32):
  scores   fp32 sums of 256 products: |ds| <= e = 2^-24 * 256 * scale * max|q| max|k|
           (Euclidean norms), also the relative error of P, plus 2^-20 for the
           fp32 exponential and sums;
  o        |do| <= w sum_j P_j |v_j| + u |o|, w = e + 2^-20 + (u for bf16: P is
           rounded for the tensor-core product);
  lse      e + 2^-20 (1 + |lse|);
  dS       |d(dS_j)| <= w |dS_j| + P_j (e2 + ddelta), e2 the fp32 error of
           dout . v, ddelta <= sum_d |dout_d| (|do_d|) + fp32;
  dq, dk   scale * sum |d(dS)| |k or q| + u |result|;   dv: w sum P |dout| + u |dv|.
Sums over many rows add 2^-24 * (number of terms) relative to the sum of
absolute values (both dtypes accumulate in fp32).
"""
import math
import types

import torch

import block_sparse_attention_22_b200 as qsa

D = 256
F64 = torch.float64


def shape(heads=24, groups=2, dtype="bf16", rope_fraction=0.25, rope_base=1e7):
    return types.SimpleNamespace(r=4, budget_tokens=2048, n_heads=heads, n_groups=groups, head_dim=D, idx_heads=4,
                                 idx_dim=64, rope_fraction=rope_fraction, rope_base=rope_base, dtype=dtype)


def torch_dtype(sh):
    return torch.bfloat16 if sh.dtype == "bf16" else torch.float32


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def workspace(cfg, segs, T, op):
    n = qsa.workspace_size(cfg, segs, T, op)
    return torch.full((max(1, n),), 0xFF, dtype=torch.uint8, device="cuda")      # NaN bytes: contents are ignored


def make_table(lens, page, gen, spare=2, pad=-7):
    """Shuffled page table for sequences of the given lengths; entries past a
    sequence's last page hold `pad`."""
    need = [(n + page - 1) // page for n in lens]
    n_pages = sum(need) + spare
    perm = torch.randperm(n_pages, generator=gen)
    table = torch.full((len(lens), max(1, max(need)) + 1), pad, dtype=torch.int32)
    at = 0
    for i, m in enumerate(need):
        table[i, :m] = perm[at:at + m].to(torch.int32)
        at += m
    return table, n_pages


def fill_pages(kp, vp, table, page, i, k, v):
    """Rows 0.. of sequence i <- k, v [L, G, D]."""
    pos = torch.arange(k.shape[0], device=kp.device)
    pg = table[i].to(kp.device).long()[pos // page]
    kp[pg, :, pos % page] = k
    vp[pg, :, pos % page] = v


def attend64(q, k, v, pos0, scale):
    """Reference of one sequence: q [n,H,D], k, v [L,G,D] (any dtype), rows at
    pos0..; returns o, lse, sum_j P|v| in fp64.  Only keys at or before a row's
    position enter (masked values may be anything)."""
    n, H, _ = q.shape
    G = k.shape[1]
    hpg = H // G
    o = torch.zeros((n, H, D), dtype=F64, device=q.device)
    av = torch.zeros_like(o)
    lse = torch.zeros((n, H), dtype=F64, device=q.device)
    for h in range(H):
        kk, vv = k[:, h // hpg].to(F64), v[:, h // hpg].to(F64)
        step = max(1, (1 << 25) // max(1, kk.shape[0]))
        for a in range(0, n, step):
            b = min(n, a + step)
            L = min(kk.shape[0], pos0 + b)
            s = (q[a:b, h].to(F64) @ kk[:L].t()) * scale
            mask = torch.arange(L, device=q.device)[None] > torch.arange(pos0 + a, pos0 + b, device=q.device)[:, None]
            s.masked_fill_(mask, -math.inf)
            lz = torch.logsumexp(s, 1)
            p = torch.exp(s - lz[:, None])
            o[a:b, h], av[a:b, h], lse[a:b, h] = p @ vv[:L], p @ vv[:L].abs(), lz
    return o, lse, av


def score_error(q, k, scale):
    """e of the module's bounds."""
    qn = q.to(F64).norm(dim=-1).max().item() if q.numel() else 0.0
    kn = k.to(F64).norm(dim=-1).max().item() if k.numel() else 0.0
    return 2.0 ** -24 * D * scale * qn * kn


def check_forward(o, lse, ref, e, dtype, where=""):
    ro, rl, av = ref
    u = half_step(dtype)
    w = e + 2.0 ** -20 + (u if dtype == torch.bfloat16 else 0.0)
    err = (o.to(F64) - ro).abs()
    tol = w * av + u * ro.abs() * (1 + w) + 1e-30
    bad = ~(err <= tol)
    assert not bad.any(), (where, "o", int(bad.sum()), (err / tol).max().item(), bad.nonzero()[:3].tolist())
    if lse is not None:
        el = (lse.to(F64) - rl).abs()
        tl = e + 2.0 ** -20 * (1 + rl.abs())
        assert (el <= tl).all(), (where, "lse", (el / tl).max().item())


def gradients64(q, k, v, dout, scale):
    """Reference gradients of one prompt and the sums of absolute values that
    the bounds need."""
    n, H, _ = q.shape
    G = k.shape[1]
    hpg = H // G
    z = lambda t: torch.zeros(t.shape, dtype=F64, device=q.device)
    dq, dk, dv = z(q), z(k), z(v)
    aq, ak, av_ = z(q), z(k), z(v)          # sum |dS| |k|, sum |dS| |q|, sum P |dout|
    pq, pk = z(q), z(k)                     # sum P ddelta |k|, sum P ddelta |q|
    u = half_step(q.dtype)
    e = score_error(q, k, scale)
    w = e + 2.0 ** -20 + (u if q.dtype == torch.bfloat16 else 0.0)
    tri = torch.ones((n, n), dtype=torch.bool, device=q.device).triu(1)
    for h in range(H):
        g = h // hpg
        qq, kk, vv, dd = (x.to(F64) for x in (q[:, h], k[:, g], v[:, g], dout[:, h]))
        s = (qq @ kk.t()) * scale
        s.masked_fill_(tri, -math.inf)
        p = torch.exp(s - torch.logsumexp(s, 1, keepdim=True))
        o = p @ vv
        do = w * (p @ vv.abs()) + u * o.abs()
        dp = dd @ vv.t()
        ds = p * (dp - (dd * o).sum(1, keepdim=True))
        dq[:, h] = scale * (ds @ kk)
        dk[:, g] += scale * (ds.t() @ qq)
        dv[:, g] += p.t() @ dd
        e2 = 2.0 ** -24 * D * (dd.norm(dim=1).max() * vv.norm(dim=1).max()).item()
        slack = (dd.abs() * do).sum(1, keepdim=True) + 2 * e2
        aq[:, h] = scale * (ds.abs() @ kk.abs())
        ak[:, g] += scale * (ds.abs().t() @ qq.abs())
        av_[:, g] += p.t() @ dd.abs()
        pq[:, h] = scale * ((p * slack) @ kk.abs())
        pk[:, g] += scale * ((p * slack).t() @ qq.abs())
    acc = 2.0 ** -24 * n * hpg
    tol = dict(dq=(w + 2.0 ** -24 * n) * aq + pq * (1 + w) + u * dq.abs(),
               dk=(w + acc) * ak + pk * (1 + w) + u * dk.abs(), dv=(w + acc) * av_ + u * dv.abs())
    return dict(dq=dq, dk=dk, dv=dv), tol


def rotate64(x, pos, rope_fraction=0.25, base=1e7):
    """x [n, heads, D] rotated to positions pos [n], in fp64."""
    rd = int(math.floor(D * rope_fraction))
    rd -= rd & 1
    y = x.to(F64).clone()
    if rd == 0:
        return y
    half = rd // 2
    ang = pos.to(F64)[:, None] * torch.tensor([base ** (-2.0 * i / rd) for i in range(half)], dtype=F64,
                                              device=x.device)
    c, s = ang.cos()[:, None], ang.sin()[:, None]
    a, b = y[..., :half].clone(), y[..., half:rd].clone()
    y[..., :half] = a * c - b * s
    y[..., half:rd] = b * c + a * s
    return y
