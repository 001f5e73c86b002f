"""Helpers of the 4-bit cache tests: records built and read in plain torch, and
attention over them in 64 bits with a bound on the kernel's roundings."""
from __future__ import annotations

import math

import torch

U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}  # half a step, relative


def pack_records(kc, vc, params):
    """Codes uint8 [..., BS, D] and params T [..., BS, 4] as records [..., BS * (D + 8)]."""
    BS, D = kc.shape[-2:]
    x = min(D, 128)

    def rows(c):
        parts = [c[..., i:i + x] for i in range(0, D, x)]  # [D/x] of [..., BS, x]
        return torch.cat([(p[..., ::2] + 16 * p[..., 1::2]).flatten(-2) for p in parts], -1)

    return torch.cat([rows(kc), rows(vc), params.contiguous().view(torch.uint8).flatten(-2)], -1)


def read_records(rec, D, dtype):
    """Records [..., R] as float64 (keys, values) [..., BS, D] and params [..., BS, 4]."""
    BS = rec.shape[-1] // (D + 8)
    x, n = min(D, 128), BS * D // 2
    out = []
    par = rec[..., 2 * n:].contiguous().view(dtype).reshape(*rec.shape[:-1], BS, 4).double()
    for i in range(2):
        b = rec[..., i * n:(i + 1) * n].reshape(*rec.shape[:-1], D // x, BS, x // 2).long()
        code = torch.stack([b % 16, b // 16], -1).flatten(-2)  # [..., D/x, BS, x]
        code = torch.cat(list(code.unbind(-3)), -1).double()
        out.append(code * par[..., 2 * i:2 * i + 1] + par[..., 2 * i + 1:2 * i + 2])
    return out[0], out[1], par


def kv4_case(seed, S, H, KH, D, BS, lens, dtype, q_len=1, MB=None, NB=None, v_spread=False):
    """Random query, records with N(0, 1)-like contents, shuffled tables."""
    g = torch.Generator().manual_seed(seed)
    MB = MB or max(1, max(-(-v // BS) for v in lens))
    NB = NB or S * MB
    q = torch.randn((S, q_len, H, D), generator=g).to(dtype)
    kc = torch.randint(0, 16, (NB, KH, BS, D), generator=g, dtype=torch.uint8)
    vc = torch.randint(0, 16, (NB, KH, BS, D), generator=g, dtype=torch.uint8)
    s = 0.15 + 0.2 * torch.rand((NB, KH, BS, 2), generator=g)
    z = -7.5 * s + 0.1 * torch.randn((NB, KH, BS, 2), generator=g)
    if v_spread:  # value scales over eight orders of magnitude
        f = 10.0 ** (-6 + 5 * torch.rand((NB, KH, BS), generator=g))
        s[..., 1] *= f
        z[..., 1] *= f
    params = torch.stack([s[..., 0], z[..., 0], s[..., 1], z[..., 1]], -1).to(dtype)
    cache = pack_records(kc, vc, params)
    if NB >= S * MB:
        bt = torch.randperm(NB, generator=g)[: S * MB].view(S, MB).to(torch.int32)
    else:
        bt = torch.randint(0, NB, (S, MB), generator=g, dtype=torch.int32)
    if q_len == 1:
        q = q[:, 0].contiguous()
    return q, cache, bt, torch.tensor(lens, dtype=torch.int32)


def attend64(q, cache, bt, lens, scale, dtype):
    """Output, log-sum-exp and their error bounds, float64, shaped as q / q's rows.

    Bound of an output element: half a step of the output's type; a relative
    2^-11 of each fp16 weight, which multiplies (code - 8) * scale; the fp32
    sums of the scores (D + 4 roundings of at most 2^-23 of the sum of the
    terms' magnitudes, M), which move every weight by a factor within
    exp(+-d), d = that error, so the quotient by at most 2 d sum p |v| (to
    first order); fp32 sums of the weights and values (2^-23 of sum p (15 s +
    |z|) per 16-token step); and subnormal weights (an absolute 2^-25 in units
    of 2^-12 of the largest value scale, doubled as it is a power of two above
    it, per token, times 8 scale).  The last factor 1.05 covers second order."""
    S, H, D = q.shape[0], q.shape[-2], q.shape[-1]
    ql = q.shape[1] if q.dim() == 4 else 1
    q4 = q.reshape(S, ql, H, D).double()
    KH = cache.shape[1]
    G = H // KH
    K, V, par = read_records(cache, D, dtype)
    BS = K.shape[2]
    sc = float(torch.tensor(scale, dtype=torch.float32))
    out, bound = torch.zeros_like(q4), torch.zeros_like(q4)
    lse = torch.full((S, ql, H), -math.inf, dtype=torch.float64)
    lse_b = torch.zeros((S, ql, H), dtype=torch.float64)
    for s in range(S):
        L = int(lens[s])
        if L == 0:
            continue
        ids = bt[s, : -(-L // BS)].long()
        k, v, pr = K[ids], V[ids], par[ids]  # [nb, KH, BS, ..]
        for h in range(H):
            kv = h // G
            kk, vv, pp = (t[:, kv].reshape(-1, t.shape[-1])[:L] for t in (k, v, pr))
            for i in range(ql):
                n = L - ql + 1 + i
                qi = q4[s, i, h]
                z = sc * (kk[:n] @ qi)
                lse[s, i, h] = torch.logsumexp(z, 0)
                p = torch.softmax(z, 0)
                o = p @ vv[:n]
                out[s, i, h] = o
                ks, kz, vs, vz = (pp[:n, j].abs() for j in range(4))
                M = abs(sc) * (15 * ks + kz) * qi.abs().sum()
                d = float((M * (D + 8) * 2.0 ** -23).max()) + 2.0 ** -21 * (1 + float(z.abs().max()))
                w = p * 8 * vs
                fp32 = 2.0 ** -23 * (n / 16 + 16) * float((p * (15 * vs + vz)).sum())
                small = n * 2.0 ** -25 * 2.0 ** -12 * 2 * 8 * float(vs.max())
                bound[s, i, h] = 1.05 * (U[dtype] * o.abs() + 2.0 ** -11 * float(w.sum()) + 2 * d *
                                         (p @ vv[:n].abs()) + fp32 + small) + (2.0 ** -25 if dtype == torch.float16 else 0)
                lse_b[s, i, h] = 1.05 * (d + 2.0 ** -20 * (1 + float(lse[s, i, h].abs())))
    shape = q.shape
    return out.view(shape), bound.view(shape), lse.view(shape[:-1]), lse_b.view(shape[:-1])


def quantise64(x):
    """The stored form of rows [..., D] (T), step by step: codes, scale, zero."""
    d = x.double()
    lo, hi = d.amin(-1, keepdim=True), d.amax(-1, keepdim=True)
    s = ((hi - lo).float().double() / 15).float().to(x.dtype).double()
    c = ((d - lo).float().double() / s).float().double().round().clamp(0, 15)
    c = torch.where(s > 0, c, torch.zeros_like(c))
    return c, s, lo + 0.0  # (a zero of either sign is stored as +0)
