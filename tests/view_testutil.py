"""Plain 64-bit restatements of windowed and tree attention over paged caches,
and error bounds from the arithmetic.  Test infrastructure only."""
from __future__ import annotations

import math

import torch

E4M3_MAX = 448.0


def visible(L: int, n: int, window: int, sinks: int, see=None) -> torch.Tensor:
    """bool [n, L]: position t is seen by row i of a sequence of L tokens.  ``see``
    (bool [n, n]): the rows are a tree's nodes and see the nodes of their row."""
    out = torch.zeros((n, L), dtype=torch.bool)
    for i in range(n):
        if see is None:
            p = L - n + i
            for t in range(p + 1):
                out[i, t] = t > p - window or t < sinks
        elif bool(see[i].any()):
            p = L - n + int(see[i].sum()) - 1
            for t in range(L - n):
                out[i, t] = window == 0 or t > p - window or t < sinks
            out[i, L - n:] = see[i]
    return out


def ancestors(parents) -> torch.Tensor:
    """bool [n, n] of one tree: node i sees itself and its ancestors; padding (parent below -1) nothing."""
    n = len(parents)
    see = torch.zeros((n, n), dtype=torch.bool)
    for i in range(n):
        j = i
        while j >= 0:
            if parents[j] < -1 or parents[j] >= j:
                see[i] = False
                break
            see[i, j] = True
            j = parents[j]
    return see


def pack(see: torch.Tensor) -> torch.Tensor:
    """bool [S, n, n] -> int32 [S, n, ceil(n / 32)]."""
    S, n, _ = see.shape
    out = torch.zeros((S, n, (n + 31) // 32), dtype=torch.int64)
    for j in range(n):
        out[:, :, j // 32] |= see[:, :, j].long() << (j % 32)
    return torch.where(out >= 2 ** 31, out - 2 ** 32, out).to(torch.int32)


def tokens64(key_cache, value_cache, ids, k_scale=None, v_scale=None):
    """K and V [KH, tokens, D] in fp64 of the blocks ``ids`` (uint8 caches: E4M3 codes)."""
    out = []
    for c, s in ((key_cache, k_scale), (value_cache, v_scale)):
        b = c[ids]
        b = b.view(torch.float8_e4m3fn).double() * s if c.dtype == torch.uint8 else b.double()
        b = b.permute(1, 0, 3, 2, 4).flatten(3) if b.dim() == 5 else b.permute(1, 0, 3, 2)
        out.append(b.flatten(1, 2))
    return out


def attend64(q, key_cache, value_cache, tables, lens, scale, window, sinks, see=None, k_scale=1.0, v_scale=1.0):
    """Output, log-sum-exp, and a bound on the output's error.  q [S, n, H, D];
    ``see`` bool [S, n, n] or None.  Only tokens that a row sees take part.

    The bound: the output is rounded to its type (half a step); a weight is off by
    its own rounding (fp16: 2^-11, and 2^-25 where it is subnormal; the others:
    2^-16) and by the score's error, D + 8 sums of fp32 that tensor cores may
    truncate (2^-23 each); exponentials and sums add 2^-20."""
    S, n, H, D = q.shape
    KH, BS = key_cache.shape[1], key_cache.shape[3]
    G = H // KH
    out = torch.zeros((S, n, H, D), dtype=torch.float64)
    lse = torch.full((S, n, H), -math.inf, dtype=torch.float64)
    bound = torch.zeros_like(out)
    fp16_weights = q.dtype == torch.float16 or key_cache.dtype == torch.uint8
    weps = 0.0 if q.dtype == torch.float32 else 2.0 ** -11 if fp16_weights else 2.0 ** -16
    for s in range(S):
        L = int(lens[s])
        if L < n:
            continue
        seen = visible(L, n, window, sinks, None if see is None else see[s])
        any_row = seen.any(0)
        ids = tables[s, : -(-L // BS)].long().clone()
        for b in range(ids.numel()):  # blocks that no row sees may have any id
            if not bool(any_row[b * BS:(b + 1) * BS].any()):
                ids[b] = 0
        K, V = tokens64(key_cache, value_cache, ids, k_scale, v_scale)
        for i in range(n):
            t = seen[i].nonzero().flatten()
            if not t.numel():
                continue
            for h in range(H):
                k, v, x = K[h // G][t], V[h // G][t], q[s, i, h].double()
                z = scale * (k @ x)
                lse[s, i, h] = torch.logsumexp(z, 0)
                w = torch.softmax(z, 0)
                out[s, i, h] = w @ v
                dz = float((k.abs() @ x.abs()).max()) * abs(scale) * (D + 8) * 2.0 ** -23
                av = w @ v.abs()
                bound[s, i, h] = av * (weps + 2 * dz + 2.0 ** -20)
                if fp16_weights:
                    bound[s, i, h] += t.numel() * 2.0 ** -25 * float(v.abs().max())
    half = torch.finfo(q.dtype).eps / 2
    bound += half * (out.abs() + bound) + (2.0 ** -25 if q.dtype == torch.float16 else 0.0)
    return out, lse, bound


def caches(seed, NB, KH, D, BS, dtype):
    """Random paged caches; dtype uint8: E4M3 codes."""
    g = torch.Generator().manual_seed(seed)
    esz = torch.empty((), dtype=dtype).element_size()
    x = 16 // esz
    k = torch.randn((NB, KH, D // x, BS, x), generator=g)
    v = torch.randn((NB, KH, D, BS), generator=g)
    if dtype == torch.uint8:
        return tuple(t.to(torch.float8_e4m3fn).view(torch.uint8) for t in (k, v))
    return k.to(dtype), v.to(dtype)


def tree_parents(seed, n, live=None):
    g = torch.Generator().manual_seed(seed)
    out = []
    for i in range(n):
        if live is not None and i >= live:
            out.append(-2)
        elif i == 0 or int(torch.randint(0, 6, (1,), generator=g)) == 0:
            out.append(-1)
        else:
            out.append(int(torch.randint(max(0, i - 4), i, (1,), generator=g)))
    return out
