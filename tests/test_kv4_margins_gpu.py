"""Decode over 4-bit caches whose value scales differ by many orders of
magnitude, or whose query has infinities and NaN: what one token or row holds
leaves the others' results alone.

Bound of an output element o = sum P_t v_t (P the softmax): half a step of the
type, |o| u; the weights P_t vs_t go through fp16, which multiplies the code's
distance from 8, at most 8: 2^-11 * 8 P_t vs_t, or half a subnormal step where
that is more: the weights of a row are scaled so that the largest that its warp
has met is 2^5 or more (the target is 2^6, met to a factor of two), hence 2^-25
2^-5 max(P vs) a token, or, where the scale of P binds (2^36 or more for the
largest), 2^-25 2^-36; the scores' fp32 error d moves a weight by a factor within exp(+-d):
D + 8 roundings of the terms' magnitudes, those of the reference (the largest
score, log2 of a scale and 40), and 2^-21 for the exponential; fp32 sums, 2^-23 a 16-token
step and 16 for the merges."""
import math

import pytest
import torch

from decode_attention_paged_pa_gb300 import binding
from kv4_testutil import U, kv4_case, read_records

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16


def reference(q, cache, bt, lens, scale, dtype, pick):
    """(output, bound) of the sequences `pick`, float64, [n, q_len, H, D]."""
    S, H, D = q.shape[0], q.shape[-2], q.shape[-1]
    ql = q.shape[1] if q.dim() == 4 else 1
    q4 = q.reshape(S, ql, H, D).double()
    KH = cache.shape[1]
    G = H // KH
    sc = float(torch.tensor(scale, dtype=torch.float32))
    out = torch.zeros((len(pick), ql, H, D), dtype=torch.float64)
    bound = torch.zeros_like(out)
    for a, s in enumerate(pick):
        L = int(lens[s])
        BS = cache.shape[-1] // (D + 8)
        k, v, par = read_records(cache[bt[s, : -(-L // BS)].long()], D, dtype)
        for kv in range(KH):
            kk, vv, pp = (t[:, kv].reshape(-1, t.shape[-1])[:L] for t in (k, v, par))
            ks, kz, vs, vz = (pp[:, j].abs() for j in range(4))
            for i in range(ql):
                n = L - ql + 1 + i
                r = q4[s, i, kv * G:(kv + 1) * G]
                z = sc * (r @ kk[:n].T)
                p = torch.softmax(z, 1)
                o = p @ vv[:n]
                M = abs(sc) * ((15 * ks + kz)[:n] * r.abs().sum(1, keepdim=True))
                lg = torch.log2(vs[:n].clamp(min=2.0 ** -40)).abs().max()
                d = M.amax(1) * (D + 8) * 2.0 ** -23 + 2.0 ** -21 + (2 * z.abs().amax(1) + lg + 46) * 2.0 ** -23
                w = p * vs[:n]
                small = 8 * n * (2.0 ** -30 * w.amax(1) + 2.0 ** -61)
                fp32 = 2.0 ** -23 * (n / 16 + 16) * (p @ (15 * vs + vz)[:n])
                t = 8 * 2.0 ** -11 * w.sum(1) + small + fp32
                out[a, i, kv * G:(kv + 1) * G] = o
                bound[a, i, kv * G:(kv + 1) * G] = 1.05 * (U[dtype] * o.abs() + t[:, None] + 2 * d[:, None] *
                                                           (p @ vv[:n].abs()))
    return out, bound + (2.0 ** -25 if dtype == F16 else 0)


def run(q, cache, bt, lens, scale, P):
    dev = torch.device("cuda")
    q, cache, bt, lens = (t.to(dev) for t in (q, cache, bt, lens))
    out, lse = torch.full_like(q, float("nan")), torch.full(q.shape[:-1], float("nan"), device=dev)
    call = binding.pa_decode_v2_kv4 if q.dim() == 3 else binding.pa_decode_v2_mq_kv4
    assert binding.device_status(call(out, q, cache, bt, lens, scale, partition_size=P, lse=lse)) == binding.PA_OK
    return out.cpu(), lse.cpu()


def check(q, cache, bt, lens, scale, P, pick=None):
    pick = list(range(q.shape[0])) if pick is None else pick
    out, _ = run(q, cache, bt, lens, scale, P)
    ref, bound = reference(q, cache, bt, lens, scale, q.dtype, pick)
    err = (out[pick].reshape(ref.shape).double() - ref).abs()
    assert bool((err <= bound).all()), f"worst {float((err / bound).max()):.3g} of the bound"
    return out


def params(cache, D, dtype):
    """The parameters [NB, KH, BS, 4] of a cache, a view to write to."""
    BS = cache.shape[-1] // (D + 8)
    return cache[..., BS * D:].view(dtype).view(*cache.shape[:-1], BS, 4)


def at(bt, s, pos, BS):
    return int(bt[s, pos // BS]), pos % BS


# (sequences, heads, kv heads, head size, block size, new tokens): two kv heads a
# unit, eight rows, sixteen rows, head size 256; and the first two with more units than warps.
FORMS = [(3, 8, 2, 128, 16, 1), (3, 16, 2, 64, 64, 1), (3, 8, 2, 128, 16, 4), (3, 4, 2, 256, 32, 2),
         (700, 8, 8, 64, 16, 1), (500, 16, 4, 80, 8, 2)]


def case(form, dtype, seed=1):
    S, H, KH, D, BS, ql = form
    lens = [150 + 37 * (s % 7) for s in range(S)]
    q, cache, bt, L = kv4_case(seed, S, H, KH, D, BS, lens, dtype, q_len=ql, NB=3 * (-(-372 // BS)) if S > 3 else None)
    if S > 3:  # the checked sequences' blocks are their own
        MB = bt.shape[1]
        bt[:3] = torch.arange(3 * MB, dtype=torch.int32).view(3, MB) if 3 * MB <= cache.shape[0] else bt[:3]
    return q.abs(), cache, bt, L  # (positive queries: a negative key zero is a low score)


@pytest.mark.parametrize("dtype,big,small", [(F16, 4000.0, 1e-3), (BF16, 4000.0, 1e-3), (BF16, 1e18, 0.3),
                                             (BF16, 1.0, 1e-12)])
@pytest.mark.parametrize("form", FORMS, ids=str)
def test_a_scale_that_no_row_attends_to(form, dtype, big, small):
    """One token of a huge value scale and a score far below all others: its
    weight is nothing, and the others keep their precision."""
    q, cache, bt, L = case(form, dtype)
    D, BS = form[3], form[4]
    par = params(cache, D, dtype)
    par[..., 2:] = (par[..., 2:].float() * (small / 0.25)).to(dtype)
    for s in range(3):
        for pos in (3, 77, int(L[s]) - 12):
            b, o = at(bt, s, pos, BS)
            par[b, :, o] = torch.tensor([0.0, -200.0, big, -7.5 * big]).to(dtype)
    check(q, cache, bt, L, 0.09, 64, [0, 1, 2])


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("form", FORMS, ids=str)
def test_another_heads_scale_changes_no_bit(form, dtype):
    q, cache, bt, L = case(form, dtype)
    S, H, KH, D, BS, ql = form
    base, lse = run(q, cache, bt, L, 0.09, 64)
    par = params(cache, D, dtype)
    par[:, 1, :, 2:] = (par[:, 1, :, 2:].float() * 8000.0).to(dtype)
    out, lse2 = run(q, cache, bt, L, 0.09, 64)
    G = H // KH
    keep = [h for h in range(H) if h // G != 1]
    assert torch.equal(out[..., keep, :], base[..., keep, :]) and torch.equal(lse[..., keep], lse2[..., keep])


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("form", FORMS, ids=str)
def test_a_first_token_that_takes_the_weight(form, dtype):
    """Nearly all weight on a first token that holds one value for every dim (its
    scale is 0): what the others add is small and keeps its precision."""
    q, cache, bt, L = case(form, dtype)
    D, BS = form[3], form[4]
    par = params(cache, D, dtype)
    for s in range(3):
        b, o = at(bt, s, 0, BS)
        par[b, :, o] = torch.tensor([0.0, 1.5, 0.0, 0.0]).to(dtype)
    check(q, cache, bt, L, 0.09, 64, [0, 1, 2])


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("form", FORMS, ids=str)
def test_scales_of_zero_then_large_then_small(form, dtype):
    """Partitions (and stretches of one) whose value scales are 0, large, tiny and of both signs."""
    q, cache, bt, L = case(form, dtype)
    D, BS = form[3], form[4]
    par = params(cache, D, dtype)
    top, low = (300.0, 1e-5) if dtype == F16 else (1e6, 1e-9)
    for s in range(3):
        for pos in range(int(L[s])):
            b, o = at(bt, s, pos, BS)
            if pos < 70:
                par[b, :, o, 2] = 0
            elif pos < 100:
                par[b, :, o, 2:] = (par[b, :, o, 2:].float() * top).to(dtype)
            elif pos % 3 == 0:
                par[b, :, o, 2:] = (par[b, :, o, 2:].float() * -low).to(dtype)
    for P in (64, 128, 1024):
        check(q, cache, bt, L, 0.09, P, [0, 1, 2])
        check(q, cache, bt, L, 1.0, P, [0, 1, 2])


@pytest.mark.parametrize("mag", [1e-13, 1e-6, 1e4, 1e15])
@pytest.mark.parametrize("form", FORMS[:4], ids=str)
def test_caches_of_every_magnitude(form, mag):
    q, cache, bt, L = case(form, BF16)
    par = params(cache, form[3], BF16)
    par[..., 2:] = (par[..., 2:].float() * mag).to(BF16)
    check(q, cache, bt, L, 0.09, 64, [0, 1, 2])


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("form", FORMS, ids=str)
def test_scores_that_rise_by_hundreds(form, dtype):
    """Each token's score far above the one before it: the reference rises all the way."""
    q, cache, bt, L = case(form, dtype)
    D, BS = form[3], form[4]
    par = params(cache, D, dtype)
    for s in range(3):
        for pos in range(int(L[s])):
            b, o = at(bt, s, pos, BS)
            par[b, :, o, 0] = 0.01
            par[b, :, o, 1] = pos // 5 * 0.5  # scores of about 0.09 * 0.8 D * that
    check(q, cache, bt, L, 0.09, 1024, [0, 1, 2])

@pytest.mark.parametrize("form", FORMS, ids=str)
def test_states_of_partitions(form):
    """What is left of a partition in the workspace: its weight sum lies in [1, 16),
    and with its reference gives the log of its sum; unused ones are (-inf, 0)."""
    q, cache, bt, L = case(form, BF16)
    S, H, KH, D, BS, ql = form
    params(cache, D, BF16)[..., 2:] *= 1000.0
    dev, P = torch.device("cuda"), 64
    qd, cd, bd, ld = (t.to(dev) for t in (q, cache, bt, L))
    out = torch.empty_like(qd)
    call = binding.pa_decode_v2_kv4 if ql == 1 else binding.pa_decode_v2_mq_kv4
    ws = call(out, qd, cd, bd, ld, 0.09, partition_size=P)
    assert binding.device_status(ws) == binding.PA_OK
    (om, ol, _, _, _), pmax = binding.workspace_layout(S * ql, H, KH, D, bt.shape[1], BS, P)
    m, l = (ws[o:o + S * ql * H * pmax * 4].view(torch.float32).view(S, ql * H, pmax).cpu() for o in (om, ol))
    G = H // KH
    for s in range(3):
        n = int(L[s])
        np = -(-n // P)
        assert bool((m[s, :, np:] == -math.inf).all()) and not bool(l[s, :, np:].any())
        k, _, _ = read_records(cache[bt[s, : -(-n // BS)].long()], D, BF16)
        for r in range(H * ql):  # row head r: kv head, token, head of the group
            kv, i, g = r // (G * ql), r % (G * ql) // G, r % G
            row = (q[s] if ql == 1 else q[s, i])[kv * G + g].double()
            z = float(torch.tensor(0.09)) * (k[:, kv].reshape(-1, D)[: n - ql + 1 + i] @ row)
            for p in range(np):
                part = z[p * P:(p + 1) * P]
                if part.numel() == 0:
                    assert m[s, r, p] == -math.inf and l[s, r, p] == 0
                    continue
                assert 1 <= float(l[s, r, p]) < 16
                got = float(m[s, r, p]) + math.log(float(l[s, r, p]))
                # (The scores' fp32 error, as in the bound above with M below 400; one of fp32 for m.)
                assert abs(got - float(torch.logsumexp(part, 0))) <= 400 * (D + 8) * 2.0 ** -23 + 2.0 ** -15


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("mag,dtype", [(1.0, F16), (1.0, BF16), (1e7, BF16), (1e-8, BF16), (2e-5, F16)])
@pytest.mark.parametrize("form", FORMS[:4], ids=str)
def test_a_row_of_infinities_or_nan_leaves_the_others(form, mag, dtype, bad):
    """Query rows that hold one: NaN; every other row of the sequence keeps its bits."""
    q, cache, bt, L = case(form, dtype)
    q = (q.float() * mag).to(dtype)
    q[:, ..., 1, 5] = 0
    base, lse = run(q, cache, bt, L, 0.09 / mag, 64)
    check(q, cache, bt, L, 0.09 / mag, 64)
    q[:, ..., 1, 5] = bad
    out, lse2 = run(q, cache, bt, L, 0.09 / mag, 64)
    keep = [h for h in range(form[1]) if h != 1]
    assert torch.equal(out[..., keep, :], base[..., keep, :]) and torch.equal(lse[..., keep], lse2[..., keep])
    if math.isnan(bad):
        assert bool(out[..., 1, :].isnan().all())
