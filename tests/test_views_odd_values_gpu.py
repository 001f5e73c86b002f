"""Values that are not finite under windows and trees with many rows a kv head: they
reach the rows that see them, no others, and cost little.  What a row gets is known
without arithmetic: where it sees such a value in a dim it is not finite, elsewhere it
is bit for bit what the same call gives with zeros in their place."""
import math

import pytest
import torch

from decode_attention_paged_pa_gb300 import binding
from test_views_gpu import K_SCALE, NAN_E4M3, T, V_SCALE, make, run
from view_testutil import ancestors, pack, tree_parents, visible

pytestmark = pytest.mark.gpu


def place(vc, bt, s, t, kv, d, BS, value):
    vc[bt[s, t // BS], kv, d, t % BS] = value


def check(case, spots, cache, n, window, sinks, see, P, scale=0.09):
    """spots: (sequence, position, kv head, dim, +1, -1 or 0 for NaN)."""
    q, kc, vc, bt, lens = case
    BS, H, KH = vc.shape[3], q.shape[2], vc.shape[1]
    clean = vc.clone()
    for s, t, kv, d, _ in spots:
        place(clean, bt, s, t, kv, d, BS, 0)
    for s, t, kv, d, sign in spots:
        place(vc, bt, s, t, kv, d, BS, NAN_E4M3 if cache == "e4m3" else sign * math.inf)
    got, lse = run(q, kc, vc, bt, lens, scale, window, sinks, see, P=P)
    ref, ref_lse = run(q, kc, clean, bt, lens, scale, window, sinks, see, P=P)
    assert bool(ref.isfinite().all())
    odd = torch.zeros_like(got, dtype=torch.bool)
    seen = [visible(int(L), n, window, sinks, None if see is None else see[s]) for s, L in enumerate(lens)]
    for s, t, kv, d, _ in spots:
        odd[s, :, kv * (H // KH):(kv + 1) * (H // KH), d] |= seen[s][:, t, None]
    assert torch.equal(~got.isfinite(), odd)
    assert torch.equal(got[~odd], ref[~odd]) and torch.equal(lse, ref_lse)
    return got


SHAPES = [("fp16", "same", 8, 2, 128, 16), ("bf16", "same", 4, 1, 64, 8), ("bf16", "same", 6, 2, 80, 64),
          ("fp16", "same", 4, 1, 256, 32), ("bf16", "same", 5, 1, 112, 32), ("fp16", "e4m3", 8, 2, 128, 16),
          ("bf16", "e4m3", 4, 1, 64, 8), ("fp16", "e4m3", 4, 1, 256, 64), ("bf16", "e4m3", 6, 2, 96, 32)]


@pytest.mark.parametrize("n,window,sinks,P", [(33, 0, 0, 4096), (40, 90, 30, 4096), (90, 300, 500, 256), (140, 200, 0, 192),
                                              (24, 2000, 7, 512)])
@pytest.mark.parametrize("shape", SHAPES, ids=["-".join(map(str, s)) for s in SHAPES])
def test_everywhere(shape, n, window, sinks, P):
    """Dozens of values over first tokens, skipped blocks, windows' edges, whole tiles,
    nodes and the last token, alone and several in a tile."""
    dtype, cache, H, KH, D, BS = shape
    lens = [n + 900, n + 77, n]
    g = torch.Generator().manual_seed(n + D)
    see = torch.stack([ancestors(tree_parents(n + s, n, n - 3 * s)) for s in range(len(lens))])
    for tree in (True, False):
        w = window if not tree or window == 0 or window >= n else n + 5
        if not tree and w == 0:
            w = 150
        case = make(D + n, T[dtype], cache, n, H, KH, D, BS, lens, w, sinks, see if tree else None, poison=False)
        spots = []
        for s, L in enumerate(lens):
            at = torch.randint(0, L, (24,), generator=g).tolist() + [0, max(0, sinks - 1), max(0, L - n + 1 - w), L - n, L - 1]
            for t in at:
                spots.append((s, min(t, L - 1), int(torch.randint(0, KH, (1,), generator=g)),
                              int(torch.randint(0, D, (1,), generator=g)), int(torch.randint(0, 2, (1,), generator=g)) * 2 - 1))
        check(case, spots, cache, n, w, sinks, see if tree else None, P)


def test_signs():
    """In partly seen tiles: +infinity, -infinity, and NaN where a row sees both."""
    n, H, KH, D, BS, L = 36, 4, 1, 128, 16, 500
    see = ancestors([-1, 0, 0, 1] + [-1] * (n - 4))[None]
    for dtype in ("fp16", "bf16"):
        case = make(4, T[dtype], "same", n, H, KH, D, BS, [L], 0, 0, see, poison=False)
        base = L - n
        spots = [(0, base, 0, 1, 1), (0, base + 1, 0, 2, -1), (0, base + 2, 0, 1, -1), (0, base + 3, 0, 2, -1)]
        got = check(case, spots, "same", n, 0, 0, see, 4096)[0, :, 0]
        assert got[0, 1] == math.inf and got[1, 1] == math.inf and got[1, 2] == -math.inf and got[3, 2] == -math.inf
        assert bool(got[2, 1].isnan())


@pytest.mark.parametrize("shape", [("fp16", "same", 4, 4, 64, 16, 3), ("bf16", "same", 8, 2, 128, 32, 1), ("bf16", "same", 4, 1, 80, 8, 2),
                                   ("fp16", "same", 2, 1, 256, 64, 4), ("fp16", "e4m3", 8, 2, 128, 16, 1), ("bf16", "e4m3", 4, 2, 64, 8, 4),
                                   ("bf16", "e4m3", 2, 1, 256, 64, 3), ("fp32", "same", 2, 1, 64, 16, 4), ("fp16", "same", 8, 2, 128, 16, 9),
                                   ("bf16", "e4m3", 8, 2, 64, 32, 9)], ids=lambda s: "-".join(map(str, s)))
def test_also_where_the_weight_is_zero(shape):
    """Scores hundreds apart: almost every weight is 0 in fp32.  A value that is not finite
    reaches the rows that see it all the same, in nodes and at windows' edges."""
    dtype, cache, H, KH, D, BS, n = shape
    lens = [n + 60, n + 7, n]
    see = torch.stack([ancestors(tree_parents(s, n)) for s in range(len(lens))])
    g = torch.Generator().manual_seed(D)
    for window, v in ((0, see), (20, None)):
        case = make(D + n, T[dtype], cache, n, H, KH, D, BS, lens, window, 3 if v is None else 0, v, poison=False)
        spots = []
        for s, L in enumerate(lens):
            for t in [0, L - 1, L - n, min(L - 1, max(0, L - n + 1 - window))] + torch.randint(0, L, (8,), generator=g).tolist():
                spots.append((s, t, int(torch.randint(0, KH, (1,), generator=g)), int(torch.randint(0, D, (1,), generator=g)),
                              int(torch.randint(0, 3, (1,), generator=g)) - 1))
        # (One value a place: a later one replaces an earlier one in either form.)
        check(case, list({x[:4]: x for x in spots}.values()), cache, n, window, 3 if v is None else 0, v, 4096, scale=30.0)


def call_time(f):
    f()
    best = math.inf
    for _ in range(3):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        f()
        b.record()
        b.synchronize()
        best = min(best, a.elapsed_time(b))
    return best  # ms


@pytest.mark.parametrize("cache,H,D", [("same", 4, 128), ("same", 2, 256), ("e4m3", 4, 128)])
def test_one_value_of_a_long_sequence_costs_little(cache, H, D):
    """One node's value is not finite, in trees over 20000 tokens: gone through token by
    token and element by element for every row the call took hundreds of times as long
    (and at greater lengths more than its waits allow)."""
    dev, S, n, BS, L = torch.device("cuda"), 20, 16, 16, 20000
    MB, esz = L // BS, 1 if cache == "e4m3" else 2
    NB, x = S * MB, 16 // esz
    ct = torch.uint8 if cache == "e4m3" else torch.float16
    fill = lambda shape: (torch.randint(0, 64, shape, dtype=torch.uint8, device=dev) if cache == "e4m3" else
                          torch.randn(shape, dtype=ct, device=dev))
    kc, vc = fill((NB, 1, D // x, BS, x)), fill((NB, 1, D, BS))
    bt = torch.randperm(NB, generator=torch.Generator().manual_seed(0)).view(S, MB).to(torch.int32)
    lens = torch.full((S,), L, dtype=torch.int32, device=dev)
    q = torch.randn((S, n, H, D), dtype=torch.float16, device=dev)
    see = torch.stack([ancestors(tree_parents(s, n)) for s in range(S)])
    masks, btd, ws = pack(see).to(dev), bt.to(dev), None
    more = dict(k_scale=0.5, v_scale=0.25) if cache == "e4m3" else {}
    fn = binding.pa_decode_v2_tree_fp8 if cache == "e4m3" else binding.pa_decode_v2_tree
    out = torch.empty_like(q)
    ws = fn(out, q, kc, vc, btd, lens, masks, 0.05, partition_size=1 << 15, **more)
    f = lambda: fn(out, q, kc, vc, btd, lens, masks, 0.05, partition_size=1 << 15, workspace=ws, **more)
    clean = call_time(f)
    ref = out.clone()
    node, s = 3, 7
    t = L - n + node
    vc[bt[s, t // BS], 0, 9, t % BS] = NAN_E4M3 if cache == "e4m3" else math.inf
    with_one = call_time(f)
    assert binding.device_status(ws) == binding.PA_OK
    odd = torch.zeros(out.shape, dtype=torch.bool)
    odd[s, :, :, 9] = see[s, :, node][:, None]
    assert torch.equal(~out.isfinite().cpu(), odd)
    assert torch.equal(out.cpu()[~odd], ref.cpu()[~odd])
    assert with_one < 3 * clean + 1, f"{with_one:.3f} ms, {clean:.3f} without"


@pytest.mark.parametrize("shape", SHAPES, ids=["-".join(map(str, s)) for s in SHAPES])
def test_keys_with_many_rows(shape):
    """A key with a NaN (or infinities, whose products with a row are an infinity or NaN):
    the rows of its kv head that see it are NaN with a NaN log-sum-exp; in nodes, at
    windows' edges and in tiles that every row sees.  Others: as with the key replaced."""
    dtype, cache, H, KH, D, BS = shape
    n, lens = 40, [40 + 700, 40 + 3]
    see = torch.stack([ancestors(tree_parents(s, n, n - s)) for s in range(len(lens))])
    for window, v in ((0, see), (300, None)):
        q, kc, vc, bt, L = make(D, T[dtype], cache, n, H, KH, D, BS, lens, window, 2, v, poison=False)
        seen = [visible(length, n, window, 2, None if v is None else v[s]) for s, length in enumerate(lens)]
        ref, ref_lse = run(q, kc, vc, bt, L, 0.09, window, 2, v, P=256)
        bad = [NAN_E4M3] if cache == "e4m3" else [math.nan, math.inf, -math.inf]
        for s, length in enumerate(lens):
            for i, t in enumerate([length - 2, length - n + 5, max(0, length - n + 3 - window), max(0, length - 130)]):
                k2 = kc.clone()
                k2[bt[s, t // BS], KH - 1, :, t % BS] = bad[i % len(bad)]
                got, lse = run(q, k2, vc, bt, L, 0.09, window, 2, v, P=256)
                hit = torch.zeros(lse.shape, dtype=torch.bool)
                hit[s, :, (KH - 1) * (H // KH):] = seen[s][:, t, None]
                # (An infinity times a row of both signs is NaN; the rows are not of one sign.)
                assert bool(got[hit].isnan().all()) and bool(lse[hit].isnan().all())
                assert torch.equal(lse[~hit], ref_lse[~hit]) and torch.equal(got[~hit], ref[~hit])
