"""Windowed and tree attention (pa_decode_v2_window, pa_decode_v2_tree and their
forms over E4M3 caches) against plain 64-bit attention over the tokens each row
sees, within bounds derived in view_testutil."""
import math

import pytest
import torch

from decode_attention_paged_pa_gb300 import PaError, binding
from view_testutil import ancestors, attend64, caches, pack, tree_parents, visible

pytestmark = pytest.mark.gpu

K_SCALE, V_SCALE = 0.5, 1.25
NAN_E4M3 = 0x7F


def make(seed, dtype, cache, n, H, KH, D, BS, lens, window, sinks, see=None, poison=True):
    """Inputs on the CPU: shuffled pages; table entries of blocks that no row sees
    are -1, and every slot that no row sees holds NaN."""
    S, MB = len(lens), max(1, max(-(-v // BS) for v in lens) + 1)
    g = torch.Generator().manual_seed(seed)
    q = torch.randn((S, n, H, D), generator=g).to(dtype)
    kc, vc = caches(seed + 1, S * MB, KH, D, BS, torch.uint8 if cache == "e4m3" else dtype)
    bt = torch.randperm(S * MB, generator=g).view(S, MB).to(torch.int32)
    if poison:
        bad = NAN_E4M3 if cache == "e4m3" else float("nan")
        for s, L in enumerate(lens):
            seen = visible(L, n, window, sinks, None if see is None else see[s]).any(0)
            for b in range(MB):
                part = seen[b * BS:(b + 1) * BS]
                for o in range(BS):
                    if o >= part.numel() or not bool(part[o]):
                        kc[bt[s, b], :, :, o] = bad
                        vc[bt[s, b], :, :, o] = bad
                if not bool(part.any()) and not (see is not None and L - n < (b + 1) * BS and b * BS < L):
                    bt[s, b] = -1  # (blocks of a tree's nodes are all there)
    return q, kc, vc, bt, torch.tensor(lens, dtype=torch.int32)


def run(q, kc, vc, bt, lens, scale, window, sinks, see=None, P=64, single=False, status=binding.PA_OK, ws=None):
    dev = torch.device("cuda")
    d = [t.to(dev) for t in (q, kc, vc, bt, lens)]
    if single:
        d[0] = d[0].squeeze(1)
    out = torch.full_like(d[0], float("nan"))
    lse = torch.full(d[0].shape[:-1], float("nan"), device=dev)
    more = dict(partition_size=P, lse=lse, workspace=ws)
    fp8 = kc.dtype == torch.uint8
    if fp8:
        more |= dict(k_scale=K_SCALE, v_scale=V_SCALE)
    if see is None:
        call = binding.pa_decode_v2_window_fp8 if fp8 else binding.pa_decode_v2_window
        ws = call(out, *d, scale, window, sinks, **more)
    else:
        call = binding.pa_decode_v2_tree_fp8 if fp8 else binding.pa_decode_v2_tree
        ws = call(out, *d, pack(see).to(dev), scale, window=window, sinks=sinks, **more)
    assert binding.device_status(ws) == status
    return out.cpu().view(q.shape), lse.cpu().view(q.shape[:-1])


def check(got, lse, q, kc, vc, bt, lens, scale, window, sinks, see=None):
    ref, ref_lse, bound = attend64(q, kc, vc, bt, lens, scale, window, sinks, see, K_SCALE, V_SCALE)
    err = (got.double() - ref).abs()
    assert bool((err <= bound).all()), f"worst excess {float((err - bound).max()):.3e}, NaN {int(got.isnan().sum())}"
    empty = ref_lse.isinf()
    assert bool((lse[empty] == -math.inf).all())
    assert bool((got[empty] == 0).all())
    # fp32 sums of at most a few thousand terms, and scores of about 10 or less.
    assert bool(((lse.double() - ref_lse)[~empty].abs() <= 1e-4 + 1e-5 * ref_lse[~empty].abs()).all())


LENS = [1, 15, 16, 17, 64, 65, 127, 300, 5]
SHAPES = [("fp16", "same", 4, 4, 64, 16), ("bf16", "same", 8, 2, 128, 16), ("fp16", "same", 4, 1, 128, 32),
          ("bf16", "same", 6, 2, 96, 8), ("fp16", "same", 8, 2, 80, 8), ("bf16", "same", 5, 1, 256, 16),
          ("fp16", "same", 2, 2, 112, 64), ("bf16", "same", 12, 1, 64, 32), ("fp32", "same", 2, 1, 64, 16),
          ("fp32", "same", 2, 2, 128, 64), ("fp32", "same", 1, 1, 256, 8), ("fp16", "e4m3", 8, 2, 128, 16),
          ("bf16", "e4m3", 4, 4, 64, 8), ("fp16", "e4m3", 6, 2, 112, 32), ("bf16", "e4m3", 3, 1, 256, 64),
          ("bf16", "e4m3", 8, 2, 64, 8)]
T = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
IDS = ["-".join(map(str, s)) for s in SHAPES]


@pytest.mark.parametrize("window,sinks", [(1, 0), (2, 1), (16, 4), (17, 33), (100, 0), (64, 300), (1 << 31, 7)])
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_window_single(shape, window, sinks):
    dtype, cache, H, KH, D, BS = shape
    lens = LENS + [0, 200]
    case = make(7 + D + window % 1000, T[dtype], cache, 1, H, KH, D, BS, lens, window, sinks)
    got, lse = run(*case, 0.11, window, sinks, single=True)
    check(got, lse, *case, 0.11, window, sinks)


@pytest.mark.parametrize("n,window,sinks", [(2, 1, 0), (4, 3, 2), (7, 40, 20), (33, 17, 4), (3, 1000, 4)])
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_window_rows(shape, n, window, sinks):
    dtype, cache, H, KH, D, BS = shape
    lens = [n + v for v in (0, 1, 15, 16, 60, 190)]
    case = make(70 + D + n, T[dtype], cache, n, H, KH, D, BS, lens, window, sinks)
    got, lse = run(*case, 0.11, window, sinks)
    check(got, lse, *case, 0.11, window, sinks)


@pytest.mark.parametrize("n,window,sinks", [(1, 0, 0), (2, 0, 0), (7, 0, 0), (7, 7, 3), (16, 40, 20), (33, 0, 0),
                                            (65, 70, 0)])
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_tree(shape, n, window, sinks):
    dtype, cache, H, KH, D, BS = shape
    lens = [n + v for v in (0, 1, 16, 47, 190)]
    see = torch.stack([ancestors(tree_parents(n + s, n, max(1, n - s))) for s in range(len(lens))])
    case = make(700 + D + n, T[dtype], cache, n, H, KH, D, BS, lens, window, sinks, see)
    got, lse = run(*case, 0.11, window, sinks, see)
    check(got, lse, *case, 0.11, window, sinks, see)


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_values_that_are_not_finite_reach_the_rows_that_see_them(shape):
    """Nodes 1 and 2 are siblings: 1's key and value are NaN, 2's value has an
    infinity of each sign; neither reaches the other's row, nor node 3's below 0."""
    dtype, cache, H, KH, D, BS = shape
    n, lens = 4, [40, 21]
    see = ancestors([-1, 0, 0, 0]).expand(2, 4, 4).clone()
    q, kc, vc, bt, L = make(5, T[dtype], cache, n, H, KH, D, BS, lens, 0, 0, see, poison=False)
    clean = kc.clone(), vc.clone()
    for s, length in enumerate(lens):
        b1, o1 = bt[s, (length - 3) // BS], (length - 3) % BS
        b2, o2 = bt[s, (length - 2) // BS], (length - 2) % BS
        kc[b1, :, :, o1] = NAN_E4M3 if cache == "e4m3" else float("nan")
        vc[b1, :, :, o1] = NAN_E4M3 if cache == "e4m3" else float("nan")
        if cache != "e4m3":
            vc[b2, :, 0, o2], vc[b2, :, 1, o2] = float("inf"), -float("inf")
    got, lse = run(q, kc, vc, bt, L, 0.11, 0, 0, see)
    ref, ref_lse, bound = attend64(q, *clean, bt, L, 0.11, 0, 0, see, K_SCALE, V_SCALE)
    assert bool(got[:, 1].isnan().all()) and bool(lse[:, 1].isnan().all())
    rows = [0, 3]
    assert bool(((got.double() - ref).abs() <= bound)[:, rows].all())
    if cache != "e4m3":
        assert bool((got[:, 2, :, 0] == math.inf).all()) and bool((got[:, 2, :, 1] == -math.inf).all())
        assert bool(((got.double() - ref).abs() <= bound)[:, 2, :, 2:].all())


@pytest.mark.parametrize("cache", ["same", "e4m3"])
def test_window_of_everything_is_multi_query_decode(cache):
    q, kc, vc, bt, L = make(3, torch.float16, cache, 4, 8, 2, 128, 16, [4, 90, 700], 1000, 0, poison=False)
    got, lse = run(q, kc, vc, bt, L, 0.1, 1000, 0, P=128)
    dev = torch.device("cuda")
    out = torch.empty_like(q, device=dev)
    d = [t.to(dev) for t in (q, kc, vc, bt, L)]
    if cache == "e4m3":
        binding.pa_decode_v2_mq_fp8(out, *d, 0.1, k_scale=K_SCALE, v_scale=V_SCALE, partition_size=128)
    else:
        binding.pa_decode_v2_mq(out, *d, 0.1, partition_size=128)
    # Two orders of the same fp32 sums, each rounded to fp16 (and its weights).
    assert bool(((got - out.cpu()).abs() <= 2.0 ** -9 * (1 + got.abs())).all())


@pytest.mark.parametrize("P", [16, 64, 512, 1 << 30])
def test_partitions(P):
    """Windows over long sequences: one or many partitions, the same workspace
    reused with a larger one's contents."""
    lens, window, sinks = [5000, 4097, 1030, 64, 1], 1024, 20
    case = make(9, torch.bfloat16, "same", 1, 8, 2, 128, 16, lens, window, sinks)
    for _ in range(2):
        got, lse = run(*case, 0.09, window, sinks, P=P, single=True)
        check(got, lse, *case, 0.09, window, sinks)


def test_many_sequences_and_a_poisoned_workspace():
    """More sequences than one launch takes; the workspace starts as 0x7f bytes."""
    g = torch.Generator().manual_seed(4)
    lens = torch.randint(3, 120, (600,), generator=g).tolist()
    case = make(11, torch.float16, "same", 3, 4, 2, 64, 16, lens, 24, 2)
    n = binding.view_workspace_bytes(600, 3, 4, 2, 64, case[3].shape[1], 16, 16, 24, 2)
    ws = torch.full((n,), 0x7F, dtype=torch.uint8, device="cuda")
    got, lse = run(*case, 0.12, 24, 2, P=16, ws=ws)
    check(got, lse, *case, 0.12, 24, 2)


def test_bad_lengths_and_ids_are_recorded():
    q, kc, vc, bt, L = make(13, torch.float16, "same", 4, 4, 2, 64, 16, [50, 3, 40], 16, 0, poison=False)
    got, lse = run(q, kc, vc, bt, L, 0.1, 16, 0, status=binding.PA_ERR_DEVICE_BOUNDS)
    assert bool((got[1] == 0).all()) and bool((lse[1] == -math.inf).all())
    ref, _, bound = attend64(q, kc, vc, bt, L, 0.1, 16, 0)
    assert bool(((got.double() - ref).abs() <= bound)[[0, 2]].all())
    L2 = torch.tensor([50, 60, 40], dtype=torch.int32)
    bt2 = bt.clone()
    bt2[2, 2] = kc.shape[0]
    got, _ = run(q, kc, vc, bt2, L2, 0.1, 16, 0, status=binding.PA_ERR_DEVICE_BOUNDS)
    ref, _, bound = attend64(q, kc, vc, bt, L2, 0.1, 16, 0)
    assert bool(((got.double() - ref).abs() <= bound)[:2].all())
    see = ancestors([-1, 0, 0, 1]).expand(3, 4, 4).clone()
    got, lse = run(q, kc, vc, bt, torch.tensor([50, 0, 40], dtype=torch.int32), 0.1, 0, 0, see,
                   status=binding.PA_ERR_DEVICE_BOUNDS)
    assert bool((got[1] == 0).all())


@pytest.mark.parametrize("op", ["window", "tree"])
def test_captured_and_on_another_stream(op):
    """A captured call replayed with other lengths, masks and queries; then two
    calls at once on two streams with workspaces of their own."""
    dev = torch.device("cuda")
    n, H, KH, D, BS, P = 5, 8, 2, 128, 16, 64
    see_a = ancestors([-1, 0, 1, 0, 3]).expand(3, n, n).clone()
    see_b = ancestors([-1, -1, 1, 2, 3]).expand(3, n, n).clone()
    window, sinks = (32, 4) if op == "window" else (0, 0)
    see = (None, None) if op == "window" else (see_a, see_b)
    a = make(1, torch.float16, "same", n, H, KH, D, BS, [200, 30, 7], window, sinks, see[0], poison=False)
    b = make(1, torch.float16, "same", n, H, KH, D, BS, [40, 190, 111], window, sinks, see[1], poison=False)
    q2, lens2 = torch.flip(a[0], [0]), b[4]
    d = [t.to(dev) for t in a]
    masks = pack(see_a).to(dev)
    out = torch.empty_like(d[0])
    ws = torch.empty(binding.view_workspace_bytes(3, n, H, KH, D, a[3].shape[1], BS, P, window, sinks),
                     dtype=torch.uint8, device=dev)

    def call(o, x, w, stream=None):
        if op == "window":
            binding.pa_decode_v2_window(o, *x, 0.1, window, sinks, partition_size=P, workspace=w, stream=stream)
        else:
            binding.pa_decode_v2_tree(o, *x, masks, 0.1, partition_size=P, workspace=w, stream=stream)

    call(out, d, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out, d, ws)
    for q, lens, s in ((a[0], a[4], see[0]), (q2, lens2, see[1]), (a[0], a[4], see[0])):
        d[0].copy_(q)
        d[4].copy_(lens)
        if s is not None:
            masks.copy_(pack(s))
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert binding.device_status(ws) == binding.PA_OK
        ref, _, bound = attend64(q, a[1], a[2], a[3], lens, 0.1, window, sinks, s)
        assert bool(((out.cpu().double() - ref).abs() <= bound).all())
    outs = [torch.full_like(out, float("nan")) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for o, st in zip(outs, streams):
            st.wait_stream(torch.cuda.current_stream())
            call(o, d, None, st)
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, out)


def test_repeats_are_bitwise_equal():
    case = make(21, torch.bfloat16, "same", 16, 32, 8, 128, 16, [900, 333, 1500, 64], 0, 0,
                see := torch.stack([ancestors(tree_parents(s, 16)) for s in range(4)]), poison=False)
    first = run(*case, 0.09, 0, 0, see, P=256)
    for _ in range(3):
        again = run(*case, 0.09, 0, 0, see, P=256)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_pool_past_4_gb():
    """Blocks whose bytes lie past 2^32 of the caches."""
    dev = torch.device("cuda")
    KH, D, BS = 8, 128, 16
    NB = (1 << 32) // (KH * D * BS * 2) * 5 // 4
    kc = torch.zeros((NB, KH, D // 8, BS, 8), dtype=torch.float16, device=dev)
    vc = torch.zeros((NB, KH, D, BS), dtype=torch.float16, device=dev)
    small = make(31, torch.float16, "same", 2, 8, 8, D, BS, [100, 70], 50, 4, poison=False)
    used = torch.tensor([NB - 1 - 3 * i for i in range(small[1].shape[0])])
    kc[used.to(dev)] = small[1].to(dev)
    vc[used.to(dev)] = small[2].to(dev)
    bt = used[small[3].long()].to(torch.int32)
    out = torch.empty_like(small[0], device=dev)
    ws = binding.pa_decode_v2_window(out, small[0].to(dev), kc, vc, bt.to(dev), small[4].to(dev), 0.1, 50, 4)
    assert binding.device_status(ws) == binding.PA_OK
    ref, _, bound = attend64(*small, 0.1, 50, 4)
    assert bool(((out.cpu().double() - ref).abs() <= bound).all())


def test_refusals():
    dev = torch.device("cuda")
    q, kc, vc, bt, L = (t.to(dev) for t in make(1, torch.float16, "same", 4, 4, 2, 64, 16, [40, 30], 16, 0,
                                                 poison=False))
    out = torch.empty_like(q)
    masks = torch.zeros((2, 4, 1), dtype=torch.int32, device=dev)
    ok = lambda **kw: binding.pa_decode_v2_tree(out, q, kc, vc, bt, L, masks, 0.1, **kw)
    ok(window=4)
    for bad in (dict(window=3), dict(window=-1), dict(sinks=-1), dict(partition_size=24)):
        with pytest.raises(PaError):
            ok(**bad)
    for window, sinks in ((0, 0), (-5, 0), (4, -1)):
        with pytest.raises(PaError):
            binding.pa_decode_v2_window(out, q, kc, vc, bt, L, 0.1, window, sinks)
    with pytest.raises(PaError):
        binding.pa_decode_v2_window(out, q, kc, vc, bt, L, 0.1, 16, workspace=torch.empty(256, dtype=torch.uint8, device=dev))
    with pytest.raises(ValueError):
        binding.pa_decode_v2_tree(out, q, kc, vc, bt, L, masks[:, :3], 0.1)
    with pytest.raises(TypeError):
        binding.pa_decode_v2_tree(out, q, kc, vc, bt, L, masks.long(), 0.1)
    with pytest.raises(ValueError):
        binding.pa_decode_v2_tree(out[:, 0], q[:, 0], kc, vc, bt, L, masks, 0.1)
    with pytest.raises(TypeError):
        binding.pa_decode_v2_window_fp8(out, q, kc, vc, bt, L, 0.1, 16)
    with pytest.raises(ValueError):
        binding.pa_decode_v2_window(out, q, kc.cpu(), vc, bt, L, 0.1, 16)


MANY = [("fp16", 16, 4, 128, 16), ("bf16", 12, 1, 128, 32), ("bf16", 8, 2, 64, 8), ("fp16", 6, 2, 80, 64),
        ("bf16", 5, 1, 256, 16), ("fp16", 4, 2, 256, 64), ("fp16", 10, 1, 96, 32), ("bf16", 4, 4, 112, 16),
        ("fp16", 4, 1, 256, 8), ("bf16", 3, 1, 256, 32)]


@pytest.mark.parametrize("n,window,sinks,P", [(40, 0, 0, 128), (100, 0, 0, 1024), (130, 200, 10, 256), (70, 70, 300, 192)])
@pytest.mark.parametrize("shape", MANY, ids=["-".join(map(str, s)) for s in MANY])
def test_many_rows(shape, n, window, sinks, P):
    """Row counts that are and are not whole tiles; one, two and more tiles of 128
    rows a kv head; partitions of one and of several tiles of tokens."""
    dtype, H, KH, D, BS = shape
    lens = [n, n + 1, n + 333, n + 700]
    see = torch.stack([ancestors(tree_parents(n + s, n, n - 9 * s)) for s in range(len(lens))])
    for tree in (True, False):
        w = window if tree or window else 150
        case = make(D + n, T[dtype], "same", n, H, KH, D, BS, lens, w, sinks, see if tree else None)
        got, lse = run(*case, 0.07 if tree else -0.07, w, sinks, see if tree else None, P=P)
        check(got, lse, *case, 0.07 if tree else -0.07, w, sinks, see if tree else None)


def test_many_rows_that_see_values_that_are_not_finite():
    """Values of the tree and of a window's edge that are not finite reach the rows
    that see them; keys that are not finite too."""
    n, H, KH, D, BS, L = 36, 4, 1, 128, 16, 400
    for dtype in (torch.float16, torch.bfloat16):
        q, kc, vc, bt, lens = make(3, dtype, "same", n, H, KH, D, BS, [L], 100, 0, poison=False)
        vc[bt[0, (L - 5) // BS], :, 3, (L - 5) % BS] = float("inf")        # seen by the last five rows
        lo = L - n + 1 - 100                                               # the first row's window starts here
        vc[bt[0, (lo + 2) // BS], :, 7, (lo + 2) % BS] = float("nan")      # seen by the first three rows
        got, _ = run(q, kc, vc, bt, lens, 0.1, 100, 0)
        odd = torch.zeros(n, D, dtype=torch.bool)
        odd[n - 5:, 3] = True
        odd[:3, 7] = True
        assert torch.equal(~got[0].isfinite(), odd[:, None].expand(n, H, D))
        assert bool((got[0, n - 5:, :, 3] == math.inf).all())
        clean = vc.clone()
        clean[~clean.isfinite()] = 0
        ref, _, bound = attend64(q, kc, clean, bt, lens, 0.1, 100, 0)
        fine = ~odd[None, :, None].expand(1, n, H, D)
        assert bool(((got.double() - ref).abs() <= bound)[fine].all())


def test_many_rows_of_large_scores():
    """Scores that grow along the sequence: the rows' references are set again and
    again.  The tokens' keys are one direction times their position."""
    n, H, KH, D, BS, L = 32, 4, 1, 128, 16, 900
    for dtype in (torch.float16, torch.bfloat16):
        q, kc, vc, bt, lens = make(8, dtype, "same", n, H, KH, D, BS, [L], 5000, 0, poison=False)
        q = (q.abs() + 0.5).to(dtype)
        for t in range(L):
            kc[bt[0, t // BS], :, :, t % BS] = (t / 256.0) * (1.0 if t % 7 else -1.0)
        got, lse = run(q, kc, vc, bt, lens, 0.15, 5000, 0, P=1024)
        check(got, lse, q, kc, vc, bt, lens, 0.15, 5000, 0)


MANY8 = [("fp16", 16, 4, 128, 16), ("bf16", 12, 1, 128, 32), ("bf16", 8, 2, 64, 8), ("fp16", 6, 2, 80, 64),
         ("bf16", 5, 1, 256, 16), ("fp16", 4, 2, 256, 64), ("fp16", 10, 1, 96, 32), ("bf16", 4, 4, 112, 16),
         ("fp16", 4, 1, 256, 8), ("bf16", 3, 1, 256, 32), ("fp16", 4, 1, 128, 8), ("bf16", 4, 1, 128, 64)]


@pytest.mark.parametrize("n,window,sinks,P", [(40, 0, 0, 128), (130, 200, 10, 256), (70, 70, 300, 192)])
@pytest.mark.parametrize("shape", MANY8, ids=["-".join(map(str, s)) for s in MANY8])
def test_many_rows_over_e4m3(shape, n, window, sinks, P):
    """As above over an E4M3 cache; slots that no row sees hold NaN codes."""
    dtype, H, KH, D, BS = shape
    lens = [n, n + 1, n + 333, n + 700]
    see = torch.stack([ancestors(tree_parents(n + s, n, n - 9 * s)) for s in range(len(lens))])
    for tree in (True, False):
        w = window if tree or window else 150
        case = make(D + n, T[dtype], "e4m3", n, H, KH, D, BS, lens, w, sinks, see if tree else None)
        got, lse = run(*case, 0.07 if tree else -0.07, w, sinks, see if tree else None, P=P)
        check(got, lse, *case, 0.07 if tree else -0.07, w, sinks, see if tree else None)


def test_many_rows_over_e4m3_of_any_size():
    """bf16 queries far outside fp16's range, each row by a power of two of its own,
    and one row of zeros: exact in the kernel, so the usual bound holds."""
    n, H, KH, D, BS, L = 40, 4, 1, 128, 16, 300
    for up, scale in ((2.0 ** 90, 0.1 * 2.0 ** -90), (2.0 ** -60, 0.1 * 2.0 ** 60)):
        q, kc, vc, bt, lens = make(6, torch.bfloat16, "e4m3", n, H, KH, D, BS, [L], 120, 3)
        q = (q.float() * up).to(torch.bfloat16)
        q[0, 5] = 0
        got, lse = run(q, kc, vc, bt, lens, scale, 120, 3)
        check(got, lse, q, kc, vc, bt, lens, scale, 120, 3)


def test_many_rows_that_see_nan_codes():
    """A NaN code in a value reaches the rows that see it, in tiles that every row sees
    (dim 9) and at the edges of windows (dims 3 and 7)."""
    n, H, KH, D, BS, L = 36, 4, 1, 128, 16, 400
    for dtype in (torch.float16, torch.bfloat16):
        q, kc, vc, bt, lens = make(3, dtype, "e4m3", n, H, KH, D, BS, [L], 200, 0, poison=False)
        lo = L - n + 1 - 200
        clean = vc.clone()
        vc[bt[0, (L - 5) // BS], 0, 3, (L - 5) % BS] = 0xFF
        vc[bt[0, (lo + 2) // BS], 0, 7, (lo + 2) % BS] = NAN_E4M3
        vc[bt[0, 290 // BS], 0, 9, 290 % BS] = NAN_E4M3
        got, _ = run(q, kc, vc, bt, lens, 0.1, 200, 0)
        odd = torch.zeros(n, D, dtype=torch.bool)
        odd[n - 5:, 3] = True
        odd[:3, 7] = True
        odd[:, 9] = True
        assert torch.equal(got[0].isnan(), odd[:, None].expand(n, H, D))
        ref, _, bound = attend64(q, kc, clean, bt, lens, 0.1, 200, 0, None, K_SCALE, V_SCALE)
        fine = ~odd[None, :, None].expand(1, n, H, D)
        assert bool(((got.double() - ref).abs() <= bound)[fine].all())


@pytest.mark.parametrize("P", [128, 4096])
def test_many_rows_into_tensors_aligned_to_16_bytes(P):
    """An output and a workspace that start 16 bytes past a 32-byte boundary."""
    n, H, KH, D, BS = 40, 4, 1, 80, 16
    for cache in ("same", "e4m3"):
        case = make(2, torch.bfloat16, cache, n, H, KH, D, BS, [n, 300], 150, 2)
        d = [t.to("cuda") for t in case]
        out = torch.full((d[0].numel() + 8,), float("nan"), dtype=d[0].dtype, device="cuda")[8:].view(d[0].shape)
        size = binding.view_workspace_bytes(2, n, H, KH, D, d[3].shape[1], BS, P, 150, 2)
        ws = torch.full((size + 16,), 0x7F, dtype=torch.uint8, device="cuda")[16:]
        assert out.data_ptr() % 32 == 16 and ws.data_ptr() % 32 == 16
        if cache == "e4m3":
            binding.pa_decode_v2_window_fp8(out, *d, 0.1, 150, 2, k_scale=K_SCALE, v_scale=V_SCALE, partition_size=P,
                                            workspace=ws)
        else:
            binding.pa_decode_v2_window(out, *d, 0.1, 150, 2, partition_size=P, workspace=ws)
        assert binding.device_status(ws) == binding.PA_OK
        ref, _, bound = attend64(*case, 0.1, 150, 2, None, K_SCALE, V_SCALE)
        assert bool(((out.cpu().double() - ref).abs() <= bound).all())


@pytest.mark.parametrize("cache", ["same", "e4m3"])
def test_pools_past_32_bits(cache):
    """Blocks whose first element lies past 2^31 elements (2^32 bytes for fp16): written by
    their slots, read by one row, many rows and a tree, and moved by an accepted path."""
    dev, BS, D, S, MB, n = torch.device("cuda"), 16, 64, 2, 40, 12
    NB = (1 << 21) + 128
    ct, x = (torch.uint8, 16) if cache == "e4m3" else (torch.float16, 8)
    kc = torch.empty((NB, 1, D // x, BS, x), dtype=ct, device=dev)
    vc = torch.empty((NB, 1, D, BS), dtype=ct, device=dev)
    g = torch.Generator().manual_seed(12)
    ids = torch.randperm(128, generator=g)[:S * MB] + (1 << 21)
    ids[3], ids[45] = 5, (1 << 20) + 1
    bt = ids.view(S, MB).to(torch.int32)
    lens = [600, 333]
    t = [torch.arange(L) for L in lens]
    slots = torch.cat([bt[s, t[s] // BS].long() * BS + t[s] % BS for s in range(S)])
    key, value = (torch.randn((sum(lens), 1, D), generator=g).half() for _ in range(2))
    more = dict(k_scale=K_SCALE, v_scale=V_SCALE) if cache == "e4m3" else {}
    ws = binding.pa_cache_write(kc, vc, key.to(dev), value.to(dev), slots.to(dev), **more)
    assert binding.device_status(ws) == binding.PA_OK
    small = torch.arange(S * MB).view(S, MB).to(torch.int32)
    see = torch.stack([ancestors(tree_parents(s, n)) for s in range(S)])

    def check_rows(q, lens, window, see):
        pages = [c[ids.to(dev)].cpu() for c in (kc, vc)]
        L = torch.tensor(lens, dtype=torch.int32)
        out = torch.full_like(q, float("nan"), device=dev)
        d = (out, q.to(dev), kc, vc, bt.to(dev), L.to(dev))
        if see is None:
            call = binding.pa_decode_v2_window_fp8 if cache == "e4m3" else binding.pa_decode_v2_window
            ws = call(*d, 0.1, window, 3, partition_size=128, **more)
        else:
            call = binding.pa_decode_v2_tree_fp8 if cache == "e4m3" else binding.pa_decode_v2_tree
            ws = call(*d, pack(see).to(dev), 0.1, partition_size=128, **more)
        assert binding.device_status(ws) == binding.PA_OK
        ref, _, bound = attend64(q, *pages, small, L, 0.1, window, 3, see, K_SCALE, V_SCALE)
        assert bool(((out.cpu().double() - ref).abs() <= bound).all())
        return pages

    check_rows(torch.randn((S, 1, 4, D), generator=g).half(), lens, 200, None)
    check_rows(torch.randn((S, n, 4, D), generator=g).half(), lens, 200, None)
    pages = check_rows(torch.randn((S, n, 4, D), generator=g).half(), lens, 0, see)
    for s, L in enumerate(lens):  # what was written is what is there
        want = value[sum(lens[:s]):][:L]
        if cache == "e4m3":
            want = (want.float() / torch.tensor(V_SCALE)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        assert torch.equal(pages[1][s * MB + t[s] // BS, :, :, t[s] % BS], want)
    path = [1, 4, 5, 9]
    new = torch.empty((S,), dtype=torch.int32, device=dev)
    ws = binding.pa_tree_accept(new, kc, vc, bt.to(dev), torch.tensor(lens, dtype=torch.int32, device=dev),
                                torch.tensor([path] * S, dtype=torch.int32, device=dev),
                                torch.tensor([4] * S, dtype=torch.int32, device=dev), n)
    assert binding.device_status(ws) == binding.PA_OK and new.tolist() == [L - n + 4 for L in lens]
    for c, before in zip((kc, vc), pages):
        after = c[ids.to(dev)].cpu()
        for s, L in enumerate(lens):
            for i, node in enumerate(path):
                to, at = L - n + i, L - n + node
                a, b = after[s * MB + to // BS], before[s * MB + at // BS]
                assert torch.equal(a[:, :, to % BS], b[:, :, at % BS])
    lens = new.tolist()
    check_rows(torch.randn((S, n, 4, D), generator=g).half(), lens, 200, None)
