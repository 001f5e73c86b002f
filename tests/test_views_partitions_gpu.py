"""Partitions of view rows follow the lengths on the device, not the room in the tables:
long sequences among short ones, tables far wider than the lengths, several launches of
one call, and captured calls replayed with other lengths."""
import pytest
import torch

from decode_attention_paged_pa_gb300 import binding
from test_views_gpu import K_SCALE, T, V_SCALE, check, make, run
from view_testutil import ancestors, attend64, pack, tree_parents, visible

pytestmark = pytest.mark.gpu

SMS = 152


def header(ws):
    """(units handed out, tokens of a partition) of the last call that used the workspace."""
    h = ws[:256].view(torch.int32).tolist()
    return h[1], h[6]


def call(lens, MB, n, H, KH, P, window=0, D=64, BS=16, cache="same", garbage=True):
    """A tree of n nodes (n = 1: a windowed row) over random pages; the workspace."""
    dev = torch.device("cuda")
    S = len(lens)
    NB = sum(-(-L // BS) for L in lens) + 1
    x = 8 if cache == "same" else 16
    if cache == "same":
        kc, vc = torch.randn((NB, KH, D // x, BS, x), device=dev).half(), torch.randn((NB, KH, D, BS), device=dev).half()
    else:
        kc, vc = (torch.randint(0, 100, s, dtype=torch.uint8, device=dev) for s in ((NB, KH, D // x, BS, x), (NB, KH, D, BS)))
    bt = torch.full((S, MB), -1, dtype=torch.int32)
    at, ids = 0, torch.randperm(NB).int()
    for s, L in enumerate(lens):
        m = -(-L // BS)
        bt[s, :m] = ids[at:at + m]
        at += m
    q = torch.randn((S, n, H, D), device=dev).half()
    out = torch.empty_like(q)
    L = torch.tensor(lens, dtype=torch.int32, device=dev)
    size = binding.view_workspace_bytes(S, n, H, KH, D, MB, BS, P, window, 0)
    ws = torch.full((size,), 0x7F, dtype=torch.uint8, device=dev)
    see = torch.stack([ancestors(tree_parents(s, n)) for s in range(S)])
    binding.pa_decode_v2_tree(out, q, kc, vc, bt.to(dev), L, pack(see).to(dev), 0.1, window=window, partition_size=P, workspace=ws)
    assert binding.device_status(ws) == binding.PA_OK
    assert bool(out.isfinite().all())
    return ws


@pytest.mark.parametrize("n,H,KH", [(16, 32, 8), (1, 32, 8), (1, 64, 8), (40, 8, 8)])
@pytest.mark.parametrize("lens,MB", [([2000] * 15 + [32768], 2048), ([2000] * 15 + [32768], 8192), ([20000], 8192),
                                     ([3000] * 4, 8192), ([40000, 9000, 3000, 700, 300, 100, 64, 50], 8192)],
                         ids=["one-long", "one-long-wide", "one-wide", "few-wide", "skew-wide"])
def test_no_unit_is_far_above_an_sm_s_share(lens, MB, n, H, KH):
    """Counted in tokens of a kv head's rows: the longest unit is at most 1.3 times what an
    SM gets if all get the same, or a partition of the caller's size."""
    units, part = header(call(lens, MB, n, H, KH, 512))
    rows = n * H // KH
    groups = KH * -(-rows // 128) if rows > 8 else KH // 2 if rows == 4 else KH
    share = sum(lens) * groups / SMS
    assert part % 512 == 0
    assert min(part, max(lens)) <= max(512, 1.3 * share)
    assert units == groups * sum(-(-L // part) for L in lens)


def test_even_batches_keep_whole_sequences():
    """48 sequences of about one length over 8 kv heads: 2.5 units an SM without a split."""
    lens = [4000 - 10 * i for i in range(48)]
    units, part = header(call(lens, 313, 16, 32, 8, 512))
    assert part >= max(lens) and units == 48 * 8


SHAPES = [("fp16", "same", 8, 2, 64, 16, 16), ("bf16", "same", 4, 1, 128, 8, 12), ("bf16", "e4m3", 4, 2, 64, 32, 9),
          ("fp16", "same", 4, 2, 64, 16, 1), ("bf16", "e4m3", 8, 2, 96, 8, 1), ("fp32", "same", 2, 1, 64, 16, 2)]


@pytest.mark.parametrize("P", [64, 512])
@pytest.mark.parametrize("shape", SHAPES, ids=["-".join(map(str, s)) for s in SHAPES])
def test_skewed_lengths(shape, P):
    dtype, cache, H, KH, D, BS, n = shape
    lens = [3000, n, 40, 17 + n, 500, n + 1, 64, 100]
    see = torch.stack([ancestors(tree_parents(s, n)) for s in range(len(lens))])
    for window, sinks, s in ((0, 0, see), (600, 70, None)):
        case = make(D + n, T[dtype], cache, n, H, KH, D, BS, lens, window, sinks, s)
        got, lse = run(*case, 0.1, window, sinks, s, P=P)
        check(got, lse, *case, 0.1, window, sinks, s)


@pytest.mark.parametrize("cache,tree", [("same", True), ("e4m3", False), ("same", False)])
def test_many_rows_of_several_launches(cache, tree):
    """More sequences than a launch takes, short ones first: each launch has partitions of
    its own.  The workspace starts as 0x7f bytes."""
    n, H, KH, D, BS, P, S = 3, 8, 2, 64, 16, 32, 300
    window, sinks = (0, 0) if tree else (100, 5)
    g = torch.Generator().manual_seed(2)
    lens = torch.randint(n, 40, (S,), generator=g).tolist()
    lens[256:] = torch.randint(n, 300, (S - 256,), generator=g).tolist()
    lens[270] = 900
    see = torch.stack([ancestors(tree_parents(s, n, n - s % 2)) for s in range(S)]) if tree else None
    case = make(5, torch.float16, cache, n, H, KH, D, BS, lens, window, sinks, see, poison=False)
    size = binding.view_workspace_bytes(S, n, H, KH, D, case[3].shape[1], BS, P, window, sinks)
    ws = torch.full((size,), 0x7F, dtype=torch.uint8, device="cuda")
    got, lse = run(*case, 0.12, window, sinks, see, P=P, ws=ws)
    check(got, lse, *case, 0.12, window, sinks, see)


@pytest.mark.parametrize("n", [1, 14])
def test_replayed_with_other_lengths(n):
    """One captured call: even lengths, one long sequence, all short, and back."""
    dev = torch.device("cuda")
    H, KH, D, BS, P, MB = 8, 2, 64, 16, 64, 200
    batches = [[700, 640, 600, 660], [3000, n, 20, 30], [n, n + 1, 40, n], [700, 640, 600, 660]]
    see = torch.stack([ancestors(tree_parents(s, n)) for s in range(4)])
    q, kc, vc, _, _ = make(3, torch.float16, "same", n, H, KH, D, BS, [MB * BS - BS] * 4, 0, 0, see, poison=False)
    bt = torch.randperm(4 * MB, generator=torch.Generator().manual_seed(1)).view(4, MB).to(torch.int32)
    d = [t.to(dev) for t in (q, kc, vc, bt, torch.tensor(batches[0], dtype=torch.int32))]
    masks, out = pack(see).to(dev), torch.empty_like(d[0])
    ws = torch.empty(binding.view_workspace_bytes(4, n, H, KH, D, MB, BS, P, 0, 0), dtype=torch.uint8, device=dev)
    go = lambda: binding.pa_decode_v2_tree(out, *d, masks, 0.1, partition_size=P, workspace=ws)
    go()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    parts = []
    for lens in batches:
        d[4].copy_(torch.tensor(lens, dtype=torch.int32))
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert binding.device_status(ws) == binding.PA_OK
        parts.append(header(ws)[1])
        ref, _, bound = attend64(q, kc, vc, bt, lens, 0.1, 0, 0, see)
        assert bool(((out.cpu().double() - ref).abs() <= bound).all())
    assert parts[0] == parts[3] and all(p >= P for p in parts)


def test_the_order_of_a_batch_does_not_matter():
    """16 sequences of 3000 to 8000 tokens whose partitions are whole: shortest first or longest
    first, the long ones start first and the call takes the same time (without that it
    took a fifth longer with the longest last)."""
    dev, S, n, H, KH, D, BS, P = torch.device("cuda"), 16, 64, 32, 8, 128, 16, 512
    lens = [3000 + 5000 * i // (S - 1) for i in range(S)]
    MB = -(-lens[-1] // BS)
    NB = S * MB
    kc, vc = (torch.randn(s, dtype=torch.bfloat16, device=dev) for s in ((NB, KH, D // 8, BS, 8), (NB, KH, D, BS)))
    bt = torch.randperm(NB, device=dev).view(S, MB).to(torch.int32)
    q = torch.randn((S, n, H, D), dtype=torch.bfloat16, device=dev)
    masks = pack(torch.stack([ancestors(tree_parents(s, n)) for s in range(S)])).to(dev)
    ws = torch.empty(binding.view_workspace_bytes(S, n, H, KH, D, MB, BS, P, 0, 0), dtype=torch.uint8, device=dev)
    times = []
    for order in (lens, lens[::-1]):
        L, out = torch.tensor(order, dtype=torch.int32, device=dev), torch.empty_like(q)
        best = float("inf")
        for _ in range(5):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            for _ in range(10):
                binding.pa_decode_v2_tree(out, q, kc, vc, bt, L, masks, 0.1, partition_size=P, workspace=ws)
            b.record()
            b.synchronize()
            best = min(best, a.elapsed_time(b))
        assert header(ws)[0] == S * KH * 2
        times.append(best)
    assert max(times) <= 1.1 * min(times), times
