"""Slot maps, tree masks, cache writes and accepted paths against plain Python
restatements: whole numbers and copied values equal, E4M3 codes equal to torch's
rounding of the quotient."""
import math

import pytest
import torch

from decode_attention_paged_pa_gb300 import PaError, binding
from view_testutil import ancestors, caches, pack, tree_parents

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def status(ws):
    return binding.device_status(ws)


# ------------------------------------------------------------------ slots
def plain_slots(tables, lens, new, BS, N):
    slots, pos, seq, cu = [], [], [], [0]
    MB = len(tables[0]) if tables else 1
    for s, (L, n) in enumerate(zip(lens, new)):
        n = max(n, 0)
        for i in range(n):
            ok = n <= L <= MB * BS
            t = L - n + i
            b = tables[s][t // BS] if ok else -1
            slots.append(b * BS + t % BS if ok and b >= 0 else -1)
            pos.append(t if ok else -1)
            seq.append(s)
        cu.append(cu[-1] + n)
    pad = [-1] * max(0, N - len(slots))
    return (slots + pad)[:N], (pos + pad)[:N], (seq + pad)[:N], cu


def run_slots(tables, lens, new, BS, N, MB=None, ws=None, extras=True):
    S = len(lens)
    out = [torch.full((N,), 77, dtype=torch.int64, device=DEV), torch.full((N,), 77, dtype=torch.int32, device=DEV),
           torch.full((N,), 77, dtype=torch.int32, device=DEV), torch.full((S + 1,), 77, dtype=torch.int32, device=DEV)]
    bt = i32(tables).view(S, MB or len(tables[0]))
    ws = binding.pa_pages_slots(out[0], out[1] if extras else None, out[2] if extras else None, out[3], bt, i32(lens),
                                i32(new), BS, workspace=ws)
    return [t.tolist() for t in out], status(ws)


def step(seed, S, top, ctx, BS):
    g = torch.Generator().manual_seed(seed)
    new = torch.randint(0, top + 1, (S,), generator=g).tolist()
    lens = [n + int(torch.randint(0, ctx + 1, (1,), generator=g)) for n in new]
    MB = max(1, max(-(-v // BS) for v in lens))
    tables = torch.randperm(S * MB, generator=g).view(S, MB).tolist()
    return tables, lens, new


@pytest.mark.parametrize("S,top,ctx,BS,room", [
    (1, 1, 0, 16, 0), (1, 0, 5, 16, 3), (7, 3, 100, 8, 0), (128, 1, 4000, 16, 0), (128, 1, 4000, 16, 511),
    (300, 40, 300, 64, 1), (5, 3000, 50, 7, 600), (513, 2, 30, 16, 0), (2049, 1, 30, 16, 5), (9001, 3, 20, 32, 100)])
def test_slots(S, top, ctx, BS, room):
    tables, lens, new = step(S + top, S, top, ctx, BS)
    N = sum(new) + room
    want = plain_slots(tables, lens, new, BS, N)
    got, st = run_slots(tables, lens, new, BS, N, ws=torch.full((256,), 0x7F, dtype=torch.uint8, device=DEV))
    assert st == binding.PA_OK
    for a, b in zip(got, want):
        assert a == list(b)
    got, st = run_slots(tables, lens, new, BS, N, extras=False)
    assert got[0] == list(want[0]) and set(got[1]) <= {77}


def test_slots_of_nothing():
    got, st = run_slots([[0, 1]], [5], [0], 16, 4)
    assert got == [[-1] * 4, [-1] * 4, [-1] * 4, [0, 0]] and st == binding.PA_OK
    cu = torch.full((1,), 9, dtype=torch.int32, device=DEV)
    empty = torch.empty((0,), dtype=torch.int32, device=DEV)
    ws = binding.pa_pages_slots(torch.empty((0,), dtype=torch.int64, device=DEV), None, None, cu,
                                torch.empty((0, 3), dtype=torch.int32, device=DEV), empty, empty, 16)
    assert cu.tolist() == [0] and status(ws) == binding.PA_OK


@pytest.mark.parametrize("room", [0, 1000])
def test_slots_refused_sequences(room):
    tables, lens, new = step(3, 40, 30, 60, 16)
    MB = len(tables[0])
    new[3], lens[3] = 9, 4             # shorter than its new tokens
    lens[8], new[8] = MB * 16 + 1, 2   # past the table
    new[11] = -3
    lens[20], new[20] = 20, 20
    tables[20][1] = -1
    N = sum(max(n, 0) for n in new) + room
    got, st = run_slots(tables, lens, new, 16, N)
    assert st == binding.PA_ERR_DEVICE_BOUNDS
    for a, b in zip(got, plain_slots(tables, lens, new, 16, N)):
        assert a == list(b)
    # More rows than there is room for; then a good call clears the status.
    tables, lens, new = step(4, 40, 30, 60, 16)
    N = sum(new) - 5
    ws = torch.empty(256, dtype=torch.uint8, device=DEV)
    got, st = run_slots(tables, lens, new, 16, N, ws=ws)
    assert st == binding.PA_ERR_DEVICE_BOUNDS
    for a, b in zip(got, plain_slots(tables, lens, new, 16, N)):
        assert a == list(b)
    assert run_slots(tables, lens, new, 16, N + 5, ws=ws)[1] == binding.PA_OK


def test_slots_past_32_bits():
    """Blocks of a pool whose slots pass 2^31."""
    got, st = run_slots([[2 ** 31 - 1, 2 ** 28]], [20], [20], 16, 20)
    assert st == binding.PA_OK
    assert got[0] == [(2 ** 31 - 1) * 16 + i for i in range(16)] + [2 ** 32 + i for i in range(4)]


# ------------------------------------------------------------------ masks
@pytest.mark.parametrize("S,n", [(1, 1), (3, 7), (40, 16), (5, 32), (4, 33), (9, 100), (3, 512), (200, 64)])
def test_masks(S, n):
    parents = [tree_parents(s + n, n, max(1, n - s % 5)) for s in range(S)]
    if n == 512:
        parents[0] = list(range(-1, n - 1))  # a chain
    lens = [n + 3 * s for s in range(S)]
    see = torch.stack([ancestors(p) for p in parents])
    masks = torch.full((S, n, (n + 31) // 32), 77, dtype=torch.int32, device=DEV)
    pos = torch.full((S, n), 77, dtype=torch.int32, device=DEV)
    ws = binding.pa_tree_masks(masks, pos, i32(parents), i32(lens))
    assert status(ws) == binding.PA_OK
    assert torch.equal(masks.cpu(), pack(see))
    depth = see.sum(-1)
    want = torch.where(depth > 0, torch.tensor(lens)[:, None] - n + depth - 1, -1)
    assert torch.equal(pos.cpu().long(), want)
    masks2 = torch.zeros_like(masks)
    binding.pa_tree_masks(masks2, None, i32(parents), i32(lens))
    assert torch.equal(masks, masks2)


@pytest.mark.parametrize("copies", [1, 600])
def test_masks_of_bad_trees(copies):
    bad = [[0, -1, 1], [-1, 2, 0], [-1, 5, 0], [-2, 0, -1], [-1, 0, 1]]
    for parents in bad[:4]:
        rows = [[-1, 0, 0]] * (copies - 1) + [parents]
        masks = torch.zeros((copies, 3, 1), dtype=torch.int32, device=DEV)
        pos = torch.zeros((copies, 3), dtype=torch.int32, device=DEV)
        ws = binding.pa_tree_masks(masks, pos, i32(rows), i32([9] * copies))
        assert status(ws) == binding.PA_ERR_DEVICE_BOUNDS
        assert torch.equal(masks[-1].cpu(), pack(ancestors(parents)[None])[0])
        assert torch.equal(masks[:-1].cpu(), pack(ancestors([-1, 0, 0])[None]).expand(copies - 1, 3, 1))
    pos = torch.zeros((2, 3), dtype=torch.int32, device=DEV)
    ws = binding.pa_tree_masks(torch.zeros((2, 3, 1), dtype=torch.int32, device=DEV), pos, i32([[-1, 0, -2]] * 2),
                               i32([3, 2]))
    assert status(ws) == binding.PA_ERR_DEVICE_BOUNDS and pos.tolist() == [[0, 1, -1], [-1, -1, -1]]


# ------------------------------------------------------------------ write
T = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


def plain_write(kc, vc, key, value, slots, k_scale, v_scale):
    kc, vc = kc.clone(), vc.clone()
    BS = kc.shape[3]
    keep = (slots >= 0) & (slots < kc.shape[0] * BS)
    blk, off = slots[keep] // BS, slots[keep] % BS
    key, value = key[keep], value[keep]
    if kc.dtype == torch.uint8:
        key, value = ((t.float() / torch.tensor(s, dtype=torch.float32)).clamp(-448, 448).to(torch.float8_e4m3fn)
                      .view(torch.uint8) for t, s in ((key, k_scale), (value, v_scale)))
    kc[blk, :, :, off] = key.reshape(key.shape[0], kc.shape[1], kc.shape[2], kc.shape[4])
    vc[blk, :, :, off] = value
    return kc, vc


def check_write(kc, vc, key, value, slots, ks=1.0, vs=1.0, st=binding.PA_OK):
    want = plain_write(kc, vc, key, value, slots, ks, vs)
    d = [t.to(DEV) for t in (kc, vc)]
    # Rows as slices of a wider projection.
    KH, D = key.shape[1:]
    qkv = torch.zeros((key.shape[0], 3 * KH, D), dtype=key.dtype, device=DEV)
    qkv[:, KH:2 * KH], qkv[:, 2 * KH:] = key.to(DEV), value.to(DEV)
    ws = binding.pa_cache_write(*d, qkv[:, KH:2 * KH], qkv[:, 2 * KH:], slots.to(DEV), k_scale=ks, v_scale=vs)
    assert status(ws) == st
    for got, ref in zip(d, want):
        same = got.cpu().view(torch.uint8) == ref.view(torch.uint8) if got.dtype != torch.uint8 else (
            (got.cpu() == ref) | ((got.cpu() & 127 == 127) & (ref & 127 == 127)))
        assert bool(same.all())


def runs(seed, lengths, NB, BS, skip=0.0):
    """Slots of runs of consecutive tokens from random offsets, each in blocks of its own."""
    g = torch.Generator().manual_seed(seed)
    ids = torch.randperm(NB, generator=g).tolist()
    out, used = [], 0
    for n in lengths:
        first = int(torch.randint(0, BS, (1,), generator=g))
        nb = -(-(first + n) // BS)
        out += [ids[used + t // BS] * BS + t % BS for t in range(first, first + n)]
        used += nb
    slots = torch.tensor(out, dtype=torch.int64)
    if skip:
        slots[torch.rand(slots.shape, generator=g) < skip] = -1
    return slots


WRITES = [("fp16", "same"), ("bf16", "same"), ("fp32", "same"), ("fp16", "e4m3"), ("bf16", "e4m3"), ("fp32", "e4m3")]


@pytest.mark.parametrize("dtype,cache", WRITES, ids=["-".join(w) for w in WRITES])
@pytest.mark.parametrize("KH,D,BS,lengths,skip", [
    (2, 64, 16, [1] * 9, 0), (1, 80, 8, [1, 7, 8, 9, 30], 0), (8, 128, 16, [300, 1, 15, 16, 17, 64], 0),
    (3, 112, 32, [70, 5, 33], 0.1), (2, 256, 64, [200, 3], 0), (4, 96, 16, [1000, 40, 1], 0.02), (1, 64, 16, [1], 0),
    (16, 128, 32, [129, 63, 65], 0)])
def test_write(dtype, cache, KH, D, BS, lengths, skip):
    NB = sum(n // BS + 2 for n in lengths) + 1
    kc, vc = caches(1, NB, KH, D, BS, torch.uint8 if cache == "e4m3" else T[dtype])
    slots = runs(D + BS, lengths, NB, BS, skip)
    g = torch.Generator().manual_seed(2)
    key, value = ((torch.randn((slots.numel(), KH, D), generator=g) * 3).to(T[dtype]) for _ in range(2))
    scales = (0.37, 1.3) if cache == "e4m3" else (1.0, 1.0)
    check_write(kc, vc, key, value, slots, *scales)
    check_write(kc, vc, key, value, slots.flip(0), *scales)  # nothing follows anything


def test_write_rounds_every_pattern():
    """All 65536 fp16 patterns (and bf16 ones) as E4M3 codes: ties, subnormals, infinities, NaN."""
    for dtype in (torch.float16, torch.bfloat16):
        x = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(dtype).view(-1, 2, 64)
        kc, vc = caches(3, 32, 2, 64, 16, torch.uint8)
        for ks, vs in ((1.0, 0.5), (0.37, 3.0), (448.0, 1e-3)):
            check_write(kc, vc, x, x.flip(0), torch.arange(512, dtype=torch.int64), ks, vs)


def test_write_divides_exactly():
    """Scales that are powers of two and not, tiny and huge ones; zeros of either
    sign, infinities and NaN; rows of every type."""
    kc, vc = caches(4, 8, 2, 64, 16, torch.uint8)
    g = torch.Generator().manual_seed(2)
    for dtype in T.values():
        for ks, vs in ((0.3, 0.7), (1e-30, 1e-25), (3e25, 0.0625), (448.0, 1e-3)):
            x = [(torch.randn((100, 2, 64), generator=g) * min(abs(s) * 40, 1e4)).to(dtype) for s in (ks, vs)]
            for t in x:
                t[::7, 0, 5], t[::9, 1, 6], t[3, 0, 7], t[4, 1, 8], t[5, 0, 9] = 0.0, -0.0, math.inf, -math.inf, math.nan
            check_write(kc, vc, *x, torch.arange(3, 103, dtype=torch.int64), ks, vs)


@pytest.mark.parametrize("dtype,cache,BS", [("fp16", None, 16), ("fp32", None, 8), ("bf16", torch.uint8, 16),
                                            ("fp16", torch.uint8, 32), ("fp32", torch.uint8, 64)])
def test_write_into_caches_aligned_to_16_bytes(dtype, cache, BS):
    kc, vc = caches(4, 6, 2, 80, BS, cache or T[dtype])
    key, value = (torch.randn((3 * BS, 2, 80), generator=torch.Generator().manual_seed(i)).to(T[dtype]) for i in (1, 2))
    slots = torch.arange(5, 5 + 3 * BS, dtype=torch.int64)
    want = plain_write(kc, vc, key, value, slots, 1.0, 1.0)
    got = []
    for t in (kc, vc):
        size = t.numel() * t.element_size()
        room = torch.zeros(size + 16, dtype=torch.uint8, device=DEV)[16:]
        assert room.data_ptr() % 32 == 16
        got.append(room.view(t.dtype).view(t.shape))
        got[-1].copy_(t)
    assert status(binding.pa_cache_write(*got, key.to(DEV), value.to(DEV), slots.to(DEV))) == binding.PA_OK
    for a, b in zip(got, want):
        assert torch.equal(a.cpu().view(torch.uint8), b.view(torch.uint8))


def test_write_edges():
    kc, vc = caches(5, 6, 2, 64, 16, torch.float16)
    g = torch.Generator().manual_seed(1)
    key, value = (torch.randn((5, 2, 64), generator=g).half() for _ in range(2))
    key[1] = float("nan")
    value[2] = float("inf")
    check_write(kc, vc, key, value, torch.tensor([-1, 95, -(2 ** 40), 0, 17]))
    check_write(kc, vc, key, value, torch.tensor([3, 96, 2 ** 40, 4, 5]), st=binding.PA_ERR_DEVICE_BOUNDS)
    check_write(kc, vc, key, value, torch.tensor([94, 95, 96, 97, 1]), st=binding.PA_ERR_DEVICE_BOUNDS)
    check_write(kc, vc, key[:0], value[:0], torch.empty((0,), dtype=torch.int64))
    # Four-dimensional rows, and refusals.
    d = [t.to(DEV) for t in (kc, vc)]
    k4, v4 = key[:4].view(2, 2, 2, 64).to(DEV), value[:4].view(2, 2, 2, 64).to(DEV)
    slots = torch.tensor([7, 8, 20, 21], device=DEV)
    assert status(binding.pa_cache_write(*d, k4, v4, slots)) == binding.PA_OK
    want = plain_write(kc, vc, key[:4], value[:4], slots.cpu(), 1, 1)
    assert torch.equal(d[1].cpu().view(torch.int16), want[1].view(torch.int16))
    for bad in (lambda: binding.pa_cache_write(*d, k4, v4, slots.int()), lambda: binding.pa_cache_write(*d, k4.float(), v4.float(), slots),
                lambda: binding.pa_cache_write(*d, k4, v4, slots, k_scale=0.5), lambda: binding.pa_cache_write(*d, k4[..., ::2], v4, slots),
                lambda: binding.pa_cache_write(*d, k4, v4[:1], slots), lambda: binding.pa_cache_write(d[0], d[0], k4, v4, slots),
                lambda: binding.pa_cache_write(*d, k4[:, :, :1], v4[:, :, :1], slots)):
        with pytest.raises((PaError, TypeError, ValueError)):
            bad()


def test_write_past_4_gb():
    KH, D, BS = 8, 128, 16
    NB = (1 << 32) // (KH * D * BS * 2) * 5 // 4
    kc = torch.zeros((NB, KH, D // 8, BS, 8), dtype=torch.float16, device=DEV)
    vc = torch.zeros((NB, KH, D, BS), dtype=torch.float16, device=DEV)
    n = 40
    key, value = (torch.randn((n, KH, D), device=DEV).half() for _ in range(2))
    slots = (NB - 3) * BS + 5 + torch.arange(n, device=DEV)
    assert status(binding.pa_cache_write(kc, vc, key, value, slots)) == binding.PA_OK
    blk, off = slots // BS, slots % BS
    assert torch.equal(kc[blk, :, :, off].flatten(2), key) and torch.equal(vc[blk, :, :, off], value)
    assert int(vc.count_nonzero()) == int(value.count_nonzero())


# ------------------------------------------------------------------ accept
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32, torch.uint8],
                         ids=["fp16", "bf16", "fp32", "e4m3"])
@pytest.mark.parametrize("KH,D,BS,n,layers", [(2, 64, 16, 7, 1), (1, 80, 8, 30, 2), (8, 128, 16, 16, 3), (3, 112, 32, 70, 1),
                                              (2, 256, 64, 5, 2), (1, 96, 16, 1, 66)])
def test_accept(dtype, KH, D, BS, n, layers):
    g = torch.Generator().manual_seed(n)
    lens = [n, n + 1, n + 17, n + 50, n + 3, n + 9]
    S, MB = len(lens), -(-max(lens) // BS)
    bt = torch.randperm(S * MB, generator=g).view(S, MB).to(torch.int32)
    paths = [[], [0], list(range(n)), [n - 1], sorted(torch.randperm(n, generator=g)[: n // 2].tolist()),
             list(range(n // 2, n))]
    A = n
    acc = torch.full((S, A), -9, dtype=torch.int32)
    for s, p in enumerate(paths):
        acc[s, : len(p)] = torch.tensor(p, dtype=torch.int32)
    pairs = [caches(i, S * MB, KH, D, BS, dtype) for i in range(layers)]
    ks, vs = [p[0].to(DEV) for p in pairs], [p[1].to(DEV) for p in pairs]
    new = torch.full((S,), 77, dtype=torch.int32, device=DEV)
    ws = binding.pa_tree_accept(new, ks, vs, bt.to(DEV), i32(lens), acc.to(DEV), i32([len(p) for p in paths]), n)
    assert status(ws) == binding.PA_OK
    assert new.tolist() == [L - n + len(p) for L, p in zip(lens, paths)]
    for layer in range(layers):
        for got, ref in ((ks[layer].cpu(), pairs[layer][0]), (vs[layer].cpu(), pairs[layer][1])):
            ref = ref.clone()
            for s, p in enumerate(paths):
                rows = []
                for node in p:
                    t = lens[s] - n + node
                    rows.append(ref[bt[s, t // BS], :, :, t % BS].clone())
                for i, row in enumerate(rows):
                    t = lens[s] - n + i
                    ref[bt[s, t // BS], :, :, t % BS] = row
            assert torch.equal(got.view(torch.uint8), ref.view(torch.uint8))


def test_accept_refuses_paths():
    n, BS, lens = 4, 16, [20, 21, 22, 23, 24, 3, 70, 30]
    paths = [[1, 1], [2, 1], [0, 4], [-1], [1, 3], [1], [1], [1, 2]]
    counts = [2, 2, 2, 1, 5, 1, 1, 2]
    S, MB = len(lens), 4
    bt = torch.arange(S * MB, dtype=torch.int32).view(S, MB)
    bt[7, 1] = S * MB
    kc, vc = caches(1, S * MB, 2, 64, BS, torch.float16)
    d = kc.to(DEV), vc.to(DEV)
    acc = i32([p + [0] * (4 - len(p)) for p in paths])
    new = torch.zeros((S,), dtype=torch.int32, device=DEV)
    ws = binding.pa_tree_accept(new, *d, bt.to(DEV), i32(lens), acc, i32(counts), n)
    assert status(ws) == binding.PA_ERR_DEVICE_BOUNDS
    assert new.tolist() == lens  # every one of them refused
    assert torch.equal(d[0].cpu(), kc) and torch.equal(d[1].cpu(), vc)
    bt[7, 1] = 0
    ws2 = binding.pa_tree_accept(new[:1], *d, bt.to(DEV)[:1].contiguous(), i32(lens[:1]), acc[:1, 1:].contiguous(), i32([1]), n,
                                 workspace=ws)
    assert status(ws2) == binding.PA_OK and new[0] == 17
    with pytest.raises(PaError):
        lens_d = i32(lens)
        binding.pa_tree_accept(lens_d, *d, bt.to(DEV), lens_d, acc, i32(counts), n)
    with pytest.raises(ValueError):
        binding.pa_tree_accept(new, [d[0]], [], bt.to(DEV), i32(lens), acc, i32(counts), n)


def test_captured_step():
    """Slots, masks, writes and accepted paths of a step captured once and replayed
    with other lengths; eager calls give the same bytes."""
    S, n, KH, D, BS, MB = 3, 4, 2, 64, 16, 6
    bt = torch.randperm(S * MB).view(S, MB).to(torch.int32).to(DEV)
    lens, new, num = i32([40, 20, 9]), i32([4, 4, 4]), i32([2, 0, 3])
    parents, acc = i32([[-1, 0, 0, 1], [-1, -1, 1, -2], [-1, 0, 1, 2]]), i32([[1, 3, 0], [0, 0, 0], [0, 1, 3]])
    slots = torch.empty((S * n + 2,), dtype=torch.int64, device=DEV)
    pos, npos, cu, out_lens = torch.empty((S * n + 2,), dtype=torch.int32, device=DEV), i32([[0] * n] * S), i32([0] * (S + 1)), i32([0] * S)
    masks = torch.zeros((S, n, 1), dtype=torch.int32, device=DEV)
    kc, vc = (t.to(DEV) for t in caches(1, S * MB, KH, D, BS, torch.float16))
    rows = torch.randn((S * n + 2, 2, KH, D), device=DEV).half()
    ws = [torch.empty(256, dtype=torch.uint8, device=DEV) for _ in range(4)]

    def go():
        binding.pa_pages_slots(slots, pos, None, cu, bt, lens, new, BS, workspace=ws[0])
        binding.pa_tree_masks(masks, npos, parents, lens, workspace=ws[1])
        binding.pa_cache_write(kc, vc, rows[:, 0], rows[:, 1], slots, workspace=ws[2])
        binding.pa_tree_accept(out_lens, kc, vc, bt, lens, acc, num, n, workspace=ws[3])

    start = kc.clone(), vc.clone()
    go()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    for L in ([40, 20, 9], [96, 4, 33], [5, 60, 17]):
        results = []
        for run in (go, graph.replay):
            lens.copy_(i32(L))
            kc.copy_(start[0])
            vc.copy_(start[1])
            run()
            results.append([t.clone() for t in (slots, pos, npos, cu, out_lens, masks, kc, vc)])
        assert all(torch.equal(a, b) for a, b in zip(*results))
        assert all(status(w) == binding.PA_OK for w in ws)
        assert out_lens.tolist() == [L[0] - 2, L[1] - 4, L[2] - 1]
