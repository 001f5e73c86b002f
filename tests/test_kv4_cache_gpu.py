"""Tokens written into a 4-bit cache and read back (pa_kv4_append,
pa_kv4_gather).  What is stored is compared bit for bit with the definition in
64 bits (every step of it is an fp32 operation or a rounding to T, and the
quotients' 64-bit values round to fp32 as the fp32 division does); what is read
back has to be the nearest value of the type."""
import pytest
import torch

from decode_attention_paged_pa_gb300 import binding
from kv4_testutil import pack_records, quantise64, read_records

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16


def pool(seed, S, KH, D, BS, lens, extra=3):
    g = torch.Generator().manual_seed(seed)
    MB = max(1, max(-(-v // BS) for v in lens))
    NB = S * MB + extra
    cache = torch.randint(0, 256, (NB, KH, BS * (D + 8)), generator=g, dtype=torch.uint8)
    bt = torch.randperm(NB, generator=g)[: S * MB].view(S, MB).to(torch.int32)
    return cache, bt, torch.tensor(lens, dtype=torch.int32), g


def expected(cache, bt, lens, new, key, value):
    """The records after the append: the definition applied row by row."""
    want = cache.clone()
    KH, D = key.shape[1:]
    BS = cache.shape[-1] // (D + 8)
    x, n = min(D, 128), BS * D // 2
    kc, ks, kz = quantise64(key)
    vc, vs, vz = quantise64(value)
    row = 0
    for s, m in enumerate(new):
        for i in range(m):
            pos = int(lens[s]) - m + i
            rec = want[int(bt[s, pos // BS])]
            o = pos % BS
            for k, c in enumerate((kc, vc)):
                b = (c[row, :, ::2] + 16 * c[row, :, 1::2]).to(torch.uint8)
                codes = rec[:, k * n:(k + 1) * n].view(KH, D // x, BS, x // 2)
                codes[:, :, o] = b.view(KH, D // x, x // 2)
            p = torch.cat([ks[row], kz[row], vs[row], vz[row]], -1).to(key.dtype)
            rec[:, 2 * n:].view(KH, BS, 8)[:, o] = p.view(torch.uint8).view(KH, 8)
            row += 1
    return want


def cu_of(new):
    return torch.tensor([0] + new, dtype=torch.int32).cumsum(0, dtype=torch.int32)


def rows(g, N, KH, D, dtype):
    x = torch.randn((N, KH, D), generator=g)
    x[..., 0] += 5
    return x.to(dtype)


def nearest(got, ref):
    """Every value is the nearest of its type to scale * code + zero (rounded once)."""
    err = (got.double() - ref).abs()
    for step in (1, -1):  # the neighbouring patterns
        near = (got.view(torch.int16) + step).view(got.dtype).double()
        assert bool((err <= (near - ref).abs())[near.isfinite()].all())


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("BS", [8, 16, 32, 64])
@pytest.mark.parametrize("D", [64, 80, 96, 112, 128, 256])
def test_append_and_gather(D, BS, dtype):
    new, ctx = [1, 0, BS + 3, 2 * BS, 7], [0, 5, BS - 1, 0, 2 * BS - 3]
    lens = [a + b for a, b in zip(new, ctx)]
    KH = 3
    cache, bt, L, g = pool(D + BS, 5, KH, D, BS, lens)
    key, value = rows(g, sum(new), KH, D, dtype), rows(g, sum(new), KH, D, dtype)
    dev = torch.device("cuda")
    cd, bd, ld, cu = cache.to(dev), bt.to(dev), L.to(dev), cu_of(new).to(dev)
    ws = binding.pa_kv4_append(cd, key.to(dev), value.to(dev), bd, ld, cu_tokens=cu)
    assert binding.device_status(ws) == binding.PA_OK
    want = expected(cache, bt, L, new, key, value)
    assert torch.equal(cd.cpu(), want)  # the new slots, and nothing else
    ko = torch.full((sum(new) + 2, KH, D), 7.0, dtype=dtype, device=dev)
    vo = ko.clone()
    ws = binding.pa_kv4_gather(ko, vo, cd, bd, ld, cu_tokens=cu)
    assert binding.device_status(ws) == binding.PA_OK
    K, V, _ = read_records(want, D, dtype)
    at = [(s, int(L[s]) - m + i) for s, m in enumerate(new) for i in range(m)]
    for got, ref in ((ko, K), (vo, V)):
        w = torch.stack([ref[int(bt[s, p // BS]), :, p % BS] for s, p in at])
        nearest(got[: len(at)].cpu(), w)
        assert bool((got[len(at):] == 7).all())  # rows behind the last sequence


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["fp16", "bf16"])
def test_uniform_rows_strided_slices_and_4d(dtype):
    S, QL, KH, D, BS = 6, 3, 2, 128, 16
    lens = [3, 20, 16, 17, 33, 4]
    cache, bt, L, g = pool(3, S, KH, D, BS, lens)
    dev = torch.device("cuda")
    qkv = rows(g, S * QL, 4 * KH, D, dtype)
    k, v = qkv[:, 2 * KH:3 * KH], qkv[:, 3 * KH:]
    want = expected(cache, bt, L, [QL] * S, k, v)
    d = qkv.to(dev)
    for kk, vv in ((d[:, 2 * KH:3 * KH], d[:, 3 * KH:]),
                   (d.view(S, QL, 4 * KH, D)[:, :, 2 * KH:3 * KH], d.view(S, QL, 4 * KH, D)[:, :, 3 * KH:])):
        cd = cache.to(dev)
        ws = binding.pa_kv4_append(cd, kk, vv, bt.to(dev), L.to(dev))
        assert binding.device_status(ws) == binding.PA_OK
        assert torch.equal(cd.cpu(), want)


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["fp16", "bf16"])
def test_values_of_every_kind(dtype):
    """Constant vectors, tiny and huge spreads, one outlier, subnormals, zeros of both signs."""
    g = torch.Generator().manual_seed(2)
    D, KH, BS = 128, 1, 16
    top = 60000.0 if dtype == F16 else 1e38
    r = torch.randn((12, KH, D), generator=g)
    r[0] = 3.25
    r[1] = 0.0
    r[2] *= 1e-7
    r[3] *= top / 10
    r[4] = 1e-3 * r[4]
    r[4, 0, 17] = 1000.0
    r[5] = 100.0 + r[5]
    r[6, 0, ::2], r[6, 0, 1::2] = 0.0, -0.0
    r[7], r[7, 0, 3] = -top, top / 2
    r[8] = torch.randint(0, 31, (KH, D), generator=g) * 0.5      # quotients on the ties
    r[9] = torch.randint(-4, 5, (KH, D), generator=g).float()
    key = r.to(dtype)
    cache, bt, L, _ = pool(4, 1, KH, D, BS, [12])
    dev = torch.device("cuda")
    cd = cache.to(dev)
    binding.pa_kv4_append(cd, key.to(dev), key.flip(0).contiguous().to(dev), bt.to(dev), L.to(dev))
    want = expected(cache, bt, L, [12], key, key.flip(0))
    assert torch.equal(cd.cpu(), want)


def test_nan_and_inf_are_stored_as_nan():
    D, KH, BS = 64, 2, 16
    cache, bt, L, g = pool(5, 1, KH, D, BS, [4])
    key = rows(g, 4, KH, D, BF16)
    value = rows(g, 4, KH, D, BF16)
    key[0, 1, 5] = float("nan")
    key[1, 0, 63] = float("inf")
    value[2, 1, 0] = -float("inf")
    value[3, 0, 1], value[3, 0, 2] = 3e38, -3e38  # a spread that fp32 does not hold
    dev = torch.device("cuda")
    cd = cache.to(dev)
    ws = binding.pa_kv4_append(cd, key.to(dev), value.to(dev), bt.to(dev), L.to(dev))
    ko, vo = torch.empty((4, KH, D), dtype=BF16, device=dev), torch.empty((4, KH, D), dtype=BF16, device=dev)
    binding.pa_kv4_gather(ko, vo, cd, bt.to(dev), L.to(dev), workspace=ws)
    kn, vn = ko.isnan().all(-1).cpu(), vo.isnan().all(-1).cpu()
    assert kn.tolist() == [[False, True], [True, False], [False, False], [False, False]]
    assert vn.tolist() == [[False, False], [False, False], [False, True], [True, False]]
    assert torch.equal(ko.isnan().any(-1).cpu(), kn) and torch.equal(vo.isnan().any(-1).cpu(), vn)


def test_bad_sequences_are_recorded_and_skipped():
    D, KH, BS = 128, 2, 16
    lens = [20, 5, 18]
    cache, bt, L, g = pool(6, 3, KH, D, BS, lens)
    new = [4, 2, 3]
    key, value = rows(g, 9, KH, D, F16), rows(g, 9, KH, D, F16)
    dev = torch.device("cuda")

    def call(bt, L, cu):
        cd = cache.to(dev)
        ws = binding.pa_kv4_append(cd, key.to(dev), value.to(dev), bt.to(dev), L.to(dev), cu_tokens=cu.to(dev))
        ko = torch.full_like(key, 9.0, device=dev)
        vo = ko.clone()
        w2 = binding.pa_kv4_gather(ko, vo, cd, bt.to(dev), L.to(dev), cu_tokens=cu.to(dev))
        assert binding.device_status(ws) == binding.device_status(w2)
        return cd.cpu(), binding.device_status(ws), ko.cpu()

    full = expected(cache, bt, L, new, key, value)
    for bad_id in (-1, cache.shape[0], 2 ** 31 - 1):
        b = bt.clone()
        b[0, 1] = bad_id  # rows 0..3 go to positions 16..19
        got, st, ko = call(b, L, cu_of(new))
        assert st == binding.PA_ERR_DEVICE_BOUNDS
        want = full.clone()
        want[int(bt[0, 1])] = cache[int(bt[0, 1])]
        assert torch.equal(got, want) and bool((ko[:4] == 9).all()) and not bool((ko[4:] == 9).all())
    for bad_len in (1, -3, 10 ** 6):  # sequence 1: fewer than its two rows, negative, past the table
        l = L.clone()
        l[1] = bad_len
        got, st, ko = call(bt, l, cu_of(new))
        assert st == binding.PA_ERR_DEVICE_BOUNDS
        want = full.clone()
        want[int(bt[1, 0])] = cache[int(bt[1, 0])]
        assert torch.equal(got, want) and bool((ko[4:6] == 9).all())
    for cu in ([0, 4, 6, 12], [0, 6, 4, 9], [-2, 4, 6, 9]):
        assert call(bt, L, torch.tensor(cu, dtype=torch.int32))[1] == binding.PA_ERR_DEVICE_BOUNDS
    got, st, _ = call(bt, L, cu_of(new))
    assert st == binding.PA_OK and torch.equal(got, full)


def test_many_sequences_large_rows_and_empty_calls():
    """More sequences than one step of the offset search takes, zero-length ones among them."""
    D, KH, BS = 64, 1, 8
    g = torch.Generator().manual_seed(9)
    new = torch.randint(0, 4, (1100,), generator=g).tolist()
    lens = [v + (i % 5) for i, v in enumerate(new)]
    cache, bt, L, g = pool(8, 1100, KH, D, BS, lens)
    key, value = rows(g, sum(new), KH, D, F16), rows(g, sum(new), KH, D, F16)
    dev = torch.device("cuda")
    cd = cache.to(dev)
    ws = binding.pa_kv4_append(cd, key.to(dev), value.to(dev), bt.to(dev), L.to(dev), cu_tokens=cu_of(new).to(dev))
    assert binding.device_status(ws) == binding.PA_OK
    assert torch.equal(cd.cpu(), expected(cache, bt, L, new, key, value))
    ws.fill_(255)
    ws = binding.pa_kv4_append(cd, key[:0].to(dev), value[:0].to(dev), bt.to(dev), L.to(dev), workspace=ws)
    assert binding.device_status(ws) == binding.PA_OK
    assert torch.equal(cd.cpu(), expected(cache, bt, L, new, key, value))


def test_replays_from_a_cuda_graph():
    """A step captured once (append, then the context read back), replayed as the lengths grow."""
    D, KH, BS, S, dev = 128, 2, 16, 4, torch.device("cuda")
    lens = [15, 1, 40, 64]
    cache, bt, L, g = pool(12, S, KH, D, BS, [v + 4 for v in lens])
    L = torch.tensor(lens, dtype=torch.int32)
    cd, bd, ld = cache.to(dev), bt.to(dev), L.to(dev)
    k, v = (torch.zeros((S, KH, D), dtype=BF16, device=dev) for _ in range(2))
    ko, vo = torch.empty_like(k), torch.empty_like(k)
    ws, ws2 = (torch.empty(256, dtype=torch.uint8, device=dev) for _ in range(2))

    def step():
        binding.pa_kv4_append(cd, k, v, bd, ld, workspace=ws)
        binding.pa_kv4_gather(ko, vo, cd, bd, ld, workspace=ws2)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    want = expected(cache, bt, L, [1] * S, k.cpu(), v.cpu())
    for i in range(4):
        key, value = rows(g, S, KH, D, BF16), rows(g, S, KH, D, BF16)
        k.copy_(key)
        v.copy_(value)
        L += 1
        ld.copy_(L)
        graph.replay()
        assert binding.device_status(ws) == binding.device_status(ws2) == binding.PA_OK
        want = expected(want, bt, L, [1] * S, key, value)
        assert torch.equal(cd.cpu(), want)
        K, V, _ = read_records(want, D, BF16)
        for got, ref in ((ko, K), (vo, V)):
            nearest(got.cpu(), torch.stack([ref[int(bt[s, p // BS]), :, p % BS] for s, p in enumerate((L - 1).tolist())]))


def test_refusals():
    dev = torch.device("cuda")
    D, KH, BS = 128, 2, 16
    cache, bt, L, g = pool(6, 3, KH, D, BS, [20, 5, 18])
    c, b, l = cache.to(dev), bt.to(dev), L.to(dev)
    k = rows(g, 9, KH, D, F16).to(dev)
    with pytest.raises(TypeError):
        binding.pa_kv4_append(c, k.float(), k.float(), b, l)
    with pytest.raises(ValueError):
        binding.pa_kv4_append(c, k, k[:6], b, l)
    with pytest.raises(binding.PaError):       # 8 rows over 3 sequences
        binding.pa_kv4_append(c, k[:8], k[:8], b, l)
    with pytest.raises(ValueError):            # heads of a token apart
        binding.pa_kv4_append(c, k.expand(9, KH, D).transpose(0, 1).contiguous().transpose(0, 1), k, b, l)
    with pytest.raises(ValueError):
        binding.pa_kv4_append(c, k, k, b.cpu(), l)
    with pytest.raises(binding.PaError):       # rows not 16 bytes apart
        wide = torch.zeros((9, KH * D + 4), dtype=F16, device=dev)
        binding.pa_kv4_append(c, wide[:, :KH * D].unflatten(1, (KH, D)), k, b, l)
    with pytest.raises(binding.PaError):
        binding.pa_kv4_append(c, k, k, b, l, workspace=torch.empty(64, dtype=torch.uint8, device=dev))


def slots(rec, D):
    """Records [KH, BS * (D + 8)] as the bytes of each token: [BS, KH, D + 8]."""
    KH, BS, x = rec.shape[0], rec.shape[-1] // (D + 8), min(D, 128)
    n = BS * D // 2
    codes = rec[:, :2 * n].view(KH, 2, D // x, BS, x // 2).permute(3, 0, 1, 2, 4).reshape(BS, KH, D)
    return torch.cat([codes, rec[:, 2 * n:].view(KH, BS, 8).transpose(0, 1)], -1)


@pytest.mark.parametrize("cu,refused", [
    ([0, 4, 6, 12], [2]),           # passes the nine rows
    ([-2, 4, 6, 9], [0]),           # starts below 0
    ([0, 4, 2 ** 31 - 1, 2 ** 31 - 1], [1, 2]),
    ([0, 6, 4, 9], [1]),            # descend
    ([0, 4, -2 ** 31, 9], [1, 2]),
    ([7, 5, 6, 3], [0, 2]),
])
def test_rows_of_refused_offsets_are_skipped(cu, refused):
    """Every slot of a refused sequence keeps its bytes, its rows what they held.
    The other sequences get their rows; where offsets descend, some or none of them."""
    D, KH, BS = 128, 2, 16
    lens = [20, 9, 18]
    cache, bt, L, g = pool(6, 3, KH, D, BS, lens)
    key, value = rows(g, 9, KH, D, F16), rows(g, 9, KH, D, F16)
    dev = torch.device("cuda")
    cd, cud = cache.to(dev), torch.tensor(cu, dtype=torch.int32, device=dev)
    ws = binding.pa_kv4_append(cd, key.to(dev), value.to(dev), bt.to(dev), L.to(dev), cu_tokens=cud)
    assert binding.device_status(ws) == binding.PA_ERR_DEVICE_BOUNDS
    ko = torch.full_like(key, 9.0, device=dev)
    vo = ko.clone()
    ws = binding.pa_kv4_gather(ko, vo, cd, bt.to(dev), L.to(dev), cu_tokens=cud)
    assert binding.device_status(ws) == binding.PA_ERR_DEVICE_BOUNDS
    descend = any(a > b for a, b in zip(cu, cu[1:]))
    claims = {}  # row -> (sequence, position)
    for s in range(3):
        if s not in refused:
            for t in range(cu[s], cu[s + 1]):
                claims.setdefault(t, []).append((s, lens[s] - (cu[s + 1] - cu[s]) + t - cu[s]))
    allowed = {(s, p): t for t, c in claims.items() for s, p in c}
    got = cd.cpu()
    for s in range(3):
        for p in range(lens[s]):
            b, o = int(bt[s, p // BS]), p % BS
            now, old = slots(got[b], D)[o], slots(cache[b], D)[o]
            if (s, p) not in allowed:
                assert torch.equal(now, old), (s, p)
                continue
            t = allowed[s, p]
            at, one = torch.zeros(3, dtype=torch.int32), [int(i == s) for i in range(3)]
            at[s] = p + 1
            new = slots(expected(cache, bt, at, one, key[t:t + 1], value[t:t + 1])[b], D)[o]
            assert torch.equal(now, new) or (descend and torch.equal(now, old)), (s, p)
    held = {int(bt[s, j]) for s in range(3) for j in range(-(-lens[s] // BS))}
    for b in set(range(cache.shape[0])) - held:
        assert torch.equal(got[b], cache[b])
    for t in range(9):
        kept = bool((ko[t] == 9).all()) and bool((vo[t] == 9).all())
        assert kept if t not in claims else descend or not kept
