"""Decode over a cache held in 4 bits (pa_decode_v2_kv4, pa_decode_v2_mq_kv4)
against attention in 64 bits over the same records, element by element within
the bound that kv4_testutil.attend64 derives."""
import math

import pytest
import torch

from decode_attention_paged_pa_gb300 import binding
from kv4_testutil import attend64, kv4_case, read_records

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16


def run(q, cache, bt, lens, scale, P=512, expect=binding.PA_OK, **kw):
    dev = torch.device("cuda")
    q, cache, bt, lens = (t.to(dev) for t in (q, cache, bt, lens))
    out = torch.full_like(q, float("nan"))
    lse = torch.full(q.shape[:-1], float("nan"), device=dev)
    call = binding.pa_decode_v2_kv4 if q.dim() == 3 else binding.pa_decode_v2_mq_kv4
    ws = call(out, q, cache, bt, lens, scale, partition_size=P, lse=lse, **kw)
    assert binding.device_status(ws) == expect
    return out.cpu(), lse.cpu()


def check(q, cache, bt, lens, scale, P=512):
    out, lse = run(q, cache, bt, lens, scale, P)
    ref, bound, rl, rb = attend64(q, cache, bt, lens, scale, q.dtype)
    err = (out.double() - ref).abs()
    assert bool((err <= bound).all()), f"worst {float((err / bound.clamp(min=1e-30)).max()):.2f} of the bound"
    same = (lse.double() == rl) | ((lse.double() - rl).abs() <= rb)
    assert bool(same.all()), float((lse.double() - rl).abs().max())


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("BS", [8, 16, 32, 64])
@pytest.mark.parametrize("D", [64, 80, 96, 112, 128, 256])
def test_shapes(D, BS, dtype):
    # no token, one, a ragged block, block and partition edges (P = 64), several partitions
    lens = [1, 0, 5, BS, BS + 1, 63, 64, 65, 700]
    for H, KH in ((8, 2), (3, 3)):
        check(*kv4_case(D + BS + H, len(lens), H, KH, D, BS, lens, dtype), 1.0 / math.sqrt(D), P=64)


@pytest.mark.parametrize("H,KH", [(1, 1), (2, 2), (4, 2), (6, 2), (5, 1), (8, 1), (12, 1), (20, 2), (32, 4), (10, 5)])
def test_group_sizes(H, KH):
    lens = [17, 130, 1, 600]
    check(*kv4_case(H * 100 + KH, len(lens), H, KH, 128, 16, lens, BF16), 0.09, P=128)


@pytest.mark.parametrize("H,KH,D,BS", [(8, 2, 128, 16), (4, 4, 64, 8), (12, 3, 80, 32), (16, 1, 256, 64)])
@pytest.mark.parametrize("q_len", [2, 4, 7])
def test_multi_query(H, KH, D, BS, q_len):
    lens = [q_len, q_len + 1, 64, 63 + q_len, 65, 500]
    check(*kv4_case(q_len + D + BS, len(lens), H, KH, D, BS, lens, F16, q_len=q_len), 0.1, P=64)


def test_long_sequence_and_many_partitions():
    check(*kv4_case(7, 2, 8, 2, 128, 32, [20000, 33], BF16), 0.0884, P=512)


def test_more_sequences_than_a_launch_takes():
    lens = [(i * 37) % 90 for i in range(530)]
    check(*kv4_case(8, 530, 4, 2, 64, 16, lens, F16, NB=700), 0.125, P=64)


@pytest.mark.parametrize("S,H,KH,D,BS,q_len,dtype", [
    (420, 32, 8, 64, 16, 1, BF16),     # two kv heads a unit
    (300, 16, 2, 128, 8, 1, F16),      # eight rows a kv head
    (300, 16, 4, 80, 32, 4, BF16),     # sixteen rows
    (300, 3, 3, 256, 16, 1, F16),      # head size 256
    (300, 5, 5, 128, 64, 1, BF16),     # 64-token blocks
    (300, 20, 4, 112, 16, 1, F16),     # five rows
])
def test_batches_of_many_units(S, H, KH, D, BS, q_len, dtype):
    """Thousands of units: warps take whole ones, the rest goes to teams.  A
    sample of the sequences is checked, and that a second run is bitwise the same."""
    g = torch.Generator().manual_seed(S + D)
    lens = [int(v) for v in torch.randint(q_len, 900, (S,), generator=g)]
    lens[5], lens[6] = q_len, 899
    if q_len == 1:
        lens[7] = 0
    q, cache, bt, L = kv4_case(S + D, S, H, KH, D, BS, lens, dtype, q_len=q_len, NB=1500)
    out, lse = run(q, cache, bt, L, 0.1, P=64)
    again, lse2 = run(q, cache, bt, L, 0.1, P=64)
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    pick = [0, 5, 6, 7, S - 1] + [int(v) for v in torch.randint(0, S, (9,), generator=g)]
    ref, bound, rl, rb = attend64(q[pick], cache, bt[pick], L[pick], 0.1, dtype)
    err = (out[pick].double() - ref).abs()
    assert bool((err <= bound).all()), f"worst {float((err / bound.clamp(min=1e-30)).max()):.2f} of the bound"
    same = (lse[pick].double() == rl) | ((lse[pick].double() - rl).abs() <= rb)
    assert bool(same.all())


def test_partition_sizes_from_one_block_to_past_the_table():
    case = kv4_case(21, 3, 8, 2, 128, 16, [300, 17, 64], BF16)
    for P in (16, 48, 80, 4096, 2 ** 31 - 16):
        check(*case, 0.09, P=P)


def test_another_stream_and_two_calls_at_once():
    """Calls on two streams at a time, each with a workspace of its own."""
    dev = torch.device("cuda")
    cases = [[t.to(dev) for t in kv4_case(30 + i, 40, 8, 2, 128, 16, [(37 * j) % 700 for j in range(40)], F16)]
             for i in range(2)]
    want = []
    for q, c, b, l in cases:
        o = torch.empty_like(q)
        binding.pa_decode_v2_kv4(o, q, c, b, l, 0.1, partition_size=64)
        want.append(o)
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in cases], [torch.empty_like(c[0]) for c in cases]
    keep = []
    for _ in range(5):
        for s, o, (q, c, b, l) in zip(streams, outs, cases):
            keep.append(binding.pa_decode_v2_kv4(o, q, c, b, l, 0.1, partition_size=64, stream=s,
                                                 workspace=torch.empty(1 << 24, dtype=torch.uint8, device=dev)))
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["fp16", "bf16"])
def test_value_scales_of_every_magnitude(dtype):
    """Value scales over eight orders of magnitude in one sequence: the bound
    that the weights are scaled by rises as the sequence goes."""
    check(*kv4_case(9, 3, 8, 2, 128, 16, [40, 300, 1000], dtype, v_spread=True), 0.09, P=256)


def test_slots_past_the_end_may_hold_anything():
    """NaN and Inf parameters behind the last token (and in unused blocks) reach nothing."""
    lens = [5, 33, 70]
    q, cache, bt, L = kv4_case(10, 3, 8, 2, 128, 16, lens, BF16)
    clean = run(q, cache, bt, L, 0.09, P=64)
    n = 16 * 128
    par = cache[..., n:].view(BF16).view(*cache.shape[:-1], 16, 4)
    for s, v in enumerate(lens):
        for j in range(bt.shape[1]):
            first = max(0, min(16, v - 16 * j))
            par[bt[s, j].long(), :, first:] = torch.tensor([float("nan"), float("inf"), float("nan"), -float("inf")])
    dirty = run(q, cache, bt, L, 0.09, P=64)
    assert torch.equal(clean[0], dirty[0]) and torch.equal(clean[1], dirty[1])


def test_nan_token_reaches_the_rows_that_see_it_only():
    """A token stored as NaN makes every row that sees it NaN, and no other:
    causal rows before it and other kv heads keep their values."""
    q, cache, bt, L = kv4_case(11, 2, 8, 2, 128, 16, [40, 50], F16, q_len=4)
    base = run(q, cache, bt, L, 0.1)[0]
    par = cache[..., 16 * 128:].view(F16).view(*cache.shape[:-1], 16, 4)
    pos = 38  # rows 0, 1 of sequence 0 see positions 0..36, 0..37
    par[bt[0, pos // 16].long(), 1, pos % 16, 2:] = float("nan")  # kv head 1's value
    out = run(q, cache, bt, L, 0.1)[0]
    assert torch.equal(out[1], base[1]) and torch.equal(out[0, :, :4], base[0, :, :4])
    assert torch.equal(out[0, :2], base[0, :2])
    assert bool(out[0, 2:, 4:].isnan().all())
    par[bt[0, pos // 16].long(), 1, pos % 16] = float("nan")      # its key too
    out = run(q, cache, bt, L, 0.1)[0]
    assert torch.equal(out[0, :2], base[0, :2]) and bool(out[0, 2:, 4:].isnan().all())
    assert torch.equal(out[0, :, :4], base[0, :, :4])


def test_one_token_returns_its_value():
    q, cache, bt, L = kv4_case(12, 4, 4, 2, 96, 8, [1, 1, 1, 1], F16)
    out, _ = run(q, cache, bt, L, 0.1)
    V = read_records(cache, 96, F16)[1]
    want = V[bt[:, 0].long(), :, 0].repeat_interleave(2, 1)
    # one weight of 1: the code's product is exact, the scale's rounding 2^-11 of 8 scale
    s = read_records(cache, 96, F16)[2][bt[:, 0].long(), :, 0, 2].repeat_interleave(2, 1)[..., None]
    assert bool(((out.double() - want).abs() <= 2.0 ** -11 * (want.abs() + 8 * s) * 1.05).all())


def test_bad_block_ids_and_lengths_are_recorded():
    q, cache, bt, L = kv4_case(13, 2, 4, 2, 64, 16, [40, 20], F16)
    bad = bt.clone()
    bad[0, 1] = cache.shape[0]
    run(q, cache, bad, L, 0.1, expect=binding.PA_ERR_DEVICE_BOUNDS)
    bad[0, 1] = -1
    run(q, cache, bad, L, 0.1, expect=binding.PA_ERR_DEVICE_BOUNDS)
    run(q, cache, bt, torch.tensor([40, 1000], dtype=torch.int32), 0.1, expect=binding.PA_ERR_DEVICE_BOUNDS)
    run(q, cache, bt, L, 0.1)


def test_repeats_and_replays_are_bitwise_equal():
    q, cache, bt, L = kv4_case(14, 5, 16, 4, 128, 16, [1, 300, 64, 1000, 90], BF16)
    want = run(q, cache, bt, L, 0.09, P=128)
    dev = torch.device("cuda")
    qd, cd, bd, ld = (t.to(dev) for t in (q, cache, bt, L))
    out = torch.empty_like(qd)
    ws = torch.empty(binding.workspace_bytes(5, 16, 4, 128, bt.shape[1], 16, 128), dtype=torch.uint8, device=dev)
    call = lambda: binding.pa_decode_v2_kv4(out, qd, cd, bd, ld, 0.09, partition_size=128, workspace=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out.cpu(), want[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.cpu(), want[0])


def test_refusals():
    dev = torch.device("cuda")
    q, cache, bt, L = (t.to(dev) for t in kv4_case(15, 2, 4, 2, 64, 16, [40, 20], F16))
    out = torch.empty_like(q)
    with pytest.raises(TypeError):
        binding.pa_decode_v2_kv4(out.float(), q.float(), cache, bt, L, 0.1)
    with pytest.raises(ValueError):
        binding.pa_decode_v2_kv4(out, q, cache[:, :, :-8].contiguous(), bt, L, 0.1)
    with pytest.raises(ValueError):
        binding.pa_decode_v2_kv4(out, q, cache, bt.cpu(), L, 0.1)
    with pytest.raises(binding.PaError):
        binding.pa_decode_v2_kv4(out, q, cache, bt, L, float("nan"))
    with pytest.raises(binding.PaError):
        binding.pa_decode_v2_kv4(out, q, cache, bt, L, 0.1, workspace=torch.empty(256, dtype=torch.uint8, device=dev))
