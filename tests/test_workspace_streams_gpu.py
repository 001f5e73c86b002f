"""Calls on a stream that is not the current one, their workspaces dropped at
once, while the current stream makes tensors of the same sizes and fills them:
every result is that of the call on the current stream."""
import pytest
import torch

from decode_attention_paged_pa_gb300 import binding
from kv4_testutil import kv4_case
from pa_testutil import random_case

pytestmark = pytest.mark.gpu

DEV = "cuda"


def decode_kv4(q_len):
    q, c, bt, L = (t.to(DEV) for t in kv4_case(3, 6, 8, 2, 128, 16, [40 + 90 * i for i in range(6)], torch.bfloat16,
                                               q_len=q_len))
    call = binding.pa_decode_v2_kv4 if q_len == 1 else binding.pa_decode_v2_mq_kv4

    def run(stream):
        out = torch.empty_like(q)
        call(out, q, c, bt, L, 0.09, partition_size=64, stream=stream)
        return [out]
    return run


def decode_16bit(q_len):
    q, kc, vc, bt, L = (t.to(DEV) for t in random_case(3, S=6, H=8, KH=2, D=128, BS=16, lens=[40 + 90 * i for i in range(6)]))
    if q_len > 1:
        q = q[:, None].expand(-1, q_len, -1, -1).contiguous()
    call = binding.pa_decode_v2 if q_len == 1 else binding.pa_decode_v2_mq

    def run(stream):
        out = torch.empty_like(q)
        call(out, q, kc, vc, bt, L, 0.09, partition_size=64, stream=stream)
        return [out]
    return run


def decode_fp8(q_len):
    g = torch.Generator().manual_seed(5)
    S, H, KH, D, BS, MB = 4, 8, 2, 128, 16, 20
    q = torch.randn((S, q_len, H, D) if q_len > 1 else (S, H, D), generator=g).to(torch.float16).to(DEV)
    codes = torch.randint(0, 120, (2, S * MB, KH * D * BS), generator=g, dtype=torch.uint8).to(DEV)
    kc, vc = codes[0].view(S * MB, KH, D // 16, BS, 16), codes[1].view(S * MB, KH, D, BS)
    bt = torch.randperm(S * MB, generator=g).view(S, MB).to(torch.int32).to(DEV)
    L = torch.tensor([300, 17, 64, 220], dtype=torch.int32, device=DEV)
    call = binding.pa_decode_v2_fp8 if q_len == 1 else binding.pa_decode_v2_mq_fp8

    def run(stream):
        out = torch.empty_like(q)
        call(out, q, kc, vc, bt, L, 0.01, partition_size=64, stream=stream)
        return [out]
    return run


def pages():
    S, MB, NB, BS = 40, 12, 1200, 16
    g = torch.Generator().manual_seed(6)
    lens = torch.randint(1, MB * BS // 2, (S,), generator=g)
    tables = torch.randperm(NB, generator=g)[: S * MB].view(S, MB).to(torch.int32)
    refs = torch.zeros(NB, dtype=torch.int32)
    for s in range(S):
        refs[tables[s, : -(-int(lens[s]) // BS)].long()] += 1
    cache = torch.randint(0, 256, (NB, 64), generator=g, dtype=torch.uint8)
    new = (lens + torch.randint(-20, 60, (S,), generator=g)).clamp(0, MB * BS).to(torch.int32).to(DEV)
    start = [t.to(DEV) for t in (tables, lens.to(torch.int32), refs, cache)]
    parents = torch.arange(S, dtype=torch.int32, device=DEV)

    def run(stream):
        t, L, r, c = (x.clone() for x in start)
        out, lo = torch.zeros_like(t), torch.zeros_like(L)
        zero = torch.zeros_like(L)
        stream.wait_stream(torch.cuda.current_stream())
        binding.pa_pages_resize(t, L, new, r, c, BS, stream=stream)
        binding.pa_pages_fork(out, lo, t, L, parents, r, c, BS, stream=stream)
        binding.pa_pages_resize(t, L, zero, r, c, BS, stream=stream)
        binding.pa_pages_compact(out, lo, r, c, BS, stream=stream)
        return [t, L, r, c, out, lo, zero]  # (zero: kept as long as the calls read it)
    return run


@pytest.mark.parametrize("make", [lambda: decode_kv4(1), lambda: decode_kv4(4), lambda: decode_16bit(1),
                                  lambda: decode_16bit(3), lambda: decode_fp8(1), lambda: decode_fp8(2), pages],
                         ids=["kv4", "mq_kv4", "16bit", "mq", "fp8", "mq_fp8", "pages"])
def test_dropped_workspaces(make):
    run = make()
    current = torch.cuda.current_stream()
    want = [t.clone() for t in run(current)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    raw = torch.cuda.ExternalStream(side.cuda_stream)
    for stream in (side, raw):
        side.wait_stream(current)
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)  # (some 10 ms: the calls wait behind it)
        got = run(stream)
        junk = [torch.full((n,), 255, dtype=torch.uint8, device=DEV)
                for n in (256, 1 << 12, 1 << 15, 1 << 17, 1 << 19, 1 << 20, 1 << 21, 1 << 23) for _ in range(4)]
        torch.cuda.synchronize()
        del junk
        for g, w in zip(got, want):
            assert torch.equal(g, w)
