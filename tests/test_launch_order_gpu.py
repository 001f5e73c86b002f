"""Calls enqueued one behind the other, without a synchronisation: sequences
that all fit one partition of a table that holds many (short chats, tables for
the longest context), more units than the GPU has warps, one workspace for every
decode.  Each output is bitwise that of the same call alone."""
import pytest
import torch

from decode_attention_paged_pa_gb300 import binding
from kv4_testutil import kv4_case
from pa_testutil import random_case

pytestmark = pytest.mark.gpu

S, H, KH, D, BS, P = 480, 8, 8, 64, 16, 64


def lengths():
    return [(i * 29) % 65 for i in range(S)]


def case(kind, MB):
    """(decode(out, query, workspace), queries, caches, tables, lens)."""
    dev = torch.device("cuda")
    lens = lengths()
    if kind == "kv4":
        q, cache, bt, L = kv4_case(1, S, H, KH, D, BS, lens, torch.float16, MB=4, NB=6 * S)
        caches = [cache.to(dev)]
    else:
        q, kc, vc, bt, L = random_case(1, S=S, H=H, KH=KH, D=D, BS=BS, lens=[max(v, 1) for v in lens])
        lens = L.tolist()
        caches = [kc.to(dev), vc.to(dev)]
    NB = caches[0].shape[0]
    # A pool with holes: one block, one holder.
    ids = torch.randperm(NB, generator=torch.Generator().manual_seed(2)).to(torch.int32)
    tables = torch.zeros((S, MB), dtype=torch.int32)
    refs = torch.zeros(NB, dtype=torch.int32)
    at = 0
    for s, v in enumerate(lens):
        n = -(-v // BS)
        tables[s, :n] = ids[at:at + n]
        at += n
    refs[ids[:at].long()] = 1
    L = L.to(dev)
    call = binding.pa_decode_v2_kv4 if kind == "kv4" else binding.pa_decode_v2

    def decode(out, query, t, c, ws):
        call(out, query, *c, t, L, 0.11, partition_size=P, workspace=ws)

    queries = [torch.randn((S, H, D), generator=torch.Generator().manual_seed(i)).to(q.dtype).to(dev)
               for i in range(3)]
    return decode, queries, caches, tables.to(dev), L, refs.to(dev)


@pytest.mark.parametrize("MB", [32, 128])  # tables of 8 and of 32 partitions: both combine launches
@pytest.mark.parametrize("kind", ["kv4", "fp16"])
def test_decode_decode_compact_decode(kind, MB):
    decode, queries, caches, tables, L, refs = case(kind, MB)
    ws = torch.empty(binding.workspace_bytes(S, H, KH, D, MB, BS, P), dtype=torch.uint8, device="cuda")
    want = []
    for q in queries:
        o = torch.full_like(q, float("nan"))
        decode(o, q, tables, caches, ws)
        torch.cuda.synchronize()
        assert binding.device_status(ws) == binding.PA_OK
        want.append(o)
    plan = torch.empty(binding.pages_workspace_bytes(S, MB, refs.numel()), dtype=torch.uint8, device="cuda")
    for _ in range(20):
        now = [t.clone() for t in (tables, refs)] + [c.clone() for c in caches]
        outs = [torch.full_like(q, float("nan")) for q in queries]
        torch.cuda.synchronize()
        t, r, c = now[0], now[1], now[2:]
        decode(outs[0], queries[0], t, c, ws)
        decode(outs[1], queries[1], t, c, ws)
        binding.pa_pages_compact(t, L, r, c, BS, workspace=plan)
        decode(outs[2], queries[2], t, c, ws)
        torch.cuda.synchronize()
        assert binding.device_status(ws) == binding.device_status(plan) == binding.PA_OK
        used = int((refs > 0).sum())
        assert bool((r[:used] == 1).all()) and not bool(r[used:].any())
        for got, w in zip(outs, want):
            assert torch.equal(got, w)
