"""A decode step over a 4-bit cache whose pool is full: the resize is refused and
its status says so before anything is appended, and the tokens that were cached
are as they were; with blocks freed the step goes on."""
import pytest
import torch

import decode_attention_paged_pa_gb300 as pa
from kv4_testutil import kv4_case

pytestmark = pytest.mark.gpu


def step(out, query, key, value, kv_cache, block_tables, seq_lens, refcounts, scale, block_size):
    ws = pa.pa_pages_resize(block_tables, seq_lens, seq_lens + 1, refcounts, [kv_cache], block_size)
    if pa.device_status(ws) != pa.PA_OK:
        return pa.device_status(ws)
    for ws in (pa.pa_kv4_append(kv_cache, key, value, block_tables, seq_lens),
               pa.pa_decode_v2_kv4(out, query, kv_cache, block_tables, seq_lens, scale)):
        assert pa.device_status(ws) == pa.PA_OK
    return pa.PA_OK


def test_a_step_of_a_full_pool():
    dev = torch.device("cuda")
    D, KH, H, BS, dtype = 128, 2, 8, 16, torch.bfloat16
    lens = [32, 16, 40]  # the first two need a block for their next token
    query, cache, _, L = (t.to(dev) for t in kv4_case(1, 3, H, KH, D, BS, lens, dtype, MB=4, NB=7))
    tables = torch.tensor([[4, 2, 0, 0], [6, 0, 0, 0], [1, 5, 3, 0]], dtype=torch.int32, device=dev)
    refs = torch.tensor([0, 1, 1, 1, 1, 1, 1], dtype=torch.int32, device=dev)  # block 0 is free
    g = torch.Generator().manual_seed(2)
    key, value = (torch.randn((3, KH, D), generator=g).to(dtype).to(dev) for _ in range(2))
    args = (torch.empty_like(query), query, key, value, cache, tables, L, refs, 0.09, BS)
    before = [t.clone() for t in (cache, tables, L, refs)]
    assert step(*args) == pa.PA_ERR_NO_BLOCKS
    for a, b in zip((cache, tables, L, refs), before):
        assert torch.equal(a, b)
    # The last sequence ends: its blocks are free for the next step.
    ws = pa.pa_pages_resize(tables, L, torch.tensor([32, 16, 0], dtype=torch.int32, device=dev), refs, cache, BS)
    assert pa.device_status(ws) == pa.PA_OK
    assert step(*args) == pa.PA_OK
    assert L.tolist() == [33, 17, 1] and int(refs.sum()) == 6
    ko, vo = torch.empty_like(key), torch.empty_like(value)
    ws = pa.pa_kv4_gather(ko, vo, cache, tables, L)
    assert pa.device_status(ws) == pa.PA_OK
    # A value is off by half the width of a code, and two roundings to bf16 (the scale, 15 codes of it; the value).
    for got, x in ((ko, key), (vo, value)):
        x, got = x.double(), got.double()
        width = (x.amax(-1, keepdim=True) - x.amin(-1, keepdim=True)) / 15
        assert bool(((got - x).abs() <= width * (0.5 + 15 * 2.0 ** -8) * 1.01 + 2.0 ** -8 * (x.abs() + width)).all())
