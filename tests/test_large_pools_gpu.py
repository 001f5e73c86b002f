"""4-bit caches and pages whose byte offsets pass 32 bits: the same records at
low ids of a small pool and all over a large one give the same bits."""
import pytest
import torch

from decode_attention_paged_pa_gb300 import binding
from kv4_testutil import kv4_case

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16
GB = 1 << 30


@pytest.mark.parametrize("H,KH,q_len", [(8, 2, 1), (6, 3, 1), (8, 2, 3)])
def test_records_past_four_gigabytes(H, KH, q_len):
    D, BS = 128, 16
    lens = [5, 700, 64, 1, 333]
    q, cache, bt, L = kv4_case(H + q_len, len(lens), H, KH, D, BS, [max(v, q_len) for v in lens], BF16, q_len=q_len)
    nb = cache.shape[0]
    NB = 5 * GB // (KH * BS * (D + 8))
    dev = torch.device("cuda")
    where = torch.linspace(0, NB - 1, nb, dtype=torch.float64).long().to(dev)  # of the small pool's blocks
    large = torch.empty((NB,) + cache.shape[1:], dtype=torch.uint8, device=dev)
    small, bs = cache.to(dev), bt.to(dev)
    large[where] = small
    bl = where[bs.long()].to(torch.int32)
    ld, qd = L.to(dev), q.to(dev)
    g = torch.Generator().manual_seed(3)
    new = torch.randn((len(lens), KH, D), generator=g).to(BF16).to(dev)
    got = []
    for c, t in ((small, bs), (large, bl)):
        assert binding.device_status(binding.pa_kv4_append(c, new, new + 1, t, ld)) == binding.PA_OK
        out, ko = torch.empty_like(qd), torch.empty((int(L.sum()), KH, D), dtype=BF16, device=dev)
        vo = torch.empty_like(ko)
        call = binding.pa_decode_v2_kv4 if q_len == 1 else binding.pa_decode_v2_mq_kv4
        assert binding.device_status(call(out, qd, c, t, ld, 0.09, partition_size=128)) == binding.PA_OK
        cu = torch.cat([ld.new_zeros(1), ld.cumsum(0, dtype=torch.int32)])
        assert binding.device_status(binding.pa_kv4_gather(ko, vo, c, t, ld, cu_tokens=cu)) == binding.PA_OK
        got.append((out, ko, vo))
    assert torch.equal(large[where], small)
    for a, b in zip(*got):
        assert torch.equal(a, b)


def test_pages_past_four_gigabytes():
    page, BS, MB = 1 << 16, 16, 4
    NB = 5 * GB // page
    dev = torch.device("cuda")
    cache = torch.zeros((NB, page), dtype=torch.uint8, device=dev)
    # Two rows at the pool's end; free are three blocks before them and, below, block 7.
    refs = torch.ones(NB, dtype=torch.int32, device=dev)
    refs[NB - 8:NB - 5] = 0
    refs[7] = 0
    t = torch.tensor([[NB - 1, NB - 2, -1, -1], [NB - 3, -1, -1, -1]], dtype=torch.int32, device=dev)
    lens = torch.tensor([20, 9], dtype=torch.int32, device=dev)
    src = torch.randint(0, 256, (2, page), dtype=torch.uint8, generator=torch.Generator().manual_seed(1)).to(dev)
    cache[NB - 2], cache[NB - 3] = src[0], src[1]
    out = torch.full((3, MB), -1, dtype=torch.int32, device=dev)
    lo = torch.zeros(3, dtype=torch.int32, device=dev)
    par = torch.tensor([1, 0, 1], dtype=torch.int32, device=dev)
    ws = binding.pa_pages_fork(out, lo, t, lens, par, refs, [cache], BS)
    assert binding.device_status(ws) == binding.PA_OK
    assert out.tolist() == [[7, -1, -1, -1], [NB - 1, NB - 8, -1, -1], [NB - 7, -1, -1, -1]]
    assert lo.tolist() == [9, 20, 9]
    for at, i in ((7, 1), (NB - 8, 0), (NB - 7, 1)):
        assert torch.equal(cache[at], src[i])
    # The rest of the pool empties; what is left moves to the front.
    refs.zero_()
    refs[NB - 1], refs[NB - 2], refs[NB - 3] = 1, 1, 1
    ids = torch.empty(NB, dtype=torch.int32, device=dev)
    ws = binding.pa_pages_compact(t, lens, refs, [cache], BS, new_ids=ids)
    assert binding.device_status(ws) == binding.PA_OK
    assert t.tolist() == [[2, 1, -1, -1], [0, -1, -1, -1]] and ids[NB - 3:].tolist() == [0, 1, 2]
    assert torch.equal(cache[1], src[0]) and torch.equal(cache[0], src[1])
    assert refs[:3].tolist() == [1, 1, 1] and int(refs.sum()) == 3
