"""Failure detection of the 4-bit kernel without a fault: a call whose waits are
bounded by 1 ns gives up at its first wait that does not succeed at once, records
PA_ERR_TIMEOUT, lets its copies land and ends; the context stays usable, and the
next call with the same workspace is right.  Whole units of single warps, then
teams, with warps that have given up among them."""
import pytest
import torch

from decode_attention_paged_pa_gb300 import binding
from kv4_testutil import attend64, kv4_case

pytestmark = pytest.mark.gpu


# A pool of this many copies of a small one, larger than the L2 cache, and
# batches that the memory bounds: hundreds of their waits run out.  (The other
# kinds of unit compute for longer than their pages take to come.)
COPIES = 100


@pytest.mark.parametrize("S,H,KH,D,BS,P", [
    (400, 8, 2, 128, 16, 512),
    (300, 8, 8, 128, 64, 512),
    (300, 8, 8, 128, 8, 1024),
])
def test_wait_bound_reports_timeout_and_context_survives(S, H, KH, D, BS, P):
    lens = [2048 + 5 * (s % 9) for s in range(S)]
    case = kv4_case(S + D, S, H, KH, D, BS, lens, torch.bfloat16, NB=600)
    q, cache, bt, L = (t.cuda() for t in case)
    large = cache.repeat(COPIES, 1, 1)
    bt = bt + 600 * torch.randint(0, COPIES, bt.shape, device="cuda", dtype=torch.int32)
    call = binding.pa_decode_v2_kv4
    out = torch.empty_like(q)
    flush = torch.zeros(1 << 28, dtype=torch.uint8, device="cuda")
    ws = call(out, q, large, bt, L, 0.09, partition_size=P, timeout_ns=1)
    assert binding.device_status(ws) == binding.PA_ERR_TIMEOUT
    out.fill_(float("nan"))
    flush.fill_(1)
    call(out, q, large, bt, L, 0.09, partition_size=P, workspace=ws)
    assert binding.device_status(ws) == binding.PA_OK
    pick = [0, S // 2, S - 1]
    ref, bound, _, _ = attend64(case[0][pick], case[1], case[2][pick], case[3][pick], 0.09, torch.bfloat16)
    assert bool(((out[pick].cpu().double() - ref).abs() <= bound).all())
    assert not bool(out.isnan().any())
