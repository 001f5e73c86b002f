"""Long runs of a warp over a 4-bit cache: partitions of more than 32 blocks
(the block ids come 32 at a time), rings that wrap many times, units that run on
into the next claimed one, and grids of a few CTAs whose warps take many units
each before the teams."""
import pytest
import torch

from decode_attention_paged_pa_gb300 import binding
from kv4_testutil import attend64, kv4_case

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16

# (heads, kv heads, head size, new tokens): two kv heads a unit, eight rows, one
# row, sixteen rows, head size 256.
UNITS = [(8, 2, 128, 1), (16, 2, 64, 1), (3, 3, 96, 1), (8, 2, 128, 4), (4, 2, 256, 1)]


def check(case, P, pick, dtype, **kw):
    q, cache, bt, L = case
    call = binding.pa_decode_v2_kv4 if q.dim() == 3 else binding.pa_decode_v2_mq_kv4
    dev = torch.device("cuda")
    qd, cd, bd, ld = (t.to(dev) for t in case)
    out, lse = torch.full_like(qd, float("nan")), torch.full(q.shape[:-1], float("nan"), device=dev)
    ws = call(out, qd, cd, bd, ld, 0.09, partition_size=P, lse=lse, **kw)
    assert binding.device_status(ws) == binding.PA_OK
    ref, bound, rl, rb = attend64(q[pick], cache, bt[pick], L[pick], 0.09, dtype)
    err = (out[pick].cpu().double() - ref).abs()
    assert bool((err <= bound).all()), f"worst {float((err / bound.clamp(min=1e-30)).max()):.2f} of the bound"
    assert bool(((lse[pick].cpu().double() - rl).abs() <= rb).all())
    assert not bool(out.isnan().any())


@pytest.mark.parametrize("BS,P", [(8, 512), (16, 1024), (8, 1024), (8, 2048), (64, 4096)])
@pytest.mark.parametrize("H,KH,D,q_len", UNITS)
def test_partitions_of_many_blocks(H, KH, D, q_len, BS, P):
    """Few units: teams, whose warps take parts of a partition."""
    lens = [1100, 2049, 1024, 3001, 257]
    case = kv4_case(BS + P + H, 5, H, KH, D, BS, lens, BF16, q_len=q_len)
    check(case, P, [0, 1, 2, 3, 4], BF16)


@pytest.mark.parametrize("BS,P", [(8, 512), (16, 1024), (8, 1024)])
@pytest.mark.parametrize("H,KH,D,q_len", UNITS)
def test_units_of_many_blocks_taken_whole(H, KH, D, q_len, BS, P):
    """More units than the GPU has warps; every block of a few sequences is
    looked at, the others draw on one pool."""
    units = KH // 2 if (H // KH) * q_len <= 4 and KH % 2 == 0 and D <= 128 else KH
    S = -(-2000 // (units * (2 if P == 512 else 1)))
    g = torch.Generator().manual_seed(S)
    lens = [int(v) for v in torch.randint(P + 40, P + 500, (S,), generator=g)]
    case = kv4_case(S + BS, S, H, KH, D, BS, lens, F16, q_len=q_len, NB=700)
    check(case, P, [0, S // 2, S - 1], F16)


@pytest.mark.parametrize("max_ctas", [1, 2, 5])
@pytest.mark.parametrize("H,KH,D,q_len", UNITS)
def test_a_few_ctas(H, KH, D, q_len, max_ctas):
    """Each warp takes many units, of one token to many stages, and joins teams at the end."""
    lens = [1, 700, 64, 33, 1025, 2, 513, 90, 300, 5, 64, 65]
    lens = [max(v, q_len) for v in lens]
    case = kv4_case(H + max_ctas, 12, H, KH, D, 8, lens, BF16, q_len=q_len)
    check(case, 64, list(range(12)), BF16, max_ctas=max_ctas)
    check(case, 512, list(range(12)), BF16, max_ctas=max_ctas)
