"""Failure detection of windowed and tree attention without a fault: a call whose waits
are bounded by less than its work takes gives up, records PA_ERR_TIMEOUT, lets its copies
and products complete and ends; the context stays usable, and the next call with the same
workspace is right.  With a bound of 1 ns almost the first wait runs out, with
microseconds one in the middle of the work, with copies and products on their way."""
import pytest
import torch

from decode_attention_paged_pa_gb300 import binding
from test_views_gpu import T, make
from view_testutil import ancestors, attend64, pack, tree_parents

pytestmark = pytest.mark.gpu
DEV = "cuda"

# Pages of a pool larger than the L2 cache, so that its copies take their time.
COPIES = 64


@pytest.mark.parametrize("n,H,KH,D,BS,dtype,cache", [
    (16, 8, 2, 128, 16, "bf16", "same"), (40, 4, 1, 128, 8, "fp16", "same"), (16, 8, 2, 128, 16, "bf16", "e4m3"),
    (16, 4, 1, 256, 32, "fp16", "same"), (20, 4, 1, 256, 16, "bf16", "e4m3"), (33, 6, 2, 64, 64, "fp16", "e4m3"),
    (1, 8, 2, 128, 16, "bf16", "same"), (2, 4, 2, 64, 32, "fp16", "e4m3"), (3, 2, 1, 64, 16, "fp32", "same"),
])
@pytest.mark.parametrize("op", ["tree", "window"])
def test_wait_bound_reports_timeout_and_context_survives(op, n, H, KH, D, BS, dtype, cache):
    S = 96
    lens = [n + 900 + 16 * (s % 7) for s in range(S)]
    see = torch.stack([ancestors(tree_parents(s, n)) for s in range(S)]) if op == "tree" else None
    window = 0 if op == "tree" else 700
    case = make(S + D, T[dtype], cache, n, H, KH, D, BS, lens, window, 0, see, poison=False)
    q, kc, vc, bt, L = (t.to(DEV) for t in case)
    NB = kc.shape[0]
    copies = COPIES if kc.nbytes < 1 << 26 else 8
    kc, vc = kc.repeat(copies, 1, 1, 1, 1), vc.repeat(copies, 1, 1, 1)
    bt = bt + NB * torch.randint(0, copies, bt.shape, device=DEV, dtype=torch.int32)
    more = dict(k_scale=0.5, v_scale=1.25) if cache == "e4m3" else {}
    args = (q, kc, vc, bt, L) + ((pack(see).to(DEV), 0.09) if op == "tree" else (0.09, window))
    call = getattr(binding, "pa_decode_v2_" + op + ("_fp8" if cache == "e4m3" else ""))
    flush = torch.zeros(1 << 28, dtype=torch.uint8, device=DEV)
    want = torch.empty_like(q)
    ws = call(want, *args, partition_size=256, **more)
    assert binding.device_status(ws) == binding.PA_OK
    pick = [0, S - 1]
    ref, _, bound = attend64(case[0][pick], case[1], case[2], case[3][pick], case[4][pick], 0.09, window, 0,
                             None if see is None else see[pick], 0.5, 1.25)
    assert bool(((want[pick].cpu().double() - ref).abs() <= bound).all())
    out = torch.empty_like(q)
    for timeout in (1, 1, 2000, 5000, 10000, 20000):
        flush.fill_(1)
        call(out, *args, partition_size=256, workspace=ws, timeout_ns=timeout, **more)
        status = binding.device_status(ws)
        assert status == binding.PA_ERR_TIMEOUT or (timeout > 1 and status == binding.PA_OK and torch.equal(out, want))
        out.fill_(float("nan"))
        call(out, *args, partition_size=256, workspace=ws, **more)
        assert binding.device_status(ws) == binding.PA_OK
        assert torch.equal(out, want)


@pytest.mark.parametrize("n", [1, 16])
def test_results_do_not_depend_on_the_grid(n):
    """(A unit's sums are the same whichever CTA runs it.)"""
    see = torch.stack([ancestors(tree_parents(s, n)) for s in range(6)])
    case = make(5, torch.bfloat16, "same", n, 8, 2, 128, 16, [n, 900, 300, 77, 500, 64], 0, 0, see, poison=False)
    d = [t.to(DEV) for t in case] + [pack(see).to(DEV), 0.1]
    outs = []
    for ctas in (0, 1, 3, 40):
        outs.append(torch.full_like(d[0], float("nan")))
        assert binding.device_status(binding.pa_decode_v2_tree(outs[-1], *d, partition_size=64, max_ctas=ctas)) == binding.PA_OK
    assert all(torch.equal(outs[0], o) for o in outs[1:])
