"""Arguments that the step's operators record or refuse, at the ends of their ranges:
paths that are no paths, and empty calls."""
import pytest
import torch

from decode_attention_paged_pa_gb300 import binding
from view_testutil import caches

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32, torch.uint8], ids=["fp16", "fp32", "e4m3"])
def test_accept_reads_no_entry_outside_its_row_for_a_bad_path(dtype):
    """Entries that ascend from far below 0 or that come down and go up again beyond the
    nodes' number, in the first row and in the last one of the tables: each entry follows
    the one before it, and none of them, taken as a position, is in its row."""
    n, BS, A, MB = 4, 16, 512, 2
    paths = [[-(2 ** 31) + 5 * i for i in range(A)], [-900000, -800000, -5, 0], [2, 3] * (A // 2), [0, 1, 2, 3] * (A // 4),
             [2 ** 31 - 1 - i for i in range(A)], [1, 3], [-(2 ** 30), 2], [2, 3] * (A // 2)]
    counts = [A, 4, A, A, A, 2, 2, 300]
    lens = [4, 4, 32, 31, 4, 20, 4, 32]
    S = len(lens)
    bt = torch.randperm(S * MB, generator=torch.Generator().manual_seed(1)).view(S, MB).to(torch.int32)
    kc, vc = caches(2, S * MB, 2, 64, BS, dtype)
    d = kc.to(DEV), vc.to(DEV)
    acc = torch.full((S, A), 7, dtype=torch.int64)
    for s, p in enumerate(paths):
        acc[s, :len(p)] = torch.tensor(p)
    new = torch.zeros((S,), dtype=torch.int32, device=DEV)
    ws = binding.pa_tree_accept(new, *d, bt.to(DEV), i32(lens), acc.to(torch.int32).to(DEV), i32(counts), n)
    assert binding.device_status(ws) == binding.PA_ERR_DEVICE_BOUNDS
    assert new.tolist() == [18 if s == 5 else L for s, L in enumerate(lens)]
    for got, ref in ((d[0].cpu(), kc), (d[1].cpu(), vc)):
        ref = ref.clone()
        rows = [ref[bt[5, t // BS], :, :, t % BS].clone() for t in (17, 19)]
        for t, row in zip((16, 17), rows):
            ref[bt[5, t // BS], :, :, t % BS] = row
        assert torch.equal(got.view(torch.uint8), ref.view(torch.uint8))


@pytest.mark.parametrize("given", [True, False])
@pytest.mark.parametrize("op", ["accept", "window", "tree"])
def test_a_call_without_sequences_has_a_status(op, given):
    """On a workspace full of 0x7f bytes, on a side stream too; nothing else is touched."""
    kc, vc = (t.to(DEV) for t in caches(1, 4, 2, 64, 16, torch.float16))
    before = kc.clone(), vc.clone()
    bt, none = torch.empty((0, 2), dtype=torch.int32, device=DEV), torch.empty((0,), dtype=torch.int32, device=DEV)
    for stream in (None, torch.cuda.Stream()):
        ws = torch.full((1024,), 0x7F, dtype=torch.uint8, device=DEV) if given else None
        torch.cuda.synchronize()
        if op == "accept":
            ws = binding.pa_tree_accept(none, kc, vc, bt, none, torch.empty((0, 3), dtype=torch.int32, device=DEV), none, 4,
                                        workspace=ws, stream=stream)
        else:
            q = torch.empty((0, 3, 4, 64), dtype=torch.float16, device=DEV)
            args = (torch.empty_like(q), q, kc, vc, bt, none)
            if op == "window":
                ws = binding.pa_decode_v2_window(*args, 0.1, 16, workspace=ws, stream=stream)
            else:
                ws = binding.pa_decode_v2_tree(*args, torch.empty((0, 3, 1), dtype=torch.int32, device=DEV), 0.1, workspace=ws,
                                               stream=stream)
        assert binding.device_status(ws, stream) == binding.PA_OK
        assert torch.equal(kc, before[0]) and torch.equal(vc, before[1])
