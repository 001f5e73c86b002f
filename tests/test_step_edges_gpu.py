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
