"""Calls of thousands of rows (chunks of prompts, whole contexts): several
tokens a CTA, sequence boundaries and empty sequences inside a CTA's run, a
ragged last run, vectors taken in several passes.  Stored bits against the
definition in 64 bits, read-back the nearest value of the type."""
import pytest
import torch

from decode_attention_paged_pa_gb300 import binding
from kv4_testutil import quantise64

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16


def lengths(N, seed):
    """Rows of the sequences: 0, 1, a few, thousands; N in all."""
    g = torch.Generator().manual_seed(seed)
    new, left = [0, 0, 1, 0, 33], N - 34
    while left > 0:
        kind = int(torch.randint(0, 4, (1,), generator=g))
        n = 0 if kind == 0 else min(left, int(torch.randint(1, (0, 4, 100, 3000)[kind], (1,), generator=g)))
        new.append(n)
        left -= n
    return new + [0]


# N past 2 * 8 * 152 rows gives a CTA two tokens or more, up to 16384 elements' worth and 32.
@pytest.mark.parametrize("N,KH,D,BS,dtype", [
    (3001, 8, 128, 16, BF16),    # 2 tokens a CTA
    (3001, 1, 80, 8, F16),
    (5003, 3, 96, 64, BF16),     # 4
    (10007, 8, 128, 16, F16),    # 8, as many as 8 heads of 128 dims get
    (10007, 4, 256, 32, BF16),
    (9001, 32, 64, 16, F16),     # 4, as many as 32 heads of 64 dims get
    (2500, 70, 128, 16, BF16),   # one: more than a CTA's elements in a token
    (41003, 1, 64, 8, BF16),     # 32, the most there are
    (41003, 1, 112, 16, F16),
    (40960, 2, 128, 32, F16),    # no ragged end
])
@pytest.mark.parametrize("uniform", [False, True], ids=["ragged", "uniform"])
def test_rows_by_the_thousand(N, KH, D, BS, dtype, uniform):
    dev = torch.device("cuda")
    if uniform:
        N -= N % 7
        new = [N // 7] * 7
    else:
        new = lengths(N, N + KH + D)
    S = len(new)
    ctx = [(s * 5) % 19 for s in range(S)]
    lens = [a + b for a, b in zip(new, ctx)]
    MB = max(1, max(-(-v // BS) for v in lens))
    need = sum(-(-v // BS) for v in lens)
    NB = need + 5
    g = torch.Generator().manual_seed(N)
    ids = torch.randperm(NB, generator=g).to(torch.int32)
    bt, at = torch.full((S, MB), -1, dtype=torch.int32), 0
    for s, v in enumerate(lens):
        n = -(-v // BS)
        bt[s, :n] = ids[at:at + n]
        at += n
    behind = 0 if uniform else 6  # rows behind the last sequence
    key, value = (torch.randn((N + behind, KH, D), generator=g).to(dtype) for _ in range(2))
    cache = torch.randint(0, 256, (NB, KH, BS * (D + 8)), generator=g, dtype=torch.uint8)
    # The definition, by rows: position, block and slot.
    n = torch.tensor(new)
    seq = torch.repeat_interleave(torch.arange(S), n)
    cu = torch.cat([torch.zeros(1, dtype=torch.long), n.cumsum(0)])
    pos = torch.tensor(lens)[seq] - n[seq] + torch.arange(N) - cu[seq]
    blk, slot = bt[seq, pos // BS].long(), pos % BS
    want, half, x = cache.clone(), BS * D // 2, min(D, 128)
    par = []
    for i, t in enumerate((key[:N], value[:N])):
        c, s, z = quantise64(t)
        b = (c[..., ::2] + 16 * c[..., 1::2]).to(torch.uint8).unflatten(-1, (D // x, x // 2))
        codes = want[..., i * half:(i + 1) * half].unflatten(-1, (D // x, BS, x // 2))
        codes[blk, :, :, slot] = b
        par += [s, z]
    p = torch.cat(par, -1).to(dtype).view(torch.uint8)
    want[..., 2 * half:].unflatten(-1, (BS, 8))[blk, :, slot] = p
    cd, bd, ld = cache.to(dev), bt.to(dev), torch.tensor(lens, dtype=torch.int32, device=dev)
    cud = None if uniform else cu.to(torch.int32).to(dev)
    ws = binding.pa_kv4_append(cd, key.to(dev), value.to(dev), bd, ld, cu_tokens=cud)
    assert binding.device_status(ws) == binding.PA_OK
    assert torch.equal(cd.cpu(), want)
    ko, vo = (torch.full((N + behind, KH, D), 7.0, dtype=dtype, device=dev) for _ in range(2))
    ws = binding.pa_kv4_gather(ko, vo, cd, bd, ld, cu_tokens=cud)
    assert binding.device_status(ws) == binding.PA_OK
    for i, got in enumerate((ko.cpu(), vo.cpu())):
        assert bool((got[N:] == 7).all())
        c, s, z = quantise64((key, value)[i][:N])
        ref = c * s + z
        err = (got[:N].double() - ref).abs()
        for step in (1, -1):  # the neighbouring patterns are no nearer
            near = (got[:N].view(torch.int16) + step).view(dtype).double()
            assert bool((err <= (near - ref).abs())[near.isfinite()].all())
