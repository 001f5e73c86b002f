"""The README's decode step over a 4-bit cache whose pool is full: the resize is
refused and its status says so, nothing is appended, and the tokens that were
cached are as they were; with blocks freed the step goes on."""
import os
import re

import pytest
import torch

import decode_attention_paged_pa_gb300 as pa
from kv4_testutil import kv4_case

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def readme_step():
    """The step's lines, up to the decode."""
    text = open(os.path.join(ROOT, "README.md")).read()
    code = next(c for c in re.findall(r"```python\n(.*?)```", text, flags=re.S) if "pa_pages_resize" in c)
    return code[:code.index("# samples or beams")]


def test_a_step_of_a_full_pool():
    dev = torch.device("cuda")
    D, KH, H, BS, dtype = 128, 2, 8, 16, torch.bfloat16
    lens = [32, 16, 40]  # the first two need a block for their next token
    query, cache, _, L = (t.to(dev) for t in kv4_case(1, 3, H, KH, D, BS, lens, dtype, MB=4, NB=7))
    tables = torch.tensor([[4, 2, 0, 0], [6, 0, 0, 0], [1, 5, 3, 0]], dtype=torch.int32, device=dev)
    refs = torch.tensor([0, 1, 1, 1, 1, 1, 1], dtype=torch.int32, device=dev)  # block 0 is free
    g = torch.Generator().manual_seed(2)
    key, value = (torch.randn((3, KH, D), generator=g).to(dtype).to(dev) for _ in range(2))
    names = dict(query=query, out=torch.empty_like(query), kv_cache=cache, block_tables=tables, seq_lens=L,
                 refcounts=refs, key=key, value=value, scale=0.09, block_size=BS)
    before = [t.clone() for t in (cache, tables, L, refs)]
    with pytest.raises(RuntimeError, match="no room"):
        exec(readme_step(), names)
    for a, b in zip((cache, tables, L, refs), before):
        assert torch.equal(a, b)
    # The last sequence ends: its blocks are free for the next step.
    ws = pa.pa_pages_resize(tables, L, torch.tensor([32, 16, 0], dtype=torch.int32, device=dev), refs, cache, BS)
    assert pa.device_status(ws) == pa.PA_OK
    exec(readme_step(), names)
    assert L.tolist() == [33, 17, 1] and int(refs.sum()) == 6
    ko, vo = torch.empty_like(key), torch.empty_like(value)
    ws = pa.pa_kv4_gather(ko, vo, cache, tables, L)
    assert pa.device_status(ws) == pa.PA_OK
    # A value is off by half a step of its code, and two roundings to bf16 (the scale, 15 codes of it; the value).
    for got, x in ((ko, key), (vo, value)):
        x, got = x.double(), got.double()
        step = (x.amax(-1, keepdim=True) - x.amin(-1, keepdim=True)) / 15
        assert bool(((got - x).abs() <= step * (0.5 + 15 * 2.0 ** -8) * 1.01 + 2.0 ** -8 * (x.abs() + step)).all())
