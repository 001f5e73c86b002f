"""A key or value that is not finite stays in its kv head: the rows of the others, also of
one that shares a work unit with it, are bit for bit what they are without it."""
import math

import pytest
import torch

from decode_attention_paged_pa_gb300 import binding
from test_views_gpu import NAN_E4M3, T, make
from view_testutil import ancestors, pack, tree_parents

pytestmark = pytest.mark.gpu
DEV = "cuda"


def call(op, fp8, q, kc, vc, bt, lens, n):
    d = [t.to(DEV) for t in (q, kc, vc, bt, lens)]
    if op == "decode":
        d[0] = d[0].squeeze(1)
    out = torch.full_like(d[0], float("nan"))
    lse = torch.full(out.shape[:-1], float("nan"), device=DEV)
    more = dict(partition_size=128, lse=lse) | (dict(k_scale=0.5, v_scale=1.25) if fp8 else {})
    fn = {"decode": "pa_decode_v2", "mq": "pa_decode_v2_mq", "window": "pa_decode_v2_window", "tree": "pa_decode_v2_tree"}[op]
    args = [0.1]
    if op == "window":
        args += [1000, 0]
    if op == "tree":
        args = [pack(torch.stack([ancestors(tree_parents(s, n)) for s in range(len(lens))])).to(DEV), 0.1]
    ws = getattr(binding, fn + ("_fp8" if fp8 else ""))(out, *d, *args, **more)
    assert binding.device_status(ws) == binding.PA_OK
    return out.cpu().view(q.shape), lse.cpu().view(q.shape[:-1])


SHAPES = [("fp16", "same", 8, 2, 128, 16), ("bf16", "same", 16, 4, 64, 32), ("bf16", "same", 8, 2, 96, 8),
          ("bf16", "same", 8, 2, 128, 32), ("fp16", "same", 8, 2, 80, 8), ("fp16", "e4m3", 8, 2, 128, 16),
          ("bf16", "e4m3", 16, 4, 64, 8), ("bf16", "e4m3", 8, 2, 112, 32), ("fp16", "same", 4, 4, 64, 16),
          ("bf16", "same", 10, 2, 128, 64), ("fp32", "same", 4, 2, 64, 16)]


@pytest.mark.parametrize("op,n", [("decode", 1), ("mq", 2), ("window", 1), ("window", 2), ("tree", 1), ("tree", 2), ("window", 5)])
@pytest.mark.parametrize("shape", SHAPES, ids=["-".join(map(str, s)) for s in SHAPES])
def test_kv_heads_are_apart(shape, op, n):
    dtype, cache, H, KH, D, BS = shape
    if op == "mq" or (op != "decode" and n == 2):
        H = H // 2 if H // KH % 2 == 0 else H  # (two rows of half the heads: as many rows a kv head)
    fp8, G = cache == "e4m3", H // KH
    lens = [400, 70, n + 1]
    see = torch.stack([ancestors(tree_parents(s, n)) for s in range(len(lens))]) if op == "tree" else None
    q, kc, vc, bt, L = make(D + n, T[dtype], cache, n, H, KH, D, BS, lens, 1000 if see is None else 0, 0, see, poison=False)
    ref, ref_lse = call(op, fp8, q, kc, vc, bt, L, n)
    bad = [NAN_E4M3] if fp8 else [math.inf, -math.inf, math.nan]
    for what in ("value", "key"):
        k2, v2 = kc.clone(), vc.clone()
        for s, length in enumerate(lens):
            for kv in range(1, KH, 2):
                for i, x in enumerate(bad):
                    t = (17 * i + 5) % length
                    b, o = bt[s, t // BS], t % BS
                    if what == "value":
                        v2[b, kv, 3 + i, o] = x
                    else:
                        k2[b, kv, :, o] = x
        got, lse = call(op, fp8, q, k2, v2, bt, L, n)
        other = [h for h in range(H) if h // G % 2 == 0]
        hit = [h for h in range(H) if h // G % 2 == 1]
        assert torch.equal(got[:, :, other], ref[:, :, other]) and torch.equal(lse[:, :, other], ref_lse[:, :, other])
        # (The last row of a window or a chain sees every token; of a tree, those before it.)
        rows = got[:2, -1, :][:, hit]
        if what == "value":
            assert not bool(rows[..., 3].isfinite().any())
            assert bool(rows[..., 3 + len(bad):].isfinite().all())
        else:
            assert not bool(rows.isfinite().any())
