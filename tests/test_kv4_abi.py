"""The 4-bit entry points refuse bad arguments before they touch the GPU."""
import ctypes

import pytest

from decode_attention_paged_pa_gb300 import binding

FAKE = 0x10000  # a 16-byte aligned non-null address; never dereferenced by these calls


def test_block_bytes():
    for D in (64, 80, 96, 112, 128, 256):
        for BS in (8, 16, 32, 64):
            assert binding.kv4_block_bytes(D, BS) == BS * (D + 8)
    for D, BS in ((72, 16), (128, 24), (0, 16), (128, 0), (-64, 16), (512, 16)):
        assert binding.kv4_block_bytes(D, BS) == 0


def decode(q_len=None, **kw):
    a = dict(out=FAKE, lse=None, query=FAKE, cache=FAKE, bt=FAKE, lens=FAKE, scale=0.125, S=2, H=4, KH=2, D=128,
             BS=16, P=512, dtype=0, stream=None, MB=4, NB=8, ws=FAKE, n=1 << 30)
    a.update(kw)
    head = [a[k] for k in ("out", "lse", "query", "cache", "bt", "lens")] + [ctypes.c_float(a["scale"]), a["S"]]
    tail = [a[k] for k in ("H", "KH", "D", "BS", "P", "dtype", "stream", "MB", "NB", "ws", "n")]
    if q_len is None:
        return binding.lib().pa_decode_v2_kv4(*head, *tail)
    return binding.lib().pa_decode_v2_mq_kv4(*head, q_len, *tail)


@pytest.mark.parametrize("kw,status", [
    (dict(H=6, KH=4), binding.PA_ERR_INVALID_ARG),
    (dict(dtype=2), binding.PA_ERR_UNSUPPORTED),
    (dict(dtype=3), binding.PA_ERR_INVALID_ARG),
    (dict(D=72), binding.PA_ERR_UNSUPPORTED),
    (dict(BS=4), binding.PA_ERR_UNSUPPORTED),
    (dict(P=100), binding.PA_ERR_UNSUPPORTED),
    (dict(cache=None), binding.PA_ERR_INVALID_ARG),
    (dict(cache=FAKE + 8), binding.PA_ERR_INVALID_ARG),
    (dict(lse=FAKE + 2), binding.PA_ERR_INVALID_ARG),
    (dict(scale=float("inf")), binding.PA_ERR_INVALID_ARG),
    (dict(n=1024), binding.PA_ERR_WORKSPACE),
    (dict(S=0), binding.PA_OK),
    (dict(q_len=0), binding.PA_ERR_INVALID_ARG),
    (dict(q_len=1025), binding.PA_ERR_INVALID_ARG),
    (dict(q_len=4, n=1024), binding.PA_ERR_WORKSPACE),
    (dict(q_len=4, S=0), binding.PA_OK),
])
def test_decode_rejects(kw, status):
    assert decode(**kw) == status


def tokens(fn, **kw):
    a = dict(cache=FAKE, key=FAKE, value=FAKE, bt=FAKE, lens=FAKE, cu=FAKE, S=2, N=6, KH=2, D=128, BS=16, ks=256,
             vs=256, dtype=0, stream=None, MB=4, NB=8, ws=FAKE, n=256)
    a.update(kw)
    order = ("cache", "key", "value") if fn == "pa_kv4_append" else ("key", "value", "cache")
    return getattr(binding.lib(), fn)(*[a[k] for k in order], *[a[k] for k in (
        "bt", "lens", "cu", "S", "N", "KH", "D", "BS", "ks", "vs", "dtype", "stream", "MB", "NB", "ws", "n")])


@pytest.mark.parametrize("fn", ["pa_kv4_append", "pa_kv4_gather"])
@pytest.mark.parametrize("kw,status", [
    (dict(N=-1), binding.PA_ERR_INVALID_ARG),
    (dict(S=-1), binding.PA_ERR_INVALID_ARG),
    (dict(S=0), binding.PA_ERR_INVALID_ARG),
    (dict(KH=0), binding.PA_ERR_INVALID_ARG),
    (dict(MB=0), binding.PA_ERR_INVALID_ARG),
    (dict(NB=0), binding.PA_ERR_INVALID_ARG),
    (dict(MB=1 << 30), binding.PA_ERR_INVALID_ARG),
    (dict(dtype=2), binding.PA_ERR_UNSUPPORTED),
    (dict(dtype=-1), binding.PA_ERR_INVALID_ARG),
    (dict(D=72, ks=1024, vs=1024), binding.PA_ERR_UNSUPPORTED),
    (dict(BS=24), binding.PA_ERR_UNSUPPORTED),
    (dict(ks=248), binding.PA_ERR_INVALID_ARG),
    (dict(vs=260), binding.PA_ERR_INVALID_ARG),
    (dict(cu=None, N=7), binding.PA_ERR_INVALID_ARG),
    (dict(key=None), binding.PA_ERR_INVALID_ARG),
    (dict(value=FAKE + 8), binding.PA_ERR_INVALID_ARG),
    (dict(cache=None), binding.PA_ERR_INVALID_ARG),
    (dict(bt=None), binding.PA_ERR_INVALID_ARG),
    (dict(lens=FAKE + 2), binding.PA_ERR_INVALID_ARG),
    (dict(cu=FAKE + 1), binding.PA_ERR_INVALID_ARG),
    (dict(ws=None), binding.PA_ERR_INVALID_ARG),
    (dict(ws=FAKE + 4), binding.PA_ERR_INVALID_ARG),
    (dict(n=128), binding.PA_ERR_WORKSPACE),
])
def test_tokens_rejects(fn, kw, status):
    assert tokens(fn, **kw) == status


@pytest.mark.parametrize("max_ctas,timeout_ns,kw,status", [
    (-1, 0, {}, binding.PA_ERR_INVALID_ARG),
    (0, -1, {}, binding.PA_ERR_INVALID_ARG),
    (4, 1000, dict(S=0), binding.PA_OK),
    (4, 1000, dict(n=1024), binding.PA_ERR_WORKSPACE),
])
def test_decode_ex_rejects(max_ctas, timeout_ns, kw, status):
    a = dict(out=FAKE, lse=None, query=FAKE, cache=FAKE, bt=FAKE, lens=FAKE, scale=0.125, S=2, q_len=2, H=4, KH=2,
             D=128, BS=16, P=512, dtype=0, stream=None, MB=4, NB=8, ws=FAKE, n=1 << 30)
    a.update(kw)
    assert binding.lib().pa_decode_v2_kv4_ex(*a.values(), max_ctas, timeout_ns) == status
