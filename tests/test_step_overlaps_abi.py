"""Cache writes and accepted paths refuse arrays that overlap what they write, before they
touch the GPU."""
import ctypes

import pytest

from decode_attention_paged_pa_gb300 import binding

M = 1 << 24  # addresses 16 MB apart; never dereferenced: every call here is refused
BAD = binding.PA_ERR_INVALID_ARG
F = ctypes.c_float
CACHE = 8 * 2 * 64 * 16 * 2  # bytes of the caches below


def write(**kw):
    a = dict(kc=M, vc=2 * M, key=3 * M, value=4 * M, slots=5 * M, ks=1.0, vs=1.0, N=5, KH=2, D=64, BS=16, kst=128, vst=128,
             dtype=0, cdt=0, stream=None, NB=8, ws=6 * M, bytes=256)
    a.update(kw)
    return binding.lib().pa_cache_write(a["kc"], a["vc"], a["key"], a["value"], a["slots"], F(a["ks"]), F(a["vs"]),
                                        *[a[k] for k in ("N", "KH", "D", "BS", "kst", "vst", "dtype", "cdt", "stream",
                                                         "NB", "ws", "bytes")])


@pytest.mark.parametrize("kw", [
    dict(vc=M), dict(vc=M + CACHE - 16), dict(kc=2 * M + CACHE - 16), dict(key=M + 1024), dict(key=M - 16), dict(value=M + 256),
    dict(key=2 * M + CACHE - 16), dict(value=2 * M), dict(slots=M + 8), dict(slots=2 * M + CACHE - 8), dict(slots=M - 8),
    dict(ws=M + 16), dict(ws=2 * M - 240), dict(ws=3 * M), dict(ws=4 * M + 4 * 256 + 240), dict(ws=5 * M + 32),
    dict(key=M - 4 * 2 * 640 - 128, kst=640),                # the last row, a slice of wider ones, reaches into the cache
    dict(cdt=3, vc=M + CACHE // 2 - 16), dict(dtype=2, cdt=2, vc=M + 2 * CACHE - 16),
])
def test_write_refuses_overlaps(kw):
    assert write(**kw) == BAD


def accept(**kw):
    a = dict(new=M, k=[8 * M, 10 * M], v=[9 * M, 11 * M], bt=2 * M, lens=3 * M, acc=4 * M, num=5 * M, S=2, n=5, A=4, KH=2, D=64,
             BS=16, cdt=0, stream=None, MB=4, NB=8, ws=6 * M, bytes=256)
    a.update(kw)
    k, v = ((ctypes.c_void_p * len(a[x]))(*a[x]) for x in "kv")
    return binding.lib().pa_tree_accept(a["new"], k, v, len(a["k"]), *[a[x] for x in (
        "bt", "lens", "acc", "num", "S", "n", "A", "KH", "D", "BS", "cdt", "stream", "MB", "NB", "ws", "bytes")])


LAYERS = [(100 + 2 * i) * M for i in range(200)]


@pytest.mark.parametrize("kw", [
    dict(k=[8 * M, 8 * M]), dict(v=[8 * M, 11 * M]), dict(v=[9 * M, 10 * M]), dict(k=[8 * M, 9 * M + CACHE - 16]),
    dict(k=[11 * M + CACHE - 16, 10 * M]), dict(k=[8 * M], v=[8 * M]), dict(cdt=3, k=[8 * M, 9 * M - CACHE // 2 + 16]),
    dict(cdt=2, k=[8 * M, 9 * M + 2 * CACHE - 16]),
    dict(k=LAYERS, v=[x + M for x in LAYERS[:-1]] + [LAYERS[3] + M]),  # more than one launch takes
    dict(new=8 * M + 64), dict(new=11 * M + CACHE - 4), dict(ws=9 * M - 240), dict(bt=10 * M), dict(lens=10 * M + 4),
    dict(acc=9 * M + CACHE - 4), dict(num=8 * M - 4),
])
def test_accept_refuses_overlaps(kw):
    assert accept(**kw) == BAD
