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
