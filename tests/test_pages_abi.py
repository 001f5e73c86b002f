"""The pages entry points refuse bad arguments before they touch the GPU."""
import ctypes

import pytest

from decode_attention_paged_pa_gb300 import binding

FAKE = 0x100000  # an aligned non-null address; never dereferenced by these calls
BAD = binding.PA_ERR_INVALID_ARG


def _align(x):
    return (x + 255) // 256 * 256


@pytest.mark.parametrize("rows,MB,NB", [(0, 1, 1), (5, 9, 100), (1000, 4, 64), (128, 513, 65536)])
def test_workspace_bytes(rows, MB, NB):
    r, b = _align(4 * rows), _align(4 * NB)
    assert binding.pages_workspace_bytes(rows, MB, NB) == 256 + 4 * r + max(r, b) + 2 * b


def test_workspace_bytes_of_invalid_sizes_is_zero():
    for a in ((-1, 4, 4), (4, 0, 4), (4, 4, 0)):
        assert binding.pages_workspace_bytes(*a) == 0


def call(fn, **kw):
    a = dict(out=FAKE * 2, lo=FAKE * 3, bt=FAKE, lens=FAKE * 4, arg=FAKE, refs=FAKE, ids=None, caches=[FAKE],
             sizes=[1024], S=2, n=3, MB=4, BS=16, NB=8, stream=None, ws=FAKE, bytes=1 << 20)
    a.update(kw)
    nc = a.get("nc", len(a["caches"]))
    c = (ctypes.c_void_p * max(1, len(a["caches"])))(*a["caches"])
    s = (ctypes.c_size_t * max(1, len(a["sizes"])))(*a["sizes"])
    if a.get("no_array"):
        c = None
    tail = [a["MB"], a["BS"], a["NB"], a["stream"], a["ws"], a["bytes"]]
    if fn == "pa_pages_fork":
        args = [a[k] for k in ("out", "lo", "bt", "lens", "arg", "refs")] + [c, s, nc, a["S"], a["n"]]
    elif fn == "pa_pages_resize":
        args = [a[k] for k in ("bt", "lens", "arg", "refs")] + [c, s, nc, a["S"]]
    else:
        args = [a[k] for k in ("bt", "lens", "refs", "ids")] + [c, s, nc, a["S"]]
    return getattr(binding.lib(), fn)(*args, *tail)


@pytest.mark.parametrize("fn", ["pa_pages_fork", "pa_pages_resize", "pa_pages_compact"])
@pytest.mark.parametrize("kw,status", [
    (dict(S=-1), BAD), (dict(MB=0), BAD), (dict(BS=0), BAD), (dict(NB=0), BAD), (dict(MB=1 << 28, BS=8), BAD),
    (dict(refs=None), BAD), (dict(refs=FAKE + 2), BAD), (dict(bt=None), BAD), (dict(lens=FAKE + 1), BAD),
    (dict(nc=-1), BAD), (dict(no_array=True), BAD), (dict(caches=[None]), BAD), (dict(caches=[FAKE + 8]), BAD),
    (dict(sizes=[0]), BAD), (dict(sizes=[24]), BAD), (dict(sizes=[2 ** 35 + 16]), BAD),
    (dict(ws=None), BAD), (dict(ws=FAKE + 8), BAD),
    (dict(bytes=256), binding.PA_ERR_WORKSPACE),
])
def test_rejects(fn, kw, status):
    assert call(fn, **kw) == status


@pytest.mark.parametrize("fn,kw", [
    ("pa_pages_fork", dict(arg=None)), ("pa_pages_fork", dict(n=-1)), ("pa_pages_fork", dict(n=1 << 24)), ("pa_pages_fork", dict(out=None)),
    ("pa_pages_fork", dict(lo=FAKE * 3 + 2)), ("pa_pages_fork", dict(out=FAKE)),
    ("pa_pages_fork", dict(out=FAKE + 2 * 16 - 4)), ("pa_pages_fork", dict(lo=FAKE * 4 + 4)),
    ("pa_pages_resize", dict(arg=None)), ("pa_pages_compact", dict(ids=FAKE + 2)),
])
def test_rejects_of_one_call(fn, kw):
    assert call(fn, **kw) == BAD


def test_status_string_of_a_full_pool():
    assert "free blocks" in binding.status_string(binding.PA_ERR_NO_BLOCKS)
