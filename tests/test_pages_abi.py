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


# Arrays that lie apart: two rows of four blocks, three children, a pool of eight blocks.
APART = dict(bt=FAKE, lens=FAKE * 2, arg=FAKE * 3, out=FAKE * 4, lo=FAKE * 5, refs=FAKE * 6, caches=[FAKE * 7],
             ws=FAKE * 8)
SIZE = dict(bt=32, lens=8, arg=8, out=48, lo=12, refs=32, ids=32, caches=8 * 1024, ws=binding.pages_workspace_bytes(2, 4, 8))


@pytest.mark.parametrize("fn,written,other", [
    # The children's rows and lengths, over what the call reads and over one another.
    *[("pa_pages_fork", w, o) for w in ("out", "lo") for o in ("bt", "lens", "arg", "refs", "caches", "ws")],
    ("pa_pages_fork", "out", "lo"),
    ("pa_pages_fork", "refs", "bt"), ("pa_pages_fork", "refs", "arg"), ("pa_pages_fork", "ws", "arg"),
    # The tables and lengths in place; new lengths that overlap the lengths in part.
    *[("pa_pages_resize", w, o) for w in ("bt", "lens", "refs", "ws") for o in ("arg", "caches")],
    ("pa_pages_resize", "bt", "lens"), ("pa_pages_resize", "bt", "refs"), ("pa_pages_resize", "lens", "refs"),
    *[("pa_pages_compact", w, o) for w in ("bt", "refs", "ids") for o in ("lens", "caches", "ws")],
    ("pa_pages_compact", "ids", "refs"), ("pa_pages_compact", "ids", "bt"),
])
@pytest.mark.parametrize("end", ["first", "last"])
def test_rejects_what_is_written_over_another_array(fn, written, other, end):
    """`other` begins at the last word of `written`, or ends at its first one."""
    a = dict(APART)
    base = FAKE * 32
    off = SIZE[written] - 4 if end == "last" else 4 - SIZE[other]
    if other in ("ws", "caches") or written in ("ws", "caches"):
        off = off // 16 * 16 if end == "last" else -(-off // 16) * 16
        off = off if end == "last" else min(off, 0)
    a[written] = [base] if written == "caches" else base
    a[other] = [base + off] if other == "caches" else base + off
    assert call(fn, **a) == BAD
