"""The entry points of windowed and tree attention, slot maps, cache writes and
accepted paths refuse bad arguments before they touch the GPU."""
import ctypes

import pytest

from decode_attention_paged_pa_gb300 import binding

FAKE = 0x100000  # an aligned non-null address; never dereferenced by these calls
BAD, UNS, WS = binding.PA_ERR_INVALID_ARG, binding.PA_ERR_UNSUPPORTED, binding.PA_ERR_WORKSPACE
F = ctypes.c_float


def view(op, **kw):
    a = dict(out=FAKE, lse=None, query=FAKE, kc=FAKE, vc=FAKE, bt=FAKE, lens=FAKE, masks=FAKE, scale=0.125, ks=1.0,
             vs=1.0, window=16, sinks=4, S=2, n=4, H=4, KH=2, D=128, BS=16, P=512, dtype=0, stream=None, MB=4, NB=8,
             ws=FAKE, bytes=1 << 30)
    a.update(kw)
    args = [a[k] for k in ("out", "lse", "query", "kc", "vc", "bt", "lens")]
    if op.startswith("tree"):
        args.append(a["masks"])
    args.append(F(a["scale"]))
    if op.endswith("fp8"):
        args += [F(a["ks"]), F(a["vs"])]
    args += [a[k] for k in ("window", "sinks", "S", "n", "H", "KH", "D", "BS", "P", "dtype", "stream", "MB", "NB",
                            "ws", "bytes")]
    return getattr(binding.lib(), "pa_decode_v2_" + op)(*args)


@pytest.mark.parametrize("op", ["window", "window_fp8", "tree", "tree_fp8"])
@pytest.mark.parametrize("kw,status", [
    (dict(sinks=-1), BAD), (dict(window=-1), BAD), (dict(n=0), BAD), (dict(n=513), BAD), (dict(H=3), BAD),
    (dict(H=4096, KH=2, n=64), BAD), (dict(D=72), UNS), (dict(BS=24), UNS), (dict(P=100), UNS), (dict(P=0), BAD),
    (dict(out=None), BAD), (dict(query=FAKE + 8), BAD), (dict(kc=None), BAD), (dict(lens=FAKE + 2), BAD),
    (dict(lse=FAKE + 2), BAD), (dict(scale=float("nan")), BAD), (dict(dtype=3), BAD), (dict(NB=0), BAD),
    (dict(MB=0), BAD), (dict(ws=FAKE + 8), BAD), (dict(bytes=256), WS), (dict(S=0), binding.PA_OK), (dict(S=-1), BAD),
])
def test_attention_refuses(op, kw, status):
    assert view(op, **kw) == status


def test_attention_refuses_of_one_call():
    assert view("window", window=0) == BAD
    assert view("tree", window=3) == BAD      # a window that does not hold the tree
    assert view("tree", masks=None) == BAD
    assert view("tree", masks=FAKE + 2) == BAD
    assert view("tree_fp8", ks=float("inf")) == BAD
    assert view("window_fp8", vs=float("nan")) == BAD
    assert view("window_fp8", dtype=2) == UNS
    assert view("window", dtype=2, D=256, BS=64) == UNS


def _align(x):
    return (x + 255) // 256 * 256


@pytest.mark.parametrize("S,n,H,KH,D,MB,BS,P,window,sinks", [
    (4, 1, 4, 4, 64, 100, 16, 512, 128, 4), (3, 7, 8, 2, 128, 4, 16, 64, 1000, 0), (2, 16, 8, 2, 128, 300, 32, 64, 0, 0),
    (5, 3, 6, 2, 96, 1000, 8, 64, 33, 9)])
def test_workspace_counts_the_visible_blocks(S, n, H, KH, D, MB, BS, P, window, sinks):
    # A window's rows look at window + n - 1 tokens, which touch at most one block more than they fill.
    blocks = min(MB, -(-sinks // BS) + -(-(window + n - 1) // BS) + 1) if window else MB
    pmax = -(-blocks * BS // P)
    m = 256
    l = _align(m + S * n * H * pmax * 4)
    o = _align(l + S * n * H * pmax * 4)
    want = _align(o + S * n * H * pmax * D * 4)
    assert binding.view_workspace_bytes(S, n, H, KH, D, MB, BS, P, window, sinks) == want
    for bad in ((S, 0), (S, 513), (-1, n)):
        assert binding.view_workspace_bytes(*bad, H, KH, D, MB, BS, P, window, sinks) == 0
    assert binding.view_workspace_bytes(S, n, H, KH, D, MB, BS, P, -1, sinks) == 0
    assert binding.view_workspace_bytes(S, n, H, KH, D, MB, BS, P, window, -1) == 0


def slots(**kw):
    a = dict(slots=FAKE, pos=FAKE * 2, seq=FAKE * 3, cu=FAKE * 4, bt=FAKE * 5, lens=FAKE * 6, new=FAKE * 7, S=3, N=10,
             MB=4, BS=16, stream=None, ws=FAKE * 8, bytes=256)
    a.update(kw)
    return binding.lib().pa_pages_slots(*[a[k] for k in ("slots", "pos", "seq", "cu", "bt", "lens", "new", "S", "N",
                                                         "MB", "BS", "stream", "ws", "bytes")])


@pytest.mark.parametrize("kw,status", [
    (dict(S=-1), BAD), (dict(N=-1), BAD), (dict(MB=0), BAD), (dict(BS=0), BAD), (dict(MB=1 << 28, BS=8), BAD),
    (dict(S=(1 << 24) + 1), BAD), (dict(slots=None), BAD), (dict(slots=FAKE + 4), BAD), (dict(pos=FAKE + 2), BAD),
    (dict(seq=FAKE * 3 + 1), BAD), (dict(cu=None), BAD), (dict(bt=None), BAD), (dict(lens=FAKE + 2), BAD),
    (dict(new=None), BAD), (dict(ws=None), BAD), (dict(ws=FAKE + 8), BAD), (dict(bytes=128), WS),
    (dict(pos=FAKE + 76), BAD), (dict(cu=FAKE * 7 + 8), BAD), (dict(slots=FAKE * 6), BAD), (dict(seq=FAKE * 2), BAD),
])
def test_slots_refuses(kw, status):
    assert slots(**kw) == status


def masks(**kw):
    a = dict(masks=FAKE, pos=FAKE * 2, par=FAKE * 3, lens=FAKE * 4, S=3, n=10, stream=None, ws=FAKE * 5, bytes=256)
    a.update(kw)
    return binding.lib().pa_tree_masks(*[a[k] for k in ("masks", "pos", "par", "lens", "S", "n", "stream", "ws",
                                                        "bytes")])


@pytest.mark.parametrize("kw,status", [
    (dict(S=-1), BAD), (dict(n=0), BAD), (dict(n=513), BAD), (dict(masks=None), BAD), (dict(masks=FAKE + 2), BAD),
    (dict(pos=FAKE + 2), BAD), (dict(par=None), BAD), (dict(lens=FAKE + 2), BAD), (dict(ws=None), BAD),
    (dict(bytes=255), WS), (dict(masks=FAKE * 3 + 4), BAD), (dict(pos=FAKE * 4 + 4), BAD),
])
def test_masks_refuses(kw, status):
    assert masks(**kw) == status


def write(**kw):
    a = dict(kc=FAKE, vc=FAKE, key=FAKE, value=FAKE, slots=FAKE, ks=1.0, vs=1.0, N=5, KH=2, D=64, BS=16, kst=128,
             vst=128, dtype=0, cdt=0, stream=None, NB=8, ws=FAKE, bytes=256)
    a.update(kw)
    return binding.lib().pa_cache_write(a["kc"], a["vc"], a["key"], a["value"], a["slots"], F(a["ks"]), F(a["vs"]),
                                        *[a[k] for k in ("N", "KH", "D", "BS", "kst", "vst", "dtype", "cdt", "stream",
                                                         "NB", "ws", "bytes")])


@pytest.mark.parametrize("kw,status", [
    (dict(N=-1), BAD), (dict(KH=0), BAD), (dict(NB=0), BAD), (dict(D=72), UNS), (dict(BS=12), UNS), (dict(dtype=3), BAD),
    (dict(cdt=1), BAD), (dict(cdt=2), BAD), (dict(cdt=4), BAD), (dict(ks=0.5), BAD), (dict(vs=2.0), BAD),
    (dict(cdt=3, ks=0.0), BAD), (dict(cdt=3, vs=float("nan")), BAD), (dict(cdt=3, ks=-1.0), BAD),
    (dict(cdt=3, ks=float("inf")), BAD), (dict(kst=120), BAD), (dict(vst=132), BAD), (dict(dtype=2, cdt=2, kst=130), BAD),
    (dict(kc=None), BAD), (dict(vc=FAKE + 8), BAD), (dict(key=None), BAD), (dict(value=FAKE + 8), BAD),
    (dict(slots=None), BAD), (dict(slots=FAKE + 4), BAD), (dict(ws=None), BAD), (dict(bytes=16), WS),
])
def test_write_refuses(kw, status):
    assert write(**kw) == status


def accept(**kw):
    a = dict(new=FAKE, k=[FAKE * 9], v=[FAKE * 10], bt=FAKE * 2, lens=FAKE * 3, acc=FAKE * 4, num=FAKE * 5, S=2, n=5, A=4,
             KH=2, D=64, BS=16, cdt=0, stream=None, MB=4, NB=8, ws=FAKE * 6, bytes=256)
    a.update(kw)
    k, v = ((ctypes.c_void_p * len(a[x]))(*a[x]) for x in "kv")
    if a.get("no_array"):
        k = None
    return binding.lib().pa_tree_accept(a["new"], k, v, a.get("nc", len(a["k"])), *[a[x] for x in (
        "bt", "lens", "acc", "num", "S", "n", "A", "KH", "D", "BS", "cdt", "stream", "MB", "NB", "ws", "bytes")])


@pytest.mark.parametrize("kw,status", [
    (dict(S=-1), BAD), (dict(n=0), BAD), (dict(n=513), BAD), (dict(A=-1), BAD), (dict(A=513), BAD), (dict(KH=0), BAD),
    (dict(D=72), UNS), (dict(BS=12), UNS), (dict(cdt=4), BAD), (dict(NB=0), BAD), (dict(MB=0), BAD),
    (dict(nc=-1), BAD), (dict(no_array=True), BAD), (dict(k=[None]), BAD), (dict(v=[FAKE + 8]), BAD),
    (dict(new=None), BAD), (dict(bt=FAKE + 2), BAD), (dict(lens=None), BAD), (dict(acc=None), BAD),
    (dict(num=FAKE + 1), BAD), (dict(new=FAKE * 3), BAD), (dict(new=FAKE * 5 + 4), BAD), (dict(ws=None), BAD),
    (dict(bytes=16), WS), (dict(S=0), binding.PA_OK),
])
def test_accept_refuses(kw, status):
    assert accept(**kw) == status
