"""pa_decode_v2_view_ex refuses bad arguments before it touches the GPU."""
import ctypes

import pytest

from decode_attention_paged_pa_gb300 import binding

FAKE = 0x100000  # an aligned non-null address; never dereferenced by these calls
BAD, UNS, WS = binding.PA_ERR_INVALID_ARG, binding.PA_ERR_UNSUPPORTED, binding.PA_ERR_WORKSPACE
F = ctypes.c_float


def view_ex(**kw):
    a = dict(out=FAKE, lse=None, query=FAKE, kc=FAKE, vc=FAKE, bt=FAKE, lens=FAKE, masks=FAKE, scale=0.125, ks=1.0, vs=1.0,
             window=16, sinks=4, S=2, n=4, H=4, KH=2, D=128, BS=16, P=512, dtype=0, tree=1, fp8=0, stream=None, MB=4, NB=8,
             ws=FAKE, bytes=1 << 30, max_ctas=0, timeout_ns=0)
    a.update(kw)
    for k in ("scale", "ks", "vs"):
        a[k] = F(a[k])
    return binding.lib().pa_decode_v2_view_ex(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(max_ctas=-1), BAD), (dict(timeout_ns=-1), BAD), (dict(ks=0.5), BAD), (dict(vs=2.0), BAD),
    (dict(fp8=1, ks=float("inf")), BAD), (dict(masks=None), BAD), (dict(masks=FAKE + 2), BAD), (dict(window=3), BAD),
    (dict(tree=0, window=0), BAD), (dict(tree=0, sinks=-1), BAD), (dict(fp8=1, dtype=2), UNS), (dict(D=72), UNS),
    (dict(H=3, n=2), BAD), (dict(H=3, n=2, tree=0), BAD), (dict(bytes=256), WS), (dict(out=None), BAD),
    (dict(S=0), binding.PA_OK), (dict(S=0, tree=0, masks=None), binding.PA_OK),
])
def test_view_ex_refuses(kw, status):
    assert view_ex(**kw) == status
