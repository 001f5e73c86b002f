"""Multi-query calls refuse heads that are not whole groups of the kv heads, also where
their rows would be (three heads over two kv heads, two rows of each)."""
import ctypes

import pytest

from decode_attention_paged_pa_gb300 import binding

FAKE = 0x100000  # an aligned non-null address; never dereferenced: every call is refused
F = ctypes.c_float


@pytest.mark.parametrize("H,KH,n", [(3, 2, 2), (6, 4, 2), (2, 4, 2), (10, 4, 4), (1, 2, 2)])
@pytest.mark.parametrize("op", ["mq", "mq_fp8", "mq_kv4"])
def test_heads_are_whole_groups(op, H, KH, n):
    caches = [FAKE] if op == "mq_kv4" else [FAKE, FAKE]
    scales = [F(1.0), F(1.0)] if op == "mq_fp8" else []
    fn = getattr(binding.lib(), "pa_decode_v2_" + op)
    assert fn(FAKE, None, FAKE, *caches, FAKE, FAKE, F(0.1), *scales, 2, n, H, KH, 128, 16, 512, 0, None, 4, 8, FAKE,
              1 << 30) == binding.PA_ERR_INVALID_ARG
