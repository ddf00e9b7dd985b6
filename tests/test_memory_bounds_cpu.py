"""What a workspace query says of a call that is refused, and arguments that only the
header has spoken of (no GPU needed)."""
import math
import os

import pytest

from gemm_decode_q1_amd import q1 as B
from test_memory_refusals_cpu import FAKE, kv, query, said

pytestmark = pytest.mark.skipif(not os.path.exists(B.LIB_PATH), reason="libq1.so not built")


@pytest.mark.parametrize("scale", [math.inf, -math.inf, math.nan])
def test_attention_scale_is_finite(scale):
    L = B.load_library()
    assert L.q1_kv_attn(kv(), query(scale=scale), FAKE, 1 << 40, None) == -1 and "scale" in said()
    assert L.q1_kv_attn_workspace_bytes(kv(), query(scale=scale)) == 0 and "scale" in said()
    for fine in (0.0, -0.0, -2.5, 1e-45, 3.4e38):
        assert L.q1_kv_attn(kv(), query(scale=fine, q=None), FAKE, 1 << 40, None) == -1 and "NULL" in said()
