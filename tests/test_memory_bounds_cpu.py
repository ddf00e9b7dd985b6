"""What a workspace query says of a call that is refused, and arguments that only the
header has spoken of (no GPU needed)."""
import math
import os

import pytest

from gemm_decode_q1_amd import q1 as B
from test_memory_refusals_cpu import FAKE, kv, query, said, scan

pytestmark = pytest.mark.skipif(not os.path.exists(B.LIB_PATH), reason="libq1.so not built")


@pytest.mark.parametrize("scale", [math.inf, -math.inf, math.nan])
def test_attention_scale_is_finite(scale):
    L = B.load_library()
    assert L.q1_kv_attn(kv(), query(scale=scale), FAKE, 1 << 40, None) == -1 and "scale" in said()
    assert L.q1_kv_attn_workspace_bytes(kv(), query(scale=scale)) == 0 and "scale" in said()
    for fine in (0.0, -0.0, -2.5, 1e-45, 3.4e38):
        assert L.q1_kv_attn(kv(), query(scale=fine, q=None), FAKE, 1 << 40, None) == -1 and "NULL" in said()


def test_workspace_of_a_refused_scan():
    """Calls that are too large have no size to allocate first."""
    L = B.load_library()
    wide = dict(Di=1 << 18, x_ld=1 << 18, dt_ld=1 << 18, z_ld=1 << 18)
    for tokens, nseq, kw in (((1 << 31) - 1, 4, dict(Di=1 << 12, x_ld=1 << 12, dt_ld=1 << 12, z_ld=1 << 12)),
                             (10, 1 << 20, dict(slots=1 << 20, Di=128, N=64, x_ld=128, dt_ld=128, z_ld=128, b_ld=64, c_ld=64))):
        assert L.q1_scan_prefill(scan(**kw), tokens, nseq, FAKE, FAKE, 1 << 50, None) == -2 and "too large" in said()
        assert L.q1_scan_prefill_workspace_bytes(scan(**kw), tokens, nseq) == 0 and "too large" in said()
    assert L.q1_scan_prefill_workspace_bytes(scan(**wide), 1 << 18, 1) > 0 and said() == ""


def test_workspace_of_a_refused_attention():
    L = B.load_library()
    c = kv(pages=1 << 20, page_size=16, Hkv=64, D=64)
    a = dict(B=1 << 18, max_pages=1 << 20, Hq=64, q_ld=64 * 64)
    assert L.q1_kv_attn(c, query(**a), FAKE, 1 << 50, None) == -2 and "too large" in said()
    assert L.q1_kv_attn_workspace_bytes(c, query(**a)) == 0 and "too large" in said()


@pytest.mark.parametrize("tokens,nseq,Di", [(16895, 512, 512), (16384 + 255, 256, 1024), (8480, 61, 5120), (1 << 20, 5000, 64)])
def test_a_long_sequence_among_many_is_cut(tokens, nseq, Di):
    """Whatever the batch, a piece of a prompt's scan has at most 512 tokens: one sequence that has nearly all
    tokens would else be left to few workgroups.  The workspace has N + 1 numbers for each channel of each piece."""
    kw = dict(Di=Di, x_ld=Di, dt_ld=Di, z_ld=Di, slots=nseq)
    got = B.load_library().q1_scan_prefill_workspace_bytes(scan(**kw), tokens, nseq)
    assert got >= (tokens // 512 + nseq) * Di * 17 * 4


def test_pieces_of_a_small_batch():
    """Sequences that fill the chip but have few tokens are cut as a single one is, not less."""
    L = B.load_library()
    for tokens, most in ((400, 64), (1000, 128), (3000, 384)):
        kw = dict(Di=5120, x_ld=5120, dt_ld=5120, z_ld=5120, slots=64)
        assert L.q1_scan_prefill_workspace_bytes(scan(**kw), tokens, 64) >= (tokens // most + 64) * 5120 * 17 * 4
