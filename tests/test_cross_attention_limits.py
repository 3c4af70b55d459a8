"""Cross attention's limits on what it is given, on the host (no GPU is needed)."""
import numpy as np
import pytest

from audio_encoder_aut_b200 import _lib as A

P = 1 << 20  # an aligned address that is never read
MOST = 0x7ffff000


@pytest.mark.parametrize("rows,heads", [(MOST + 1, 1), ((1 << 31) - 17, 1), ((1 << 31) - 15, 1), ((1 << 31) - 1, 1), ((1 << 30) - 8, 2)])
def test_rows_near_2_31_are_refused(rows, heads):
    """A kernel counts a block's spare rows in 32 bits too: (rows + 255) / 256 must not pass them."""
    cu_q, cu_k = np.array([0, rows], np.int32), np.array([0, 0], np.int32)
    assert A.aut_cross_attention_workspace_bytes(heads, heads, 16, cu_q, cu_k) == 0
    assert A.aut_cross_attention(P, 16 * heads, None, 16 * heads, None, 16 * heads, P, 16 * heads, A.BF16, heads, heads, 16, cu_q, cu_k, None,
                                 1.0, P, 1 << 30, None, 0, 0) == A.AUT_ERR_UNSUPPORTED


def test_the_largest_row_count_is_planned():
    assert A.aut_cross_attention_workspace_bytes(1, 1, 16, np.array([0, MOST], np.int32), np.array([0, 0], np.int32)) >= 256


@pytest.mark.parametrize("far", [1 << 31, (1 << 32) + 100, -(1 << 32) + 100])
@pytest.mark.parametrize("make", [list, tuple, np.array])
def test_offsets_past_32_bits_are_refused(make, far):
    """Not wrapped to offsets that can be planned for."""
    size = A.aut_cross_attention_workspace_bytes
    ok, bad = [0, 100], make([0, far])
    assert size(4, 2, 64, ok, bad) == 0 and size(4, 2, 64, bad, ok) == 0
    for cu_q, cu_k in ((ok, bad), (bad, ok)):
        assert A.aut_cross_attention(P, 256, P, 128, P, 128, P, 256, A.BF16, 4, 2, 64, cu_q, cu_k, None, 0.125, P, 0, None, 0,
                                     0) == A.AUT_ERR_INVALID_ARG


def test_a_copy_is_left_out_of_prompts_only():
    arg = dict(q=P, ld_q=256, k=P, ld_k=128, v=P, ld_v=128, out=P, ld_out=256, dtype=A.BF16, heads_q=4, heads_kv=2, head_dim=64,
               cu_q=[0, 1], cu_k=[0, 500], key_mask=None, scale=0.125, workspace=P, ws_bytes=1 << 30, status=None, timeout_ms=0, stream=0)
    for flags in (A.CROSS_FAULT_K, A.CROSS_FAULT_V):
        assert A.aut_cross_attention_ex(**arg, flags=flags) == A.AUT_ERR_UNSUPPORTED
        assert A.aut_cross_attention_ex(**(arg | dict(cu_q=[0, 0])), flags=flags) == A.AUT_ERR_UNSUPPORTED
    for flags in (3, 4, -1):
        assert A.aut_cross_attention_ex(**arg, flags=flags) == A.AUT_ERR_INVALID_ARG


@pytest.mark.parametrize("scale,ok", [(3e38, False), (2.4e38, False), (2.3e38, True), (1e-45, True)])
def test_a_scale_that_overflows_in_base_2_is_refused(scale, ok):
    """scale log2(e) has to be finite in fp32: scores of zero would otherwise become NaN."""
    st = A.aut_cross_attention(P, 256, P, 128, P, 128, P, 256, A.BF16, 4, 2, 64, [0, 1], [0, 100], None, scale, P, 0, None, 0, 0)
    assert st == (A.AUT_ERR_WORKSPACE if ok else A.AUT_ERR_INVALID_ARG)
