"""The decoder-side operators refuse bad arguments on the host, before anything
touches a GPU (none is needed), and the workspace helper plans without one."""
import ctypes

import numpy as np
import pytest

from audio_encoder_aut_b200 import _lib as A

P = 1 << 20  # an aligned address that is never read
BAD, UNS, WS = A.AUT_ERR_INVALID_ARG, A.AUT_ERR_UNSUPPORTED, A.AUT_ERR_WORKSPACE


@pytest.mark.parametrize("over,want", [
    (dict(dtype=3), BAD), (dict(dtype=-1), BAD), (dict(M=-1), BAD), (dict(K=0), BAD), (dict(K=24), UNS), (dict(K=131088), UNS),
    (dict(M=(1 << 31) - 1), UNS), (dict(x=None), BAD), (dict(q=None), BAD), (dict(scale=None), BAD), (dict(x=P + 8), BAD), (dict(q=P + 8), BAD),
    (dict(scale=P + 2), BAD), (dict(ld_x=48), BAD), (dict(ld_x=68), BAD), (dict(ld_x=1 << 41), BAD), (dict(M=0, x=None), A.AUT_OK)])
def test_quantize_rows_refuses(over, want):
    arg = dict(x=P, dtype=A.BF16, ld_x=64, M=4, K=64, q=P, scale=P, stream=0) | over
    assert A.aut_quantize_rows(**arg) == want


@pytest.mark.parametrize("M", [4, 400])
@pytest.mark.parametrize("over,want", [
    (dict(N=24), UNS), (dict(K=40), UNS), (dict(K=131088), UNS), (dict(M=(1 << 31) - 1), UNS), (dict(N=0), BAD), (dict(K=-16), BAD), (dict(epilogue=4), BAD),
    (dict(epilogue=-1), BAD), (dict(timeout_ms=-1), BAD), (dict(flags=A.LINEAR_F16), BAD), (dict(flags=8), BAD), (dict(xq=None), BAD),
    (dict(x_scale=None), BAD), (dict(wq=None), BAD), (dict(w_scale=None), BAD), (dict(y=None), BAD), (dict(xq=P + 8), BAD),
    (dict(wq=P + 4), BAD), (dict(w_scale=P + 4), BAD), (dict(x_scale=P + 1), BAD), (dict(bias=P + 2), BAD), (dict(y=P + 8), BAD)])
def test_linear_i8_refuses(over, want, M):
    arg = dict(xq=P, x_scale=P, wq=P, w_scale=P, bias=None, y=P, M=M, N=64, K=64, epilogue=0, status=None, timeout_ms=0, flags=0,
               stream=0) | over
    assert A.aut_linear_i8(**arg) == want


def test_linear_i8_few_rows_has_no_wait_to_inject_into():
    assert A.aut_linear_i8(P, P, P, P, None, P, 4, 64, 64, 0, None, 0, A.LINEAR_FAULT_INJECT, 0) == UNS
    assert A.aut_linear_i8(None, None, None, None, None, None, 0, 64, 64, 0, None, 0, 0, 0) == A.AUT_OK


def _rows(**over):
    return A.aut_head_rows(**(dict(x=P, ld_x=128, y=P, ld_y=128, gamma=P, positions=P, rows=3, heads=2) | over))


@pytest.mark.parametrize("over,want", [
    (dict(rows=-1), BAD), (dict(heads=0), BAD), (dict(heads=1 << 20), BAD), (dict(x=None), BAD), (dict(y=None), BAD), (dict(x=P + 2), BAD),
    (dict(y=P + 8), BAD), (dict(gamma=P + 2), BAD), (dict(positions=P + 2), BAD), (dict(ld_x=120), BAD), (dict(ld_y=64), BAD),
    (dict(ld_x=132), BAD), (dict(rows=0, x=None, y=None), A.AUT_OK), (dict(ld_y=1 << 41), BAD)])
def test_norm_rope_refuses_a_side(over, want):
    side = _rows(**over)
    none = _rows(rows=0)
    assert A.aut_qk_norm_rope(side, None, 64, 0, 0, 64, 1e4, False, 1e-6, 0) == want
    assert A.aut_qk_norm_rope(none, side, 64, 0, 0, 64, 1e4, False, 1e-6, 0) == want


@pytest.mark.parametrize("over,want", [
    (dict(head_dim=80), UNS), (dict(head_dim=512), UNS), (dict(rot_dim=24), UNS), (dict(rot_dim=-16), BAD), (dict(rot_dim=80), BAD),
    (dict(theta=0.5), BAD), (dict(theta=float("nan")), BAD), (dict(theta=float("inf")), BAD), (dict(eps=-1.0), BAD),
    (dict(eps=float("nan")), BAD), (dict(eps=float("inf")), BAD), (dict(x_dtype=3), BAD), (dict(y_dtype=-1), BAD)])
def test_norm_rope_refuses(over, want):
    arg = dict(q=_rows(), k=_rows(), head_dim=64, x_dtype=0, y_dtype=0, rot_dim=64, theta=1e4, interleaved=False, eps=1e-6, stream=0) | over
    assert A.aut_qk_norm_rope(**arg) == want


def test_norm_rope_nothing_to_do():
    assert A.aut_qk_norm_rope(None, None, 64, 0, 0, 64, 1e4, False, 1e-6, 0) == A.AUT_OK


@pytest.mark.parametrize("over,want", [
    (dict(heads_q=0), BAD), (dict(heads_q=5), BAD), (dict(heads_kv=0), BAD), (dict(head_dim=96), UNS), (dict(head_dim=256), UNS),
    (dict(heads_q=1 << 20), UNS), (dict(dtype=A.F32), BAD), (dict(dtype=7), BAD), (dict(scale=0.0), BAD), (dict(scale=-1.0), BAD),
    (dict(scale=float("inf")), BAD), (dict(scale=float("nan")), BAD), (dict(timeout_ms=-1), BAD), (dict(cu_q=[1, 3, 9]), BAD),
    (dict(cu_k=[2, 5, 5]), BAD), (dict(cu_q=[0, 4, 3]), BAD), (dict(cu_k=[0, 9, 3]), BAD), (dict(cu_q=[0, 4]), BAD), (dict(cu_q=[]), BAD),
    (dict(cu_q=[0, 3, 1 << 30]), UNS), (dict(cu_k=[0, 3, (1 << 31) - 1]), UNS), (dict(q=None), BAD), (dict(k=None), BAD), (dict(v=None), BAD), (dict(out=None), BAD),
    (dict(q=P + 8), BAD), (dict(k=P + 2), BAD), (dict(v=P + 8), BAD), (dict(out=P + 4), BAD), (dict(ld_q=248), BAD), (dict(ld_k=120), BAD),
    (dict(ld_v=64), BAD), (dict(ld_out=255), BAD), (dict(ld_q=260), BAD), (dict(ld_k=132), BAD), (dict(ld_q=1 << 39), BAD),
    (dict(workspace=None), BAD), (dict(workspace=P + 128), BAD), (dict(ws_bytes=0), WS), (dict(status=P + 2), BAD)])
def test_cross_attention_refuses(over, want):
    arg = dict(q=P, ld_q=256, k=P, ld_k=128, v=P, ld_v=128, out=P, ld_out=256, dtype=A.BF16, heads_q=4, heads_kv=2, head_dim=64,
               cu_q=[0, 3, 9], cu_k=[0, 5, 5], key_mask=None, scale=0.125, workspace=P, ws_bytes=1 << 30, status=None, timeout_ms=0,
               stream=0) | over
    assert A.aut_cross_attention(**arg) == want


def test_cross_attention_workspace():
    size = A.aut_cross_attention_workspace_bytes
    assert size(4, 2, 64, [0, 1], [0, 100]) >= 256
    long = size(4, 2, 128, [0, 1], [0, 100_000])  # split: at least the partial rows of 2 splits
    assert long >= 2 * 4 * 128 * 4
    need = dict(q=P, ld_q=512, k=P, ld_k=256, v=P, ld_v=256, out=P, ld_out=512, dtype=A.BF16, heads_q=4, heads_kv=2, head_dim=128,
                cu_q=[0, 1], cu_k=[0, 100_000], key_mask=None, scale=0.125, workspace=P, status=None, timeout_ms=0, stream=0)
    assert A.aut_cross_attention(ws_bytes=long - 1, **need) == WS
    assert size(4, 3, 64, [0, 1], [0, 100]) == 0
    assert size(4, 2, 48, [0, 1], [0, 100]) == 0
    assert size(4, 2, 64, [0, 2, 1], [0, 1, 1]) == 0
    many = np.arange(2001, dtype=np.int32)
    assert size(4, 2, 64, many, many) > size(4, 2, 64, many[:100], many[:100])
    assert A.lib().aut_cross_attention_workspace_bytes(4, 2, 64, None, None, 1) == 0
    none = (ctypes.c_int32 * 1)(0)
    assert A.lib().aut_cross_attention_workspace_bytes(4, 2, 64, none, none, 0) >= 256


def test_cross_attention_without_queries_launches_nothing():
    assert A.aut_cross_attention(None, 0, P, 128, P, 128, None, 0, A.BF16, 4, 2, 64, [0, 0], [0, 5], None, 1.0, P, 256, None, 0, 0) == A.AUT_OK
