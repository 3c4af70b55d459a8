"""Cross attention's prompt kernel when a copy never arrives: its waits run out, it says so and the GPU stays usable."""
import math

import numpy as np
import pytest

import decoder_ops_ref as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from audio_encoder_aut_b200 import _lib as A  # noqa: E402


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("flag", [A.CROSS_FAULT_K, A.CROSS_FAULT_V], ids=["first_k", "first_v"])
@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("nq,nk", [(8001, 100), (4000, 700), (1500, 3000), (900, 20000)])  # one tile of keys, a few, more than the ring, split
def test_a_copy_that_never_arrives(nq, nk, masked, flag, hd):
    heads = 2
    g = torch.Generator(device="cuda")
    g.manual_seed(nk)
    q = torch.randn(nq, heads * hd, device="cuda", generator=g).bfloat16()
    kv = torch.randn(nk, 2 * hd, device="cuda", generator=g).bfloat16()
    mask = (torch.rand(nk, device="cuda", generator=g) < 0.8).to(torch.uint8) if masked else None
    cu_q, cu_k = np.array([0, nq], np.int32), np.array([0, nk], np.int32)
    ws = torch.zeros(A.aut_cross_attention_workspace_bytes(heads, 1, hd, cu_q, cu_k), dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((nq + 1, heads * hd), 7.0, dtype=torch.bfloat16, device="cuda")

    def call(flags, timeout_ms):
        return A.aut_cross_attention_ex(q.data_ptr(), heads * hd, kv.data_ptr(), 2 * hd, kv.data_ptr() + 2 * hd, 2 * hd, out.data_ptr(),
                                        heads * hd, A.BF16, heads, 1, hd, cu_q, cu_k, None if mask is None else mask.data_ptr(),
                                        1 / math.sqrt(hd), ws.data_ptr(), ws.numel(), status.data_ptr(), timeout_ms, flags,
                                        torch.cuda.current_stream().cuda_stream)

    assert call(flag, 20) == A.AUT_OK
    torch.cuda.synchronize()
    assert A.aut_check_status_word(status.data_ptr()) == A.AUT_ERR_TIMEOUT
    assert (out[nq] == 7).all()
    assert call(0, 0) == A.AUT_OK
    torch.cuda.synchronize()
    assert A.aut_check_status_word(status.data_ptr()) == A.AUT_OK
    kn = kv.double().cpu().numpy()
    ref, tol = R.cross_attention(q.double().cpu().numpy(), kn[:, :hd], kn[:, hd:], cu_q, cu_k, heads, 1, hd,
                                 None if mask is None else mask.cpu().numpy(), 1 / math.sqrt(hd), "bf16")
    got = out[:nq].double().cpu().numpy()
    assert (np.abs(got - ref) <= tol).all()
