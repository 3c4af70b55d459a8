"""Cross attention on the GPU: how finely the softmax's weights are held."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from audio_encoder_aut_b200 import _lib as A  # noqa: E402

CODE = {torch.bfloat16: A.BF16, torch.float16: A.F16}


def _attend(q, kv, heads, hd, scale):
    """Every query over all keys, one request, every head with keys of its own."""
    nq, nk, w = q.shape[0], kv.shape[0], heads * hd
    out = torch.empty_like(q)
    cu_q, cu_k = np.array([0, nq], np.int32), np.array([0, nk], np.int32)
    ws = torch.empty(A.aut_cross_attention_workspace_bytes(heads, heads, hd, cu_q, cu_k), dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert A.aut_cross_attention(q.data_ptr(), w, kv.data_ptr(), 2 * w, kv.data_ptr() + 2 * w, 2 * w, out.data_ptr(), w, CODE[q.dtype], heads,
                                 heads, hd, cu_q, cu_k, None, scale, ws.data_ptr(), ws.numel(), status.data_ptr(), 0,
                                 torch.cuda.current_stream().cuda_stream) == A.AUT_OK
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    return out


@pytest.mark.parametrize("hd", [16, 64, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("nq,nk", [(1, 3000), (300, 3000), (1, 60000), (700, 60000)])
def test_many_small_weights_count(nq, nk, dtype, hd):
    """One key of every 16 has the row's maximum and a value of zero, the others weights of e^-17.75, below half of
    fp16's smallest step, and values of 4096: the result is theirs alone, whichever keys a warp or split takes."""
    q = torch.zeros(nq, hd, device="cuda", dtype=dtype)
    q[:, 0] = 1
    kv = torch.zeros(nk, 2 * hd, device="cuda", dtype=dtype)
    kv[:, 0] = -17.75
    kv[:, hd:] = 4096
    kv[::16] = 0
    out = _attend(q, kv, 1, hd, 1.0)
    few, p = len(range(0, nk, 16)), math.exp(-17.75)
    total = few + (nk - few) * p
    want = (nk - few) * p * 4096 / total
    # Half a step for every weight and for the output; a weight's exponent, 25.6, off by 3 steps of fp32 (product, sum and
    # exponential), the sums by nk; fp16: half a step of 2^-24 under the lift of 2^7, for every weight.
    u = torch.finfo(dtype).eps / 2
    tol = want * (2 * u + 3 * 26 * 2.0 ** -24 + 2 * nk * 2.0 ** -24)
    if dtype == torch.float16:
        tol += 2.0 ** -32 * (nk - few) * 4096 / total + 2.0 ** -25
    assert (out.double() - want).abs().max().item() <= tol, (out[0, 0].item(), out[-1, 0].item(), want, tol)
