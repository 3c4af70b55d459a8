"""The 8-bit linear layer's longest exact sums with -128 among the operands."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from audio_encoder_aut_b200 import _lib as A  # noqa: E402


@pytest.mark.parametrize("M", [3, 40])
@pytest.mark.parametrize("K,x,w", [(131056, -128, -128), (131056, -128, 127), (131072, -128, 127), (131072, 127, -128), (131072, -127, -127)])
def test_longest_sums_with_the_lowest_byte(K, x, w, M):
    """2^14 K stays below 2^31 up to K = 131056; at 131072 only -128 times -128 all along would not."""
    N = 16
    xq = torch.full((M, K), x, dtype=torch.int8, device="cuda")
    wq = torch.full((N, K), w, dtype=torch.int8, device="cuda")
    one = torch.ones(max(M, N), device="cuda")
    y = torch.empty(M, N, device="cuda")
    assert A.aut_linear_i8(xq.data_ptr(), one.data_ptr(), wq.data_ptr(), one.data_ptr(), None, y.data_ptr(), M, N, K, A.EPI_F32, None, 0, 0,
                           torch.cuda.current_stream().cuda_stream) == A.AUT_OK
    torch.cuda.synchronize()
    assert (y.double() - x * w * K).abs().max().item() <= abs(x * w * K) * 2.0 ** -24
