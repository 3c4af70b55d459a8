"""The decoder-side operators on the GPU, through the C ABI, against their
definitions in 64 bits (decoder_ops_ref): 8-bit linear layers, head norms with
rotation, cross attention; alone, captured, on other streams and in a row."""
import itertools
import math

import numpy as np
import pytest

import aut_synth as S
import decoder_ops_ref as R
import oracle as O
from gpu_util import assert_rows_close

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from audio_encoder_aut_b200 import _lib as A  # noqa: E402

TORCH = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
CODE = {"bf16": A.BF16, "f16": A.F16, "f32": A.F32}


def _stream():
    return torch.cuda.current_stream().cuda_stream


def _draw(shape, dtype, seed, scale=1.0):
    g = np.random.default_rng(seed)
    return torch.from_numpy(g.standard_normal(shape).astype(np.float32) * np.float32(scale)).to(TORCH[dtype]).cuda()


def _np(t):
    return t.detach().double().cpu().numpy()


# ------------------------------------------------------------------ quantise

def _quantize(x, dtype, ld, M, K):
    q = torch.full((M, K), 99, dtype=torch.int8, device="cuda")
    s = torch.full((M,), -1.0, device="cuda")
    assert A.aut_quantize_rows(x.data_ptr(), CODE[dtype], ld, M, K, q.data_ptr(), s.data_ptr(), _stream()) == A.AUT_OK
    torch.cuda.synchronize()
    return q, s


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,K", [(1, 16), (1, 2048), (7, 1040), (1500, 80), (1187, 2048), (1201, 2064), (3, 16384), (2, 16400), (2, 40000)])
def test_quantize_rows_is_exact(M, K, dtype):
    x = _draw((M, K), dtype, M + K)
    if M > 2:
        x[1] = 0
        x[2] = torch.arange(K, device="cuda").to(x.dtype) % 128 - 63.5  # many halves: ties to even
    q, s = _quantize(x, dtype, K, M, K)
    rq, rs = R.quantize(x.float().cpu().numpy())
    np.testing.assert_array_equal(s.cpu().numpy(), rs)
    np.testing.assert_array_equal(q.cpu().numpy(), rq)


def test_quantize_rows_ties_and_tiny_scales():
    """Scale a power of two and every quotient on a rounding border; denormal rows."""
    K = 256
    x = np.zeros((4, K), np.float32)
    x[0] = np.arange(K) / 2 - 63.5
    x[0, 0] = 127
    x[1] = 1e-40 * np.arange(K)
    x[2, 3] = 1e-45
    x[3] = 3e38 * np.linspace(-1, 1, K)
    q, s = _quantize(torch.from_numpy(x).cuda(), "f32", K, 4, K)
    rq, rs = R.quantize(x)
    np.testing.assert_array_equal(s.cpu().numpy(), rs)
    np.testing.assert_array_equal(q.cpu().numpy(), rq)


@pytest.mark.parametrize("M", [2, 1300])
def test_quantize_rows_strided_and_not_finite(M):
    K, ld = 96, 104
    buf = _draw((M, ld), "bf16", 3)
    buf[:, K:] = 1e30  # between the rows: never read
    buf[0, 5], buf[1, 7] = float("inf"), float("nan")
    q, s = _quantize(buf, "bf16", ld, M, K)
    assert math.isinf(s[0].item()) and math.isnan(s[1].item())
    assert not q[:2].any()
    if M > 2:
        rq, rs = R.quantize(buf[2:, :K].float().cpu().numpy())
        np.testing.assert_array_equal(q[2:].cpu().numpy(), rq)
        np.testing.assert_array_equal(s[2:].cpu().numpy(), rs)


# --------------------------------------------------------------- 8-bit linear

EPIS = {"bf16": A.EPI_BF16, "gelu": A.EPI_BF16_GELU, "resid": A.EPI_RESID_F32, "f32": A.EPI_F32}


def _i8(M, N, K, epi, bias=True, flags=0, seed=0):
    g = np.random.default_rng(seed + M * 7 + N + K)
    xq = g.integers(-127, 128, (M, K)).astype(np.int8)
    wq = g.integers(-127, 128, (N, K)).astype(np.int8)
    sx = (g.uniform(0.2, 1, M) / (40 * math.sqrt(K))).astype(np.float32)
    sw = (g.uniform(0.2, 1, N) / 40).astype(np.float32)
    b = S.round_bf16(g.standard_normal(N).astype(np.float32)) if bias else None
    y0 = g.standard_normal((M, N)).astype(np.float32)
    ref, tol = R.linear_i8(xq, sx, wq, sw, b)
    dev = [torch.from_numpy(t).cuda() for t in (xq, sx, wq, sw)]
    bd = torch.from_numpy(b).cuda().to(torch.bfloat16) if bias else None
    rows = M + 3  # three rows behind the last: left alone
    if epi in ("resid", "f32"):
        y = torch.full((rows, N), 7.0, device="cuda")
        if epi == "resid":
            y[:M] = torch.from_numpy(y0).cuda()
            # acc + (x + b): the inner sum is rounded too
            tol = tol + R.U32 * (np.abs(y0 + (0 if b is None else b)) + np.abs(ref + y0))
            ref = ref + y0
        tol = tol + 1e-30
    else:
        y = torch.full((rows, N), 7.0, device="cuda", dtype=torch.bfloat16)
        if epi == "gelu":
            ref, tol = O.gelu(ref), 1.13 * tol + 6e-7  # GELU' < 1.13; the kernel's GELU is within 5e-7
        tol = tol * (1 + R.HALF["bf16"]) + R.HALF["bf16"] * np.abs(ref)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    st = A.aut_linear_i8(*[t.data_ptr() for t in dev], bd.data_ptr() if bias else None, y.data_ptr(), M, N, K, EPIS[epi],
                         status.data_ptr(), 0, flags, _stream())
    assert st == A.AUT_OK
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    got = _np(y)
    assert (got[M:] == 7).all()
    excess = np.abs(got[:M] - ref) - tol
    i = np.unravel_index(int(excess.argmax()), excess.shape)
    assert excess.max() <= 0, (i, got[i], ref[i], tol[i])


I8_SHAPES = [(1, 16, 16), (1, 2048, 2048), (5, 48, 80), (8, 1024, 4096), (9, 32, 1040), (16, 240, 64), (17, 64, 144), (32, 512, 5120),
             (33, 16, 16), (33, 48, 80), (77, 240, 144), (128, 256, 128), (129, 96, 272), (300, 1280, 1280), (390, 2048, 1024),
             (1000, 32, 896), (2600, 2048, 208), (4000, 5120, 256)]


@pytest.mark.parametrize("epi", list(EPIS))
@pytest.mark.parametrize("M,N,K", I8_SHAPES)
def test_linear_i8_matches_definition(M, N, K, epi):
    _i8(M, N, K, epi)


@pytest.mark.parametrize("M,N,K,flags", [(4, 64, 64, 0), (300, 256, 256, A.LINEAR_SINGLE_CTA), (4000, 1280, 144, A.LINEAR_SINGLE_CTA),
                                         (600, 128, 16, 0)])
def test_linear_i8_without_bias_and_on_single_ctas(M, N, K, flags):
    for epi in ("bf16", "resid"):
        _i8(M, N, K, epi, bias=False, flags=flags)


@pytest.mark.parametrize("M", [3, 40])
def test_linear_i8_longest_sum(M):
    """K at its limit and every product 127^2: the int32 sum is near 2^31."""
    K, N = 131072, 16
    xq = torch.full((M, K), 127, dtype=torch.int8, device="cuda")
    wq = torch.full((N, K), 127, dtype=torch.int8, device="cuda")
    wq[1] = -127
    one = torch.ones(max(M, N), device="cuda")
    y = torch.empty(M, N, device="cuda")
    assert A.aut_linear_i8(xq.data_ptr(), one.data_ptr(), wq.data_ptr(), one.data_ptr(), None, y.data_ptr(), M, N, K, A.EPI_F32, None, 0,
                           0, _stream()) == A.AUT_OK
    torch.cuda.synchronize()
    want = np.full((M, N), 127.0 * 127 * K)
    want[:, 1] *= -1
    assert np.abs(_np(y) - want).max() <= 127.0 * 127 * K * R.U32


@pytest.mark.parametrize("flags", [0, A.LINEAR_SINGLE_CTA], ids=["auto", "single_cta"])
def test_linear_i8_wait_that_runs_out_is_reported(flags):
    """The first block leaves its first operand load out: the kernel gives up after
    its time limit, says so in the status word and leaves the GPU usable."""
    M, N, K = 512, 256, 256
    x = torch.ones(M, K, dtype=torch.int8, device="cuda")
    w = torch.ones(N, K, dtype=torch.int8, device="cuda")
    one = torch.ones(M, device="cuda")
    y = torch.zeros(M, N, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def call(extra):
        return A.aut_linear_i8(x.data_ptr(), one.data_ptr(), w.data_ptr(), one.data_ptr(), None, y.data_ptr(), M, N, K, A.EPI_F32,
                               status.data_ptr(), 20, flags | extra, _stream())
    assert call(A.LINEAR_FAULT_INJECT) == A.AUT_OK
    torch.cuda.synchronize()
    assert A.aut_check_status_word(status.data_ptr()) == A.AUT_ERR_TIMEOUT
    assert call(0) == A.AUT_OK
    torch.cuda.synchronize()
    assert A.aut_check_status_word(status.data_ptr()) == A.AUT_OK
    assert (y == K).all()


def test_linear_i8_spoilt_row_is_nan_alone():
    M, N, K = 40, 32, 64
    x = _draw((M, K), "f32", 1)
    x[3, 2] = float("nan")
    x[7, 1] = float("-inf")
    q, s = _quantize(x, "f32", K, M, K)
    w, sw = _quantize(_draw((N, K), "f32", 2), "f32", K, N, K)
    y = torch.empty(M, N, device="cuda")
    assert A.aut_linear_i8(q.data_ptr(), s.data_ptr(), w.data_ptr(), sw.data_ptr(), None, y.data_ptr(), M, N, K, A.EPI_F32, None, 0, 0,
                           _stream()) == A.AUT_OK
    torch.cuda.synchronize()
    bad = torch.isnan(y).all(1).cpu().numpy()
    assert list(np.flatnonzero(bad)) == [3, 7] and not torch.isnan(y[[0, 39]]).any()


# ------------------------------------------------------------ norm and rotation

def _norm_rope_case(Tq, Tk, hq, hk, hd, rot, x, y, theta, inter, gamma, pos0, pad=0, seed=0):
    sides, refs = [], []
    for n, T, heads in (("q", Tq, hq), ("k", Tk, hk)):
        buf = _draw((max(T, 1), heads * hd + pad), x, seed + len(sides), 2.0)
        out = torch.full((max(T, 1) + 2, heads * hd + 2 * pad), 7.0, dtype=TORCH[y], device="cuda")
        gm = (1 + 0.3 * _draw((hd,), "f32", 5 + seed)).to(torch.bfloat16) if gamma else None
        pos = torch.arange(T, dtype=torch.int32, device="cuda") * 3 + pos0 if pos0 is not None else None
        sides.append(A.aut_head_rows(buf.data_ptr(), buf.shape[1], out.data_ptr(), out.shape[1], gm.data_ptr() if gamma else None,
                                     pos.data_ptr() if pos0 is not None else None, T, heads))
        refs.append((buf, out, gm, pos, T, heads))
    st = A.aut_qk_norm_rope(sides[0], sides[1], hd, CODE[x], CODE[y], rot, theta, inter, 1e-6, _stream())
    assert st == A.AUT_OK
    torch.cuda.synchronize()
    for buf, out, gm, pos, T, heads in refs:
        got = _np(out)
        assert (got[T:] == 7).all() and (got[:, heads * hd:] == 7).all()
        if T == 0:
            continue
        xin = _np(buf)[:T, :heads * hd].reshape(T, heads, hd)
        ref, norm = R.norm_rope(xin, None if gm is None else _np(gm), None if pos is None else pos.cpu().numpy(), hd, rot, theta, inter,
                                1e-6)
        ref, norm = ref.reshape(T, -1), norm.reshape(T, -1)
        # fp32 steps: 16.5 half steps for the norm (20 in the sum count half, rsqrt 4, two products), the sine's and
        # cosine's 7.15 times |a| + |b| <= 1.42 pair norms, three in the rotation: under 32 in all.
        tol = 32 * R.U32 * norm * (1 + R.HALF[y]) + R.HALF[y] * np.abs(ref) + R.TINY[y] + 1e-30
        excess = np.abs(got[:T, :heads * hd] - ref) - tol
        i = np.unravel_index(int(excess.argmax()), excess.shape)
        assert excess.max() <= 0, (i, got[i], ref[i], tol[i])


@pytest.mark.parametrize("hd", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("Tq,Tk,hq,hk", [(1, 1, 4, 1), (3, 37, 5, 2), (0, 5, 3, 3), (9, 0, 1, 1)])
def test_norm_rope_heads_and_lengths(Tq, Tk, hq, hk, inter, hd):
    _norm_rope_case(Tq, Tk, hq, hk, hd, hd, "bf16", "bf16", 1e4, inter, True, 11)


@pytest.mark.parametrize("x,y", list(itertools.product(["bf16", "f16", "f32"], repeat=2)))
def test_norm_rope_types(x, y):
    _norm_rope_case(5, 19, 6, 2, 64, 32, x, y, 1e6, False, True, 100, pad=8)
    _norm_rope_case(1700, 900, 3, 1, 128, 128, x, y, 1e4, True, False, 0, pad=16)


@pytest.mark.parametrize("rot", [0, 16, 48, 112, 128])
@pytest.mark.parametrize("inter", [False, True])
def test_norm_rope_partial(rot, inter):
    _norm_rope_case(4, 33, 3, 7, 128, rot, "f32", "f32", 500.0, inter, True, 77)


@pytest.mark.parametrize("pos0", [-5, 1 << 20, 2147483000, -2147483648])
def test_norm_rope_far_and_negative_positions(pos0):
    _norm_rope_case(50, 50, 2, 1, 64, 64, "f32", "f32", 1e4, False, True, pos0)


def test_norm_rope_without_positions():
    _norm_rope_case(20, 30, 4, 2, 64, 64, "bf16", "f32", 1e4, False, True, None)


def test_norm_rope_in_place_on_a_fused_projection():
    """Queries and keys normed where the projection left them; values untouched."""
    T, hq, hk, hd = 300, 6, 2, 64
    qkv = _draw((T, (hq + 2 * hk) * hd), "bf16", 9)
    before = qkv.clone()
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    ld, p = qkv.shape[1], qkv.data_ptr()
    q = A.aut_head_rows(p, ld, p, ld, None, pos.data_ptr(), T, hq)
    k = A.aut_head_rows(p + 2 * hq * hd, ld, p + 2 * hq * hd, ld, None, pos.data_ptr(), T, hk)
    assert A.aut_qk_norm_rope(q, k, hd, A.BF16, A.BF16, hd, 1e4, False, 1e-6, _stream()) == A.AUT_OK
    torch.cuda.synchronize()
    ref, norm = R.norm_rope(_np(before)[:, :(hq + hk) * hd].reshape(T, hq + hk, hd), None, pos.cpu().numpy(), hd, hd, 1e4, False, 1e-6)
    got = _np(qkv)[:, :(hq + hk) * hd].reshape(ref.shape)
    assert (np.abs(got - ref) <= 32 * R.U32 * norm * 1.01 + R.HALF["bf16"] * np.abs(ref) + 1e-30).all()
    assert torch.equal(qkv[:, (hq + hk) * hd:], before[:, (hq + hk) * hd:])


def test_norm_rope_one_side_and_zero_head():
    x = torch.zeros(2, 64, device="cuda")
    x[1, 0] = 3.0
    y = torch.empty_like(x)
    pos = torch.zeros(2, dtype=torch.int32, device="cuda")
    side = A.aut_head_rows(x.data_ptr(), 64, y.data_ptr(), 64, None, pos.data_ptr(), 2, 1)
    for q, k in ((side, None), (None, side)):
        y.fill_(7)
        assert A.aut_qk_norm_rope(q, k, 64, A.F32, A.F32, 64, 1e4, False, 1e-6, _stream()) == A.AUT_OK
        torch.cuda.synchronize()
        want = 3 / math.sqrt(9 / 64 + 1e-6)  # eps takes 2.8e-5 off 8
        assert not y[0].any() and abs(y[1, 0].item() - want) < 1e-5 and not y[1, 1:].any()


# -------------------------------------------------------------- cross attention

class Cross:
    """One call's inputs on the GPU; its output has sentinel rows behind it.  `large`: with
    one more request behind the others, of so many rows and keys that the requests of
    more than 32 rows (16, with head_dim 64 and 128) run on the tile kernel."""

    def __init__(self, hq, hk, hd, dtype, q_lens, k_lens, mask=None, scale=None, seed=0, pad=0, qk_scale=1.0, large=False):
        if large:
            if mask is not None and not isinstance(mask, str):
                mask = np.concatenate([mask, np.arange(2999) % 5 != 0])
            q_lens, k_lens = list(q_lens) + [2000 * hk // hq], list(k_lens) + [2999]
        self.hq, self.hk, self.hd, self.dtype = hq, hk, hd, dtype
        self.cu_q = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
        self.cu_k = np.concatenate([[0], np.cumsum(k_lens)]).astype(np.int32)
        self.scale = scale or 1 / math.sqrt(hd)
        tq, tk = int(self.cu_q[-1]), int(self.cu_k[-1])
        self.q = _draw((max(tq, 1), hq * hd + pad), dtype, seed, qk_scale)
        self.kv = _draw((max(tk, 1), 2 * hk * hd + pad), dtype, seed + 1)
        self.mask = None
        if isinstance(mask, str):  # "random"
            self.mask = torch.from_numpy((np.random.default_rng(seed).random(tk) < 0.6).astype(np.uint8) * 255).cuda()
        elif mask is not None:
            self.mask = torch.from_numpy(np.asarray(mask, np.uint8)).cuda()
        self.tq, self.pad = tq, pad
        need = A.aut_cross_attention_workspace_bytes(hq, hk, hd, self.cu_q, self.cu_k)
        assert need > 0
        self.ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")  # any contents will do
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.out = torch.full((tq + 3, hq * hd + 2 * pad), 7.0, dtype=TORCH[dtype], device="cuda")

    def call(self, **over):
        wk = self.hk * self.hd
        arg = dict(q=self.q.data_ptr(), ld_q=self.q.shape[1], k=self.kv.data_ptr(), ld_k=self.kv.shape[1], v=self.kv.data_ptr() + 2 * wk,
                   ld_v=self.kv.shape[1], out=self.out.data_ptr(), ld_out=self.out.shape[1], dtype=CODE[self.dtype], heads_q=self.hq,
                   heads_kv=self.hk, head_dim=self.hd, cu_q=self.cu_q, cu_k=self.cu_k,
                   key_mask=None if self.mask is None else self.mask.data_ptr(), scale=self.scale, workspace=self.ws.data_ptr(),
                   ws_bytes=self.ws.numel(), status=self.status.data_ptr(), timeout_ms=0, stream=_stream())
        return A.aut_cross_attention(**(arg | over))

    def check(self, bad_masked=False):
        wk = self.hk * self.hd
        ref, tol = R.cross_attention(_np(self.q)[:self.tq, :self.hq * self.hd], _np(self.kv)[:, :wk], _np(self.kv)[:, wk:2 * wk], self.cu_q,
                                     self.cu_k, self.hq, self.hk, self.hd, None if self.mask is None else self.mask.cpu().numpy(),
                                     self.scale, self.dtype)
        if bad_masked:
            drop = torch.ones(self.kv.shape[0], dtype=torch.bool, device="cuda")
            drop[:len(self.mask)] = self.mask == 0
            rows = torch.nonzero(drop).flatten()
            self.kv[rows[0::3]] = float("nan")
            self.kv[rows[1::3]] = float("inf")
            self.kv[rows[2::3]] = float("-inf")
        assert self.call() == A.AUT_OK
        torch.cuda.synchronize()
        assert int(self.status.item()) == 0
        got = _np(self.out)
        assert (got[self.tq:] == 7).all() and (got[:, self.hq * self.hd:] == 7).all()
        if self.tq == 0:
            return
        excess = np.abs(got[:self.tq, :self.hq * self.hd] - ref) - tol
        i = np.unravel_index(int(np.nan_to_num(excess, nan=np.inf).argmax()), excess.shape)
        assert excess[i] <= 0, (i, got[i], ref[i], tol[i])


K_EDGES = [0, 1, 2, 31, 32, 33, 127, 128, 129, 255, 257, 500]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("hd", [16, 32, 64, 128])
@pytest.mark.parametrize("hq,hk", [(1, 1), (4, 4), (6, 2), (8, 1), (20, 1)])
def test_cross_single_tokens(hq, hk, hd, dtype):
    Cross(hq, hk, hd, dtype, [1] * len(K_EDGES), K_EDGES).check()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("hd", [16, 32, 64, 128])
@pytest.mark.parametrize("mask", [None, "random"])
@pytest.mark.parametrize("large", [False, True])
def test_cross_ragged_prompts(large, mask, hd, dtype):
    Cross(6, 2, hd, dtype, [0, 1, 5, 6, 43, 130, 0, 129, 257, 17], [3, 0, 1, 129, 128, 500, 40, 127, 33, 300], mask, pad=8,
          large=large).check()


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("hq,hk", [(1, 1), (3, 1), (10, 2), (16, 16)])
@pytest.mark.parametrize("large", [False, True])
def test_cross_longer_prompts(large, hq, hk, hd):
    Cross(hq, hk, hd, "bf16", [300, 1, 128], [700, 1000, 385], large=large).check()


@pytest.mark.parametrize("hd", [64, 128])
def test_cross_prompts_of_one_to_three_row_blocks(hd):
    """15 to 49 rows a request: on the row kernel alone, and beside longer prompts."""
    for large in (False, True):
        Cross(1, 1, hd, "f16", [15, 16, 17, 31, 32, 33, 48, 49], [100, 0, 300, 40, 129, 64, 1, 257], large=large).check()
    Cross(16, 16, hd, "bf16", [32] * 16, [1500] * 16).check()  # many, none longer than two blocks


@pytest.mark.parametrize("hd", [32, 64, 128])
@pytest.mark.parametrize("q_len", [1, 40, 200])
@pytest.mark.parametrize("large", [False, True])
def test_cross_masked_rows_may_hold_anything(large, q_len, hd):
    """Masked keys and values (and rows behind the last request) with infinities
    and NaN; a request whose mask leaves nothing; whole blocks masked first."""
    k_lens = [300, 64, 129, 400]
    m = (np.random.default_rng(1).random(sum(k_lens)) < 0.5).astype(np.uint8)
    m[300:364] = 0
    m[493:493 + 260] = 0
    Cross(4, 2, hd, "bf16", [q_len] * 4, k_lens, m, large=large).check(bad_masked=True)


@pytest.mark.parametrize("hd", [32, 64, 128])
@pytest.mark.parametrize("q_len", [1, 150])
@pytest.mark.parametrize("k_len,at", [(300, 290), (9000, 4321)])
@pytest.mark.parametrize("large", [False, True])
def test_cross_keys_that_are_read_do_reach_the_result(large, k_len, at, q_len, hd):
    """NaN and infinity in a key that counts spoil every query of its request and
    key head, NaN in a query that query's head, and nothing else."""
    for bad in (float("nan"), float("inf")):
        c = Cross(4, 2, hd, "bf16", [q_len, q_len], [k_len, 200], large=large)
        c.kv[at, 0] = bad           # key head 0: query heads 0 and 1 of the first request
        c.kv[k_len + 3, hd] = 0.0
        if bad != bad:
            c.q[2 * q_len - 1, 3 * hd] = bad
        assert c.call() == A.AUT_OK
        torch.cuda.synchronize()
        out = c.out[:2 * q_len, :4 * hd].view(2 * q_len, 4, hd)
        spoilt = torch.isnan(out).all(-1).cpu().numpy()
        want = np.zeros((2 * q_len, 4), bool)
        want[:q_len, :2] = True
        if bad != bad:
            want[2 * q_len - 1, 3] = True
        else:  # infinity times a negative query element is -infinity: that row's key just drops out
            want[:q_len, :2] = (c.q[:q_len, :4 * hd].view(q_len, 4, hd)[:, :2, 0] > 0).cpu().numpy()
        np.testing.assert_array_equal(spoilt, want)
        assert torch.isfinite(out[torch.from_numpy(~want).cuda()]).all()


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("q_len", [1, 3, 70])
@pytest.mark.parametrize("mask", [None, "random"])
@pytest.mark.parametrize("large", [False, True])
def test_cross_split_keys(large, mask, q_len, hd):
    Cross(4, 2, hd, "bf16", [q_len, 1, q_len], [5000, 13, 9001], mask, large=large).check()


@pytest.mark.parametrize("qk_scale", [1e-3, 8.0])
def test_cross_flat_and_sharp_softmax(qk_scale):
    """Nearly equal weights, and weights that all but select one key (a row
    maximum that keeps rising along the keys)."""
    for hd, q, large in ((64, 130, False), (64, 130, True), (128, 1, False), (128, 140, False), (128, 140, True)):
        c = Cross(2, 1, hd, "f16", [q], [900], qk_scale=qk_scale, large=large)
        ramp = torch.linspace(0.1, 1.0, 900, device="cuda")[:, None]
        c.kv[:900, :hd] = (c.kv[:900, :hd].float() * ramp).half()
        c.check()


@pytest.mark.parametrize("n", [512, 513, 1300])
def test_cross_many_requests(n):
    g = np.random.default_rng(n)
    Cross(2, 2, 64, "bf16", g.integers(0, 3, n), g.integers(0, 40, n)).check()


def test_cross_many_requests_with_splits_and_prompts():
    g = np.random.default_rng(4)
    q, k = g.integers(0, 2, 600), g.integers(0, 20, 600)
    q[77], k[77], q[300], k[300], q[599], k[599] = 1, 6000, 150, 90, 3, 7000
    for large in (False, True):
        Cross(2, 1, 64, "bf16", q, k, "random", large=large).check()


def test_cross_nothing_to_do():
    Cross(2, 1, 64, "bf16", [], []).check()
    Cross(2, 1, 64, "bf16", [0, 0], [5, 0]).check()
    Cross(2, 1, 64, "bf16", [2, 0], [0, 0]).check()


@pytest.mark.parametrize("hd", [64, 128])
def test_cross_requests_without_keys_among_prompts(hd):
    """Zeros for the rows of requests without keys, call after call: nothing else of
    such a block may reach its output."""
    c = Cross(16, 8, hd, "bf16", [29, 300, 200, 64, 17, 128], [0, 0, 5, 0, 0, 0], large=True)
    c.check()
    first = c.out.clone()
    for _ in range(200):
        c.out.fill_(7)
        assert c.call() == A.AUT_OK
        assert torch.equal(c.out, first)
    assert not first[:329].any() and not first[529:738].any()


def test_cross_mixed_offsets_as_lists_and_arrays():
    c = Cross(4, 2, 64, "bf16", [1, 20], [50, 60])
    assert c.call() == A.AUT_OK
    first = c.out.clone()
    c.out.fill_(7)
    assert c.call(cu_q=[int(v) for v in c.cu_q], cu_k=torch.from_numpy(c.cu_k).tolist()) == A.AUT_OK
    strided = np.stack([c.cu_k, c.cu_k * 0], 1)[:, 0]  # not contiguous: copied
    assert torch.equal(first, c.out)
    assert c.call(cu_k=strided) == A.AUT_OK
    torch.cuda.synchronize()
    assert torch.equal(first, c.out)


@pytest.mark.parametrize("q_lens,k_lens", [([1, 1], [5000, 40]), ([200, 1, 300], [400, 70, 50]), ([600, 1, 900], [4000, 700, 50])])
def test_cross_same_bits_every_time_and_when_captured(q_lens, k_lens):
    c = Cross(8, 2, 128, "bf16", q_lens, k_lens, "random")
    c.check()
    first = c.out.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        assert c.call() == A.AUT_OK
    for _ in range(3):
        c.out.fill_(7)
        c.ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(first, c.out)
    # replay on new contents of the same buffers
    c.q.copy_(_draw(tuple(c.q.shape), "bf16", 77))
    graph.replay()
    torch.cuda.synchronize()
    replayed = c.out.clone()
    c.out.fill_(7)
    c.check()
    assert torch.equal(replayed, c.out)


def test_cross_two_streams_with_a_workspace_each():
    a = Cross(4, 1, 128, "bf16", [1], [9000], seed=1)
    b = Cross(4, 1, 128, "bf16", [150], [3000], seed=2, large=True)
    a.check()
    b.check()
    wants = a.out.clone(), b.out.clone()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(10):
        a.call(stream=sa.cuda_stream)
        b.call(stream=sb.cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(wants[0], a.out) and torch.equal(wants[1], b.out)


@pytest.mark.parametrize("q_len", [1, 160, 16000])
def test_cross_rows_beyond_32_bit_offsets(q_len):
    """Key rows so far apart that element offsets pass 2^32."""
    hd, nk, ld = 64, 700, 7_000_000
    buf = torch.zeros(nk * ld, dtype=torch.bfloat16, device="cuda")
    rows = buf.view(nk, ld)
    rows[:, :2 * hd] = _draw((nk, 2 * hd), "bf16", 3)
    c = Cross(1, 1, hd, "bf16", [q_len], [nk])
    c.kv = rows[:, :2 * hd].contiguous()
    ref, tol = R.cross_attention(_np(c.q), _np(c.kv)[:, :hd], _np(c.kv)[:, hd:], c.cu_q, c.cu_k, 1, 1, hd, None, c.scale, "bf16")
    assert c.call(k=buf.data_ptr(), ld_k=ld, v=buf.data_ptr() + 2 * hd, ld_v=ld) == A.AUT_OK
    torch.cuda.synchronize()
    assert (np.abs(_np(c.out)[:q_len] - ref) <= tol).all()


# ------------------------------------------------------------------- together

@pytest.mark.parametrize("q_lens", [[1, 1, 1], [33, 150, 4]])
def test_decoder_layer_reads_the_encoder(q_lens):
    """The encoder's own output -> 8-bit key/value projection -> key norm with
    rotation -> cross attention of 8-bit projected, normed, rotated queries, against
    the same chain in 64 bits."""
    from audio_encoder_aut_b200.encoder import Encoder
    cfg = S.TINY
    enc = Encoder(cfg, S.weights(cfg), 0)
    lens = [237, 61, 400]
    states = enc.encode(enc.features_to_device(S.features(lens)), lens)
    tokens, _, total, _, _ = enc.plan(lens)
    D, hq, hk, hd = cfg.output_dim, 4, 2, 64
    st = _stream()
    wkv, wq_ = _draw((2 * hk * hd, D), "f32", 1, D ** -0.5), _draw((hq * hd, D), "f32", 2, D ** -0.5)
    x = _draw((sum(q_lens), D), "bf16", 3)
    gq, gk = _draw((hd,), "bf16", 4), _draw((hd,), "bf16", 5)

    def project(inp, dtype, w):
        xq, sx = _quantize(inp, dtype, D, inp.shape[0], D)
        wq, sw = _quantize(w, "f32", D, w.shape[0], D)
        y = torch.empty(inp.shape[0], w.shape[0], dtype=torch.bfloat16, device="cuda")
        assert A.aut_linear_i8(xq.data_ptr(), sx.data_ptr(), wq.data_ptr(), sw.data_ptr(), None, y.data_ptr(), y.shape[0], y.shape[1], D,
                               A.EPI_BF16, None, 0, 0, st) == A.AUT_OK
        ref, _ = R.linear_i8(xq.cpu().numpy(), sx.cpu().numpy(), wq.cpu().numpy(), sw.cpu().numpy(), None)
        return y, ref

    kv, kv_ref = project(states, "f32", wkv)
    q, q_ref = project(x, "bf16", wq_)
    pk = torch.arange(total, dtype=torch.int32, device="cuda")
    pq = torch.arange(sum(q_lens), dtype=torch.int32, device="cuda") + 50
    assert A.aut_qk_norm_rope(
        A.aut_head_rows(q.data_ptr(), hq * hd, q.data_ptr(), hq * hd, gq.data_ptr(), pq.data_ptr(), len(pq), hq),
        A.aut_head_rows(kv.data_ptr(), 2 * hk * hd, kv.data_ptr(), 2 * hk * hd, gk.data_ptr(), pk.data_ptr(), total, hk),
        hd, A.BF16, A.BF16, hd, 1e4, False, 1e-6, st) == A.AUT_OK
    c = Cross(hq, hk, hd, "bf16", q_lens, tokens)
    c.q, c.kv = q, kv
    assert c.call() == A.AUT_OK
    torch.cuda.synchronize()
    qn, _ = R.norm_rope(q_ref.reshape(-1, hq, hd), _np(gq), pq.cpu().numpy(), hd, hd, 1e4, False, 1e-6)
    kn, _ = R.norm_rope(kv_ref[:, :hk * hd].reshape(-1, hk, hd), _np(gk), pk.cpu().numpy(), hd, hd, 1e4, False, 1e-6)
    ref, _ = R.cross_attention(qn.reshape(len(pq), -1), kn.reshape(total, -1), kv_ref[:, hk * hd:], c.cu_q, c.cu_k, hq, hk, hd, None,
                               c.scale, "bf16")
    assert_rows_close(_np(c.out)[:c.tq], ref, "decoder layer over the encoder's output", rel_max=4e-2)
