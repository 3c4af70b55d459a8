"""The decoder-side operators' definitions in 64 bits (numpy), with the error
bounds that their kernels' roundings allow."""
import math

import numpy as np

U32 = 2.0 ** -24                         # half a step of fp32, relative
HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": U32}
TINY = {"bf16": 0.0, "f16": 2.0 ** -25, "f32": 0.0}  # half a step of the denormals (bf16, fp32: nothing)


def quantize(x):
    """int8 rows and fp32 scales, by the definition's own fp32 steps."""
    x = np.asarray(x, np.float32)
    amax = np.abs(x).max(1)
    with np.errstate(all="ignore"):
        scale = np.where(np.isfinite(amax), amax * (np.float32(1) / np.float32(127)), amax)
        s = np.where((scale > 0) & np.isfinite(scale), scale, np.float32(1))
        q = np.clip(np.rint((x / s[:, None]).astype(np.float32)), -127, 127)
    q[~(np.isfinite(scale) & (scale > 0))] = 0
    return q.astype(np.int8), scale


def linear_i8(xq, sx, wq, sw, bias):
    """Scaled sum in 64 bits, and how far the kernel's fp32 steps may be off: three
    roundings (to fp32, times each scale) of the product and one of the sum with
    the bias, each 2^-24 of what it rounds, the first three with a second-order margin."""
    acc = (xq.astype(np.int64) @ wq.astype(np.int64).T).astype(np.float64)
    prod = acc * sx.astype(np.float64)[:, None] * sw.astype(np.float64)[None]
    y = prod + (0.0 if bias is None else bias.astype(np.float64)[None])
    return y, 3.01 * U32 * np.abs(prod) + U32 * np.abs(y)


def norm_rope(x, gamma, pos, hd, rot, theta, interleaved, eps):
    """[rows, heads, hd] in 64 bits, and every element's pair norm."""
    x = np.asarray(x, np.float64)
    y = x / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps)
    if gamma is not None:
        y = y * np.asarray(gamma, np.float64)
    out, norm = y.copy(), np.abs(y)
    if pos is None or rot == 0:
        return out, norm
    h = rot // 2
    for i in range(h):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + h)
        ang = np.asarray(pos, np.float64) * theta ** (-2.0 * i / rot)
        c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
        out[..., a] = y[..., a] * c - y[..., b] * s
        out[..., b] = y[..., b] * c + y[..., a] * s
        norm[..., a] = norm[..., b] = np.hypot(y[..., a], y[..., b])
    return out, norm


def cross_attention(q, k, v, cu_q, cu_k, heads_q, heads_kv, hd, mask, scale, dtype):
    """Output in 64 bits and the bound of its error.

    With u half a step of the type (P and the output are rounded to it): a score's
    product sum in fp32 is off by at most hd 2^-24 sum |q||k|, its scaling, the
    subtraction of the maximum and the exponential by a few 2^-24 of the exponent
    and 2^-22; every p is then off by a relative e, out = sum p v / sum p by
    (2 e + u) sum p |v| / sum p, the sums by another nk 2^-24 of that, and out's own
    rounding by u |out|."""
    q, k, v = (np.asarray(t, np.float64) for t in (q, k, v))
    u = HALF[dtype]
    group = heads_q // heads_kv
    out = np.zeros((q.shape[0], heads_q * hd))
    tol = np.zeros_like(out)
    for r in range(len(cu_q) - 1):
        rows = np.arange(cu_k[r], cu_k[r + 1])
        if mask is not None:
            rows = rows[np.asarray(mask)[rows] != 0]
        if len(rows) == 0 or cu_q[r] == cu_q[r + 1]:
            continue
        for h in range(heads_q):
            qs = q[cu_q[r]:cu_q[r + 1], h * hd:(h + 1) * hd]
            g = h // group
            ks, vs = k[rows, g * hd:(g + 1) * hd], v[rows, g * hd:(g + 1) * hd]
            s = qs @ ks.T * scale
            big = (np.abs(qs) @ np.abs(ks).T).max(1, keepdims=True) * scale
            e = U32 * (hd * big + 4 * big + 8) * math.log2(math.e)
            p = np.exp(s - s.max(1, keepdims=True))
            tot = p.sum(1, keepdims=True)
            o, oa = p @ vs / tot, p @ np.abs(vs) / tot
            at = np.s_[cu_q[r]:cu_q[r + 1], h * hd:(h + 1) * hd]
            out[at] = o
            tol[at] = ((2 * e + u + 2 * len(rows) * U32) * oa + TINY[dtype] * np.abs(vs).sum(0) / tot
                       + u * np.abs(o) + TINY[dtype])
    return out, tol
