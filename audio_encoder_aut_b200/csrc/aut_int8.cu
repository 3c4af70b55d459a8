// The 8-bit integer linear layer's own kernels and entry points: quantising
// rows (tokens or weight channels) to int8 with a scale each, and the product
// for a few tokens.  Larger products run on the tcgen05 GEMM (aut_gemm.cuh, I8).
//
// Each kernel starts while the one before it ends, and that one may be writing its
// tokens, scales or weights: coherent loads after the wait, no read-only ones (which
// ask that the data stays as it is from the kernel's start).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "aut_elem.cuh"
#include "aut_internal.h"
#include "aut_kernels.h"
#include "aut_ptx.cuh"

namespace aut {
namespace {

// ---------------------------------------------------------------- quantise --
// scale = max |x| (1 / 127), q = rint(x / scale): the row's maximum first, then the
// row again, so a row is kept in registers between the two (the rest of a row too
// long for them is read a second time).  One read of x and one write of q; an element
// costs about ten instructions and none on the conversion pipe: the maximum is taken
// on the bits, two 16-bit elements at a time, and rounding is an addition.  15600 x
// 5120: from fp32 64 us (6.2 TB/s), bound by HBM; from bf16 61 us (3.9 TB/s), which is
// not: a warp has no load in flight while it reduces and stores its row.

constexpr int kQuantThreads = 256;

// max(top, |elements|) as bits, for 16-bit types two halves at a time: their order is
// the values', infinity above every number and NaN above that.
template <typename T>
AUT_DEV uint32_t top_bits(const Pack8<T> &r, uint32_t t) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 8; ++i) t = max(t, r.w[i] & 0x7fffffffu);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) t = __vmaxu2(t, r.w[i] & 0x7fff7fffu);
    }
    return t;
}
template <typename T>
AUT_DEV uint32_t fold_bits(uint32_t t) {
    return sizeof(T) == 4 ? t : max(t & 0xffffu, t >> 16);
}
template <typename T>
AUT_DEV float bits_value(uint32_t t) {
    if constexpr (sizeof(T) == 4)
        return __uint_as_float(t);
    else
        return Pack8<T>::pair(t).x;
}

// Eight values / scale, rounded to nearest even, as bytes.  The quotient is taken as
// x * inv, off by less than 4e-5 for |x / scale| <= 127 (the reciprocal's rounding, the
// product's and the quotient's, each 2^-24 of it); adding 1.5 2^23 rounds it and
// leaves the integer in the low bits.  Only where a quotient lies within 1e-4 of a
// rounding border (or a denormal scale has spoilt it) are the eight divided.
AUT_DEV uint2 quantise8(const float (&x)[8], float scale, float inv) {
    constexpr float kMagic = 12582912.f;
    float t[8], off = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float r = x[e] * inv;
        t[e] = r + kMagic;
        off = fmaxf(off, fabsf(r - (t[e] - kMagic)));
    }
    // An infinite inv or product is no distance from its own rounding: refused by
    // the scale's own size.
    if (off > 0.4999f || scale < 1e-37f) {
#pragma unroll
        for (int e = 0; e < 8; ++e) t[e] = fmaxf(-127.f, fminf(127.f, x[e] / scale)) + kMagic;
    }
    uint32_t o[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t a = __byte_perm(__float_as_uint(t[4 * h]), __float_as_uint(t[4 * h + 1]), 0x0040);
        const uint32_t b = __byte_perm(__float_as_uint(t[4 * h + 2]), __float_as_uint(t[4 * h + 3]), 0x0040);
        o[h] = __byte_perm(a, b, 0x5410);
    }
    return make_uint2(o[0], o[1]);
}

// W warps per row, 8 / W rows a block; a thread keeps C chunks of 8 elements.
template <typename T, int W, int C>
__global__ void __launch_bounds__(kQuantThreads, C == 4 ? 4 : 3) quantize_rows_kernel(
    const T *x, long long ld, int M, int K, int8_t *q, float *scale) {
    __shared__ uint32_t warp_max[kQuantThreads / 32];
    pdl_trigger();
    pdl_wait();
    const int warp = threadIdx.x >> 5;
    constexpr int kStep = W * 32;  // chunks one pass of the row's threads covers
    const int team = warp / W, row = (int)blockIdx.x * (kQuantThreads / 32 / W) + team;
    if (row >= M) return;  // whole teams
    const int t = threadIdx.x & (kStep - 1), chunks = K / 8;
    const T *xr = x + (size_t)row * ld;
    Pack8<T> v[C];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int c = t + i * kStep;
        if (c < chunks) v[i].load(xr + c * 8);
    }
#pragma unroll
    for (int i = 0; i < C; ++i)
        if (t + i * kStep < chunks) top = top_bits(v[i], top);
    for (int c = t + C * kStep; c < chunks; c += kStep) {
        Pack8<T> w;
        w.load(xr + c * 8);
        top = top_bits(w, top);
    }
    top = __reduce_max_sync(0xffffffffu, fold_bits<T>(top));
    if constexpr (W > 1) {
        if ((threadIdx.x & 31) == 0) warp_max[warp] = top;
        asm volatile("barrier.cta.sync %0, %1;" ::"r"(team + 1), "n"(W * 32) : "memory");
#pragma unroll
        for (int w = 0; w < W; ++w) top = max(top, warp_max[team * W + w]);
    }
    const float amax = bits_value<T>(top);
    const bool finite = amax < INFINITY;
    const float s = finite ? amax * (1.f / 127.f) : amax;
    if (t == 0) scale[row] = s;
    const bool zero = !finite || s == 0.f;
    const float inv = 1.f / s;
    int8_t *qr = q + (size_t)row * K;
    auto store = [&](int c, const Pack8<T> &raw) {
        float f[8];
        raw.values(f);
        *reinterpret_cast<uint2 *>(qr + c * 8) = zero ? make_uint2(0, 0) : quantise8(f, s, inv);
    };
#pragma unroll
    for (int i = 0; i < C; ++i)
        if (t + i * kStep < chunks) store(t + i * kStep, v[i]);
    for (int c = t + C * kStep; c < chunks; c += kStep) {
        Pack8<T> w;
        w.load(xr + c * 8);
        store(c, w);
    }
}

template <typename T>
cudaError_t launch_quantize(const void *x, long long ld, int M, int K, void *q, void *scale,
                            cudaStream_t st) {
    const auto go = [&](auto kernel, int rows) {
        return launch_pdl(kernel, dim3((M + rows - 1) / rows), dim3(kQuantThreads), 0, st, 1,
                          static_cast<const T *>(x), ld, M, K, static_cast<int8_t *>(q),
                          static_cast<float *>(scale));
    };
    // All eight warps to a row while there are too few rows to fill the GPU
    // otherwise (390 x 1024 fp32: 2.3 us); else the fewest that keep it in their
    // registers, so that more rows are in flight: fp32 in 4 chunks a thread
    // (15600 x 1280: 17 to 19 us, 24 us in 8), 16-bit types in 8 (14.4 us, 15.3 us in
    // 4: a row of 1280 then takes two warps and a barrier).
    constexpr int C = sizeof(T) == 4 ? 4 : 8;
    if (M >= 8 * sm_count_cached()) {
        if (K <= 32 * 8 * C) return go(quantize_rows_kernel<T, 1, C>, 8);
        if (K <= 2 * 32 * 8 * C) return go(quantize_rows_kernel<T, 2, C>, 4);
        if (K <= 4 * 32 * 8 * C) return go(quantize_rows_kernel<T, 4, C>, 2);
    }
    return go(quantize_rows_kernel<T, 8, 4>, 1);
}

// ------------------------------------------------- product for a few tokens --
// Up to 32 tokens: the weights are read once.  A block takes 16 output
// channels, its eight warps share K in blocks of 64 bytes.  One m16n8k32 product
// has the 16 channels as its rows and 8 tokens as its columns; since the sum over
// K may run in any order, a lane's 16 consecutive bytes of a row serve as its
// operand words of two products (the same permutation of K on both sides), so
// weights (read once: past L1) and tokens go from global memory to registers in
// 16-byte loads with no shared memory between.  The warps' int32 sums meet in shared
// memory: exact, so in any order.  One token, 2048 x 2048 in L2: 2.4 us, a launch's
// latency.  Weights from HBM, N x K: 1 token 13824 x 5120 13.7 us (5.2 TB/s), 5120 x
// 13824 21.7 us (3.3), 4096 x 4096 7.6 us (2.2).  On 5120 x 13824, 8 tokens take 22.2
// us, 16 31.6 us and 32 64.4 us (every block reads the tokens anew, with 32 of them
// twice the weights' bytes in all), where 33 tokens take 38.0 us on the tcgen05 GEMM.

constexpr int kFewThreads = 256;
constexpr int kFewTokens = 32;

AUT_DEV void mma_s8(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                    uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// NT: tiles of 8 tokens.
template <int NT>
__global__ void __launch_bounds__(kFewThreads) linear_i8_few_kernel(
    const int8_t *x, const float *x_scale, const int8_t *w, const float *w_scale,
    const __nv_bfloat16 *bias, void *y, int M, int N, int K, int epi) {
    __shared__ int part[kFewThreads / 32][NT][8][16 + 1];  // [warp][tile][token][channel]
    pdl_trigger();
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int n0 = blockIdx.x * 16;
    const int8_t *w0 = w + (size_t)(n0 + g) * K + 16 * t;
    const int8_t *w1 = w0 + (size_t)8 * K;
    int acc[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[j][e] = 0;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    constexpr int kUnroll = NT > 2 ? 2 : 4;
    constexpr int kStep = 64 * (kFewThreads / 32);
    for (int k0 = warp * 64; k0 < K; k0 += kUnroll * kStep) {
        uint4 a[kUnroll][2], b[kUnroll][NT];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int k = k0 + u * kStep;
            const bool in = k + 16 * t < K;
            a[u][0] = in ? __ldcg(reinterpret_cast<const uint4 *>(w0 + k)) : zero;
            a[u][1] = in ? __ldcg(reinterpret_cast<const uint4 *>(w1 + k)) : zero;
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const int tok = j * 8 + g;
                b[u][j] = in && tok < M
                              ? *reinterpret_cast<const uint4 *>(x + (size_t)tok * K + k + 16 * t)
                              : zero;
            }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                mma_s8(acc[j], a[u][0].x, a[u][1].x, a[u][0].y, a[u][1].y, b[u][j].x, b[u][j].y);
                mma_s8(acc[j], a[u][0].z, a[u][1].z, a[u][0].w, a[u][1].w, b[u][j].z, b[u][j].w);
            }
    }
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) part[warp][j][2 * t + (e & 1)][g + 8 * (e >> 1)] = acc[j][e];
    __syncthreads();
    for (int i = threadIdx.x; i < NT * 8 * 16; i += kFewThreads) {
        const int n = i & 15, m = i >> 4;
        if (m >= M) break;
        int sum = 0;
#pragma unroll
        for (int v = 0; v < kFewThreads / 32; ++v) sum += part[v][m >> 3][m & 7][n];
        float r = __int2float_rn(sum) * x_scale[m] * w_scale[n0 + n];
        const float b = bias ? __bfloat162float(bias[n0 + n]) : 0.f;
        const size_t o = (size_t)m * N + n0 + n;
        float *yf = static_cast<float *>(y);
        __nv_bfloat16 *yh = static_cast<__nv_bfloat16 *>(y);
        switch (epi) {
            case kEpiResidF32: yf[o] = r + (yf[o] + b); break;
            case kEpiF32: yf[o] = r + b; break;
            case kEpiBf16Gelu: yh[o] = __float2bfloat16_rn(gelu_fast(r + b)); break;
            default: yh[o] = __float2bfloat16_rn(r + b); break;
        }
    }
}

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

constexpr int kMaxK8 = 131072;         // 127 * 128 * 131072 < 2^31 (128^2 * 131072 is not)
constexpr int kMaxRows = 0x7ffff000;   // row indexes are 32-bit, a block's spare rows included

}  // namespace
}  // namespace aut

using namespace aut;

extern "C" aut_status aut_quantize_rows(const void *x, int32_t dtype, int64_t ld_x, int32_t M,
                                        int32_t K, void *q, void *scale, aut_stream_t stream) {
    if (dtype < AUT_BF16 || dtype > AUT_F32 || M < 0 || K <= 0) return AUT_ERR_INVALID_ARG;
    if (K % 16 || K > kMaxK8 || M > kMaxRows) return AUT_ERR_UNSUPPORTED;
    if (M == 0) return AUT_OK;
    const int64_t es = dtype == AUT_F32 ? 4 : 2;
    if (!x || !q || !scale || ld_x < K || (ld_x * es) % 16 || ld_x > (int64_t)1 << 40)
        return AUT_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(q, 16) || !aligned(scale, 4)) return AUT_ERR_INVALID_ARG;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (dtype == AUT_BF16)
        e = launch_quantize<__nv_bfloat16>(x, ld_x, M, K, q, scale, st);
    else if (dtype == AUT_F16)
        e = launch_quantize<__half>(x, ld_x, M, K, q, scale, st);
    else
        e = launch_quantize<float>(x, ld_x, M, K, q, scale, st);
    return e == cudaSuccess ? AUT_OK : AUT_ERR_CUDA;
}

extern "C" aut_status aut_linear_i8(const void *xq, const void *x_scale, const void *wq,
                                    const void *w_scale, const void *bias, void *y, int32_t M,
                                    int32_t N, int32_t K, int32_t epilogue, int32_t *status,
                                    int32_t timeout_ms, int32_t flags, aut_stream_t stream) {
    if (M < 0 || N <= 0 || K <= 0 || epilogue < 0 || epilogue > 3 || timeout_ms < 0)
        return AUT_ERR_INVALID_ARG;
    if (flags & ~(AUT_LINEAR_FAULT_INJECT | AUT_LINEAR_SINGLE_CTA)) return AUT_ERR_INVALID_ARG;
    if (K % 16 || N % 16 || K > kMaxK8 || M > kMaxRows) return AUT_ERR_UNSUPPORTED;
    if (M == 0) return AUT_OK;
    if (!xq || !x_scale || !wq || !w_scale || !y) return AUT_ERR_INVALID_ARG;
    if (!aligned(xq, 16) || !aligned(wq, 16) || !aligned(w_scale, 16) || !aligned(y, 16) ||
        !aligned(x_scale, 4) || (bias && !aligned(bias, 16)))
        return AUT_ERR_INVALID_ARG;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const int epi = epilogue == 3 ? kEpiF32 : epilogue;
    if (M <= kFewTokens) {
        if (flags & AUT_LINEAR_FAULT_INJECT) return AUT_ERR_UNSUPPORTED;
        const auto launch = [&](auto kernel) {
            return launch_pdl(kernel, dim3(N / 16), dim3(kFewThreads), 0, st, 1,
                              static_cast<const int8_t *>(xq), static_cast<const float *>(x_scale),
                              static_cast<const int8_t *>(wq), static_cast<const float *>(w_scale),
                              static_cast<const __nv_bfloat16 *>(bias), y, (int)M, (int)N, (int)K,
                              epi);
        };
        const cudaError_t e = M <= 8    ? launch(linear_i8_few_kernel<1>)
                              : M <= 16 ? launch(linear_i8_few_kernel<2>)
                                        : launch(linear_i8_few_kernel<4>);
        return e == cudaSuccess ? AUT_OK : AUT_ERR_CUDA;
    }
    LinearLaunch L{};
    L.a = xq;
    L.w = wq;
    L.bias = bias;
    L.out = y;
    L.M = M;
    L.N = N;
    L.K = K;
    L.ldo = N;
    L.epi = epi;
    L.status = reinterpret_cast<int *>(status);
    L.timeout_ns = timeout_ms ? (unsigned long long)timeout_ms * 1000000ull : 4000ull * 1000000ull;
    L.fault_inject = (flags & AUT_LINEAR_FAULT_INJECT) ? 1 : 0;
    L.single_cta = (flags & AUT_LINEAR_SINGLE_CTA) != 0;
    L.x_scale = static_cast<const float *>(x_scale);
    L.w_scale = static_cast<const float *>(w_scale);
    switch (launch_linear(L, st)) {
        case GemmStatus::kOk: return AUT_OK;
        case GemmStatus::kBadShape: return AUT_ERR_INVALID_ARG;
        default: return AUT_ERR_CUDA;
    }
}
