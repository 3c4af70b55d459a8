// RMS norm of query and key heads with the rotation by position, in one pass.
//
//   y = R(pos) (x / sqrt(mean x^2 + eps) * gamma)  over every head of every row
//
// Bound by HBM: every element is read once and written once (15600 rows of 16 heads
// of 64, fp32 to bf16: 18.7 us, 5.4 TB/s; 3253 rows of 24 heads of 128, bf16: 10.7
// us, 3.8 TB/s, of which 2 us are the launch's).  A warp takes one
// row and some of its heads, 16 elements of a head per lane: the two 8-element
// blocks that a rotation in halves pairs with each other, so the rotation needs
// no exchange, and the sum of squares log2(lanes per head) shuffles.
//
// The angle of pair i is pos * theta^(-2 i / rot) radians.  In turns it is
// pos * f with f = theta^(-2 i / rot) / 2 pi, and only its fraction matters.  With f
// held as a 64-bit binary fraction, the wrapping 64-bit product pos * f is that
// fraction exactly as far as f is exact (2^-64 of a turn times pos): no position
// is too far, and no sine table is read.  Sine and cosine of a row are computed
// once per warp and shared by its heads through shared memory.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "aut_elem.cuh"
#include "aut_internal.h"
#include "aut_kernels.h"
#include "aut_ptx.cuh"

namespace aut {
namespace {

constexpr int kWarps = 4;
constexpr int kMaxPairs = 128;  // head_dim 256

struct Side {
    const void *x;
    void *y;
    const __nv_bfloat16 *gamma;
    const int *pos;
    long long ld_x, ld_y;
    int rows, heads;
    int parts, part_heads;  // warps per row and heads per warp
};

struct NormRopeArgs {
    Side side[2];
    int tasks0, tasks;        // warps' tasks of side 0; of both
    int rot;                  // rotated elements, rot / 2 pairs
    int interleaved;
    float eps;
    unsigned long long turn[kMaxPairs];  // f of every pair, in 2^-64 turns
};

// G lanes per head: head_dim = 16 G.
template <typename TX, typename TY, int G>
__global__ void __launch_bounds__(kWarps * 32, 6)
    qk_norm_rope_kernel(const __grid_constant__ NormRopeArgs a) {
    constexpr int HD = 16 * G, kHeads = 32 / G;  // heads a warp handles at a time
    __shared__ unsigned long long turn[HD / 2];
    __shared__ float2 cs[kWarps][HD / 2];
    pdl_trigger();
    for (int i = threadIdx.x; i < a.rot / 2; i += kWarps * 32) turn[i] = a.turn[i];
    __syncthreads();
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int task = (int)blockIdx.x * kWarps + warp;
    if (task >= a.tasks) return;
    const Side &s = a.side[task >= a.tasks0];
    if (task >= a.tasks0) task -= a.tasks0;
    const int row = task / s.parts, part = task - row * s.parts;
    const int h_end = min(s.heads, (part + 1) * s.part_heads);
    const int c = lane % G, rb = a.rot / 16;  // this lane's place in its head; rotated block pairs
    // The lane's two blocks of 8 elements: a pair of the rotation, or two
    // neighbours of the part behind it.
    const int b0 = c < rb ? c : 2 * rb + 2 * (c - rb);
    const int b1 = c < rb ? c + rb : b0 + 1;
    const TX *x = static_cast<const TX *>(s.x) + (size_t)row * s.ld_x;
    TY *y = static_cast<TY *>(s.y) + (size_t)row * s.ld_y;
    int h = part * s.part_heads + lane / G;
    float v0[8], v1[8];
    if (h < h_end) {
        load8(x + h * HD + b0 * 8, v0);
        load8(x + h * HD + b1 * 8, v1);
    }
    const bool rotate = s.pos != nullptr && rb > 0;  // the same for the whole warp
    if (rotate) {
        const long long pos = s.pos[row];
        for (int i = lane; i < a.rot / 2; i += 32) {
            const long long t = (long long)((unsigned long long)pos * turn[i]);
            float sn, cn;  // of 2^-31 (t >> 32) half turns
            sincospif((float)(int)(t >> 32) * 0x1p-31f, &sn, &cn);
            cs[warp][i] = make_float2(cn, sn);
        }
        __syncwarp();
    }
    float g0[8], g1[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) g0[e] = g1[e] = 1.f;
    if (s.gamma) {
        load8(s.gamma + b0 * 8, g0);
        load8(s.gamma + b1 * 8, g1);
    }
    for (int hw = part * s.part_heads; hw < h_end; hw += kHeads, h += kHeads) {
        const bool in = h < h_end;
        float n0[8], n1[8];
        if (h + kHeads < h_end) {  // the next heads' elements, before this one's arithmetic
            load8(x + (h + kHeads) * HD + b0 * 8, n0);
            load8(x + (h + kHeads) * HD + b1 * 8, n1);
        }
        float sum = 0.f;
        if (in)
#pragma unroll
            for (int e = 0; e < 8; ++e) sum = fmaf(v0[e], v0[e], fmaf(v1[e], v1[e], sum));
#pragma unroll
        for (int o = G / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (in) {
            const float r = rsqrtf(sum * (1.f / HD) + a.eps);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                v0[e] = v0[e] * r * g0[e];
                v1[e] = v1[e] * r * g1[e];
            }
            if (rotate && c < rb) {
                if (a.interleaved) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 p = cs[warp][b0 * 4 + e], q = cs[warp][b1 * 4 + e];
                        const float a0 = v0[2 * e], a1 = v1[2 * e];
                        v0[2 * e] = a0 * p.x - v0[2 * e + 1] * p.y;
                        v0[2 * e + 1] = v0[2 * e + 1] * p.x + a0 * p.y;
                        v1[2 * e] = a1 * q.x - v1[2 * e + 1] * q.y;
                        v1[2 * e + 1] = v1[2 * e + 1] * q.x + a1 * q.y;
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float2 p = cs[warp][b0 * 8 + e];
                        const float a0 = v0[e];
                        v0[e] = a0 * p.x - v1[e] * p.y;
                        v1[e] = v1[e] * p.x + a0 * p.y;
                    }
                }
            }
            store8(y + h * HD + b0 * 8, v0);
            store8(y + h * HD + b1 * 8, v1);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            v0[e] = n0[e];
            v1[e] = n1[e];
        }
    }
}

template <typename TX, typename TY>
cudaError_t launch_norm_rope(const NormRopeArgs &a, int hd, unsigned blocks, cudaStream_t st) {
    const auto go = [&](auto kernel) {
        return launch_pdl(kernel, dim3(blocks), dim3(kWarps * 32), 0, st, 1, a);
    };
    switch (hd) {
        case 16: return go(qk_norm_rope_kernel<TX, TY, 1>);
        case 32: return go(qk_norm_rope_kernel<TX, TY, 2>);
        case 64: return go(qk_norm_rope_kernel<TX, TY, 4>);
        case 128: return go(qk_norm_rope_kernel<TX, TY, 8>);
        case 256: return go(qk_norm_rope_kernel<TX, TY, 16>);
        default: return cudaErrorInvalidValue;
    }
}

template <typename TX>
cudaError_t launch_norm_rope(const NormRopeArgs &a, int hd, int y_dtype, unsigned blocks,
                             cudaStream_t st) {
    switch (y_dtype) {
        case AUT_BF16: return launch_norm_rope<TX, __nv_bfloat16>(a, hd, blocks, st);
        case AUT_F16: return launch_norm_rope<TX, __half>(a, hd, blocks, st);
        default: return launch_norm_rope<TX, float>(a, hd, blocks, st);
    }
}

int elem_size(int dtype) { return dtype == AUT_F32 ? 4 : 2; }

bool side_ok(const aut_head_rows &r, int hd, int x_dtype, int y_dtype) {
    if (r.rows < 0 || r.heads <= 0 || r.heads > (1 << 20) / hd) return false;
    if (r.rows == 0) return true;
    const int64_t width = (int64_t)r.heads * hd, most = (int64_t)1 << 40;
    if (!r.x || !r.y || r.ld_x < width || r.ld_y < width || r.ld_x > most || r.ld_y > most) return false;
    if ((r.ld_x * elem_size(x_dtype)) % 16 || (r.ld_y * elem_size(y_dtype)) % 16) return false;
    const uintptr_t p = reinterpret_cast<uintptr_t>(r.x) | reinterpret_cast<uintptr_t>(r.y) |
                        reinterpret_cast<uintptr_t>(r.gamma);
    if (p & 15u || reinterpret_cast<uintptr_t>(r.positions) & 3u) return false;
    return true;
}

}  // namespace
}  // namespace aut

using namespace aut;

extern "C" aut_status aut_qk_norm_rope(const aut_head_rows *q, const aut_head_rows *k,
                                       int32_t head_dim, int32_t x_dtype, int32_t y_dtype,
                                       int32_t rot_dim, double theta, int32_t interleaved,
                                       float eps, aut_stream_t stream) {
    if (x_dtype < AUT_BF16 || x_dtype > AUT_F32 || y_dtype < AUT_BF16 || y_dtype > AUT_F32)
        return AUT_ERR_INVALID_ARG;
    if (head_dim != 16 && head_dim != 32 && head_dim != 64 && head_dim != 128 && head_dim != 256)
        return AUT_ERR_UNSUPPORTED;
    if (rot_dim < 0 || rot_dim > head_dim || !(theta >= 1.0) || !std::isfinite(theta) ||
        !(eps >= 0.f) || !std::isfinite(eps))
        return AUT_ERR_INVALID_ARG;
    if (rot_dim % 16) return AUT_ERR_UNSUPPORTED;
    NormRopeArgs a{};
    const aut_head_rows *in[2] = {q, k};
    const int at_once = 32 / (head_dim / 16);
    for (int i = 0; i < 2; ++i) {
        if (!in[i]) continue;
        if (!side_ok(*in[i], head_dim, x_dtype, y_dtype)) return AUT_ERR_INVALID_ARG;
    }
    // A warp takes all heads of its row (its sines serve them all) unless that
    // leaves most of the GPU idle; then each takes what it can at once.
    const int64_t rows = (q ? q->rows : 0) + (int64_t)(k ? k->rows : 0);
    const bool whole_rows = rows >= 16ll * sm_count_cached();
    int64_t tasks = 0;
    for (int i = 0; i < 2; ++i) {
        Side &s = a.side[i];
        s.parts = 1;
        if (in[i] && in[i]->rows > 0) {
            s.x = in[i]->x;
            s.y = in[i]->y;
            s.gamma = static_cast<const __nv_bfloat16 *>(in[i]->gamma);
            s.pos = in[i]->positions;
            s.ld_x = in[i]->ld_x;
            s.ld_y = in[i]->ld_y;
            s.rows = in[i]->rows;
            s.heads = in[i]->heads;
            s.part_heads = whole_rows ? s.heads : at_once;
            s.parts = (s.heads + s.part_heads - 1) / s.part_heads;
        }
        tasks += (int64_t)s.rows * s.parts;
        if (tasks > 0x7fffff00ll) return AUT_ERR_UNSUPPORTED;
        a.tasks = (int)tasks;
        if (i == 0) a.tasks0 = a.tasks;
    }
    if (a.tasks == 0) return AUT_OK;
    const unsigned blocks = ((unsigned)a.tasks + kWarps - 1) / kWarps;
    a.rot = rot_dim;
    a.interleaved = interleaved != 0;
    a.eps = eps;
    if (rot_dim > 0) {
        // theta^(-2 i / rot) / 2 pi < 0.16 as a 64-bit fraction of a turn.
        const long double ratio = powl((long double)theta, -2.0L / rot_dim);
        long double f = 0.159154943091895335768883763372514362L * 0x1p64L;
        for (int i = 0; i < rot_dim / 2; ++i, f *= ratio)
            a.turn[i] = (unsigned long long)(f + 0.5L);
    }
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (x_dtype == AUT_BF16)
        e = launch_norm_rope<__nv_bfloat16>(a, head_dim, y_dtype, blocks, st);
    else if (x_dtype == AUT_F16)
        e = launch_norm_rope<__half>(a, head_dim, y_dtype, blocks, st);
    else
        e = launch_norm_rope<float>(a, head_dim, y_dtype, blocks, st);
    return e == cudaSuccess ? AUT_OK : AUT_ERR_CUDA;
}
