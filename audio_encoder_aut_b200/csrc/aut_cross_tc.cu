// Cross attention on the 5th-generation tensor cores, for prompts: head_dim 64
// and 128, tiles of 128 rows (query, head of the group) against 128 keys.
//
//   S = Q K^T (fp32, tensor memory) -> P = 2^(S scale log2(e) - m), rounded to the
//   inputs' type -> O += P V (fp32, tensor memory), O and the row sums scaled
//   down when a row's maximum has grown by more than 2^8 since O last was: until
//   then the old maximum serves as the softmax's reference, which cancels in
//   O / sum, and P stays at most 2^8.
//
// Warp roles (192 threads, one tile of rows and one split of keys per block):
//   warps 0-3  softmax: thread r owns row r (TMEM lane r), so maximum and sum
//              need no exchange; also Q into shared memory and O out
//   warp 4     TMA producer: K and V tiles (128 keys, 128-byte swizzle) in
//              turn through a ring of slots
//   warp 5     TMEM allocation; one thread issues the products.  P is the A
//              operand from tensor memory
// Two blocks share a SM (256 tensor-memory columns and half the shared memory
// each): while one runs its softmax, the other's products run, without any
// exchange between them.  With head_dim 64 the P columns fit beside S, and the
// next tile's S is computed while this tile's softmax runs; with 128 P takes the
// place of the S it came from, and the next S follows P V in the tensor pipe's
// order.
//
// Keys past the request's end or masked out score -inf, and their V rows are
// zeroed in shared memory (they may hold anything, and 0 * NaN is NaN).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "aut_cross.h"
#include "aut_elem.cuh"
#include "aut_kernels.h"
#include "aut_ptx.cuh"

namespace aut {
namespace {

constexpr int kM = kCrossTileRows, kN = kCrossTileKeys;
constexpr int kThreads = 192;
constexpr uint32_t kTmemCols = 256;

template <int HD>
struct TcCfg {
    static constexpr int kTileBytes = kN * HD * 2;    // K or V of a tile; Q as well
    static constexpr int kAtom = kN * 128;            // 128 rows of 64 elements
    static constexpr int kSlots = HD == 64 ? 5 : 2;   // K and V tiles in shared memory
    static constexpr bool kEarlyS = HD == 64;         // the next S before this P V
    static constexpr uint32_t kColO = kN;             // O behind S
    static constexpr uint32_t kColP = kEarlyS ? kN + HD : 0;
    static constexpr int kOffBar = kTileBytes * (1 + kSlots);
    // full, empty [kSlots]; q_full, s_full, s_read, p_full, pv_done, mma_done
    static constexpr int kBars = 2 * kSlots + 6;
    static constexpr int kSmem = 1024 + kOffBar + kBars * 8 + 16;
    static_assert(kColO + HD + (kEarlyS ? kN / 2 : 0) <= kTmemCols, "tensor memory");
    static_assert(2 * (kSmem + 1024) <= 228 * 1024, "two blocks a SM");
};

template <typename T>
constexpr uint32_t idesc_qk(int n) {
    return std::is_same<T, __half>::value ? idesc_f16_f32(kM, n) : idesc_bf16_f32(kM, n);
}
// B (V) MN-major.
template <typename T, int HD>
constexpr uint32_t idesc_pv() {
    return idesc_qk<T>(HD) | (1u << 16);
}

template <typename T, int HD>
__global__ void __launch_bounds__(kThreads, 2)
    cross_tiles_kernel(const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v,
                       const __grid_constant__ CrossArgs a) {
    using Cfg = TcCfg<HD>;
    constexpr int kSlots = Cfg::kSlots;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t *slots = sm + Cfg::kTileBytes;  // Q first
    uint64_t *full = reinterpret_cast<uint64_t *>(sm + Cfg::kOffBar);
    uint64_t *empty = full + kSlots;
    uint64_t *q_full = empty + kSlots;
    uint64_t *s_full = q_full + 1;
    uint64_t *s_read = s_full + 1;
    uint64_t *p_full = s_read + 1;
    uint64_t *pv_done = p_full + 1;
    uint64_t *mma_done = pv_done + 1;
    uint32_t *tslot = reinterpret_cast<uint32_t *>(mma_done + 1);
    int *abort_flag = reinterpret_cast<int *>(tslot + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile int *abort_v = abort_flag;
    const uint64_t lim = a.timeout_ns;
    auto signal_abort = [&] {
        if (a.status) atomicCAS(a.status, 0, kDevTimeout);
        *abort_v = 1;
    };

    if (threadIdx.x == 0) {
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(full + i, 1);
            mbar_init(empty + i, 1);
        }
        mbar_init(q_full, 4);
        mbar_init(s_full, 1);
        mbar_init(s_read, 4);
        mbar_init(p_full, 4);
        mbar_init(pv_done, 1);
        mbar_init(mma_done, 1);
        *abort_flag = 0;
        fence_barrier_init();
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
    }
    pdl_wait();  // before the tensor memory: the previous kernel's blocks have all left
    if (warp == 5) {
        tmem_alloc(tslot, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_trigger();  // the next kernel's early blocks cannot take columns this one needs
    const uint32_t tmem = *tslot;

    const CrossSeq *seqs = a.seqs ? a.seqs : a.inline_seqs;
    const int seq = cross_find(seqs, a.n_seq, blockIdx.x, lane);
    const CrossSeq s = seqs[seq], nx = seqs[seq + 1];
    const int nq = nx.q0 - s.q0, nk = nx.k0 - s.k0;
    const int rows = nq * a.group, tiles = (rows + kM - 1) / kM;
    int item = (int)blockIdx.x - s.item;
    const int tile = item % tiles;
    item /= tiles;
    const int hk = item % a.heads_kv, split = item / a.heads_kv;
    const int splits = max(1, (nk + a.chunk - 1) / a.chunk);
    const int key0 = s.k0 + split * a.chunk, key1 = min(nx.k0, key0 + a.chunk);
    const int n = (key1 - key0 + kN - 1) / kN;  // key tiles; 0 for a request without keys

    if (warp == 4) {
        if (lane == 0) {
            // ------------------------------------------------ TMA producer --
            // Copy t: K (t even) or V (t odd) of key tile t / 2, in slot t % kSlots.
            bool ok = true;
            int t = 0;
            for (; t < 2 * n; ++t) {
                const int i = t % kSlots;
                if (t >= kSlots && !mbar_wait(empty + i, (uint32_t)(t / kSlots - 1) & 1u, abort_v, lim)) {
                    ok = false;
                    break;
                }
                mbar_arrive_expect_tx(full + i, Cfg::kTileBytes);
#pragma unroll
                for (int c = 0; c < HD / 64; ++c)
                    tma_load_2d(slots + i * Cfg::kTileBytes + c * Cfg::kAtom, t & 1 ? &tm_v : &tm_k,
                                full + i, hk * HD + 64 * c, key0 + (t >> 1) * kN);
            }
            if (!ok) signal_abort();
            // The last copies have landed before the block may exit.
            const uint64_t t0 = global_timer_ns();
            for (int u = t - kSlots < 0 ? 0 : t - kSlots; u < t; ++u) {
                const uint64_t used = global_timer_ns() - t0;
                if (used < lim)
                    mbar_wait(full + u % kSlots, (uint32_t)(u / kSlots) & 1u, nullptr, lim - used);
            }
        }
    } else if (warp == 5) {
        if (lane == 0) {
            // -------------------------------------------------- MMA issuer --
            auto n16 = [&](int j) { return min(kN, (key1 - key0 - j * kN + 15) & ~15); };
            auto issue_s = [&](int j) -> bool {
                const int t = 2 * j, i = t % kSlots;
                if (!mbar_wait(full + i, (uint32_t)(t / kSlots) & 1u, abort_v, lim)) return false;
                tc_fence_after();
                const uint32_t id = idesc_qk<T>(n16(j));
#pragma unroll
                for (int c = 0; c < HD / 16; ++c) {
                    const int at = (c >> 2) * Cfg::kAtom;
                    tc_mma_bf16(tmem, smem_desc_sw128(sm + at) + 2 * (c & 3),
                                smem_desc_sw128(slots + i * Cfg::kTileBytes + at) + 2 * (c & 3), id,
                                c > 0);
                }
                tc_commit(s_full);
                tc_commit(empty + i);
                return true;
            };
            bool ok = n == 0 || mbar_wait(q_full, 0, abort_v, lim);
            if (ok && n > 0) ok = issue_s(0);
            for (int j = 0; ok && j < n; ++j) {
                if (Cfg::kEarlyS && j + 1 < n) {
                    ok = mbar_wait(s_read, (uint32_t)j & 1u, abort_v, lim);
                    if (ok) tc_fence_after();
                    ok = ok && issue_s(j + 1);
                }
                const int t = 2 * j + 1, i = t % kSlots;
                ok = ok && mbar_wait(p_full, (uint32_t)j & 1u, abort_v, lim) &&
                     mbar_wait(full + i, (uint32_t)(t / kSlots) & 1u, abort_v, lim);
                if (!ok) break;
                tc_fence_after();
                const int steps = n16(j) / 16;
                for (int c = 0; c < steps; ++c)
                    tc_mma_f16_ts(tmem + Cfg::kColO, tmem + Cfg::kColP + 8 * c,
                                  smem_desc_sw128_mn(slots + i * Cfg::kTileBytes + c * 16 * 128,
                                                     Cfg::kAtom),
                                  idesc_pv<T, HD>(), j > 0 || c > 0);
                tc_commit(pv_done);
                tc_commit(empty + i);
                if (!Cfg::kEarlyS && j + 1 < n) ok = issue_s(j + 1);
            }
            if (!ok) signal_abort();
            // Every product this thread issued has completed before TMEM is released.
            tc_commit(mma_done);
            mbar_wait(mma_done, 0, nullptr, lim);
        }
    } else {
        // ------------------------------------------------------- softmax --
        // Q: 16 bytes a thread, rows of the tile one after the other.
        constexpr int kChunks = HD / 8;
        for (int i = threadIdx.x; i < kM * kChunks; i += 128) {
            const int r = i / kChunks, c = i % kChunks, at = tile * kM + r;
            const int tok = at / a.group, head = hk * a.group + at - tok * a.group;
            uint4 v = make_uint4(0, 0, 0, 0);
            if (at < rows)
                v = *reinterpret_cast<const uint4 *>(static_cast<const T *>(a.q) +
                                                     (size_t)(s.q0 + tok) * a.ld_q + head * HD + c * 8);
            *reinterpret_cast<uint4 *>(sm + (c >> 3) * Cfg::kAtom + r * 128 + (((c & 7) ^ (r & 7)) << 4)) = v;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(q_full);

        const int row = warp * 32 + lane;
        const bool active = tile * kM + warp * 32 < rows;  // some row of the warp exists
        const uint32_t trow = tmem + ((uint32_t)(warp * 32) << 16);
        const float2 scale2 = make_float2(a.scale_log2e, a.scale_log2e);
        float m = -INFINITY, l = 0.f;  // the softmax's reference (unscaled) and the row's sum
        bool ok = true;
        // Which of key tile j's keys are read, as 4 words of 32 keys.
        auto tile_keys = [&](int j, uint32_t(&w)[4]) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int key = key0 + j * kN + c * 32 + lane;
                w[c] = __ballot_sync(0xffffffffu,
                                     j < n && key < key1 && (!a.mask || a.mask[key] != 0));
            }
        };
        uint32_t next[4];
        tile_keys(0, next);
        for (int j = 0; j < n; ++j) {
            const uint32_t keys[4] = {next[0], next[1], next[2], next[3]};
            const bool whole = (keys[0] & keys[1] & keys[2] & keys[3]) == 0xffffffffu;
            tile_keys(j + 1, next);
            if (!mbar_wait_warp(s_full, (uint32_t)j & 1u, abort_v, lim)) {
                ok = false;
                break;
            }
            tc_fence_after();
            float v[4][32];
            if (active) {
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld32(trow + 32 * c, v[c]);
                tc_wait_ld();
            }
            if (Cfg::kEarlyS) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(s_read);
            }
            float neg = 0.f;  // -(reference) in units of the exponent
            bool shrink = false;
            float f = 1.f;
            if (active) {
                if (!whole) {
#pragma unroll
                    for (int c = 0; c < 4; ++c)
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            v[c][e] = keys[c] & (1u << e) ? v[c][e] : -INFINITY;
                }
                float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int e = 0; e < 32; e += 2) top[c] = fmax3(top[c], v[c][e], v[c][e + 1]);
                const float mn = fmaxf(m, fmaxf(fmax3(top[0], top[1], top[2]), top[3]));
                const bool grown = (mn - m) * a.scale_log2e > 8.f;  // also from no key at all
                shrink = __any_sync(0xffffffffu, grown);
                if (grown) {
                    f = ex2_approx((m - mn) * a.scale_log2e);
                    m = mn;
                    l *= f;
                }
                neg = m == -INFINITY ? 0.f : -m * a.scale_log2e;
            }
            // P into tensor memory (over S, or over the last P) and O scaled only
            // once the previous P V is done.
            if (j > 0 && !mbar_wait_warp(pv_done, (uint32_t)(j - 1) & 1u, abort_v, lim)) {
                ok = false;
                break;
            }
            tc_fence_after();
            if (active) {
                const float2 neg2 = make_float2(neg, neg);
                float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t p[32];
#pragma unroll
                    for (int e = 0; e < 64; e += 2) {
                        const float *x = &v[2 * h + (e >> 5)][e & 31];
                        const float2 y = ffma2(make_float2(x[0], x[1]), scale2, neg2);
                        const float2 q = make_float2(ex2_approx(y.x), ex2_approx(y.y));
                        sum[(e >> 1) & 1] = fadd2(sum[(e >> 1) & 1], q);
                        p[e >> 1] = pack2<T>(q.x, q.y);
                    }
                    tmem_st32(trow + Cfg::kColP + 32 * h, p);
                }
                const float2 all = fadd2(sum[0], sum[1]);
                l += all.x + all.y;
                if (shrink && j > 0) {
#pragma unroll 1
                    for (int c = 0; c < HD; c += 16) {
                        float o[16];
                        tmem_ld16(trow + Cfg::kColO + c, o);
                        tc_wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[e] *= f;
                        tmem_st16(trow + Cfg::kColO + c, o);
                    }
                }
                tc_wait_st();
            }
            if (!whole) {  // this thread's key's V row, if it is not read
                const int t = 2 * j + 1, i = t % kSlots;
                if (!mbar_wait_warp(full + i, (uint32_t)(t / kSlots) & 1u, abort_v, lim)) {
                    ok = false;
                    break;
                }
                if (!((keys[warp] >> lane) & 1u))
#pragma unroll
                    for (int c = 0; c < kChunks; ++c)
                        *reinterpret_cast<uint4 *>(slots + i * Cfg::kTileBytes + (c >> 3) * Cfg::kAtom +
                                                   row * 128 + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
                fence_proxy_async_smem();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(p_full);
        }
        if (ok && n > 0) ok = mbar_wait_warp(pv_done, (uint32_t)(n - 1) & 1u, abort_v, lim);
        if (!ok && lane == 0) signal_abort();
        if (ok && active) {
            tc_fence_after();
            const int at = tile * kM + row, tok = at / a.group, head = hk * a.group + at - tok * a.group;
            const bool in = at < rows;
            const float inv = splits > 1 ? 1.f : l == 0.f ? 0.f : 1.f / l;  // no key: zeros
            const size_t prow = (size_t)s.part + ((size_t)split * nq + tok) * a.heads_q + head;
            T *dst = static_cast<T *>(a.out) + (size_t)(s.q0 + tok) * a.ld_out + head * HD;
#pragma unroll
            for (int c = 0; c < HD; c += 32) {
                float o[32];
                if (n > 0) {
                    tmem_ld32(trow + Cfg::kColO + c, o);
                    tc_wait_ld();
                }
                if (in) {
#pragma unroll
                    for (int e = 0; e < 32; e += 8) {
                        float w[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) w[i] = n > 0 ? o[e + i] * inv : 0.f;
                        if (splits > 1)
                            store8(a.part_o + prow * HD + c + e, w);
                        else
                            store8(dst + c + e, w);
                    }
                }
                __syncwarp();  // converged again before the next warp-wide load
            }
            if (in && splits > 1) a.part_ml[prow] = make_float2(m * a.scale_log2e, l);
        }
    }
    tc_fence_before();
    __syncwarp();
    __syncthreads();
    if (warp == 5) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

template <typename T, int HD>
cudaError_t launch(const CrossArgs &a, const CUtensorMap &tk, const CUtensorMap &tv, cudaStream_t st) {
    const cudaError_t e = smem_attr_once<cross_tiles_kernel<T, HD>>(TcCfg<HD>::kSmem);
    if (e != cudaSuccess) return e;
    return launch_pdl(cross_tiles_kernel<T, HD>, dim3(a.items), dim3(kThreads), TcCfg<HD>::kSmem, st, 1,
                      tk, tv, a);
}

}  // namespace

cudaError_t launch_cross_tiles(const CrossArgs &a, int hd, bool f16, int tk, cudaStream_t st) {
    CUtensorMap maps[2];
    const uint64_t dims[2] = {(uint64_t)a.heads_kv * hd, (uint64_t)std::max(tk, 1)};
    const uint32_t box[2] = {64, kN};
    for (int i = 0; i < 2; ++i) {
        // Without any key no copy runs; the map then only has to encode.
        const void *p = tk > 0 ? (i ? a.v : a.k) : a.q;
        const uint64_t stride[1] = {tk > 0 ? (uint64_t)(i ? a.ld_v : a.ld_k) * 2 : dims[0] * 2};
        // 16-bit copies: the maps of bf16 serve fp16 as well (the zero fill is zero in both).
        if (!make_tensor_map_bf16_sw128(&maps[i], 2, p, dims, stride, box)) return cudaErrorInvalidValue;
    }
    if (hd == 64)
        return f16 ? launch<__half, 64>(a, maps[0], maps[1], st)
                   : launch<__nv_bfloat16, 64>(a, maps[0], maps[1], st);
    return f16 ? launch<__half, 128>(a, maps[0], maps[1], st)
               : launch<__nv_bfloat16, 128>(a, maps[0], maps[1], st);
}

}  // namespace aut
