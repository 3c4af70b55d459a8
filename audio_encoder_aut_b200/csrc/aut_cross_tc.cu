// Cross attention on the 5th-generation tensor cores, for prompts: head_dim 64
// and 128, tiles of 128 rows (query, head of the group) against 128 keys.
//
//   S = Q K^T (fp32, tensor memory) -> P = 2^(S scale log2(e) - m), rounded to the
//   inputs' type -> O += P V (fp32, tensor memory), O and the row sums scaled
//   down when a row's maximum has grown by more than 2^8 since O last was: until
//   then the old maximum serves as the softmax's reference, which cancels in
//   O / sum, and P stays at most 2^8 (fp16: 2^15).
//
// Warp roles (384 threads; two tiles of rows, 256 rows in all, and one split of
// keys per block):
//   warps 0-7  softmax, four warps a tile: thread r owns row r (TMEM lane r), so
//              maximum and sum need no exchange; also Q into shared memory and O
//              out
//   warp 8     TMA producer: K and V tiles (128 keys, 128-byte swizzle) in
//              turn through a ring of slots, each read by both row tiles
//   warp 9     TMEM allocation, and the products.  P is the A operand from tensor
//              memory
//   warps 10, 11  zeros over the V rows of keys that are not read
// The one issuer alternates between the row tiles, so that while one tile's
// softmax runs the other's products do.  (As two blocks a SM with one tile each,
// the two issuers' products share the tensor pipe instruction by instruction, and
// both blocks fall into step: softmax against softmax, products against products,
// 528 us where the alternating issuer, otherwise the same, took 386 us for 16
// requests of 512 x 4096, 16 heads of 128.)  With head_dim 64 the P columns fit beside S, and the next tile's S is
// computed while this tile's softmax runs; with 128 P takes the place of the S
// it came from, and the next S follows P V in the tensor pipe's order.
//
// Bound by the chain S -> softmax -> P V -> S of a row tile, of which the tensor
// cores are busy 45%: 16 requests of 512 x 4096, 16 heads of 128: 271 us, 1012
// TFLOP/s, 0.61 of the measured bf16 peak; head_dim 64 (32 heads) 440 us, 625
// TFLOP/s, the exponentials' pipe busy 58%, the tensor cores 29%, issue slots 40%:
// there too no pipe is full, the chain is what is long.  Tried without gain: a part of
// the exponentials as a polynomial on the FMA pipe, two threads a row (registers
// spill), P V of a tile's first 96 keys before the rest's P is made, and persistent
// blocks (the loop's registers).
//
// Keys past the request's end or masked out score -inf, and their V rows are
// zeroed in shared memory (they may hold anything, and 0 * NaN is NaN).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "aut_cross.h"
#include "aut_elem.cuh"
#include "aut_kernels.h"
#include "aut_ptx.cuh"

namespace aut {
namespace {

constexpr int kM = 128, kN = kCrossTileKeys;  // rows of a tile, keys of a tile
constexpr int kSoftmaxWarps = 8;              // four per row tile
constexpr int kThreads = 32 * (kSoftmaxWarps + 4);  // three warpgroups
// Registers a thread: 168 at launch (three warps to a quarter of the register
// file), of which the third warpgroup gives some to the softmax, for its rows of 128
// scores.  256 * 208 + 128 * 80 <= 384 * 168.  (The compiler still reports 36 to 48
// bytes of spill stores.)
constexpr int kSoftmaxRegs = 208, kOtherRegs = 80;
constexpr uint32_t kTmemCols = 512;

template <int HD>
struct TcCfg {
    static constexpr int kTileBytes = kN * HD * 2;    // K or V of a tile; Q of a row tile as well
    static constexpr int kAtom = kN * 128;            // 128 rows of 64 elements
    static constexpr int kSlots = HD == 64 ? 10 : 5;  // K and V tiles in shared memory
    static constexpr bool kEarlyS = HD == 64;         // the next S before this P V
    // Tensor memory: S of the row tiles, then their O; P beside them or over S.
    static constexpr uint32_t kColO = 2 * kN;
    static constexpr uint32_t kColP = kEarlyS ? kColO + 2 * HD : 0;
    static constexpr uint32_t kStepP = kEarlyS ? kN / 2 : kN;  // from one row tile's P to the other's
    static constexpr int kOffBar = kTileBytes * (2 + kSlots);
    // V tiles until one takes the same slot again.
    static constexpr int kCleanRing = kSlots % 2 ? kSlots : kSlots / 2;
    // full, empty [kSlots]; q_full; s_full, s_read, p_full, pv_done [2]; mma_done;
    // loading, clean [kCleanRing]
    static constexpr int kBars = 2 * kSlots + 10 + 2 * kCleanRing;
    static constexpr int kSmem = 1024 + kOffBar + kBars * 8 + 16;
    static_assert(kColO + 2 * HD + (kEarlyS ? kN : 0) <= kTmemCols, "tensor memory");
    static_assert(kSmem <= 232448, "shared memory of a block");
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

// Bounded waits for this kernel's chain of short steps: a plain try_wait (which
// suspends the thread for as long as the hardware likes) comes back 30 to 60
// clocks sooner than one with a suspend-time hint.
AUT_DEV bool wait_try(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(ok)
        : "r"(smem_addr(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}
AUT_DEV bool wait_one(uint64_t *bar, uint32_t parity, volatile int *abort, uint64_t limit_ns) {
    if (wait_try(bar, parity)) return true;
    uint64_t t0 = 0;
#pragma unroll 1
    for (uint32_t i = 1;; ++i) {
        if (wait_try(bar, parity)) return true;
        if ((i & 63u) == 0) {
            const uint64_t now = global_timer_ns();
            if (i == 64) t0 = now;
            if ((abort && *abort) || now - t0 > limit_ns) return false;
        }
    }
}
AUT_DEV bool wait_warp(uint64_t *bar, uint32_t parity, volatile int *abort, uint64_t limit_ns) {
    return __all_sync(0xffffffffu, wait_one(bar, parity, abort, limit_ns));
}

// Maximum of a row's 128 scores, in four chains.
AUT_DEV float row_max(const float (&v)[4][32]) {
    float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int e = 0; e < 32; e += 2) top[c] = fmax3(top[c], v[c][e], v[c][e + 1]);
    return fmaxf(fmax3(top[0], top[1], top[2]), top[3]);
}

template <typename T, int HD>
__global__ void __launch_bounds__(kThreads, 1)
    cross_tiles_kernel(const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v,
                       const __grid_constant__ CrossArgs a) {
    using Cfg = TcCfg<HD>;
    constexpr int kSlots = Cfg::kSlots;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t *slots = sm + 2 * Cfg::kTileBytes;  // behind the row tiles' Q
    uint64_t *full = reinterpret_cast<uint64_t *>(sm + Cfg::kOffBar);
    uint64_t *empty = full + kSlots;
    uint64_t *q_full = empty + kSlots;
    uint64_t *s_full = q_full + 1;    // [2] per row tile, as the next three
    uint64_t *s_read = s_full + 2;
    uint64_t *p_full = s_read + 2;
    uint64_t *pv_done = p_full + 2;
    uint64_t *mma_done = pv_done + 2;
    // V tiles that may miss keys, one after the other: on their way, and ready.
    uint64_t *loading = mma_done + 1;  // [kCleanRing]
    uint64_t *clean = loading + Cfg::kCleanRing;
    uint32_t *tslot = reinterpret_cast<uint32_t *>(clean + Cfg::kCleanRing);
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
        mbar_init(q_full, kSoftmaxWarps);
        for (int i = 0; i < 2; ++i) {
            mbar_init(s_full + i, 1);
            mbar_init(s_read + i, 4);
            mbar_init(p_full + i, 4);
            mbar_init(pv_done + i, 1);
        }
        mbar_init(mma_done, 1);
        for (int i = 0; i < Cfg::kCleanRing; ++i) {
            mbar_init(loading + i, 1);
            mbar_init(clean + i, 2);
        }
        *abort_flag = 0;
        fence_barrier_init();
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
    }
    // The item, from the parameters, while the previous kernel ends.
    const CrossSeq *seqs = a.seqs ? a.seqs : a.inline_seqs;
    int seq = 0;
    if (!a.seqs) seq = cross_find(seqs, a.n_seq, blockIdx.x, lane);
    pdl_wait();  // before the tensor memory: the previous kernel's blocks have all left
    if (a.seqs) seq = cross_find(seqs, a.n_seq, blockIdx.x, lane);
    const CrossSeq s = seqs[seq];
    const int nq = s.nq, rows = nq * a.group, tiles = (rows + kCrossTileRows - 1) / kCrossTileRows;
    int item = (int)blockIdx.x - s.item;
    const int row0 = item % tiles * kCrossTileRows;
    item /= tiles;
    const int hk = item % a.heads_kv, split = item / a.heads_kv;
    const int key0 = s.k0 + split * s.keys, key1 = min(s.k0 + s.nk, key0 + s.keys);
    const int n = (key1 - key0 + kN - 1) / kN;  // key tiles; 0 for a request without keys
    const int n_rt = rows - row0 > kM ? 2 : 1;  // row tiles in use
    const int n_whole = a.mask ? 0 : max(0, key1 - key0) / kN;  // key tiles known to miss no key

    // Q: 16 bytes a thread, rows one after the other; the loads run while the block
    // sets itself up.
    constexpr int kChunks = HD / 8, kLoads = 2 * kM * kChunks / (32 * kSoftmaxWarps);
    constexpr int kStep = 32 * kSoftmaxWarps / kChunks;  // rows from one load to the next
    uint4 qv[kLoads];
    if (warp < kSoftmaxWarps) {
        const int step_tok = kStep / a.group, step_rem = kStep - step_tok * a.group;
        int at = row0 + (int)threadIdx.x / kChunks, tok = at / a.group, rem = at - tok * a.group;
        const T *qp = static_cast<const T *>(a.q) + (size_t)s.q0 * a.ld_q + hk * a.group * HD +
                      threadIdx.x % kChunks * 8;
#pragma unroll
        for (int u = 0; u < kLoads; ++u) {
            qv[u] = make_uint4(0, 0, 0, 0);
            if (at < rows) qv[u] = *reinterpret_cast<const uint4 *>(qp + (size_t)tok * a.ld_q + rem * HD);
            at += kStep;
            tok += step_tok;
            if ((rem += step_rem) >= a.group) {
                rem -= a.group;
                ++tok;
            }
        }
    }

    if (warp == kSoftmaxWarps + 1) {
        tmem_alloc(tslot, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_trigger();  // the next kernel's early blocks cannot take columns this one needs
    const uint32_t tmem = *tslot;

    if (warp >= kSoftmaxWarps) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        if (warp == kSoftmaxWarps && lane == 0) {
            // ------------------------------------------------ TMA producer --
            // Copy t: K (t even) or V (t odd) of key tile t / 2, in slot t % kSlots.
            bool ok = true;
            int t = 0;
            for (; t < 2 * n; ++t) {
                const int i = t % kSlots;
                if (t >= kSlots && !wait_one(empty + i, (uint32_t)(t / kSlots - 1) & 1u, abort_v, lim)) {
                    ok = false;
                    break;
                }
                if (t + 1 != a.left_out || blockIdx.x != 0) {
                    mbar_arrive_expect_tx(full + i, Cfg::kTileBytes);
#pragma unroll
                    for (int c = 0; c < HD / 64; ++c)
                        tma_load_2d(slots + i * Cfg::kTileBytes + c * Cfg::kAtom, t & 1 ? &tm_v : &tm_k,
                                    full + i, hk * HD + 64 * c, key0 + (t >> 1) * kN);
                }
                if ((t & 1) && (t >> 1) >= n_whole) mbar_arrive(loading + ((t >> 1) - n_whole) % Cfg::kCleanRing);
            }
            if (!ok) signal_abort();
            // The last copies have landed before the block may exit.
            const uint64_t t0 = global_timer_ns();
            for (int u = t - kSlots < 0 ? 0 : t - kSlots; u < t; ++u) {
                const uint64_t used = global_timer_ns() - t0;
                if (used < lim)
                    wait_one(full + u % kSlots, (uint32_t)(u / kSlots) & 1u, nullptr, lim - used);
            }
        }
        if (warp == kSoftmaxWarps + 1) {
            // -------------------------------------------------- MMA issuer --
            // The whole warp runs the loop, so that descriptors are warp-uniform
            // values (kept in uniform registers, which the products take); one
            // lane issues.
            const bool leader = elect_one();
            auto n16 = [&](int j) { return min(kN, (key1 - key0 - j * kN + 15) & ~15); };
            // Slots of the next K and V tile and their phases.
            int ki = 0, vi = 1 % kSlots;
            uint32_t kp = 0, vp = 0;
            const uint64_t slot_k = smem_desc_sw128(slots), slot_v = smem_desc_sw128_mn(slots, Cfg::kAtom);
            const uint64_t q_desc = smem_desc_sw128(sm);
            constexpr uint32_t kTile16 = Cfg::kTileBytes >> 4, kAtom16 = Cfg::kAtom >> 4;
            // The wait for a slot belongs to its first user, its release to its last.
            auto wait_k = [&] { return wait_warp(full + ki, kp, abort_v, lim); };
            auto wait_v = [&] { return wait_warp(full + vi, vp, abort_v, lim); };
            auto issue_s = [&](int j, int rt) {
                const uint32_t id = idesc_qk<T>(n16(j));
                const uint64_t qd = q_desc + rt * kTile16, kd = slot_k + ki * kTile16;
                if (leader) {
#pragma unroll
                    for (int c = 0; c < HD / 16; ++c)
                        tc_mma_bf16(tmem + rt * kN, qd + (c >> 2) * kAtom16 + 2 * (c & 3),
                                    kd + (c >> 2) * kAtom16 + 2 * (c & 3), id, c > 0);
                    tc_commit(s_full + rt);
                    if (rt == n_rt - 1) tc_commit(empty + ki);
                }
                __syncwarp();
                if (rt == n_rt - 1) {
                    if ((ki += 2) >= kSlots) {
                        ki -= kSlots;
                        kp ^= 1u;
                    }
                }
            };
            auto issue_pv = [&](int j, int rt) {
                const int steps = n16(j) / 16;
                const uint64_t vd = slot_v + vi * kTile16;
                const uint32_t d = tmem + Cfg::kColO + rt * HD, p = tmem + Cfg::kColP + rt * Cfg::kStepP;
                if (leader) {
#pragma unroll
                    for (int c = 0; c < kN / 16; ++c)
                        if (c < steps)
                            tc_mma_f16_ts(d, p + 8 * c, vd + c * (16 * 128 / 16), idesc_pv<T, HD>(),
                                          (j | c) > 0);
                    tc_commit(pv_done + rt);
                    if (rt == n_rt - 1) tc_commit(empty + vi);
                }
                __syncwarp();
                if (rt == n_rt - 1) {
                    if ((vi += 2) >= kSlots) {
                        vi -= kSlots;
                        vp ^= 1u;
                    }
                }
            };
            bool ok = n > 0 && wait_warp(q_full, 0, abort_v, lim) && wait_k();
            if (ok) {
                tc_fence_after();
                for (int rt = 0; rt < n_rt; ++rt) issue_s(0, rt);
            }
            for (int j = 0; ok && j < n; ++j) {
                // V of this tile and K of the next, long there, before the wait for P.
                ok = wait_v() && (j + 1 == n || wait_k());
                for (int rt = 0; ok && rt < n_rt; ++rt) {
                    if (Cfg::kEarlyS && j + 1 < n) {
                        ok = wait_warp(s_read + rt, (uint32_t)j & 1u, abort_v, lim);
                        if (!ok) break;
                        tc_fence_after();
                        issue_s(j + 1, rt);
                    }
                    if (rt == 0 && j >= n_whole) {
                        const int u = j - n_whole;
                        ok = wait_warp(clean + u % Cfg::kCleanRing, (uint32_t)(u / Cfg::kCleanRing) & 1u,
                                       abort_v, lim);
                    }
                    ok = ok && wait_warp(p_full + rt, (uint32_t)j & 1u, abort_v, lim);
                    if (!ok) break;
                    tc_fence_after();
                    issue_pv(j, rt);
                    if (!Cfg::kEarlyS && j + 1 < n) issue_s(j + 1, rt);
                }
            }
            // Every product the leader issued has completed before TMEM is released.
            if (leader) {
                if (!ok && n > 0) signal_abort();
                tc_commit(mma_done);
                wait_one(mma_done, 0, nullptr, lim);
            }
            __syncwarp();
        }
        if (warp >= kSoftmaxWarps + 2) {
            // ------------------------------------------------------ V rows --
            // Zeros over the V rows of keys that are not read, 64 keys a warp.  (Left
            // to the softmax, between its P and the product, this took 6 of 43 us
            // on masked prompts.)
            const int first = (warp - kSoftmaxWarps - 2) * 64;
            bool ok = true;
            uint8_t next[2];
            auto load_mask = [&](int j) {
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int key = key0 + j * kN + first + c * 32 + lane;
                    next[c] = j < n && key < key1 && (!a.mask || a.mask[key] != 0);
                }
            };
            load_mask(n_whole);
            for (int j = n_whole; ok && j < n; ++j) {
                uint32_t keys[2];
#pragma unroll
                for (int c = 0; c < 2; ++c) keys[c] = __ballot_sync(0xffffffffu, next[c] != 0);
                load_mask(j + 1);
                // Once its copy is on its way the slot's barrier is in this tile's phase
                // (and stays there until its P V).
                const int t = 2 * j + 1, i = t % kSlots, u = j - n_whole;
                ok = wait_warp(loading + u % Cfg::kCleanRing, (uint32_t)(u / Cfg::kCleanRing) & 1u, abort_v,
                               lim) &&
                     wait_warp(full + i, (uint32_t)(t / kSlots) & 1u, abort_v, lim);
                if (!ok) break;
                if ((keys[0] & keys[1]) != 0xffffffffu) {
                    const int c = lane % kChunks;
#pragma unroll 4
                    for (int r = lane / kChunks; r < 64; r += 32 / kChunks)
                        if (!((keys[r >> 5] >> (r & 31)) & 1u))
                            *reinterpret_cast<uint4 *>(slots + i * Cfg::kTileBytes + (c >> 3) * Cfg::kAtom +
                                                       (first + r) * 128 + (c & 7) * 16) =
                                make_uint4(0, 0, 0, 0);
                    fence_proxy_async_smem();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(clean + u % Cfg::kCleanRing);
            }
            if (!ok && lane == 0) signal_abort();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
        // ------------------------------------------------------- softmax --
        // Q into shared memory.
        if (n > 0) {
            // Not for a request without keys: nothing would order these writes before
            // the output's, which goes out through the same place.
#pragma unroll
            for (int u = 0; u < kLoads; ++u) {
                const int i = threadIdx.x + u * 32 * kSoftmaxWarps, r = i / kChunks, c = i % kChunks;
                *reinterpret_cast<uint4 *>(sm + (r >> 7) * Cfg::kTileBytes + (c >> 3) * Cfg::kAtom +
                                           (r & 127) * 128 + (((c & 7) ^ (r & 7)) << 4)) = qv[u];
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(q_full);
        }

        const int rt = warp >> 2, quad = warp & 3;
        const int row = quad * 32 + lane;  // of the row tile, and TMEM lane
        const bool used = rt < n_rt;
        const bool active = row0 + rt * kM + quad * 32 < rows;  // some row of the warp exists
        const uint32_t trow = tmem + ((uint32_t)(quad * 32) << 16);
        const uint32_t t_s = trow + rt * kN, t_o = trow + Cfg::kColO + rt * HD,
                       t_p = trow + Cfg::kColP + rt * Cfg::kStepP;
        const float2 scale2 = make_float2(a.scale_log2e, a.scale_log2e);
        float m = -INFINITY, l = 0.f;  // the softmax's reference (unscaled) and the row's sum
        bool ok = true;
        // Which of key tile j's keys are read, as 4 words of 32 keys, for tiles that
        // may miss some; their mask bytes are loaded one tile ahead.
        auto load_mask = [&](int j, uint8_t(&w)[4]) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int key = key0 + j * kN + c * 32 + lane;
                w[c] = j < n && key < key1 && (!a.mask || a.mask[key] != 0);
            }
        };
        uint8_t next[4] = {0, 0, 0, 0};
        if (n_whole == 0) load_mask(0, next);
        for (int j = 0; used && j < n; ++j) {
            uint32_t keys[4] = {0, 0, 0, 0};
            bool whole = true;
            if (j >= n_whole) {
#pragma unroll
                for (int c = 0; c < 4; ++c) keys[c] = __ballot_sync(0xffffffffu, next[c] != 0);
                whole = (keys[0] & keys[1] & keys[2] & keys[3]) == 0xffffffffu;
            }
            if (j + 1 >= n_whole) load_mask(j + 1, next);
            if (!wait_warp(s_full + rt, (uint32_t)j & 1u, abort_v, lim)) {
                ok = false;
                break;
            }
            tc_fence_after();
            float v[4][32];
            if (active) {
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld32(t_s + 32 * c, v[c]);
                tc_wait_ld();
            }
            if (Cfg::kEarlyS) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(s_read + rt);
            }
            // P over the last P, and O scaled, only once the last P V is done.  (With
            // P over S, this S came after it.)
            if (Cfg::kEarlyS && j > 0 && !wait_warp(pv_done + rt, (uint32_t)(j - 1) & 1u, abort_v, lim)) {
                ok = false;
                break;
            }
            if (active) {
                tc_fence_after();
                if (!whole) {
#pragma unroll
                    for (int c = 0; c < 4; ++c)
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            v[c][e] = keys[c] & (1u << e) ? v[c][e] : -INFINITY;
                }
                if (j == 0) m = row_max(v);
                // P by the reference so far, the maximum beside it; once more by
                // the new one in the rare case that it has grown too much.
                float f = 1.f, sum;
                while (true) {
                    const float neg = (m == -INFINITY ? 0.f : -m * a.scale_log2e) + kCrossLift<T>;
                    const float2 neg2 = make_float2(neg, neg);
                    float2 s2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                    float top[4] = {m, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint32_t p[16];
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            const float *x = &v[c][e];
                            top[(e >> 1) & 3] = fmax3(top[(e >> 1) & 3], x[0], x[1]);
                            const float2 y = ffma2(make_float2(x[0], x[1]), scale2, neg2);
                            const float2 q = make_float2(ex2_approx(y.x), ex2_approx(y.y));
                            s2[(e >> 1) & 1] = fadd2(s2[(e >> 1) & 1], q);
                            p[e >> 1] = pack2<T>(q.x, q.y);
                        }
                        tmem_st16u(t_p + 16 * c, p);
                    }
                    const float2 all = fadd2(s2[0], s2[1]);
                    sum = all.x + all.y;
                    const float mn = fmaxf(fmax3(top[0], top[1], top[2]), top[3]);
                    const bool grown = (mn - m) * a.scale_log2e > 8.f;  // also from no key at all
                    if (!__any_sync(0xffffffffu, grown)) break;
                    if (grown) {
                        f *= ex2_approx((m - mn) * a.scale_log2e);
                        m = mn;
                    }
                }
                l = l * f + sum;
                if (j > 0 && __any_sync(0xffffffffu, f != 1.f)) {
#pragma unroll 1
                    for (int c = 0; c < HD; c += 16) {
                        float o[16];
                        tmem_ld16(t_o + c, o);
                        tc_wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[e] *= f;
                        tmem_st16(t_o + c, o);
                    }
                }
                tc_wait_st();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(p_full + rt);
        }
        if (ok && used && n > 0) ok = wait_warp(pv_done + rt, (uint32_t)(n - 1) & 1u, abort_v, lim);
        if (!ok && lane == 0) signal_abort();
        if (ok && active) {
            tc_fence_after();
            const int at = row0 + rt * kM + row, tok = at / a.group, head = hk * a.group + at - tok * a.group;
            const bool in = at < rows;
            const float inv = s.splits > 1 ? 1.f : l == 0.f ? 0.f : 1.f / l;  // no key: zeros
            const size_t prow = (size_t)s.part + ((size_t)split * nq + tok) * a.heads_q + head;
            // Out through the warp's 32 rows of the Q tile, which every S of this row
            // tile has read: a thread's row becomes whole lines of the warp's stores.
            uint8_t *const box = sm + rt * Cfg::kTileBytes + quad * 32 * HD * 2;
            char *const dst =
                in ? (s.splits > 1 ? reinterpret_cast<char *>(a.part_o + prow * HD)
                               : reinterpret_cast<char *>(static_cast<T *>(a.out) +
                                                          (size_t)(s.q0 + tok) * a.ld_out + head * HD))
                   : nullptr;
            // 16-byte chunks lane by lane: kRowChunks to a row of `box`, `at` bytes into the row.
            auto flush = [&](auto row_chunks, int at_bytes) {
                constexpr int kRowChunks = decltype(row_chunks)::value;
                __syncwarp();
#pragma unroll
                for (int u = 0; u < kRowChunks; ++u) {
                    const int i = u * 32 + lane, r = i / kRowChunks, c = i % kRowChunks;
                    char *to = reinterpret_cast<char *>(
                        __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(dst), r));
                    if (to)
                        *reinterpret_cast<uint4 *>(to + at_bytes + c * 16) =
                            *reinterpret_cast<const uint4 *>(box + r * kRowChunks * 16 +
                                                             ((c ^ (r & 7)) << 4));
                }
                __syncwarp();
            };
#pragma unroll
            for (int c = 0; c < HD; c += 32) {
                float o[32];
                if (n > 0) {
                    tmem_ld32(t_o + c, o);
                    tc_wait_ld();
                }
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = n > 0 ? o[e] * inv : 0.f;
                if (s.splits > 1) {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        *reinterpret_cast<float4 *>(box + lane * 128 + ((e ^ (lane & 7)) << 4)) =
                            make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                    flush(std::integral_constant<int, 8>(), c * 4);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        *reinterpret_cast<uint4 *>(box + lane * HD * 2 + (((c / 8 + e) ^ (lane & 7)) << 4)) =
                            make_uint4(pack2<T>(o[8 * e], o[8 * e + 1]), pack2<T>(o[8 * e + 2], o[8 * e + 3]),
                                       pack2<T>(o[8 * e + 4], o[8 * e + 5]),
                                       pack2<T>(o[8 * e + 6], o[8 * e + 7]));
                }
            }
            if (s.splits == 1) flush(std::integral_constant<int, kChunks>(), 0);
            if (in && s.splits > 1) a.part_ml[prow] = make_float2(m * a.scale_log2e, l);
        }
    }
    tc_fence_before();
    __syncwarp();
    __syncthreads();
    if (warp == kSoftmaxWarps + 1) {
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
