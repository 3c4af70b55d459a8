// Cross attention over an encoder's packed states: the host plan, the kernel for
// a few query rows, the join of split requests, and the entry point.  (Many rows
// of head_dim 64 and 128 run on the tcgen05 kernel, aut_cross_tc.cu.)
//
//   out[i, h] = sum_j p_ij v[j, h'] / sum_j p_ij,   p_ij = 2^(s_ij - max_j s_ij),
//   s_ij = (q[i, h] . k[j, h']) scale log2(e),   h' = h / group
//
// over the keys j of query i's request that the mask leaves.  One pass over the
// keys with the running maximum and sum of the softmax.
//
// cross_rows_kernel: 16 rows (query, head of the group) of one request and key
// head per block.  With so few rows the work is reading keys and values once (256
// requests of one token on 780 keys, 16 heads of 128 over 8: 122 us for 818 MB, far
// more than L2 holds, 6.7 TB/s: reads alone pass the measured copy's 6.46), so
// the block's warps each stream key blocks of their own (block w, w + W, ...)
// through a private ring of cp.async copies, with no barrier between warps until
// their results are joined at the end.  A masked key, or one past the end, is
// zero-filled by its copy: whatever stands there never enters.  Scores and P V
// are m16n8k16 products: a tcgen05 tile has 128 rows, and would leave
// seven eighths of them empty here.
//
// A request whose keys take longer than its share of the GPU is split along
// them; every split leaves its unnormalised rows, their maximum and their sum in
// the workspace, and cross_join_kernel adds them up in a fixed order.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <new>

#include "aut_cross.h"
#include "aut_elem.cuh"
#include "aut_internal.h"
#include "aut_kernels.h"
#include "aut_ptx.cuh"

namespace aut {
namespace {

// Small rings, so that three blocks share a SM: most requests of a batch are a step
// or two long, and a block's start and end are then most of its time (256 requests
// of 6 to 780 keys: 37 us; 65 us with 32 keys and 3 stages, one block a SM).
constexpr int kRows = 16;    // rows of one block
constexpr int kRowWarps = 4;
// With no more blocks than SMs there is room for twice the warps, and half the
// steps (one token, 16 heads of 128: 6.6 us against 9.2 us on 2000 keys; on a full GPU
// they cost, 65 us against 37 us for 256 requests).
constexpr int kRowWarpsAlone = 8;
constexpr int kKeys = 16;    // keys of a warp's block (at most a lane each, for the mask)
constexpr int kStages = 2;   // blocks a warp holds in its ring

template <int HD, int W>
struct RowsCfg {
    static constexpr int kRowBytes = HD * 2;
    static constexpr int kTile = kKeys * kRowBytes;  // K or V of one block
    static constexpr int kWarpBytes = kStages * 2 * kTile;
    static constexpr int kJoin = W * kRows * (HD + 4) * 4;  // the warps' O, padded rows
    static constexpr int kSmem = W * kWarpBytes > kJoin ? W * kWarpBytes : kJoin;
};

// Byte offset of the 16-byte chunk c of row r of a K or V block; the chunks of
// any 8 consecutive rows at one c fall in different banks (ldmatrix).
template <int HD>
AUT_DEV uint32_t row_chunk(int r, int c) {
    if constexpr (HD >= 64) return r * (HD * 2) + ((c ^ (r & 7)) << 4);
    if constexpr (HD == 32) return r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
    return r * 32 + ((c ^ ((r >> 2) & 1)) << 4);
}

// 16 bytes global -> shared, or 16 zero bytes.
AUT_DEV void copy16(uint32_t dst, const void *src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(in ? 16 : 0)
                 : "memory");
}
AUT_DEV void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
AUT_DEV void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
AUT_DEV void ldmatrix4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
AUT_DEV void ldmatrix4_trans(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
template <typename T>
AUT_DEV void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <>
AUT_DEV void mma16816<__nv_bfloat16>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                     uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
AUT_DEV void mma16816<__half>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <typename T, int HD, int W>
__global__ void __launch_bounds__(W * 32, W == kRowWarps ? 3 : 1)
    cross_rows_kernel(const __grid_constant__ CrossArgs a) {
    using Cfg = RowsCfg<HD, W>;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float2 join_ml[W][kRows];
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    // The item: from the parameters, if the list is there, while the previous
    // kernel ends.
    if (a.seqs) pdl_wait();
    const CrossSeq *seqs = a.seqs ? a.seqs : a.inline_seqs;
    const CrossSeq s = seqs[cross_find(seqs, a.n_seq, blockIdx.x, lane)];
    const int nq = s.nq, rows = nq * a.group, tiles = (rows + kRows - 1) / kRows;
    int item = (int)blockIdx.x - s.item;
    const int tile = item % tiles;
    item /= tiles;
    const int hk = item % a.heads_kv, split = item / a.heads_kv;
    const int key0 = s.k0 + split * s.keys, key1 = min(s.k0 + s.nk, key0 + s.keys);
    const int n_blocks = (key1 - key0 + kKeys - 1) / kKeys;  // 0 for a request without keys

    pdl_wait();

    // Row r of the tile: query (tile 16 + r) / group, head hk group + (tile 16 + r) % group.
    auto row_at = [&](int r, int &tok, int &head) {
        const int i = tile * kRows + r;
        tok = i / a.group;
        head = hk * a.group + i - tok * a.group;
        return i < rows;
    };
    const T *kp = static_cast<const T *>(a.k) + hk * HD, *vp = static_cast<const T *>(a.v) + hk * HD;
    uint8_t *ring = smem + warp * Cfg::kWarpBytes;
    // Which of block b's keys are read (lane i: key i).
    auto block_keys = [&](int b) -> uint32_t {
        const int key = key0 + b * kKeys + lane;
        const bool in = lane < kKeys && b < n_blocks && key < key1 && (!a.mask || a.mask[key] != 0);
        return __ballot_sync(0xffffffffu, in);
    };
    constexpr int kChunks = HD / 8;         // 16-byte chunks of a row
    constexpr int kRowsAtOnce = 32 / kChunks > 0 ? 32 / kChunks : 1;
    const int cr = lane / kChunks, cc = lane % kChunks;
    auto copy_block = [&](int b, uint32_t keys, int stage) {
        const uint32_t dst = smem_addr(ring + stage * 2 * Cfg::kTile);
        if (keys) {
#pragma unroll
            for (int r0 = 0; r0 < kKeys; r0 += kRowsAtOnce) {
                const int r = r0 + cr;
                const bool in = (keys >> r) & 1u;
                const size_t key = in ? (size_t)(key0 + b * kKeys + r) : (size_t)key0;
                copy16(dst + row_chunk<HD>(r, cc), kp + key * a.ld_k + cc * 8, in);
                copy16(dst + Cfg::kTile + row_chunk<HD>(r, cc), vp + key * a.ld_v + cc * 8, in);
            }
        }
        copy_commit();
    };

    uint32_t keys[kStages];  // of the blocks in the ring
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) {
        keys[i] = block_keys(warp + i * W);
        copy_block(warp + i * W, keys[i], i);
    }
    uint32_t ahead = block_keys(warp + (kStages - 1) * W);
    // Queries as product operands: rows g and g + 8, columns 16 c + 2 t (+ 8).
    uint32_t qf[HD / 16][4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        int tok, head;
        const bool in = row_at(g + 8 * i, tok, head);
        const T *qp = static_cast<const T *>(a.q) + (size_t)(s.q0 + (in ? tok : 0)) * a.ld_q + head * HD;
#pragma unroll
        for (int c = 0; c < HD / 16; ++c) {
            qf[c][i] = in ? *reinterpret_cast<const uint32_t *>(qp + 16 * c + 2 * t) : 0u;
            qf[c][2 + i] = in ? *reinterpret_cast<const uint32_t *>(qp + 16 * c + 2 * t + 8) : 0u;
        }
    }
    float o[HD / 8][4];
#pragma unroll
    for (int c = 0; c < HD / 8; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[c][e] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};  // rows g, g + 8; l: this lane's share

    int stage = 0;
    for (int b = warp; b < n_blocks; b += W) {
        {  // the block kStages - 1 ahead, into the stage the previous step has read
            const int fill = stage == 0 ? kStages - 1 : stage - 1;
#pragma unroll
            for (int i = 0; i < kStages; ++i)
                if (i == fill) keys[i] = ahead;
            copy_block(b + (kStages - 1) * W, ahead, fill);
            ahead = block_keys(b + kStages * W);
        }
        copy_wait<kStages - 1>();
        __syncwarp();
        uint32_t live = 0;
#pragma unroll
        for (int i = 0; i < kStages; ++i)
            if (i == stage) live = keys[i];
        const uint32_t ks = smem_addr(ring + stage * 2 * Cfg::kTile), vs = ks + Cfg::kTile;
        if (live) {
            // S: 16 rows x 16 keys, two tiles of 8 keys.
            float sc[kKeys / 8][4];
#pragma unroll
            for (int j = 0; j < kKeys / 8; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) sc[j][e] = 0.f;
#pragma unroll
            for (int j = 0; j < kKeys / 8; j += 2)
#pragma unroll
                for (int c = 0; c < HD / 16; ++c) {
                    uint32_t kf[4];  // keys 8 j .. (chunks 2 c, 2 c + 1), keys 8 j + 8 .. (the same)
                    ldmatrix4(ks + row_chunk<HD>(8 * j + (lane & 7) + (lane >> 4) * 8,
                                                 2 * c + ((lane >> 3) & 1)),
                              kf);
                    mma16816<T>(sc[j], qf[c], kf[0], kf[1]);
                    mma16816<T>(sc[j + 1], qf[c], kf[2], kf[3]);
                }
            float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int j = 0; j < kKeys / 8; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const bool in = (live >> (8 * j + 2 * t + (e & 1))) & 1u;
                    sc[j][e] = in ? sc[j][e] * a.scale_log2e : -INFINITY;
                    top[e >> 1] = fmaxf(top[e >> 1], sc[j][e]);
                }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 1));
                top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 2));
                const float mn = fmaxf(m[i], top[i]);
                // No finite score yet: 2^(-inf - 0) = 0 keeps sums and rows at zero.
                const float base = mn == -INFINITY ? 0.f : mn;
                const float shrink = ex2_approx(m[i] - base);
                m[i] = mn;
                l[i] *= shrink;
#pragma unroll
                for (int c = 0; c < HD / 8; ++c) {
                    o[c][2 * i] *= shrink;
                    o[c][2 * i + 1] *= shrink;
                }
#pragma unroll
                for (int j = 0; j < kKeys / 8; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        sc[j][2 * i + e] = ex2_approx(sc[j][2 * i + e] - (base - kCrossLift<T>));
                        l[i] += sc[j][2 * i + e];
                    }
            }
            // O += P V.  P in 16 bits: in [0, 1] (fp16: [0, 2^7]), off by half a step
            // of its type, the same rounding the output gets once more: for values
            // independent of each other the two make an error of at most sqrt(2)
            // times the output's own (one token: 1.06 to 1.11 times).  A second bf16
            // term took one token from 4.0 to 4.3 us on 390 keys and from 13.8 to 14.9
            // us on 15600.
#pragma unroll
            for (int j = 0; j < kKeys / 16; ++j) {
                const uint32_t pf[4] = {pack2<T>(sc[2 * j][0], sc[2 * j][1]),
                                        pack2<T>(sc[2 * j][2], sc[2 * j][3]),
                                        pack2<T>(sc[2 * j + 1][0], sc[2 * j + 1][1]),
                                        pack2<T>(sc[2 * j + 1][2], sc[2 * j + 1][3])};
#pragma unroll
                for (int c = 0; c < HD / 16; ++c) {
                    uint32_t vf[4];  // chunk 2 c (keys 16 j, 16 j + 8), chunk 2 c + 1 (the same)
                    ldmatrix4_trans(vs + row_chunk<HD>(16 * j + (lane & 15), 2 * c + (lane >> 4)), vf);
                    mma16816<T>(o[2 * c], pf, vf[0], vf[1]);
                    mma16816<T>(o[2 * c + 1], pf, vf[2], vf[3]);
                }
            }
        }
        __syncwarp();  // every lane has read the stage before it is filled again
        stage = stage + 1 == kStages ? 0 : stage + 1;
    }
    copy_wait<0>();
    __syncthreads();  // every warp is done with its ring; the join reuses it

    constexpr int kLd = HD + 4;
    float *join = reinterpret_cast<float *>(smem);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
        if (t == 0) join_ml[warp][g + 8 * i] = make_float2(m[i], l[i]);
#pragma unroll
        for (int c = 0; c < HD / 8; ++c)
            *reinterpret_cast<float2 *>(join + (warp * kRows + g + 8 * i) * kLd + 8 * c + 2 * t) =
                make_float2(o[c][2 * i], o[c][2 * i + 1]);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < kRows * (HD / 8); i += W * 32) {
        const int r = i / (HD / 8), c = i % (HD / 8);
        int tok, head;
        if (!row_at(r, tok, head)) continue;
        float mx = -INFINITY;
#pragma unroll
        for (int w = 0; w < W; ++w) mx = fmaxf(mx, join_ml[w][r].x);
        const float base = mx == -INFINITY ? 0.f : mx;
        float sum = 0.f, v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const float f = ex2_approx(join_ml[w][r].x - base);
            sum = fmaf(f, join_ml[w][r].y, sum);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = fmaf(f, join[(w * kRows + r) * kLd + 8 * c + e], v[e]);
        }
        if (s.splits > 1) {
            const size_t row = (size_t)s.part + ((size_t)split * nq + tok) * a.heads_q + head;
            store8(a.part_o + row * HD + 8 * c, v);
            if (c == 0) a.part_ml[row] = make_float2(mx, sum);
        } else {
            const float inv = sum == 0.f ? 0.f : 1.f / sum;  // no key: zeros
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] *= inv;
            store8(static_cast<T *>(a.out) + (size_t)(s.q0 + tok) * a.ld_out + head * HD + 8 * c, v);
        }
    }
}

// Adds the splits of every row of the split requests.  HD / 8 threads take a row's
// columns, 8 each; `groups` such teams share a row's splits (a.join_groups, a power
// of two: one team reading 49 splits one after the other took 7 us) and meet in
// shared memory, each time in the same order.
constexpr int kJoinThreads = 256;

int join_groups(int splits, int hd) {
    int g = 1;
    while (g * 2 < splits && g < kJoinThreads / (hd / 8)) g *= 2;
    return g;
}

template <typename T, int HD>
__global__ void __launch_bounds__(kJoinThreads) cross_join_kernel(const __grid_constant__ CrossArgs a) {
    constexpr int kLanes = HD / 8, kTeams = kJoinThreads / kLanes;
    __shared__ float4 team_v[kTeams][kLanes][2];
    __shared__ float2 team_ml[kTeams];
    pdl_trigger();
    if (a.seqs) pdl_wait();
    const int lane = threadIdx.x & 31, team = threadIdx.x / kLanes, c = threadIdx.x % kLanes;
    const int groups = a.join_groups, g = team % groups;
    const int first = (int)blockIdx.x * (kTeams / groups), item = first + team / groups;
    const CrossSeq *seqs = a.seqs ? a.seqs : a.inline_seqs;
    // The block's rows may belong to several requests.
    int seq = cross_find(seqs, a.n_seq, first, lane);
    const bool in = item < a.items;
    while (in && seqs[seq + 1].item <= item) ++seq;
    const CrossSeq s = seqs[seq];
    const int r = item - s.item, tok = r / a.heads_q, head = r - tok * a.heads_q;
    const int splits = in ? s.splits : 0;
    const size_t step = (size_t)s.nq * a.heads_q, row0 = (size_t)s.part + r;
    pdl_wait();
    float mx = -INFINITY, sum = 0.f, v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = 0.f;
#pragma unroll 4
    for (int i = g; i < splits; i += groups) {
        const float2 ml = a.part_ml[row0 + i * step];
        float w[8];
        load8(a.part_o + (row0 + i * step) * HD + 8 * c, w);
        const float mn = fmaxf(mx, ml.x), base = mn == -INFINITY ? 0.f : mn;
        const float f = ex2_approx(mx - base), h = ex2_approx(ml.x - base);
        mx = mn;
        sum = sum * f + ml.y * h;
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = v[e] * f + w[e] * h;
    }
    if (groups > 1) {
        team_v[team][c][0] = make_float4(v[0], v[1], v[2], v[3]);
        team_v[team][c][1] = make_float4(v[4], v[5], v[6], v[7]);
        if (c == 0) team_ml[team] = make_float2(mx, sum);
        __syncthreads();
        if (g != 0) return;
        for (int t = team; t < team + groups; ++t) mx = fmaxf(mx, team_ml[t].x);
        const float base = mx == -INFINITY ? 0.f : mx;
        sum = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = 0.f;
        for (int t = team; t < team + groups; ++t) {
            const float f = ex2_approx(team_ml[t].x - base);
            const float4 x = team_v[t][c][0], y = team_v[t][c][1];
            sum = fmaf(f, team_ml[t].y, sum);
            v[0] = fmaf(f, x.x, v[0]);
            v[1] = fmaf(f, x.y, v[1]);
            v[2] = fmaf(f, x.z, v[2]);
            v[3] = fmaf(f, x.w, v[3]);
            v[4] = fmaf(f, y.x, v[4]);
            v[5] = fmaf(f, y.y, v[5]);
            v[6] = fmaf(f, y.z, v[6]);
            v[7] = fmaf(f, y.w, v[7]);
        }
    }
    if (!in) return;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= inv;
    store8(static_cast<T *>(a.out) + (size_t)(s.q0 + tok) * a.ld_out + head * HD + 8 * c, v);
}

// -------------------------------------------------------------------- plan --

// The kernels a request may run on, and the join after them.
enum { kRowsKernel = 0, kTilesKernel = 1, kJoin = 2, kLists = 3 };

// Blocks that the row kernel's splits aim for (three a SM); the fewest keys worth a
// split of their own; and the keys a split is rounded to (whole steps of the row
// kernel's four warps; whole tiles).  One token on 15600 keys, 8 key heads of 128:
// 13.9 us with these, 16.0 us with splits of at least 512.  (Aiming for one block a
// SM, which then has eight warps, takes that single call 11.9 us; batches have not
// been measured so.)  148 SMs are the B200's: a plan asks no GPU, for the workspace
// helper needs none.
constexpr int kRowsTarget = 3 * 148;
constexpr int kMinChunk[2] = {256, 512};
constexpr int kUnit[2] = {kRowWarps * kKeys, kCrossTileKeys};

// No request of up to so many keys is split: one block then ends before a second
// kernel has joined two (390 keys, 16 heads of 64: 4.0 us whole, 4.8 us in two).
constexpr int kCrossWhole = 512;

struct CrossPlan {
    int64_t items[kLists] = {0, 0, 0};  // of each kernel; of the join: rows of split requests
    int64_t part_rows = 0;              // partial rows
    int max_splits = 1;
    int chunk[2] = {0, 0};              // most keys of a split
    bool small_call = false;            // everything on the row kernel
    bool long_prompts = false;          // some request has more than two row blocks
};

struct Splits {
    int n, keys;  // splits, and keys of each but the last
};

// A request's splits: as few as the kernel's chunk allows (at least one), as even
// as whole units of keys allow.
Splits split_keys(int nk, int kernel, const CrossPlan &p) {
    const unsigned chunk = (unsigned)p.chunk[kernel], unit = (unsigned)kUnit[kernel];  // chunk <= 2^30
    if (nk <= kCrossWhole || (unsigned)nk <= chunk) return {1, nk};
    const unsigned n = ((unsigned)nk + chunk - 1) / chunk;
    const unsigned keys = (((unsigned)nk + n - 1) / n + unit - 1) / unit * unit;
    return {(int)(((unsigned)nk + keys - 1) / keys), (int)keys};
}

// Which kernel a request runs on.  One 16-row block is the row kernel's.  Two still
// are: the second read of the keys (out of L2) costs less than the tile kernel's
// longer start (16 requests of 1500 keys, 16 heads of 64, 32 rows: 34 us against
// 44 us; 48 rows of 128: 70 us against 58 us), unless the call runs the tile kernel
// anyway: a kernel of their own then takes longer (16 prompts, one of them of 29
// rows: 55 us against 50 us).  On a small call, everything is the row kernel's.
int kernel_of(int64_t nq, int group, int hd, const CrossPlan &p) {
    const int64_t rows = nq * group;
    if (hd < 64 || p.small_call || rows <= kRows) return kRowsKernel;
    return rows <= 2 * kRows && !p.long_prompts ? kRowsKernel : kTilesKernel;
}

bool head_dim_ok(int hd) { return hd == 16 || hd == 32 || hd == 64 || hd == 128; }

aut_status check_shape(int heads_q, int heads_kv, int hd, const int32_t *cu_q, const int32_t *cu_k,
                       int n_seq) {
    if (heads_q <= 0 || heads_kv <= 0 || heads_q % heads_kv || n_seq < 0 || !cu_q || !cu_k)
        return AUT_ERR_INVALID_ARG;
    if (!head_dim_ok(hd)) return AUT_ERR_UNSUPPORTED;
    if (heads_q > (1 << 20) / hd) return AUT_ERR_UNSUPPORTED;
    if (cu_q[0] != 0 || cu_k[0] != 0) return AUT_ERR_INVALID_ARG;
    for (int i = 0; i < n_seq; ++i)
        if (cu_q[i + 1] < cu_q[i] || cu_k[i + 1] < cu_k[i]) return AUT_ERR_INVALID_ARG;
    // Row indexes (query, head of a group) and key indexes are 32-bit in the kernels,
    // a block's spare rows and a few tiles past the last key included.
    if ((int64_t)cu_q[n_seq] * heads_q > 0x7ffff000 || cu_k[n_seq] > 0x7ffff000)
        return AUT_ERR_UNSUPPORTED;
    return AUT_OK;
}

// Items of one split of a request.
int64_t split_items(int kernel, int64_t nq, int group, int heads_kv) {
    const int rows = kernel == kTilesKernel ? kCrossTileRows : kRows;
    return (nq * group + rows - 1) / rows * heads_kv;
}

// The tile kernel's chunk.  Its items run one a SM, so a few more than a whole
// number of waves cost a wave, and a split pays only if it fills the last one:
// of a few candidates, the one with the least estimated time.  An item takes 3.5 us
// and 2.05 us a tile of keys (1.95 with head_dim 64), a join 2 us and the partial
// rows' way to memory and back.  (16 heads of 128 over 8, 512 x 4096: 4 requests
// take 68 us whole, and took 90 us in the halves that an even share of the work would
// ask for; one request takes 31 us in its splits, and took 69 us whole.)
int tile_chunk(int heads_q, int heads_kv, int hd, const int32_t *cu_q, const int32_t *cu_k,
               int n_seq, CrossPlan p) {
    const int group = heads_q / heads_kv, unit = kUnit[kTilesKernel];
    int longest = 0;
    for (int i = 0; i < n_seq; ++i)
        if (kernel_of(cu_q[i + 1] - cu_q[i], group, hd, p) == kTilesKernel)
            longest = std::max(longest, cu_k[i + 1] - cu_k[i]);
    const int whole = std::max(longest, 1);
    double best = 0;
    int best_chunk = whole;
    for (int s : {1, 2, 3, 4, 6, 8, 12, 16, 24, 32, 48}) {
        p.chunk[kTilesKernel] = (int)(((int64_t)whole / s + unit) / unit * unit);
        if (s > 1 && p.chunk[kTilesKernel] < kMinChunk[kTilesKernel]) break;
        double items = 0, sum = 0, most = 0, least = 1e30, joined = 0;
        for (int i = 0; i < n_seq; ++i) {
            const int64_t nq = cu_q[i + 1] - cu_q[i];
            if (nq == 0 || kernel_of(nq, group, hd, p) != kTilesKernel) continue;
            const Splits sp = split_keys(cu_k[i + 1] - cu_k[i], kTilesKernel, p);
            const double n = (double)split_items(kTilesKernel, nq, group, heads_kv) * sp.n;
            const double us = 3.5 + (hd > 64 ? 2.05 : 1.95) * (((int64_t)sp.keys + unit - 1) / unit);
            items += n;
            sum += n * us;
            most = std::max(most, us);
            least = std::min(least, us);
            if (sp.n > 1) joined += (double)nq * heads_q * sp.n;
        }
        if (items == 0) break;
        const double waves = items / 148;
        const double us = std::max(most, sum / 148 + (std::ceil(waves) - waves) * least) +
                          (joined > 0 ? 2.0 + joined * hd * 2e-6 : 0.0);
        if (s == 1 || us < best) {
            best = us;
            best_chunk = p.chunk[kTilesKernel];
        }
        if (waves > 4) break;  // the last wave is a small part of the whole
    }
    return best_chunk;
}

// Whether the row kernel would end a call's requests of more than one row block
// before the tile kernel does.  Estimates in us from what both measured over 20 to 512 rows, 100
// to 4000 keys, 1 and 16 requests: the row kernel takes 3.3 (4.3 with head_dim
// 128) and 19 (32) ns for every key of a block, three blocks a SM; the tile kernel
// 5.2 (7) an item and 1.45 (2) a tile of keys, one item a SM, and 2 for a join.
// One request, 16 heads of 64, 128 rows: 4.6 against 10.5 us on 400 keys, 24.2
// against 16.4 us on 4000.  Of 150 calls (1, 4 and 16 requests of 24 to 512 queries on
// 100 to 4000 keys, 16 heads of 64 and of 128) 147 take the faster kernel or one
// within 8% of it, the others one within 20%.  (The constants are not tile_chunk's:
// those weigh the splits of long calls, these whole calls of about a wave.)
bool small_call(int heads_q, int heads_kv, int hd, const int32_t *cu_q, const int32_t *cu_k,
                int n_seq) {
    const int group = heads_q / heads_kv;
    double block_keys = 0, items = 0, tiles = 0, most = 0;
    for (int i = 0; i < n_seq; ++i) {
        const int64_t nq = cu_q[i + 1] - cu_q[i], nk = cu_k[i + 1] - cu_k[i];
        if (nq * group <= kRows) continue;
        const double it = (double)split_items(kTilesKernel, nq, group, heads_kv);
        const double ti = (double)((nk + kCrossTileKeys - 1) / kCrossTileKeys);
        block_keys += (double)split_items(kRowsKernel, nq, group, heads_kv) * (double)nk;
        items += it;
        tiles += it * ti;
        most = std::max(most, ti);
    }
    const bool wide = hd > 64;
    const double share = tiles / 148, whole = (double)kMinChunk[kTilesKernel] / kCrossTileKeys;
    const double rows_us =
        (wide ? 4.3 : 3.3) + (wide ? 0.032 : 0.019) * block_keys / kRowsTarget;
    const double tiles_us = (wide ? 7.0 : 5.2) * std::max(1.0, items / 148) +
                            (wide ? 2.0 : 1.45) * std::max(share, std::min(most, whole)) +
                            (most > whole ? 2.0 : 0.0);
    return rows_us < tiles_us;
}

aut_status plan_cross(int heads_q, int heads_kv, int hd, const int32_t *cu_q, const int32_t *cu_k,
                      int n_seq, CrossPlan *p) {
    const int group = heads_q / heads_kv;
    p->small_call = small_call(heads_q, heads_kv, hd, cu_q, cu_k, n_seq);
    for (int i = 0; i < n_seq; ++i)
        p->long_prompts |= (int64_t)(cu_q[i + 1] - cu_q[i]) * group > 2 * kRows;
    int64_t work = 0;  // keys read by all of the row kernel's items, unsplit
    for (int i = 0; i < n_seq; ++i) {
        const int64_t nq = cu_q[i + 1] - cu_q[i];
        if (kernel_of(nq, group, hd, *p) == kRowsKernel)
            work += split_items(kRowsKernel, nq, group, heads_kv) * (cu_k[i + 1] - cu_k[i]);
    }
    // Every split about as long as one block's share of the whole.
    const int64_t share = std::min<int64_t>((work + kRowsTarget - 1) / kRowsTarget, 1 << 30);
    const int unit = kUnit[kRowsKernel];
    p->chunk[kRowsKernel] = std::max(((int)share + unit - 1) / unit * unit, kMinChunk[kRowsKernel]);
    p->chunk[kTilesKernel] = tile_chunk(heads_q, heads_kv, hd, cu_q, cu_k, n_seq, *p);
    for (int i = 0; i < n_seq; ++i) {
        const int64_t nq = cu_q[i + 1] - cu_q[i], nk = cu_k[i + 1] - cu_k[i];
        if (nq == 0) continue;
        const int kernel = kernel_of(nq, group, hd, *p);
        const int64_t splits = split_keys((int)nk, kernel, *p).n;
        p->items[kernel] += split_items(kernel, nq, group, heads_kv) * splits;
        if (splits > 1) {
            p->items[kJoin] += nq * heads_q;
            p->part_rows += nq * heads_q * splits;
            p->max_splits = std::max(p->max_splits, (int)splits);
        }
    }
    if (p->part_rows > 0x7fffffffll) return AUT_ERR_UNSUPPORTED;
    for (int64_t n : p->items)
        if (n > 0x7fffffffll) return AUT_ERR_UNSUPPORTED;
    return AUT_OK;
}

// The requests as kernel `list` (or the join) sees them: those with items, in
// order, for the kernels those with long splits first (their blocks end together
// only if the last ones are short).  Returns how many.
int fill_seqs(CrossSeq *out, int list, const CrossPlan &p, int heads_q, int heads_kv, int hd,
              const int32_t *cu_q, const int32_t *cu_k, int n_seq) {
    constexpr int kBuckets = 64;  // of steps of keys, the first for all longer splits
    const int group = heads_q / heads_kv;
    int64_t items = 0, part = 0;
    int n = 0, first[kBuckets + 1] = {0};
    const auto bucket = [&](int keys) {
        const int unit = kUnit[list];
        const int steps = (int)(((int64_t)keys + unit - 1) / unit);
        return kBuckets - 1 - std::min(steps, kBuckets - 1);
    };
    const auto visit = [&](auto &&use) {
        part = 0;
        for (int i = 0; i < n_seq; ++i) {
            const int nq = cu_q[i + 1] - cu_q[i], nk = cu_k[i + 1] - cu_k[i];
            if (nq == 0) continue;
            const int kernel = kernel_of(nq, group, hd, p);
            const Splits s = split_keys(nk, kernel, p);
            if (list == kernel || (list == kJoin && s.n > 1))
                use(CrossSeq{cu_q[i], nq, cu_k[i], nk, 0, (int)part, s.n, s.keys});
            if (s.n > 1) part += (int64_t)nq * heads_q * s.n;
        }
    };
    if (list != kJoin) {
        visit([&](const CrossSeq &s) { ++first[bucket(s.keys) + 1]; });
        for (int b = 0; b < kBuckets; ++b) first[b + 1] += first[b];
        n = first[kBuckets];
        visit([&](const CrossSeq &s) { out[first[bucket(s.keys)]++] = s; });
    } else {
        visit([&](const CrossSeq &s) { out[n++] = s; });
    }
    for (int i = 0; i < n; ++i) {
        out[i].item = (int)items;
        items += list == kJoin ? (int64_t)out[i].nq * heads_q
                               : split_items(list, out[i].nq, group, heads_kv) * out[i].splits;
    }
    out[n] = CrossSeq{};
    out[n].item = (int)items;
    return n;
}

struct CrossLayout {
    size_t list[kLists], part_o, part_ml, total;
};
CrossLayout cross_layout(const CrossPlan &p, int hd, int n_seq) {
    CrossLayout l{};
    size_t off = 0;
    const auto take = [&](size_t bytes) {
        const size_t o = off;
        off += (bytes + 255) / 256 * 256;
        return o;
    };
    const size_t list = n_seq > kCrossInline ? ((size_t)n_seq + 1) * sizeof(CrossSeq) : 0;
    for (size_t &at : l.list) at = take(list);
    l.part_o = take((size_t)p.part_rows * hd * 4);
    l.part_ml = take((size_t)p.part_rows * 8);
    l.total = std::max<size_t>(off, 256);
    return l;
}

template <typename T, int HD, int W>
cudaError_t launch_rows(const CrossArgs &a, cudaStream_t st) {
    constexpr int smem = RowsCfg<HD, W>::kSmem;
    const cudaError_t e = smem_attr_once<cross_rows_kernel<T, HD, W>>(smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(cross_rows_kernel<T, HD, W>, dim3(a.items), dim3(W * 32), smem, st, 1, a);
}
template <typename T, int HD>
cudaError_t launch_rows(const CrossArgs &a, cudaStream_t st) {
    return a.items <= sm_count_cached() ? launch_rows<T, HD, kRowWarpsAlone>(a, st)
                                        : launch_rows<T, HD, kRowWarps>(a, st);
}

template <typename T, int HD>
cudaError_t launch_join(const CrossArgs &a, cudaStream_t st) {
    const int rows = kJoinThreads / (HD / 8) / a.join_groups;  // of a block
    return launch_pdl(cross_join_kernel<T, HD>, dim3((unsigned)((a.items + (int64_t)rows - 1) / rows)),
                      dim3(kJoinThreads), 0, st, 1, a);
}

template <typename T>
cudaError_t launch_kernel(bool join, int hd, const CrossArgs &a, cudaStream_t st) {
    switch (hd) {
        case 16: return join ? launch_join<T, 16>(a, st) : launch_rows<T, 16>(a, st);
        case 32: return join ? launch_join<T, 32>(a, st) : launch_rows<T, 32>(a, st);
        case 64: return join ? launch_join<T, 64>(a, st) : launch_rows<T, 64>(a, st);
        default: return join ? launch_join<T, 128>(a, st) : launch_rows<T, 128>(a, st);
    }
}

}  // namespace
}  // namespace aut

using namespace aut;

extern "C" size_t aut_cross_attention_workspace_bytes(int32_t heads_q, int32_t heads_kv,
                                                      int32_t head_dim, const int32_t *cu_q,
                                                      const int32_t *cu_k, int32_t n_seq) {
    CrossPlan p;
    if (check_shape(heads_q, heads_kv, head_dim, cu_q, cu_k, n_seq) != AUT_OK ||
        plan_cross(heads_q, heads_kv, head_dim, cu_q, cu_k, n_seq, &p) != AUT_OK)
        return 0;
    return cross_layout(p, head_dim, n_seq).total;
}

extern "C" aut_status aut_cross_attention(
    const void *q, int64_t ld_q, const void *k, int64_t ld_k, const void *v, int64_t ld_v,
    void *out, int64_t ld_out, int32_t dtype, int32_t heads_q, int32_t heads_kv, int32_t head_dim,
    const int32_t *cu_q, const int32_t *cu_k, int32_t n_seq, const uint8_t *key_mask, float scale,
    void *workspace, size_t ws_bytes, int32_t *status, int32_t timeout_ms, aut_stream_t stream) {
    return aut_cross_attention_ex(q, ld_q, k, ld_k, v, ld_v, out, ld_out, dtype, heads_q, heads_kv,
                                  head_dim, cu_q, cu_k, n_seq, key_mask, scale, workspace, ws_bytes,
                                  status, timeout_ms, 0, stream);
}

extern "C" aut_status aut_cross_attention_ex(
    const void *q, int64_t ld_q, const void *k, int64_t ld_k, const void *v, int64_t ld_v,
    void *out, int64_t ld_out, int32_t dtype, int32_t heads_q, int32_t heads_kv, int32_t head_dim,
    const int32_t *cu_q, const int32_t *cu_k, int32_t n_seq, const uint8_t *key_mask, float scale,
    void *workspace, size_t ws_bytes, int32_t *status, int32_t timeout_ms, int32_t flags,
    aut_stream_t stream) {
    if (flags != 0 && flags != AUT_CROSS_FAULT_K && flags != AUT_CROSS_FAULT_V)
        return AUT_ERR_INVALID_ARG;
    aut_status st = check_shape(heads_q, heads_kv, head_dim, cu_q, cu_k, n_seq);
    if (st != AUT_OK) return st;
    const float scale_log2e = (float)((double)scale * 1.4426950408889634);
    if ((dtype != AUT_BF16 && dtype != AUT_F16) || timeout_ms < 0 || !(scale > 0.f) ||
        !std::isfinite(scale_log2e))
        return AUT_ERR_INVALID_ARG;
    const int64_t tq = cu_q[n_seq], tk = cu_k[n_seq], most = (int64_t)1 << 38;
    const int64_t wq = (int64_t)heads_q * head_dim, wk = (int64_t)heads_kv * head_dim;
    if (tq > 0 && (!q || !out || ld_q < wq || ld_out < wq || ld_q > most || ld_out > most ||
                   ld_q % 8 || ld_out % 8))
        return AUT_ERR_INVALID_ARG;
    if (tk > 0 && (!k || !v || ld_k < wk || ld_v < wk || ld_k > most || ld_v > most || ld_k % 8 ||
                   ld_v % 8))
        return AUT_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k) |
         reinterpret_cast<uintptr_t>(v) | reinterpret_cast<uintptr_t>(out)) & 15u)
        return AUT_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(status) & 3u) return AUT_ERR_INVALID_ARG;
    CrossPlan p;
    st = plan_cross(heads_q, heads_kv, head_dim, cu_q, cu_k, n_seq, &p);
    if (st != AUT_OK) return st;
    const CrossLayout lay = cross_layout(p, head_dim, n_seq);
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u)) return AUT_ERR_INVALID_ARG;
    if (ws_bytes < lay.total) return AUT_ERR_WORKSPACE;
    if (flags && p.items[kTilesKernel] == 0) return AUT_ERR_UNSUPPORTED;  // no wait to run out
    if (tq == 0) return AUT_OK;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    CrossArgs a;
    a.q = q;
    a.k = k;
    a.v = v;
    a.out = out;
    a.mask = key_mask;
    a.ld_q = ld_q;
    a.ld_k = ld_k;
    a.ld_v = ld_v;
    a.ld_out = ld_out;
    a.heads_q = heads_q;
    a.heads_kv = heads_kv;
    a.group = heads_q / heads_kv;
    a.scale_log2e = scale_log2e;
    a.status = reinterpret_cast<int *>(status);
    a.timeout_ns = timeout_ms ? (unsigned long long)timeout_ms * 1000000ull : 4000ull * 1000000ull;
    a.left_out = flags == AUT_CROSS_FAULT_K ? 1 : flags == AUT_CROSS_FAULT_V ? 2 : 0;
    a.part_o = reinterpret_cast<float *>(ws + lay.part_o);
    a.part_ml = reinterpret_cast<float2 *>(ws + lay.part_ml);
    const bool listed = n_seq > kCrossInline;
    CrossSeq *list = listed ? new (std::nothrow) CrossSeq[(size_t)n_seq + 1] : a.inline_seqs;
    if (!list) return AUT_ERR_WORKSPACE;
    aut_status result = AUT_OK;
    for (int i = 0; i < kLists && result == AUT_OK; ++i) {
        if (p.items[i] == 0) continue;
        a.items = (int)p.items[i];
        a.join_groups = join_groups(p.max_splits, head_dim);
        a.n_seq = fill_seqs(list, i, p, heads_q, heads_kv, head_dim, cu_q, cu_k, n_seq);
        a.seqs = nullptr;
        if (listed) {
            CrossSeq *dev = reinterpret_cast<CrossSeq *>(ws + lay.list[i]);
            a.seqs = dev;
            if (launch_upload(reinterpret_cast<const int32_t *>(list), ((size_t)a.n_seq + 1) * (sizeof(CrossSeq) / 4),
                              reinterpret_cast<int32_t *>(dev), s) != cudaSuccess)
                result = AUT_ERR_CUDA;
        }
        if (result != AUT_OK) break;
        cudaError_t e;
        if (i == kTilesKernel)
            e = launch_cross_tiles(a, head_dim, dtype == AUT_F16, (int)tk, s);
        else if (dtype == AUT_BF16)
            e = launch_kernel<__nv_bfloat16>(i == kJoin, head_dim, a, s);
        else
            e = launch_kernel<__half>(i == kJoin, head_dim, a, s);
        if (e != cudaSuccess) result = AUT_ERR_CUDA;
    }
    if (listed) delete[] list;
    return result;
}
