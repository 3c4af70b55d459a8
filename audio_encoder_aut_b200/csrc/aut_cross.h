// Cross attention: what its host plan hands to its kernels.
#pragma once

#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

namespace aut {

// Up to kCrossInline requests travel in the kernels' parameters; longer lists are
// uploaded to the workspace, a launch for each kernel that reads one, and blocks then
// look their item up only once that has ended: 257 requests of one token take 27.7 us
// on 100 keys each and 39.5 us on 6 to 780, 256 take 26.0 and 36.9 us.  Not more, since
// every launch, of one request too, carries the whole list (8 KB).
constexpr int kCrossInline = 256;

// The kernels' probabilities are 2^(s - reference + lift), which cancels in O / sum.
// fp16 ends at 2^-24 and weights below half of that would drop out of P V (but not out
// of the sum, which is fp32): many such weights together are no small part of a long
// row. Lifted by 2^7 those from 2^-32 of the maximum on count; the tile kernel's
// reference may be 2^8 too low, and 2^15 is within fp16's range. bf16 has fp32's.
template <typename T>
constexpr float kCrossLift = std::is_same<T, __half>::value ? 7.f : 0.f;

// One request as one kernel sees it; the entry behind the last one only has `item`.
// Its work items are item .. next item (none, if another kernel handles it):
// [split][key head][row tile].  With more than one split its partial results start
// at row `part` of the partial buffer: [split][query][query head].
struct CrossSeq {
    int q0, nq, k0, nk;  // first row and rows of its queries and keys
    int item, part;
    int splits, keys;    // splits, and keys of each but the last
};

struct CrossArgs {
    const void *q, *k, *v;
    void *out;
    const uint8_t *mask;
    long long ld_q, ld_k, ld_v, ld_out;  // elements
    int heads_q, heads_kv, group;
    float scale_log2e;
    int n_seq, items;
    int join_groups;  // of the join: teams that share a row's splits
    float *part_o;    // [partial rows][head_dim], fp32, over each split's own row maximum
    float2 *part_ml;  // that maximum (times scale_log2e) and the sum of 2^(s - max)
    int *status;
    unsigned long long timeout_ns;
    int left_out;  // tests: 1 + the tile kernel's first block's copy that never starts
    const CrossSeq *seqs;  // in the workspace; null: `inline_seqs`
    CrossSeq inline_seqs[kCrossInline + 1];
};

// The item's request: the last one that begins at or before `item`.  The whole
// warp searches, 32 probes a round.
__device__ __forceinline__ int cross_find(const CrossSeq *seqs, int n_seq, int item, int lane) {
    int lo = 0, n = n_seq;
    while (n > 1) {
        const int step = (n + 31) >> 5;
        const int at = lane * step;
        const bool before = at < n && seqs[lo + at].item <= item;
        const int last = 31 - __clz(__ballot_sync(0xffffffffu, before));  // probe 0 always is
        lo += last * step;
        n = min(step, n - last * step);
    }
    return lo;
}

// The tcgen05 kernel (aut_cross_tc.cu), for head_dim 64 and 128: kCrossTileRows
// rows (query, head of the group) a block, keys in tiles of 128.
constexpr int kCrossTileRows = 256;
constexpr int kCrossTileKeys = 128;
// tk: rows of k and v.  f16: the element type (bf16 otherwise).
cudaError_t launch_cross_tiles(const CrossArgs &a, int head_dim, bool f16, int tk, cudaStream_t st);

}  // namespace aut
