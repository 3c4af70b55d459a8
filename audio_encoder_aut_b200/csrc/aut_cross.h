// Cross attention: what its host plan hands to its kernels.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace aut {

// Up to kCrossInline requests travel in the kernels' parameters (one launch
// less); longer lists are uploaded to the workspace.
constexpr int kCrossInline = 512;

// One request as one kernel sees it; entry n closes the list.  Its work items
// are item .. next item (none, if another kernel handles it): [split][key
// head][row tile].  With more than one split its partial results are rows
// part .. next part of the partial buffer: [split][query][query head].
struct CrossSeq {
    int q0, k0, item, part;
};

struct CrossArgs {
    const void *q, *k, *v;
    void *out;
    const uint8_t *mask;
    long long ld_q, ld_k, ld_v, ld_out;  // elements
    int heads_q, heads_kv, group;
    float scale_log2e;
    int chunk;        // most keys of a split
    int unit;         // its keys come in multiples of this
    int n_seq, items;
    int join_groups;  // of the join: teams that share a row's splits
    float *part_o;    // [partial rows][head_dim], fp32, over each split's own row maximum
    float2 *part_ml;  // that maximum (times scale_log2e) and the sum of 2^(s - max)
    int *status;
    unsigned long long timeout_ns;
    const CrossSeq *seqs;  // in the workspace; null: `inline_seqs`
    CrossSeq inline_seqs[kCrossInline + 1];
};

// No request of up to so many keys is split: one block then ends before a second
// kernel has joined two (390 keys, 16 heads of 64: 4.9 us whole, 6.2 us in two).
constexpr int kCrossWhole = 512;

// A request's splits: as few as `chunk` allows (at least one), as even as whole
// units of keys allow.
struct CrossSplits {
    int n, keys;  // splits, and keys of each but the last
};
__host__ __device__ inline CrossSplits cross_splits(int nk, int chunk, int unit) {
    if (nk <= chunk || nk <= kCrossWhole) return {1, nk};
    const unsigned n = ((unsigned)nk + (unsigned)chunk - 1) / (unsigned)chunk;  // chunk <= 2^30
    const unsigned keys = (((unsigned)nk + n - 1) / n + unit - 1) / unit * unit;
    return {(int)(((unsigned)nk + keys - 1) / keys), (int)keys};
}

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
