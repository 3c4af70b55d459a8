// Cross attention: what its host plan hands to its kernels.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace aut {

// Up to kCrossInline requests travel in the kernels' parameters (one launch
// less); longer lists are uploaded to the workspace.
constexpr int kCrossInline = 512;

// One request as one kernel sees it; entry n closes the list.  Its work items
// are item .. next item: [split][key head][row tile].  With more than one
// split its partial results start at row `part` of the partial buffer:
// [split][query][query head].
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
    int chunk;        // keys of a split (a request has ceil(keys / chunk) of them, at least one)
    int n_seq, items;
    float *part_o;    // [partial rows][head_dim], fp32, over each split's own row maximum
    float2 *part_ml;  // that maximum (times scale_log2e) and the sum of 2^(s - max)
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

}  // namespace aut
