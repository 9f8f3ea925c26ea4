// attention_split.cuh -- what the split decode kernel (decode_attention_scored.cu) and the shared-prefix call
// (decode_attention_shared.cu) have in common.
#pragma once

#include "attention_scores.cuh"

namespace pkv {

// Groups of sequences with a shared prefix, as the call has them.
struct GroupArgs {
    const int32_t* start;   // [N + 1]
    const int32_t* shared;  // [N]
    int N;
};

// How a call is laid out; computed on the host.
struct SplitPlan {
    int HG, NG;      // KV heads per group, groups (the last one may have fewer heads)
    int QC;          // chunks of query heads per KV head (8 or 16 heads each)
    int slots;       // a step is slots x kSub units along the cache
    int units;       // units a step
    int R;           // query rows per group: HG * G
    int UB;          // units of 16 positions per block
    int nst;         // ring stages
    int stage_bytes, q_bytes, scratch_bytes;
    int qslots;      // sequences' queries in shared memory
    int direct;      // one CTA per (sequence, group), no join
    int B, Hq, Hkv, G, D, BS, NB, max_blocks;
    ScoreArgs sc;
    GroupArgs groups;
    uint32_t polls;
    int silent_cta;
};
// Units of a step that a warp takes: steps of about 64 KB.
__host__ __device__ constexpr int split_sub(int DP) { return DP <= 64 ? 2 : 1; }

// A range that begins inside a piece: the sequence and head group, the piece's first range and the ranges it spans
// (0: nothing to join here).
struct SplitCut {
    int b, g, f, pieces;
};
struct SplitHead {
    int W;  // steps per range (shared prefixes only)
};
struct SplitSpace {
    SplitHead* head;
    SplitCut* cuts;  // one per range
    int2* info;      // shared prefixes: (first step, steps per head group) of every sequence
    float2* ml;      // (max, sum) of every partial result
    float* o;        // its sums of products
};

// Whether group g's bounds can be those of a group (all groups': start is an array of such).
__device__ __forceinline__ bool group_valid(const GroupArgs& ga, int B, int g) {
    const int s = ga.start[g], e = ga.start[g + 1];
    return s <= e && s >= 0 && e <= B && (g > 0 || s == 0);
}
// The group of sequence b, -1 where it has none (start non-decreasing).
__device__ __forceinline__ int group_of(const GroupArgs& ga, int b) {
    int lo = 0, hi = ga.N;
    if (hi == 0 || b < ga.start[0] || b >= ga.start[hi]) return -1;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (ga.start[mid] <= b) lo = mid;
        else hi = mid;
    }
    return lo;
}
// Positions of the prefix that group g reads once: whole blocks, 0 for groups of one; -1 where the shared length is
// outside the table.
__device__ __forceinline__ int group_prefix(const GroupArgs& ga, int max_blocks, int BS, int g) {
    const int shared = ga.shared[g];
    if (shared < 0 || static_cast<long long>(shared) > static_cast<long long>(max_blocks) * BS) return -1;
    return ga.start[g + 1] - ga.start[g] > 1 ? shared / BS * BS : 0;
}
__device__ __forceinline__ int shared_prefix(const GroupArgs& ga, int max_blocks, int BS, int b) {
    const int g = group_of(ga, b);
    return g < 0 ? 0 : group_prefix(ga, max_blocks, BS, g);
}

}  // namespace pkv
