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
    int TQ;  // members of a group in a tile of 128 rows (shared prefixes)
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

// Positions of the prefix that a group of n with this shared length reads once; 0 where the length is none.
__device__ __forceinline__ int group_prefix_of(int n, int shared, int max_blocks, int BS) {
    return n > 1 && shared > 0 && static_cast<long long>(shared) <= static_cast<long long>(max_blocks) * BS ? shared / BS * BS : 0;
}

// What a call over shared prefixes has to do, and how its two kernels divide the SMs.  One after the other, the second pays
// its start (lengths, block ids, first tiles) and each leaves idle what the other would use: the prefixes the tensor
// cores, the sequences' own positions HBM.  So where the estimate says that it gains, `own_ctas` SMs take the own positions
// from the beginning, and the prefix kernel leaves them free.
// The estimate, in us, was fitted to 40 batches: the start, 4 a piece and 0.65 (capped 1.15) a tile of 64 keys and 128 rows
// for a prefix CTA; the start, 4 a piece and 0.8 (capped 1.04) a step for an own one.  Together only where that is below 85%
// of one after the other, whose overlap it does not know.  One group of 64 behind 8192 with 64-1024 of their own, 32 and 8
// heads of 128: 52 us for 67; 6 of 3 behind 11667, 56 and 8 heads of 64: 51 for 58; a batch that stays as it was pays 1
// us for the estimate.  With more than 8 query heads a KV head the steps take anything from 1 to 5 us, and the estimate
// lost as often as it gained: those stay one after the other.
__host__ __device__ constexpr bool shares_sms(int G) { return G <= 8; }
struct SharedWork {
    int behind = 0;  // units of 16 positions behind the prefixes
    int tiles = 0;   // the prefixes' key tiles, of one KV head
    int halves = 0;  // the same, those of more than 128 rows counted twice

    __device__ __forceinline__ void group(int from, int to, int shared, int max_blocks, int BS, int TQ) {
        const int n = to - from, prefix = group_prefix_of(n, shared, max_blocks, BS);
        if (prefix == 0) return;
        const int nt = (prefix + 63) / 64, rows = (n + TQ - 1) / TQ;
        tiles += (rows + 1) / 2 * nt;
        halves += rows * nt;
        behind -= n * (prefix / 16);
    }
    __device__ __forceinline__ void sequence(int L, int max_blocks, int BS) {
        if (L > 0 && static_cast<long long>(L) <= static_cast<long long>(max_blocks) * BS) behind += L / 16;
    }
    // The CTA's sum: put, a barrier, get; at: three ints per warp.
    __device__ __forceinline__ void put(int* at, int warp, int lane) {
        const int a = __reduce_add_sync(0xffffffffu, behind), b = __reduce_add_sync(0xffffffffu, tiles),
                  c = __reduce_add_sync(0xffffffffu, halves);
        if (lane == 0) {
            at[3 * warp] = a;
            at[3 * warp + 1] = b;
            at[3 * warp + 2] = c;
        }
    }
    __device__ __forceinline__ void get(const int* at, int warps, int lane) {
        const bool in = lane < warps;
        behind = __reduce_add_sync(0xffffffffu, in ? at[3 * lane] : 0);
        tiles = __reduce_add_sync(0xffffffffu, in ? at[3 * lane + 1] : 0);
        halves = __reduce_add_sync(0xffffffffu, in ? at[3 * lane + 2] : 0);
    }
    // CTAs of P for the own positions, 0: all take the prefixes and then those.  A whole warp calls it: its lanes try 32
    // numbers.  Both kernels give the same arguments.
    __device__ __forceinline__ int own_ctas(int P, int B, int N, int Hkv, int NG, int units, bool cap, int lane) const {
        if (behind <= 0 || tiles <= 0) return 0;
        const float pieces = static_cast<float>(NG) * static_cast<float>(B);
        const float steps = static_cast<float>(NG) * __fdividef(static_cast<float>(behind), static_cast<float>(units)) + 0.5f * pieces;
        const float all_tiles = static_cast<float>(Hkv) * static_cast<float>(tiles);
        const float tile = __fdividef((cap ? 1.15f : 0.65f) * static_cast<float>(halves), static_cast<float>(tiles));
        const float step = cap ? 1.04f : 0.8f;
        const float tile_pieces = __fdividef(static_cast<float>(N), static_cast<float>(tiles)), step_pieces = __fdividef(pieces, steps);
        auto prefixes = [&](int n) {
            const float w = fmaxf(2.f, ceilf(__fdividef(all_tiles, static_cast<float>(n))));
            return 10.f + w * (tile + 4.f * tile_pieces);
        };
        auto own = [&](int n) {
            const float w = ceilf(__fdividef(steps, static_cast<float>(n)));
            return 8.f + w * (step + 4.f * step_pieces);
        };
        const int e = P * (lane + 1) / 40;  // up to 4/5 of them
        const float t = e > 0 ? fmaxf(prefixes(P - e), own(e) + 3.f) : INFINITY;
        const unsigned best = __reduce_min_sync(0xffffffffu, __float_as_uint(t));
        const int at = __ffs(__ballot_sync(0xffffffffu, __float_as_uint(t) == best)) - 1;
        return __uint_as_float(best) < 0.85f * (prefixes(P) + own(P)) ? P * (at + 1) / 40 : 0;
    }
};

}  // namespace pkv
