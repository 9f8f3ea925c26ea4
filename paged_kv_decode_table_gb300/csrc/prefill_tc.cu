// prefill_tc.cu -- chunked-prefill attention on the fifth-generation tensor
// cores: tcgen05 MMAs with accumulators in tensor memory (TMEM), operands
// staged in shared memory by TMA.  Same results as prefill_attn_kernel (the
// chunk's causal GQA attention over the paged cache; "Suy luan & Toi uu hoa
// (Inference)" 2.1 and 4.1, the lab's prefill step, "LLM inference serving
// tutorial" 5.4) for bf16, D = 128, G = Hq / Hkv from 1 to 8, block_size a
// multiple of 16 and 16-byte aligned q / out / pools.
//
//  * One CTA per (two query tiles of 128 rows, KV head h).  Row r of query
//    tile t is (chunk token t TQ + r / G, query head h G + r % G), TQ =
//    floor(128 / G): 2 TQ consecutive tokens of one sequence times the G heads
//    that share K/V head h, so each K/V tile serves up to 256 rows (rows TQ G
//    .. 127 of a tile, when G does not divide 128, are padding: computed on
//    zero queries and not stored).  The CTAs take the chunk tiles
//    longest first (by the number of key tiles they read; the KV head is the
//    innermost grid index), so that the longest start in the first wave.
//  * K and V of head h stream in 64-key tiles through a five-stage ring.  The
//    paged layout allows TMA boxes of one block's 16 keys at most.  K comes in
//    one 4 KB box per 16 keys through a 4-D view of the pool that lands the
//    two 64-dimension halves interleaved at 1 KB, so that for either half the
//    8-row groups of the tile sit 2 KB apart (one N = 64 MMA per k-step); V in
//    one 4 KB box per 16 keys (a 3-D view, both halves, one box per PV k-step).
//    Three producer warps issue a tile's eight boxes, each on its own (its
//    own window of the block table in shared memory, its own arrival on the
//    stage's barrier).  Each CTA walks its key tiles starting at a different
//    tile, so that the CTAs sharing a sequence do not read the same blocks at
//    the same time.
//  * Tensor memory, per query tile t (256 columns): Q (bf16, two per column)
//    at 256 t, S at 256 t + 64, O at 256 t + 128.  One warp issues
//    S = Q K^T (M 128, N 64, K 128; A = Q from tensor memory, B = K from the
//    stage), another O += P V (M 128, N 128, K 64; A = P from a K-major,
//    128-byte-swizzled shared tile per query tile, B = V as stored, MN-major,
//    one 16-key group per k-step).  The softmax releases S as soon as it has
//    read it, so S of tile j + 1 runs during the softmax of tile j; P of tile
//    j + 1 is written once the PV of tile j is complete.  The two query tiles
//    interleave on the tensor pipe.  Completion is signalled through
//    mbarriers (tcgen05.commit).
//  * Eight softmax warps, four per query tile: thread r owns row r (TMEM lane
//    r).  It reads its 64 scores (tcgen05.ld), applies the causal mask and the
//    scale in the log2 domain, and exponentiates against a reference maximum
//    that is raised only when the row maximum exceeds it by more than 8, in
//    which case the row of O in TMEM and the running sum are rescaled first;
//    P (bf16, values at most 2^8) goes to shared memory for the PV MMA, and
//    the sum accumulates the fp32 values.  Rows past the chunk are
//    computed on zero queries and not stored.  The V rows of the last tile's
//    keys past the CTA's last position (which may hold anything, NaN included)
//    are cleared before the last PV MMAs.
//  * Epilogue: O / sum from TMEM to the bf16 output rows.
// Every mbarrier wait is bounded; a CTA that gives up records PKV_ERR_TIMEOUT,
// waits (bounded) for its own TMA copies and MMAs, frees its TMEM, and sets the
// rows that it did not finish to zero.
#include <cuda.h>
#include <math.h>

#include <algorithm>

#include "tensor_core.cuh"

namespace pkv {

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn get_encode_fn();
uint32_t attention_wait_polls();
int attention_silent_cta();
bool encode_pool_box_halves(CUtensorMap* map, const void* pool, int NB, int Hkv, int BS, int box_rows);

constexpr int kTcDim = 128;
constexpr int kTcRows = 128;                 // query rows per query tile (TMEM lanes)
constexpr int kTcQT = 2;                     // query tiles per CTA, sharing every K/V tile
constexpr int kTcKeys = 64;                  // keys per tile
constexpr int kTcStages = 5;                 // K/V ring depth
constexpr int kTcPBytes = kTcRows * kTcKeys * 2;          // 16 KB: P of one query tile, one atom of 128 rows
constexpr int kTcKBytes = kTcKeys * kTcDim * 2;           // 16 KB per operand tile
constexpr int kTcGroupBytes = 16 * kTcDim * 2;            // 4 KB: 16 keys x 128 dimensions
constexpr int kTcStageBytes = 2 * kTcKBytes;              // K then V
constexpr int kTcProd = 3;                   // producer warps
constexpr int kTcWin = 640;                  // block-table entries kept in shared memory, per producer warp
// warps 0-7: softmax (warp w: query tile w / 4, TMEM lanes 32 (w % 4) ..); warps 8,
// 11 and 12: producers; warp 9: S MMAs (and the TMEM allocation); warp 10: PV MMAs
constexpr int kTcWarpProd = 8, kTcWarpS = 9, kTcWarpPV = 10;
constexpr int kTcThreads = 13 * 32;
// With changed scores a softmax thread needs more than the 128 registers that 13 warps leave it: 16 warps (13-15 idle),
// which can pass theirs on by warpgroup.
constexpr int kTcScoredThreads = 16 * 32;
enum : int { kPlain = 0, kMasked = 1, kCapped = 2, kSloped = 4 };
constexpr int kTcTmemCols = 512;             // query tile t: Q at 256 t, S at 256 t + 64, O at 256 t + 128

struct TcSmem {  // follows the 1024-aligned operand area
    uint64_t kv_full[kTcStages], kv_empty[kTcStages];
    uint64_t s_full[kTcQT], s_free[kTcQT], p_full[kTcQT], o_done[kTcQT];
    uint64_t last[2];  // of a thread that leaves: its MMAs are complete
    uint32_t tmem_base;
    int b, tile, bad;
    int tbl[kTcProd][kTcWin];
};
constexpr size_t kTcOperandBytes = kTcQT * static_cast<size_t>(kTcPBytes) + kTcStages * static_cast<size_t>(kTcStageBytes);
constexpr size_t kTcSmemBytes = 1024 + kTcOperandBytes + sizeof(TcSmem);
static_assert(kTcSmemBytes <= 227 * 1024, "shared memory of one CTA");

__device__ __forceinline__ int warp_sum_i(int x) { return __reduce_add_sync(0xffffffffu, x); }
__device__ __forceinline__ int warp_max_i(int x) { return __reduce_max_sync(0xffffffffu, x); }
// Chunk tiles of one sequence (n chunk tokens, length L after the chunk, TC
// tokens per tile) that read more than v key tiles.  Full tile c reads up to
// position L - n + TC (c + 1) - 1, the last tile up to L - 1; the count grows
// with c.  L below n (an invalid length, reported by the CTA that owns the
// tile) is taken as n, so that the order is defined for any input.
__device__ __forceinline__ int tc_tiles_longer(int n, int L, int TC, int v) {
    if (n <= 0) return 0;
    const int tiles = (n + TC - 1) / TC;
    const long long Lc = max(L, n), P = Lc - n;
    int cnt = (Lc - 1) / kTcKeys + 1 > v ? 1 : 0;
    const long long x = static_cast<long long>(kTcKeys) * v - P + 1;  // full tile c qualifies iff TC (c + 1) >= x
    const int cmin = x <= 0 ? 0 : static_cast<int>((static_cast<unsigned>(x) + TC - 1) / static_cast<unsigned>(TC)) - 1;
    cnt += max(0, tiles - 1 - cmin);
    return cnt;
}

// The 64 products of a row with the keys from kbase on become scores in the log2 domain (without cap and slopes they stay
// products, which the softmax scales), -infinity where the row at position `pos` does not see the key.  from: the key that the
// row's bias is measured from; first, last: the positions of the query tile's rows; slope: of the row's head, times log2(e).
template <int kKind>
__device__ __forceinline__ void score_tile(uint32_t (&sr)[2][32], int kbase, int pos, int from, int first, int last, int pfx,
                                           float slope, const ScoreArgs& sc) {
    if constexpr ((kKind & (kCapped | kSloped)) != 0)
        tc_scores<(kKind & kCapped) != 0, (kKind & kSloped) != 0>(sr, kbase - from, slope, sc);
    // some key is hidden from some row of the query tile
    if (kbase + kTcKeys > pfx && (kbase + kTcKeys - 1 > first || (sc.window > 0 && kbase <= last - sc.window))) {
        const int lo = sc.window > 0 ? pos - sc.window + 1 - kbase : -kbase, hi = pos - kbase, near = pfx - kbase;
#pragma unroll
        for (int c = 0; c < kTcKeys; ++c)
            if (!(c < near || (c <= hi && c >= lo))) sr[c >> 5][c & 31] = __float_as_uint(-INFINITY);
    }
}

// The eight softmax warps.
__device__ __forceinline__ void softmax_barrier() { asm volatile("barrier.sync 1, 256;" ::: "memory"); }

// Few query tiles over long key ranges (scored): S CTAs take a share of a pair of query tiles' keys each and leave
// maxima, sums and float32 O of their rows, [T_new * Hq][S], to prefill_join_kernel.
struct TcSplit {
    int S;
    float2* ml;
    float* o;
};
// Polls of a wait, and the CTA whose loaders issue no copy (test hook).
struct TcWaits {
    uint32_t polls;
    int silent_cta;
};

// What bounds it: the chain of a query tile (S from tensor memory, scores, maximum, exponentials, P to shared memory, PV),
// which only the other query tile hides: two softmax warps a scheduler, and no pipe near full by the counters.  A tile of 64 keys
// and 256 rows takes 2000-2300 clocks plain, 2800 with slopes, 3500 capped (eight FMAs a score).  8 chunks of 256-512
// behind 512-4096 (32 and 8 heads): plain 109 us (tensor pipe 33% busy, issue slots 31%), slopes 132 (25%, 38%), capped 166 (20%,
// 39%; FMA pipe 31%).  16 such chunks: 258 us plain, 368 with every score capped; 4 of up to 2048 behind 16384-32768 that see
// 1024 + 100 positions, with slopes, 412 (109 at the measured bf16 rate).
// Of a plain tile the MMAs, one after the other, are 1900 clocks: with M 128, K 16 one takes 84 with A in tensor memory (N 64; 88
// for N 128), 70 with A in shared memory (N 128), and there are 16 of S and 8 of PV.  Q in shared memory (52 clocks an MMA of S)
// was no way out: shared memory then carries 224 KB a tile at 118 bytes a clock, 1900 again, and the ring is two stages
// shorter (16 chunks of 512 behind 512-4096: 354 us where the layout kept took 311 then and takes 279 now).
// kKind: kPlain, or kMasked (the masks of attention_scores.cuh) with kCapped and kSloped where its scores are.
template <int kKind>
__global__ void __launch_bounds__(kKind == kPlain ? kTcThreads : kTcScoredThreads, 1)
    prefill_tc_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                      const __nv_bfloat16* q, __nv_bfloat16* out,
                      const int32_t* block_tables, int max_blocks, const int32_t* seq_lens,
                      const int32_t* q_start, int B, int Hq, int Hkv, int BS, int NB, float scale_log2,
                      const __grid_constant__ ScoreArgs sc, const __grid_constant__ TcSplit split,
                      const __grid_constant__ TcWaits waits, int32_t* status) {
    constexpr bool kScored = kKind != kPlain;
    const int S = kScored ? split.S : 1;  // CTAs along the keys of a pair of query tiles
    extern __shared__ uint8_t tc_raw[];
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(tc_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sP = base;                          // P of query tile t at t kTcPBytes
    uint8_t* sKV = base + kTcQT * kTcPBytes;
    TcSmem* sm = reinterpret_cast<TcSmem*>(base + kTcOperandBytes);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = Hq / Hkv, h = static_cast<int>(blockIdx.x) % Hkv;
    const int TQ = kTcRows / G;    // chunk tokens per query tile (rows TQ G .. 127 are padding)
    const int TC = kTcQT * TQ;     // chunk tokens per CTA
    [[maybe_unused]] const int share = kScored ? static_cast<int>(blockIdx.x) / Hkv % S : 0;

    // ---- prologue, independent of the inputs
    if (tid == 0) {
        for (int s = 0; s < kTcStages; ++s) {
            mbar_init(&sm->kv_full[s], kTcProd);  // one arrival (with its bytes) per producer warp
            mbar_init(&sm->kv_empty[s], 1);
        }
        for (int t = 0; t < kTcQT; ++t) {
            mbar_init(&sm->s_full[t], 1);
            mbar_init(&sm->s_free[t], kTcRows);
            mbar_init(&sm->p_full[t], kTcRows);
            mbar_init(&sm->o_done[t], 1);
            mbar_init(&sm->last[t], 1);
        }
        fence_mbar_init();
        prefetch_tmap(&tmK);
        prefetch_tmap(&tmV);
        sm->b = -1;
        sm->tile = 0;
        sm->bad = 0;
    }
    if (warp == kTcWarpS) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(&sm->tmem_base)),
                     "r"(kTcTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the chunk's K/V are in the cache
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __syncthreads();
    if (warp == 0) {
        // This CTA's chunk tile: the one of rank k when the chunk tiles of all
        // sequences are ordered by their number of key tiles, longest first (ties:
        // sequence order, then tile order), so that the longest start in the first
        // wave.  v = the rank's key-tile count, found by bisection on the counts.
        const int k = static_cast<int>(blockIdx.x) / Hkv / S;
        int total = 0, vmax = 0;
        for (int b0 = 0; b0 < B; b0 += 32) {
            const int bb = b0 + lane;
            if (bb < B) {
                const int n = q_start[bb + 1] - q_start[bb];
                if (n > 0) {
                    total += (n + TC - 1) / TC;
                    vmax = max(vmax, (max(seq_lens[bb], n) - 1) / kTcKeys + 1);
                }
            }
        }
        total = warp_sum_i(total);
        vmax = warp_max_i(vmax);
        if (k < total) {
            auto longer = [&](int v) {  // chunk tiles (all sequences) with more than v key tiles
                int c = 0;
                for (int bb = lane; bb < B; bb += 32) c += tc_tiles_longer(q_start[bb + 1] - q_start[bb], seq_lens[bb], TC, v);
                return warp_sum_i(c);
            };
            int lo = 1, hi = vmax;  // the smallest v with longer(v) <= k
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (longer(mid) <= k) hi = mid;
                else lo = mid + 1;
            }
            const int v = lo;
            int idx = k - longer(v);  // among the tiles with exactly v key tiles, in sequence order
            for (int b0 = 0; b0 < B; b0 += 32) {
                const int bb = b0 + lane;
                int e = 0, first = 0;
                if (bb < B) {
                    const int n = q_start[bb + 1] - q_start[bb], L = seq_lens[bb];
                    const int ge = tc_tiles_longer(n, L, TC, v - 1);
                    e = ge - tc_tiles_longer(n, L, TC, v);
                    first = (n > 0 ? (n + TC - 1) / TC : 0) - ge;  // the counts grow along the chunk
                }
                int inc = e;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, inc, o);
                    if (lane >= o) inc += y;
                }
                const int ex = inc - e;
                if (e > 0 && ex <= idx && idx < inc) {
                    sm->b = bb;
                    sm->tile = first + (idx - ex);
                }
                const int tot = __shfl_sync(0xffffffffu, inc, 31);
                if (idx < tot) break;
                idx -= tot;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm->tmem_base;
    const int b = sm->b, tile = sm->tile;
    bool active = b >= 0;  // a spare CTA of the upper-bound grid has no tile
    int n = 0, L = 0, t0 = 0, nt = 0, p0 = 0;
    if (active) {
        n = q_start[b + 1] - q_start[b];
        L = seq_lens[b];
        t0 = q_start[b] + TC * tile;
        nt = min(TC, n - TC * tile);
        p0 = L - n + TC * tile;  // position of the CTA's first token
    }
    const bool bad_len = active && (L < n || static_cast<long long>(L) > static_cast<long long>(max_blocks) * BS);
    // this thread's row (softmax warps): query tile qt, row r = token tl of the CTA, query head qh
    const bool softmax_warp = warp < 4 * kTcQT;
    const int qt = warp >> 2, r = tid & (kTcRows - 1);
    // scored: where all rows fit into one query tile, both hold them: tile t takes every other key tile from t on, and the
    // epilogue joins the two.  Two chains of products and softmax over half the keys each, instead of one over padding: 9
    // sequences of 2 tokens behind 141-8220, 15 and 5 heads, capped 49 us for 77; 29 of 6 behind 1216-1541, 63 and 9 77 for
    // 131.  (Barriers then count the key tiles of a query tile, u.)
    const bool dual = kScored && active && nt <= TQ;
    const int tl = (dual ? 0 : qt * TQ) + r / G, qh = h * G + r % G;
    const bool row_valid = active && softmax_warp && r < TQ * G && tl < nt;  // rows TQ G .. 127: padding
    if (bad_len) {
        if (tid == 0) report(status, PKV_ERR_DEVICE_BOUNDS);
        if (row_valid && S > 1) {  // a share that cannot be read makes the row zero
            split.ml[(static_cast<size_t>(t0 + tl) * Hq + qh) * S + share] = make_float2(-INFINITY, -1.f);
        } else if (row_valid) {
            uint4* o = reinterpret_cast<uint4*>(out + (static_cast<size_t>(t0 + tl) * Hq + qh) * kTcDim);
            for (int c = 0; c < 16; ++c) o[c] = make_uint4(0u, 0u, 0u, 0u);
        }
        active = false;
    }
    // scored: keys below pfx are seen by every row, keys below wlo (and not below pfx) by no row of the CTA
    [[maybe_unused]] int pfx = 0, wlo = 0;
    if constexpr (kScored) {
        if (active && sc.prefix_lens != nullptr) pfx = min(max(sc.prefix_lens[b], 0), L);
        if (active && sc.window > 0) wlo = max(0, p0 - sc.window + 1);
    }
    const int plast = max(p0 + nt, pfx) - 1;          // the CTA's last key (keys 0 .. plast are read)
    // key tile i of the walk is tile i, behind the prefix's tiles (near) tile i + skip
    [[maybe_unused]] const int near = (pfx + kTcKeys - 1) / kTcKeys, skip = max(0, wlo / kTcKeys - near);
    const int nall = active ? plast / kTcKeys + 1 - (kScored ? skip : 0) : 0;
    // this CTA's share of them: [first, first + ntiles)
    const int first = kScored ? static_cast<int>(static_cast<long long>(nall) * share / S) : 0;
    const int ntiles = kScored ? static_cast<int>(static_cast<long long>(nall) * (share + 1) / S) - first : nall;
    auto key_tile = [&](int i) { return kScored ? (i + first >= near ? i + first + skip : i + first) : i; };
    // iteration j handles key tile (j + rot) mod ntiles (any order gives the same softmax)
    const int rot = ntiles > 0 ? static_cast<int>((blockIdx.x * 13u) % static_cast<unsigned>(ntiles)) : 0;
    const int nblk_used = active ? plast / BS + 1 : 0;
    const int pos = row_valid ? p0 + tl : plast;      // the row's position (rows past the chunk: the last)

    // ---- the query tiles: row r of tile qt into TMEM lane r, columns 256 qt .. + 63 (two
    // bf16 per column; rows past the chunk: zeros), the A operand of S = Q K^T
    if (active && softmax_warp) {
        const uint4* src = reinterpret_cast<const uint4*>(q + (static_cast<size_t>(t0 + (row_valid ? tl : 0)) * Hq + qh) * kTcDim);
        const uint32_t lrow = static_cast<uint32_t>((warp & 3) * 32) << 16;
#pragma unroll
        for (int hv = 0; hv < 2; ++hv) {
            uint32_t w[32];
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const uint4 v = row_valid ? src[8 * hv + c] : make_uint4(0u, 0u, 0u, 0u);
                w[4 * c] = v.x;
                w[4 * c + 1] = v.y;
                w[4 * c + 2] = v.z;
                w[4 * c + 3] = v.w;
            }
            tc_st32(tmem + 256 * qt + lrow + 32 * hv, w);
        }
    }
    tc_fence_before();
    if (softmax_warp || warp == kTcWarpS) asm volatile("barrier.sync 2, 288;" ::: "memory");  // Q is there; the producers go on
    tc_fence_after();

    bool fail = false;
    // A thread that issues MMAs waits until they are complete before it leaves: tensor memory is given back behind it, and
    // no arrival may be outstanding when the CTA exits.
    auto land = [&](int i) {
        tc_commit(&sm->last[i]);
        mbar_wait(&sm->last[i], 0);
    };
    if ((warp == kTcWarpProd || (warp > kTcWarpPV && warp < kTcThreads / 32)) && active) {
        if constexpr (kScored) tc_fewer_registers();
        // ------------------------------------------------ producer warps 8, 11, 12
        // The three warps work independently: warp pw issues boxes i = pw, pw + 3,
        // pw + 6 of every tile (box i: K of 16-key group i for i < 4, V of group
        // i - 4 otherwise), with block ids from its own window of the block table;
        // it waits for the stage itself and arms the stage's transaction count
        // with its own bytes (the stage's full barrier expects one arrival per
        // producer warp), so one warp's bookkeeping overlaps the others' copies.
        const int pw = warp == kTcWarpProd ? 0 : warp - kTcWarpPV;
        const int nbox = pw < 2 ? 3 : 2;  // boxes of this warp per tile
        int* tbl = sm->tbl[pw];
        const int32_t* trow = block_tables + static_cast<size_t>(b) * max_blocks;
        int win0 = -kTcWin, j = 0;
        const int stop = static_cast<int>(blockIdx.x) == waits.silent_cta ? 0 : ntiles;
        for (; j < stop; ++j) {
            const int s = j % kTcStages;
            const int kt = key_tile(j + rot < ntiles ? j + rot : j + rot - ntiles);
            const int kb0 = (kt * kTcKeys) / BS, kb1 = min(nblk_used - 1, (kt * kTcKeys + kTcKeys - 1) / BS);
            if (kb0 < win0 || kb1 >= win0 + kTcWin) {  // move this warp's window of the block table
                __syncwarp();
                win0 = kb0;
                for (int i = lane; i < kTcWin; i += 32) tbl[i] = win0 + i < nblk_used ? trow[win0 + i] : 0;
                __syncwarp();
            }
            if (lane == 0) fail = !mbar_wait(&sm->kv_empty[s], ((j / kTcStages) & 1) ^ 1, waits.polls);
            fail = __shfl_sync(0xffffffffu, fail, 0);
            if (fail) break;
            const int bi = pw + 3 * lane;
            int row = 0;
            if (lane < nbox) {  // the pool row of box bi's first key
                const int key0 = kt * kTcKeys + 16 * (bi & 3);
                const int kb = key0 / BS;
                int blk = 0, slot = 0;
                // later keys and those that no row sees: any valid rows (masked; their V rows are cleared)
                if (kb < nblk_used && !(kScored && key0 + 16 <= wlo && key0 >= pfx)) {
                    blk = tbl[kb - win0];
                    slot = key0 - kb * BS;
                    if (blk < 0 || blk >= NB) {
                        sm->bad = 1;
                        report(status, PKV_ERR_DEVICE_BOUNDS);
                        blk = 0;
                    }
                }
                row = (blk * Hkv + h) * BS + slot;
            }
            if (lane == 0) mbar_arrive_expect_tx(&sm->kv_full[s], nbox * kTcGroupBytes);
            __syncwarp();  // the arrival precedes this warp's copies
            if (lane < nbox) {
                uint8_t* st = sKV + static_cast<size_t>(s) * kTcStageBytes;
                if (bi < 4)  // K of group bi: [8-row half][64-dimension half][8 rows][128 B]
                    tma_load_4d(st + kTcGroupBytes * bi, &tmK, 0, 0, 0, row >> 3, &sm->kv_full[s]);
                else  // V of group bi - 4: [64-dimension half][16 rows][128 B]
                    tma_load_3d(st + kTcKBytes + kTcGroupBytes * (bi - 4), &tmV, 0, row, 0, &sm->kv_full[s]);
            }
            __syncwarp();
        }
        // no copy of this CTA may still be in flight when it exits
        if (lane == 0)
            for (int i = max(0, j - kTcStages); i < j; ++i)
                mbar_wait(&sm->kv_full[i % kTcStages], (i / kTcStages) & 1, kTcLandPolls);
    } else if (warp == kTcWarpS && active) {
        if constexpr (kScored) tc_fewer_registers();
        // ------------------------------------------------ S = Q K^T for both query tiles (lane 0 issues)
        // Q (A) from tensor memory, K (B) from the stage.  S_j of query tile t
        // overwrites S_{j-1} once the softmax has read it, so it runs while the
        // softmax works on tile j - 1.
        if (lane == 0) {
            constexpr uint32_t idS = tc_idesc(kTcRows, kTcKeys, false);
            const uint32_t kva = smem_u32(sKV);
            for (int j = 0; j < ntiles && !fail; ++j) {
                const int s = j % kTcStages;
                if (!mbar_wait(&sm->kv_full[s], (j / kTcStages) & 1, waits.polls)) {
                    fail = true;
                    break;
                }
                const uint32_t kb = kva + s * kTcStageBytes;
                const int ta = dual ? j & 1 : 0, tb = dual ? ta : kTcQT - 1, u = dual ? j >> 1 : j;
                for (int t = ta; t <= tb; ++t) {
                    if (u >= 1 && !mbar_wait(&sm->s_free[t], (u - 1) & 1, waits.polls)) {
                        fail = true;
                        break;
                    }
                    tc_fence_after();
#pragma unroll
                    for (int kk = 0; kk < kTcDim / 16; ++kk)
                        tc_mma_ta(tmem + 256 * t + 64, tmem + 256 * t + 8 * kk,
                                  tc_desc(kb + (kk >> 2) * 1024 + 32 * (kk & 3), 16, 2048), idS, kk > 0 ? 1u : 0u);
                    tc_commit(&sm->s_full[t]);
                }
            }
            land(0);  // (the softmax may have given up and not wait for the last ones)
        }
        __syncwarp();
    } else if (warp == kTcWarpPV && active) {
        if constexpr (kScored) tc_fewer_registers();
        // ------------------------------------------------ O += P V for both query tiles (lane 0 issues)
        // P of query tile t (bf16, a K-major 128-byte-swizzled shared tile) is
        // the A operand.  Both P tiles of key tile j were written after the
        // softmax read S_j, so once their PV MMAs are complete nothing reads the
        // stage any more.
        if (lane == 0) {
            constexpr uint32_t idO = tc_idesc(kTcRows, kTcDim, true);
            const uint32_t pa = smem_u32(sP), kva = smem_u32(sKV);
            for (int j = 0; j < ntiles && !fail; ++j) {
                const int s = j % kTcStages;
                const uint32_t vb = kva + s * kTcStageBytes + kTcKBytes;
                const int ta = dual ? j & 1 : 0, tb = dual ? ta : kTcQT - 1, u = dual ? j >> 1 : j;
                for (int t = ta; t <= tb; ++t) {  // query tile 0 first: its softmax warps clear V rows past L
                    if (!mbar_wait(&sm->p_full[t], u & 1, waits.polls)) {
                        fail = true;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t pb = pa + t * kTcPBytes;
#pragma unroll
                    for (int kk = 0; kk < kTcKeys / 16; ++kk)
                        tc_mma(tmem + 256 * t + 128, tc_desc(pb + 32 * kk, 16, 1024),
                               tc_desc(vb + kTcGroupBytes * kk, kTcGroupBytes / 2, 1024), idO,
                               (u > 0 || kk > 0) ? 1u : 0u);
                    tc_commit(&sm->o_done[t]);
                }
                if (!fail) tc_commit(&sm->kv_empty[s]);
            }
            // no arrival of this CTA may be outstanding when it exits: the last one follows all others
            if (!fail && ntiles > 0 && !mbar_wait(&sm->kv_empty[(ntiles - 1) % kTcStages], ((ntiles - 1) / kTcStages) & 1)) fail = true;
            if (fail) land(1);
        }
        __syncwarp();
    } else if (softmax_warp && active) {
        if constexpr (kScored) tc_more_registers();
        // ------------------------------------------------ softmax warps: thread r of query tile qt owns row r
        const uint32_t lrow = static_cast<uint32_t>((warp & 3) * 32) << 16;  // this warp's TMEM lanes
        const uint32_t tq = tmem + 256 * qt;
        const int p0t = p0 + (dual ? 0 : qt * TQ);  // the query tile's first position
        const int step = dual ? 1 : 0, mine = dual ? (ntiles + 1 - qt) >> 1 : ntiles;  // its key tiles
        float m_ref = -INFINITY, lsum = 0.f;
        [[maybe_unused]] float slope = 0.f;
        if constexpr (kScored) slope = kKind & kSloped ? sc.slopes[qh] * kLog2e : 0.f;
        // the key that the bias is measured from: the last one that the row sees, or the first
        [[maybe_unused]] int from = max(pos, pfx - 1);
        if ((kKind & kSloped) != 0 && slope < 0.f) from = pfx > 0 || sc.window <= 0 ? 0 : max(0, pos - sc.window + 1);
        for (int u = 0; u < mine; ++u) {
            const int j = (u << step) + (step & qt);
            if (!__all_sync(0xffffffffu, tc_wait(&sm->s_full[qt], u & 1, waits.polls))) {  // tcgen05.ld needs the whole warp
                fail = true;
                break;
            }
            tc_fence_after();
            uint32_t sr[2][32];
            tc_ld32(tq + lrow + 64, sr[0]);
            tc_ld32(tq + lrow + 96, sr[1]);
            tc_fence_before();
            mbar_arrive(&sm->s_free[qt]);  // S may take the next tile
            const int kt = key_tile(j + rot < ntiles ? j + rot : j + rot - ntiles);
            const int kbase = kt * kTcKeys;
            if constexpr (kScored) score_tile<kKind>(sr, kbase, pos, from, p0t, min(p0t + TQ, p0 + nt) - 1, pfx, slope, sc);
            // maximum of the raw scores (the scale is positive), eight chains;
            // the causal mask only on tiles that reach past the query tile's first position
            // (three-input maxima: two scores per instruction, four chains)
            float mxs[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) mxs[k] = -INFINITY;
            if (!kScored && kbase + kTcKeys - 1 > p0t) {
#pragma unroll
                for (int c = 0; c < kTcKeys; ++c) {
                    const float v = kbase + c <= pos ? __uint_as_float(sr[c >> 5][c & 31]) : -INFINITY;
                    sr[c >> 5][c & 31] = __float_as_uint(v);
                }
            }
#pragma unroll
            for (int c = 0; c < kTcKeys; c += 2)
                mxs[(c >> 1) & 3] = tc_max3(mxs[(c >> 1) & 3], __uint_as_float(sr[c >> 5][c & 31]),
                                            __uint_as_float(sr[(c + 1) >> 5][(c + 1) & 31]));
            const float mul = kKind == kPlain ? scale_log2 : kKind == kMasked ? sc.mul : 1.f;
            const float mx = fmaxf(fmaxf(mxs[0], mxs[1]), fmaxf(mxs[2], mxs[3])) * mul;
            // the reference maximum moves only when the row maximum passes it by more than 8
            const float m_new = mx > m_ref + 8.f ? mx : m_ref;
            const bool resc = m_new != m_ref;
            const float a = resc ? tc_ex2(m_ref - m_new) : 1.f;
            m_ref = m_new;
            const float nmu = m_ref == -INFINITY ? 0.f : -m_ref;
            // P = 2^(s scale - m_ref) (masked scores give 0), the sum in four chains of
            // pairs (the scale, the offset and the sum as paired fp32 operations)
            uint32_t pk[kTcKeys / 2];
            float ls[4][2];
#pragma unroll
            for (int k = 0; k < 4; ++k) ls[k][0] = ls[k][1] = 0.f;
#pragma unroll
            for (int c = 0; c < kTcKeys / 2; ++c) {
                float t0, t1;
                tc_fma2(t0, t1, __uint_as_float(sr[(2 * c) >> 5][(2 * c) & 31]),
                        __uint_as_float(sr[(2 * c + 1) >> 5][(2 * c + 1) & 31]), mul, nmu);
                const float e0 = tc_ex2(t0), e1 = tc_ex2(t1);
                pk[c] = pack_bf16x2(e0, e1);
                tc_add2(ls[c & 3][0], ls[c & 3][1], e0, e1);
            }
            lsum = lsum * a + (((ls[0][0] + ls[0][1]) + (ls[1][0] + ls[1][1])) +
                               ((ls[2][0] + ls[2][1]) + (ls[3][0] + ls[3][1])));
            // the PV of the tile before is complete: O may be rescaled and the P tile rewritten
            if (u > 0) {
                if (!__all_sync(0xffffffffu, tc_wait(&sm->o_done[qt], (u - 1) & 1, waits.polls))) {
                    fail = true;
                    break;
                }
                tc_fence_after();
            }
            if (u > 0 && __any_sync(0xffffffffu, resc)) {
#pragma unroll 1
                for (int cc = 0; cc < kTcDim / 32; ++cc) {
                    uint32_t o[32];
                    tc_ld32(tq + lrow + 128 + 32 * cc, o);
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * a);
                    tc_st32(tq + lrow + 128 + 32 * cc, o);
                }
            }
            // the V rows of keys past the CTA's last one (not in the cache yet, past L, or another block's) may hold
            // anything: clear them (scored: those of every key that no row sees)
            if ((dual || qt == 0) && (kScored ? kbase + kTcKeys - 1 > plast || (kbase < wlo && kbase + kTcKeys > pfx) : kt == ntiles - 1)) {
                const int rlo = kScored ? 0 : plast + 1 - kbase;
                uint8_t* vb = sKV + static_cast<size_t>(j % kTcStages) * kTcStageBytes + kTcKBytes;
                for (int idx = r; idx < (kTcKeys - rlo) * 16; idx += kTcRows) {
                    const int rr = rlo + (idx >> 4), half = (idx >> 3) & 1, ch = idx & 7;
                    if (kScored && kbase + rr <= plast && (kbase + rr >= wlo || kbase + rr < pfx)) continue;
                    *reinterpret_cast<uint4*>(vb + kTcGroupBytes * (rr >> 4) + half * (kTcGroupBytes / 2) +
                                              (rr & 15) * 128 + ch * 16) = make_uint4(0u, 0u, 0u, 0u);
                }
            }
            // P row r (64 bf16 = 8 chunks of 16 bytes) into the K-major P tile of query tile qt
            uint8_t* pbuf = sP + qt * kTcPBytes;
#pragma unroll
            for (int ch = 0; ch < 8; ++ch)
                *reinterpret_cast<uint4*>(pbuf + sw128(r, ch)) =
                    make_uint4(pk[4 * ch], pk[4 * ch + 1], pk[4 * ch + 2], pk[4 * ch + 3]);
            fence_proxy_async_smem();  // P and the cleared V rows, for the PV MMA
            tc_fence_before();
            mbar_arrive(&sm->p_full[qt]);
        }
        // ---- epilogue: O / sum of the last PV
        if (!fail && mine > 0 && !__all_sync(0xffffffffu, tc_wait(&sm->o_done[qt], (mine - 1) & 1, waits.polls))) fail = true;
        // dual: query tile 1's result goes through the ring (both are done with it) to query tile 0, whose rows take
        // own O + other O' with the factors below
        [[maybe_unused]] float own = 1.f, other = 0.f;
        float4* const there = reinterpret_cast<float4*>(sKV) + r * (kTcDim / 4);  // 16-byte piece c at c ^ (r & 7)
        if constexpr (kScored) {
            if (dual) {
                float2* const ends = reinterpret_cast<float2*>(sKV + kTcRows * kTcDim * 4);
                tc_fence_after();
                softmax_barrier();
                if (qt == 1) {
                    ends[r] = make_float2(m_ref, fail ? -1.f : lsum);
#pragma unroll 1
                    for (int cc = 0; mine > 0 && !fail && cc < kTcDim / 32; ++cc) {
                        uint32_t o[32];
                        tc_ld32(tq + lrow + 128 + 32 * cc, o);
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            there[(8 * cc + i) ^ (r & 7)] = make_float4(__uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]),
                                                                        __uint_as_float(o[4 * i + 2]), __uint_as_float(o[4 * i + 3]));
                    }
                }
                softmax_barrier();
                if (qt == 0) {
                    const float2 e = ends[r];
                    fail = fail || e.y < 0.f;  // (of a whole warp)
                    const float m_new = fmaxf(m_ref, e.x), mu = m_new == -INFINITY ? 0.f : m_new;
                    own = tc_ex2(m_ref - mu);
                    other = tc_ex2(e.x - mu);
                    lsum = lsum * own + e.y * other;
                    m_ref = m_new;
                }
            }
        }
        auto joined = [&](uint32_t (&o)[32], int cc) {
            if constexpr (kScored) {
                if (!dual) return;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float4 v = ntiles > 1 ? there[(8 * cc + i) ^ (r & 7)] : make_float4(0.f, 0.f, 0.f, 0.f);
                    o[4 * i] = __float_as_uint(fmaf(v.x, other, __uint_as_float(o[4 * i]) * own));
                    o[4 * i + 1] = __float_as_uint(fmaf(v.y, other, __uint_as_float(o[4 * i + 1]) * own));
                    o[4 * i + 2] = __float_as_uint(fmaf(v.z, other, __uint_as_float(o[4 * i + 2]) * own));
                    o[4 * i + 3] = __float_as_uint(fmaf(v.w, other, __uint_as_float(o[4 * i + 3]) * own));
                }
            }
        };
        if (!fail && (!dual || qt == 0)) {
            tc_fence_after();
            if (S > 1) {
                const size_t at = row_valid ? (static_cast<size_t>(t0 + tl) * Hq + qh) * S + share : 0;
                if (row_valid) split.ml[at] = make_float2(m_ref, sm->bad ? -1.f : lsum);
                float4* to = reinterpret_cast<float4*>(split.o + at * kTcDim);
#pragma unroll 1
                for (int cc = 0; ntiles > 0 && cc < kTcDim / 32; ++cc) {
                    uint32_t o[32];
                    tc_ld32(tq + lrow + 128 + 32 * cc, o);
                    joined(o, cc);
                    if (row_valid) {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            to[8 * cc + i] = make_float4(__uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]),
                                                         __uint_as_float(o[4 * i + 2]), __uint_as_float(o[4 * i + 3]));
                    }
                }
            }
            const float inv = lsum > 0.f ? 1.f / lsum : 0.f;
            const bool store = row_valid && !sm->bad;
            uint4* dst = reinterpret_cast<uint4*>(out + (static_cast<size_t>(t0 + (row_valid ? tl : 0)) * Hq + qh) * kTcDim);
#pragma unroll 1
            for (int cc = 0; S == 1 && cc < kTcDim / 32; ++cc) {
                uint32_t o[32];
                tc_ld32(tq + lrow + 128 + 32 * cc, o);
                joined(o, cc);
                uint32_t w[16];
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    w[i] = pack_bf16x2(__uint_as_float(o[2 * i]) * inv, __uint_as_float(o[2 * i + 1]) * inv);
                if (row_valid) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        dst[4 * cc + k] = store ? make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3])
                                                : make_uint4(0u, 0u, 0u, 0u);
                }
            }
        }
    } else if (kScored && active) {
        tc_fewer_registers();
    }
    if (fail) {
        if (lane == 0) report(status, PKV_ERR_TIMEOUT);
        // what the row's results are to be made of may be missing: zeros
        if (row_valid && S > 1) {
            split.ml[(static_cast<size_t>(t0 + tl) * Hq + qh) * S + share] = make_float2(-INFINITY, -1.f);
        } else if (row_valid) {
            uint4* o = reinterpret_cast<uint4*>(out + (static_cast<size_t>(t0 + tl) * Hq + qh) * kTcDim);
            for (int c = 0; c < 16; ++c) o[c] = make_uint4(0u, 0u, 0u, 0u);
        }
    }
    // ---- every role is done with TMEM
    tc_fence_before();
    __syncthreads();
    if (warp == kTcWarpS) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTcTmemCols)
                     : "memory");
    }
}

// out = sum o_s 2^(m_s - M) / sum l_s 2^(m_s - M) over a row's shares, a warp a row; a share without keys has l = 0 and
// no O.  Rows behind the last sequence stay as they are.
__global__ void __launch_bounds__(128)
    prefill_join_kernel(__nv_bfloat16* out, const TcSplit split, const int32_t* q_start, int B, int T_new, int Hq) {
    const long long row = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    const long long rows = static_cast<long long>(min(q_start[B], T_new)) * Hq;  // older than the kernel before
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (row >= rows) return;
    const float2* ml = split.ml + row * split.S;
    const float2 mine = lane < split.S ? __ldcg(ml + lane) : make_float2(-INFINITY, 0.f);
    const float2 more = lane + 32 < split.S ? __ldcg(ml + lane + 32) : make_float2(-INFINITY, 0.f);
    float M = fmaxf(mine.x, more.x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    const float mu = M == -INFINITY ? 0.f : M, f0 = tc_ex2(mine.x - mu), f1 = tc_ex2(more.x - mu);
    const bool bad = __any_sync(0xffffffffu, mine.y < 0.f || more.y < 0.f);
    float l = mine.y * f0 + more.y * f1;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    const float4* os = reinterpret_cast<const float4*>(split.o + row * split.S * kTcDim) + lane;
#pragma unroll 4
    for (int s = 0; s < split.S; ++s) {
        const float w = __shfl_sync(0xffffffffu, s < 32 ? f0 : f1, s & 31), sum = __shfl_sync(0xffffffffu, s < 32 ? mine.y : more.y, s & 31);
        if (sum == 0.f) continue;
        const float4 v = __ldcg(os + static_cast<size_t>(s) * (kTcDim / 4));
        acc = make_float4(fmaf(v.x, w, acc.x), fmaf(v.y, w, acc.y), fmaf(v.z, w, acc.z), fmaf(v.w, w, acc.w));
    }
    const bool zero = bad || l == 0.f;
    const float inv = 1.f / l;
    const uint2 v = zero ? make_uint2(0u, 0u)
                         : make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
    reinterpret_cast<uint2*>(out + row * kTcDim)[lane] = v;
}

// The K pool [NB, Hkv, BS, 128] bf16 in four dimensions: (64 elements, 8 rows,
// the two 64-element halves of a row, groups of 8 rows), with boxes of
// 64 x 8 x 2 x 2.  One box holds 16 consecutive rows and lands as
// [8-row group][half][8 rows][128 B]: for either half, successive 8-row groups
// sit 2048 bytes apart, so a 64-key tile of four boxes is one K-major,
// 128-byte-swizzled operand per half with a 2048-byte group stride.
bool encode_pool_k16(CUtensorMap* map, const void* pool, int NB, int Hkv, int BS) {
    EncodeTiledFn enc = get_encode_fn();
    const cuuint64_t rows = static_cast<cuuint64_t>(NB) * Hkv * BS;
    if (!enc || rows % 8 != 0) return false;
    cuuint64_t gdim[4] = {64, 8, 2, rows / 8};
    cuuint64_t gstride[3] = {kTcDim * 2, 128, 8 * kTcDim * 2};
    cuuint32_t box[4] = {64, 8, 2, 2};
    cuuint32_t estr[4] = {1, 1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(pool), gdim, gstride, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool prefill_tc_supported(int Hq, int Hkv, int D, int BS, const void* q, const void* out, const void* k,
                          const void* v) {
    const int G = Hkv > 0 ? Hq / Hkv : 0;
    auto a16 = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
    return D == kTcDim && BS % 16 == 0 && G >= 1 && G <= 8 && Hq == G * Hkv && a16(q) && a16(out) && a16(k) &&
           a16(v);
}

// CTAs along the keys: as many as fill the SMs once, where the pairs of query tiles are fewer.
constexpr int kTcShares = 64;     // at most
// Key tiles a share has at least, by the table's width or the window.  16 and 2 heads: 40 tokens behind 3000 27.4 us (shares of
// 1 and more 32.9, of 8 30.1, none 62.4); 1 behind 500 12.4 (12.2, 15.9, 15.7); 1 behind 30000 27.0 (none 366).
constexpr int kTcShareTiles = 2;
static long long tc_units(int B, int T_new, int Hq, int Hkv) {
    return (static_cast<long long>(T_new) / (kTcQT * (kTcRows / (Hq / Hkv))) + B) * Hkv;
}
static int tc_shares(int B, int T_new, int Hq, int Hkv, long long longest, int P) {
    const long long units = std::max(1LL, tc_units(B, T_new, Hq, Hkv));
    const long long tiles = std::max(1LL, longest / (kTcKeys * kTcShareTiles));
    return static_cast<int>(std::max(1LL, std::min({P / units, tiles, static_cast<long long>(kTcShares)})));
}
static size_t tc_part_o(long long places) { return static_cast<size_t>((places * 8 + 255) / 256 * 256); }
size_t prefill_scored_workspace_bytes(int B, int T_new, int Hq, int Hkv, int P) {
    if (Hq / Hkv > 8) return 0;
    const int S = tc_shares(B, T_new, Hq, Hkv, 0x7fffffffLL, P);
    const long long places = static_cast<long long>(T_new) * Hq * S;
    return S == 1 ? 0 : tc_part_o(places) + static_cast<size_t>(places) * kTcDim * 4;
}

cudaError_t launch_prefill_tc(void* out, const void* q, const void* k_cache, const void* v_cache,
                              const int32_t* block_tables, int max_blocks, const int32_t* seq_lens,
                              const int32_t* q_start, int B, int T_new, int Hq, int Hkv, int BS, int NB, float scale,
                              const ScoreArgs* scored, void* workspace, int P, int32_t* status, cudaStream_t stream) {
    const int G = Hq / Hkv, TC = kTcQT * (kTcRows / G);
    const long long tiles = static_cast<long long>(T_new) / TC + B;
    if (tiles * Hkv > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    TcSplit split{1, nullptr, nullptr};
    if (scored != nullptr) {
        long long longest = std::min(static_cast<long long>(max_blocks) * BS, 0x7fffffffLL);
        if (scored->window > 0 && scored->prefix_lens == nullptr) longest = std::min(longest, static_cast<long long>(scored->window) + TC);
        split.S = tc_shares(B, T_new, Hq, Hkv, longest, P);
        split.ml = static_cast<float2*>(workspace);
        split.o = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + tc_part_o(static_cast<long long>(T_new) * Hq * split.S));
    }
    CUtensorMap tmK, tmV;
    if (!encode_pool_k16(&tmK, k_cache, NB, Hkv, BS) || !encode_pool_box_halves(&tmV, v_cache, NB, Hkv, BS, 16))
        return cudaErrorInvalidValue;
    const bool cap = scored != nullptr && scored->cap_log2 > 0.f, sloped = scored != nullptr && scored->slopes != nullptr;
    auto kern = scored == nullptr ? prefill_tc_kernel<kPlain>
                : cap             ? (sloped ? prefill_tc_kernel<kMasked | kCapped | kSloped> : prefill_tc_kernel<kMasked | kCapped>)
                                  : (sloped ? prefill_tc_kernel<kMasked | kSloped> : prefill_tc_kernel<kMasked>);
    cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           static_cast<int>(kTcSmemBytes));
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(tiles * Hkv * split.S), 1, 1);  // KV head innermost
    cfg.blockDim = dim3(scored != nullptr ? kTcScoredThreads : kTcThreads, 1, 1);
    cfg.dynamicSmemBytes = kTcSmemBytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const float scale_log2 = scale * 1.4426950408889634f;
    err = cudaLaunchKernelEx(&cfg, kern, tmK, tmV, static_cast<const __nv_bfloat16*>(q),
                             static_cast<__nv_bfloat16*>(out), block_tables, max_blocks, seq_lens, q_start, B, Hq, Hkv,
                             BS, NB, scale_log2, scored != nullptr ? *scored : ScoreArgs{}, split,
                             TcWaits{attention_wait_polls(), attention_silent_cta()}, status);
    if (err != cudaSuccess || split.S == 1) return err != cudaSuccess ? err : cudaGetLastError();
    cfg.gridDim = dim3(static_cast<unsigned>((static_cast<long long>(T_new) * Hq + 3) / 4), 1, 1);
    cfg.blockDim = dim3(128, 1, 1);
    cfg.dynamicSmemBytes = 0;
    err = cudaLaunchKernelEx(&cfg, prefill_join_kernel, static_cast<__nv_bfloat16*>(out), split, q_start, B, T_new, Hq);
    return err != cudaSuccess ? err : cudaGetLastError();
}

}  // namespace pkv
