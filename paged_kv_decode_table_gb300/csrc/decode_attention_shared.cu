// decode_attention_shared.cu -- decode attention of sequences that share prefixes ("LLM inference serving tutorial"
// 4.2: sequences hold the same physical blocks by reference count; 4.1 of "Suy luan & Toi uu hoa (Inference)":
// online softmax, whose partial results can be joined in any order).
//
// softmax over a sequence's keys is taken in two parts, the group's prefix and what the sequence has of its own; each
// leaves (max, sum, sum of products) per row, and out = sum o_c 2^(m_c - M) / sum l_c 2^(m_c - M).
//  1. prefix_tc_kernel: the queries of a group's members and of the query heads of one KV head are the rows of one
//     matrix (members x Hq / Hkv), which meets every prefix key once.  A tile of K and V serves up to 256 rows.
//  2. decode_split_kernel<.., kShared> (decode_attention_scored.cu): the positions behind the prefix, per sequence.
//  3. shared_join_kernel: a warp per row.
// 2 does not wait for 1: an SM that has no prefix work left takes up the rest, and where both have much to do they share
// the SMs out between them (SharedWork).
//
// prefix_tc_kernel: a persistent kernel, one CTA per SM.  Work = (group, KV head, tile of up to 256 rows) x key tiles of
// 64; all of it in one order, cut into one range of key tiles per CTA, so that a few rows over a long prefix and many
// groups over short ones fill the device alike.  What a range covers of one (group, head, row tile) is a piece.
//  * Where all members fit into 128 rows, both query tiles hold them and take every other key tile, each with results
//    of its own: two chains of products and softmax stay in flight (16 groups of 16 rows over 1024-4096 keys took 51 us
//    with one).
//  * Operands as in prefill_tc.cu: Q (bf16) in tensor memory, K and V by TMA in boxes of 16 keys through a ring,
//    S = Q K^T (M 128, N 64, K = D) and O += P V (M 128, N = D, K 64) by one issuing thread each, P through a
//    128-byte-swizzled shared tile, S and O in tensor memory (256 columns per query tile of 128 rows).
//  * Thread r of a query tile's four softmax warps owns row r.  A maximum is renewed (and O in tensor memory
//    rescaled) only when a score exceeds it by 2^8.
//  * A piece leaves its row maxima, sums and float32 O: 512 bytes per row of 128 dimensions, written through the P tile
//    so that a warp stores whole 128-byte lines.
//
// What bounds it.  Starts (lengths or groups, block ids, first tiles: 3-5 us) and ends of three kernels.  64 sequences of
// 64-1024 behind 8192 tokens, 32 and 8 heads of 128: 49 us, 26 at the copy rate; prefix and own positions side by side 40 (one
// after the other 22 and 25, 63 in all), the join 7.  16 groups of 4 behind 1024-4096: 63 us (34 at the copy rate): the
// prefix kernel streams at 6.6 TB/s once its ring is full.  Many rows: the chain of products and softmax, 2600 clocks a tile
// of 64 keys and 256 rows, 3900 with a cap, with two softmax warps a scheduler and no pipe near full (capped, with slopes: FMA
// pipe 37% busy, tensor pipe 18%, special functions 10%, issue slots 44%): 32 sequences behind 65536 tokens, 64 and 8 heads, cap
// and slopes 153 us (50).
// Tried and not kept: key tiles of 128 (P over S in tensor memory, half the barriers; 4000 clocks for 128 keys, but with a
// longer start as fast in all); 16 softmax warps, two threads a row.
// Every mbarrier wait is bounded; a CTA that gives up records PKV_ERR_TIMEOUT, waits (bounded) for its own TMA copies and
// MMAs, frees its tensor memory, and marks its pieces, whose rows the join then sets to zero.
#include <cuda.h>
#include <math.h>

#include <algorithm>

#include "attention_split.cuh"
#include "tensor_core.cuh"

namespace pkv {

int device_sm_count();
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn get_encode_fn();
bool split_applies(SplitPlan& pl, const void* out, const void* q, const void* k, const void* v, pkv_dtype dtype);
bool split_shape(int Hq, int Hkv, int D, int BS, int min_groups, SplitPlan& pl);
size_t split_space(const SplitPlan& pl, int P, int B, bool shared, void* base, SplitSpace* ws);
cudaError_t launch_split_shared(const SplitPlan& pl, const SplitSpace& ws, const void* q, const void* k, const void* v,
                                const int32_t* block_tables, const int32_t* seq_lens, int P, int32_t* status,
                                cudaStream_t stream, bool* done);
cudaError_t launch_decode_scored(void* out, const void* q, const void* k, const void* v, const int32_t* block_tables,
                                 int max_blocks, const int32_t* seq_lens, int B, int Hq, int Hkv, int D, int BS, int NB,
                                 const ScoreArgs& sc, const GroupArgs& groups, pkv_dtype dtype, void* workspace, int P,
                                 int32_t* status, cudaStream_t stream);
bool scored_shape_valid(int B, int Hq, int Hkv, int D, int BS, int NB, int max_blocks, pkv_dtype dtype);

constexpr int kPxRows = 128, kPxTiles = 2, kPxKeys = 64;
constexpr int kPxProd = 3;     // producer warps
constexpr int kPxMarks = 16;   // pieces of which a bad block is remembered; more than the ring has stages
constexpr int kPxPBytes = kPxRows * kPxKeys * 2;
// warps 0-7: softmax (warp w: query tile w / 4); 8, 11, 12: producers; 9: S MMAs (and the TMEM allocation); 10: PV MMAs
constexpr int kPxWarpProd = 8, kPxWarpS = 9, kPxWarpPV = 10;
constexpr int kPxThreads = 16 * 32;  // (13-15 have registers to pass on)
constexpr int kPxTmemCols = 512;  // query tile t: Q at 256 t, S at 256 t + 64, O at 256 t + 128
constexpr uint32_t kPxLoaderPolls = 1u << 20;  // of a loader's wait for a free stage: a quarter of a second or more
constexpr int kPxMinTiles = 2;    // key tiles of a range at least

template <int kD>
struct Px {
    static constexpr int kStages = kD == 128 ? 5 : 10;
    static constexpr int kKBytes = kPxKeys * kD * 2;
    static constexpr int kGroup = 16 * kD * 2;  // 16 keys
    static constexpr int kStageBytes = 2 * kKBytes;
    static constexpr size_t kOperands = kPxTiles * static_cast<size_t>(kPxPBytes) + kStages * static_cast<size_t>(kStageBytes);
};
struct PxShared {  // follows the 1024-aligned operand area
    uint64_t kv_full[10], kv_empty[10];
    uint64_t q_full[kPxTiles], s_full[kPxTiles], s_free[kPxTiles], p_full[kPxTiles], o_done[kPxTiles];
    uint64_t last[2];  // of a thread that leaves: its MMAs are complete
    uint32_t tmem_base;
    int at[7];  // where the CTA's range begins: a group as PxWalk has it
    int red[32];
    int work[3 * kPxThreads / 32];
    int bad[kPxMarks];
};
template <int kD>
constexpr size_t kPxSmem = 1024 + Px<kD>::kOperands + sizeof(PxShared);
static_assert(kPxSmem<128> <= 227 * 1024 && kPxSmem<64> <= 227 * 1024, "shared memory of one CTA");

// Written by the prefix kernel's first CTA for the join.
struct PxHead {
    int W;      // key tiles per range
    int valid;  // group_start is one
};
struct PxSpace {
    PxHead* head;
    int2* plan;   // of every group: (first key tile in the order, key tiles of a row tile)
    float2* ml;   // (max, sum): 2 slots per CTA of 256 rows, then two places per row of out
    float* o;
};
constexpr int kPxSlot = kPxTiles * kPxRows;  // rows of a slot

struct PxPlan {
    int B, Hq, Hkv, G, BS, NB, max_blocks;
    int TQ, TC;  // members per query tile and per row tile
    ScoreArgs sc;
    GroupArgs groups;
    int NG, units;  // of the split kernel
    uint32_t polls;  // of a wait
    int silent_cta;  // test hook: whose loaders issue no copy
};

// A role's walk over the CTA's pieces.
struct PxWalk {
    int g, base;          // group, its first key tile in the order
    int first, n;         // its first sequence, its members
    int prefix, nt, rt;   // positions read once; key tiles of one row tile; row tiles (0 where there is nothing to share)
    int h, tile, k0, k1;  // the piece: KV head, row tile, key tiles [k0, k1)
    // Group g from its entries, which were loaded together.
    __device__ __forceinline__ void set(const PxPlan& pl, int from, int to, int shared) {
        first = from;
        n = to - from;
        prefix = group_prefix_of(n, shared, pl.max_blocks, pl.BS);
        nt = (prefix + kPxKeys - 1) / kPxKeys;
        rt = prefix > 0 ? (n + pl.TC - 1) / pl.TC : 0;
    }
    __device__ __forceinline__ void load(const PxPlan& pl) {
        set(pl, pl.groups.start[g], pl.groups.start[g + 1], pl.groups.shared[g]);
    }
    __device__ __forceinline__ void put(int* at) const {
        at[0] = g;
        at[1] = base;
        at[2] = first;
        at[3] = n;
        at[4] = prefix;
        at[5] = nt;
        at[6] = rt;
    }
    PxWalk() = default;
    __device__ __forceinline__ explicit PxWalk(const int* at)
        : g(at[0]), base(at[1]), first(at[2]), n(at[3]), prefix(at[4]), nt(at[5]), rt(at[6]) {}
    // The piece at key tile `at` of a range that ends at `end`.
    __device__ __forceinline__ void to(const PxPlan& pl, int at, int end) {
        while (at >= base + pl.Hkv * rt * nt) {
            base += pl.Hkv * rt * nt;
            ++g;
            load(pl);
        }
        const int rel = at - base, work = rel / nt;
        k0 = rel - work * nt;
        k1 = min(nt, k0 + end - at);
        h = work / rt;
        tile = work - h * rt;
    }
    // All rows fit into one query tile: both hold them, tile t takes key tiles k0 + t, k0 + t + 2, ..
    __device__ __forceinline__ bool dual(const PxPlan& pl) const { return n - tile * pl.TC <= pl.TQ; }
};

template <int kD, bool kCap, bool kSlope>
__global__ void __launch_bounds__(kPxThreads, 1)
    prefix_tc_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                     const __grid_constant__ PxPlan pl, const __nv_bfloat16* q, const int32_t* block_tables,
                     const int32_t* seq_lens, const PxSpace ws, int32_t* status) {
    using C = Px<kD>;
    constexpr bool kScored = kCap || kSlope;
    constexpr int kStages = C::kStages;
    extern __shared__ uint8_t px_raw[];
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(px_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sP = base;  // P of query tile t at t kPxPBytes
    uint8_t* sKV = base + kPxTiles * kPxPBytes;
    PxShared* sm = reinterpret_cast<PxShared*>(base + C::kOperands);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int BS = pl.BS, G = pl.G, N = pl.groups.N;
    // groups, then block ids, then K and V: three dependent loads; the first two and q come to L2 while the
    // predecessor ends
    const unsigned worker = blockIdx.x * blockDim.x + tid;
    prefetch_l2(seq_lens, static_cast<size_t>(pl.B) * 4, worker);
    prefetch_l2(pl.groups.start, (static_cast<size_t>(N) + 1) * 4, worker);
    prefetch_l2(pl.groups.shared, static_cast<size_t>(N) * 4, worker);
    prefetch_l2(block_tables, static_cast<size_t>(pl.B) * pl.max_blocks * 4, worker);
    prefetch_l2(q, static_cast<size_t>(pl.B) * pl.Hq * kD * 2, worker);
    if (tid == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&sm->kv_full[s], kPxProd);  // one arrival (with its bytes) per producer warp
            mbar_init(&sm->kv_empty[s], 1);
        }
        for (int t = 0; t < kPxTiles; ++t) {
            mbar_init(&sm->q_full[t], kPxRows);
            mbar_init(&sm->s_full[t], 1);
            mbar_init(&sm->s_free[t], kPxRows);
            mbar_init(&sm->p_full[t], kPxRows);
            mbar_init(&sm->o_done[t], 1);
            mbar_init(&sm->last[t], 1);
        }
        fence_mbar_init();
        prefetch_tmap(&tmK);
        prefetch_tmap(&tmV);
        for (int i = 0; i < kPxMarks; ++i) sm->bad[i] = 0;
    }
    if (warp == kPxWarpS) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sm->tmem_base)),
                     "r"(kPxTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // ---- the whole work, and this CTA's range of it: key tiles [start, end)
    auto scan = [&](int v, int& total) {  // over the CTA; exclusive
        int x = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) sm->red[warp] = x;
        __syncthreads();
        int before = 0, all = 0;
        for (int w = 0; w < kPxThreads / 32; ++w) {
            const int r = sm->red[w];
            if (w < warp) before += r;
            all += r;
        }
        __syncthreads();
        total = all;
        return before + x - v;
    };
    bool wrong = false;
    int sum = 0, total, mine = 0;  // mine: key tiles of group tid
    SharedWork work;
    const bool estimate = shares_sms(G);
    const int L0 = estimate && tid < pl.B ? seq_lens[tid] : 0;  // on its way together with the group's entries
    PxWalk own;
    for (int g = N - 1 - (N - 1 - tid) % kPxThreads; g >= tid && g < N; g -= kPxThreads) {  // group tid comes last
        own.set(pl, pl.groups.start[g], pl.groups.start[g + 1], pl.groups.shared[g]);
        wrong = wrong || !group_valid(pl.groups, pl.B, g);
        mine = pl.Hkv * own.nt * own.rt;
        sum += mine;
        if (estimate) work.group(own.first, own.first + own.n, pl.groups.shared[g], pl.max_blocks, BS, pl.TQ);
    }
    if (estimate) {
        work.sequence(L0, pl.max_blocks, BS);
        for (int b = tid + kPxThreads; b < pl.B; b += kPxThreads) work.sequence(seq_lens[b], pl.max_blocks, BS);
        work.put(sm->work, warp, lane);
    }
    wrong = __syncthreads_or(wrong) != 0;
    int before = scan(sum, total);
    int P = static_cast<int>(gridDim.x);
    if (estimate) {
        work.get(sm->work, kPxThreads / 32, lane);
        P -= work.own_ctas(P, pl.B, N, pl.Hkv, pl.NG, pl.units, kCap, lane);
    }
    const int W = max(kPxMinTiles, (total + P - 1) / P);
    if (blockIdx.x == 0 && tid == 0) {
        *ws.head = PxHead{W, wrong ? 0 : 1};
        if (wrong) report(status, PKV_ERR_DEVICE_BOUNDS);
    }
    const int start = min(total, static_cast<int>(blockIdx.x) * W), end = min(total, start + W);
    const bool idle = wrong || start >= end;  // uniform over the CTA
    int carry = 0;
    for (int g0 = 0; g0 < N && !wrong && (!idle || blockIdx.x == 0); g0 += kPxThreads) {
        const int g = g0 + tid;
        int tot = total;
        if (N > kPxThreads) {  // else the scan above was this one
            mine = 0;
            if (g < N) {
                own.g = g;
                own.load(pl);
                mine = pl.Hkv * own.nt * own.rt;
            }
            before = scan(mine, tot);
        }
        const int at = carry + before;
        if (mine > 0 && at <= start && start < at + mine) {  // exactly one thread of the CTA
            own.g = g;
            own.base = at;
            own.put(sm->at);
        }
        if (blockIdx.x == 0 && g < N) ws.plan[g] = make_int2(at, own.nt);
        carry += tot;
        if (carry > start && blockIdx.x != 0) break;  // same decision in every thread
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm->tmem_base;

    bool fail = false;
    // A thread that issues MMAs waits until they are complete before it leaves: tensor memory is given back behind it, and
    // no arrival may be outstanding when the CTA exits.
    auto land = [&](int i) {
        tc_commit(&sm->last[i]);
        mbar_wait(&sm->last[i], 0);
    };
    if (idle) {
        // nothing but the tensor memory to give back
    } else if (warp == kPxWarpProd || warp == kPxWarpPV + 1 || warp == kPxWarpPV + 2) {
        tc_fewer_registers();
        // ------------------------------------------------ producer warps 8, 11, 12
        // Warp pw issues boxes i = pw, pw + 3, pw + 6 of every tile (box i: K of 16-key group i for i < 4, V of group
        // i - 4 otherwise), and arms the stage's transaction count with its own bytes.  Block
        // ids come 32 a load, a lane each, and the next 32 ahead of their use.
        const int pw = warp == kPxWarpProd ? 0 : warp - kPxWarpPV;
        const int nbox = pw < 2 ? 3 : 2;
        PxWalk w(sm->at);
        int j = 0;
        const int stop = static_cast<int>(blockIdx.x) == pl.silent_cta ? start : end;
        for (int at = start, piece = 0; at < stop && !fail; at += w.k1 - w.k0, ++piece) {
            w.to(pl, at, end);
            // The prefix is read by the table row of the first member that has all of it: a member of length 0 or of a
            // refused length may have anything there.  (Where no member has, any valid rows: all of them get zeros.)  The
            // first one's length and block ids are on their way together.
            const int32_t* trow = block_tables + static_cast<size_t>(w.first) * pl.max_blocks;
            int nblk = w.prefix / BS;
            auto ids = [&](int i) { return i < nblk ? trow[i] : 0; };
            auto has_all = [&](int L) { return L >= w.prefix && static_cast<long long>(L) <= static_cast<long long>(pl.max_blocks) * BS; };
            const int L0 = seq_lens[w.first];
            int have = (w.k0 * kPxKeys) / BS, cur = ids(have + lane), nxt = ids(have + 32 + lane);
            if (!has_all(L0)) {
                unsigned found = 0;
                int m = 1;
                for (; m < w.n; m += 32) {
                    found = __ballot_sync(0xffffffffu, m + lane < w.n && has_all(seq_lens[w.first + min(m + lane, w.n - 1)]));
                    if (found != 0) break;
                }
                if (found != 0) trow += static_cast<size_t>(m + __ffs(found) - 1) * pl.max_blocks;
                else nblk = 0;
                cur = ids(have + lane);
                nxt = ids(have + 32 + lane);
            }
            for (int kt = w.k0; kt < w.k1 && !fail; ++kt, ++j) {
                const int s = j % kStages;
                if ((kt * kPxKeys) / BS - have >= 32) {  // a tile is in at most five blocks
                    have += 32;
                    cur = nxt;
                    nxt = ids(have + 32 + lane);
                }
                // (a limit of their own: with the argument's 16 groups of 4 behind 1024-4096 take 75.4 us for 73.1)
                if (lane == 0 && !mbar_wait(&sm->kv_empty[s], ((j / kStages) & 1) ^ 1, kPxLoaderPolls)) fail = true;
                fail = __shfl_sync(0xffffffffu, fail, 0);
                if (fail) break;
                const int bi = pw + 3 * lane;
                const int key0 = kt * kPxKeys + 16 * (bi & 3), kb = key0 / BS;
                const int id0 = __shfl_sync(0xffffffffu, cur, (kb - have) & 31), id1 = __shfl_sync(0xffffffffu, nxt, (kb - have) & 31);
                int row = 0;
                if (lane < nbox) {  // the pool row of box bi's first key
                    int blk = 0, slot = 0;
                    if (kb < nblk) {  // keys behind the prefix: any valid rows (masked; their V rows are cleared)
                        blk = kb - have < 32 ? id0 : id1;
                        slot = key0 - kb * BS;
                        if (blk < 0 || blk >= pl.NB) {
                            *const_cast<volatile int*>(&sm->bad[piece % kPxMarks]) = piece + 1;
                            report(status, PKV_ERR_DEVICE_BOUNDS);
                            blk = 0;
                        }
                    }
                    row = (blk * pl.Hkv + w.h) * BS + slot;
                }
                __syncwarp();  // the marks precede the arrival
                if (lane == 0) mbar_arrive_expect_tx(&sm->kv_full[s], nbox * C::kGroup);
                __syncwarp();  // the arrival precedes this warp's copies
                if (lane < nbox) {
                    uint8_t* st = sKV + static_cast<size_t>(s) * C::kStageBytes + (bi < 4 ? 0 : C::kKBytes) + C::kGroup * (bi & 3);
                    if constexpr (kD == 64) {
                        tma_load_2d(st, bi < 4 ? &tmK : &tmV, 0, row, &sm->kv_full[s]);
                    } else {
                        if (bi < 4)  // [8-row half][64-dimension half][8 rows][128 B]
                            tma_load_4d(st, &tmK, 0, 0, 0, row >> 3, &sm->kv_full[s]);
                        else  // [64-dimension half][16 rows][128 B]
                            tma_load_3d(st, &tmV, 0, row, 0, &sm->kv_full[s]);
                    }
                }
                __syncwarp();
            }
        }
        // no copy of this CTA may still be in flight when it exits
        if (lane == 0)
            for (int i = max(0, j - kStages); i < j; ++i) mbar_wait(&sm->kv_full[i % kStages], (i / kStages) & 1, kTcLandPolls);
    } else if (warp == kPxWarpS) {
        tc_fewer_registers();
        // ------------------------------------------------ S = Q K^T (lane 0 issues)
        if (lane == 0) {
            constexpr uint32_t idS = tc_idesc(kPxRows, kPxKeys, false);
            const uint32_t kva = smem_u32(sKV);
            PxWalk w(sm->at);
            // bit t: the phase of query tile t's barriers, and whether it had a tile (indexed arrays would lie in local
            // memory)
            uint32_t free_ = 1u | 2u, had = 0, queries = 0;
            int j = 0;
            for (int at = start; at < end && !fail; at += w.k1 - w.k0) {
                w.to(pl, at, end);
                const bool dual = w.dual(pl);
                for (int kt = w.k0; kt < w.k1 && !fail; ++kt, ++j) {
                    const int s = j % kStages;
                    if (!mbar_wait(&sm->kv_full[s], (j / kStages) & 1, pl.polls)) {
                        fail = true;
                        break;
                    }
                    const uint32_t kb = kva + s * C::kStageBytes;
                    const int ta = dual ? (kt - w.k0) & 1 : 0, tb = dual ? ta : 1;
                    for (int t = ta; t <= tb; ++t) {
                        if ((kt - w.k0 < (dual ? 2 : 1) && !mbar_wait(&sm->q_full[t], (queries >> t) & 1u, pl.polls)) ||
                            ((had >> t) & 1u && !mbar_wait(&sm->s_free[t], (free_ >> t) & 1u, pl.polls))) {
                            fail = true;
                            break;
                        }
                        tc_fence_after();
#pragma unroll
                        for (int kk = 0; kk < kD / 16; ++kk)
                            tc_mma_ta(tmem + 256 * t + 64, tmem + 256 * t + 8 * kk,
                                      kD == 64 ? tc_desc(kb + 32 * kk, 16, 1024)
                                               : tc_desc(kb + (kk >> 2) * 1024 + 32 * (kk & 3), 16, 2048),
                                      idS, kk > 0 ? 1u : 0u);
                        tc_commit(&sm->s_full[t]);
                        had |= 1u << t;
                        free_ ^= 1u << t;
                    }
                }
                queries ^= 1u | (!dual || w.k1 - w.k0 > 1 ? 2u : 0u);
            }
            land(0);  // (the softmax may have given up and not wait for the last ones)
        }
        __syncwarp();
    } else if (warp == kPxWarpPV) {
        tc_fewer_registers();
        // ------------------------------------------------ O += P V (lane 0 issues)
        if (lane == 0) {
            constexpr uint32_t idO = tc_idesc(kPxRows, kD, true);
            const uint32_t pa = smem_u32(sP), kva = smem_u32(sKV);
            PxWalk w(sm->at);
            uint32_t phase = 0;  // bit t: of query tile t
            int j = 0;
            for (int at = start; at < end && !fail; at += w.k1 - w.k0) {
                w.to(pl, at, end);
                const bool dual = w.dual(pl);
                for (int kt = w.k0; kt < w.k1 && !fail; ++kt, ++j) {
                    const int s = j % kStages;
                    const uint32_t vb = kva + s * C::kStageBytes + C::kKBytes;
                    const int ta = dual ? (kt - w.k0) & 1 : 0, tb = dual ? ta : 1;
                    for (int t = ta; t <= tb; ++t) {  // query tile 0 first: its softmax warps clear V rows
                        if (!mbar_wait(&sm->p_full[t], (phase >> t) & 1u, pl.polls)) {
                            fail = true;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t pb = pa + t * kPxPBytes;
#pragma unroll
                        for (int kk = 0; kk < kPxKeys / 16; ++kk)
                            tc_mma(tmem + 256 * t + 128, tc_desc(pb + 32 * kk, 16, 1024),
                                   tc_desc(vb + C::kGroup * kk, C::kGroup / 2, 1024), idO,
                                   (kt - w.k0 >= (dual ? 2 : 1) || kk > 0) ? 1u : 0u);
                        tc_commit(&sm->o_done[t]);
                        phase ^= 1u << t;
                    }
                    if (!fail) tc_commit(&sm->kv_empty[s]);
                }
            }
            // no arrival of this CTA may be outstanding when it exits: the last one follows all others
            if (!fail && !mbar_wait(&sm->kv_empty[(j - 1) % kStages], ((j - 1) / kStages) & 1)) fail = true;
            if (fail) land(1);
        }
        __syncwarp();
    } else if (warp < 8) {
        tc_more_registers();
        // ------------------------------------------------ softmax warps: thread r of query tile qt owns row r
        const int qt = warp >> 2, r = tid & (kPxRows - 1);
        const uint32_t lrow = static_cast<uint32_t>((warp & 3) * 32) << 16;  // this warp's TMEM lanes
        const uint32_t tq = tmem + 256 * qt + lrow;
        uint8_t* pbuf = sP + qt * kPxPBytes;
        PxWalk w(sm->at);
        const int rm = r / G, rh = r - rm * G;  // the row's member in the query tile, and query head
        // The piece's queries as A of S = Q K^T; rows without a member are zero queries.
        auto put_q = [&](const PxWalk& x) {
            const bool dual = x.dual(pl);
            if (x.k0 + (dual ? qt : 0) >= x.k1) return;
            const int member = x.tile * pl.TC + (dual ? 0 : qt * pl.TQ) + rm;
            const bool valid = rm < pl.TQ && member < x.n;
            const uint4* src = reinterpret_cast<const uint4*>(
                q + (static_cast<size_t>(x.first + (valid ? member : 0)) * pl.Hq + x.h * G + rh) * kD);
#pragma unroll
            for (int hv = 0; hv < kD / 64; ++hv) {
                uint32_t y[32];
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    const uint4 v = valid ? src[8 * hv + c] : make_uint4(0u, 0u, 0u, 0u);
                    y[4 * c] = v.x;
                    y[4 * c + 1] = v.y;
                    y[4 * c + 2] = v.z;
                    y[4 * c + 3] = v.w;
                }
                tc_st32(tq + 32 * hv, y);
            }
            tc_fence_before();
            mbar_arrive(&sm->q_full[qt]);
        };
        // Where the row's part of a piece goes: a place per row of out where it is the whole prefix, else this range's slot.
        auto place = [&](const PxWalk& x, bool dual, int b) {
            return x.k0 == 0 && x.k1 == x.nt ? 2 * static_cast<size_t>(gridDim.x) * kPxSlot +
                                                   (static_cast<size_t>(dual ? qt : 0) * pl.B + b) * pl.Hq + x.h * G + rh
                                             : (2 * static_cast<size_t>(blockIdx.x) + (x.k0 > 0 ? 0 : 1)) * kPxSlot + qt * kPxRows + r;
        };
        int done = 0;  // key tiles of this query tile
        PxWalk next = w;
        next.to(pl, start, end);
        put_q(next);
        for (int at = start, piece = 0; at < end && !fail; at += w.k1 - w.k0, ++piece) {
            w = next;
            const bool dual = w.dual(pl);
            const int step = dual ? 2 : 1, k0 = w.k0 + (dual ? qt : 0);  // this query tile's first key tile
            const int member = w.tile * pl.TC + (dual ? 0 : qt * pl.TQ) + rm, qh = w.h * G + rh;
            const bool valid = rm < pl.TQ && member < w.n;
            const int b = w.first + (valid ? member : 0);
            const int prefix = w.prefix;
            [[maybe_unused]] const float slope = kSlope ? pl.sc.slopes[qh] * kLog2e : 0.f;
            [[maybe_unused]] const int from = kSlope && valid && !(slope < 0.f) ? seq_lens[b] - 1 : 0;  // the bias is 0 there
            float m_ref = -INFINITY, lsum = 0.f;
            bool broken = false;
            for (int kt = k0; kt < w.k1; kt += step, ++done) {
                if (!__all_sync(0xffffffffu, tc_wait(&sm->s_full[qt], done & 1, pl.polls))) {  // tcgen05.ld needs the whole warp
                    fail = true;
                    break;
                }
                tc_fence_after();
                uint32_t sr[2][32];
                tc_ld32(tq + 64, sr[0]);
                tc_ld32(tq + 96, sr[1]);
                tc_fence_before();
                mbar_arrive(&sm->s_free[qt]);  // S may take the next tile
                const int kbase = kt * kPxKeys;
                if constexpr (kScored) tc_scores<kCap, kSlope>(sr, kbase - from, slope, pl.sc);
                const bool tail = kbase + kPxKeys > prefix;
                if (tail) {
#pragma unroll
                    for (int c = 0; c < kPxKeys; ++c)
                        if (kbase + c >= prefix) sr[c >> 5][c & 31] = __float_as_uint(-INFINITY);
                }
                float mxs[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) mxs[k] = -INFINITY;
#pragma unroll
                for (int c = 0; c < kPxKeys; c += 2)
                    mxs[(c >> 1) & 3] = tc_max3(mxs[(c >> 1) & 3], __uint_as_float(sr[c >> 5][c & 31]),
                                                __uint_as_float(sr[(c + 1) >> 5][(c + 1) & 31]));
                const float mul = kScored ? 1.f : pl.sc.mul;
                const float mx = fmaxf(fmaxf(mxs[0], mxs[1]), fmaxf(mxs[2], mxs[3])) * mul;
                const float m_new = mx > m_ref + 8.f ? mx : m_ref;
                const bool resc = m_new != m_ref;
                const float a = resc ? tc_ex2(m_ref - m_new) : 1.f;
                m_ref = m_new;
                const float nmu = m_ref == -INFINITY ? 0.f : -m_ref;
                uint32_t pk[kPxKeys / 2];
                float ls[4][2];
#pragma unroll
                for (int k = 0; k < 4; ++k) ls[k][0] = ls[k][1] = 0.f;
#pragma unroll
                for (int c = 0; c < kPxKeys / 2; ++c) {
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
                if (kt > k0) {
                    if (!__all_sync(0xffffffffu, tc_wait(&sm->o_done[qt], (done - 1) & 1, pl.polls))) {
                        fail = true;
                        break;
                    }
                    tc_fence_after();
                    if (__any_sync(0xffffffffu, resc)) {
#pragma unroll 1
                        for (int cc = 0; cc < kD / 32; ++cc) {
                            uint32_t o[32];
                            tc_ld32(tq + 128 + 32 * cc, o);
#pragma unroll
                            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * a);
                            tc_st32(tq + 128 + 32 * cc, o);
                        }
                    }
                }
                if (tail && (dual || qt == 0)) {  // the V rows of keys behind the prefix may hold anything: clear them
                    const int rlo = prefix - kbase;
                    uint8_t* vb = sKV + static_cast<size_t>((at - start + kt - w.k0) % kStages) * C::kStageBytes + C::kKBytes;
                    constexpr int kRowChunks = kD / 8;
                    for (int idx = r; idx < (kPxKeys - rlo) * kRowChunks; idx += kPxRows) {
                        const int rr = rlo + idx / kRowChunks, half = (idx / 8) % (kRowChunks / 8), ch = idx & 7;
                        *reinterpret_cast<uint4*>(vb + C::kGroup * (rr >> 4) + half * 2048 + (rr & 15) * 128 + ch * 16) =
                            make_uint4(0u, 0u, 0u, 0u);
                    }
                }
#pragma unroll
                for (int ch = 0; ch < 8; ++ch)
                    *reinterpret_cast<uint4*>(pbuf + sw128(r, ch)) =
                        make_uint4(pk[4 * ch], pk[4 * ch + 1], pk[4 * ch + 2], pk[4 * ch + 3]);
                // before this tile is given back: the producers are at most kStages pieces ahead of it
                if (kt + step >= w.k1) broken = *const_cast<volatile int*>(&sm->bad[piece % kPxMarks]) == piece + 1;
                fence_proxy_async_smem();  // P and the cleared V rows, for the PV MMA
                tc_fence_before();
                mbar_arrive(&sm->p_full[qt]);
            }
            // all S of the piece are read: the next one's queries, whose S runs while this one's results are stored
            if (!fail && at + w.k1 - w.k0 < end) {
                next.to(pl, at + w.k1 - w.k0, end);
                put_q(next);
            }
            if (!fail && k0 < w.k1 && !__all_sync(0xffffffffu, tc_wait(&sm->o_done[qt], (done - 1) & 1, pl.polls))) fail = true;
            if (fail) {  // this piece's rows and those of the pieces to come are marked: the join sets them to zero
                for (int x = at; x < end; x += w.k1 - w.k0) {
                    w.to(pl, x, end);
                    const bool both = w.dual(pl);
                    const int m = w.tile * pl.TC + (both ? 0 : qt * pl.TQ) + rm;
                    if (rm < pl.TQ && m < w.n) ws.ml[place(w, both, w.first + m)] = make_float2(-INFINITY, -1.f);
                }
                break;
            }
            // ---- the piece's rows
            tc_fence_after();
            const size_t own = place(w, dual, b);
            if (valid) ws.ml[own] = make_float2(m_ref, broken ? -1.f : lsum);
            // the P tile is free: 32 columns of the warp's 32 rows go through its quarter of it
            float4* stage = reinterpret_cast<float4*>(pbuf + (warp & 3) * 4096);
            const int own_lo = valid ? static_cast<int>(own) : -1, own_hi = valid ? static_cast<int>(own >> 32) : -1;
            const bool any = __any_sync(0xffffffffu, valid);
#pragma unroll 1
            for (int cc = 0; any && cc < kD / 32; ++cc) {
                uint32_t o[32];
                if (k0 < w.k1) {
                    tc_ld32(tq + 128 + 32 * cc, o);
                } else {  // no key tile: nothing was summed
#pragma unroll
                    for (int c = 0; c < 32; ++c) o[c] = 0u;
                }
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    stage[lane * 8 + (c ^ (lane & 7))] =
                        make_float4(__uint_as_float(o[4 * c]), __uint_as_float(o[4 * c + 1]),
                                    __uint_as_float(o[4 * c + 2]), __uint_as_float(o[4 * c + 3]));
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int rr = 4 * i + (lane >> 3), c = lane & 7;
                    const int lo = __shfl_sync(0xffffffffu, own_lo, rr), hi = __shfl_sync(0xffffffffu, own_hi, rr);
                    const float4 v = stage[rr * 8 + (c ^ (rr & 7))];
                    if (hi >= 0) {
                        const size_t to = (static_cast<size_t>(hi) << 32) | static_cast<uint32_t>(lo);
                        *reinterpret_cast<float4*>(ws.o + to * kD + 32 * cc + 4 * c) = v;
                    }
                }
                __syncwarp();
            }
            tc_fence_before();
        }
    } else {
        tc_fewer_registers();
    }
    if (fail && lane == 0) report(status, PKV_ERR_TIMEOUT);
    // ---- every role is done with TMEM
    tc_fence_before();
    __syncthreads();
    if (warp == kPxWarpS) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kPxTmemCols) : "memory");
    }
}

// ------------------------------------------------------------------ join
// A row's pieces are those of its group's prefix, then those of what its sequence has of its own.  kUnit warps a row: one
// where the rows fill the SMs, four where they are few.
constexpr int kSjWarps = 4;
constexpr int kSjGroup = 8;  // pieces in flight, of a warp (4: 1-2% more on long prefixes, 8% less on 10000 rows of few pieces)
constexpr int kSjManyRows = 4;  // rows per SM from which one warp a row is enough (2048 rows of 20 pieces: 66 us a call for 67)

template <int kD, int kUnit>
__global__ void __launch_bounds__(kSjWarps * 32)
    shared_join_kernel(const __grid_constant__ PxPlan pl, const PxSpace px, const SplitSpace ws, const int R,
                       const int32_t* seq_lens, __nv_bfloat16* out, const int P, int32_t* status) {
    constexpr int kRows = kSjWarps / kUnit, kCols = kD / 32;  // rows of a CTA, columns of a lane
    __shared__ float part[kUnit > 1 ? kSjWarps : 1][32][kCols + 2];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, w0 = warp % kUnit;
    const long long rows = static_cast<long long>(pl.B) * pl.Hq, row0 = static_cast<long long>(blockIdx.x) * kRows + warp / kUnit;
    const long long row = min(row0, rows - 1);
    const int b = static_cast<int>(row / pl.Hq), qh = static_cast<int>(row - static_cast<long long>(b) * pl.Hq);
    // What only the inputs say comes before the wait: they are older than the prefix kernel, which started this
    // chain after its own wait.
    const int L = seq_lens[b];
    bool bad = L < 0 || static_cast<long long>(L) > static_cast<long long>(pl.max_blocks) * pl.BS;
    const int g = group_of(pl.groups, b);
    const int prefix = g < 0 ? 0 : group_prefix(pl.groups, pl.max_blocks, pl.BS, g);
    bad = bad || (L > 0 && (prefix < 0 || L < prefix));
    // the row in its row tile
    int first_seq = 0, rt = 0, tile = 0, qt = 0, r = 0;
    const int h = qh / pl.G, grp = qh / R;
    bool dual = false;
    if (prefix > 0) {
        first_seq = pl.groups.start[g];
        const int n = pl.groups.start[g + 1] - first_seq, member = b - first_seq;
        rt = (n + pl.TC - 1) / pl.TC;
        tile = member / pl.TC;
        const int in = member - tile * pl.TC;
        qt = in / pl.TQ;
        r = (in - qt * pl.TQ) * pl.G + qh - h * pl.G;
        dual = n - tile * pl.TC <= pl.TQ;
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int2 h2 = __ldcg(reinterpret_cast<const int2*>(px.head));
    const PxHead head{h2.x, h2.y};
    const int2 plan = prefix > 0 ? __ldcg(px.plan + g) : make_int2(0, 0), info = __ldcg(ws.info + b);
    const int Wo = __ldcg(&ws.head->W);
    bad = bad || head.valid == 0;
    if (bad && lane == 0 && qh == 0 && w0 == 0) report(status, PKV_ERR_DEVICE_BOUNDS);
    // pieces [0, np) lie in ranges pf .. of the prefix's key tiles (twice that many where dual), the others in ranges of
    int np = 0, pf = 0, no = 0, of = 0;
    if (!bad && L > 0) {
        if (prefix > 0) {
            const int first = plan.x + (h * rt + tile) * plan.y;
            pf = first / head.W;
            np = (first + plan.y - 1) / head.W - pf + 1;
        }
        if (info.y > 0) {
            const int first = info.x + grp * info.y;
            of = first / Wo;
            no = (first + info.y - 1) / Wo - of + 1;
        }
    }
    const int npx = dual ? 2 * np : np, n = npx + no;
    float acc[kCols] = {};
    float M = -INFINITY, l = 0.f;
    for (int x0 = w0; x0 < n; x0 += kUnit * kSjGroup) {
        float2 ml[kSjGroup];
        float o[kSjGroup][kCols];
#pragma unroll
        for (int k = 0; k < kSjGroup; ++k) {
            const int x = x0 + k * kUnit;
            ml[k] = make_float2(-INFINITY, 0.f);
#pragma unroll
            for (int i = 0; i < kCols; ++i) o[k][i] = 0.f;
            if (x < n) {
                const float2* mls;
                const float* os;
                if (x < npx) {
                    const int p = dual ? x >> 1 : x, t = dual ? x & 1 : qt;
                    const size_t at = np == 1 ? 2 * static_cast<size_t>(P) * kPxSlot + (static_cast<size_t>(dual ? t : 0) * pl.B + b) * pl.Hq + qh
                                              : (2 * static_cast<size_t>(pf + p) + (p == 0 ? 1 : 0)) * kPxSlot + t * kPxRows + r;
                    mls = px.ml + at;
                    os = px.o + at * kD;
                } else {
                    const int p = x - npx;
                    const size_t at = no == 1 ? 2 * static_cast<size_t>(P) * R + row
                                              : (2 * static_cast<size_t>(of + p) + (p == 0 ? 1 : 0)) * R + (qh - grp * R);
                    mls = ws.ml + at;
                    os = ws.o + at * kD;
                }
                ml[k] = __ldcg(mls);
                if constexpr (kCols == 4) {
                    const float4 v = __ldcg(reinterpret_cast<const float4*>(os) + lane);
                    o[k][0] = v.x;
                    o[k][1] = v.y;
                    o[k][2] = v.z;
                    o[k][3] = v.w;
                } else {
                    const float2 v = __ldcg(reinterpret_cast<const float2*>(os) + lane);
                    o[k][0] = v.x;
                    o[k][1] = v.y;
                }
            }
        }
        float mn = M;
#pragma unroll
        for (int k = 0; k < kSjGroup; ++k) mn = fmaxf(mn, ml[k].x);
        const float mu = mn == -INFINITY ? 0.f : mn, fa = ex2_approx(M - mu);
        l *= fa;
#pragma unroll
        for (int i = 0; i < kCols; ++i) acc[i] *= fa;
        M = mn;
#pragma unroll
        for (int k = 0; k < kSjGroup; ++k) {
            const float f = ex2_approx(ml[k].x - mu);
            bad = bad || ml[k].y < 0.f;  // a piece that could not be read makes the row zero
            l = fmaf(ml[k].y, f, l);
#pragma unroll
            for (int i = 0; i < kCols; ++i) acc[i] = fmaf(o[k][i], f, acc[i]);
        }
    }
    if constexpr (kUnit > 1) {
        float* mine = part[warp][lane];
        mine[0] = M;
        mine[1] = bad ? -1.f : l;
#pragma unroll
        for (int i = 0; i < kCols; ++i) mine[2 + i] = acc[i];
        __syncthreads();
        if (w0 != 0) return;
        float mn = M;
#pragma unroll
        for (int u = 1; u < kUnit; ++u) mn = fmaxf(mn, part[warp + u][lane][0]);
        const float mu = mn == -INFINITY ? 0.f : mn, fa = ex2_approx(M - mu);
        l *= fa;
#pragma unroll
        for (int i = 0; i < kCols; ++i) acc[i] *= fa;
#pragma unroll
        for (int u = 1; u < kUnit; ++u) {
            const float* other = part[warp + u][lane];
            const float f = ex2_approx(other[0] - mu);
            bad = bad || other[1] < 0.f;
            l = fmaf(other[1], f, l);
#pragma unroll
            for (int i = 0; i < kCols; ++i) acc[i] = fmaf(other[2 + i], f, acc[i]);
        }
    }
    if (row0 >= rows) return;
    const bool zero = bad || l == 0.f;
    const float inv = 1.f / l;
    __nv_bfloat16* to = out + row * kD + kCols * lane;
    if constexpr (kCols == 4)
        *reinterpret_cast<uint2*>(to) = zero ? make_uint2(0u, 0u)
                                             : make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv),
                                                          pack_bf16x2(acc[2] * inv, acc[3] * inv));
    else
        *reinterpret_cast<uint32_t*>(to) = zero ? 0u : pack_bf16x2(acc[0] * inv, acc[1] * inv);
}

// ------------------------------------------------------------------ host side
// Bytes of cache (by the table's width, each sequence's own) up to which two kernels that read a prefix per sequence take
// less time than three that read it once.  Per sequence against once: 8 groups of 8, prefix 86, 5 KV heads x 64
// (10 MB) 7.1 : 16.0 us; 5 of 32, 60, 7 x 128 (37 MB) 14.5 : 28.7; 1 of 16, 1575, 6 x 64 (39 MB) 17.9 : 15.6; 2 of 7, 1782,
// 5 x 128 (65 MB) 31.0 : 26.3; 5 of 17, 271, 8 x 128 (100 MB) 36.4 : 36.2; groups of one, 6533, 11 x 128 52 : 57.
constexpr long long kPxReadPerSequence = 48LL << 20;

bool encode_pool_k16(CUtensorMap* map, const void* pool, int NB, int Hkv, int BS);
bool encode_pool_box_halves(CUtensorMap* map, const void* pool, int NB, int Hkv, int BS, int box_rows);

// A pool of 64-element rows in boxes of 16 rows, 128-byte swizzle.
static bool encode_pool_rows64(CUtensorMap* map, const void* pool, long long rows) {
    EncodeTiledFn enc = get_encode_fn();
    if (!enc) return false;
    cuuint64_t dim[2] = {64, static_cast<cuuint64_t>(rows)}, stride[1] = {128};
    cuuint32_t box[2] = {64, 16}, one[2] = {1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(pool), dim, stride, box, one,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// [head][plan of up to B groups][(max, sum)][O]
static size_t px_space(int B, int Hq, int D, int P, void* base, PxSpace* ws) {
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    const size_t places = 2 * static_cast<size_t>(P) * kPxSlot + 2 * static_cast<size_t>(B) * Hq;
    const size_t plan = 256;
    const size_t ml = up(plan + sizeof(int2) * static_cast<size_t>(B)), o = up(ml + places * sizeof(float2));
    if (ws != nullptr) {
        uint8_t* p = static_cast<uint8_t*>(base);
        ws->head = reinterpret_cast<PxHead*>(p);
        ws->plan = reinterpret_cast<int2*>(p + plan);
        ws->ml = reinterpret_cast<float2*>(p + ml);
        ws->o = reinterpret_cast<float*>(p + o);
    }
    return up(o + places * D * sizeof(float));
}

template <int kD>
static cudaError_t launch_shared(const PxPlan& px, SplitPlan pl, void* out, const void* q, const void* k, const void* v,
                                 const int32_t* block_tables, const int32_t* seq_lens, void* workspace, int P,
                                 int32_t* status, cudaStream_t stream) {
    CUtensorMap tmK, tmV;
    const long long rows = static_cast<long long>(pl.NB) * pl.Hkv * pl.BS;
    if (kD == 64 ? !encode_pool_rows64(&tmK, k, rows) || !encode_pool_rows64(&tmV, v, rows)
                 : !encode_pool_k16(&tmK, k, pl.NB, pl.Hkv, pl.BS) || !encode_pool_box_halves(&tmV, v, pl.NB, pl.Hkv, pl.BS, 16))
        return cudaErrorInvalidValue;
    PxSpace pws = {};
    SplitSpace ws = {};
    const size_t used = px_space(pl.B, pl.Hq, pl.D, P, workspace, &pws);
    split_space(pl, P, pl.B, true, static_cast<uint8_t*>(workspace) + used, &ws);
    const bool sloped = pl.sc.slopes != nullptr;
    auto kern = pl.sc.cap_log2 > 0.f ? (sloped ? prefix_tc_kernel<kD, true, true> : prefix_tc_kernel<kD, true, false>)
                                     : (sloped ? prefix_tc_kernel<kD, false, true> : prefix_tc_kernel<kD, false, false>);
    cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kPxSmem<kD>));
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(P), 1, 1);
    cfg.blockDim = dim3(kPxThreads, 1, 1);
    cfg.dynamicSmemBytes = kPxSmem<kD>;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    err = cudaLaunchKernelEx(&cfg, kern, tmK, tmV, px, static_cast<const __nv_bfloat16*>(q), block_tables, seq_lens, pws, status);
    if (err != cudaSuccess) return err;
    bool done = false;
    err = launch_split_shared(pl, ws, q, k, v, block_tables, seq_lens, P, status, stream, &done);
    if (err != cudaSuccess || !done) return err != cudaSuccess ? err : cudaErrorInvalidValue;
    const long long n = static_cast<long long>(pl.B) * pl.Hq;
    const bool many = n >= kSjManyRows * P;
    const int per = many ? kSjWarps : 1;  // rows of a CTA
    cfg.gridDim = dim3(static_cast<unsigned>((n + per - 1) / per), 1, 1);
    cfg.blockDim = dim3(kSjWarps * 32, 1, 1);
    cfg.dynamicSmemBytes = 0;
    err = cudaLaunchKernelEx(&cfg, many ? shared_join_kernel<kD, 1> : shared_join_kernel<kD, kSjWarps>, px, pws, ws, pl.R, seq_lens, static_cast<__nv_bfloat16*>(out), P, status);
    return err != cudaSuccess ? err : cudaGetLastError();
}

}  // namespace pkv

extern "C" size_t pkv_decode_shared_workspace_bytes(int B, int Hq, int Hkv, int D, int num_sms) {
    using namespace pkv;
    const size_t plain = pkv_decode_scored_workspace_bytes(B, Hq, Hkv, D, num_sms);
    if (plain == 0) return 0;
    const int P = num_sms > 0 ? num_sms : device_sm_count();
    SplitPlan pl = {};
    pl.Hq = Hq;
    pl.D = D;
    if ((D != 64 && D != 128) || Hq / Hkv > kPxRows || !split_shape(Hq, Hkv, D, 16, 1, pl)) return plain;
    return std::max(plain, px_space(B, Hq, D, P, nullptr, nullptr) + split_space(pl, P, B, true, nullptr, nullptr));
}

extern "C" pkv_status pkv_paged_decode_attention_shared(
    void* out, const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
    int max_blocks_per_seq, const int32_t* seq_lens, const int32_t* group_start, const int32_t* shared_lens, int N,
    int B, int Hq, int Hkv, int D, int block_size, int num_blocks, float scale, float softcap, const float* slopes,
    pkv_dtype dtype, void* workspace, size_t workspace_bytes, int32_t* dev_status, void* stream) {
    using namespace pkv;
    ScoreArgs sc;
    if (!scored_shape_valid(B, Hq, Hkv, D, block_size, num_blocks, max_blocks_per_seq, dtype) ||
        !make_scores(&sc, scale, D, softcap, slopes, 0, nullptr) || N < 0 || N > B)
        return PKV_ERR_INVALID_ARG;
    if (N == 0)
        return pkv_paged_decode_attention_scored(out, q, k_cache, v_cache, block_tables, max_blocks_per_seq, seq_lens,
                                                 nullptr, B, Hq, Hkv, D, block_size, num_blocks, scale, softcap, slopes, 0,
                                                 dtype, workspace, workspace_bytes, dev_status, stream);
    if (!positions_fit(max_blocks_per_seq, block_size)) return PKV_ERR_UNSUPPORTED;
    if (!out || !q || !k_cache || !v_cache || !block_tables || !seq_lens || !group_start || !shared_lens || !workspace ||
        (reinterpret_cast<uintptr_t>(workspace) & 15u) != 0)
        return PKV_ERR_INVALID_ARG;
    SplitPlan pl = {};
    pl.B = B;
    pl.Hq = Hq;
    pl.Hkv = Hkv;
    pl.G = Hq / Hkv;
    pl.D = D;
    pl.BS = block_size;
    pl.NB = num_blocks;
    pl.max_blocks = max_blocks_per_seq;
    pl.sc = sc;
    pl.groups = GroupArgs{group_start, shared_lens, N};
    PxPlan px = {};
    px.B = B;
    px.Hq = Hq;
    px.Hkv = Hkv;
    px.G = pl.G;
    px.BS = block_size;
    px.NB = num_blocks;
    px.max_blocks = max_blocks_per_seq;
    px.TQ = pl.G <= kPxRows ? kPxRows / pl.G : 0;
    px.TC = kPxTiles * px.TQ;
    px.sc = sc;
    px.groups = pl.groups;
    if ((D != 64 && D != 128) || px.TQ == 0 || !split_applies(pl, out, q, k_cache, v_cache, dtype)) return PKV_ERR_UNSUPPORTED;
    px.NG = pl.NG;
    pl.TQ = px.TQ;
    px.units = pl.units;
    px.polls = pl.polls;
    px.silent_cta = pl.silent_cta;
    // pool rows and key tiles stay in 32 bits
    const long long tiles = (static_cast<long long>(max_blocks_per_seq) * block_size / kPxKeys + 1) * Hkv *
                            (static_cast<long long>(B) / px.TC + N);
    if (static_cast<long long>(num_blocks) * Hkv * block_size >= (1LL << 31) || tiles >= (1LL << 30)) return PKV_ERR_UNSUPPORTED;
    if (overlap(out, q, static_cast<size_t>(B) * Hq * D * 2)) return PKV_ERR_INVALID_ARG;
    const int P = device_sm_count();
    if (workspace_bytes < pkv_decode_shared_workspace_bytes(B, Hq, Hkv, D, P > 0 ? P : 1)) return PKV_ERR_INVALID_ARG;
    if (P <= 0) return PKV_ERR_CUDA;
    // Small batches, and such whose groups cannot have two members on average, are read per sequence
    const long long width = static_cast<long long>(max_blocks_per_seq) * block_size;
    if (B < 2 * N || 4LL * B * width * Hkv * D <= kPxReadPerSequence) {
        const cudaError_t err = launch_decode_scored(out, q, k_cache, v_cache, block_tables, max_blocks_per_seq, seq_lens, B, Hq,
                                                     Hkv, D, block_size, num_blocks, sc, pl.groups, dtype, workspace, P,
                                                     dev_status, static_cast<cudaStream_t>(stream));
        return err == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
    }
    const cudaError_t err = (D == 64 ? launch_shared<64> : launch_shared<128>)(
        px, pl, out, q, k_cache, v_cache, block_tables, seq_lens, workspace, P, dev_status, static_cast<cudaStream_t>(stream));
    return err == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}
