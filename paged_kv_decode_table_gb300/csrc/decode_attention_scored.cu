// decode_attention_scored.cu -- GQA paged decode attention with capped, biased and windowed scores
// (attention_scores.cuh has the definition), one query token per sequence.
//
// Fast path (bfloat16, D a multiple of 8 up to 128, block size a multiple of 16): a persistent kernel, one CTA per
// SM, over balanced ranges, and a kernel that joins the sequences that several ranges share.
//  * A tile is 16 positions of one KV head.  A step is slots x kSub units of 16 visible positions of HG KV heads,
//    fetched by TMA boxes of 64 dimensions x 16 positions x HG heads into one stage of an mbarrier ring; positions
//    that a window hides are walked past, except inside a unit.  The steps of all (sequence, head group) pairs, one
//    after the other, are cut into one range per CTA; every CTA finds its range itself from the lengths.
//  * One consumer warp per (KV head, chunk of its query heads, slot) takes kSub tiles of every step: with 8 KV heads
//    the 8 warps are the heads, with one head they are 8 slots along the cache.  The slots' results are merged in
//    shared memory when the range leaves the sequence.
//  * Both products run transposed on mma.sync m16n8k16 with float32 accumulation: S^T = K Q^T (16 positions x 8 query
//    heads) and O^T = V^T P^T (16 dimensions x 8 query heads), so the cached tile is the 16-row operand and no MMA
//    row is idle with 8 query heads.  movmatrix turns the weights from S^T's layout into P^T's.
//  * Scores, maxima, sums and products are float32; a weight is rounded once, to bfloat16 for the MMA (2^-8 of it;
//    V is bfloat16 and the MMA takes one type), its sum is of the unrounded ones.
//  * The maximum is renewed (shuffles, rescaled sums) only when a score exceeds it by 2^kSplitLag: a vote decides.
// mma.sync and not tcgen05: one query per sequence gives a KV head 1 to 16 rows, a 128-row tile would be empty rows, and
// the tensor pipe is 8% busy.
// What bounds it: HBM where the cache is large.  8 sequences of 32768-131072, 64 and 8 heads of 128: 412 us for 2.85 GB, 102%
// of the measured copy rate; 64 of 512-4096, 32 and 8 heads, capped: 94.8 us for 584 MB, 91%; 512 of 128-4096 that see 4 + 512
// positions: 175.0 us for 1.05 GB, 88% (units that a window cuts are read whole).  More than 8 query heads a KV head: 71%
// (two n-tiles a warp, whose chain of products is longer than its share of the copies).  One short sequence: 7 us, four
// dependent trips to memory.
//
// Generic kernel (float32, other shapes): one CTA per (sequence, KV head, up to 8 of its query heads, share of the visible
// positions).  Tiles of 32 visible positions come to shared memory as float32; warp w takes the scores of two query
// heads (a lane a position) and their running maxima and sums, then a thread takes four dimensions of two heads'
// outputs.  Positions that the mask hides are never loaded.  The shares' results are joined by a second kernel.
//
// No input is read through the read-only path (__ldg, const __restrict__): these kernels start while their
// predecessor still writes what they read after griddepcontrol.wait.
#include <cuda.h>
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "attention_split.cuh"

namespace pkv {

int device_sm_count();
int max_optin_smem();
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn get_encode_fn();
uint32_t attention_wait_polls();
int attention_silent_cta();

// ------------------------------------------------------------------ fast kernel
constexpr int kSplitStages = 12;  // at most
constexpr int kUnit = 16;         // positions per tile
constexpr int kSplitWarps = 8;    // consumer warps at most
// A score may exceed the running maximum that the weights are relative to by this many powers of two before
// the maximum is renewed: weights stay below 2^8, far inside float32 and bfloat16.
constexpr float kSplitLag = 8.f;

struct SplitMeta {
    int vb;  // sequence * NG + group
    int flags;
    int unit;  // the step's first unit of the walk
    int L, lo, pfx, near, gap;
};
enum : int { kSFirst = 1, kSLast = 2, kSWhole = 4, kSHead = 8, kSBad = 16 };

// What the walk over a sequence's visible units of 16 positions needs: unit u is unit u of the cache, from
// `near` on unit u + gap; n of them.
struct Span {
    Seen seen;
    int n, near, gap;
};
template <bool kShared>
__device__ __forceinline__ Span span_of(const SplitPlan& pl, const int32_t* seq_lens, int b) {
    Span s;
    s.near = s.gap = s.n = 0;
    const int L = seq_lens[b];
    s.seen = Seen{L, 0, 0};
    if (L <= 0 || static_cast<long long>(L) > static_cast<long long>(pl.max_blocks) * pl.BS) return s;
    if constexpr (kShared) {
        s.seen.lo = shared_prefix(pl.groups, pl.max_blocks, pl.BS, b);  // a multiple of the block size
        if (s.seen.lo < 0 || s.seen.lo >= L) return s;
    } else {
        s.seen = decode_seen(pl.sc, b, L);
        if (pl.groups.N > 0) {  // a call with shared prefixes that reads them per sequence: the same refusals
            const int shared = shared_prefix(pl.groups, pl.max_blocks, pl.BS, b);
            if (shared < 0 || L < shared) return s;
        }
    }
    s.near = (s.seen.pfx + kUnit - 1) / kUnit;
    const int first = max(s.near, s.seen.lo / kUnit);
    s.gap = first - s.near;
    s.n = s.near + (L + kUnit - 1) / kUnit - first;
    return s;
}
template <bool kShared>
__device__ __forceinline__ int steps_of(const SplitPlan& pl, const int32_t* seq_lens, int b) {
    const int per = pl.units;
    return (span_of<kShared>(pl, seq_lens, b).n + per - 1) / per;
}

// Sum over the CTA and this thread's exclusive prefix; red holds 33 ints.
__device__ __forceinline__ int split_scan(int v, int* red, int& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = (blockDim.x + 31) >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) red[warp] = x;
    __syncthreads();
    int before = 0, all = 0;
    for (int w = 0; w < nw; ++w) {
        const int r = red[w];
        if (w < warp) before += r;
        all += r;
    }
    __syncthreads();
    total = all;
    return before + x - v;
}

__device__ __forceinline__ void split_cp16(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
// One arrival on the barrier once this thread's earlier cp.async copies have landed.
__device__ __forceinline__ void split_cp_arrive(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// 8x8 16-bit numbers: row g, columns 2r, 2r + 1 -> row 2r (and 2r + 1) as column g
__device__ __forceinline__ uint32_t split_transpose(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

// What a consumer warp does whose wait ran out in step `left` of the CTA's range, which ends at `end` and begins at `from` (-1: a
// direct plan's only piece) in sequence b, whose first step is `at`.  Slot 0's warps, which leave the results, write zeros,
// or marks that become zeros in the join, for their heads' rows in the pieces that are not done.  (Another slot's warp
// that gives up lets slot 0's wait for it run out.)
template <int kHeads, bool kShared>
__device__ __noinline__ void split_give_up(const SplitPlan& pl, const int32_t* seq_lens, float2* ml, __nv_bfloat16* out,
                                           int32_t* status, int b, int at, int from, int left, int end, int slot, int hh,
                                           int qc) {
    const int lane = threadIdx.x & 31;
    if (lane == 0) report(status, PKV_ERR_TIMEOUT);
    if (slot != 0) return;
    if (from < 0) from = end - steps_of<kShared>(pl, seq_lens, b);
    for (; at < end; ++b) {
        const int n = steps_of<kShared>(pl, seq_lens, b);
        for (int g = 0; g < pl.NG; ++g, at += n) {
            if (min(at + n, end) <= max(left, at) || at + n <= from) continue;
            const bool whole = at >= from && at + n <= end;
            for (int head = qc * kHeads; head < min(pl.G, (qc + 1) * kHeads); ++head) {
                const int qr = hh * pl.G + head;
                if (g * pl.R + qr >= pl.Hq) continue;
                const size_t row = static_cast<size_t>(b) * pl.Hq + g * pl.R + qr;
                if (!kShared && whole) {
                    for (int e = lane; e < pl.D; e += 32) out[row * pl.D + e] = from_f32<__nv_bfloat16>(0.f);
                } else if (lane == 0) {
                    ml[whole ? 2 * static_cast<size_t>(gridDim.x) * pl.R + row
                             : (2 * static_cast<size_t>(blockIdx.x) + (at < from ? 0 : 1)) * pl.R + qr] =
                        make_float2(-INFINITY, -1.f);
                }
            }
        }
    }
}

// DP: dimensions computed, 64 or 128 (D may be smaller: the copies fill in zeros).  kN: n-tiles of 8 query heads
// per warp.  kShared: positions behind the shared prefix only, every piece left as a partial result.
template <int DP, int kN, bool kShared>
__global__ void __launch_bounds__((kSplitWarps + 1) * 32, 1)
    decode_split_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                        const __grid_constant__ SplitPlan pl, const __nv_bfloat16* q, __nv_bfloat16* out,
                        const int32_t* block_tables, const int32_t* seq_lens, const SplitSpace ws, int32_t* status) {
    constexpr bool kEstimate = kShared && shares_sms(8 * kN);
    constexpr int kHalves = DP / 64, kChunks = DP / 16, kSub = split_sub(DP), kHeads = 8 * kN;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int nst = pl.nst, HG = pl.HG, QC = pl.QC, slots = pl.slots;
    const int HV = HG * QC, CW = HV * slots, units = pl.units;
    const int half_bytes = HG * 2048, unit_bytes = kHalves * half_bytes, v_at = units * unit_bytes;
    uint8_t* qring = smem + static_cast<size_t>(nst) * pl.stage_bytes;
    float* scratch = reinterpret_cast<float*>(qring + pl.qslots * static_cast<size_t>(pl.q_bytes));
    uint64_t* full = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(scratch) + pl.scratch_bytes);
    uint64_t* empty = full + kSplitStages;
    uint64_t* qfull = empty + kSplitStages;
    uint64_t* qempty = qfull + 2;
    uint64_t* mfull = qempty + 2;  // merge slots: one per consumer warp
    uint64_t* mempty = mfull + kSplitWarps;
    SplitMeta* meta = reinterpret_cast<SplitMeta*>(mempty + kSplitWarps);
    int* sch = reinterpret_cast<int*>(meta + kSplitStages);  // [0, 33) scan scratch, 33: b0, 34: s0, 35: n, 36: start

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto finish = [] {  // before every exit
        if constexpr (kShared) asm volatile("griddepcontrol.wait;" ::: "memory");
    };
    // lengths, then block ids, then K and V: three dependent loads; the first two and q come to L2 while the
    // predecessor ends
    const unsigned worker = blockIdx.x * blockDim.x + threadIdx.x;
    prefetch_l2(seq_lens, static_cast<size_t>(pl.B) * 4, worker);
    prefetch_l2(block_tables, static_cast<size_t>(pl.B) * pl.max_blocks * 4, worker);
    prefetch_l2(q, static_cast<size_t>(pl.B) * pl.Hq * pl.D * 2, worker);
    if (threadIdx.x == 0) {
        for (int s = 0; s < nst; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], CW);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&qfull[s], 32);  // each producer lane's copies
            mbar_init(&qempty[s], CW);
        }
        for (int s = 0; s < kSplitWarps; ++s) {
            mbar_init(&mfull[s], 1);
            mbar_init(&mempty[s], 1);
        }
        fence_mbar_init();
        prefetch_tmap(&tmK);
        prefetch_tmap(&tmV);
    }
    // kShared: the predecessor is the prefix kernel, which started its dependents after its own wait; this kernel
    // reads nothing of it, and waits for it before it ends.
    if constexpr (!kShared) asm volatile("griddepcontrol.wait;" ::: "memory");
    // Only after the wait: the joining kernel's predecessors are complete then.
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    const int nthr = blockDim.x, B = pl.B, NG = pl.NG;
    if (!kShared && pl.groups.N > 0) {  // group_start is none: zeros for every sequence
        bool wrong = false;
        for (int g = threadIdx.x; g < pl.groups.N; g += nthr) wrong = wrong || !group_valid(pl.groups, B, g);
        if (__syncthreads_or(wrong)) {
            const size_t all = static_cast<size_t>(B) * pl.Hq * pl.D, step = static_cast<size_t>(gridDim.x) * nthr;
            for (size_t e = worker; e < all; e += step) out[e] = from_f32<__nv_bfloat16>(0.f);
            if (threadIdx.x == 0) {
                report(status, PKV_ERR_DEVICE_BOUNDS);
                if (!pl.direct) ws.cuts[blockIdx.x] = SplitCut{0, 0, 0, 0};
            }
            return;
        }
    }
    // ---- this CTA's range of steps: [start, end), which begins in sequence b0, whose first step is s0
    int W = 1, start, end, b0, s0;
    if (!kShared && pl.direct) {
        b0 = static_cast<int>(blockIdx.x) / NG;
        const int g = static_cast<int>(blockIdx.x) - b0 * NG, n = steps_of<kShared>(pl, seq_lens, b0);
        start = g * n;
        end = start + n;
        s0 = 0;
        if (n == 0) {  // empty or invalid: zeros
            const int rows = min(pl.R, pl.Hq - g * pl.R);
            __nv_bfloat16* o = out + (static_cast<size_t>(b0) * pl.Hq + g * pl.R) * pl.D;
            for (int e = threadIdx.x; e < rows * pl.D; e += nthr) o[e] = from_f32<__nv_bfloat16>(0.f);
            if (threadIdx.x == 0 && seq_lens[b0] != 0) report(status, PKV_ERR_DEVICE_BOUNDS);
            return;
        }
        __syncthreads();  // the barriers are initialised
    } else {
        [[maybe_unused]] int from = 0, to = 0, shared = 0;  // of group threadIdx.x: asked for before the lengths' chain
        if (kEstimate && static_cast<int>(threadIdx.x) < pl.groups.N) {
            from = pl.groups.start[threadIdx.x];
            to = pl.groups.start[threadIdx.x + 1];
            shared = pl.groups.shared[threadIdx.x];
        }
        const int n_first = static_cast<int>(threadIdx.x) < B ? NG * steps_of<kShared>(pl, seq_lens, threadIdx.x) : 0;
        int tsum = n_first;
        for (int b = threadIdx.x + nthr; b < B; b += nthr) tsum += NG * steps_of<kShared>(pl, seq_lens, b);
        int ranges = static_cast<int>(gridDim.x);
        [[maybe_unused]] SharedWork work;
        [[maybe_unused]] int* sums = reinterpret_cast<int*>(qring);  // (no query is there yet)
        if constexpr (kEstimate) {
            work.group(from, to, shared, pl.max_blocks, pl.BS, pl.TQ);
            for (int g = threadIdx.x + nthr; g < pl.groups.N; g += nthr)
                work.group(pl.groups.start[g], pl.groups.start[g + 1], pl.groups.shared[g], pl.max_blocks, pl.BS, pl.TQ);
            for (int b = threadIdx.x; b < B; b += nthr) work.sequence(seq_lens[b], pl.max_blocks, pl.BS);
            work.put(sums, warp, lane);
        }
        int total, before = split_scan(tsum, sch, total);
        if constexpr (kEstimate) {
            work.get(sums, nthr >> 5, lane);
            const int own = work.own_ctas(ranges, B, pl.groups.N, pl.Hkv, NG, pl.units, pl.sc.cap_log2 > 0.f, lane);
            if (own > 0) ranges = own;
        }
        if (total > 0) W = (total + ranges - 1) / ranges;
        start = min(total, static_cast<int>(blockIdx.x) * W);
        end = min(total, start + W);
        if constexpr (!kShared) {
            for (int b = blockIdx.x; b < B; b += gridDim.x) {  // sequences without steps: zeros
                if (steps_of<kShared>(pl, seq_lens, b) > 0) continue;
                __nv_bfloat16* o = out + static_cast<size_t>(b) * pl.Hq * pl.D;
                for (int e = threadIdx.x; e < pl.Hq * pl.D; e += nthr) o[e] = from_f32<__nv_bfloat16>(0.f);
                if (threadIdx.x == 0 && seq_lens[b] != 0) report(status, PKV_ERR_DEVICE_BOUNDS);
            }
        } else if (blockIdx.x == 0 && threadIdx.x == 0) {
            ws.head->W = W;
        }
        const bool idle = start >= end;
        if (idle && (!kShared || blockIdx.x != 0)) {  // uniform over the CTA
            if (!kShared && threadIdx.x == 0) ws.cuts[blockIdx.x] = SplitCut{0, 0, 0, 0};
            finish();
            return;
        }
        int carry = 0;
        for (int base = 0; base < B; base += nthr) {
            const int b = base + threadIdx.x;
            int n = n_first, tot = total;
            if (B > nthr) {  // else the scan above was this one
                if (base > 0) n = b < B ? NG * steps_of<kShared>(pl, seq_lens, b) : 0;
                before = split_scan(n, sch, tot);
            }
            const int sb = carry + before;
            if (n > 0 && sb <= start && start < sb + n) {  // exactly one thread of the CTA
                sch[33] = b;
                sch[34] = sb;
                sch[35] = n / NG;
            }
            if (kShared && blockIdx.x == 0 && b < B) ws.info[b] = make_int2(sb, n / NG);
            carry += tot;
            if (carry > start && !(kShared && blockIdx.x == 0)) break;  // same decision in every thread
        }
        if (idle) {
            finish();
            return;
        }
        if (threadIdx.x == 0) sch[36] = start;
        __syncthreads();
        b0 = sch[33];
        s0 = sch[34];
        if (!kShared && threadIdx.x == 0) {
            // the first range that begins inside a piece (a sequence's steps in one head group) has it joined
            const int n = sch[35], g = (start - s0) / n, first = s0 + g * n, f = first / W;
            const bool mine = first < start && f == static_cast<int>(blockIdx.x) - 1;
            ws.cuts[blockIdx.x] = SplitCut{b0, g, f, mine ? (first + n - 1) / W - f + 1 : 0};
        }
    }

    if (warp == CW) {
        // ------------------------------------------------ producer warp
        // Lane u fetches unit u of the step (slot u % slots).  Block ids are read two steps ahead.
        int b = b0, cs = s0, g = 0;
        Span sp = span_of<kShared>(pl, seq_lens, b);
        int cn = (sp.n + units - 1) / units;
        struct Step {
            int b, g, j, n, cs;
            Span sp;
            bool in;  // lane u: unit u lies before the end
            int blk;  // lane u: the block of unit u as the table has it, any integer
            int tok;  // lane u: the unit's first slot in its block
        };
        auto fetch = [&](int i) {  // walk on to step i
            while (cs + cn <= i) {
                cs += cn;
                if (++g == NG || cn == 0) {
                    g = 0;
                    ++b;
                    sp = span_of<kShared>(pl, seq_lens, b);
                    cn = (sp.n + units - 1) / units;
                }
            }
            Step s{b, g, i - cs, cn, cs, sp, false, -1, 0};
            const int u = s.j * units + lane;
            if (lane < units && u < sp.n) {
                const unsigned at = static_cast<unsigned>(u < sp.near ? u : u + sp.gap);
                s.in = true;
                const unsigned lb = pl.UB == 1 ? at : at / static_cast<unsigned>(pl.UB);
                s.tok = static_cast<int>(at - lb * pl.UB) * kUnit;
                s.blk = block_tables[static_cast<size_t>(b) * pl.max_blocks + lb];
            }
            return s;
        };
        if (static_cast<int>(blockIdx.x) == pl.silent_cta) {  // test hook: no copy is issued
            finish();
            return;
        }
        Step cur = fetch(start), nxt = cur;
        if (start + 1 < end) nxt = fetch(start + 1);
        const uint32_t unit_tx = 2u * unit_bytes;
        int piece = 0;
        // before every exit: wait for this warp's copies in flight, so that none writes into shared memory after
        // the CTA is gone, whether its consumers still wait for them or have given up (bounded, but not by the limit that a
        // test lowers: copies that were issued land)
        auto drain = [&](int it) {
            asm volatile("cp.async.wait_all;" ::: "memory");
            if (lane != 0) return;
            for (int k = max(0, it - nst); k < it; ++k)
                mbar_wait(&full[k % nst], static_cast<uint32_t>(k / nst) & 1u);
        };
        // 16-byte chunks of a row of q; this lane's first one, and the step to its next one
        const int q_chunks = pl.D / 8;
        const int q_row = lane / q_chunks, q_col = lane - q_row * q_chunks;
        const int q_drow = 32 / q_chunks, q_dcol = 32 - q_drow * q_chunks;
        int stage = 0;
        uint32_t parity = 1;  // of the empty barriers: the first round finds them free
        for (int i = start, it = 0; i < end; ++i, ++it) {
            const Step s = cur;
            cur = nxt;
            if (i + 2 < end) nxt = fetch(i + 2);
            const bool first = s.j == 0 || i == start, last = s.j == s.n - 1 || i == end - 1;
            const bool good = s.in && s.blk >= 0 && s.blk < pl.NB;
            const unsigned live = __ballot_sync(0xffffffffu, good);
            const bool bad = __any_sync(0xffffffffu, s.in && !good);
            bool ok = mbar_wait(&empty[stage], parity, pl.polls);
            if (first && ok)
                ok = mbar_wait(&qempty[pl.qslots == 2 ? piece & 1 : 0],
                               (static_cast<uint32_t>(piece >> (pl.qslots - 1)) & 1u) ^ 1u, pl.polls);
            if (!__all_sync(0xffffffffu, ok)) {
                if (lane == 0) report(status, PKV_ERR_TIMEOUT);
                drain(it);
                finish();
                return;
            }
            if (lane == 0) {
                SplitMeta mt;
                mt.vb = s.b * NG + s.g;
                mt.flags = (first ? kSFirst : 0) | (last ? kSLast : 0) |
                           (s.cs >= start && s.cs + s.n <= end ? kSWhole : 0) | (s.cs < start ? kSHead : 0) |
                           (bad ? kSBad : 0);
                mt.unit = s.j * units;
                mt.L = s.sp.seen.L;
                mt.lo = s.sp.seen.lo;
                mt.pfx = s.sp.seen.pfx;
                mt.near = s.sp.near;
                mt.gap = s.sp.gap;
                meta[stage] = mt;
                mbar_arrive_expect_tx(&full[stage], __popc(live) * unit_tx);  // releases the metadata
            }
            __syncwarp();
            if (good) {
                const int row = s.blk * pl.Hkv + s.g * HG;
                uint8_t* kd = smem + static_cast<size_t>(stage) * pl.stage_bytes + lane * unit_bytes;
#pragma unroll
                for (int x = 0; x < kHalves; ++x) tma_load_3d(kd + x * half_bytes, &tmK, 64 * x, s.tok, row, &full[stage]);
#pragma unroll
                for (int x = 0; x < kHalves; ++x)
                    tma_load_3d(kd + v_at + x * half_bytes, &tmV, 64 * x, s.tok, row, &full[stage]);
            }
            if (first) {
                const int qs = pl.qslots == 2 ? piece & 1 : 0;
                const int rows = min(pl.R, pl.Hq - s.g * pl.R);  // the last group may have fewer heads
                const uint8_t* src = reinterpret_cast<const uint8_t*>(
                    q + (static_cast<size_t>(s.b) * pl.Hq + static_cast<size_t>(s.g) * pl.R) * pl.D);
                uint8_t* dst = qring + static_cast<size_t>(qs) * pl.q_bytes;
                int row = q_row, col = q_col;
                for (int x = lane; x < rows * q_chunks; x += 32) {
                    split_cp16(dst + row * (2 * DP) + ((col ^ (row & 7)) << 4), src + static_cast<size_t>(x) * 16);
                    row += q_drow;
                    col += q_dcol;
                    if (col >= q_chunks) {
                        col -= q_chunks;
                        ++row;
                    }
                }
                split_cp_arrive(&qfull[qs]);
                ++piece;
            }
            if (bad && lane == 0) report(status, PKV_ERR_DEVICE_BOUNDS);
            if (++stage == nst) {
                stage = 0;
                parity ^= 1u;
            }
        }
        drain(end - start);
        finish();
        return;
    }

    // ---------------------------------------------------- consumers
    const int slot = warp / HV, vh = warp - slot * HV, hh = vh / QC, qc = vh - hh * QC;
    const int g = lane >> 2, r = lane & 3, mi = lane >> 3, rr = lane & 7;
    // O^T: [16-dim chunk][n-tile][dim g of head 2r, 2r + 1, dim g + 8 of head 2r, 2r + 1]
    float O[kChunks][kN][4];
    uint32_t qb[kN][kChunks][2];
    float slope[kN][2], m[kN][2], mu[kN][2], l[kN][2];  // of heads 8 n + 2 r + e; mu: m, 0 while m is -infinity
    bool poisoned = false;
    int piece = 0, stage = 0;
    uint32_t parity = 0;
    const uint32_t smem_base = smem_u32(smem);
    const bool capped = pl.sc.cap_log2 > 0.f, sloped = pl.sc.slopes != nullptr;
    // ldmatrix: lane group mi gives the rows of matrix mi: (positions 8 (mi & 1) .., 16-byte chunk + (mi >> 1))
    uint32_t lm[4];
#pragma unroll
    for (int c = 0; c < 4; ++c)
        lm[c] = hh * 2048 + ((mi & 1) * 8 + rr) * 128 + (((2 * c + (mi >> 1)) ^ rr) << 4);

    // One step's kSub tiles.
    auto tiles = [&](const SplitMeta& mt) {
        const uint32_t kb0 = smem_base + static_cast<uint32_t>(stage) * pl.stage_bytes + slot * unit_bytes;
        float x[kSub][kN][4];  // scores of position g (+ 8 for 2, 3), heads 2r, 2r + 1
        bool over = false;
        float tmax[kN][2];
        int p0[kSub];  // the tile's first position; -1: no such tile
        bool part[kSub];  // some positions do not take part
#pragma unroll
        for (int n = 0; n < kN; ++n) tmax[n][0] = tmax[n][1] = -INFINITY;
        const Seen seen{mt.L, mt.lo, mt.pfx};
#pragma unroll
        for (int k = 0; k < kSub; ++k) {
            const int u = mt.unit + k * slots + slot;
            p0[k] = kUnit * (u < mt.near ? u : u + mt.gap);
            part[k] = p0[k] + kUnit > mt.L || (p0[k] < mt.lo && p0[k] + kUnit > mt.pfx);
            if (p0[k] >= mt.L) {  // uniform over the warp
                p0[k] = -1;
                continue;
            }
            // ---- S^T = K Q^T, in two independent chains
            const uint32_t kb = kb0 + k * slots * unit_bytes;
            float s[kN][2][4];
#pragma unroll
            for (int n = 0; n < kN; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[n][0][e] = s[n][1][e] = 0.f;
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
                uint32_t a[4];
                ldmatrix_x4(a[0], a[1], a[2], a[3], kb + (c >> 2) * half_bytes + lm[c & 3]);
#pragma unroll
                for (int n = 0; n < kN; ++n) mma_bf16_16816(s[n][c & 1], a, qb[n][c][0], qb[n][c][1]);
            }
            // ---- scores
            if (capped) {
                float z[kN][4];
                bool large = false;
#pragma unroll
                for (int n = 0; n < kN; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        z[n][e] = (s[n][0][e] + s[n][1][e]) * pl.sc.in;
                        large = large || fabsf(z[n][e]) > 1.f;
                    }
                if (__any_sync(0xffffffffu, large)) {
#pragma unroll
                    for (int n = 0; n < kN; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            x[k][n][e] = pl.sc.cap_log2 * (fabsf(z[n][e]) > 1.f ? tanh_beyond(z[n][e]) : tanh_within(z[n][e]));
                } else {
#pragma unroll
                    for (int n = 0; n < kN; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) x[k][n][e] = pl.sc.cap_log2 * tanh_within(z[n][e]);
                }
            } else {
#pragma unroll
                for (int n = 0; n < kN; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[k][n][e] = (s[n][0][e] + s[n][1][e]) * pl.sc.mul;
            }
            if (sloped) {
                // the bias's distances: from the last key, and from the sequence's first one that takes part
                const float dist = static_cast<float>(p0[k] + g - (mt.L - 1)),
                            dist_first = static_cast<float>(p0[k] + g - (kShared ? 0 : seen.first()));
#pragma unroll
                for (int n = 0; n < kN; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        x[k][n][e] = fmaf(slope[n][e & 1], (slope[n][e & 1] < 0.f ? dist_first : dist) + static_cast<float>(8 * (e >> 1)),
                                          x[k][n][e]);
            }
            if (part[k]) {
                const bool in0 = seen.at(p0[k] + g), in1 = seen.at(p0[k] + g + 8);
#pragma unroll
                for (int n = 0; n < kN; ++n) {
                    if (!in0) x[k][n][0] = x[k][n][1] = -INFINITY;
                    if (!in1) x[k][n][2] = x[k][n][3] = -INFINITY;
                }
            }
#pragma unroll
            for (int n = 0; n < kN; ++n) {
                tmax[n][0] = fmaxf(tmax[n][0], fmaxf(x[k][n][0], x[k][n][2]));
                tmax[n][1] = fmaxf(tmax[n][1], fmaxf(x[k][n][1], x[k][n][3]));
            }
        }
#pragma unroll
        for (int n = 0; n < kN; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) over = over || tmax[n][e] > m[n][e] + kSplitLag;
        if (__any_sync(0xffffffffu, over)) {  // renew the maxima, rescale what was summed so far
#pragma unroll
            for (int n = 0; n < kN; ++n) {
                float al[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float mx = tmax[n][e];
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                    const float mn = fmaxf(m[n][e], mx);
                    mu[n][e] = mn == -INFINITY ? 0.f : mn;
                    al[e] = ex2_approx(m[n][e] - mu[n][e]);
                    m[n][e] = mn;
                    l[n][e] *= al[e];
                }
#pragma unroll
                for (int c = 0; c < kChunks; ++c) {
                    O[c][n][0] *= al[0];
                    O[c][n][1] *= al[1];
                    O[c][n][2] *= al[0];
                    O[c][n][3] *= al[1];
                }
            }
        }
        // ---- weights, in P^T's layout; their sum is of the float32 ones
        uint32_t pb[kSub][kN][2];
        float lsum[kN][2];
#pragma unroll
        for (int n = 0; n < kN; ++n) lsum[n][0] = lsum[n][1] = 0.f;
#pragma unroll
        for (int k = 0; k < kSub; ++k) {
            if (p0[k] < 0) break;
#pragma unroll
            for (int n = 0; n < kN; ++n)
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const float w0 = ex2_approx(x[k][n][2 * t] - mu[n][0]), w1 = ex2_approx(x[k][n][2 * t + 1] - mu[n][1]);
                    lsum[n][0] += w0;
                    lsum[n][1] += w1;
                    pb[k][n][t] = split_transpose(pack_bf16x2(w0, w1));
                }
        }
#pragma unroll
        for (int n = 0; n < kN; ++n) {
            l[n][0] += lsum[n][0];
            l[n][1] += lsum[n][1];
        }
        // V rows that do not take part have weight 0, but may hold anything: cleared
        uint32_t keep[kSub][2];
#pragma unroll
        for (int k = 0; k < kSub; ++k)
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const int j = p0[k] + 8 * t + 2 * r;
                keep[k][t] = (seen.at(j) ? 0xffffu : 0u) | (seen.at(j + 1) ? 0xffff0000u : 0u);
            }
        // ---- O^T += V^T P^T.  A step's products are summed apart and added by rounded additions: the MMA
        // truncates what it adds to about 2^-24 of its accumulator, which over a long sequence is a bias.
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            float F[kN][4];
#pragma unroll
            for (int n = 0; n < kN; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) F[n][e] = 0.f;
#pragma unroll
            for (int k = 0; k < kSub; ++k) {
                if (p0[k] < 0) break;
                uint32_t a[4];
                ldmatrix_x4_trans(a[0], a[2], a[1], a[3], kb0 + k * slots * unit_bytes + v_at + (c >> 2) * half_bytes + lm[c & 3]);
                if (part[k]) {
                    a[0] &= keep[k][0];
                    a[1] &= keep[k][0];
                    a[2] &= keep[k][1];
                    a[3] &= keep[k][1];
                }
#pragma unroll
                for (int n = 0; n < kN; ++n) mma_bf16_16816(F[n], a, pb[k][n][0], pb[k][n][1]);
            }
#pragma unroll
            for (int n = 0; n < kN; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) O[c][n][e] += F[n][e];
        }
    };

    // The step in which a wait ran out, or `end`.
    auto consume = [&]() -> int {
        for (int i = start; i < end; ++i) {
            if (!mbar_wait(&full[stage], parity, pl.polls)) return i;
            const SplitMeta mt = meta[stage];
            if (mt.flags & kSFirst) {
                const int qs = pl.qslots == 2 ? piece & 1 : 0;
                if (!mbar_wait(&qfull[qs], static_cast<uint32_t>(piece >> (pl.qslots - 1)) & 1u, pl.polls)) return i;
                const uint8_t* qsm = qring + static_cast<size_t>(qs) * pl.q_bytes;
                const int head0 = ((mt.vb % NG) * HG + hh) * pl.G;
                // (none for the heads that a last, smaller group lacks)
                const int qrows = (mt.vb % NG) * HG + hh < pl.Hkv ? pl.G : 0;
#pragma unroll
                for (int n = 0; n < kN; ++n) {
                    const int row = qc * kHeads + 8 * n + g;
#pragma unroll
                    for (int c = 0; c < kChunks; ++c)
#pragma unroll
                        for (int p = 0; p < 2; ++p) {
                            const int at = hh * pl.G + row;
                            qb[n][c][p] = row < qrows && 16 * c + 8 * p < pl.D
                                              ? *reinterpret_cast<const uint32_t*>(
                                                    qsm + at * (2 * DP) + (((2 * c + p) ^ (at & 7)) << 4) + 4 * r) : 0u;
                        }
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int hd = qc * kHeads + 8 * n + 2 * r + e;
                        slope[n][e] = pl.sc.slopes != nullptr && hd < qrows ? pl.sc.slopes[head0 + hd] * kLog2e : 0.f;
                        m[n][e] = -INFINITY;
                        mu[n][e] = l[n][e] = 0.f;
                    }
#pragma unroll
                    for (int c = 0; c < kChunks; ++c) O[c][n][0] = O[c][n][1] = O[c][n][2] = O[c][n][3] = 0.f;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&qempty[qs]);
                poisoned = false;
            }
            poisoned = poisoned || (mt.flags & kSBad);
            if (!poisoned) tiles(mt);
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[stage]);
            if (++stage == nst) {
                stage = 0;
                parity ^= 1u;
            }
            if (!(mt.flags & kSLast)) continue;

            // ---------------------------------------------- the range leaves (sequence, group) mt.vb
#pragma unroll
            for (int n = 0; n < kN; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], o);
            if (slots > 1) {
                // merge the slots: at distance d = slots / 2, .., 1 warp slot in [d, 2d) hands its result to slot - d
                // through its own scratch tile (rows padded by 4 floats so that the 4 pairs of heads a store touches
                // fall on different banks).  Each wait is bounded.
                constexpr int kRow = DP + 4, kTile = kHeads * (kRow + 2);
                const uint32_t ph = static_cast<uint32_t>(piece) & 1u;
                bool sent = false;
                for (int d = slots >> 1; d > 0; d >>= 1) {
                    if (slot >= d) {
                        float* t = scratch + ((slot - 1) * HV + vh) * kTile;
                        if (!mbar_wait(&mempty[warp], ph ^ 1u, pl.polls)) return i;
#pragma unroll
                        for (int n = 0; n < kN; ++n)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const int head = 8 * n + 2 * r + e;
#pragma unroll
                                for (int c = 0; c < kChunks; ++c) {
                                    t[head * kRow + 16 * c + g] = O[c][n][e];
                                    t[head * kRow + 16 * c + 8 + g] = O[c][n][2 + e];
                                }
                                if (g == 0)
                                    *reinterpret_cast<float2*>(t + kHeads * kRow + 2 * head) = make_float2(m[n][e], l[n][e]);
                            }
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&mfull[warp]);
                        sent = true;
                        break;
                    }
                    const int from = warp + d * HV;
                    const float* t = scratch + ((slot + d - 1) * HV + vh) * kTile;
                    if (!mbar_wait(&mfull[from], ph, pl.polls)) return i;
#pragma unroll
                    for (int n = 0; n < kN; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int head = 8 * n + 2 * r + e;
                            const float2 ml = *reinterpret_cast<const float2*>(t + kHeads * kRow + 2 * head);
                            const float mn = fmaxf(m[n][e], ml.x), base = mn == -INFINITY ? 0.f : mn;
                            const float fa = ex2_approx(m[n][e] - base), fb = ex2_approx(ml.x - base);
                            m[n][e] = mn;
                            l[n][e] = fmaf(l[n][e], fa, ml.y * fb);
#pragma unroll
                            for (int c = 0; c < kChunks; ++c) {
                                O[c][n][e] = fmaf(O[c][n][e], fa, t[head * kRow + 16 * c + g] * fb);
                                O[c][n][2 + e] = fmaf(O[c][n][2 + e], fa, t[head * kRow + 16 * c + 8 + g] * fb);
                            }
                        }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&mempty[from]);
                }
                ++piece;
                if (sent) continue;
            } else {
                ++piece;
            }
            const int vb_g = mt.vb % NG, vb_b = mt.vb / NG;
#pragma unroll
            for (int n = 0; n < kN; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int head = qc * kHeads + 8 * n + 2 * r + e;
                    const int qr = hh * pl.G + head;  // row in the group
                    if (head >= pl.G || vb_g * pl.R + qr >= pl.Hq) continue;
                    const size_t row = static_cast<size_t>(vb_b) * pl.Hq + vb_g * pl.R + qr;  // row of out
                    if (!kShared && (mt.flags & kSWhole)) {
                        const float inv = poisoned || l[n][e] == 0.f ? 0.f : 1.f / l[n][e];
                        __nv_bfloat16* o = out + row * pl.D + g;
#pragma unroll
                        for (int c = 0; c < kChunks; ++c) {
                            if (16 * c < pl.D) o[16 * c] = from_f32<__nv_bfloat16>(poisoned ? 0.f : O[c][n][e] * inv);
                            if (16 * c + 8 < pl.D) o[16 * c + 8] = from_f32<__nv_bfloat16>(poisoned ? 0.f : O[c][n][2 + e] * inv);
                        }
                    } else {
                        size_t at = (2 * static_cast<size_t>(blockIdx.x) + ((mt.flags & kSHead) ? 0 : 1)) * pl.R + qr;
                        if (kShared && (mt.flags & kSWhole)) at = 2 * static_cast<size_t>(gridDim.x) * pl.R + row;
                        if (g == 0) ws.ml[at] = make_float2(m[n][e], poisoned ? -1.f : l[n][e]);
                        float* o = ws.o + at * pl.D + g;
#pragma unroll
                        for (int c = 0; c < kChunks; ++c) {
                            if (16 * c < pl.D) o[16 * c] = O[c][n][e];
                            if (16 * c + 8 < pl.D) o[16 * c + 8] = O[c][n][2 + e];
                        }
                    }
                }
        }
        return end;
    };
    const int left = consume();
    if (left < end) {
        const int bb = !kShared && pl.direct ? static_cast<int>(blockIdx.x) / NG : sch[33];
        split_give_up<kHeads, kShared>(pl, seq_lens, ws.ml, out, status, bb, !kShared && pl.direct ? 0 : sch[34],
                                       !kShared && pl.direct ? -1 : sch[36], left, end, slot, hh, qc);
    }
    finish();
}

// ------------------------------------------------------------------ join
// M = max m_c, out = sum o_c 2^(m_c - M) / sum l_c 2^(m_c - M) over the pieces of a sequence that several ranges
// share: the piece of its first range f in slot 2f + 1, of a later range c in slot 2c.  CTAs go over the ranges'
// starts; the first start inside a piece joins it, a warp a row.
constexpr int kJoinWarps = 4;
constexpr int kJoinGroup = 8;  // pieces in flight

__global__ void __launch_bounds__(kJoinWarps * 32)
    decode_split_join_kernel(const __grid_constant__ SplitPlan pl, const SplitSpace ws, __nv_bfloat16* out) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int per = (pl.R + kJoinWarps - 1) / kJoinWarps, c = 1 + static_cast<int>(blockIdx.x) / per;
    const int4 c4 = __ldcg(reinterpret_cast<const int4*>(ws.cuts + c));
    const SplitCut cut{c4.x, c4.y, c4.z, c4.w};
    const int row = (static_cast<int>(blockIdx.x) - (c - 1) * per) * kJoinWarps + warp;
    if (cut.pieces == 0 || row >= min(pl.R, pl.Hq - cut.g * pl.R)) return;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float M = -INFINITY, l = 0.f;
    bool bad = false;
    const bool col = 4 * lane < pl.D;
    for (int p0 = 0; p0 < cut.pieces; p0 += kJoinGroup) {
        float2 ml[kJoinGroup];
        float4 o[kJoinGroup];
#pragma unroll
        for (int k = 0; k < kJoinGroup; ++k) {
            const int p = p0 + k;
            const size_t at = (static_cast<size_t>(2 * (cut.f + p) + (p == 0 ? 1 : 0))) * pl.R + row;
            ml[k] = p < cut.pieces ? __ldcg(ws.ml + at) : make_float2(-INFINITY, 0.f);
            o[k] = p < cut.pieces && col ? __ldcg(reinterpret_cast<const float4*>(ws.o + at * pl.D + 4 * lane))
                                         : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        float mn = M;
#pragma unroll
        for (int k = 0; k < kJoinGroup; ++k) mn = fmaxf(mn, ml[k].x);
        const float mu = mn == -INFINITY ? 0.f : mn, fa = ex2_approx(M - mu);
        l *= fa;
        acc = make_float4(acc.x * fa, acc.y * fa, acc.z * fa, acc.w * fa);
        M = mn;
#pragma unroll
        for (int k = 0; k < kJoinGroup; ++k) {
            const float w = ex2_approx(ml[k].x - mu);
            bad = bad || ml[k].y < 0.f;  // a piece that could not be read makes the row zero
            l = fmaf(ml[k].y, w, l);
            acc.x = fmaf(o[k].x, w, acc.x);
            acc.y = fmaf(o[k].y, w, acc.y);
            acc.z = fmaf(o[k].z, w, acc.z);
            acc.w = fmaf(o[k].w, w, acc.w);
        }
    }
    if (!col) return;
    const float inv = 1.f / l;
    const bool zero = bad || l == 0.f;
    const uint2 v = zero ? make_uint2(0u, 0u)
                         : make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
    *reinterpret_cast<uint2*>(out + (static_cast<size_t>(cut.b) * pl.Hq + cut.g * pl.R + row) * pl.D + 4 * lane) = v;
}

// ------------------------------------------------------------------ generic kernel
constexpr int kGenThreads = 128;
constexpr int kGenPos = 32;    // positions a tile
constexpr int kGenHeads = 8;   // query heads a CTA, two a warp
constexpr int kGenShares = 64;  // at most

struct GenericPlan {
    int B, Hq, Hkv, G, D, BS, NB, max_blocks;
    int chunks, shares;  // CTAs along the heads and along the positions of a (sequence, KV head)
    int stride;          // floats between rows in shared memory
    ScoreArgs sc;
};

// Rows a multiple of 4 floats apart with an odd quotient: eight rows' 16-byte reads fall on different banks.
static int generic_stride(int D) {
    const int quads = (D + 3) / 4;
    return 4 * (quads | 1);
}
// float32 rows of whole 16 bytes are copied as they are, a tile ahead; other rows are converted on their way.
template <typename T, bool kVec>
constexpr bool kGenAhead = kVec && sizeof(T) == 4;

// Bound by the chain of a tile (copy, scores, products, with a barrier between them) and by shared-memory reads: a position's
// K and V row are read once for two heads, 12 bytes of shared memory a byte of cache with 8 heads.  16 sequences of 512-4096, 32
// and 8 heads of 128 in float32: 145 us for 302 MB, 31% of the copy rate.  Short batches: lengths, block ids, rows and the join one
// after the other; 37 sequences of up to 1500 (window 300), 21 and 3 heads of 80 in float32 17.4 us for 20 MB.
template <typename T, bool kVec>
__global__ void __launch_bounds__(kGenThreads)
    decode_scored_generic_kernel(const __grid_constant__ GenericPlan pl, T* out, const T* q, const T* k_cache,
                                 const T* v_cache, const int32_t* block_tables, const int32_t* seq_lens, float* part,
                                 int32_t* status) {
    constexpr bool kAhead = kGenAhead<T, kVec>;
    extern __shared__ __align__(16) float gen_smem[];
    __shared__ __align__(16) float ps[kGenHeads][kGenPos];
    __shared__ float factor[kGenHeads], ends[kGenHeads][2];
    __shared__ long long rows[2][kGenPos];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, D = pl.D, DS = pl.stride;
    const int tile_floats = 2 * kGenPos * DS;  // K rows, V rows
    float* qs = gen_smem + (kAhead ? 2 : 1) * tile_floats;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    unsigned u = blockIdx.x;
    const int share = static_cast<int>(u % pl.shares);
    u /= pl.shares;
    const int chunk = static_cast<int>(u % pl.chunks);
    u /= pl.chunks;
    const int h = static_cast<int>(u % pl.Hkv), b = static_cast<int>(u / pl.Hkv);
    const int nh = min(kGenHeads, pl.G - chunk * kGenHeads);  // heads of this CTA
    const size_t row0 = static_cast<size_t>(b) * pl.Hq + h * pl.G + chunk * kGenHeads;
    const int L = seq_lens[b];
    bool bad = L < 0 || static_cast<long long>(L) > static_cast<long long>(pl.max_blocks) * pl.BS;
    const Seen seen = decode_seen(pl.sc, b, bad ? 0 : L);
    const int visible = seen.pfx + seen.L - seen.lo, tiles = (visible + kGenPos - 1) / kGenPos;
    const int per = (tiles + pl.shares - 1) / pl.shares, t0 = min(tiles, share * per), t1 = min(tiles, t0 + per);
    bool miss = false;
    auto position = [&](int i) { return i < seen.pfx ? i : seen.lo + (i - seen.pfx); };
    // warp 0: the block of its lane's position in tile t, asked for early; and the rows of the tile's positions
    auto ask = [&](int t) {
        const int i = t * kGenPos + lane;
        return t < t1 && i < visible ? block_tables[static_cast<size_t>(b) * pl.max_blocks + position(i) / pl.BS] : -1;
    };
    auto locate = [&](int t, int blk) {
        const int i = t * kGenPos + lane;
        long long row = -1;
        if (i < visible) {
            if (blk < 0 || blk >= pl.NB) miss = true;
            else row = (static_cast<long long>(blk) * pl.Hkv + h) * pl.BS + position(i) % pl.BS;
        }
        rows[t & 1][lane] = row;
    };
    int blk = -1;
    // Tile t to its place; rows that are not there, or behind the last, are left out.
    auto fetch = [&](int t) {
        float* to = gen_smem + (kAhead ? (t & 1) * tile_floats : 0);
        const int n = min(kGenPos, visible - t * kGenPos);
        if constexpr (kVec) {
            constexpr int kPer = 16 / static_cast<int>(sizeof(T));
            const int vecs = D / kPer;
            int p = tid / vecs, c = tid - p * vecs;
            const int dp = kGenThreads / vecs, dc = kGenThreads - dp * vecs;
            while (p < 2 * n) {
                const int which = p >= n, x = p - which * n;
                const long long row = rows[t & 1][x];
                if (row >= 0) {
                    const T* from = (which ? v_cache : k_cache) + row * D + c * kPer;
                    float* at = to + (which * kGenPos + x) * DS + c * kPer;
                    if constexpr (kAhead) {
                        split_cp16(at, from);
                    } else {
                        const uint4 z = *reinterpret_cast<const uint4*>(from);
                        reinterpret_cast<float4*>(at)[0] = make_float4(bf16_lo(z.x), bf16_hi(z.x), bf16_lo(z.y), bf16_hi(z.y));
                        reinterpret_cast<float4*>(at)[1] = make_float4(bf16_lo(z.z), bf16_hi(z.z), bf16_lo(z.w), bf16_hi(z.w));
                    }
                }
                p += dp;
                c += dc;
                if (c >= vecs) {
                    c -= vecs;
                    ++p;
                }
            }
        } else {
            for (int p = warp; p < n; p += kGenThreads / 32) {
                const long long row = rows[t & 1][p];
                if (row < 0) continue;
                const T *kr = k_cache + row * D, *vr = v_cache + row * D;
                for (int d = lane; d < D; d += 32) {
                    to[p * DS + d] = to_f32(kr[d]);
                    to[(kGenPos + p) * DS + d] = to_f32(vr[d]);
                }
            }
        }
        if constexpr (kAhead) asm volatile("cp.async.commit_group;" ::: "memory");
    };
    if (warp == 0) {
        const int blk0 = ask(t0), blk1 = ask(t0 + 1);
        blk = ask(t0 + 2);
        if (t0 < t1) locate(t0, blk0);
        if (t0 + 1 < t1) locate(t0 + 1, blk1);
    }
    // the dimensions between D and the next multiple of 4 are zeros
    for (int e = tid; e < kGenHeads * DS; e += kGenThreads) {
        const int hd = e / DS, d = e - hd * DS;
        qs[e] = hd < nh && d < D ? to_f32(q[(row0 + hd) * D + d]) : 0.f;
    }
    if ((D & 3) != 0)
        for (int e = tid; e < tile_floats; e += kGenThreads) gen_smem[e] = 0.f;
    bad = __syncthreads_or(miss) != 0 || bad;
    if constexpr (kAhead)
        if (!bad && t0 < t1) fetch(t0);
    const int quads = (D + 3) / 4;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};  // of heads 2 warp, 2 warp + 1
    float4 acc[2][2];  // [quad tid % .. of this thread][head of the pair]
#pragma unroll
    for (int a = 0; a < 2; ++a) acc[a][0] = acc[a][1] = make_float4(0.f, 0.f, 0.f, 0.f);
    float slope[2];
#pragma unroll
    for (int e = 0; e < 2; ++e)
        slope[e] = pl.sc.slopes != nullptr && 2 * warp + e < nh
                       ? pl.sc.slopes[h * pl.G + chunk * kGenHeads + 2 * warp + e] * kLog2e : 0.f;
    for (int t = t0; t < t1 && !bad; ++t) {
        const int n = min(kGenPos, visible - t * kGenPos);
        const float* ks = gen_smem + (kAhead ? (t & 1) * tile_floats : 0);
        const float* vs = ks + kGenPos * DS;
        if constexpr (kAhead) {
            if (t + 1 < t1) {
                fetch(t + 1);
                asm volatile("cp.async.wait_group 1;" ::: "memory");
            } else {
                asm volatile("cp.async.wait_group 0;" ::: "memory");
            }
        } else {
            fetch(t);
        }
        __syncthreads();  // the tile is there; the rows of tile t are used
        if (warp == 0 && t + 2 < t1) {
            locate(t + 2, blk);
            blk = ask(t + 3);
        }
        if (2 * warp < nh) {
            float x[2] = {-INFINITY, -INFINITY};
            if (lane < n) {
                const float4 *kr = reinterpret_cast<const float4*>(ks + lane * DS),
                             *q0 = reinterpret_cast<const float4*>(qs + 2 * warp * DS),
                             *q1 = reinterpret_cast<const float4*>(qs + (2 * warp + 1) * DS);
                float s[2][2] = {{0.f, 0.f}, {0.f, 0.f}};
#pragma unroll 4
                for (int c = 0; c < quads; ++c) {
                    const float4 a = kr[c], w0 = q0[c], w1 = q1[c];
                    s[0][0] = fmaf(a.x, w0.x, fmaf(a.y, w0.y, s[0][0]));
                    s[0][1] = fmaf(a.z, w0.z, fmaf(a.w, w0.w, s[0][1]));
                    s[1][0] = fmaf(a.x, w1.x, fmaf(a.y, w1.y, s[1][0]));
                    s[1][1] = fmaf(a.z, w1.z, fmaf(a.w, w1.w, s[1][1]));
                }
                const int j = position(t * kGenPos + lane);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    x[e] = s[e][0] + s[e][1];
                    x[e] = pl.sc.cap_log2 > 0.f ? pl.sc.cap_log2 * tanhf(x[e] * pl.sc.in) : x[e] * pl.sc.mul;
                    x[e] = fmaf(slope[e], static_cast<float>(j - (slope[e] < 0.f ? seen.first() : L - 1)), x[e]);
                }
            }
            float mx[2] = {x[0], x[1]};
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
#pragma unroll
                for (int e = 0; e < 2; ++e) mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], o));
            float w[2], sum[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float mn = fmaxf(m[e], mx[e]), mu = mn == -INFINITY ? 0.f : mn, f = exp2f(m[e] - mu);
                w[e] = lane < n ? exp2f(x[e] - mu) : 0.f;
                sum[e] = w[e];
                l[e] *= f;
                m[e] = mn;
                ps[2 * warp + e][lane] = w[e];
                if (lane == 0) factor[2 * warp + e] = f;
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
#pragma unroll
                for (int e = 0; e < 2; ++e) sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], o);
            l[0] += sum[0];
            l[1] += sum[1];
        }
        __syncthreads();
#pragma unroll
        for (int a = 0; a < 2; ++a) {
            const int x = tid + a * kGenThreads, hp = x / quads, c = x - hp * quads;  // a pair of heads, four dimensions
            if (2 * hp >= nh) continue;
            const float f0 = factor[2 * hp], f1 = factor[2 * hp + 1];
            float4 o0 = acc[a][0], o1 = acc[a][1];
            o0 = make_float4(o0.x * f0, o0.y * f0, o0.z * f0, o0.w * f0);
            o1 = make_float4(o1.x * f1, o1.y * f1, o1.z * f1, o1.w * f1);
            const float* v = vs + 4 * c;
            auto take = [&](int p, float w0, float w1) {
                const float4 z = *reinterpret_cast<const float4*>(v + p * DS);
                o0 = make_float4(fmaf(w0, z.x, o0.x), fmaf(w0, z.y, o0.y), fmaf(w0, z.z, o0.z), fmaf(w0, z.w, o0.w));
                o1 = make_float4(fmaf(w1, z.x, o1.x), fmaf(w1, z.y, o1.y), fmaf(w1, z.z, o1.z), fmaf(w1, z.w, o1.w));
            };
            int p = 0;
            for (; p + 4 <= n; p += 4) {
                const float4 w0 = *reinterpret_cast<const float4*>(&ps[2 * hp][p]), w1 = *reinterpret_cast<const float4*>(&ps[2 * hp + 1][p]);
                take(p, w0.x, w1.x);
                take(p + 1, w0.y, w1.y);
                take(p + 2, w0.z, w1.z);
                take(p + 3, w0.w, w1.w);
            }
            for (; p < n; ++p) take(p, ps[2 * hp][p], ps[2 * hp + 1][p]);
            acc[a][0] = o0;
            acc[a][1] = o1;
        }
        bad = __syncthreads_or(miss) != 0;  // of tile t + 2; this one's rows, weights and factors are used
    }
    if constexpr (kAhead) asm volatile("cp.async.wait_all;" ::: "memory");
    if (bad && tid == 0) report(status, PKV_ERR_DEVICE_BOUNDS);
    if (lane == 0) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            ends[2 * warp + e][0] = m[e];
            ends[2 * warp + e][1] = bad ? -1.f : l[e];  // a share that cannot be read makes the row zero
        }
    }
    __syncthreads();
    // a share's row: maximum, sum, D sums of products
    const int DR = 2 + 4 * quads;
#pragma unroll
    for (int a = 0; a < 2; ++a) {
        const int x = tid + a * kGenThreads, hp = x / quads, c = x - hp * quads;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int hd = 2 * hp + e;
            if (hd >= nh) continue;
            const float o[4] = {acc[a][e].x, acc[a][e].y, acc[a][e].z, acc[a][e].w};
            const float sum = ends[hd][1];
            if (pl.shares == 1) {
                const bool some = sum > 0.f || sum != sum;
                const float inv = 1.f / sum;
                for (int i = 0; i < 4; ++i)
                    if (4 * c + i < D) out[(row0 + hd) * D + 4 * c + i] = from_f32<T>(some ? o[i] * inv : 0.f);
            } else {
                float* to = part + ((row0 + hd) * pl.shares + share) * DR;
                if (c == 0) *reinterpret_cast<float2*>(to) = make_float2(ends[hd][0], sum);
                for (int i = 0; i < 2; ++i) *reinterpret_cast<float2*>(to + 2 + 4 * c + 2 * i) = make_float2(o[2 * i], o[2 * i + 1]);
            }
        }
    }
}

// out = sum o_s 2^(m_s - M) / sum l_s 2^(m_s - M) over a row's shares (at most 64); a warp a row.
template <typename T>
__global__ void __launch_bounds__(128)
    decode_scored_shares_kernel(T* out, const float* part, long long nrows, int shares, int D) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const long long row = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (row >= nrows) return;
    const int DR = 2 + (D + 3) / 4 * 4;
    const float* p = part + row * shares * DR;
    float2 ml[2];
#pragma unroll
    for (int k = 0; k < 2; ++k)
        ml[k] = lane + 32 * k < shares ? __ldcg(reinterpret_cast<const float2*>(p + (lane + 32 * k) * DR)) : make_float2(-INFINITY, 0.f);
    float M = fmaxf(ml[0].x, ml[1].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    const float mu = M == -INFINITY ? 0.f : M, f0 = exp2f(ml[0].x - mu), f1 = exp2f(ml[1].x - mu);
    const bool bad = __any_sync(0xffffffffu, ml[0].y < 0.f || ml[1].y < 0.f);
    float l = ml[0].y * f0 + ml[1].y * f1, acc[8] = {};
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
#pragma unroll 4
    for (int s = 0; s < shares; ++s) {
        const float w = __shfl_sync(0xffffffffu, s < 32 ? f0 : f1, s & 31);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (lane + 32 * i < D) acc[i] = fmaf(__ldcg(p + s * DR + 2 + lane + 32 * i), w, acc[i]);
    }
    const float inv = 1.f / l;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (lane + 32 * i < D) out[row * D + lane + 32 * i] = from_f32<T>(bad || l == 0.f ? 0.f : acc[i] * inv);
}

static size_t generic_smem(int D, bool ahead) {
    return ((ahead ? 4 : 2) * kGenPos + kGenHeads) * static_cast<size_t>(generic_stride(D)) * sizeof(float);
}
// CTAs along the positions: as many as an SM holds at once (37 sequences of up to 1500 in float32: 17.5 us, twice as many
// 22.0); where that leaves shares of more than 12 tiles, up to four times as many, which evens out lengths (16 sequences
// of 512-4096, 8 x 128 in float32: 140 for 170 us); and not more than the longest sequence (by the table's width, or the
// window) has tiles.
static int generic_shares(long long units, int D, bool ahead, int longest, int P) {
    const long long held = std::min<long long>(12, 225 * 1024 / (generic_smem(D, ahead) + 3 * 1024));
    const long long tiles = (static_cast<long long>(longest) + kGenPos - 1) / kGenPos;
    const long long once = held * P / units, more = std::min(4 * held * P / units, tiles / 12);
    return static_cast<int>(std::max(1LL, std::min({std::max(once, more), tiles, static_cast<long long>(kGenShares)})));
}

static size_t generic_workspace(int B, int Hq, int Hkv, int D, int P) {
    const long long units = static_cast<long long>(B) * Hkv * ((Hq / Hkv + kGenHeads - 1) / kGenHeads);
    const int shares = generic_shares(std::max(1LL, units), D, false, 0x7fffffff, P);  // (ahead holds fewer)
    return shares == 1 ? 0 : static_cast<size_t>(B) * Hq * shares * (2 + (D + 3) / 4 * 4) * sizeof(float);
}

template <typename T>
static cudaError_t launch_generic(GenericPlan pl, void* out, const void* q, const void* k, const void* v,
                                  const int32_t* block_tables, const int32_t* seq_lens, void* workspace, int P,
                                  int32_t* status, cudaStream_t stream) {
    auto aligned16 = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
    const bool vec = pl.D * sizeof(T) % 16 == 0 && aligned16(k) && aligned16(v);
    pl.chunks = (pl.G + kGenHeads - 1) / kGenHeads;
    pl.stride = generic_stride(pl.D);
    const long long units = static_cast<long long>(pl.B) * pl.Hkv * pl.chunks;
    const long long width = std::min(static_cast<long long>(pl.max_blocks) * pl.BS, 0x7fffffffLL);
    const bool windowed = pl.sc.window > 0 && pl.sc.prefix_lens == nullptr;
    const bool ahead = sizeof(T) == 4 && vec;
    pl.shares = generic_shares(units, pl.D, ahead, static_cast<int>(windowed ? std::min<long long>(width, pl.sc.window) : width), P);
    const size_t smem = generic_smem(pl.D, ahead);
    auto kern = vec ? decode_scored_generic_kernel<T, true> : decode_scored_generic_kernel<T, false>;
    // the limit belongs to the kernel, not to the call: always the same value
    constexpr int kMost = (4 * kGenPos + kGenHeads) * (256 + 4) * 4;
    cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(units * pl.shares), 1, 1);
    cfg.blockDim = dim3(kGenThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    float* part = static_cast<float*>(workspace);
    err = cudaLaunchKernelEx(&cfg, kern, pl, static_cast<T*>(out), static_cast<const T*>(q), static_cast<const T*>(k),
                             static_cast<const T*>(v), block_tables, seq_lens, part, status);
    if (err != cudaSuccess || pl.shares == 1) return err != cudaSuccess ? err : cudaGetLastError();
    const long long nrows = static_cast<long long>(pl.B) * pl.Hq;
    cfg.gridDim = dim3(static_cast<unsigned>((nrows + 3) / 4), 1, 1);
    cfg.blockDim = dim3(128, 1, 1);
    cfg.dynamicSmemBytes = 0;
    err = cudaLaunchKernelEx(&cfg, decode_scored_shares_kernel<T>, static_cast<T*>(out), static_cast<const float*>(part),
                             nrows, pl.shares, pl.D);
    return err != cudaSuccess ? err : cudaGetLastError();
}

// ------------------------------------------------------------------ host side
// Steps of a sequence up to which a join is not worth it.
constexpr int kDirectSteps = 3;  // 1 sequence of 100-300, 8 and 2 heads of 64: 6.8 us, with the join 9.4

// Group size and slots for a shape, with at least min_groups head groups where the heads allow it; false where the
// fast kernel does not apply.
bool split_shape(int Hq, int Hkv, int D, int BS, int min_groups, SplitPlan& pl) {
    if (D % 8 != 0 || D > 128 || BS % kUnit != 0) return false;
    const int G = Hq / Hkv, rows = G <= 8 ? 8 : 16;  // query heads per warp
    pl.QC = (G + rows - 1) / rows;
    if (pl.QC > kSplitWarps) return false;
    // as few groups as the warps allow, of equal size (the last one up to NG - 1 heads smaller: 11 heads are 6 + 5;
    // the tile of the missing head is read and not used)
    const int most = kSplitWarps / pl.QC;
    pl.NG = std::max((Hkv + most - 1) / most, std::min(min_groups, Hkv));
    pl.HG = (Hkv + pl.NG - 1) / pl.NG;
    pl.NG = (Hkv + pl.HG - 1) / pl.HG;
    pl.UB = BS / kUnit;
    pl.slots = 1;
    while (pl.slots * 2 * pl.HG * pl.QC <= kSplitWarps) pl.slots *= 2;
    pl.units = pl.slots * split_sub(D <= 64 ? 64 : 128);
    pl.G = G;
    pl.R = pl.HG * G;
    return true;
}

static size_t up256(size_t x) { return (x + 255) / 256 * 256; }

// [head][cuts][info of B sequences][(max, sum)][sums of products]; two partial results per CTA of R rows and, for
// shared prefixes, one per row of out.
size_t split_space(const SplitPlan& pl, int P, int B, bool shared, void* base, SplitSpace* ws) {
    const size_t slots = static_cast<size_t>(2) * P * pl.R + (shared ? static_cast<size_t>(B) * pl.Hq : 0);
    const size_t cuts = 256, info = up256(cuts + sizeof(SplitCut) * P);
    const size_t ml = up256(info + (shared ? sizeof(int2) * static_cast<size_t>(B) : 0));
    const size_t o = up256(ml + slots * sizeof(float2));
    if (ws != nullptr) {
        uint8_t* p = static_cast<uint8_t*>(base);
        ws->head = reinterpret_cast<SplitHead*>(p);
        ws->cuts = reinterpret_cast<SplitCut*>(p + cuts);
        ws->info = reinterpret_cast<int2*>(p + info);
        ws->ml = reinterpret_cast<float2*>(p + ml);
        ws->o = reinterpret_cast<float*>(p + o);
    }
    return up256(o + slots * pl.D * sizeof(float));
}

// A pool [NB * Hkv][BS][D] in boxes of 64 dimensions x 16 positions x HG heads; dimensions from D on read as zeros.
static bool split_map(CUtensorMap* map, const void* pool, const SplitPlan& pl) {
    EncodeTiledFn enc = get_encode_fn();
    if (!enc) return false;
    cuuint64_t dim[3] = {static_cast<cuuint64_t>(pl.D), static_cast<cuuint64_t>(pl.BS),
                         static_cast<cuuint64_t>(pl.NB) * pl.Hkv};
    cuuint64_t stride[2] = {static_cast<cuuint64_t>(pl.D) * 2, static_cast<cuuint64_t>(pl.D) * pl.BS * 2};
    cuuint32_t box[3] = {64, kUnit, static_cast<cuuint32_t>(pl.HG)};
    cuuint32_t one[3] = {1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(pool), dim, stride, box, one,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The fast kernel's shared memory; false where two stages do not fit.
static bool split_layout(SplitPlan& pl, int DP, int kN, size_t budget, size_t* smem) {
    pl.stage_bytes = 2 * pl.units * (DP / 64) * pl.HG * 2048;
    pl.q_bytes = pl.R * 2 * DP;
    pl.scratch_bytes = (pl.slots - 1) * pl.HG * pl.QC * (8 * kN * (DP + 6)) * 4;
    const size_t fixed = 1024 + pl.scratch_bytes + (2 * kSplitStages + 4 + 2 * kSplitWarps) * sizeof(uint64_t) +
                         kSplitStages * sizeof(SplitMeta) + 40 * sizeof(int) + 16;
    auto stages = [&](int qslots) {
        const size_t all = fixed + static_cast<size_t>(qslots) * pl.q_bytes;
        return all >= budget ? 0 : static_cast<int>(std::min<size_t>(kSplitStages, (budget - all) / pl.stage_bytes));
    };
    // two sequences' queries where that costs no stage
    pl.qslots = stages(2) == stages(1) ? 2 : 1;
    pl.nst = stages(pl.qslots);
    *smem = fixed + static_cast<size_t>(pl.qslots) * pl.q_bytes + static_cast<size_t>(pl.nst) * pl.stage_bytes;
    return pl.nst >= 2;
}

template <int DP, int kN, bool kShared>
static cudaError_t launch_split_kernel(SplitPlan pl, const SplitSpace& ws, void* out, const void* q, const void* k,
                                       const void* v, const int32_t* block_tables, const int32_t* seq_lens, int P,
                                       int32_t* status, cudaStream_t stream, bool* done) {
    *done = false;
    size_t smem;
    const size_t budget = static_cast<size_t>(max_optin_smem());
    CUtensorMap tmK, tmV;
    if (!split_layout(pl, DP, kN, budget, &smem) || !split_map(&tmK, k, pl) || !split_map(&tmV, v, pl)) return cudaSuccess;
    auto kern = decode_split_kernel<DP, kN, kShared>;
    // The limit belongs to the kernel, not to the call: always the device's largest, so that another thread's call
    // with other sizes cannot lower it between here and the launch.
    cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(budget));
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(pl.direct ? pl.B * pl.NG : P), 1, 1);
    cfg.blockDim = dim3(static_cast<unsigned>((pl.HG * pl.QC * pl.slots + 1) * 32), 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    err = cudaLaunchKernelEx(&cfg, kern, tmK, tmV, pl, static_cast<const __nv_bfloat16*>(q),
                             static_cast<__nv_bfloat16*>(out), block_tables, seq_lens, ws, status);
    if (err != cudaSuccess) return err;
    *done = true;
    if (kShared || pl.direct || P == 1) return cudaGetLastError();
    cfg.gridDim = dim3(static_cast<unsigned>((P - 1) * ((pl.R + kJoinWarps - 1) / kJoinWarps)), 1, 1);
    cfg.blockDim = dim3(kJoinWarps * 32, 1, 1);
    cfg.dynamicSmemBytes = 0;
    err = cudaLaunchKernelEx(&cfg, decode_split_join_kernel, pl, ws, static_cast<__nv_bfloat16*>(out));
    return err != cudaSuccess ? err : cudaGetLastError();
}

template <bool kShared>
static cudaError_t launch_split_any(const SplitPlan& pl, const SplitSpace& ws, void* out, const void* q, const void* k,
                                    const void* v, const int32_t* block_tables, const int32_t* seq_lens, int P,
                                    int32_t* status, cudaStream_t stream, bool* done) {
    auto kern = pl.D <= 64 ? (pl.G <= 8 ? launch_split_kernel<64, 1, kShared> : launch_split_kernel<64, 2, kShared>)
                           : (pl.G <= 8 ? launch_split_kernel<128, 1, kShared> : launch_split_kernel<128, 2, kShared>);
    return kern(pl, ws, out, q, k, v, block_tables, seq_lens, P, status, stream, done);
}

// The positions behind the shared prefixes (decode_attention_shared.cu).
cudaError_t launch_split_shared(const SplitPlan& pl, const SplitSpace& ws, const void* q, const void* k, const void* v,
                                const int32_t* block_tables, const int32_t* seq_lens, int P, int32_t* status,
                                cudaStream_t stream, bool* done) {
    return launch_split_any<true>(pl, ws, nullptr, q, k, v, block_tables, seq_lens, P, status, stream, done);
}

// Whether the fast kernel takes a call; fills in the plan.
bool split_applies(SplitPlan& pl, const void* out, const void* q, const void* k, const void* v, pkv_dtype dtype) {
    auto aligned16 = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
    if (dtype != PKV_BF16 || !aligned16(q) || !aligned16(out) || !aligned16(k) || !aligned16(v) ||
        !split_shape(pl.Hq, pl.Hkv, pl.D, pl.BS, 1, pl))
        return false;
    // step and row counts stay in 32 bits
    const long long steps = (static_cast<long long>(pl.max_blocks) * pl.BS) / (kUnit * pl.slots) + 1;
    pl.polls = attention_wait_polls();
    pl.silent_cta = attention_silent_cta();
    return steps * pl.B * pl.NG < (1LL << 30) && static_cast<long long>(pl.NB) * pl.Hkv < (1LL << 31);
}

size_t decode_scored_workspace_bytes(int B, int Hq, int Hkv, int D, int P) {
    SplitPlan pl = {};
    pl.Hq = Hq;
    pl.D = D;
    const size_t fast = split_shape(Hq, Hkv, D, kUnit, 1, pl) ? split_space(pl, P, B, false, nullptr, nullptr) : 0;
    return std::max({static_cast<size_t>(256), fast, generic_workspace(B, Hq, Hkv, D, P)});
}

// Arguments checked; B > 0.
cudaError_t launch_decode_scored(void* out, const void* q, const void* k, const void* v, const int32_t* block_tables,
                                 int max_blocks, const int32_t* seq_lens, int B, int Hq, int Hkv, int D, int BS, int NB,
                                 const ScoreArgs& sc, const GroupArgs& groups, pkv_dtype dtype, void* workspace, int P,
                                 int32_t* status, cudaStream_t stream) {
    SplitPlan pl = {};
    pl.groups = groups;
    pl.B = B;
    pl.Hq = Hq;
    pl.Hkv = Hkv;
    pl.G = Hq / Hkv;
    pl.D = D;
    pl.BS = BS;
    pl.NB = NB;
    pl.max_blocks = max_blocks;
    pl.sc = sc;
    if (split_applies(pl, out, q, k, v, dtype)) {
        SplitSpace ws = {};
        bool done = false;
        // Few and short sequences (by the table's width, or the window): a CTA for each (sequence, head group) and
        // no join, with as many groups as there are SMs for.
        long long longest = static_cast<long long>(max_blocks) * BS;
        if (sc.window > 0 && sc.prefix_lens == nullptr) longest = std::min(longest, sc.window + kUnit - 1LL);
        SplitPlan one = pl;
        if (B <= P && split_shape(Hq, Hkv, D, BS, P / B, one) && B * one.NG <= P &&
            longest <= static_cast<long long>(kDirectSteps) * one.units * kUnit) {
            one.direct = 1;
            const cudaError_t err = launch_split_any<false>(one, ws, out, q, k, v, block_tables, seq_lens, P, status, stream, &done);
            if (err != cudaSuccess || done) return err;
        }
        split_space(pl, P, B, false, workspace, &ws);
        const cudaError_t err = launch_split_any<false>(pl, ws, out, q, k, v, block_tables, seq_lens, P, status, stream, &done);
        if (err != cudaSuccess || done) return err;
    }
    GenericPlan gp = {};
    gp.B = B;
    gp.Hq = Hq;
    gp.Hkv = Hkv;
    gp.G = Hq / Hkv;
    gp.D = D;
    gp.BS = BS;
    gp.NB = NB;
    gp.max_blocks = max_blocks;
    gp.sc = sc;
    return (dtype == PKV_F32 ? launch_generic<float> : launch_generic<__nv_bfloat16>)(
        gp, out, q, k, v, block_tables, seq_lens, workspace, P, status, stream);
}

// False where a shape is none that the calls with changed scores take.
bool scored_shape_valid(int B, int Hq, int Hkv, int D, int BS, int NB, int max_blocks, pkv_dtype dtype) {
    return B >= 0 && Hq >= 1 && Hkv >= 1 && Hq % Hkv == 0 && D >= 1 && D <= 256 && BS >= 1 && NB >= 1 &&
           max_blocks >= 1 && (dtype == PKV_F32 || dtype == PKV_BF16) &&
           static_cast<long long>(B) * Hq <= 0x7fffffffLL;
}

}  // namespace pkv

extern "C" size_t pkv_decode_scored_workspace_bytes(int B, int Hq, int Hkv, int D, int num_sms) {
    using namespace pkv;
    if (!scored_shape_valid(B, Hq, Hkv, D, 1, 1, 1, PKV_BF16)) return 0;
    const int P = num_sms > 0 ? num_sms : device_sm_count();
    return P > 0 ? decode_scored_workspace_bytes(B, Hq, Hkv, D, P) : 0;
}

extern "C" pkv_status pkv_paged_decode_attention_scored(
    void* out, const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
    int max_blocks_per_seq, const int32_t* seq_lens, const int32_t* prefix_lens, int B, int Hq, int Hkv, int D,
    int block_size, int num_blocks, float scale, float softcap, const float* slopes, int window, pkv_dtype dtype,
    void* workspace, size_t workspace_bytes, int32_t* dev_status, void* stream) {
    using namespace pkv;
    ScoreArgs sc;
    if (!scored_shape_valid(B, Hq, Hkv, D, block_size, num_blocks, max_blocks_per_seq, dtype) ||
        !make_scores(&sc, scale, D, softcap, slopes, window, prefix_lens))
        return PKV_ERR_INVALID_ARG;
    if (B == 0) return PKV_OK;
    if (!positions_fit(max_blocks_per_seq, block_size)) return PKV_ERR_UNSUPPORTED;
    if (!out || !q || !k_cache || !v_cache || !block_tables || !seq_lens || !workspace ||
        (reinterpret_cast<uintptr_t>(workspace) & 15u) != 0)
        return PKV_ERR_INVALID_ARG;
    if (overlap(out, q, static_cast<size_t>(B) * Hq * D * (dtype == PKV_F32 ? 4 : 2))) return PKV_ERR_INVALID_ARG;
    const int P = device_sm_count();
    if (workspace_bytes < pkv_decode_scored_workspace_bytes(B, Hq, Hkv, D, P > 0 ? P : 1)) return PKV_ERR_INVALID_ARG;
    if (P <= 0) return PKV_ERR_CUDA;
    const cudaError_t err =
        launch_decode_scored(out, q, k_cache, v_cache, block_tables, max_blocks_per_seq, seq_lens, B, Hq, Hkv, D,
                             block_size, num_blocks, sc, GroupArgs{}, dtype, workspace, P, dev_status,
                             static_cast<cudaStream_t>(stream));
    return err == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}
