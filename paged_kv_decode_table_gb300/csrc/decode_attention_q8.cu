// decode_attention_q8.cu -- GQA paged decode attention over the 8-bit KV cache.
//
// For query head qh of sequence b, KV head h = qh / G, L = seq_lens[b]:
//   s_j = scale * ks_j * <q, kv_j>,   out = sum_j softmax(s)_j * vs_j * vv_j
// with kv_j, vv_j the 8-bit numbers of position j's rows and ks_j, vs_j their
// float32 scales (quant8.cuh): a K scale multiplies a score, a V scale a
// softmax weight.
//
// Fast path (D a multiple of 16 up to 128, block size a multiple of 16): a
// persistent kernel, one CTA per SM, over balanced ranges, and a kernel that
// joins the sequences that several ranges share.
//  * A tile is 16 positions of one KV head.  A step is slots x kSub tiles of
//    consecutive positions of `HG` KV heads (at most 8 x kSub tiles), fetched by TMA
//    boxes of 16 positions x HG heads into one stage of an mbarrier ring.  The steps of
//    all (sequence, head group) pairs, one after the other, are cut into one range per
//    CTA; every CTA finds its range itself from seq_lens.
//  * One consumer warp per (KV head, chunk of its query heads, slot) takes kSub
//    tiles of every step: with 8 KV heads the 8 warps are the heads, with one head
//    they are 8 slots along the cache, so a model split over devices keeps every
//    warp busy.  The slots' results are merged in shared memory when the range
//    leaves the sequence.
//  * The 8-bit numbers become float16 in registers (exact for both types) and
//    both products run transposed on mma.sync m16n8k16 with float32 accumulation:
//    S^T = K Q^T (16 positions x 8 query heads) and O^T = V^T P^T (16 dimensions x 8
//    query heads), so the cached tile is the 16-row operand and no MMA row is idle
//    with 8 query heads.  K's order of dimensions inside a 16-byte chunk is permuted
//    the same way in q, so a 4-byte fragment of K is one register; V is read
//    transposed in 16-bit units, which yields even and odd dimensions of two
//    positions, and rows g and g + 8 of the MMA are dimensions 2g and 2g + 1.
//    movmatrix turns the weights from S^T's layout into P^T's.
//  * bf16 queries are exact in float16 and the weights are rounded to it (2^-11 of a
//    weight, at least 2^-34 of the largest);
//    float32 queries carry what that rounding leaves of q and of the weights in a
//    second float16, the weights' 2^11 times as large, and a second MMA (kSplit: 2^-22
//    and 2^-45), and sum each step apart before adding it.  The 2-norm of the error is
//    below 6e-7 of the result for random float32 queries over 500 to 60000 positions;
//    with one weight 2^25 times as large as each of 32767 behind it, all in one warp,
//    1.1e-5, the roundings of the float32 running sums.
//  * Weights are normalised by a running maximum of s_j + log2(vs_j), the largest
//    contribution rather than the largest score, so that p_j * vs_j fits float16
//    whatever the V scales are.  Scales below 2^-64 count as 2^-64 there, which
//    bounds p_j by 2^77.  The maximum is renewed (shuffles, rescaled sums) only
//    when a contribution exceeds it by 2^kLag: a vote decides.
//  * q is multiplied by a power of two per head that puts its largest element into
//    [2^14, 2^15).
// Other shapes: one CTA per (sequence, query head), CUDA-core fp32.
// No input is read through the read-only path (__ldg, const __restrict__): these kernels start
// while their predecessor still writes what they read after griddepcontrol.wait, and the
// join while the main kernel writes its partial results.
//
// What bounds it: HBM where the cache is large.  8 sequences of 32768-131072 positions, 64
// query and 8 KV heads of 128 in int8: 234 us for 1.53 GB, 6.5 TB/s, 98% of the measured
// copy rate.  64 sequences of 512-4096, 32 and 8 heads: 58 us for 332 MB, 86%; the rest is
// the start (2.5 us), the end of the slowest SM (2.3 us) and the join (3.5 us).  With the
// arithmetic left out the same kernel takes 57 us, so the tensor and issue pipes (17% and
// 32% busy) hide behind the copies.  They do not with 16 query heads a group (128 and 8
// heads: 85 us, 59%) and with float32 queries (64 us, 78%; two MMAs for one).  One short
// sequence is a chain of latencies, lengths -> block ids -> K and V -> result: 6.4 us.
// mma.sync and not tcgen05: a float16 query needs float16 keys, so the converted numbers, twice
// the bytes that came, would go back to shared memory before tcgen05.mma could read them,
// and the tensor pipe is not what the kernel waits for.
#include <cuda.h>
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "quant8.cuh"

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
constexpr int kQ8MaxStages = 12;
constexpr int kQ8Tok = 16;  // positions per tile
constexpr int kQ8Warps = 8;  // consumer warps at most
// Steps of a sequence up to which a join is not worth it.  Direct against split: 1 sequence of
// up to 256 positions, 32 and 8 heads 6.4 : 8.5 us, 16 of up to 512 8.5 : 11.2 us; at 1024 (4
// steps) 9.1 : 8.8 us for one, 10.8 : 9.0 for four, 12.2 : 12.6 for 16.
constexpr int kDirectSteps = 3;
// Contributions stay below 2^kLag of the running maximum, and weights are 2^kShift times as
// large as relative to it, so that the float16 ones, at most 2^13, reach down to 2^-34 of the
// largest.  (The 2^3 up to float16's limit are for scores so large that their own rounding is
// a factor.)
constexpr float kLag = 4.f, kShift = 9.f;
constexpr float kLowUp = 2048.f;  // what the second float16 of a weight is scaled by

// How a call is laid out; computed on the host, passed to both kernels.
struct Q8Plan {
    int HG, NG;      // KV heads per group, groups (the last one may have fewer heads)
    int QC;          // chunks of query heads per KV head (8 or 16 heads each)
    int slots, sub;  // a step is slots x sub tiles along the cache, sub of them a warp's
    int R;           // query rows per group: HG * G
    int UB;          // units of 16 positions per block
    int nst;         // ring stages
    int stage_bytes, scale_unit, q_bytes, scratch_bytes;
    int q_stride;    // bytes between q's rows in shared memory
    int direct;      // one CTA per (sequence, group), no join
    int layout;      // of a tile in shared memory: kSwizzled, kPacked or kDense
    int tok_shift;   // log2 of the positions per row of the tensor map
    int B, Hq, Hkv, G, D, BS, NB, max_blocks;
    float scale_log2;
    uint32_t polls;
    int silent_cta;
};

// D = 128: rows of 128 bytes, one per position, 128-byte swizzle.  D = 64: two positions
// per such row.  Other D: rows of D bytes one behind the other (copied as one run per
// head, because the TMA takes as long for a row of 80 bytes as for two of 128); ldmatrix
// reads them without bank conflicts where D / 16 is odd, with two-way ones at 32 and 96.
enum : int { kSwizzled, kPacked, kDense };

struct Q8Meta {
    int vb;     // sequence * NG + group
    int left;   // positions from the step's first one to the end
    int flags;
    int pad;
};
enum : int { kQFirst = 1, kQLast = 2, kQWhole = 4, kQHead = 8, kQBad = 16 };

__device__ __forceinline__ float ex2f(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// With subnormal results: a weight p_j is about 1 / vs_j, and with V scales near 2^119 (rows
// near the largest float) weights of 2^-7 of the largest would be flushed to zero.
__device__ __forceinline__ float ex2f_subnormal(float x) {
    float y;
    asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// 2^d, d <= 0, as the square of 2^(d / 2): what sums are multiplied by when the maximum they are relative to
// changes.  A sum of weights is up to 2^77 a position where V scales are 2^-64 (rows of zeros),
// and the maximum may rise by 2^185 where rows near the largest float follow, so that
// 2^d alone would be flushed to zero while the product with the sum is not negligible.
struct Shrink {
    float half;  // 2^(d / 2)
    __device__ __forceinline__ explicit Shrink(float d) : half(ex2f(0.5f * d)) {}
    __device__ __forceinline__ float of(float sum) const { return sum * half * half; }
    __device__ __forceinline__ float both() const { return half * half; }
};
__device__ __forceinline__ float lg2f(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void mma_f16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 8x8 halves: row g, columns 2r, 2r + 1 -> row 2r (and 2r + 1) as column g
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

__device__ __forceinline__ float4 load_row4(const __nv_bfloat16* p) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    return make_float4(bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y));
}
__device__ __forceinline__ float4 load_row4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ void store_row2(__nv_bfloat16* p, float x, float y) {
    *reinterpret_cast<uint32_t*>(p) = pack_bf16x2(x, y);
}
__device__ __forceinline__ void store_row2(float* p, float x, float y) {
    *reinterpret_cast<float2*>(p) = make_float2(x, y);
}
__device__ __forceinline__ void store_row4(__nv_bfloat16* p, float4 v) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
}
__device__ __forceinline__ void store_row4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }

__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
// One arrival on the barrier once this thread's earlier cp.async copies have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// Steps of sequence b in one head group (0 for a length outside [0, max_blocks * BS]).
__device__ __forceinline__ int q8_steps(const int32_t* seq_lens, int b, const Q8Plan& pl) {
    const int L = seq_lens[b], T = pl.slots * pl.sub * kQ8Tok;
    return (L >= 0 && static_cast<long long>(L) <= static_cast<long long>(pl.max_blocks) * pl.BS)
               ? static_cast<int>((static_cast<long long>(L) + T - 1) / T)
               : 0;
}

// Sum over the CTA and this thread's exclusive prefix; red holds 33 ints.
__device__ __forceinline__ int q8_scan(int v, int* red, int& total) {
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

// Byte offset of 16-byte chunk c of position `tok` in a tile.
__device__ __forceinline__ uint32_t q8_at(int tok, int c, const Q8Plan& pl) {
    if (pl.layout == kDense) return static_cast<uint32_t>(tok * pl.D + c * 16);
    if (pl.layout == kPacked) {
        c += (tok & 1) * 4;
        tok >>= 1;
    }
    return static_cast<uint32_t>(tok * 128 + ((c ^ (tok & 7)) << 4));
}

// Floats of a warp's place for accumulators set aside: its heads' sums and maxima.
__host__ __device__ constexpr int q8_aside_floats(int DP, int kN) { return 8 * kN * DP + 64 * kN; }

// DP: dimensions computed (32, 64, 96 or 128; D may be smaller).  96 of 128 for D = 80 took 37
// float32 sequences of up to 1500 from 15.6 to 14.3 us, 32 of 64 for D = 32 169 sequences of
// 1733-3682 with 10 query heads a group from 107 to 86 us.  kN: n-tiles of 8 query heads per
// warp; kSplit: float32 accuracy (see above); kSub: tiles a warp takes of a step.
template <typename T, typename Fmt, int DP, int kN, bool kSplit, int kSub>
__global__ void __launch_bounds__((kQ8Warps + 1) * 32, 1)
    decode_q8_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                     const __grid_constant__ Q8Plan pl, const T* q, T* out, const float* k_scale,
                     const float* v_scale, const int32_t* block_tables, const int32_t* seq_lens, float* part_ml,
                     float* part_o, float* aside, int32_t* status) {
    constexpr int kChunks = DP / 16;
    // the last chunk may lie behind D: a K byte there is the next row's, and an e4m3 NaN
    // survives the product with q's zero
    constexpr int kMaybe = !Fmt::kHasNaN ? kChunks : kChunks - 1;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int nst = pl.nst, HG = pl.HG, QC = pl.QC, slots = pl.slots;
    const int HV = HG * QC, CW = HV * slots;
    const int units = slots * kSub;  // 16-position units per step
    const int tile_bytes = kQ8Tok * pl.D, unit_bytes = HG * tile_bytes, half_stage = units * unit_bytes;
    const int scale_half = units * pl.scale_unit;
    uint8_t* scales = smem + static_cast<size_t>(nst) * pl.stage_bytes;
    uint8_t* qring = scales + static_cast<size_t>(nst) * 2 * scale_half;
    float* scratch = reinterpret_cast<float*>(qring + 2 * static_cast<size_t>(pl.q_bytes));
    uint64_t* full = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(scratch) + pl.scratch_bytes);
    uint64_t* empty = full + kQ8MaxStages;
    uint64_t* qfull = empty + kQ8MaxStages;
    uint64_t* qempty = qfull + 2;
    uint64_t* mfull = qempty + 2;   // merge slots: one per consumer warp
    uint64_t* mempty = mfull + kQ8Warps;
    Q8Meta* meta = reinterpret_cast<Q8Meta*>(mempty + kQ8Warps);
    int* sch = reinterpret_cast<int*>(meta + kQ8MaxStages);  // [0, 33) scan scratch, 33: b0, 34: s0

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // lengths, then block ids, then K and V: three dependent loads, from HBM where the
    // caches of the last step have pushed them out of L2; the first two and q come to L2
    // while the predecessor ends
    const unsigned worker = blockIdx.x * blockDim.x + threadIdx.x;
    prefetch_l2(seq_lens, static_cast<size_t>(pl.B) * 4, worker);
    prefetch_l2(block_tables, static_cast<size_t>(pl.B) * pl.max_blocks * 4, worker);
    prefetch_l2(q, static_cast<size_t>(pl.B) * pl.Hq * pl.D * sizeof(T), worker);
    if (threadIdx.x == 0) {
        for (int s = 0; s < nst; ++s) {
            mbar_init(&full[s], 1 + 32);  // the TMA bytes, and each producer lane's scale copies
            mbar_init(&empty[s], CW);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&qfull[s], 32);  // each producer lane's copies
            mbar_init(&qempty[s], CW);
        }
        for (int s = 0; s < kQ8Warps; ++s) {
            mbar_init(&mfull[s], 1);
            mbar_init(&mempty[s], 1);
        }
        fence_mbar_init();
        prefetch_tmap(&tmK);
        prefetch_tmap(&tmV);
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // Only after the wait: the joining kernel reads seq_lens before its own wait.
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // ---- this CTA's range of steps: [start, end), which begins in sequence b0, whose
    // first step is s0
    const int nthr = blockDim.x, B = pl.B, NG = pl.NG;
    int W = 1, start, end, b0, s0;
    if (pl.direct) {
        b0 = static_cast<int>(blockIdx.x) / NG;
        start = (static_cast<int>(blockIdx.x) - b0 * NG);
        const int n = q8_steps(seq_lens, b0, pl);
        start *= n;
        end = start + n;
        s0 = 0;
        if (n == 0) {  // empty or invalid: zeros
            const int g = static_cast<int>(blockIdx.x) - b0 * NG, rows = min(pl.R, pl.Hq - g * pl.R);
            T* o = out + (static_cast<size_t>(b0) * pl.Hq + g * pl.R) * pl.D;
            for (int e = threadIdx.x; e < rows * pl.D; e += nthr) o[e] = from_f32<T>(0.f);
            if (threadIdx.x == 0 && seq_lens[b0] != 0) report(status, PKV_ERR_DEVICE_BOUNDS);
            return;
        }
        __syncthreads();  // the barriers are initialised
    } else {
        const int n_first = static_cast<int>(threadIdx.x) < B ? NG * q8_steps(seq_lens, threadIdx.x, pl) : 0;
        int tsum = n_first;
        for (int b = threadIdx.x + nthr; b < B; b += nthr) tsum += NG * q8_steps(seq_lens, b, pl);
        int total, before = q8_scan(tsum, sch, total);
        if (total > 0) W = (total + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x);
        start = blockIdx.x * W;
        end = min(total, start + W);
        if (start >= end) return;  // uniform over the CTA
        int carry = 0;
        for (int base = 0; base < B; base += nthr) {
            const int b = base + threadIdx.x;
            int n = n_first, tot = total;
            if (B > nthr) {  // else the scan above was this one
                if (base > 0) n = b < B ? NG * q8_steps(seq_lens, b, pl) : 0;
                before = q8_scan(n, sch, tot);
            }
            const int sb = carry + before;
            if (n > 0 && sb <= start && start < sb + n) {  // exactly one thread of the CTA
                sch[33] = b;
                sch[34] = sb;
            }
            carry += tot;
            if (carry > start) break;  // same decision in every thread
        }
        __syncthreads();
        b0 = sch[33];
        s0 = sch[34];
    }

    if (warp == CW) {
        // ------------------------------------------------ producer warp
        // Lane u fetches the K and V tiles of unit u (slot u % slots) by TMA; the
        // scales, 64 bytes per unit and head, come by 16-byte cp.async of the whole warp
        // (a TMA copy of 64 bytes costs as much issue time as one of 16 KB).  The
        // block ids are read two steps ahead.
        // b, g: the walk's sequence and head group; cn steps per group from cs on.
        int b = b0, cs = s0;
        int cn = q8_steps(seq_lens, b, pl), cL = seq_lens[b], g = 0;
        struct Step {
            int b, g, j, n, cs, L;
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
                    cn = q8_steps(seq_lens, b, pl);
                    cL = seq_lens[b];
                }
            }
            Step s{b, g, i - cs, cn, cs, cL, false, -1, 0};
            const unsigned u = static_cast<unsigned>(s.j) * units + lane;
            if (lane < units && u * kQ8Tok < static_cast<unsigned>(cL)) {
                s.in = true;
                const unsigned lb = pl.UB == 1 ? u : u / static_cast<unsigned>(pl.UB);
                s.tok = static_cast<int>(u - lb * pl.UB) * kQ8Tok;
                s.blk = block_tables[static_cast<size_t>(b) * pl.max_blocks + lb];
            }
            return s;
        };
        if (static_cast<int>(blockIdx.x) == pl.silent_cta) return;  // test hook: no copy is issued
        Step cur = fetch(start), nxt = cur;
        if (start + 1 < end) nxt = fetch(start + 1);
        // this lane's chunks of the scales: (unit, head, quarter) of chunk lane + 32 x
        const int chunks = units * HG * 4;
        constexpr int kScaleChunks = kQ8Warps * kSub * 4 / 32;
        int su[kScaleChunks], srow[kScaleChunks], sq[kScaleChunks];
#pragma unroll
        for (int x = 0; x < kScaleChunks; ++x) {
            const int c = lane + 32 * x;
            su[x] = c < chunks ? c / (HG * 4) : -1;
            srow[x] = (c >> 2) - max(su[x], 0) * HG;
            sq[x] = c & 3;
        }
        const uint32_t unit_tx = 2u * unit_bytes;
        int piece = 0;
        // before every exit: wait for this warp's copies in flight, so that none writes
        // into shared memory after the CTA is gone, whether its consumers still wait for
        // them or have given up (bounded, but not by the limit that a test lowers: copies
        // that were issued land)
        auto drain = [&](int it) {
            asm volatile("cp.async.wait_all;" ::: "memory");
            if (lane != 0) return;
            for (int k = max(0, it - nst); k < it; ++k)
                mbar_wait(&full[k % nst], static_cast<uint32_t>(k / nst) & 1u);
        };
        // 16-byte chunks of a row of q; this lane's first one, and the step to its next one
        const int q_chunks = pl.D * static_cast<int>(sizeof(T)) / 16;
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
            if (first && ok) ok = mbar_wait(&qempty[piece & 1], (static_cast<uint32_t>(piece >> 1) & 1u) ^ 1u, pl.polls);
            if (!__all_sync(0xffffffffu, ok)) {
                if (lane == 0) report(status, PKV_ERR_TIMEOUT);
                drain(it);
                return;
            }
            if (lane == 0) {
                Q8Meta mt;
                mt.vb = s.b * NG + s.g;
                mt.left = s.L - s.j * units * kQ8Tok;
                mt.flags = (first ? kQFirst : 0) | (last ? kQLast : 0) | (s.cs >= start && s.cs + s.n <= end ? kQWhole : 0) |
                           (s.cs < start ? kQHead : 0) | (bad ? kQBad : 0);
                mt.pad = 0;
                meta[stage] = mt;
                mbar_arrive_expect_tx(&full[stage], __popc(live) * unit_tx);  // releases the metadata
            }
            __syncwarp();
            const int row = s.blk * pl.Hkv + s.g * HG;
            if (good) {
                uint8_t* kd = smem + static_cast<size_t>(stage) * pl.stage_bytes + lane * unit_bytes;
                tma_load_3d(kd, &tmK, 0, s.tok >> pl.tok_shift, row, &full[stage]);
                tma_load_3d(kd + half_stage, &tmV, 0, s.tok >> pl.tok_shift, row, &full[stage]);
            }
            if (first) {
                const int qs = piece & 1;
                const int rows = min(pl.R, pl.Hq - s.g * pl.R);  // the last group may have fewer heads
                const uint8_t* src = reinterpret_cast<const uint8_t*>(
                    q + (static_cast<size_t>(s.b) * pl.Hq + static_cast<size_t>(s.g) * pl.R) * pl.D);
                uint8_t* dst = qring + static_cast<size_t>(qs) * pl.q_bytes;
                int row = q_row, col = q_col;
                for (int x = lane; x < rows * q_chunks; x += 32) {
                    cp_async16(dst + row * pl.q_stride + col * 16, src + x * 16);
                    row += q_drow;
                    col += q_dcol;
                    if (col >= q_chunks) {
                        col -= q_chunks;
                        ++row;
                    }
                }
                cp_async_arrive(&qfull[qs]);
                ++piece;
            }
            if (bad && lane == 0) report(status, PKV_ERR_DEVICE_BOUNDS);
            uint8_t* sd = scales + static_cast<size_t>(stage) * 2 * scale_half;
#pragma unroll
            for (int x = 0; x < kScaleChunks; ++x) {
                const int u = max(su[x], 0);
                const int r0 = __shfl_sync(0xffffffffu, row, u), t0 = __shfl_sync(0xffffffffu, s.tok, u);
                // heads behind the last one (a group with fewer) have no scales to read
                if (su[x] >= 0 && ((live >> u) & 1u) && s.g * HG + srow[x] < pl.Hkv) {
                    const size_t at = static_cast<size_t>(r0 + srow[x]) * pl.BS + t0 + 4 * sq[x];
                    uint8_t* d = sd + u * pl.scale_unit + (4 * srow[x] + sq[x]) * 16;
                    cp_async16(d, k_scale + at);
                    cp_async16(d + scale_half, v_scale + at);
                }
            }
            cp_async_arrive(&full[stage]);
            if (++stage == nst) {
                stage = 0;
                parity ^= 1u;
            }
        }
        drain(end - start);
        return;
    }

    // ---------------------------------------------------- consumers
    const int slot = warp / HV, vh = warp - slot * HV, hh = vh / QC, qc = vh - hh * QC;
    const int g = lane >> 2, r = lane & 3, mi = lane >> 3, rr = lane & 7;
    constexpr int kHeads = 8 * kN;
    // O^T: [16-dim chunk][n-tile][dims 2g, 2g + 1 of head 2r at 0, 2, of head 2r + 1 at 1, 3]
    float O[kChunks][kN][4];
    uint32_t qb[kN][kChunks][2];
    [[maybe_unused]] uint32_t ql[kSplit ? kN : 1][kSplit ? kChunks : 1][2];
    float smul[kN][2];  // what a score of heads 8 n + 2 r + e is multiplied by
    float m[kN][2], mu[kN][2], l[kN][2];  // of heads 8 n + 2 r + e; mu: m - kShift where m is finite
    bool poisoned = false;
    int piece = 0, stage = 0;
    uint32_t parity = 0;
    const uint32_t smem_base = smem_u32(smem);
    // this warp's tile k of a step is unit k * slots + slot
    const int tile_off = (slot * HG + hh) * tile_bytes, tile_next = slots * unit_bytes;
    const int scale_off = slot * pl.scale_unit + hh * (kQ8Tok * 4), scale_next = slots * pl.scale_unit;
    const int tok_next = slots * kQ8Tok;
    // ldmatrix: lane group mi gives the rows of matrix mi: (positions 8 (mi & 1) ..,
    // chunk + (mi >> 1))
    uint32_t lm[kChunks / 2];
#pragma unroll
    for (int c = 0; c < kChunks / 2; ++c) lm[c] = q8_at((mi & 1) * 8 + rr, 2 * c + (mi >> 1), pl);

    // One step's kSub tiles; kPart: some of their positions lie behind the end.
    auto tiles = [&](auto part, int ntok) {
        constexpr bool kPart = decltype(part)::value;
        const uint32_t kb0 = smem_base + static_cast<uint32_t>(stage) * pl.stage_bytes + tile_off;
        const uint8_t* sc0 = scales + static_cast<size_t>(stage) * 2 * scale_half + scale_off;
        float x[kSub][kN][4];  // scores of position g (+ 8 for 2, 3), heads 2r, 2r + 1
        float vsc[kSub][2];
        bool over = false;
        float tmax[kN][2];
#pragma unroll
        for (int n = 0; n < kN; ++n) tmax[n][0] = tmax[n][1] = -INFINITY;
#pragma unroll
        for (int k = 0; k < kSub; ++k) {
            if (kPart && k * tok_next >= ntok) {  // no such tile
                vsc[k][0] = vsc[k][1] = 0.f;
#pragma unroll
                for (int n = 0; n < kN; ++n) x[k][n][0] = x[k][n][1] = x[k][n][2] = x[k][n][3] = -INFINITY;
                continue;
            }
            // ---- S^T = K Q^T, in two independent chains
            const uint32_t kb = kb0 + k * tile_next;
            float s[kN][2][4];
#pragma unroll
            for (int n = 0; n < kN; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[n][0][e] = s[n][1][e] = 0.f;
#pragma unroll
            for (int c = 0; c < kChunks; c += 2) {
                uint32_t w[4];
                ldmatrix_x4(w[0], w[1], w[2], w[3], kb + lm[c / 2]);
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    if (c + u >= kMaybe && 16 * (c + u) >= pl.D) break;
                    uint32_t a[4];
                    Fmt::decode4(w[2 * u], a[0], a[2]);
                    Fmt::decode4(w[2 * u + 1], a[1], a[3]);
#pragma unroll
                    for (int n = 0; n < kN; ++n) {
                        if constexpr (kSplit) {
                            float z[4] = {0.f, 0.f, 0.f, 0.f};
                            mma_f16_16816(z, a, ql[n][c + u][0], ql[n][c + u][1]);
                            mma_f16_16816(z, a, qb[n][c + u][0], qb[n][c + u][1]);
#pragma unroll
                            for (int e = 0; e < 4; ++e) s[n][u][e] += z[e];
                        } else {
                            mma_f16_16816(s[n][u], a, qb[n][c + u][0], qb[n][c + u][1]);
                        }
                    }
                }
            }
            // ---- scaled scores, and the largest contribution s_j + log2(vs_j)
            const float* ks = reinterpret_cast<const float*>(sc0 + k * scale_next);
            const float* vs = reinterpret_cast<const float*>(sc0 + k * scale_next + scale_half);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const bool in = !kPart || k * tok_next + 8 * t + g < ntok;
                const float kk = ks[8 * t + g], vv = vs[8 * t + g];
                const float lg = lg2f(fmaxf(fabsf(vv), kMinScale));
                vsc[k][t] = in ? vv : 0.f;
#pragma unroll
                for (int n = 0; n < kN; ++n) {
                    const float2 sum = add2(make_float2(s[n][0][2 * t], s[n][0][2 * t + 1]),
                                            make_float2(s[n][1][2 * t], s[n][1][2 * t + 1]));
                    const float2 a = mul2(sum, mul2(make_float2(kk, kk), make_float2(smul[n][0], smul[n][1])));
                    const float2 c = add2(a, make_float2(lg, lg));
                    x[k][n][2 * t] = in ? a.x : -INFINITY;
                    x[k][n][2 * t + 1] = in ? a.y : -INFINITY;
                    tmax[n][0] = fmaxf(tmax[n][0], in ? c.x : -INFINITY);
                    tmax[n][1] = fmaxf(tmax[n][1], in ? c.y : -INFINITY);
                }
            }
        }
#pragma unroll
        for (int n = 0; n < kN; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) over = over || tmax[n][e] > m[n][e] + kLag;
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
                    const float base = mn == -INFINITY ? 0.f : mn;
                    mu[n][e] = base - kShift;
                    const Shrink by(m[n][e] - base);
                    al[e] = by.both();
                    m[n][e] = mn;
                    l[n][e] = by.of(l[n][e]);
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
        // ---- weights, float16, in P^T's layout.  Their sum is taken over the step first: one
        // by one, those below 2^-24 of the running sum would leave it as it is.
        float2 lsum[kN];
#pragma unroll
        for (int n = 0; n < kN; ++n) lsum[n] = make_float2(0.f, 0.f);
        auto weights = [&](int k, uint32_t (&hi)[kN][2], uint32_t (&lo)[kSplit ? kN : 1][2]) {
#pragma unroll
            for (int n = 0; n < kN; ++n)
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const float2 d = add2(make_float2(x[k][n][2 * t], x[k][n][2 * t + 1]), make_float2(-mu[n][0], -mu[n][1]));
                    const float2 p = make_float2(ex2f_subnormal(d.x), ex2f_subnormal(d.y));
                    lsum[n] = add2(lsum[n], p);
                    const float2 wt = mul2(p, make_float2(vsc[k][t], vsc[k][t]));
                    const uint32_t h = pack_f16x2(wt.x, wt.y);
                    hi[n][t] = transpose_8x8(h);
                    if constexpr (kSplit) {
                        const float2 f = unpack_f16x2(h);
                        lo[n][t] = transpose_8x8(pack_f16x2((wt.x - f.x) * kLowUp, (wt.y - f.y) * kLowUp));
                    }
                }
        };
        // V of tile k, chunks c and c + 1.  Positions behind the end have weight 0; their bytes are
        // cleared because an e4m3 NaN would survive the product.
        auto load_v = [&](int k, int c, uint32_t (&w)[4]) {
            ldmatrix_x4_trans(w[0], w[1], w[2], w[3], kb0 + half_stage + k * tile_next + lm[c / 2]);
            if (!kPart) return;
            const int left = ntok - k * tok_next - 2 * r;
            const uint32_t keep0 = (left > 0 ? 0xffffu : 0u) | (left > 1 ? 0xffff0000u : 0u);
            const uint32_t keep1 = (left > 8 ? 0xffffu : 0u) | (left > 9 ? 0xffff0000u : 0u);
            w[0] &= keep0;
            w[1] &= keep1;
            w[2] &= keep0;
            w[3] &= keep1;
        };
        // ---- O^T += V^T P^T
        if constexpr (kSplit) {
            // A step's products are summed apart (F; with the weights' second float16, 2^11 times as
            // large, E) and added by rounded additions: the MMA truncates what it adds to about 2^-24
            // of its accumulator.
            uint32_t pb[kSub][kN][2], pl2[kSub][kN][2];
#pragma unroll
            for (int k = 0; k < kSub; ++k) {
                if (kPart && k * tok_next >= ntok) break;
                weights(k, pb[k], pl2[k]);
            }
#pragma unroll
            for (int c = 0; c < kChunks; c += 2) {
                float F[2][kN][4], E[2][kN][4];
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int n = 0; n < kN; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) F[u][n][e] = E[u][n][e] = 0.f;
#pragma unroll
                for (int k = 0; k < kSub; ++k) {
                    if (kPart && k * tok_next >= ntok) break;
                    uint32_t w[4];
                    load_v(k, c, w);
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        uint32_t a[4];
                        Fmt::decode4_pairs(w[2 * u], a[0], a[1]);
                        Fmt::decode4_pairs(w[2 * u + 1], a[2], a[3]);
#pragma unroll
                        for (int n = 0; n < kN; ++n) {
                            mma_f16_16816(E[u][n], a, pl2[k][n][0], pl2[k][n][1]);
                            mma_f16_16816(F[u][n], a, pb[k][n][0], pb[k][n][1]);
                        }
                    }
                }
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int n = 0; n < kN; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) O[c + u][n][e] += fmaf(E[u][n][e], 1.f / kLowUp, F[u][n][e]);
            }
        } else {
#pragma unroll
            for (int k = 0; k < kSub; ++k) {
                if (kPart && k * tok_next >= ntok) break;
                uint32_t pb[kN][2], none[1][2];
                weights(k, pb, none);
#pragma unroll
                for (int c = 0; c < kChunks; c += 2) {
                    uint32_t w[4];
                    load_v(k, c, w);
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        uint32_t a[4];
                        Fmt::decode4_pairs(w[2 * u], a[0], a[1]);
                        Fmt::decode4_pairs(w[2 * u + 1], a[2], a[3]);
#pragma unroll
                        for (int n = 0; n < kN; ++n) mma_f16_16816(O[c + u][n], a, pb[n][0], pb[n][1]);
                    }
                }
            }
        }
#pragma unroll
        for (int n = 0; n < kN; ++n) {
            const float2 sum = add2(make_float2(l[n][0], l[n][1]), lsum[n]);
            l[n][0] = sum.x;
            l[n][1] = sum.y;
        }
    };

    // bf16: the MMA truncates what it adds to about 2^-24 of its accumulator, so that of a long
    // tail behind one large weight little would be left.  Every kAside steps (8192 positions of a
    // warp, at most 2^-11 of the result lost in them) the accumulators are added, rescaled, to this
    // warp's place in the workspace and begin again at zero; a range's last ones fetch what is there.
    // The code for it costs 0-1% (64 x 512-4096 58.0 -> 58.2 us; with heads of 32 dimensions
    // 81 -> 84), 4096 positions 1% more on ranges just longer than that, summing every step apart as
    // above up to 5%, and 16 heads a group have no registers for that (128 and 8 heads 84 -> 103).
    constexpr int kAside = 8192 / (kQ8Tok * kSub);
    [[maybe_unused]] int steps = 0;  // of this piece so far, but for its last
    [[maybe_unused]] auto set_aside = [&](bool leave) {
        float* tile = aside + (static_cast<size_t>(blockIdx.x) * kQ8Warps + warp) * q8_aside_floats(DP, kN);
        float4* to = reinterpret_cast<float4*>(tile) + lane;
        float2* to_m = reinterpret_cast<float2*>(tile + DP * kHeads) + lane;
        const bool old = leave || steps > kAside;
#pragma unroll
        for (int n = 0; n < kN; ++n) {
            float f[2] = {0.f, 0.f};
            if (old) {
                const float2 mo = to_m[n * 32];
                f[0] = ex2f(mo.x - (m[n][0] == -INFINITY ? 0.f : m[n][0]));
                f[1] = ex2f(mo.y - (m[n][1] == -INFINITY ? 0.f : m[n][1]));
            }
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
                float4* at = to + (c * kN + n) * 32;
                float4 v = make_float4(O[c][n][0], O[c][n][1], O[c][n][2], O[c][n][3]);
                if (old) {
                    const float4 o = *at;
                    v = make_float4(fmaf(o.x, f[0], v.x), fmaf(o.y, f[1], v.y), fmaf(o.z, f[0], v.z), fmaf(o.w, f[1], v.w));
                }
                if (!leave) {
                    *at = v;
                    v = make_float4(0.f, 0.f, 0.f, 0.f);
                }
                O[c][n][0] = v.x;
                O[c][n][1] = v.y;
                O[c][n][2] = v.z;
                O[c][n][3] = v.w;
            }
            if (!leave) to_m[n * 32] = make_float2(m[n][0], m[n][1]);
        }
    };

    for (int i = start; i < end; ++i) {
        if (!mbar_wait(&full[stage], parity, pl.polls)) {
            if (lane == 0) report(status, PKV_ERR_TIMEOUT);
            return;
        }
        const Q8Meta mt = meta[stage];
        if (mt.flags & kQFirst) {
            const int qs = piece & 1;
            if (!mbar_wait(&qfull[qs], static_cast<uint32_t>(piece >> 1) & 1u, pl.polls)) {
                if (lane == 0) report(status, PKV_ERR_TIMEOUT);
                return;
            }
            // head g (of each n-tile): dims 16 c + 4 r .. + 3
            const uint8_t* qsm = qring + static_cast<size_t>(qs) * pl.q_bytes + hh * pl.G * pl.q_stride;
            // (none for the heads that a last, smaller group lacks)
            const int qrows = (mt.vb % NG) * HG + hh < pl.Hkv ? pl.G : 0;
#pragma unroll
            for (int n = 0; n < kN; ++n) {
                const int row = qc * kHeads + 8 * n + g;
                float v[kChunks][4], amax = 0.f;
#pragma unroll
                for (int c = 0; c < kChunks; ++c) {
                    const int d = c * 16 + 4 * r;
                    float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (row < qrows && d < pl.D) z = load_row4(reinterpret_cast<const T*>(qsm + row * pl.q_stride) + d);
                    v[c][0] = z.x;
                    v[c][1] = z.y;
                    v[c][2] = z.z;
                    v[c][3] = z.w;
                    amax = fmaxf(amax, fmaxf(fmaxf(fabsf(z.x), fabsf(z.y)), fmaxf(fabsf(z.z), fabsf(z.w))));
                }
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
                // amax in [2^(ex-127), 2^(ex-126)) -> [2^14, 2^15); not below 2^-100, infinite: 255
                const int ex = max(static_cast<int>(__float_as_uint(amax) >> 23), 27);
                const float fac = __uint_as_float(static_cast<uint32_t>(268 - ex) << 23);
                const float mul = __uint_as_float(static_cast<uint32_t>(ex - 14) << 23) * pl.scale_log2;
#pragma unroll
                for (int e = 0; e < 2; ++e) smul[n][e] = __shfl_sync(0xffffffffu, mul, 4 * (2 * r + e));
#pragma unroll
                for (int c = 0; c < kChunks; ++c)
#pragma unroll
                    for (int p = 0; p < 2; ++p) {
                        const float a = v[c][2 * p] * fac, b = v[c][2 * p + 1] * fac;
                        qb[n][c][p] = pack_f16x2(a, b);
                        if constexpr (kSplit) {
                            const float2 f = unpack_f16x2(qb[n][c][p]);
                            ql[n][c][p] = pack_f16x2(a - f.x, b - f.y);
                        }
                    }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&qempty[qs]);
            poisoned = false;
            if constexpr (!kSplit) steps = 0;
#pragma unroll
            for (int n = 0; n < kN; ++n) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    m[n][e] = -INFINITY;
                    mu[n][e] = l[n][e] = 0.f;
                }
#pragma unroll
                for (int c = 0; c < kChunks; ++c) O[c][n][0] = O[c][n][1] = O[c][n][2] = O[c][n][3] = 0.f;
            }
        }
        const int ntok = mt.left - slot * kQ8Tok;  // positions from this warp's first one to the end
        poisoned = poisoned || (mt.flags & kQBad);
        if (!poisoned) {
            if (ntok >= (kSub - 1) * tok_next + kQ8Tok)
                tiles(std::false_type(), ntok);
            else if (ntok > 0)
                tiles(std::true_type(), ntok);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[stage]);
        if (++stage == nst) {
            stage = 0;
            parity ^= 1u;
        }
        const bool leave = mt.flags & kQLast;
        if constexpr (kSplit) {
            if (!leave) continue;
        } else {
            // the one way back for nearly all steps comes first (12 heads 85.2 -> 83.8 us), but for
            // 16 heads of 128, whose registers spill (91 us for 85)
            if constexpr (kN * DP < 256) {
                if (!leave && ++steps % kAside != 0) continue;
                if (!leave || steps >= kAside) set_aside(leave);
            } else {
                if (!leave) ++steps;
                if (leave ? steps >= kAside : steps % kAside == 0) set_aside(leave);
            }
            if (!leave) continue;
        }

        // ---------------------------------------------- the range leaves (sequence, group) mt.vb
#pragma unroll
        for (int n = 0; n < kN; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], o);
        if (slots > 1) {
            // merge the slots: at distance d = slots / 2, .., 1 warp slot in [d, 2d) hands its
            // result to slot - d through its own scratch tile (rows padded by 4 floats
            // so that the 4 heads a quarter-warp touches fall on different banks).
            // Each wait is bounded.
            constexpr int kRow = DP + 4, kTile = kHeads * (kRow + 2);
            const uint32_t ph = static_cast<uint32_t>(piece) & 1u;
            bool sent = false;
            for (int d = slots >> 1; d > 0; d >>= 1) {
                if (slot >= d) {
                    float* t = scratch + ((slot - 1) * HV + vh) * kTile;
                    if (!mbar_wait(&mempty[warp], ph ^ 1u, pl.polls)) {
                        if (lane == 0) report(status, PKV_ERR_TIMEOUT);
                        return;
                    }
#pragma unroll
                    for (int n = 0; n < kN; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int head = 8 * n + 2 * r + e;
#pragma unroll
                            for (int c = 0; c < kChunks; ++c)
                                *reinterpret_cast<float2*>(t + head * kRow + 16 * c + 2 * g) =
                                    make_float2(O[c][n][e], O[c][n][2 + e]);
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
                if (!mbar_wait(&mfull[from], ph, pl.polls)) {
                    if (lane == 0) report(status, PKV_ERR_TIMEOUT);
                    return;
                }
#pragma unroll
                for (int n = 0; n < kN; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int head = 8 * n + 2 * r + e;
                        const float2 ml = *reinterpret_cast<const float2*>(t + kHeads * kRow + 2 * head);
                        const float mn = fmaxf(m[n][e], ml.x), base = mn == -INFINITY ? 0.f : mn;
                        const Shrink sa(m[n][e] - base), sb(ml.x - base);
                        const float fa = sa.both(), fb = sb.both();
                        m[n][e] = mn;
                        l[n][e] = sa.of(l[n][e]) + sb.of(ml.y);
#pragma unroll
                        for (int c = 0; c < kChunks; ++c) {
                            const float2 o = *reinterpret_cast<const float2*>(t + head * kRow + 16 * c + 2 * g);
                            O[c][n][e] = fmaf(O[c][n][e], fa, o.x * fb);
                            O[c][n][2 + e] = fmaf(O[c][n][2 + e], fa, o.y * fb);
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
#pragma unroll
        for (int n = 0; n < kN; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int head = qc * kHeads + 8 * n + 2 * r + e;
                const int qr = hh * pl.G + head;  // row in the group
                const int vb_g = mt.vb % NG, row = (mt.vb / NG) * pl.Hq + vb_g * pl.R + qr;  // row of out
                if (head >= pl.G || vb_g * pl.R + qr >= pl.Hq) continue;
                if (mt.flags & kQWhole) {
                    const float inv = poisoned || l[n][e] == 0.f ? 0.f : 1.f / l[n][e];
                    T* o = out + static_cast<size_t>(row) * pl.D + 2 * g;
#pragma unroll
                    for (int c = 0; c < kChunks; ++c)
                        if (16 * c < pl.D)
                            store_row2(o + 16 * c, poisoned ? 0.f : O[c][n][e] * inv, poisoned ? 0.f : O[c][n][2 + e] * inv);
                } else {
                    const size_t at = (2 * static_cast<size_t>(blockIdx.x) + ((mt.flags & kQHead) ? 0 : 1)) * pl.R + qr;
                    if (g == 0)
                        *reinterpret_cast<float2*>(part_ml + 2 * at) = make_float2(m[n][e], poisoned ? -1.f : l[n][e]);
#pragma unroll
                    for (int c = 0; c < kChunks; ++c)
                        if (16 * c < pl.D)
                            *reinterpret_cast<float2*>(part_o + at * pl.D + 16 * c + 2 * g) =
                                make_float2(O[c][n][e], O[c][n][2 + e]);
                }
            }
    }
}

// ------------------------------------------------------------------ join
// M = max m_c, out = sum o_c 2^(m_c - M) / sum l_c 2^(m_c - M) over the pieces of
// a sequence that several ranges share: the piece of its first range f in slot
// 2f + 1, of a later range c in slot 2c.  kUnitWarps warps per (sequence, query
// head): one where there are many, four (over the pieces) where there are few.  The whole
// call with one and with four: 64 x 32 of them 57.7 and 60.8 us, 512 x 32 114 and 138 us;
// 8 x 32 in sequences of 100-1000 12.3 and 10.1 us, 8 x 64 in long ones 236 and 231 us.
// kCuts: the units are the rows at the starts of ranges instead of those of all sequences,
// where there are fewer of them; a start that cuts a (sequence, group) first joins it (1000
// sequences of 100-500, 32 and 8 heads 131 -> 118 us, 512 of 128-1024 114 -> 109).
// Sequences within one range were written by the main kernel; empty and invalid ones get
// zeros here, with kCuts from CTAs of their own.
constexpr int kZeroSeqs = 16;
constexpr int kJoinWarps = 4;
constexpr int kJoinGroup = 8;

template <typename T, int kUnitWarps, bool kCuts>
__global__ void __launch_bounds__(kJoinWarps * 32)
    decode_q8_join_kernel(const __grid_constant__ Q8Plan pl, const int32_t* seq_lens, const float* part_ml,
                          const float* part_o, T* out, int P, int32_t* status) {
    __shared__ float4 accsh[kJoinWarps][32];
    __shared__ float mlsh[kJoinWarps][2];
    __shared__ int sums[kCuts ? 36 : 2 * kJoinWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, w0 = warp % kUnitWarps;
    // Where the sequence's steps lie in the order, from the lengths: they are older than the
    // main kernel, which launched this one after its own wait, so everything up to the
    // partials' addresses is done before the wait.
    int pieces = 0, f = 0, row = 0;
    bool invalid = false, empty = false;
    unsigned u = 0;  // row of out
    if constexpr (kCuts) {
        static_assert(kUnitWarps == 1, "rows of a cut");
        const int per = (pl.R + kJoinWarps - 1) / kJoinWarps, c = 1 + static_cast<int>(blockIdx.x) / per;
        if (c >= P) {  // a CTA for kZeroSeqs sequences: zeros for those without steps
            asm volatile("griddepcontrol.wait;" ::: "memory");
            asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
            const int b0 = (static_cast<int>(blockIdx.x) - (P - 1) * per) * kZeroSeqs;
            for (int b = b0 + warp; b < min(pl.B, b0 + kZeroSeqs); b += kJoinWarps) {
                if (q8_steps(seq_lens, b, pl) != 0) continue;
                T* o = out + static_cast<size_t>(b) * pl.Hq * pl.D;
                for (int e = lane; e < pl.Hq * pl.D; e += 32) o[e] = from_f32<T>(0.f);
                if (lane == 0 && seq_lens[b] != 0) report(status, PKV_ERR_DEVICE_BOUNDS);
            }
            return;
        }
        row = (static_cast<int>(blockIdx.x) - (c - 1) * per) * kJoinWarps + warp;
        int sum = 0, total, carry = 0;
        for (int x = threadIdx.x; x < pl.B; x += kJoinWarps * 32) sum += pl.NG * q8_steps(seq_lens, x, pl);
        q8_scan(sum, sums, total);
        const int W = (total + P - 1) / P;
        const long long at = static_cast<long long>(c) * W;
        if (at < total) {  // uniform over the CTA; then one sequence holds step `at`
            const int start = static_cast<int>(at);
            for (int base = 0; base < pl.B; base += kJoinWarps * 32) {
                const int x = base + threadIdx.x, n = x < pl.B ? pl.NG * q8_steps(seq_lens, x, pl) : 0;
                int tot;
                const int sb = carry + q8_scan(n, sums, tot);
                if (n > 0 && sb <= start && start < sb + n) {
                    sums[33] = x;
                    sums[34] = sb;
                    sums[35] = n;
                }
                carry += tot;
                if (carry > start) break;  // same decision in every thread
            }
            __syncthreads();
            const int b = sums[33], n = sums[35] / pl.NG, grp = (start - sums[34]) / n, first = sums[34] + grp * n;
            f = first / W;
            if (first < start && f == c - 1 && row < min(pl.R, pl.Hq - grp * pl.R)) {
                pieces = (first + n - 1) / W - f + 1;
                u = static_cast<unsigned>(b) * pl.Hq + grp * pl.R + row;
            }
        }
    } else {
        const unsigned units = static_cast<unsigned>(pl.B) * pl.Hq;
        const unsigned u0 = blockIdx.x * (kJoinWarps / kUnitWarps);
        u = u0 + warp / kUnitWarps;
        const bool in = u < units;
        const int b = static_cast<int>((in ? u : u0) / pl.Hq), bfirst = static_cast<int>(u0 / pl.Hq);
        const int qh = in ? static_cast<int>(u - static_cast<unsigned>(b) * pl.Hq) : 0, grp = qh / pl.R;
        const int n = q8_steps(seq_lens, b, pl);
        int all = 0, before = 0;
        for (int x = threadIdx.x; x < pl.B; x += kJoinWarps * 32) {
            const int k = q8_steps(seq_lens, x, pl);
            all += k;
            before += x < bfirst ? k : 0;
        }
        all = __reduce_add_sync(0xffffffffu, all);
        before = __reduce_add_sync(0xffffffffu, before);
        if (lane == 0) {
            sums[2 * warp] = all;
            sums[2 * warp + 1] = before;
        }
        __syncthreads();
        all = before = 0;
#pragma unroll
        for (int w = 0; w < kJoinWarps; ++w) {
            all += sums[2 * w];
            before += sums[2 * w + 1];
        }
        for (int x = bfirst; x < b; ++x) before += q8_steps(seq_lens, x, pl);
        if (in && n > 0) {
            const int W = (all * pl.NG + P - 1) / P, first = before * pl.NG + grp * n;
            f = first / W;
            pieces = (first + n - 1) / W - f + 1;
        }
        empty = in && n == 0;
        invalid = empty && seq_lens[b] != 0 && qh == 0 && w0 == 0;
        row = qh - grp * pl.R;
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (invalid && lane == 0) report(status, PKV_ERR_DEVICE_BOUNDS);
    const bool write = empty || pieces > 1;
    if (kUnitWarps == 1 && !write) return;
    if (pieces == 1) pieces = 0;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float M = -INFINITY, l = 0.f;
    const bool col = 4 * lane < pl.D;
    // pieces w0, w0 + kUnitWarps, ..: kJoinGroup of them in flight
    for (int p0 = w0; p0 < pieces; p0 += kUnitWarps * kJoinGroup) {
        float2 ml[kJoinGroup];
        float4 o[kJoinGroup];
#pragma unroll
        for (int k = 0; k < kJoinGroup; ++k) {
            const int p = p0 + k * kUnitWarps;
            const size_t at = (static_cast<size_t>(2 * (f + p) + (p == 0 ? 1 : 0))) * pl.R + row;
            ml[k] = p < pieces ? __ldcg(reinterpret_cast<const float2*>(part_ml + 2 * at)) : make_float2(kCuts ? -INFINITY : ml[0].x, 0.f);
            o[k] = p < pieces && col ? __ldcg(reinterpret_cast<const float4*>(part_o + at * pl.D + 4 * lane))
                                     : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        float mn = M;
#pragma unroll
        for (int k = 0; k < kJoinGroup; ++k) mn = fmaxf(mn, ml[k].x);
        const float mu = mn == -INFINITY ? 0.f : mn;
        const Shrink by(M - mu);
        const float fa = by.both();
        bool bad = l < 0.f, flushed = false;
        l = by.of(l);
        acc = make_float4(acc.x * fa, acc.y * fa, acc.z * fa, acc.w * fa);
        M = mn;
#pragma unroll
        for (int k = 0; k < kJoinGroup; ++k) {
            float w;
            // 2^d first and the flushed ones again where there are any, against Shrink for all: 64 x
            // 512-4096 58.0 : 58.6 us, 37 x 0-1500 13.6 : 14.3; with cuts, whose many short CTAs want
            // few registers (56 : 72), 512 x 128-1024 112.6 : 110.5.
            if constexpr (kCuts) {
                const Shrink byk(ml[k].x - mu);
                w = byk.both();
                l += byk.of(ml[k].y);
            } else {
                w = ex2f(ml[k].x - mu);
                flushed = flushed || w == 0.f;
                l = fmaf(ml[k].y, w, l);
            }
            bad = bad || ml[k].y < 0.f;
            acc.x = fmaf(o[k].x, w, acc.x);
            acc.y = fmaf(o[k].y, w, acc.y);
            acc.z = fmaf(o[k].z, w, acc.z);
            acc.w = fmaf(o[k].w, w, acc.w);
        }
        if (flushed) {  // a sum may make up for the zero
#pragma unroll
            for (int k = 0; k < kJoinGroup; ++k)
                if (ex2f(ml[k].x - mu) == 0.f) l += Shrink(ml[k].x - mu).of(ml[k].y);
        }
        if (bad) l = -INFINITY;  // stays: a poisoned piece makes the row zero
    }
    if (kUnitWarps > 1) {
        accsh[warp][lane] = acc;
        if (lane == 0) {
            mlsh[warp][0] = M;
            mlsh[warp][1] = l;
        }
        __syncthreads();
        if (w0 != 0 || !write) return;
        float mn = M;
        for (int w = 1; w < kUnitWarps; ++w) mn = fmaxf(mn, mlsh[warp + w][0]);
        const float mu = mn == -INFINITY ? 0.f : mn;
        bool bad = l < 0.f;
        const Shrink by(M - mu);
        const float fa = by.both();
        l = by.of(l);
        acc = make_float4(acc.x * fa, acc.y * fa, acc.z * fa, acc.w * fa);
        for (int w = 1; w < kUnitWarps; ++w) {
            const Shrink byw(mlsh[warp + w][0] - mu);
            const float f2 = byw.both();
            const float4 o = accsh[warp + w][lane];
            bad = bad || mlsh[warp + w][1] < 0.f;
            l += byw.of(mlsh[warp + w][1]);
            acc.x = fmaf(o.x, f2, acc.x);
            acc.y = fmaf(o.y, f2, acc.y);
            acc.z = fmaf(o.z, f2, acc.z);
            acc.w = fmaf(o.w, f2, acc.w);
        }
        if (bad) l = -INFINITY;
    }
    if (!col) return;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (l != 0.f && l != -INFINITY) {
        const float inv = 1.f / l;
        v = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    }
    store_row4(out + static_cast<size_t>(u) * pl.D + 4 * lane, v);
}

// ------------------------------------------------------------------ generic kernel
// D not a multiple of 16 or above 128, block sizes that are not multiples of 16, addresses that
// are not 16-byte aligned, more than 64 (float32) or 128 query heads a KV head.  A thread takes
// one position's score, then one or two dimensions of the output; bound by the latency of
// its byte loads.
constexpr int kGen8Threads = 128;

template <typename T, typename Fmt>
__global__ void __launch_bounds__(kGen8Threads)
    decode_q8_generic_kernel(T* out, const T* q, const uint8_t* k_cache, const uint8_t* v_cache, const float* k_scale,
                             const float* v_scale, const int32_t* block_tables, int max_blocks,
                             const int32_t* seq_lens, int Hq, int Hkv, int D, int BS, int NB, float scale,
                             int32_t* status) {
    __shared__ float qs[256];
    __shared__ float ps[kGen8Threads];
    __shared__ long long rows[kGen8Threads];
    __shared__ float red[kGen8Threads / 32];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int b = blockIdx.x / Hq, qh = blockIdx.x % Hq, h = qh / (Hq / Hkv);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    T* o = out + (static_cast<size_t>(b) * Hq + qh) * D;
    const int L = seq_lens[b];
    bool bad = L < 0 || static_cast<long long>(L) > static_cast<long long>(max_blocks) * BS;
    for (int d = tid; d < D; d += kGen8Threads) qs[d] = to_f32(q[(static_cast<size_t>(b) * Hq + qh) * D + d]);
    float m = -INFINITY, l = 0.f, acc[2] = {0.f, 0.f};
    for (int t0 = 0; !bad && t0 < L; t0 += kGen8Threads) {
        __syncthreads();
        const int n = min(kGen8Threads, L - t0);
        float s = -INFINITY, vs = 0.f;
        bool miss = false;
        if (tid < n) {
            const int pos = t0 + tid;
            const int blk = block_tables[static_cast<size_t>(b) * max_blocks + pos / BS];
            if (blk < 0 || blk >= NB) {
                miss = true;
            } else {
                const long long row = (static_cast<long long>(blk) * Hkv + h) * BS + pos % BS;
                const uint8_t* kr = k_cache + row * D;
                float dot = 0.f;
                for (int d = 0; d < D; ++d) dot = fmaf(qs[d], Fmt::decode(kr[d]), dot);
                s = dot * k_scale[row] * scale;
                vs = v_scale[row];
                rows[tid] = row;
            }
        }
        if (__syncthreads_or(miss)) {
            bad = true;
            break;
        }
        float mx = s;
        for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
        if (lane == 0) red[warp] = mx;
        __syncthreads();
        mx = red[0];
        for (int w = 1; w < kGen8Threads / 32; ++w) mx = fmaxf(mx, red[w]);
        __syncthreads();
        const float mn = fmaxf(m, mx), mu = mn == -INFINITY ? 0.f : mn;
        const float alpha = expf(m - mu);
        const float p = tid < n ? expf(s - mu) : 0.f;
        ps[tid] = p * (vs * 0x1p-40f);  // sums of up to 2^31 rows near the largest float stay finite
        float sm = p;
        for (int off = 16; off > 0; off >>= 1) sm += __shfl_xor_sync(0xffffffffu, sm, off);
        if (lane == 0) red[warp] = sm;
        __syncthreads();
        float psum = 0.f;
        for (int w = 0; w < kGen8Threads / 32; ++w) psum += red[w];
        l = l * alpha + psum;
        m = mn;
        for (int k = 0; k < 2; ++k) {
            const int d = tid + k * kGen8Threads;
            if (d >= D) continue;
            float a = acc[k] * alpha;
            for (int t = 0; t < n; ++t) a = fmaf(ps[t], Fmt::decode(v_cache[rows[t] * D + d]), a);
            acc[k] = a;
        }
    }
    if (bad && tid == 0) report(status, PKV_ERR_DEVICE_BOUNDS);
    const float inv = bad || l == 0.f ? 0.f : 0x1p40f / l;
    for (int k = 0; k < 2; ++k) {
        const int d = tid + k * kGen8Threads;
        if (d < D) o[d] = from_f32<T>(bad ? 0.f : acc[k] * inv);
    }
}

// ------------------------------------------------------------------ host side
struct Q8Layout {  // workspace
    size_t o, aside, total;
};

// Group size and slots for a shape, with at least min_groups head groups where the heads
// allow it; false where the fast kernel does not apply.
static bool q8_shape(int Hq, int Hkv, int D, int BS, pkv_dtype dt, int min_groups, Q8Plan& pl) {
    if (D % 16 != 0 || D > 128 || BS % 16 != 0) return false;
    const int G = Hq / Hkv, rows = dt == PKV_F32 || G <= 8 ? 8 : 16;  // query heads per warp
    pl.QC = (G + rows - 1) / rows;
    if (pl.QC > kQ8Warps) return false;
    // as few groups as the warps allow, of equal size (the last one up to NG - 1 heads
    // smaller: 11 heads are 6 + 5; the tile of the missing head is read and not used)
    const int most = kQ8Warps / pl.QC;
    pl.NG = std::max((Hkv + most - 1) / most, std::min(min_groups, Hkv));
    pl.HG = (Hkv + pl.NG - 1) / pl.NG;
    pl.NG = (Hkv + pl.HG - 1) / pl.HG;
    pl.UB = BS / kQ8Tok;
    pl.layout = D == 128 ? kSwizzled : D == 64 ? kPacked : kDense;
    pl.tok_shift = D == 128 ? 0 : D == 64 ? 1 : 4;
    pl.sub = D <= 64 ? 4 : 2;  // steps of about 64 KB (D 64, 64 x 512-8192: 60.7 us with 2, 56.1 with 4)
    pl.slots = 1;
    while (pl.slots * 2 * pl.HG * pl.QC <= kQ8Warps) pl.slots *= 2;
    pl.G = G;
    pl.R = pl.HG * G;
    return true;
}

// Two partial results per CTA of (max, sum) and D floats for every row of a group.
// With aside: the accumulators that a CTA's warps set aside (bf16; of up to 16 heads).
static Q8Layout q8_layout(int R, int D, int P, bool aside) {
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    Q8Layout w;
    w.o = up(static_cast<size_t>(2) * P * R * 2 * sizeof(float));
    w.aside = up(w.o + static_cast<size_t>(2) * P * R * D * sizeof(float));
    const int DP = (D + 31) / 32 * 32;
    w.total = up(w.aside + (aside ? static_cast<size_t>(P) * kQ8Warps * q8_aside_floats(DP, 2) * sizeof(float) : 0));
    return w;
}

// A pool [NB * Hkv][BS][D] of bytes in boxes of 16 positions x HG heads, the positions in
// rows of 2^tok_shift (128-byte rows, or for kDense one row of 16 D bytes a head).
static bool q8_map(CUtensorMap* map, const void* pool, const Q8Plan& pl) {
    EncodeTiledFn enc = get_encode_fn();
    if (!enc) return false;
    const bool dense = pl.layout == kDense;
    const cuuint64_t row = static_cast<cuuint64_t>(pl.D) << pl.tok_shift, elem = dense ? 8 : 1;
    cuuint64_t dim[3] = {row / elem, static_cast<cuuint64_t>(pl.BS) >> pl.tok_shift,
                         static_cast<cuuint64_t>(pl.NB) * pl.Hkv};
    cuuint64_t stride[2] = {row, static_cast<cuuint64_t>(pl.D) * pl.BS};
    cuuint32_t box[3] = {static_cast<cuuint32_t>(row / elem), static_cast<cuuint32_t>(kQ8Tok) >> pl.tok_shift,
                         static_cast<cuuint32_t>(pl.HG)};
    cuuint32_t one[3] = {1, 1, 1};
    return enc(map, dense ? CU_TENSOR_MAP_DATA_TYPE_UINT64 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(pool),
               dim, stride, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
               dense ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, typename Fmt, int DP, int kN>
static cudaError_t launch_q8_fast(Q8Plan pl, void* out, const void* q, const void* k, const void* v, const float* ks,
                                  const float* vs, const int32_t* block_tables, const int32_t* seq_lens,
                                  void* workspace, int P, int32_t* status, cudaStream_t stream, bool* done) {
    *done = false;
    constexpr bool kSplit = sizeof(T) == 4;
    constexpr int kSub = DP <= 64 ? 4 : 2;
    const int tiles = pl.HG * pl.slots * kSub;
    pl.stage_bytes = 2 * tiles * kQ8Tok * pl.D;
    pl.scale_unit = pl.HG * kQ8Tok * 4;
    // rows 32 (bf16) or 64 bytes apart modulo 128, so that the 8 heads a warp reads at
    // once fall on different banks
    pl.q_stride = (pl.D * static_cast<int>(sizeof(T)) + 127) / 128 * 128 + 16 * static_cast<int>(sizeof(T));
    pl.q_bytes = pl.R * pl.q_stride;
    pl.scratch_bytes = (pl.slots - 1) * pl.HG * pl.QC * (8 * kN * (DP + 6)) * 4;
    const size_t fixed = 1024 + 2 * static_cast<size_t>(pl.q_bytes) + pl.scratch_bytes +
                         (2 * kQ8MaxStages + 4 + 2 * kQ8Warps) * sizeof(uint64_t) + kQ8MaxStages * sizeof(Q8Meta) +
                         40 * sizeof(int) + 16;
    const size_t per = pl.stage_bytes + 2 * static_cast<size_t>(pl.slots) * kSub * pl.scale_unit;
    const size_t budget = static_cast<size_t>(max_optin_smem());
    if (fixed + 2 * per > budget) return cudaSuccess;
    pl.nst = static_cast<int>(std::min<size_t>(kQ8MaxStages, (budget - fixed) / per));
    const size_t smem = fixed + pl.nst * per;
    CUtensorMap tmK, tmV;
    if (!q8_map(&tmK, k, pl) || !q8_map(&tmV, v, pl)) return cudaSuccess;
    const Q8Layout wl = q8_layout(pl.R, pl.D, P, !kSplit);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    float* part_ml = reinterpret_cast<float*>(ws);
    float* part_o = reinterpret_cast<float*>(ws + wl.o);
    float* aside = reinterpret_cast<float*>(ws + wl.aside);
    auto kern = decode_q8_kernel<T, Fmt, DP, kN, kSplit, kSub>;
    // The limit belongs to the kernel, not to the call: always the device's largest, so that
    // another thread's call with other sizes cannot lower it between here and the launch.
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
    err = cudaLaunchKernelEx(&cfg, kern, tmK, tmV, pl, static_cast<const T*>(q), static_cast<T*>(out),
                             ks, vs, block_tables, seq_lens, part_ml, part_o, aside, status);
    if (err != cudaSuccess) return err;
    if (pl.direct) {
        *done = true;
        return cudaGetLastError();
    }
    const long long units = static_cast<long long>(pl.B) * pl.Hq;
    const bool many = units >= 8LL * P, cuts = many && pl.B * static_cast<long long>(pl.NG) > P && P > 1;
    const long long per_cut = (pl.R + kJoinWarps - 1) / kJoinWarps;
    cfg.gridDim = dim3(static_cast<unsigned>(cuts   ? (P - 1) * per_cut + (pl.B + kZeroSeqs - 1) / kZeroSeqs
                                             : many ? (units + kJoinWarps - 1) / kJoinWarps
                                                    : units),
                       1, 1);
    cfg.blockDim = dim3(kJoinWarps * 32, 1, 1);
    cfg.dynamicSmemBytes = 0;
    auto join = cuts   ? decode_q8_join_kernel<T, 1, true>
                : many ? decode_q8_join_kernel<T, 1, false>
                       : decode_q8_join_kernel<T, kJoinWarps, false>;
    err = cudaLaunchKernelEx(&cfg, join, pl, seq_lens, static_cast<const float*>(part_ml),
                             static_cast<const float*>(part_o), static_cast<T*>(out), P, status);
    if (err != cudaSuccess) return err;
    *done = true;
    return cudaGetLastError();
}

template <typename T, typename Fmt>
static cudaError_t launch_q8(Q8Plan pl, bool fast, void* out, const void* q, const void* k, const void* v,
                             const float* ks, const float* vs, const int32_t* block_tables, const int32_t* seq_lens,
                             float scale, void* workspace, int P, int32_t* status, cudaStream_t stream) {
    if (fast) {
        bool done = false;
        cudaError_t err = cudaSuccess;
        auto run = [&](auto dp, auto n) {
            return launch_q8_fast<T, Fmt, decltype(dp)::value, decltype(n)::value>(
                pl, out, q, k, v, ks, vs, block_tables, seq_lens, workspace, P, status, stream, &done);
        };
        using I1 = std::integral_constant<int, 1>;
        using I2 = std::integral_constant<int, 2>;
        using I32 = std::integral_constant<int, 32>;
        using I64 = std::integral_constant<int, 64>;
        using I96 = std::integral_constant<int, 96>;
        using I128 = std::integral_constant<int, 128>;
        auto go = [&]() {
            if constexpr (sizeof(T) == 2) {
                if (pl.G > 8)
                    return pl.D <= 32   ? run(I32(), I2())
                           : pl.D <= 64 ? run(I64(), I2())
                           : pl.D <= 96 ? run(I96(), I2())
                                        : run(I128(), I2());
            }
            return pl.D <= 32   ? run(I32(), I1())
                   : pl.D <= 64 ? run(I64(), I1())
                   : pl.D <= 96 ? run(I96(), I1())
                                : run(I128(), I1());
        };
        // Few and short sequences (by the table's width): a CTA for each (sequence, head
        // group) and no join, with as many groups as there are SMs for.
        const Q8Plan split = pl;
        auto short_table = [](const Q8Plan& p) {
            return static_cast<long long>(p.max_blocks) * p.BS <= kDirectSteps * p.slots * p.sub * kQ8Tok;
        };
        pl.direct = pl.B <= P && q8_shape(pl.Hq, pl.Hkv, pl.D, pl.BS, sizeof(T) == 4 ? PKV_F32 : PKV_BF16, P / pl.B, pl) &&
                    pl.B * pl.NG <= P && short_table(pl);
        if (pl.direct) {
            err = go();
            if (err != cudaSuccess || done) return err;
        }
        pl = split;
        err = go();
        if (err != cudaSuccess || done) return err;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(pl.B) * pl.Hq, 1, 1);
    cfg.blockDim = dim3(kGen8Threads, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t err = cudaLaunchKernelEx(
        &cfg, decode_q8_generic_kernel<T, Fmt>, static_cast<T*>(out), static_cast<const T*>(q),
        static_cast<const uint8_t*>(k), static_cast<const uint8_t*>(v), ks, vs, block_tables, pl.max_blocks, seq_lens,
        pl.Hq, pl.Hkv, pl.D, pl.BS, pl.NB, scale, status);
    return err != cudaSuccess ? err : cudaGetLastError();
}

}  // namespace pkv

extern "C" size_t pkv_decode_q8_workspace_bytes(int B, int Hq, int Hkv, int D, int num_sms) {
    using namespace pkv;
    if (B < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || D < 1) return 0;
    const int P = num_sms > 0 ? num_sms : device_sm_count();
    if (P <= 0) return 0;
    // the block size and the type do not change the layout's size, but for the chunk
    // of query heads: take the larger
    size_t need = 256;
    for (pkv_dtype dt : {PKV_F32, PKV_BF16}) {
        Q8Plan pl = {};
        if (q8_shape(Hq, Hkv, D, 16, dt, 1, pl)) need = std::max(need, q8_layout(pl.R, D, P, dt == PKV_BF16).total);
    }
    return need;
}

extern "C" pkv_status pkv_paged_decode_attention_q8(
    void* out, const void* q, const void* k_cache, const void* v_cache, const float* k_scale, const float* v_scale,
    const int32_t* block_tables, int max_blocks_per_seq, const int32_t* seq_lens, int B, int Hq, int Hkv, int D,
    int block_size, int num_blocks, float scale, pkv_dtype dtype, pkv_dtype cache_dtype, void* workspace,
    size_t workspace_bytes, int32_t* dev_status, void* stream) {
    using namespace pkv;
    if (B < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || D < 1 || D > 256 || block_size < 1 || num_blocks < 1 ||
        max_blocks_per_seq < 1 || (dtype != PKV_F32 && dtype != PKV_BF16) ||
        (cache_dtype != PKV_E4M3 && cache_dtype != PKV_I8))
        return PKV_ERR_INVALID_ARG;
    if (static_cast<long long>(B) * Hq > 0x7fffffffLL) return PKV_ERR_INVALID_ARG;
    if (B == 0) return PKV_OK;
    if (!out || !q || !k_cache || !v_cache || !k_scale || !v_scale || !block_tables || !seq_lens || !workspace)
        return PKV_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(workspace) & 15u) != 0) return PKV_ERR_INVALID_ARG;
    const int P = device_sm_count();
    if (workspace_bytes < pkv_decode_q8_workspace_bytes(B, Hq, Hkv, D, P > 0 ? P : 1)) return PKV_ERR_INVALID_ARG;
    if (P <= 0) return PKV_ERR_CUDA;
    if (scale <= 0.f) scale = 1.0f / sqrtf(static_cast<float>(D));
    Q8Plan pl = {};
    bool fast = q8_shape(Hq, Hkv, D, block_size, dtype, 1, pl);
    pl.G = Hq / Hkv;
    pl.B = B;
    pl.Hq = Hq;
    pl.Hkv = Hkv;
    pl.D = D;
    pl.BS = block_size;
    pl.NB = num_blocks;
    pl.max_blocks = max_blocks_per_seq;
    pl.scale_log2 = scale * 1.4426950408889634f;
    pl.polls = attention_wait_polls();
    pl.silent_cta = attention_silent_cta();
    auto aligned16 = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
    fast = fast && aligned16(q) && aligned16(out) && aligned16(k_cache) && aligned16(v_cache) && aligned16(k_scale) &&
           aligned16(v_scale);
    // step and row counts stay in 32 bits
    if (fast) {
        const long long steps = (static_cast<long long>(max_blocks_per_seq) * block_size) / (16 * pl.slots) + 1;
        fast = steps * B * pl.NG < (1LL << 30) && static_cast<long long>(num_blocks) * Hkv < (1LL << 31);
    }
    auto go = dtype == PKV_F32 ? (cache_dtype == PKV_E4M3 ? launch_q8<float, FmtE4M3> : launch_q8<float, FmtI8>)
                               : (cache_dtype == PKV_E4M3 ? launch_q8<__nv_bfloat16, FmtE4M3>
                                                          : launch_q8<__nv_bfloat16, FmtI8>);
    const cudaError_t err = go(pl, fast, out, q, k_cache, v_cache, k_scale, v_scale, block_tables, seq_lens, scale,
                               workspace, P, dev_status, static_cast<cudaStream_t>(stream));
    return err == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}
