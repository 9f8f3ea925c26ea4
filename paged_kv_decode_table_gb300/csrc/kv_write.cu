// kv_write.cu -- new tokens on their way into the paged cache: the append that
// quantises to 8 bits, and the pass that normalises and rotates queries and keys
// before the append.
//
// For token t of sequence b at position pos (the last position of the sequence,
// or chunk token i at seq_lens[b] - n_b + i), with row x of D values:
//   norm      y_i = x_i * rsqrt(mean(x^2) + eps) * w_i           (q and k, w per kind)
//   rotation  (y_a, y_c) -> (y_a cos - y_c sin, y_c cos + y_a sin), angle pos * f_j,
//             pairs (j, j + rot/2) or (2j, 2j + 1), j < rot/2
//   store     q -> q_out; k, v -> the slot of position pos, as they are or in
//             8 bits with a scale (quant8.cuh).
// Everything between the load and the store is float32 and each result is
// rounded once.  The frequency comes as turns per position in units of 2^-64
// (a 64-bit integer): pos * f wraps modulo one turn in integer arithmetic, and the
// nearest quarter turn is taken off there too, before the one rounding to float32:
// the angle is off by at most 2^-28 of a turn, at every position alike.
//
// Vector kernel (D a multiple of 8, 16-byte aligned rows): a lane holds 8 elements of
// a row in two runs of 4, D / 8 lanes a row, 32 / (D / 8) rows a warp and pass.  A lane's
// dimensions are the same in every row, so cosines, sines and norm weights are
// read once per token into registers, and for pairs (j, j + half) the second run
// holds the partners of the first (half a multiple of 4; else they come through
// shared memory).  The first rows are loaded before the token's place and angles
// are known, which hides that chain of loads, and later ones a pass early.
// Two rows per lane are in work at once, two queries or a key and a value, which overlaps
// their reductions' shuffles; head sizes 64 and 128 have the lanes of a row as constants
// (64 tokens of 32 + 8 heads 3.2 -> 3.0 us).  The other kernel (any D and alignment) gives a
// warp one row, one element per lane and step.
//
// Bound by instruction issue, then HBM: 6147 tokens of 32 + 8 heads of 128 in bf16, normalised
// and rotated into a bf16 cache, 27.4 us for 151 MB, 5.5 TB/s, 82% of the measured copy rate,
// two thirds of the issue slots.  The quantising append of 5226 tokens of 8 heads 9.5 us for
// 32 MB, 50%, at as many issue slots.  64 tokens 2.8 us, 1 token 2.3 us: launch and three
// dependent loads.  Two designs that fed consumer warps by bulk copies, one CTA or two an SM,
// took 34.8 and 37.5 us on the first case when this one took 35.8.
#include <algorithm>
#include <type_traits>

#include "quant8.cuh"

namespace pkv {

constexpr int kWriteWarps = 8;
constexpr int kWriteMaxD = 256;
constexpr int kSmShared = 228 * 1024;  // an SM's, of which a CTA takes 1 KB besides its own
// Pairs of passes of one token, where there are enough tokens.  128 + 8 heads, 2420 and 10697
// tokens: 4 pairs 36.5 and 147, 8 31.6 and 124, 16 33.5 and 120 us.
constexpr int kPairsPerWarp = 8;

int device_sm_count();

struct WriteArgs {
    void* q_out;
    const void *q, *k, *v;
    long long q_stride, k_stride, v_stride;  // elements between tokens
    const void *q_weight, *k_weight;         // null: no norm
    float eps;
    const int64_t* freqs;
    int half;  // rot_dim / 2 (0: no rotation)
    int interleaved;
    void *k_cache, *v_cache;
    float *k_scale, *v_scale;
    const int32_t *block_tables, *seq_lens, *q_start;
    int max_blocks, B, T, Hq, Hkv, D, BS, NB;
    int32_t* status;
};

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}
__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}

// Where token t goes.  live: a token of some sequence (the rows behind the last one are
// not); ok: the sequence's length and chunk are valid, and pos and slot are set.
// blk_raw is the table's entry, still unchecked: its load is not waited for here.
struct Place {
    int live, ok, pos, slot, blk_raw;
    __device__ __forceinline__ int blk(int NB) const { return ok && blk_raw >= 0 && blk_raw < NB ? blk_raw : -1; }
};

// Called by a whole warp with one t < T.
__device__ __forceinline__ Place place_of(const WriteArgs& a, int t) {
    Place p{1, 0, 0, 0, -1};
    int b = t, n = 1, i = 0, L;
    if (a.q_start != nullptr) {
        // the last b with q_start[b] <= t: 32 probes per round, and with at most 32
        // sequences left one round trip brings their starts, ends and lengths
        const int lane = threadIdx.x & 31;
        const int tend = a.q_start[a.B];
        int lo = 0, count = a.B;  // in [lo, lo + count)
        while (count > 32) {
            const int step = (count + 31) / 32, at = lane * step;
            const unsigned below = __ballot_sync(0xffffffffu, at < count && (at == 0 || a.q_start[lo + at] <= t));
            const int hit = 31 - __clz(below);  // lane 0 always is
            lo += hit * step;
            count = min(step, count - hit * step);
        }
        const int mine = lo + min(lane, count - 1);
        const int s0 = a.q_start[mine], s1 = a.q_start[mine + 1], len = a.seq_lens[mine];
        const unsigned below = __ballot_sync(0xffffffffu, lane < count && (lane == 0 || s0 <= t));
        const int hit = 31 - __clz(below);
        b = lo + hit;
        const int start = __shfl_sync(0xffffffffu, s0, hit);
        n = __shfl_sync(0xffffffffu, s1, hit) - start;
        L = __shfl_sync(0xffffffffu, len, hit);
        i = t - start;
        p.live = t < tend;
    } else {
        L = a.seq_lens[b];
    }
    if (i < 0 || i >= n || L < n || static_cast<long long>(L) > static_cast<long long>(a.max_blocks) * a.BS) return p;
    p.ok = 1;
    p.pos = L - n + i;
    const int lb = static_cast<int>(static_cast<unsigned>(p.pos) / static_cast<unsigned>(a.BS));
    p.slot = p.pos - lb * a.BS;
    p.blk_raw = a.block_tables[static_cast<size_t>(b) * a.max_blocks + lb];
    return p;
}

// Asks for the token-independent inputs of the kernels below before the predecessor ends.
__device__ __forceinline__ void write_prefetch(const WriteArgs& a) {
    const unsigned worker = (blockIdx.x * gridDim.y + blockIdx.y) * blockDim.x + threadIdx.x;
    prefetch_l2(a.seq_lens, static_cast<size_t>(a.B) * 4, worker);
    prefetch_l2(a.block_tables, static_cast<size_t>(a.B) * a.max_blocks * 4, worker);
    if (a.q_start != nullptr) prefetch_l2(a.q_start, static_cast<size_t>(a.B + 1) * 4, worker);
    if (a.half > 0) prefetch_l2(a.freqs, static_cast<size_t>(a.half) * 8, worker);
}

// cos and sin of pos * freq (turns in units of 2^-64, whole turns wrap away).  What is left of
// the nearest quarter turn is within 1/4 of a half-turn, where float32 rounds by 2^-27.
__device__ __forceinline__ float2 turn_of(int pos, int64_t freq) {
    const uint64_t f = static_cast<uint64_t>(pos) * static_cast<uint64_t>(freq);
    const unsigned quarter = static_cast<unsigned>((f + (1ull << 61)) >> 62);
    const int64_t rest = static_cast<int64_t>(f - (static_cast<uint64_t>(quarter) << 62));
    float s, c;
    sincospif(static_cast<float>(rest) * 1.0842021724855044e-19f, &s, &c);  // 2^-63
    const float x = quarter & 1 ? s : c, y = quarter & 1 ? c : s;
    return make_float2(quarter == 1 || quarter == 2 ? -x : x, quarter >= 2 ? -y : y);
}

// T: element type of the rows; Fmt: the 8-bit format, or FmtNone for a cache of T.
template <typename T, typename Fmt>
__global__ void __launch_bounds__(kWriteWarps * 32) kv_write_any_kernel(const WriteArgs a) {
    write_prefetch(a);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    constexpr int kPer = kWriteMaxD / 32;
    __shared__ float2 turn[kWriteMaxD / 2];
    __shared__ float rowbuf[kWriteWarps][kWriteMaxD];
    const int t = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Place p = place_of(a, t);
    if (!p.live) return;  // rows behind the last sequence stay as they are
    const int blk = p.blk(a.NB);
    if (blk < 0 && threadIdx.x == 0 && blockIdx.y == 0) report(a.status, PKV_ERR_DEVICE_BOUNDS);
    for (int j = threadIdx.x; j < a.half; j += blockDim.x) turn[j] = turn_of(p.pos, a.freqs[j]);
    __syncthreads();
    const int rows = a.Hq + 2 * a.Hkv;
    for (int r = blockIdx.y * kWriteWarps + warp; r < rows; r += gridDim.y * kWriteWarps) {
        const bool is_q = r < a.Hq, is_v = r >= a.Hq + a.Hkv;
        const int h = is_q ? r : is_v ? r - a.Hq - a.Hkv : r - a.Hq;
        const T* src = is_q   ? static_cast<const T*>(a.q) + t * a.q_stride
                       : is_v ? static_cast<const T*>(a.v) + t * a.v_stride
                              : static_cast<const T*>(a.k) + t * a.k_stride;
        src += static_cast<size_t>(h) * a.D;
        if (!is_q && blk < 0) continue;
        float x[kPer];
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const int i = lane + 32 * k;
            x[k] = i < a.D ? to_f32(src[i]) : 0.f;
        }
        const T* w = static_cast<const T*>(is_q ? a.q_weight : a.k_weight);
        if (!is_v && w != nullptr) {
            float ss = 0.f;
#pragma unroll
            for (int k = 0; k < kPer; ++k) ss = fmaf(x[k], x[k], ss);
            const float inv = rsqrtf(warp_sum(ss) / static_cast<float>(a.D) + a.eps);
#pragma unroll
            for (int k = 0; k < kPer; ++k) {
                const int i = lane + 32 * k;
                if (i < a.D) x[k] = x[k] * inv * to_f32(w[i]);
            }
        }
        if (!is_v && a.half > 0) {
            __syncwarp();
#pragma unroll
            for (int k = 0; k < kPer; ++k) rowbuf[warp][lane + 32 * k] = x[k];
            __syncwarp();
#pragma unroll
            for (int k = 0; k < kPer; ++k) {
                const int i = lane + 32 * k;
                if (i >= 2 * a.half) continue;
                const int j = a.interleaved ? i >> 1 : (i < a.half ? i : i - a.half);
                const bool second = a.interleaved ? i & 1 : i >= a.half;
                const float other = rowbuf[warp][a.interleaved ? i ^ 1 : (second ? i - a.half : i + a.half)];
                const float2 cs = turn[j];
                x[k] = second ? fmaf(x[k], cs.x, other * cs.y) : fmaf(x[k], cs.x, -other * cs.y);
            }
        }
        if (is_q) {
            T* dst = static_cast<T*>(a.q_out) + (static_cast<size_t>(t) * a.Hq + h) * a.D;
#pragma unroll
            for (int k = 0; k < kPer; ++k) {
                const int i = lane + 32 * k;
                if (i < a.D) dst[i] = from_f32<T>(p.ok ? x[k] : 0.f);
            }
            continue;
        }
        const size_t row = (static_cast<size_t>(blk) * a.Hkv + h) * a.BS + p.slot;
        if constexpr (Fmt::kQuant) {
            float amax = 0.f;
            bool finite = true;
#pragma unroll
            for (int k = 0; k < kPer; ++k) {
                amax = fmaxf(amax, fabsf(x[k]));
                finite = finite && isfinite(x[k]);
            }
            finite = __all_sync(0xffffffffu, finite);
            const float scale = row_scale(warp_max(amax), Fmt::kInvQ);
            const float inv = __frcp_rn(scale);
            uint8_t* dst = static_cast<uint8_t*>(is_v ? a.v_cache : a.k_cache) + row * a.D;
#pragma unroll
            for (int k = 0; k < kPer; ++k) {
                const int i = lane + 32 * k;
                if (i < a.D) dst[i] = finite ? static_cast<uint8_t>(Fmt::encode2(__fmul_rn(x[k], inv), 0.f)) : 0;
            }
            if (lane == 0) {
                (is_v ? a.v_scale : a.k_scale)[row] = finite ? scale : __int_as_float(0x7fffffff);
                if (!finite) report(a.status, PKV_ERR_NONFINITE);
            }
        } else {
            T* dst = static_cast<T*>(is_v ? a.v_cache : a.k_cache) + row * a.D;
#pragma unroll
            for (int k = 0; k < kPer; ++k) {
                const int i = lane + 32 * k;
                if (i < a.D) dst[i] = is_v ? src[i] : from_f32<T>(x[k]);
            }
        }
    }
}

// ------------------------------------------------------------------ vector kernel
// max(|a|, |b|, |c|), NaN if one of them is.
__device__ __forceinline__ float abs_max(float a, float b, float c) {
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// A lane's 8 elements are two runs of 4, A and B, each as two packed pairs of floats.
// The two runs as loaded (bf16: 8 bytes each, float: 16).
template <typename T>
struct Runs;
template <>
struct Runs<__nv_bfloat16> {
    uint2 v[2];
};
template <>
struct Runs<float> {
    float4 v[2];
};
template <typename Run, typename T>
__device__ __forceinline__ void copy_run(Run* to, const T* from) {  // asynchronous
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem_u32(to)), "l"(from), "n"(sizeof(Run)) : "memory");
}
template <typename T>
__device__ __forceinline__ Runs<T> load_runs(const T* p, int gap) {  // run B lies gap elements behind run A
    Runs<T> r;
    using V = std::remove_reference_t<decltype(r.v[0])>;
    r.v[0] = *reinterpret_cast<const V*>(p);
    r.v[1] = *reinterpret_cast<const V*>(p + gap);
    return r;
}
__device__ __forceinline__ void to_floats(const Runs<__nv_bfloat16>& r, float2 (&x)[4]) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        x[2 * k] = make_float2(bf16_lo(r.v[k].x), bf16_hi(r.v[k].x));
        x[2 * k + 1] = make_float2(bf16_lo(r.v[k].y), bf16_hi(r.v[k].y));
    }
}
__device__ __forceinline__ void to_floats(const Runs<float>& r, float2 (&x)[4]) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        x[2 * k] = make_float2(r.v[k].x, r.v[k].y);
        x[2 * k + 1] = make_float2(r.v[k].z, r.v[k].w);
    }
}
__device__ __forceinline__ void store_runs(__nv_bfloat16* p, int gap, const float2 (&x)[4]) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(x[0].x, x[0].y), pack_bf16x2(x[1].x, x[1].y));
    *reinterpret_cast<uint2*>(p + gap) = make_uint2(pack_bf16x2(x[2].x, x[2].y), pack_bf16x2(x[3].x, x[3].y));
}
__device__ __forceinline__ void store_runs(float* p, int gap, const float2 (&x)[4]) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0].x, x[0].y, x[1].x, x[1].y);
    *reinterpret_cast<float4*>(p + gap) = make_float4(x[2].x, x[2].y, x[3].x, x[3].y);
}

// Layout of the vector kernel, from the host.
struct WritePlan {
    int lanes, per;  // lanes a row, rows a pass
    int qpasses, kvpasses;  // passes over a token's query rows, and over its key (or value) rows
    float inv_d;
    int magic;       // lane / lanes = lane * magic >> 16
    int wpt_log2;    // warps per token
    int warps_log2;  // warps per CTA
};

// op over the lanes of a row, for two rows at once (their shuffles overlap).  kLanes: lanes a
// row where that is a power of two, else 0 (l: this lane's index among w.lanes, base: their
// first lane).
template <int kLanes, typename V, typename Op>
__device__ __forceinline__ void row_reduce(V (&x)[2], const WritePlan& w, int l, int base, Op op) {
    if constexpr (kLanes > 0) {
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1)
#pragma unroll
            for (int k = 0; k < 2; ++k) x[k] = op(x[k], __shfl_xor_sync(0xffffffffu, x[k], o));
    } else {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const V y = __shfl_down_sync(0xffffffffu, x[k], o);
                if (l + o < w.lanes) x[k] = op(x[k], y);
            }
#pragma unroll
        for (int k = 0; k < 2; ++k) x[k] = __shfl_sync(0xffffffffu, x[k], base);
    }
}

// Dynamic shared memory of a warp: its ring, its token's cosines and sines, its rows.
template <typename T, int kRot>
struct WriteShared {
    static constexpr bool kRing = kRot != 0;
    static constexpr int kDepth = !kRing || (kRot == 2 && sizeof(T) == 4) ? 1 : 2;
    static constexpr int kRingBytes = kRing ? kDepth * 4 * 32 * 4 * static_cast<int>(sizeof(T)) : 0;
    static constexpr int kTable = kRot == 0 ? 0 : kWriteMaxD / 2;             // float2
    static constexpr int kRows = kRot == 2 ? 2 * (kWriteMaxD + kWriteMaxD / 8) : 0;  // float
    static constexpr int kBytes = kRingBytes + kTable * 8 + kRows * 4;
    static_assert(kBytes % 16 == 0 && kWriteWarps * kBytes <= 48 * 1024, "default limit");
};

// kRot: 0 no rotation, 1 pairs (j, j + half) with half a multiple of 4, 2 such pairs
// with any half, 3 pairs (2j, 2j + 1).
template <typename T, typename Fmt, int kRot, int kLanes>
__global__ void __launch_bounds__(kWriteWarps * 32, kRot == 2 || sizeof(T) == 4 ? 2 : 3)
    kv_write_kernel(const __grid_constant__ WriteArgs a, const __grid_constant__ WritePlan w) {
    write_prefetch(a);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    using Shared = WriteShared<T, kRot>;
    extern __shared__ __align__(16) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int wpt = 1 << w.wpt_log2, tok = warp >> w.wpt_log2;
    const int t = (blockIdx.x << (w.warps_log2 - w.wpt_log2)) + tok;
    const int lanes = kLanes > 0 ? kLanes : w.lanes, per = kLanes > 0 ? 32 / kLanes : w.per;
    const int sub = kLanes > 0 ? lane / kLanes : (lane * w.magic) >> 16, base = sub * lanes, l = lane - base;
    // the lane's elements: at0 .. at0 + 3 and at0 + gap .. + 3; with kRot 1 the second run
    // holds the partners of the first, so that no element has to travel
    const bool turns = kRot == 1 && 4 * l < a.half;
    const int at0 = turns ? 4 * l : 8 * l, gap = turns ? a.half : 4;
    const bool in = t < a.T && sub < per;
    // this warp's passes: first, first + stride, .. of the queries', two at a time, then of the
    // keys' with the values' beside them
    const int stride = wpt * gridDim.y, first = blockIdx.y * wpt + (warp & (wpt - 1));
    const int qpass = w.qpasses, kvpass = w.kvpasses;
    int kv0 = (first - qpass) % stride;
    if (kv0 < 0) kv0 += stride;
    const T* qp = static_cast<const T*>(a.q) + t * a.q_stride + at0;
    const T* kp = static_cast<const T*>(a.k) + t * a.k_stride + at0;
    const T* vp = static_cast<const T*>(a.v) + t * a.v_stride + at0;
    // With a rotation, pairs of rows come through a ring of kDepth pairs per warp, of which a
    // lane reads only what it copied itself: more is in flight than registers would hold (6147
    // tokens of 32 + 8 heads 32.9 -> 29.1 us; four pairs are no faster than two).  Without one
    // (the appends: few pairs a token) the next pair waits in registers (512 tokens of 8 heads
    // 2.5 us, 2.6 with the ring).
    constexpr bool kRing = Shared::kRing;
    constexpr int kDepth = Shared::kDepth;
    using Run = std::remove_reference_t<decltype(Runs<T>().v[0])>;
    uint8_t* mine = smem + warp * Shared::kBytes;
    Run* ring = reinterpret_cast<Run*>(mine) + lane;  // [kDepth][row of the pair][run][lane]
    Runs<T> held[2];
    auto load = [&](int k, int slot, const T* src, int pass, int heads) {
        const int h = pass * per + sub;
        if (!in || h >= heads) return;
        src += h * a.D;
        if constexpr (kRing) {
            copy_run(ring + (slot * 4 + 2 * k) * 32, src);
            copy_run(ring + (slot * 4 + 2 * k + 1) * 32, src + gap);
        } else {
            held[k] = load_runs(src, gap);
        }
    };
    // the pairs: first those of queries, then the keys' passes with the values'
    int lq = first, lkv = kv0, lslot = 0;
    auto load_next = [&]() {
        if constexpr (kRing) {
            if (lq < qpass) {
                load(0, lslot, qp, lq, a.Hq);
                load(1, lslot, qp, lq + stride, a.Hq);
                lq += 2 * stride;
            } else if (lkv < kvpass) {
                load(0, lslot, kp, lkv, a.Hkv);
                load(1, lslot, vp, lkv, a.Hkv);
                lkv += stride;
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        } else {  // selects: with the branches 581 tokens of 8 heads take 3.1 us for 2.7
            const bool is_q = lq < qpass;
            load(0, 0, is_q ? qp : kp, is_q ? lq : lkv, is_q ? a.Hq : a.Hkv);
            load(1, 0, is_q ? qp : vp, is_q ? lq + stride : lkv, is_q ? a.Hq : a.Hkv);
            lkv += is_q ? 0 : stride;
            lq += is_q ? 2 * stride : 0;
        }
        if (++lslot == kDepth) lslot = 0;
    };
#pragma unroll
    for (int k = 0; k < kDepth; ++k) load_next();
    int slot = 0;
    auto take = [&](Runs<T> (&to)[2]) {
        if constexpr (kRing) {
            asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 1) : "memory");
#pragma unroll
            for (int k = 0; k < 4; ++k) to[k >> 1].v[k & 1] = ring[(slot * 4 + k) * 32];
            if (++slot == kDepth) slot = 0;
            __syncwarp();
        } else {
            to[0] = held[0];
            to[1] = held[1];
        }
        load_next();
    };
    // norm weights and frequencies do not wait for the token's place either
    Runs<T> wq, wk;
    if (a.q_weight != nullptr) wq = load_runs(static_cast<const T*>(a.q_weight) + at0, gap);
    if (a.k_weight != nullptr) wk = load_runs(static_cast<const T*>(a.k_weight) + at0, gap);
    Place p{0, 0, 0, 0, -1};
    if (t < a.T) p = place_of(a, t);
    const bool active = p.live;  // the rows behind the last sequence stay
    // cosines and sines: of the run's 4 pairs (kRot 1, 3), or of the 8 elements, the sine with
    // the sign it enters with (kRot 2)
    float2 cs[kRot == 2 ? 4 : 2], sn[kRot == 2 ? 4 : 2];
    if constexpr (kRot != 0) {
        // of the token's first warp
        float2* tt = reinterpret_cast<float2*>(smem + (tok << w.wpt_log2) * Shared::kBytes + Shared::kRingBytes);
        if (active)
            for (int j = (warp & (wpt - 1)) * 32 + lane; j < a.half; j += wpt * 32) tt[j] = turn_of(p.pos, a.freqs[j]);
        __syncthreads();
        if constexpr (kRot == 2) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int i = 8 * l + e;
                const float2 v = i < 2 * a.half ? tt[i < a.half ? i : i - a.half] : make_float2(1.f, 0.f);
                (e & 1 ? cs[e >> 1].y : cs[e >> 1].x) = v.x;
                (e & 1 ? sn[e >> 1].y : sn[e >> 1].x) = i < a.half ? -v.y : v.y;
            }
        } else if (4 * l < a.half) {  // entries behind half are unused
            const float4* row = reinterpret_cast<const float4*>(tt + 4 * l);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float4 v = row[e];
                cs[e] = make_float2(v.x, v.z);
                sn[e] = make_float2(v.y, v.w);
            }
        }
    }
    // no copy outlives its CTA
    auto settle = [] { if constexpr (kRing) asm volatile("cp.async.wait_all;" ::: "memory"); };
    if (!active) return settle();
    if (!p.ok) {  // a bad length or chunk: zero queries, no append
        const float2 zero[4] = {};
        T* qo = static_cast<T*>(a.q_out) + static_cast<size_t>(t) * a.Hq * a.D + at0;
        for (int pass = first; pass < qpass; pass += stride)
            if (in && pass * per + sub < a.Hq) store_runs(qo + (pass * per + sub) * a.D, gap, zero);
        if (first == 0 && lane == 0) report(a.status, PKV_ERR_DEVICE_BOUNDS);
        return settle();
    }

    auto square = [](const float2 (&x)[4]) {
        float2 s2 = mul2(x[0], x[0]);
#pragma unroll
        for (int e = 1; e < 4; ++e) s2 = fma2(x[e], x[e], s2);
        return s2.x + s2.y;
    };
    auto scaled = [&](float2 (&x)[4], float ss, const float2 (&g)[4]) {
        const float inv = rsqrtf(fmaf(ss, w.inv_d, a.eps));
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = mul2(mul2(x[e], make_float2(inv, inv)), g[e]);
    };
    auto sum = [](float u, float v) { return u + v; };
    auto rotate = [&](float2 (&x)[4]) {
        if constexpr (kRot == 1) {
            if (turns) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float2 u = x[e], v = x[2 + e];
                    x[e] = fma2(u, cs[e], mul2(v, make_float2(-sn[e].x, -sn[e].y)));
                    x[2 + e] = fma2(v, cs[e], mul2(u, sn[e]));
                }
            }
        } else if constexpr (kRot == 3) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float c = e & 1 ? cs[e >> 1].y : cs[e >> 1].x, s = e & 1 ? sn[e >> 1].y : sn[e >> 1].x;
                const float2 v = x[e];
                if (4 * l + e < a.half) x[e] = make_float2(fmaf(v.x, c, -v.y * s), fmaf(v.y, c, v.x * s));
            }
        } else if constexpr (kRot == 2) {
            // rows through shared memory, one word of padding per 8
            float* buf = reinterpret_cast<float*>(mine + Shared::kRingBytes + Shared::kTable * 8);
            const int at = sub * (a.D + a.D / 8);
            __syncwarp();
            if (sub < per) {
#pragma unroll
                for (int e = 0; e < 8; ++e) buf[at + 9 * l + e] = e & 1 ? x[e >> 1].y : x[e >> 1].x;
            }
            __syncwarp();
            if (sub < per) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int i = 8 * l + e, q = i < a.half ? i + a.half : i - a.half;
                    if (i < 2 * a.half) {
                        const float o = buf[at + q + (q >> 3)];
                        float& y = e & 1 ? x[e >> 1].y : x[e >> 1].x;
                        y = fmaf(y, e & 1 ? cs[e >> 1].y : cs[e >> 1].x, o * (e & 1 ? sn[e >> 1].y : sn[e >> 1].x));
                    }
                }
            }
        }
    };
    {  // queries
        float2 g[4];
        if (a.q_weight != nullptr) to_floats(wq, g);
        T* qo = static_cast<T*>(a.q_out) + static_cast<size_t>(t) * a.Hq * a.D + at0;
        for (int pass = first; pass < qpass; pass += 2 * stride) {
            Runs<T> raw[2];
            take(raw);
            float2 x[2][4];
            float ss[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                to_floats(raw[k], x[k]);
                ss[k] = square(x[k]);
            }
            if (a.q_weight != nullptr) {
                row_reduce<kLanes>(ss, w, l, base, sum);
#pragma unroll
                for (int k = 0; k < 2; ++k) scaled(x[k], ss[k], g);
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                rotate(x[k]);
                const int h = (pass + k * stride) * per + sub;
                if (in && h < a.Hq) store_runs(qo + h * a.D, gap, x[k]);
            }
        }
    }
    const int blk = p.blk(a.NB);
    if (blk < 0) {
        if (first == 0 && lane == 0) report(a.status, PKV_ERR_DEVICE_BOUNDS);
        return settle();
    }
    const size_t slot0 = static_cast<size_t>(blk) * a.Hkv * a.BS + p.slot;  // cache row of KV head 0
    float2 g[4];
    if (a.k_weight != nullptr) to_floats(wk, g);
    for (int pass = kv0; pass < kvpass; pass += stride) {  // x[0]: a key row, x[1]: the value row
        float2 x[2][4];
        Runs<T> raw[2];
        take(raw);
#pragma unroll
        for (int k = 0; k < 2; ++k) to_floats(raw[k], x[k]);
        if (a.k_weight != nullptr) {
            float ss[2] = {square(x[0]), 0.f};
            row_reduce<kLanes>(ss, w, l, base, sum);
            scaled(x[0], ss[0], g);
        }
        rotate(x[0]);
        const int h = pass * per + sub;
        const bool store = in && h < a.Hkv;
        const size_t row = slot0 + static_cast<size_t>(h) * a.BS, at = row * a.D + at0;
        if constexpr (Fmt::kQuant) {
            float top[2];  // the largest |x|, NaN if there is one
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                top[k] = abs_max(0.f, x[k][0].x, x[k][0].y);
#pragma unroll
                for (int e = 1; e < 4; ++e) top[k] = abs_max(top[k], x[k][e].x, x[k][e].y);
            }
            row_reduce<kLanes>(top, w, l, base, [](float u, float v) { return abs_max(u, u, v); });
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const bool finite = top[k] < INFINITY;
                const float scale = row_scale(top[k], Fmt::kInvQ);
                const float inv = __frcp_rn(scale);
                uint32_t v0 = 0, v1 = 0;
#pragma unroll
                for (int e = 0; e < 4; ++e) x[k][e] = mul2(x[k][e], make_float2(inv, inv));
                if (finite) {
                    v0 = Fmt::encode4(&x[k][0].x);
                    v1 = Fmt::encode4(&x[k][2].x);
                }
                if (store) {
                    uint8_t* dst = static_cast<uint8_t*>(k ? a.v_cache : a.k_cache) + at;
                    *reinterpret_cast<uint32_t*>(dst) = v0;
                    *reinterpret_cast<uint32_t*>(dst + gap) = v1;
                    if (l == 0) {
                        (k ? a.v_scale : a.k_scale)[row] = finite ? scale : __int_as_float(0x7fffffff);
                        if (!finite) report(a.status, PKV_ERR_NONFINITE);
                    }
                }
            }
        } else if (store) {
            store_runs(static_cast<T*>(a.k_cache) + at, gap, x[0]);
            T* dst = static_cast<T*>(a.v_cache) + at;  // the bits as they are
            *reinterpret_cast<Run*>(dst) = raw[1].v[0];
            *reinterpret_cast<Run*>(dst + gap) = raw[1].v[1];
        }
    }
}

template <typename T, typename Fmt>
static cudaError_t launch_typed(const WriteArgs& a, cudaStream_t stream) {
    const int rows = a.Hq + 2 * a.Hkv, sms = device_sm_count();
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kWriteWarps * 32, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    uintptr_t at = 0;  // every address a lane's 8 elements start from
    for (const void* x : {static_cast<const void*>(a.q_out), a.q, a.k, a.v, a.q_weight, a.k_weight,
                          static_cast<const void*>(a.k_cache), static_cast<const void*>(a.v_cache)})
        at |= reinterpret_cast<uintptr_t>(x);
    const long long es = sizeof(T);
    const bool vec = a.D % 8 == 0 && at % 16 == 0 && ((a.q ? a.q_stride : 0) * es) % 16 == 0 &&
                     (a.k_stride * es) % 16 == 0 && (a.v_stride * es) % 16 == 0;
    cudaError_t err;
    if (vec) {
        WritePlan w;
        w.lanes = a.D / 8;
        w.per = 32 / w.lanes;
        w.magic = 65536 / w.lanes + 1;  // exact for lane < 32, lanes <= 32
        w.qpasses = (a.Hq + w.per - 1) / w.per;
        w.kvpasses = (a.Hkv + w.per - 1) / w.per;
        w.inv_d = 1.0f / static_cast<float>(a.D);
        const int passes = (w.qpasses + 1) / 2 + w.kvpasses;  // pairs of passes
        // Many tokens: a warp takes many passes of one token, which shares the token's place,
        // angles and weights, and a CTA several tokens; fewer warps a token only where more of
        // them would not all be resident, eight only up to half of that.  32 + 8 heads x 128 in
        // bf16: 5226 tokens 24.3 us with a warp a token, 26.1 with two; 1227: 8.9 with one, 7.5
        // with two; 581: 4.9 with two, 4.3 with four; 254: 3.4 with four, 3.8 with eight.
        w.wpt_log2 = 3;
        int split = 1;
        while (w.wpt_log2 > 0 && passes < kPairsPerWarp << w.wpt_log2 &&
               (static_cast<long long>(a.T) << w.wpt_log2) >= (w.wpt_log2 == 3 ? 12LL : 24LL) * sms)
            --w.wpt_log2;
        // few: a pass per warp, over as many CTAs as that takes and the SMs hold 1.5 of each
        // (39 tokens 2.95 -> 2.69 us; two CTAs for 117 tokens 3.0 -> 3.6)
        if (w.wpt_log2 == 3)
            split = std::max(1, std::min((w.qpasses + w.kvpasses + kWriteWarps - 1) / kWriteWarps, 3 * sms / 2 / a.T));
        w.warps_log2 = std::max(w.wpt_log2, 2);  // small CTAs: less to wait for at the end (6147 tokens 29.3 -> 27.2 us)
        cfg.blockDim = dim3(32u << w.warps_log2, 1, 1);
        const int tpc = 1 << (w.warps_log2 - w.wpt_log2);
        cfg.gridDim = dim3(static_cast<unsigned>((static_cast<long long>(a.T) + tpc - 1) / tpc), static_cast<unsigned>(split), 1);
        const int rot = a.half == 0 ? 0 : a.interleaved ? 3 : a.half % 4 == 0 ? 1 : 2;
        auto pick = [&](auto lanes) {
            constexpr int kLanes = decltype(lanes)::value;
            if (rot == 0) return kv_write_kernel<T, Fmt, 0, kLanes>;
            if (rot == 1) return kv_write_kernel<T, Fmt, 1, kLanes>;
            return kv_write_kernel<T, Fmt, 3, kLanes>;
        };
        auto kern = rot == 2         ? kv_write_kernel<T, Fmt, 2, 0>
                    : w.lanes == 16 ? pick(std::integral_constant<int, 16>())
                    : w.lanes == 8  ? pick(std::integral_constant<int, 8>())
                                    : pick(std::integral_constant<int, 0>());
        const int warp_bytes = rot == 0   ? WriteShared<T, 0>::kBytes
                               : rot == 2 ? WriteShared<T, 2>::kBytes
                                          : WriteShared<T, 1>::kBytes;  // and 3
        // CTAs that are all resident at once are not dealt evenly over the SMs (660 CTAs, 4.3 an SM:
        // some get 6).  Shared memory that leaves room for just ceil of the mean evens them out:
        // 2641 tokens of 32 + 8 heads 15.2 -> 13.6 us, 953 8.1 -> 6.4.  Below 4 an SM that would
        // take more than the 48 KB a kernel has by default.
        const int per_sm = static_cast<int>((static_cast<long long>(cfg.gridDim.x) * split + sms - 1) / sms);
        const int even = per_sm >= 4 ? std::min((kSmShared / per_sm - 1024) / 128 * 128, 48 * 1024) : 0;
        cfg.dynamicSmemBytes = std::max((warp_bytes << w.warps_log2), even);
        err = cudaLaunchKernelEx(&cfg, kern, a, w);
    } else {
        // few tokens: a token's rows over several CTAs
        const unsigned split = a.T < 2 * sms ? static_cast<unsigned>((rows + kWriteWarps - 1) / kWriteWarps) : 1u;
        cfg.gridDim = dim3(static_cast<unsigned>(a.T), split, 1);
        err = cudaLaunchKernelEx(&cfg, kv_write_any_kernel<T, Fmt>, a);
    }
    return err != cudaSuccess ? err : cudaGetLastError();
}

cudaError_t launch_kv_write(const WriteArgs& a, pkv_dtype dtype, pkv_dtype cache_dtype, cudaStream_t stream) {
    if (dtype == PKV_F32) {
        if (cache_dtype == PKV_E4M3) return launch_typed<float, FmtE4M3>(a, stream);
        if (cache_dtype == PKV_I8) return launch_typed<float, FmtI8>(a, stream);
        return launch_typed<float, FmtNone>(a, stream);
    }
    if (cache_dtype == PKV_E4M3) return launch_typed<__nv_bfloat16, FmtE4M3>(a, stream);
    if (cache_dtype == PKV_I8) return launch_typed<__nv_bfloat16, FmtI8>(a, stream);
    return launch_typed<__nv_bfloat16, FmtNone>(a, stream);
}

}  // namespace pkv

namespace {
bool is8(pkv_dtype d) { return d == PKV_E4M3 || d == PKV_I8; }
bool plain(pkv_dtype d) { return d == PKV_F32 || d == PKV_BF16; }
pkv_status status_of(cudaError_t e) { return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA; }
}  // namespace

extern "C" pkv_status pkv_kv_append_q8(const void* k_new, const void* v_new, void* k_cache, void* v_cache,
                                       float* k_scale, float* v_scale, const int32_t* block_tables,
                                       int max_blocks_per_seq, const int32_t* seq_lens, const int32_t* q_start, int B,
                                       int T_new, int Hkv, int D, int block_size, int num_blocks, pkv_dtype dtype,
                                       pkv_dtype cache_dtype, int32_t* dev_status, void* stream) {
    if (B < 0 || T_new < 0 || Hkv < 1 || D < 1 || D > pkv::kWriteMaxD || block_size < 1 || num_blocks < 1 ||
        max_blocks_per_seq < 1 || !plain(dtype) || !is8(cache_dtype) || (!q_start && T_new != B) ||
        static_cast<long long>(Hkv) * D > 0x7fffffffLL)
        return PKV_ERR_INVALID_ARG;
    if (B == 0 || T_new == 0) return PKV_OK;
    if (!k_new || !v_new || !k_cache || !v_cache || !k_scale || !v_scale || !block_tables || !seq_lens)
        return PKV_ERR_INVALID_ARG;
    pkv::WriteArgs a = {};
    a.k = k_new;
    a.v = v_new;
    a.k_stride = a.v_stride = static_cast<long long>(Hkv) * D;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    a.block_tables = block_tables;
    a.seq_lens = seq_lens;
    a.q_start = q_start;
    a.max_blocks = max_blocks_per_seq;
    a.B = B;
    a.T = T_new;
    a.Hkv = Hkv;
    a.D = D;
    a.BS = block_size;
    a.NB = num_blocks;
    a.status = dev_status;
    return status_of(pkv::launch_kv_write(a, dtype, cache_dtype, static_cast<cudaStream_t>(stream)));
}

extern "C" pkv_status pkv_qk_norm_rope_append(
    void* q_out, const void* q, int64_t q_stride, const void* k_new, int64_t k_stride, const void* v_new,
    int64_t v_stride, const void* q_weight, const void* k_weight, float eps, const int64_t* freqs, int rot_dim,
    int interleaved, void* k_cache, void* v_cache, float* k_scale, float* v_scale, const int32_t* block_tables,
    int max_blocks_per_seq, const int32_t* seq_lens, const int32_t* q_start, int B, int T_new, int Hq, int Hkv, int D,
    int block_size, int num_blocks, pkv_dtype dtype, pkv_dtype cache_dtype, int32_t* dev_status, void* stream) {
    if (B < 0 || T_new < 0 || Hq < 1 || Hkv < 1 || D < 1 || D > pkv::kWriteMaxD || block_size < 1 || num_blocks < 1 ||
        max_blocks_per_seq < 1 || !plain(dtype) || (!is8(cache_dtype) && cache_dtype != dtype) ||
        (!q_start && T_new != B) || rot_dim < 0 || rot_dim > D || rot_dim % 2 != 0 || !(eps >= 0.f))
        return PKV_ERR_INVALID_ARG;
    const long long qrow = static_cast<long long>(Hq) * D, kvrow = static_cast<long long>(Hkv) * D;
    if (q_stride < qrow || k_stride < kvrow || v_stride < kvrow || qrow > 0x7fffffffLL || kvrow > 0x7fffffffLL)
        return PKV_ERR_INVALID_ARG;
    if (B == 0 || T_new == 0) return PKV_OK;
    if (!q_out || !q || !k_new || !v_new || !k_cache || !v_cache || !block_tables || !seq_lens ||
        (rot_dim > 0 && !freqs) || (is8(cache_dtype) && (!k_scale || !v_scale)))
        return PKV_ERR_INVALID_ARG;
    pkv::WriteArgs a = {};
    a.q_out = q_out;
    a.q = q;
    a.k = k_new;
    a.v = v_new;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.q_weight = q_weight;
    a.k_weight = k_weight;
    a.eps = eps;
    a.freqs = freqs;
    a.half = rot_dim / 2;
    a.interleaved = interleaved != 0;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    a.block_tables = block_tables;
    a.seq_lens = seq_lens;
    a.q_start = q_start;
    a.max_blocks = max_blocks_per_seq;
    a.B = B;
    a.T = T_new;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.D = D;
    a.BS = block_size;
    a.NB = num_blocks;
    a.status = dev_status;
    return status_of(pkv::launch_kv_write(a, dtype, cache_dtype, static_cast<cudaStream_t>(stream)));
}
