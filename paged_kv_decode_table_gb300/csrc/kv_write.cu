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
// (a 64-bit integer): pos * f wraps modulo one turn in integer arithmetic, so
// the angle keeps its full precision at any position, and sincospif needs no
// range reduction.
//
// One warp per row.
#include "quant8.cuh"

namespace pkv {

constexpr int kWriteWarps = 8;
constexpr int kWriteMaxD = 256;

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

// Where token t goes.  ok: the sequence's length and chunk are valid (pos is
// set); blk < 0: no valid block for that position.
struct Place {
    int ok, pos, blk, slot;
};

__device__ __forceinline__ Place place_of(const WriteArgs& a, int t) {
    Place p{0, 0, -1, 0};
    int b = t, n = 1, i = 0;
    if (a.q_start != nullptr) {
        int lo = 0, hi = a.B - 1;  // the last b with q_start[b] <= t
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (a.q_start[mid] <= t) lo = mid; else hi = mid - 1;
        }
        b = lo;
        n = a.q_start[b + 1] - a.q_start[b];
        i = t - a.q_start[b];
    }
    const int L = a.seq_lens[b];
    if (i < 0 || i >= n || L < n || static_cast<long long>(L) > static_cast<long long>(a.max_blocks) * a.BS) return p;
    p.ok = 1;
    p.pos = L - n + i;
    p.slot = p.pos % a.BS;
    const int blk = a.block_tables[static_cast<size_t>(b) * a.max_blocks + p.pos / a.BS];
    p.blk = blk >= 0 && blk < a.NB ? blk : -1;
    return p;
}

// T: element type of the rows; Fmt: the 8-bit format, or FmtNone for a cache of T.
template <typename T, typename Fmt>
__global__ void __launch_bounds__(kWriteWarps * 32) kv_write_kernel(const WriteArgs a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    constexpr int kPer = kWriteMaxD / 32;
    __shared__ float2 turn[kWriteMaxD / 2];
    __shared__ float rowbuf[kWriteWarps][kWriteMaxD];
    const int t = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (a.q_start != nullptr && t >= a.q_start[a.B]) return;  // rows behind the last sequence stay as they are
    const Place p = place_of(a, t);
    if ((!p.ok || p.blk < 0) && threadIdx.x == 0 && blockIdx.y == 0) report(a.status, PKV_ERR_DEVICE_BOUNDS);
    for (int j = threadIdx.x; j < a.half; j += blockDim.x) {
        const uint64_t f = static_cast<uint64_t>(p.pos) * static_cast<uint64_t>(a.freqs[j]);
        float s, c;
        sincospif(static_cast<float>(static_cast<int64_t>(f)) * 1.0842021724855044e-19f, &s, &c);  // 2^-63
        turn[j] = make_float2(c, s);
    }
    __syncthreads();
    const int rows = a.Hq + 2 * a.Hkv;
    for (int r = blockIdx.y * kWriteWarps + warp; r < rows; r += gridDim.y * kWriteWarps) {
        const bool is_q = r < a.Hq, is_v = r >= a.Hq + a.Hkv;
        const int h = is_q ? r : is_v ? r - a.Hq - a.Hkv : r - a.Hq;
        const T* src = is_q   ? static_cast<const T*>(a.q) + t * a.q_stride
                       : is_v ? static_cast<const T*>(a.v) + t * a.v_stride
                              : static_cast<const T*>(a.k) + t * a.k_stride;
        src += static_cast<size_t>(h) * a.D;
        if (!is_q && p.blk < 0) continue;
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
        const size_t row = (static_cast<size_t>(p.blk) * a.Hkv + h) * a.BS + p.slot;
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
                if (i < a.D) dst[i] = from_f32<T>(x[k]);
            }
        }
    }
}

template <typename T, typename Fmt>
static cudaError_t launch_typed(const WriteArgs& a, cudaStream_t stream) {
    const int rows = a.Hq + 2 * a.Hkv;
    // few tokens: a token's rows over several CTAs
    const unsigned split = a.T < 2 * device_sm_count() ? static_cast<unsigned>((rows + kWriteWarps - 1) / kWriteWarps) : 1u;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.T), split, 1);
    cfg.blockDim = dim3(kWriteWarps * 32, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t err = cudaLaunchKernelEx(&cfg, kv_write_kernel<T, Fmt>, a);
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
        max_blocks_per_seq < 1 || !plain(dtype) || !is8(cache_dtype) || (!q_start && T_new != B))
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
    if (q_stride < qrow || k_stride < kvrow || v_stride < kvrow) return PKV_ERR_INVALID_ARG;
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
