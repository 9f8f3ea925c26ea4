// decode_attention_scored.cu -- GQA paged decode attention with capped, biased and windowed scores
// (attention_scores.cuh has the definition), one query token per sequence.
//
// Generic kernel: one CTA per (sequence, KV head, up to 8 of its query heads, share of the visible
// positions).  Tiles of 32 visible positions come to shared memory as float32; warp w takes the 32
// scores of query head w (a lane a position) and their running maximum and sum, then a thread takes
// four dimensions of one head's output.  Positions that the mask hides are never loaded.  The shares'
// results are joined by a second kernel.
#include <cuda.h>
#include <math.h>

#include <algorithm>

#include "attention_scores.cuh"

namespace pkv {

int device_sm_count();
int max_optin_smem();

// ------------------------------------------------------------------ generic kernel
constexpr int kGenThreads = 256;
constexpr int kGenPos = 32;    // positions a tile
constexpr int kGenHeads = 8;   // query heads a CTA
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

template <typename T, bool kVec>
__global__ void __launch_bounds__(kGenThreads)
    decode_scored_generic_kernel(const __grid_constant__ GenericPlan pl, T* out, const T* q, const T* k_cache,
                                 const T* v_cache, const int32_t* block_tables, const int32_t* seq_lens, float* part,
                                 int32_t* status) {
    extern __shared__ __align__(16) float gen_smem[];
    __shared__ float ps[kGenHeads][kGenPos], factor[kGenHeads];
    __shared__ long long rows[2][kGenPos];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, D = pl.D, DS = pl.stride;
    float* ks = gen_smem;
    float* vs = ks + kGenPos * DS;
    float* qs = vs + kGenPos * DS;
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
    const int per = (tiles + pl.shares - 1) / pl.shares, t0 = share * per, t1 = min(tiles, t0 + per);
    // the dimensions between D and the next multiple of 4 are zeros
    for (int e = tid; e < kGenHeads * DS; e += kGenThreads) {
        const int hd = e / DS, d = e - hd * DS;
        qs[e] = hd < nh && d < D ? to_f32(q[(row0 + hd) * D + d]) : 0.f;
    }
    if ((D & 3) != 0)
        for (int e = tid; e < 2 * kGenPos * DS; e += kGenThreads) ks[e] = 0.f;
    bool miss = false;
    auto locate = [&](int t) {  // warp 0: the rows of tile t's positions
        const int i = t * kGenPos + lane;
        long long row = -1;
        if (i < visible) {
            const int pos = i < seen.pfx ? i : seen.lo + (i - seen.pfx);
            const int blk = block_tables[static_cast<size_t>(b) * pl.max_blocks + pos / pl.BS];
            if (blk < 0 || blk >= pl.NB) miss = true;
            else row = (static_cast<long long>(blk) * pl.Hkv + h) * pl.BS + pos % pl.BS;
        }
        rows[t & 1][lane] = row;
    };
    const int quads = (D + 3) / 4;
    float m = -INFINITY, l = 0.f;  // of head `warp`
    float4 acc[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
    const float slope = pl.sc.slopes != nullptr && warp < nh
                            ? pl.sc.slopes[h * pl.G + chunk * kGenHeads + warp] * kLog2e : 0.f;
    if (warp == 0 && t0 < t1) locate(t0);
    for (int t = t0; t < t1; ++t) {
        bad = __syncthreads_or(miss) != 0;  // the rows are there, the last tile is used
        if (bad) break;
        if (warp == 0 && t + 1 < t1) locate(t + 1);
        const int n = min(kGenPos, visible - t * kGenPos);
        if constexpr (kVec) {
            constexpr int kPer = 16 / static_cast<int>(sizeof(T));
            const int vecs = D / kPer;
            for (int e = tid; e < 2 * n * vecs; e += kGenThreads) {
                const int which = e >= n * vecs, x = e - which * n * vecs, p = x / vecs, c = x - p * vecs;
                const uint4 z = *reinterpret_cast<const uint4*>((which ? v_cache : k_cache) + rows[t & 1][p] * D + c * kPer);
                float4* to = reinterpret_cast<float4*>((which ? vs : ks) + p * DS + c * kPer);
                if constexpr (sizeof(T) == 4) {
                    to[0] = make_float4(__uint_as_float(z.x), __uint_as_float(z.y), __uint_as_float(z.z), __uint_as_float(z.w));
                } else {
                    to[0] = make_float4(bf16_lo(z.x), bf16_hi(z.x), bf16_lo(z.y), bf16_hi(z.y));
                    to[1] = make_float4(bf16_lo(z.z), bf16_hi(z.z), bf16_lo(z.w), bf16_hi(z.w));
                }
            }
        } else {
            for (int p = warp; p < n; p += kGenThreads / 32) {
                const T *kr = k_cache + rows[t & 1][p] * D, *vr = v_cache + rows[t & 1][p] * D;
                for (int d = lane; d < D; d += 32) {
                    ks[p * DS + d] = to_f32(kr[d]);
                    vs[p * DS + d] = to_f32(vr[d]);
                }
            }
        }
        __syncthreads();
        if (warp < nh) {
            float x = -INFINITY;
            if (lane < n) {
                const int i = t * kGenPos + lane, pos = i < seen.pfx ? i : seen.lo + (i - seen.pfx);
                const float4 *kr = reinterpret_cast<const float4*>(ks + lane * DS),
                             *qr = reinterpret_cast<const float4*>(qs + warp * DS);
                float s0 = 0.f, s1 = 0.f;
                for (int c = 0; c < quads; ++c) {
                    const float4 a = kr[c], w = qr[c];
                    s0 = fmaf(a.x, w.x, fmaf(a.y, w.y, s0));
                    s1 = fmaf(a.z, w.z, fmaf(a.w, w.w, s1));
                }
                x = s0 + s1;
                x = pl.sc.cap_log2 > 0.f ? pl.sc.cap_log2 * tanhf(x * pl.sc.in) : x * pl.sc.mul;
                x = fmaf(slope, static_cast<float>(pos - (L - 1)), x);
            }
            float mx = x;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            const float mn = fmaxf(m, mx), mu = mn == -INFINITY ? 0.f : mn;
            const float p = lane < n ? exp2f(x - mu) : 0.f, f = exp2f(m - mu);
            float sum = p;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            l = fmaf(l, f, sum);
            m = mn;
            ps[warp][lane] = p;
            if (lane == 0) factor[warp] = f;
        }
        __syncthreads();
#pragma unroll
        for (int a = 0; a < 2; ++a) {
            const int x = tid + a * kGenThreads, hd = x / quads, c = x - hd * quads;
            if (hd >= nh) continue;
            const float f = factor[hd];
            float4 o = make_float4(acc[a].x * f, acc[a].y * f, acc[a].z * f, acc[a].w * f);
            const float* v = vs + 4 * c;
            for (int p = 0; p < n; ++p) {
                const float w = ps[hd][p];
                const float4 z = *reinterpret_cast<const float4*>(v + p * DS);
                o.x = fmaf(w, z.x, o.x);
                o.y = fmaf(w, z.y, o.y);
                o.z = fmaf(w, z.z, o.z);
                o.w = fmaf(w, z.w, o.w);
            }
            acc[a] = o;
        }
    }
    if (bad && tid == 0) report(status, PKV_ERR_DEVICE_BOUNDS);
    __syncthreads();
    if (warp < nh && lane == 0) {
        ps[warp][0] = m;
        ps[warp][1] = bad ? -1.f : l;  // a share that cannot be read makes the row zero
    }
    __syncthreads();
    // a share's row: maximum, sum, D sums of products
    const int DR = 2 + 4 * quads;
#pragma unroll
    for (int a = 0; a < 2; ++a) {
        const int x = tid + a * kGenThreads, hd = x / quads, c = x - hd * quads;
        if (hd >= nh) continue;
        const float o[4] = {acc[a].x, acc[a].y, acc[a].z, acc[a].w};
        const float sum = ps[hd][1];
        if (pl.shares == 1) {
            const float inv = sum > 0.f || sum != sum ? 1.f / sum : 0.f;
            for (int i = 0; i < 4; ++i)
                if (4 * c + i < D) out[(row0 + hd) * D + 4 * c + i] = from_f32<T>(sum > 0.f || sum != sum ? o[i] * inv : 0.f);
        } else {
            float* to = part + ((row0 + hd) * pl.shares + share) * DR;
            if (c == 0) *reinterpret_cast<float2*>(to) = make_float2(ps[hd][0], sum);
            for (int i = 0; i < 2; ++i) *reinterpret_cast<float2*>(to + 2 + 4 * c + 2 * i) = make_float2(o[2 * i], o[2 * i + 1]);
        }
    }
}

// out = sum o_s 2^(m_s - M) / sum l_s 2^(m_s - M) over a row's shares; a warp a row.
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
    float M = -INFINITY, l = 0.f, acc[8] = {};
    bool bad = false;
    for (int s = 0; s < shares; ++s) M = fmaxf(M, __ldcg(p + s * DR));
    const float mu = M == -INFINITY ? 0.f : M;
    for (int s = 0; s < shares; ++s) {
        const float2 ml = __ldcg(reinterpret_cast<const float2*>(p + s * DR));
        const float w = exp2f(ml.x - mu);
        bad = bad || ml.y < 0.f;
        l = fmaf(ml.y, w, l);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (lane + 32 * i < D) acc[i] = fmaf(__ldcg(p + s * DR + 2 + lane + 32 * i), w, acc[i]);
    }
    const float inv = l != 0.f ? 1.f / l : 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (lane + 32 * i < D) out[row * D + lane + 32 * i] = from_f32<T>(bad || l == 0.f ? 0.f : acc[i] * inv);
}

// CTAs along the positions: four per SM in all where the batch has fewer, and not more than the longest
// sequence (by the table's width, or the window) has tiles.
static int generic_shares(long long units, int longest, int P) {
    const long long want = (4LL * P + units - 1) / units, tiles = (static_cast<long long>(longest) + kGenPos - 1) / kGenPos;
    return static_cast<int>(std::max(1LL, std::min({want, tiles, static_cast<long long>(kGenShares)})));
}

static size_t generic_workspace(int B, int Hq, int Hkv, int D, int P) {
    const long long units = static_cast<long long>(B) * Hkv * ((Hq / Hkv + kGenHeads - 1) / kGenHeads);
    const int shares = generic_shares(std::max(1LL, units), 0x7fffffff, P);
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
    pl.shares = generic_shares(units, static_cast<int>(windowed ? std::min<long long>(width, pl.sc.window) : width), P);
    const size_t smem = (2 * kGenPos + kGenHeads) * static_cast<size_t>(pl.stride) * sizeof(float);
    auto kern = vec ? decode_scored_generic_kernel<T, true> : decode_scored_generic_kernel<T, false>;
    // the limit belongs to the kernel, not to the call: always the same value
    constexpr int kMost = (2 * kGenPos + kGenHeads) * (256 + 4) * 4;
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
size_t decode_scored_workspace_bytes(int B, int Hq, int Hkv, int D, int P) {
    return std::max<size_t>(256, generic_workspace(B, Hq, Hkv, D, P));
}

// Arguments checked; B > 0.
cudaError_t launch_decode_scored(void* out, const void* q, const void* k, const void* v, const int32_t* block_tables,
                                 int max_blocks, const int32_t* seq_lens, int B, int Hq, int Hkv, int D, int BS, int NB,
                                 const ScoreArgs& sc, pkv_dtype dtype, void* workspace, int P, int32_t* status,
                                 cudaStream_t stream) {
    GenericPlan pl = {};
    pl.B = B;
    pl.Hq = Hq;
    pl.Hkv = Hkv;
    pl.G = Hq / Hkv;
    pl.D = D;
    pl.BS = BS;
    pl.NB = NB;
    pl.max_blocks = max_blocks;
    pl.sc = sc;
    return (dtype == PKV_F32 ? launch_generic<float> : launch_generic<__nv_bfloat16>)(
        pl, out, q, k, v, block_tables, seq_lens, workspace, P, status, stream);
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
    if (!out || !q || !k_cache || !v_cache || !block_tables || !seq_lens || !workspace ||
        (reinterpret_cast<uintptr_t>(workspace) & 15u) != 0)
        return PKV_ERR_INVALID_ARG;
    const int P = device_sm_count();
    if (workspace_bytes < pkv_decode_scored_workspace_bytes(B, Hq, Hkv, D, P > 0 ? P : 1)) return PKV_ERR_INVALID_ARG;
    if (P <= 0) return PKV_ERR_CUDA;
    const cudaError_t err =
        launch_decode_scored(out, q, k_cache, v_cache, block_tables, max_blocks_per_seq, seq_lens, B, Hq, Hkv, D,
                             block_size, num_blocks, sc, dtype, workspace, P, dev_status, static_cast<cudaStream_t>(stream));
    return err == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

extern "C" size_t pkv_decode_shared_workspace_bytes(int B, int Hq, int Hkv, int D, int num_sms) {
    return pkv_decode_scored_workspace_bytes(B, Hq, Hkv, D, num_sms);
}

extern "C" pkv_status pkv_paged_decode_attention_shared(
    void* out, const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
    int max_blocks_per_seq, const int32_t* seq_lens, const int32_t* group_start, const int32_t* shared_lens, int N,
    int B, int Hq, int Hkv, int D, int block_size, int num_blocks, float scale, float softcap, const float* slopes,
    pkv_dtype dtype, void* workspace, size_t workspace_bytes, int32_t* dev_status, void* stream) {
    if (N < 0 || N > B || (N > 0 && (!group_start || !shared_lens))) return PKV_ERR_INVALID_ARG;
    return pkv_paged_decode_attention_scored(out, q, k_cache, v_cache, block_tables, max_blocks_per_seq, seq_lens,
                                             nullptr, B, Hq, Hkv, D, block_size, num_blocks, scale, softcap, slopes, 0,
                                             dtype, workspace, workspace_bytes, dev_status, stream);
}
