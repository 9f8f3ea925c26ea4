// decode_attention_q8.cu -- GQA paged decode attention over the 8-bit KV cache.
//
// For query head qh of sequence b, KV head h = qh / G, L = seq_lens[b]:
//   s_j = scale * ks_j * <q, kv_j>,   out = sum_j softmax(s)_j * vs_j * vv_j
// with kv_j, vv_j the 8-bit numbers of position j's rows and ks_j, vs_j their
// float32 scales (quant8.cuh): a K scale multiplies a score, a V scale a
// softmax weight.
//
// One CTA per (sequence, query head), CUDA-core fp32, chunked online softmax.
#include <math.h>

#include "quant8.cuh"

namespace pkv {

int device_sm_count();

constexpr int kGen8Threads = 128;

template <typename T, typename Fmt>
__global__ void __launch_bounds__(kGen8Threads)
    decode_q8_generic_kernel(T* __restrict__ out, const T* __restrict__ q, const uint8_t* __restrict__ k_cache,
                             const uint8_t* __restrict__ v_cache, const float* __restrict__ k_scale,
                             const float* __restrict__ v_scale, const int32_t* __restrict__ block_tables,
                             int max_blocks, const int32_t* __restrict__ seq_lens, int Hq, int Hkv, int D, int BS,
                             int NB, float scale, int32_t* status) {
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
        ps[tid] = p * vs;
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
    const float inv = bad || l == 0.f ? 0.f : 1.f / l;
    for (int k = 0; k < 2; ++k) {
        const int d = tid + k * kGen8Threads;
        if (d < D) o[d] = from_f32<T>(bad ? 0.f : acc[k] * inv);
    }
}

}  // namespace pkv

extern "C" size_t pkv_decode_q8_workspace_bytes(int B, int Hq, int Hkv, int D, int num_sms) {
    if (B < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || D < 1) return 0;
    (void)num_sms;
    return 256;
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
    if (workspace_bytes < pkv_decode_q8_workspace_bytes(B, Hq, Hkv, D, 0)) return PKV_ERR_INVALID_ARG;
    if (scale <= 0.f) scale = 1.0f / sqrtf(static_cast<float>(D));
    auto go = [&](auto t, auto fmt) {
        using T = decltype(t);
        using Fmt = decltype(fmt);
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(B) * Hq, 1, 1);
        cfg.blockDim = dim3(kGen8Threads, 1, 1);
        cfg.stream = static_cast<cudaStream_t>(stream);
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        const cudaError_t err = cudaLaunchKernelEx(
            &cfg, decode_q8_generic_kernel<T, Fmt>, static_cast<T*>(out), static_cast<const T*>(q),
            static_cast<const uint8_t*>(k_cache), static_cast<const uint8_t*>(v_cache), k_scale, v_scale, block_tables,
            max_blocks_per_seq, seq_lens, Hq, Hkv, D, block_size, num_blocks, scale, dev_status);
        return err != cudaSuccess ? err : cudaGetLastError();
    };
    cudaError_t err;
    if (dtype == PKV_F32)
        err = cache_dtype == PKV_E4M3 ? go(float(), FmtE4M3()) : go(float(), FmtI8());
    else
        err = cache_dtype == PKV_E4M3 ? go(__nv_bfloat16(), FmtE4M3()) : go(__nv_bfloat16(), FmtI8());
    return err == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}
