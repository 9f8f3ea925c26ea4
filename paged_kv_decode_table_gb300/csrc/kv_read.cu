// kv_read.cu -- blocks of the 8-bit cache read back as bf16 or float32 blocks.
//
// For i in [0, n): out[i][h][slot][:] = value * scale of block blocks[i], one
// float32 product per element, rounded once to the output type.  The result
// has the layout of an unquantised pool of n blocks, so prefill attention (or
// anything else that reads such a pool) runs on it with a table that counts 0, 1,
// 2, ...
//
// One warp per row of D values.
#include "quant8.cuh"

namespace pkv {

constexpr int kReadWarps = 8;

template <typename T, typename Fmt>
__global__ void __launch_bounds__(kReadWarps * 32)
    kv_read_kernel(T* __restrict__ k_out, T* __restrict__ v_out, const uint8_t* __restrict__ k_cache,
                   const uint8_t* __restrict__ v_cache, const float* __restrict__ k_scale,
                   const float* __restrict__ v_scale, const int32_t* __restrict__ blocks, long long rows, int R, int D,
                   int NB, int32_t* status) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long u = static_cast<long long>(blockIdx.x) * kReadWarps + warp;  // (K or V, block, row)
    if (u >= 2 * rows) return;
    const bool is_v = u >= rows;
    const long long orow = is_v ? u - rows : u;
    const int blk = blocks[orow / R];
    T* dst = (is_v ? v_out : k_out) + orow * D;
    if (blk < 0 || blk >= NB) {
        if (lane == 0 && !is_v && orow % R == 0) report(status, PKV_ERR_DEVICE_BOUNDS);
        for (int i = lane; i < D; i += 32) dst[i] = from_f32<T>(0.f);
        return;
    }
    const long long irow = static_cast<long long>(blk) * R + orow % R;
    const float scale = (is_v ? v_scale : k_scale)[irow];
    const uint8_t* src = (is_v ? v_cache : k_cache) + irow * D;
    for (int i = lane; i < D; i += 32) dst[i] = from_f32<T>(Fmt::decode(src[i]) * scale);
}

template <typename T, typename Fmt>
static cudaError_t launch_read(void* k_out, void* v_out, const void* k_cache, const void* v_cache,
                               const float* k_scale, const float* v_scale, const int32_t* blocks, int n, int R, int D,
                               int NB, int32_t* status, cudaStream_t stream) {
    const long long rows = static_cast<long long>(n) * R;
    const long long grid = (2 * rows + kReadWarps - 1) / kReadWarps;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
    cfg.blockDim = dim3(kReadWarps * 32, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t err = cudaLaunchKernelEx(
        &cfg, kv_read_kernel<T, Fmt>, static_cast<T*>(k_out), static_cast<T*>(v_out),
        static_cast<const uint8_t*>(k_cache), static_cast<const uint8_t*>(v_cache), k_scale, v_scale, blocks, rows, R,
        D, NB, status);
    return err != cudaSuccess ? err : cudaGetLastError();
}

}  // namespace pkv

extern "C" pkv_status pkv_kv_read_blocks_q8(void* k_out, void* v_out, const void* k_cache, const void* v_cache,
                                            const float* k_scale, const float* v_scale, const int32_t* blocks, int n,
                                            int Hkv, int D, int block_size, int num_blocks, pkv_dtype out_dtype,
                                            pkv_dtype cache_dtype, int32_t* dev_status, void* stream) {
    if (n < 0 || Hkv < 1 || D < 1 || D > 256 || block_size < 1 || num_blocks < 1 ||
        (out_dtype != PKV_F32 && out_dtype != PKV_BF16) || (cache_dtype != PKV_E4M3 && cache_dtype != PKV_I8))
        return PKV_ERR_INVALID_ARG;
    if (static_cast<long long>(Hkv) * block_size > 0x7fffffffLL) return PKV_ERR_INVALID_ARG;
    if (n == 0) return PKV_OK;
    if (!k_out || !v_out || !k_cache || !v_cache || !k_scale || !v_scale || !blocks) return PKV_ERR_INVALID_ARG;
    auto launch = out_dtype == PKV_F32
                      ? (cache_dtype == PKV_E4M3 ? pkv::launch_read<float, pkv::FmtE4M3>
                                                 : pkv::launch_read<float, pkv::FmtI8>)
                      : (cache_dtype == PKV_E4M3 ? pkv::launch_read<__nv_bfloat16, pkv::FmtE4M3>
                                                 : pkv::launch_read<__nv_bfloat16, pkv::FmtI8>);
    const cudaError_t err = launch(k_out, v_out, k_cache, v_cache, k_scale, v_scale, blocks, n, Hkv * block_size, D,
                                   num_blocks, dev_status, static_cast<cudaStream_t>(stream));
    return err == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}
