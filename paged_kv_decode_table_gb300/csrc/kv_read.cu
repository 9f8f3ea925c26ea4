// kv_read.cu -- blocks of the 8-bit cache read back as bf16 or float32 blocks.
//
// For i in [0, n): out[i][h][slot][:] = value * scale of block blocks[i], one
// float32 product per element, rounded once to the output type.  The result
// has the layout of an unquantised pool of n blocks, so prefill attention (or
// anything else that reads such a pool) runs on it with a table that counts 0, 1,
// 2, ...
//
// A thread holds kVec elements of a row: 8 for bf16 (8 bytes in, 16 out), 4 for
// float32 (4 in, 16 out), so that stores are 16 bytes and neighbouring threads
// write neighbouring 16 bytes; 1 where D or an address does not allow it.  A CTA takes
// kReadPasses passes of as many whole rows as its threads cover, all loads of the
// passes first, with the streaming hint: a cached byte is read once here.  No input is read
// through the read-only path (__ldg, const __restrict__): the kernel may start while the append
// before it still writes them.
// HBM-bound.  9216 blocks of 8 heads x 16 x 128 in e4m3 to bf16 (915 MB moved):
// 4 passes 138 us, 6.63 TB/s, 99% of the measured copy rate.  With the scales through the
// read-only path 4 passes took 140 us, 2 passes 156, 8 passes 167, 4 without the hint 159.
#include "quant8.cuh"

namespace pkv {

constexpr int kReadThreads = 256;
constexpr int kReadPasses = 4;

// kVec bytes as loaded.
template <int kVec>
struct Bytes {
    uint32_t w[kVec == 8 ? 2 : 1];
};
template <int kVec>
__device__ __forceinline__ Bytes<kVec> load_bytes(const uint8_t* src) {
    Bytes<kVec> r;
    if constexpr (kVec == 8) {
        const uint2 v = __ldcs(reinterpret_cast<const uint2*>(src));
        r.w[0] = v.x;
        r.w[1] = v.y;
    } else if constexpr (kVec == 4) {
        r.w[0] = __ldcs(reinterpret_cast<const uint32_t*>(src));
    } else {
        r.w[0] = __ldcs(src);
    }
    return r;
}

template <typename Fmt, int kVec>
__device__ __forceinline__ void decode_row(const Bytes<kVec>& r, float (&x)[kVec]) {
    if constexpr (kVec == 1) {
        x[0] = Fmt::decode(static_cast<uint8_t>(r.w[0]));
    } else {
#pragma unroll
        for (int k = 0; k < kVec / 4; ++k) {
            uint32_t lo, hi;
            Fmt::decode4(r.w[k], lo, hi);
            const float2 a = unpack_f16x2(lo), b = unpack_f16x2(hi);
            x[4 * k] = a.x;
            x[4 * k + 1] = a.y;
            x[4 * k + 2] = b.x;
            x[4 * k + 3] = b.y;
        }
    }
}

template <typename T, int kVec>
__device__ __forceinline__ void store_row(T* dst, const float (&x)[kVec]) {
    if constexpr (kVec == 1) {
        *dst = from_f32<T>(x[0]);
    } else if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<float4*>(dst) = make_float4(x[0], x[1], x[2], x[3]);
    } else if constexpr (kVec == 8) {
        *reinterpret_cast<uint4*>(dst) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                                    pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
    } else {
        *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
    }
}

template <typename T, typename Fmt, int kVec>
__global__ void __launch_bounds__(kReadThreads)
    kv_read_kernel(T* k_out, T* v_out, const uint8_t* k_cache, const uint8_t* v_cache, const float* k_scale,
                   const float* v_scale, const int32_t* blocks, int chunks, int R, int D, int NB, int32_t* status) {
    prefetch_l2(blocks, static_cast<size_t>(gridDim.x / (2 * chunks)) * 4, blockIdx.x * kReadThreads + threadIdx.x);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // CTA: (block, K or V, chunk of rows)
    const unsigned chunk = blockIdx.x % chunks, bp = blockIdx.x / chunks;
    const bool is_v = bp & 1u;
    const int i = static_cast<int>(bp >> 1);
    const int blk = blocks[i];
    const bool good = blk >= 0 && blk < NB;
    if (!good && threadIdx.x == 0 && !is_v && chunk == 0) report(status, PKV_ERR_DEVICE_BOUNDS);
    const int per_row = D / kVec, rows = kReadThreads / per_row;  // threads per row, rows per pass
    const int sub = threadIdx.x / per_row, col = (threadIdx.x - sub * per_row) * kVec;
    if (sub >= rows) return;
    const int r0 = chunk * rows * kReadPasses + sub, last = R - 1;
    const uint8_t* src = (is_v ? v_cache : k_cache) + static_cast<size_t>(good ? blk : 0) * R * D + col;
    const float* sc = (is_v ? v_scale : k_scale) + static_cast<size_t>(good ? blk : 0) * R;
    T* dst = (is_v ? v_out : k_out) + static_cast<size_t>(i) * R * D + col;
    // every load before the first use; rows behind the block's end read its last row again
    Bytes<kVec> raw[kReadPasses];
    float scale[kReadPasses];
#pragma unroll
    for (int p = 0; p < kReadPasses; ++p) {
        const int r = min(r0 + p * rows, last);
        raw[p] = load_bytes<kVec>(src + r * D);
        scale[p] = sc[r];
    }
#pragma unroll
    for (int p = 0; p < kReadPasses; ++p) {
        const int r = r0 + p * rows;
        if (r > last) break;
        float x[kVec];
        decode_row<Fmt, kVec>(raw[p], x);
#pragma unroll
        for (int e = 0; e < kVec; ++e) x[e] = good ? x[e] * scale[p] : 0.f;
        store_row<T, kVec>(dst + r * D, x);
    }
}

// Blocks of few rows: the rows of all blocks in one order, cut into CTAs whatever block they
// are of.  8479 blocks of 1 head x 64 x 32 in int8 to bf16 (109 MB moved): 18.2 us, 6.0
// TB/s; a CTA per block and pool 38.7 us.  4000 blocks of 12 x 16 x 32: 27.3 against 32.4 us.
// Large blocks stay with the kernel above, which is 2% faster on them.
constexpr int kRowsPasses = 6;

template <typename T, typename Fmt, int kVec>
__global__ void __launch_bounds__(kReadThreads)
    kv_read_rows_kernel(T* k_out, T* v_out, const uint8_t* k_cache, const uint8_t* v_cache, const float* k_scale,
                        const float* v_scale, const int32_t* blocks, int chunks, int n, int R, int D, int NB,
                        int32_t* status) {
    prefetch_l2(blocks, static_cast<size_t>(n) * 4, blockIdx.x * kReadThreads + threadIdx.x);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int per_row = D / kVec, rows = kReadThreads / per_row;  // threads per row, rows per pass
    const int sub = threadIdx.x / per_row, col = (threadIdx.x - sub * per_row) * kVec;
    // CTA: (K or V, chunk of all rows)
    const unsigned chunk = blockIdx.x % static_cast<unsigned>(chunks);
    const bool is_v = blockIdx.x >= static_cast<unsigned>(chunks);
    const uint8_t* src = (is_v ? v_cache : k_cache) + col;
    const float* sc = is_v ? v_scale : k_scale;
    T* dst = (is_v ? v_out : k_out) + col;
    Bytes<kVec> raw[kRowsPasses];
    float scale[kRowsPasses];
    if (sub >= rows) return;
    const unsigned last = static_cast<unsigned>(n) * R - 1u, r0 = chunk * static_cast<unsigned>(rows * kRowsPasses) + sub;
    int blk[kRowsPasses];
    unsigned in_blk[kRowsPasses];
#pragma unroll
    for (int p = 0; p < kRowsPasses; ++p) {
        const unsigned r = min(r0 + p * rows, last), i = r / static_cast<unsigned>(R);
        blk[p] = blocks[i];
        in_blk[p] = r - i * R;
    }
#pragma unroll
    for (int p = 0; p < kRowsPasses; ++p) {
        const bool good = blk[p] >= 0 && blk[p] < NB;
        if (!good && !is_v && col == 0 && in_blk[p] == 0) report(status, PKV_ERR_DEVICE_BOUNDS);
        const size_t row = static_cast<size_t>(good ? blk[p] : 0) * R + in_blk[p];
        raw[p] = load_bytes<kVec>(src + row * D);
        scale[p] = sc[row];
        if (!good) blk[p] = -1;
    }
#pragma unroll
    for (int p = 0; p < kRowsPasses; ++p) {
        const unsigned r = r0 + p * rows;
        if (r > last) break;
        float x[kVec];
        decode_row<Fmt, kVec>(raw[p], x);
#pragma unroll
        for (int e = 0; e < kVec; ++e) x[e] = blk[p] >= 0 ? x[e] * scale[p] : 0.f;
        store_row<T, kVec>(dst + static_cast<size_t>(r) * D, x);
    }
}

template <typename T, typename Fmt>
static cudaError_t launch_read(void* k_out, void* v_out, const void* k_cache, const void* v_cache,
                               const float* k_scale, const float* v_scale, const int32_t* blocks, int n, int R, int D,
                               int NB, int32_t* status, cudaStream_t stream) {
    auto fits = [&](int vec) {
        const uintptr_t out = reinterpret_cast<uintptr_t>(k_out) | reinterpret_cast<uintptr_t>(v_out);
        const uintptr_t in = reinterpret_cast<uintptr_t>(k_cache) | reinterpret_cast<uintptr_t>(v_cache);
        return D % vec == 0 && in % vec == 0 && out % (vec * sizeof(T)) == 0;
    };
    auto run = [&](auto block_kern, auto rows_kern, int vec) {
        // blocks that would leave more than an eighth of a CTA's rows idle share CTAs
        const int pass = kReadThreads / (D / vec), rows = pass * kReadPasses;
        const long long all = static_cast<long long>(n) * R, idle = (rows - R % rows) % rows;
        const bool share = idle * 8 > R + idle && all < (1LL << 31);
        const long long per = share ? static_cast<long long>(pass) * kRowsPasses : rows;
        const long long chunks = ((share ? all : R) + per - 1) / per, grid = (share ? 2LL : 2LL * n) * chunks;
        if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
        cfg.blockDim = dim3(kReadThreads, 1, 1);
        cfg.stream = stream;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        T *ko = static_cast<T*>(k_out), *vo = static_cast<T*>(v_out);
        const uint8_t *kc = static_cast<const uint8_t*>(k_cache), *vc = static_cast<const uint8_t*>(v_cache);
        const int nch = static_cast<int>(chunks);
        const cudaError_t err = share ? cudaLaunchKernelEx(&cfg, rows_kern, ko, vo, kc, vc, k_scale, v_scale, blocks, nch,
                                                           n, R, D, NB, status)
                                      : cudaLaunchKernelEx(&cfg, block_kern, ko, vo, kc, vc, k_scale, v_scale, blocks,
                                                           nch, R, D, NB, status);
        return err != cudaSuccess ? err : cudaGetLastError();
    };
    if constexpr (sizeof(T) == 2) {
        if (fits(8)) return run(kv_read_kernel<T, Fmt, 8>, kv_read_rows_kernel<T, Fmt, 8>, 8);
    }
    if (fits(4)) return run(kv_read_kernel<T, Fmt, 4>, kv_read_rows_kernel<T, Fmt, 4>, 4);
    return run(kv_read_kernel<T, Fmt, 1>, kv_read_rows_kernel<T, Fmt, 1>, 1);
}

}  // namespace pkv

extern "C" pkv_status pkv_kv_read_blocks_q8(void* k_out, void* v_out, const void* k_cache, const void* v_cache,
                                            const float* k_scale, const float* v_scale, const int32_t* blocks, int n,
                                            int Hkv, int D, int block_size, int num_blocks, pkv_dtype out_dtype,
                                            pkv_dtype cache_dtype, int32_t* dev_status, void* stream) {
    if (n < 0 || Hkv < 1 || D < 1 || D > 256 || block_size < 1 || num_blocks < 1 ||
        (out_dtype != PKV_F32 && out_dtype != PKV_BF16) || (cache_dtype != PKV_E4M3 && cache_dtype != PKV_I8))
        return PKV_ERR_INVALID_ARG;
    if (static_cast<long long>(Hkv) * block_size * D > 0x7fffffffLL) return PKV_ERR_INVALID_ARG;
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
