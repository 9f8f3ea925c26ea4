// tensor_core.cuh -- tcgen05 and TMA wrappers of the attention kernels that run on the fifth-generation tensor cores,
// and what their softmax threads do with a tile of 64 products.
#pragma once

#include "attention_scores.cuh"

namespace pkv {

// ------------------------------------------------------------------ tcgen05 helpers
// Shared-memory matrix descriptor, 128-byte swizzle: start address, leading
// byte offset (K-major: unused; MN-major: the stride between 64-element atoms
// along M / N), stride byte offset (the stride between groups of 8 rows), the
// descriptor version of this architecture.
__device__ __forceinline__ uint64_t tc_desc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
    return static_cast<uint64_t>((addr >> 4) & 0x3FFFu) | (static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16) |
           (static_cast<uint64_t>((sbo >> 4) & 0x3FFFu) << 32) | (1ull << 46) | (2ull << 61);
}
// Instruction descriptor of kind::f16: bf16 A and B, fp32 accumulator, M x N,
// B K-major or MN-major (A always K-major here).
__host__ __device__ constexpr uint32_t tc_idesc(int M, int N, bool b_mn_major) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((b_mn_major ? 1u : 0u) << 16) |
           (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}
__device__ __forceinline__ void tc_mma(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
// The same with A (M x 16 bf16, row m in TMEM lane m, two elements per column) in tensor memory.
__device__ __forceinline__ void tc_mma_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
// Arrive on bar once every tcgen05 operation this thread issued so far is complete.
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// 32 consecutive columns of this thread's TMEM lane (warp w reads lanes 32 (w % 4) ..).
__device__ __forceinline__ void tc_ld32(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tc_st32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]),
        "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]),
        "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
// Byte offset of (row, 16-byte chunk) in a tile of 128-byte rows with the
// 128-byte swizzle (the chunk index XOR the row's low three bits).
__device__ __forceinline__ uint32_t sw128(int row, int chunk) {
    return static_cast<uint32_t>(row) * 128u + (static_cast<uint32_t>(chunk ^ (row & 7)) << 4);
}
// 4-D tiled copy (the K boxes); x, y, z, w are the box's start coordinates.
__device__ __forceinline__ void tma_load_4d(void* smem_dst, const void* tmap, int x, int y, int z, int w,
                                            uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
        "[%6];" ::"r"(smem_u32(smem_dst)),
        "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
        : "memory");
}
// max(a, b, c) in one instruction
__device__ __forceinline__ float tc_max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
// (x0, x1) = (a0 b + c, a1 b + c) and (s0, s1) += (a0, a1) as paired fp32 operations
__device__ __forceinline__ void tc_fma2(float& x0, float& x1, float a0, float a1, float b, float c) {
    asm("{\n\t.reg .b64 ra, rb, rc, rd;\n\t"
        "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %4};\n\tmov.b64 rc, {%5, %5};\n\t"
        "fma.rn.f32x2 rd, ra, rb, rc;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(x0), "=f"(x1)
        : "f"(a0), "f"(a1), "f"(b), "f"(c));
}
__device__ __forceinline__ void tc_add2(float& s0, float& s1, float a0, float a1) {
    asm("{\n\t.reg .b64 ra, rs;\n\t"
        "mov.b64 ra, {%2, %3};\n\tmov.b64 rs, {%0, %1};\n\t"
        "add.rn.f32x2 rs, rs, ra;\n\tmov.b64 {%0, %1}, rs;\n\t}"
        : "+f"(s0), "+f"(s1)
        : "f"(a0), "f"(a1));
}
__device__ __forceinline__ float tc_ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Pairs of floats in a 64-bit register.
__device__ __forceinline__ uint64_t tc_pair(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ uint64_t tc_pair(uint32_t a, uint32_t b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ void tc_unpair(uint32_t& a, uint32_t& b, uint64_t v) {
    asm("mov.b64 {%0, %1}, %2;" : "=r"(a), "=r"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t tc_mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t tc_fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

__device__ __forceinline__ uint64_t tc_add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// The products of a row with a tile's keys become scores in the log2 domain.  dist: the first key's position less
// that of the key that the row's bias is measured from; slope: of the row's head, times log2(e).  All lanes of the warp take part.  Four pairs go through each
// operation together: their chains hide one another's latency.
template <bool kCap, bool kSlope, int kChunks>
__device__ __forceinline__ void tc_scores(uint32_t (&sr)[kChunks][32], int dist, float slope, const ScoreArgs& sc) {
    constexpr int kBlock = 4;
    auto at = [&](int c) -> uint32_t& { return sr[c >> 5][c & 31]; };
    auto both = [](float v) { return tc_pair(v, v); };
    [[maybe_unused]] const uint64_t slope2 = both(slope), step2 = both(2.f * kBlock);
    [[maybe_unused]] uint64_t away[kBlock];  // positions of the block's keys less that key's, exact up to 2^24
    auto far = [&]() {
#pragma unroll
        for (int k = 0; k < kBlock; ++k) away[k] = tc_pair(static_cast<float>(dist + 2 * k), static_cast<float>(dist + 2 * k + 1));
    };
    // a * b, with slopes plus the bias, for the pairs from c on
    auto finish = [&](const uint64_t (&a)[kBlock], const uint64_t (&b)[kBlock], int c) {
        uint64_t v[kBlock];
        if constexpr (kSlope) {
#pragma unroll
            for (int k = 0; k < kBlock; ++k) v[k] = tc_mul2(slope2, away[k]);
#pragma unroll
            for (int k = 0; k < kBlock; ++k) v[k] = tc_fma2(a[k], b[k], v[k]);
#pragma unroll
            for (int k = 0; k < kBlock; ++k) away[k] = tc_add2(away[k], step2);
        } else {
#pragma unroll
            for (int k = 0; k < kBlock; ++k) v[k] = tc_mul2(a[k], b[k]);
        }
#pragma unroll
        for (int k = 0; k < kBlock; ++k) tc_unpair(at(c + 2 * k), at(c + 2 * k + 1), v[k]);
    };
    if constexpr (kSlope) far();
    if constexpr (kCap) {
        float big[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < 32 * kChunks; c += 2)
            big[(c >> 1) & 3] = tc_max3(big[(c >> 1) & 3], fabsf(__uint_as_float(at(c))), fabsf(__uint_as_float(at(c + 1))));
        const uint64_t in2 = both(sc.in);
        // x and cap log2(e) tanh(x) / x of the pairs from c on, for scores within the cap
        auto within = [&](uint64_t (&x)[kBlock], uint64_t (&p)[kBlock], const uint64_t (&coef)[6], int c) {
            uint64_t w[kBlock];
#pragma unroll
            for (int k = 0; k < kBlock; ++k) x[k] = tc_mul2(tc_pair(at(c + 2 * k), at(c + 2 * k + 1)), in2);
#pragma unroll
            for (int k = 0; k < kBlock; ++k) w[k] = tc_mul2(x[k], x[k]);
#pragma unroll
            for (int k = 0; k < kBlock; ++k) p[k] = tc_fma2(coef[5], w[k], coef[4]);
#pragma unroll
            for (int e = 3; e >= 0; --e)
#pragma unroll
                for (int k = 0; k < kBlock; ++k) p[k] = tc_fma2(p[k], w[k], coef[e]);
        };
        // (The coefficients belong to the branches: ahead of both they cost 9% of a long capped prefix.)
        if (__all_sync(0xffffffffu, !(fmaxf(fmaxf(big[0], big[1]), fmaxf(big[2], big[3])) * sc.in > 1.f))) {
            const uint64_t coef[6] = {both(kTanh0 * sc.cap_log2), both(kTanh1 * sc.cap_log2), both(kTanh2 * sc.cap_log2),
                                      both(kTanh3 * sc.cap_log2), both(kTanh4 * sc.cap_log2), both(kTanh5 * sc.cap_log2)};
#pragma unroll
            for (int c = 0; c < 32 * kChunks; c += 2 * kBlock) {
                uint64_t x[kBlock], p[kBlock];
                within(x, p, coef, c);
                finish(x, p, c);
            }
        } else {
            const uint64_t coef[6] = {both(kTanh0 * sc.cap_log2), both(kTanh1 * sc.cap_log2), both(kTanh2 * sc.cap_log2),
                                      both(kTanh3 * sc.cap_log2), both(kTanh4 * sc.cap_log2), both(kTanh5 * sc.cap_log2)};
#pragma unroll
            for (int c = 0; c < 32 * kChunks; c += 2 * kBlock) {
                uint64_t x[kBlock], p[kBlock];
                within(x, p, coef, c);
                float most = 0.f;
#pragma unroll
                for (int k = 0; k < kBlock; ++k) {
                    uint32_t x0, x1;
                    tc_unpair(x0, x1, x[k]);
                    most = tc_max3(most, fabsf(__uint_as_float(x0)), fabsf(__uint_as_float(x1)));
                }
                if (!__any_sync(0xffffffffu, most > 1.f)) {  // the block is within the cap
                    finish(x, p, c);
                    continue;
                }
#pragma unroll
                for (int k = 0; k < kBlock; ++k) {  // tanh(x) and cap log2(e) instead, for scores that are beyond it
                    uint32_t xe[2], pe[2];
                    tc_unpair(xe[0], xe[1], x[k]);
                    tc_unpair(pe[0], pe[1], p[k]);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float f = __uint_as_float(xe[e]), t = tanh_beyond(f);
                        const bool large = fabsf(f) > 1.f;
                        xe[e] = large ? __float_as_uint(t) : xe[e];
                        pe[e] = large ? __float_as_uint(sc.cap_log2) : pe[e];
                    }
                    x[k] = tc_pair(xe[0], xe[1]);
                    p[k] = tc_pair(pe[0], pe[1]);
                }
                finish(x, p, c);
            }
        }
    } else {
        const uint64_t m2 = both(sc.mul);
#pragma unroll
        for (int c = 0; c < 32 * kChunks; c += 2 * kBlock) {
            uint64_t x[kBlock], b[kBlock];
#pragma unroll
            for (int k = 0; k < kBlock; ++k) {
                x[k] = tc_pair(at(c + 2 * k), at(c + 2 * k + 1));
                b[k] = m2;
            }
            finish(x, b, c);
        }
    }
}

// mbar_wait of a softmax warp, with the first poll apart from the loop: with the limit as an argument the loop alone costs the
// key tiles 3% (16 chunks of up to 512, capped: 478 us for 465, 463 with a constant limit).
__device__ __forceinline__ bool tc_wait(uint64_t* bar, uint32_t parity, uint32_t polls) {
    return mbar_try_wait(bar, parity) || mbar_wait(bar, parity, polls);
}

// Polls for copies that were issued to land, which takes microseconds: some ten milliseconds.  Where another of a stage's
// loading warps gave up, its arrival never comes, and the wait runs out although the copies have landed.
constexpr uint32_t kTcLandPolls = 1u << 17;

// Registers move from the warps that issue copies and MMAs to those of the softmax: 512 threads are launched with 128
// each, two warpgroups of softmax take 176, the two others keep 80.
__device__ __forceinline__ void tc_more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 176;"); }
__device__ __forceinline__ void tc_fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 80;"); }

}  // namespace pkv
