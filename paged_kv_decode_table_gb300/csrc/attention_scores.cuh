// attention_scores.cuh -- the scores of the *_scored and *_shared attention calls.
//
// For query head qh at position pos and key j, with t = <q, K_j>:
//   u = cap tanh(scale t / cap)  (cap > 0),  else scale t
//   s = u + slopes[qh] (j - pos)  (slopes given),  else u
// and key j < L takes part where j < prefix, or j <= pos and (window <= 0 or j > pos - window).
// The kernels work with s log2(e), so that a weight is one exp2.
//
// A softmax stays what it is when a constant is added to a row's scores, so the bias is measured from the key that it
// favours most, the row's first one that takes part where the slope is negative and its last one otherwise, and not from
// pos.  It is 0 there and falls from there on: keys that it makes matter have a small one.  Measured from pos, a
// slope of -0.5 would give the heaviest keys of 131072 a score of -95000, whose float32 neighbours lie 2^-7 apart.  All
// parts of a row that are joined later measure from the same key.
#pragma once

#include <math.h>

#include "pkv_common.cuh"

namespace pkv {

constexpr float kLog2e = 1.4426950408889634f;

// Passed to the kernels by value.
struct ScoreArgs {
    float mul;                   // scale log2(e)
    float in, cap_log2;          // scale / cap and cap log2(e); 0: no cap
    const float* slopes;         // [Hq] or NULL
    int window;                  // <= 0: none
    const int32_t* prefix_lens;  // [B] or NULL
};
// False where a number is out of range: the cap negative, NaN or subnormal, scale / cap subnormal (in the products with it
// scores would lose their digits, and below 2^-149 be all 0), or a product of the two not finite.
inline bool make_scores(ScoreArgs* sa, float scale, int D, float cap, const float* slopes, int window,
                        const int32_t* prefix_lens) {
    if (!(scale > 0.f)) scale = 1.0f / sqrtf(static_cast<float>(D));
    *sa = ScoreArgs{scale * kLog2e, cap > 0.f ? scale / cap : 0.f, cap * kLog2e, slopes, window, prefix_lens};
    constexpr float kNormal = 1.17549435e-38f;
    return (cap == 0.f || (cap >= kNormal && sa->in >= kNormal)) && sa->mul <= 3.0e38f && sa->in <= 3.0e38f && sa->cap_log2 <= 3.0e38f;
}

// Positions stay in 32 bits, with a few tiles to spare.
inline bool positions_fit(int max_blocks, int BS) { return static_cast<long long>(max_blocks) * BS <= 0x7fff0000LL; }
// Rows of out are written while others of q are still read.
inline bool overlap(const void* out, const void* q, size_t bytes) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(out), b = reinterpret_cast<uintptr_t>(q);
    return a < b ? b - a < bytes : a - b < bytes;
}

// The positions that the one query of a decode step sees: [0, pfx) and [lo, L), pfx <= lo.
struct Seen {
    int L, lo, pfx;
    __device__ __forceinline__ bool at(int j) const { return j < L && (j >= lo || j < pfx); }
    __device__ __forceinline__ int first() const { return pfx > 0 ? 0 : lo; }
};
__device__ __forceinline__ Seen decode_seen(const ScoreArgs& sa, int b, int L) {
    Seen s{L, 0, 0};
    if (sa.window > 0 && sa.window < L) {
        s.lo = L - sa.window;
        if (sa.prefix_lens != nullptr) s.pfx = min(max(sa.prefix_lens[b], 0), L);
        if (s.pfx >= s.lo) s.pfx = s.lo = 0;
    }
    return s;
}

__device__ __forceinline__ float ex2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// tanh(x), x = scale t / cap.  For |x| <= 1, x times a polynomial in x^2: the minimax one of five for the relative
// error, 2^-20.7 of tanh(x) (found by linear programming on a grid), so that a small score keeps its relative accuracy
// whatever the cap is.  Beyond, 1 - 2 / (e^(2x) + 1), off by about 2^-23 and relatively accurate for these x only; e^(2x) =
// infinity gives 1.  The kernels vote: where all scores of a warp's tile are within the cap only the polynomial is
// computed (eight operations on the FMA pipe), else both (the second form is two on the slower special-function pipe), and
// every score takes its own: what it becomes does not depend on the tile's others, hidden ones among them.
constexpr float kTanh0 = 0.99999941f, kTanh1 = -0.33329042f, kTanh2 = 0.13281434f, kTanh3 = -0.05160567f,
                kTanh4 = 0.01674311f, kTanh5 = -0.00306706f;
__device__ __forceinline__ float tanh_within(float x) {
    const float w = x * x;
    float p = fmaf(kTanh5, w, kTanh4);
    p = fmaf(p, w, kTanh3);
    p = fmaf(p, w, kTanh2);
    p = fmaf(p, w, kTanh1);
    return x * fmaf(p, w, kTanh0);
}
__device__ __forceinline__ float tanh_beyond(float x) {
    return fmaf(-2.f, rcp_approx(ex2_approx(x * (2.f * kLog2e)) + 1.f), 1.f);
}

}  // namespace pkv
