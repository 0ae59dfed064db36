// f32x2.cuh -- two floats in one register pair, 16-byte vectors of logits as such pairs, and the hardware exponential: what the
// passes over vocabulary-wide rows share that add up exponentials of every logit.
#pragma once

#include "smcsd_internal.cuh"

namespace smcsd {

__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Two floats in one register pair, for the instructions that work on both.
struct f32x2 {
    unsigned long long v;
};
__device__ __forceinline__ f32x2 pair(float lo, float hi) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void halves(f32x2 a, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(a.v)); }
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ f32x2 exp2_2(f32x2 a) {
    float lo, hi;
    halves(a, lo, hi);
    return pair(exp2_fast(lo), exp2_fast(hi));
}

// A 16-byte vector as pairs of floats: 2 of float32, 4 of bf16.
template <int DT>
struct Vec {
    static constexpr int kPairs = Geo<DT>::kPerVec / 2;
    f32x2 x[kPairs];
    __device__ __forceinline__ explicit Vec(const uint4& v) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < kPairs; ++i)
            x[i] = DT == 0 ? pair(__uint_as_float(w[(2 * i) & 3]), __uint_as_float(w[(2 * i + 1) & 3])) : pair(bf16_lo(w[i & 3]), bf16_hi(w[i & 3]));
    }
    __device__ __forceinline__ uint4 packed() const {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
            float lo, hi;
            halves(x[i], lo, hi);
            if (DT == 0)
                w[(2 * i) & 3] = __float_as_uint(lo), w[(2 * i + 1) & 3] = __float_as_uint(hi);
            else
                asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i & 3]) : "f"(hi), "f"(lo));
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};
}  // namespace smcsd
