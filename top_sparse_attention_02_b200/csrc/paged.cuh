// paged.cuh -- device helpers of the paged-cache kernels: element types and the
// warp's matrix instructions on them.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "paged.h"

namespace tsa {

constexpr int kPagedSms = 148;

// 2^x by the special-function unit (about 2^-22 of the value; below 2^-126: 0)
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
    return y;
}

// ---- two fp32 values in one 64-bit register: one instruction for both
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};\n" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;\n" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;\n" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// The element types.  Softmax weights become elements for the second product; an fp16
// one below 2^-25 is zero, and a long flat tail of such weights may be worth more
// than an output's rounding.  So fp16 weights are formed relative to a maximum
// lowered by a bias (their sums and the maximum kept with them are, too, and the
// quotient is the same): kBias for weights of at most 1, and kBiasRef, kGrow for those
// of a shared prefix, whose reference may fall 2^kGrow behind the maximum.
//
// From 2^22 on (base 2) a step of fp32 is 1/2 and more: a maximum of 2^27 less 12 rounds to
// it less 16, and a product that is not rounded may lie several above its maximum, which
// was.  Such maxima are not lowered, and their scores are rounded before anything is
// taken from them, so that no weight exceeds 1 (in fp16 one of 2^16 would be infinite).
constexpr float kBigLogit = 4194304.f;
template <class E>
__device__ __forceinline__ float lowered(float m) { return fabsf(m) < kBigLogit ? m - E::kBias : m; }

struct Bf16 {
    static constexpr bool kHalf = false;
    static constexpr float kBias = 0.f, kBiasRef = 0.f, kGrow = 8.f;
    static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
        uint32_t r;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(hi), "f"(lo));
        return r;
    }
    static __device__ __forceinline__ float lo(uint32_t w) { return bf_lo(w); }
    static __device__ __forceinline__ float hi(uint32_t w) { return bf_hi(w); }
    static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};\n"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
    static __device__ __forceinline__ void unpack8(const uint4& r, uint64_t (&f)[4]) {
        f[0] = pack2(lo(r.x), hi(r.x)), f[1] = pack2(lo(r.y), hi(r.y));
        f[2] = pack2(lo(r.z), hi(r.z)), f[3] = pack2(lo(r.w), hi(r.w));
    }
    static __device__ __forceinline__ uint4 pack8(const uint64_t (&f)[4]) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float a, b;
            unpack2(f[j], a, b);
            w[j] = pack(a, b);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

struct F16 {
    static constexpr bool kHalf = true;
    static constexpr float kBias = 12.f, kBiasRef = 10.f, kGrow = 5.f;  // weights up to 2^12, 2^15; below 2^-37, 2^-35: zero
    static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
        uint32_t r;
        asm("cvt.rn.f16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(hi), "f"(lo));
        return r;
    }
    static __device__ __forceinline__ float lo(uint32_t w) { return __half2float(__ushort_as_half((unsigned short)w)); }
    static __device__ __forceinline__ float hi(uint32_t w) { return __half2float(__ushort_as_half((unsigned short)(w >> 16))); }
    static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};\n"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
    static __device__ __forceinline__ void unpack8(const uint4& r, uint64_t (&f)[4]) {
        f[0] = pack2(lo(r.x), hi(r.x)), f[1] = pack2(lo(r.y), hi(r.y));
        f[2] = pack2(lo(r.z), hi(r.z)), f[3] = pack2(lo(r.w), hi(r.w));
    }
    static __device__ __forceinline__ uint4 pack8(const uint64_t (&f)[4]) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float a, b;
            unpack2(f[j], a, b);
            w[j] = pack(a, b);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

}  // namespace tsa
