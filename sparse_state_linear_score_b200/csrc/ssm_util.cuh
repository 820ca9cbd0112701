// Device helpers of the state-space block's kernels (short_conv, selective_scan, block_norm).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#ifndef SDM_DEV
#define SDM_DEV __device__ __forceinline__
#endif

namespace sdm {
namespace ssm {

typedef __nv_bfloat16 bf16;

constexpr float kLog2e = 1.44269504088896340736f;

// A view's pointer and strides (elements): sequence, head (or group), token.
template <typename T>
struct View {
    T* p;
    long long sb, sh, st;
};

SDM_DEV float ld(const float* p) { return *p; }
SDM_DEV float ld(const bf16* p) { return __bfloat162float(*p); }
SDM_DEV void st(float* p, float v) { *p = v; }
SDM_DEV void st(bf16* p, float v) { *p = __float2bfloat16_rn(v); }

// V consecutive elements as floats; V = 4 wants an address aligned to the four elements.
template <int V>
struct Vec;

template <>
struct Vec<1> {
    template <typename T>
    SDM_DEV static void load(const T* p, float (&v)[1]) {
        v[0] = ld(p);
    }
    template <typename T>
    SDM_DEV static void store(T* p, const float (&v)[1]) {
        st(p, v[0]);
    }
};

SDM_DEV float bf16_lo(uint32_t x) { return __uint_as_float(x << 16); }
SDM_DEV float bf16_hi(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }
SDM_DEV uint32_t pack_bf16(float a, float b) {  // a in the low half, round to nearest even
    __nv_bfloat162 r = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&r);
}

template <>
struct Vec<4> {
    SDM_DEV static void load(const float* p, float (&v)[4]) {
        const float4 x = *reinterpret_cast<const float4*>(p);
        v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
    }
    SDM_DEV static void load(const bf16* p, float (&v)[4]) {
        const uint2 x = *reinterpret_cast<const uint2*>(p);
        v[0] = bf16_lo(x.x), v[1] = bf16_hi(x.x), v[2] = bf16_lo(x.y), v[3] = bf16_hi(x.y);
    }
    SDM_DEV static void store(float* p, const float (&v)[4]) {
        *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    }
    SDM_DEV static void store(bf16* p, const float (&v)[4]) {
        *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
    }
};

// 2^x (ex2.approx: relative error about 2^-22; 0 below the normal range).
SDM_DEV float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

SDM_DEV float sigmoid(float x) { return __fdividef(1.f, 1.f + __expf(-x)); }

// log(1 + e^x) = max(x, 0) + log(1 + e), e = e^-|x| <= 1, to a few units in the last place: a
// step's relative error goes into every state and gradient behind it, so small steps (x << 0)
// keep theirs.  log(1 + e) = 2 atanh(w), w = e / (2 + e) <= 1/3, by its Taylor series (the first
// term left out is below 2^-24 of the sum); the rounding of |x| log2(e), which would cost e up to
// |x| 2^-24, is put back to first order.
SDM_DEV float softplus(float x) {
    float a = fabsf(x);
    if (a > 128.f) a = 128.f;  // e is 0 there; a NaN stays
    const float p = a * kLog2e;
    const float lo = fmaf(a, kLog2e, -p) + a * 1.925963033500e-8f;  // log2(e) - its fp32 value
    float e = exp2_fast(-p);
    e = fmaf(e, -0.69314718f * lo, e);
    const float w = __fdividef(e, 2.f + e), q = w * w;
    float s = 2.f / 15.f;
    s = fmaf(s, q, 2.f / 13.f);
    s = fmaf(s, q, 2.f / 11.f);
    s = fmaf(s, q, 2.f / 9.f);
    s = fmaf(s, q, 2.f / 7.f);
    s = fmaf(s, q, 2.f / 5.f);
    s = fmaf(s, q, 2.f / 3.f);
    s = fmaf(s * q, w, 2.f * w);
    return fmaxf(x, 0.f) + s;
}

SDM_DEV int clamp_len(const int* lens, int b, int T) {
    if (!lens) return T;
    const int n = lens[b];
    return n < 0 ? 0 : (n > T ? T : n);
}

template <typename T>
SDM_DEV T warp_sum(T v) {
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
    return v;
}

}  // namespace ssm
}  // namespace sdm
