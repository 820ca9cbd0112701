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

template <>
struct Vec<8> {  // bf16 only: 16 bytes
    SDM_DEV static void load(const bf16* p, float (&v)[8]) {
        const uint4 x = *reinterpret_cast<const uint4*>(p);
        v[0] = bf16_lo(x.x), v[1] = bf16_hi(x.x), v[2] = bf16_lo(x.y), v[3] = bf16_hi(x.y);
        v[4] = bf16_lo(x.z), v[5] = bf16_hi(x.z), v[6] = bf16_lo(x.w), v[7] = bf16_hi(x.w);
    }
};

template <>
struct Vec<2> {
    SDM_DEV static void load(const float* p, float (&v)[2]) {
        const float2 x = *reinterpret_cast<const float2*>(p);
        v[0] = x.x, v[1] = x.y;
    }
    SDM_DEV static void load(const bf16* p, float (&v)[2]) {
        const uint32_t x = *reinterpret_cast<const uint32_t*>(p);
        v[0] = bf16_lo(x), v[1] = bf16_hi(x);
    }
    SDM_DEV static void store(float* p, const float (&v)[2]) {
        *reinterpret_cast<float2*>(p) = make_float2(v[0], v[1]);
    }
    SDM_DEV static void store(bf16* p, const float (&v)[2]) {
        *reinterpret_cast<uint32_t*>(p) = pack_bf16(v[0], v[1]);
    }
};

// 2^x (ex2.approx: relative error about 2^-22; 0 below the normal range).
SDM_DEV float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

SDM_DEV float sigmoid(float x) { return __fdividef(1.f, 1.f + __expf(-x)); }

// ---- two fp32 at a time --------------------------------------------------------------------
typedef unsigned long long f32x2;
SDM_DEV f32x2 pack2(float lo, float hi) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
SDM_DEV f32x2 dup2(float x) { return pack2(x, x); }
SDM_DEV void unpack2(f32x2 v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
SDM_DEV f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
SDM_DEV f32x2 add2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
SDM_DEV f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
SDM_DEV f32x2 exp2_pair(f32x2 x) {
    float lo, hi;
    unpack2(x, lo, hi);
    return pack2(exp2_fast(lo), exp2_fast(hi));
}
SDM_DEV f32x2 rcp_pair(f32x2 x) {  // rcp.approx: one unit in the last place
    float lo, hi, a, b;
    unpack2(x, lo, hi);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(a) : "f"(lo));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(b) : "f"(hi));
    return pack2(a, b);
}
SDM_DEV float min_nan(float a, float b) {  // a NaN stays
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
SDM_DEV float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// A state's rate for exp2(s * rate) = e^(s A).  Kept finite where A log2(e) is not (A of the type's
// lowest value, or -inf where -e^x overflowed): a step of zero, also that of a row behind the
// sequence, then leaves the state as it is instead of making it 0 * inf.
SDM_DEV float decay_rate(float A) { return max_nan(A * kLog2e, -3.402823466e38f); }

// V consecutive values as they are stored: what a load in flight leaves in registers, so that
// nothing waits for it before they are used.
template <typename T, int V>
struct Raw;
template <>
struct Raw<float, 4> {
    float4 x;
    SDM_DEV void clear() { x = make_float4(0.f, 0.f, 0.f, 0.f); }
    SDM_DEV void load(const float* p) { x = *reinterpret_cast<const float4*>(p); }
    SDM_DEV void load(const float* p, int cnt) {  // the first cnt, where p is not aligned to four
        if (cnt > 0) x.x = p[0];
        if (cnt > 1) x.y = p[1];
        if (cnt > 2) x.z = p[2];
        if (cnt > 3) x.w = p[3];
    }
    SDM_DEV void pairs(f32x2 (&v)[2]) const { v[0] = pack2(x.x, x.y), v[1] = pack2(x.z, x.w); }
};
template <>
struct Raw<bf16, 4> {
    uint2 x;
    SDM_DEV void clear() { x = make_uint2(0u, 0u); }
    SDM_DEV void load(const bf16* p) { x = *reinterpret_cast<const uint2*>(p); }
    SDM_DEV void load(const bf16* p, int cnt) {
        const uint16_t* q = reinterpret_cast<const uint16_t*>(p);
        if (cnt > 0) x.x = q[0];
        if (cnt > 1) x.x |= (uint32_t)q[1] << 16;
        if (cnt > 2) x.y = q[2];
        if (cnt > 3) x.y |= (uint32_t)q[3] << 16;
    }
    SDM_DEV void pairs(f32x2 (&v)[2]) const {
        v[0] = pack2(bf16_lo(x.x), bf16_hi(x.x)), v[1] = pack2(bf16_lo(x.y), bf16_hi(x.y));
    }
};
template <typename T>
struct Raw<T, 1> {
    T x;
    SDM_DEV void clear() { x = T(0.f); }
    SDM_DEV void load(const T* p) { x = *p; }
    SDM_DEV void pairs(f32x2 (&v)[1]) const { v[0] = pack2(ld(&x), 0.f); }
};

// x sigmoid(x) of two values.  Below -126 ln 2 the exponential passes rcp's range: the result is
// then 0 where it is above -2^-118.
SDM_DEV f32x2 silu2(f32x2 x) {
    const f32x2 e = exp2_pair(mul2(x, dup2(-kLog2e)));
    return mul2(x, rcp_pair(add2(e, dup2(1.f))));
}

// d/dx (x sigmoid(x)) = s + x s (1 - s) of two values, s = sigmoid(x).
SDM_DEV f32x2 dsilu2(f32x2 x) {
    const f32x2 s = rcp_pair(add2(exp2_pair(mul2(x, dup2(-kLog2e))), dup2(1.f)));
    const f32x2 r = fma2(s, dup2(-1.f), dup2(1.f));
    return fma2(mul2(x, s), r, s);
}

// log(1 + e^x) = max(x, 0) + log(1 + e), e = e^-|x| <= 1, to a few units in the last place: a
// step's relative error goes into every state and gradient behind it, so small steps (x << 0)
// keep theirs.  log(1 + e) = 2 atanh(w), w = e / (2 + e) <= 1/3; 2 atanh(w) / w is a polynomial of
// degree 4 in w^2, fitted at Chebyshev nodes (relative error 4e-9).  The rounding of
// |x| log2(e), which would cost e up to |x| 2^-24, is put back to first order.
SDM_DEV f32x2 softplus2(f32x2 x) {
    float x0, x1;
    unpack2(x, x0, x1);
    const f32x2 a = pack2(min_nan(fabsf(x0), 128.f), min_nan(fabsf(x1), 128.f));  // e is 0 there
    const f32x2 p = mul2(a, dup2(-kLog2e));
    f32x2 lo = fma2(a, dup2(kLog2e), p);
    lo = fma2(a, dup2(1.925963033500e-8f), lo);  // log2(e) - its fp32 value
    f32x2 e = exp2_pair(p);
    e = fma2(e, mul2(lo, dup2(-0.69314718f)), e);
    const f32x2 w = mul2(e, rcp_pair(add2(e, dup2(2.f)))), q = mul2(w, w);
    f32x2 s = fma2(dup2(0.2817465662956238f), q, dup2(0.2796141803264618f));
    s = fma2(s, q, dup2(0.40024852752685547f));
    s = fma2(s, q, dup2(0.6666631698608398f));
    s = fma2(s, q, dup2(2.f));
    s = mul2(s, w);
    return add2(pack2(max_nan(x0, 0.f), max_nan(x1, 0.f)), s);
}
SDM_DEV float softplus(float x) {
    float lo, hi;
    unpack2(softplus2(dup2(x)), lo, hi);
    return lo;
}

// Asynchronous copy of BYTES (4, 8 or 16) to shared memory, of which the first n are read and the
// rest set to zero.
template <int BYTES>
SDM_DEV void async_copy(void* dst, const void* src, int n) {
    const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst);
    if (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(src), "r"(n)
                     : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %3, %2;" ::"r"(d), "l"(src), "r"(n),
                     "n"(BYTES)
                     : "memory");
}
SDM_DEV void async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
SDM_DEV void async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
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
