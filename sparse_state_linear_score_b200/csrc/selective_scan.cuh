// Selective state-space scan, D channels of N states (B and C shared by a group's channels):
//   s_t = softplus(delta_t + dt_bias),  h_t[n] = exp(s_t A[n]) h_{t-1}[n] + s_t B_t[n] u_t,
//   y_t = (sum_n C_t[n] h_t[n] + Dskip u_t) z_t sigmoid(z_t)
//
// Per token and channel: one exponential, one product and three multiply-adds a state, against
// four activations of memory traffic.  At N = 16 in bf16 that is bound by the exponential unit
// (16 a clock and SM: 148 SMs at 1.9 GHz make 4.5e12 a second), about three times above the
// memory's time.  So: the states live in registers over the whole run, NPT a thread, LN
// neighbouring lanes a channel; products and multiply-adds go two states at a time (f32x2);
// B and C, the same for all channels of a block, are staged in shared memory as fp32; what a
// token needs once a channel (softplus, gate, the output's rounding) is split over the channel's
// lanes, token i of a group of 8 on lane i % LN.
//
// Where the channels alone do not fill the GPU the tokens are split into chunks: the decay over a
// chunk is exp(A sum s), so a chunk's effect on the state is its end state from zero and the sum
// of its steps.  scan_chunk_kernel computes those (the exponentials once more), scan_carry_kernel
// chains them, and scan_out_kernel starts every chunk from its true state.
#pragma once

#include "ssm_util.cuh"

namespace sdm {
namespace ssm {

constexpr int SCAN_THREADS = 128;
constexpr int SCAN_TILE = 16;  // tokens of B and C staged at a time
constexpr int SCAN_GRP = 8;    // tokens whose activations are loaded together

template <typename T>
struct ScanArgs {
    View<const T> u, delta, z, Bm, Cm, dy;
    View<T> y;
    const float *A, *Dskip, *dt_bias;
    float* state;
    const int* lens;
    float* E;     // [B][nchunk][D][N] states: a chunk's end from zero, then its start
    float* R;     // the same for the gradient's carry (backward), or null
    float* S;     // [B][nchunk][D] sums of steps
    const float* dstate_end;
    int B, T_, D, N, G, softplus, fresh;
    int chunk, nchunk;  // tokens of a chunk
};

// ---- two fp32 at a time --------------------------------------------------------------------
typedef unsigned long long f32x2;
SDM_DEV f32x2 pack2(float lo, float hi) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
SDM_DEV void unpack2(f32x2 v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
SDM_DEV f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
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

// Sums v[i], i < 8, over LN neighbouring lanes; lane l of them ends with token k*LN + l in v[k].
template <int LN>
SDM_DEV void spread_sum(float (&v)[SCAN_GRP], int nl) {
    int cnt = SCAN_GRP;
#pragma unroll
    for (int bit = 1; bit < LN; bit <<= 1) {
        cnt >>= 1;
        const bool up = nl & bit;
#pragma unroll
        for (int k = 0; k < SCAN_GRP / 2; ++k)
            if (k < cnt) {
                const float mine = up ? v[2 * k + 1] : v[2 * k];
                const float other = up ? v[2 * k] : v[2 * k + 1];
                v[k] = mine + __shfl_xor_sync(0xffffffffu, other, bit);
            }
    }
}

// One tile of B (and C) in flight: loaded to registers while the tile before is used, then
// stored to shared memory as fp32, zero behind t1 and N.
template <typename T, int NN, int WITH_C, int THREADS>
struct BCTile {
    static constexpr int W = NN * (1 + WITH_C);
    static constexpr int PER = (SCAN_TILE * W + THREADS - 1) / THREADS;
    float r[PER];
    SDM_DEV void load(const T* Bp, long long bst, const T* Cp, long long cst, int t, int t1, int N) {
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const int e = threadIdx.x + k * THREADS;
            const int i = e / W, c = e % W, n = c % NN;
            r[k] = 0.f;
            if (e < SCAN_TILE * W && t + i < t1 && n < N)
                r[k] = c < NN ? ld(Bp + (t + i) * bst + n) : ld(Cp + (t + i) * cst + n);
        }
    }
    SDM_DEV void put(float* s) const {
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const int e = threadIdx.x + k * THREADS;
            if (e < SCAN_TILE * W) s[e] = r[k];
        }
    }
};

// The states a block's thread holds: channel c of group g, states n0 .. n0+NPT-1.
template <int NPT, int LN>
struct ScanLane {
    int g, c, nl, n0, b;
    bool live;
    SDM_DEV ScanLane(int D, int G) {
        const int cb = SCAN_THREADS / LN, dg = D / G, tiles = (dg + cb - 1) / cb;
        g = blockIdx.x / tiles;
        const int cg = (blockIdx.x % tiles) * cb + threadIdx.x / LN;
        live = cg < dg;
        c = g * dg + (live ? cg : 0);
        nl = threadIdx.x % LN;
        n0 = nl * NPT;
        b = blockIdx.z;
    }
    SDM_DEV void load(const float* p, int N, float (&v)[NPT]) const {  // p: the channel's row
        if (N % 4 == 0) {  // rows of whole 16-byte pieces
#pragma unroll
            for (int i = 0; i < NPT; i += 4)
                if (live && n0 + i < N) {
                    const float4 x = *reinterpret_cast<const float4*>(p + n0 + i);
                    v[i] = x.x, v[i + 1] = x.y, v[i + 2] = x.z, v[i + 3] = x.w;
                } else {
                    v[i] = v[i + 1] = v[i + 2] = v[i + 3] = 0.f;
                }
        } else {
#pragma unroll
            for (int i = 0; i < NPT; ++i) v[i] = live && n0 + i < N ? p[n0 + i] : 0.f;
        }
    }
    SDM_DEV void store(float* p, int N, const float (&v)[NPT]) const {
        if (!live) return;
        if (N % 4 == 0) {
#pragma unroll
            for (int i = 0; i < NPT; i += 4)
                if (n0 + i < N)
                    *reinterpret_cast<float4*>(p + n0 + i) =
                        make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
        } else {
#pragma unroll
            for (int i = 0; i < NPT; ++i)
                if (n0 + i < N) p[n0 + i] = v[i];
        }
    }
};

// A chunk's end state from zero, the sum of its steps and (REV) what its outputs' gradients
// carry to the token before it: sum_t (prod_{s<=t} a_s) C_t dy_t.
template <typename T, int NPT, int LN, bool REV>
__global__ void __launch_bounds__(SCAN_THREADS) scan_chunk_kernel(ScanArgs<T> a) {
    constexpr int NN = NPT * LN, OWN = SCAN_GRP / LN, NP = NPT / 2, W = NN * (1 + REV);
    __shared__ __align__(16) float s_bc[2][SCAN_TILE * W];
    const ScanLane<NPT, LN> L(a.D, a.G);
    const int lane = threadIdx.x & 31;
    const int len = clamp_len(a.lens, L.b, a.T_);
    const int t0 = blockIdx.y * a.chunk, t1 = min(t0 + a.chunk, len);
    const T* up = a.u.p + L.b * a.u.sb + L.c;
    const T* dp = a.delta.p + L.b * a.delta.sb + L.c;
    const T* zp = REV && a.z.p ? a.z.p + L.b * a.z.sb + L.c : nullptr;
    const T* yp = REV ? a.dy.p + L.b * a.dy.sb + L.c : nullptr;
    const T* Bp = a.Bm.p + L.b * a.Bm.sb + L.g * a.Bm.sh;
    const T* Cp = REV ? a.Cm.p + L.b * a.Cm.sb + L.g * a.Cm.sh : nullptr;
    float tmp[NPT];
    f32x2 A2[NP], h[NP], r[NP], P[NP];
    L.load(a.A + (long long)L.c * a.N, a.N, tmp);
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        A2[i] = pack2(tmp[2 * i] * kLog2e, tmp[2 * i + 1] * kLog2e);
        h[i] = r[i] = pack2(0.f, 0.f);
        P[i] = pack2(1.f, 1.f);
    }
    const float bias = a.dt_bias ? a.dt_bias[L.c] : 0.f;
    float steps = 0.f;
    BCTile<T, NN, REV, SCAN_THREADS> bc;
    bc.load(Bp, a.Bm.st, Cp, a.Cm.st, t0, t1, a.N);
    bc.put(s_bc[0]);
    __syncthreads();
    int buf = 0;
    for (int tt = t0; tt < t1; tt += SCAN_TILE) {
        if (tt + SCAN_TILE < t1)
            bc.load(Bp, a.Bm.st, Cp, a.Cm.st, tt + SCAN_TILE, t1, a.N);
#pragma unroll
        for (int gq = 0; gq < SCAN_TILE / SCAN_GRP; ++gq) {
            const int tg = tt + gq * SCAN_GRP;
            float dt[OWN], dtu[OWN], gy[OWN];
#pragma unroll
            for (int k = 0; k < OWN; ++k) {
                const int t = tg + k * LN + L.nl;
                dt[k] = dtu[k] = gy[k] = 0.f;
                if (t < t1 && L.live) {
                    const float d = ld(dp + t * a.delta.st) + bias;
                    dt[k] = a.softplus ? softplus(d) : d;
                    dtu[k] = dt[k] * ld(up + t * a.u.st);
                    if (REV) {
                        gy[k] = ld(yp + t * a.dy.st);
                        if (zp) {
                            const float z = ld(zp + t * a.z.st);
                            gy[k] *= z * sigmoid(z);
                        }
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < SCAN_GRP; ++i) {
                float d = dt[i / LN], e = dtu[i / LN], y = gy[i / LN];
                if (LN > 1) {
                    const int src = (lane & ~(LN - 1)) | (i % LN);
                    d = __shfl_sync(0xffffffffu, d, src);
                    e = __shfl_sync(0xffffffffu, e, src);
                    if (REV) y = __shfl_sync(0xffffffffu, y, src);
                }
                steps += d;
                const f32x2 d2 = pack2(d, d), e2 = pack2(e, e), y2 = pack2(y, y);
                const float* row = s_bc[buf] + (gq * SCAN_GRP + i) * W + L.n0;
                const f32x2* Br = reinterpret_cast<const f32x2*>(row);
                const f32x2* Cr = reinterpret_cast<const f32x2*>(row + NN);
#pragma unroll
                for (int p = 0; p < NP; ++p) {
                    const f32x2 dec = exp2_pair(mul2(d2, A2[p]));
                    h[p] = fma2(dec, h[p], mul2(e2, Br[p]));
                    if (REV) {
                        P[p] = mul2(P[p], dec);
                        r[p] = fma2(P[p], mul2(y2, Cr[p]), r[p]);
                    }
                }
            }
        }
        if (tt + SCAN_TILE < t1) {
            buf ^= 1;  // last read before the barrier that ended the tile before this one
            bc.put(s_bc[buf]);
            __syncthreads();
        }
    }
    const long long at = ((long long)L.b * a.nchunk + blockIdx.y) * a.D + L.c;
#pragma unroll
    for (int i = 0; i < NP; ++i) unpack2(h[i], tmp[2 * i], tmp[2 * i + 1]);
    L.store(a.E + at * a.N, a.N, tmp);
    if (REV) {
#pragma unroll
        for (int i = 0; i < NP; ++i) unpack2(r[i], tmp[2 * i], tmp[2 * i + 1]);
        L.store(a.R + at * a.N, a.N, tmp);
    }
    if (L.live && L.nl == 0) a.S[at] = steps;
}

// Chains the chunks: E[k] becomes the state that chunk k starts from and, in the gradient, R[k]
// the carry that reaches its last token.  One thread a state; the loads of SCAN_AHEAD chunks are
// in flight together.
constexpr int SCAN_AHEAD = 8;
template <typename T>
__global__ void __launch_bounds__(256) scan_carry_kernel(ScanArgs<T> a, int rev) {
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    const long long dn = (long long)a.D * a.N;
    if (i >= a.B * dn) return;
    const long long b = i / dn, cn = i % dn;
    const float A2 = a.A[cn] * kLog2e;
    float* E = (rev ? a.R : a.E) + b * a.nchunk * dn + cn;
    const float* S = a.S + b * a.nchunk * a.D + cn / a.N;
    float h = 0.f;
    if (rev) {
        if (a.dstate_end) h = a.dstate_end[i];
    } else if (a.state && !a.fresh) {
        h = a.state[i];
    }
    for (int k = 0; k < a.nchunk; k += SCAN_AHEAD) {
        float e[SCAN_AHEAD], s[SCAN_AHEAD];
#pragma unroll
        for (int q = 0; q < SCAN_AHEAD; ++q)
            if (k + q < a.nchunk - 1) {  // the last chunk's effect is not needed
                const long long at = rev ? a.nchunk - 1 - (k + q) : k + q;
                e[q] = E[at * dn];
                s[q] = S[at * a.D];
            }
#pragma unroll
        for (int q = 0; q < SCAN_AHEAD; ++q)
            if (k + q < a.nchunk) {
                const long long at = rev ? a.nchunk - 1 - (k + q) : k + q;
                E[at * dn] = h;
                if (k + q < a.nchunk - 1) h = fmaf(exp2_fast(s[q] * A2), h, e[q]);
            }
    }
}

// The outputs of a chunk (the whole call when nchunk is 1) from its start state.
template <typename T, int NPT, int LN>
__global__ void __launch_bounds__(SCAN_THREADS) scan_out_kernel(ScanArgs<T> a) {
    constexpr int NN = NPT * LN, OWN = SCAN_GRP / LN, NP = NPT / 2, W = 2 * NN;
    __shared__ __align__(16) float s_bc[2][SCAN_TILE * W];
    const ScanLane<NPT, LN> L(a.D, a.G);
    const int lane = threadIdx.x & 31;
    const int len = clamp_len(a.lens, L.b, a.T_);
    const int t0 = blockIdx.y * a.chunk, t1 = min(t0 + a.chunk, len);
    if (t0 >= len && blockIdx.y > 0) return;
    const T* up = a.u.p + L.b * a.u.sb + L.c;
    const T* dp = a.delta.p + L.b * a.delta.sb + L.c;
    const T* zp = a.z.p ? a.z.p + L.b * a.z.sb + L.c : nullptr;
    T* yp = a.y.p + L.b * a.y.sb + L.c;
    const T* Bp = a.Bm.p + L.b * a.Bm.sb + L.g * a.Bm.sh;
    const T* Cp = a.Cm.p + L.b * a.Cm.sb + L.g * a.Cm.sh;
    float* state = a.state ? a.state + ((long long)L.b * a.D + L.c) * a.N : nullptr;
    float tmp[NPT];
    f32x2 A2[NP], h[NP];
    L.load(a.A + (long long)L.c * a.N, a.N, tmp);
#pragma unroll
    for (int i = 0; i < NP; ++i) A2[i] = pack2(tmp[2 * i] * kLog2e, tmp[2 * i + 1] * kLog2e);
#pragma unroll
    for (int i = 0; i < NPT; ++i) tmp[i] = 0.f;
    if (a.nchunk > 1)
        L.load(a.E + (((long long)L.b * a.nchunk + blockIdx.y) * a.D + L.c) * a.N, a.N, tmp);
    else if (state && !a.fresh)
        L.load(state, a.N, tmp);
#pragma unroll
    for (int i = 0; i < NP; ++i) h[i] = pack2(tmp[2 * i], tmp[2 * i + 1]);
    const float bias = a.dt_bias ? a.dt_bias[L.c] : 0.f;
    const float skip = a.Dskip ? a.Dskip[L.c] : 0.f;
    BCTile<T, NN, 1, SCAN_THREADS> bc;
    bc.load(Bp, a.Bm.st, Cp, a.Cm.st, t0, t1, a.N);
    bc.put(s_bc[0]);
    __syncthreads();
    int buf = 0;
    float un[OWN], dn[OWN], zn[OWN];  // the next group's activations
    auto fetch = [&](int tg) {
#pragma unroll
        for (int k = 0; k < OWN; ++k) {
            const int t = tg + k * LN + L.nl;
            un[k] = dn[k] = zn[k] = 0.f;
            if (t < t1 && L.live) {
                un[k] = ld(up + t * a.u.st);
                dn[k] = ld(dp + t * a.delta.st);
                if (zp) zn[k] = ld(zp + t * a.z.st);
            }
        }
    };
    fetch(t0);
    for (int tt = t0; tt < t1; tt += SCAN_TILE) {
        if (tt + SCAN_TILE < t1)
            bc.load(Bp, a.Bm.st, Cp, a.Cm.st, tt + SCAN_TILE, t1, a.N);
#pragma unroll
        for (int gq = 0; gq < SCAN_TILE / SCAN_GRP; ++gq) {
            const int tg = tt + gq * SCAN_GRP;
            float u[OWN], z[OWN], dt[OWN], dtu[OWN], y[SCAN_GRP];
#pragma unroll
            for (int k = 0; k < OWN; ++k) {
                const float d = dn[k] + bias;
                u[k] = un[k];
                z[k] = zn[k];
                // a token behind the sequence: step 0, the state stays
                dt[k] = tg + k * LN + L.nl < t1 ? (a.softplus ? softplus(d) : d) : 0.f;
                dtu[k] = dt[k] * u[k];
            }
            fetch(tg + SCAN_GRP);
#pragma unroll
            for (int i = 0; i < SCAN_GRP; ++i) {
                float d = dt[i / LN], e = dtu[i / LN];
                if (LN > 1) {
                    const int src = (lane & ~(LN - 1)) | (i % LN);
                    d = __shfl_sync(0xffffffffu, d, src);
                    e = __shfl_sync(0xffffffffu, e, src);
                }
                const f32x2 d2 = pack2(d, d), e2 = pack2(e, e);
                const float* row = s_bc[buf] + (gq * SCAN_GRP + i) * W + L.n0;
                const f32x2* Br = reinterpret_cast<const f32x2*>(row);
                const f32x2* Cr = reinterpret_cast<const f32x2*>(row + NN);
                f32x2 acc = pack2(0.f, 0.f);
#pragma unroll
                for (int p = 0; p < NP; ++p) {
                    h[p] = fma2(exp2_pair(mul2(d2, A2[p])), h[p], mul2(e2, Br[p]));
                    acc = fma2(h[p], Cr[p], acc);
                }
                float lo, hi;
                unpack2(acc, lo, hi);
                y[i] = lo + hi;
            }
            spread_sum<LN>(y, L.nl);
#pragma unroll
            for (int k = 0; k < OWN; ++k) {
                const int t = tg + k * LN + L.nl;
                if (t < t1 && L.live) {
                    float v = fmaf(skip, u[k], y[k]);
                    if (zp) v *= z[k] * sigmoid(z[k]);
                    st(yp + t * a.y.st, v);
                }
            }
        }
        if (tt + SCAN_TILE < t1) {
            buf ^= 1;
            bc.put(s_bc[buf]);
            __syncthreads();
        }
    }
    if (state && t1 == len && (len > t0 || blockIdx.y == 0)) {
#pragma unroll
        for (int i = 0; i < NP; ++i) unpack2(h[i], tmp[2 * i], tmp[2 * i + 1]);
        L.store(state, a.N, tmp);
    }
}

// One token a sequence: bound by the state, read and written once (8 N bytes a channel against
// 8 of activations in bf16).  Four states a thread, so that a warp's state accesses are whole
// contiguous lines.
template <typename T, int LN>
__global__ void __launch_bounds__(256) scan_step_kernel(ScanArgs<T> a) {
    const int nl = threadIdx.x % LN, n0 = nl * 4;
    const int c = blockIdx.x * (256 / LN) + threadIdx.x / LN, b = blockIdx.y;
    const bool live = c < a.D && n0 < a.N;
    const int cc = c < a.D ? c : 0, g = cc / (a.D / a.G);
    const bool on = clamp_len(a.lens, b, 1) > 0;
    const bool vec = a.N % 4 == 0;
    float* state = a.state ? a.state + ((long long)b * a.D + cc) * a.N + n0 : nullptr;
    float h[4] = {0.f, 0.f, 0.f, 0.f}, A[4] = {0.f, 0.f, 0.f, 0.f};
    if (live) {
        const float* Ap = a.A + (long long)cc * a.N + n0;
        if (vec) {
            Vec<4>::load(Ap, A);
            if (state && !a.fresh) Vec<4>::load(state, h);
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (n0 + k < a.N) {
                    A[k] = Ap[k];
                    if (state && !a.fresh) h[k] = state[k];
                }
        }
    }
    if (on) {
        float d = ld(a.delta.p + b * a.delta.sb + cc) + (a.dt_bias ? a.dt_bias[cc] : 0.f);
        if (a.softplus) d = softplus(d);
        const float u = ld(a.u.p + b * a.u.sb + cc);
        const T* Bp = a.Bm.p + b * a.Bm.sb + g * a.Bm.sh + n0;
        const T* Cp = a.Cm.p + b * a.Cm.sb + g * a.Cm.sh + n0;
        float y = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (live && n0 + k < a.N) {
                h[k] = fmaf(exp2_fast(d * (A[k] * kLog2e)), h[k], d * u * ld(Bp + k));
                y = fmaf(h[k], ld(Cp + k), y);
            }
#pragma unroll
        for (int m = 1; m < LN; m <<= 1) y += __shfl_xor_sync(0xffffffffu, y, m);
        if (nl == 0 && c < a.D) {
            if (a.Dskip) y = fmaf(a.Dskip[cc], u, y);
            if (a.z.p) {
                const float z = ld(a.z.p + b * a.z.sb + cc);
                y *= z * sigmoid(z);
            }
            st(a.y.p + b * a.y.sb + cc, y);
        }
    }
    if (state && live && (on || a.fresh)) {
        if (vec) {
            Vec<4>::store(state, h);
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (n0 + k < a.N) state[k] = h[k];
        }
    }
}

}  // namespace ssm
}  // namespace sdm
