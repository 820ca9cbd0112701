// The norms around a block with its gate and residual scale, over rows of D values:
//   p = f rf w_post,  rf = (mean f^2 + eps)^-1/2      o = r + scale sigmoid(gate) p
//   r_out = o,        n = o ro w_pre,  ro = (mean o^2 + eps)^-1/2
// and its gradient, with dn w_pre = m, o^ = o ro, f^ = f rf:
//   do = dr_out + ro (m - o^ mean(m o^)),  dr = do
//   dp = do scale sigmoid(gate),  q = dp w_post,  df = rf (q - f^ mean(q f^))
//   dgate = do scale p s (1-s),  dscale = sum do s p,  dw_post = sum dp f^,  dw_pre = sum dn o^
//
// Bound by memory.  A block of at most 512 threads takes whole rows of up to 4096 columns; a row is
// read once into registers (so r_out may be r) and normalised in place, eight values a thread as
// pairs (f32x2); the weights come from L1 after the first row.  Wider rows go in passes over their
// columns (see there; clusters of blocks with the row in registers took three times as long, since
// each of a cluster's barriers waits for the stores before it).  The sums of a row (two reductions;
// the gradient one, see there) are sums over the block's warps in fp32.  What hides the loads'
// latency: two blocks an SM (four, wide) that wait in turn, or (gradient, whose registers allow only
// one) the next row's loads issued ahead.
// Measured: 8192 rows of 4096, r and f fp32, gate and n bf16, 95 us, 5.3 TB/s; gradient of 4099 rows,
// all bf16, 72 us, 3.6 TB/s (a row's latency at one block an SM); 3395 rows of 8192, bf16, 69 us, 4.0
// TB/s, gradient 192 us, 2.3 TB/s; odd widths, 4096 rows of 4095, 69 and 165 us.
#pragma once

#include "ssm_util.cuh"

namespace sdm {
namespace ssm {

constexpr int NORM_THREADS = 512;
constexpr int NORM_COLS = 4096;  // columns that a block keeps in registers
constexpr int NORM_WIDE = 256;   // threads that take a wider row, forward

struct NormArgs {
    const void *r, *f, *gate, *dr_out, *dn;
    void *r_out, *n, *dr, *df, *dgate;  // r_out, n: forward
    const float *w_post, *scale, *w_pre;
    float* part;  // backward: [row groups][3][D] (dscale, dw_post, dw_pre)
    long long rows;
    int D, rb, fb, xb;  // 1: bf16
    float eps;
};

constexpr int NORM_V = 4, NORM_P = 2;  // values of a piece, pieces of a thread

// A piece of a row as it is stored, in registers until it is used: a block's loads are all in flight
// before the first is waited for.  VEC: D is a multiple of four, so pieces are whole and aligned;
// else they are loaded value by value, `cnt` of them.
template <bool VEC>
struct NormRaw {
    uint32_t x[4];
    SDM_DEV void clear() {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = 0u;
    }
    SDM_DEV void load(const void* p, bool is_bf16, long long at, int cnt) {
        if (VEC) {
            if (is_bf16) {
                const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const bf16*>(p) + at);
                x[0] = v.x, x[1] = v.y;
            } else {
                const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const float*>(p) + at);
                x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < cnt)
                    x[i] = is_bf16 ? static_cast<const uint16_t*>(p)[at + i]
                                   : static_cast<const uint32_t*>(p)[at + i];
        }
    }
    SDM_DEV void get(bool is_bf16, f32x2 (&v)[2]) const {
        if (!is_bf16) {
            v[0] = pack2(__uint_as_float(x[0]), __uint_as_float(x[1]));
            v[1] = pack2(__uint_as_float(x[2]), __uint_as_float(x[3]));
        } else if (VEC) {
            v[0] = pack2(bf16_lo(x[0]), bf16_hi(x[0]));
            v[1] = pack2(bf16_lo(x[1]), bf16_hi(x[1]));
        } else {
            v[0] = pack2(bf16_lo(x[0]), bf16_lo(x[1]));
            v[1] = pack2(bf16_lo(x[2]), bf16_lo(x[3]));
        }
    }
};
template <bool VEC>
SDM_DEV void norm_store(void* p, bool is_bf16, long long at, int cnt, const f32x2 (&v)[2]) {
    float x[4];
    unpack2(v[0], x[0], x[1]);
    unpack2(v[1], x[2], x[3]);
    if (VEC) {
        if (is_bf16) Vec<4>::store(static_cast<bf16*>(p) + at, x);
        else Vec<4>::store(static_cast<float*>(p) + at, x);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < cnt) {
                if (is_bf16) st(static_cast<bf16*>(p) + at + i, x[i]);
                else st(static_cast<float*>(p) + at + i, x[i]);
            }
    }
}
// A piece of a weight vector (1 where there is none).
template <bool VEC>
SDM_DEV void norm_weight(bool has, const float* w, int c, int cnt, f32x2 (&v)[2]) {
    v[0] = v[1] = dup2(1.f);
    if (!has) return;
    if (VEC || cnt == 4) {  // c is a multiple of four
        const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(w + c);
        v[0] = x.x, v[1] = x.y;
    } else {
        v[0] = pack2(w[c], cnt > 1 ? w[c + 1] : 1.f);
        v[1] = pack2(cnt > 2 ? w[c + 2] : 1.f, 1.f);
    }
}
SDM_DEV float sum2(f32x2 v) {
    float lo, hi;
    unpack2(v, lo, hi);
    return lo + hi;
}
SDM_DEV f32x2 sigmoid2(f32x2 x) {
    return rcp_pair(add2(exp2_pair(mul2(x, dup2(-kLog2e))), dup2(1.f)));
}

// Sums over a block, which alternate between two slots: one barrier each is enough, since a
// slot is written again only behind the barrier of the reduction after the one that read it.
constexpr int NORM_SUMS = 8;
struct NormSums {
    float s[2][NORM_SUMS][16];  // of every warp; zero where there is none
    SDM_DEV void clear() {
        float* p = &s[0][0][0];
        for (int i = threadIdx.x; i < 2 * NORM_SUMS * 16; i += blockDim.x) p[i] = 0.f;
    }
};
struct RowSum {
    NormSums& m;
    int slot;
    // v[0..K) to every thread: over the lanes by shuffles that halve the values with each step, lane
    // i ending with value i; over the warps four lanes a value.
    template <int K>
    SDM_DEV void sum(float (&v)[K]) {
        static_assert(K <= NORM_SUMS, "sums");
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        float x[NORM_SUMS];
#pragma unroll
        for (int k = 0; k < NORM_SUMS; ++k) x[k] = k < K ? v[k < K ? k : 0] : 0.f;
        if (K == 1) {
            x[0] = warp_sum(x[0]);
        } else {
            int cnt = NORM_SUMS;
#pragma unroll
            for (int bit = 1; bit < NORM_SUMS; bit <<= 1) {
                cnt >>= 1;
                const bool up = lane & bit;
#pragma unroll
                for (int k = 0; k < NORM_SUMS / 2; ++k)
                    if (k < cnt) {
                        const float mine = up ? x[2 * k + 1] : x[2 * k];
                        const float other = up ? x[2 * k] : x[2 * k + 1];
                        x[k] = mine + __shfl_xor_sync(0xffffffffu, other, bit);
                    }
            }
            x[0] += __shfl_xor_sync(0xffffffffu, x[0], 8);
            x[0] += __shfl_xor_sync(0xffffffffu, x[0], 16);
        }
        if (lane < K) m.s[slot][lane][warp] = x[0];
        __syncthreads();
        const float4 q = *reinterpret_cast<const float4*>(&m.s[slot][lane >> 2][(lane & 3) * 4]);
        float t = (q.x + q.y) + (q.z + q.w);
        t += __shfl_xor_sync(0xffffffffu, t, 1);
        t += __shfl_xor_sync(0xffffffffu, t, 2);
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] = __shfl_sync(0xffffffffu, t, 4 * k);
        slot ^= 1;
    }
};

// Piece i of thread t starts at column (i*blockDim + t)*4.  DT: which of r, f, x are bf16 (bits 0,
// 1, 2), or -1: as the arguments say.  ALL: no argument is missing.
template <bool VEC, int DT, bool ALL>
__global__ void __launch_bounds__(NORM_THREADS, 2) block_norm_kernel(NormArgs a) {
    constexpr int P = NORM_P, N = 2;
    __shared__ __align__(16) NormSums s_sum;
    const bool rb = DT < 0 ? a.rb : DT & 1, fb = DT < 0 ? a.fb : DT & 2, xb = DT < 0 ? a.xb : DT & 4;
    const bool has_gate = ALL || a.gate, has_post = ALL || a.w_post, has_scale = ALL || a.scale,
               has_pre = ALL || a.w_pre, out_r = ALL || a.r_out, out_n = ALL || a.n;
    RowSum red{s_sum, 0};
    s_sum.clear();
    __syncthreads();
    const float inv_d = 1.f / (float)a.D;
    for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const long long base = row * a.D;
        NormRaw<VEC> rf[P], rr[P], rg[P];
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int c = (i * blockDim.x + threadIdx.x) * NORM_V, cnt = min(NORM_V, a.D - c);
            rf[i].clear();
            rr[i].clear();
            rg[i].clear();
            if (c < a.D) {
                rf[i].load(a.f, fb, base + c, cnt);
                rr[i].load(a.r, rb, base + c, cnt);
                if (has_gate) rg[i].load(a.gate, xb, base + c, cnt);
            }
        }
        f32x2 f[P][N], o[P][N], s2 = dup2(0.f);
        float ss[1];
#pragma unroll
        for (int i = 0; i < P; ++i) {
            rf[i].get(fb, f[i]);
#pragma unroll
            for (int v = 0; v < N; ++v) s2 = fma2(f[i][v], f[i][v], s2);
        }
        f32x2 k = dup2(1.f);
        if (has_post) {
            ss[0] = sum2(s2);
            red.sum(ss);
            k = dup2(rsqrtf(ss[0] * inv_d + a.eps));
        }
        s2 = dup2(0.f);
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int c = (i * blockDim.x + threadIdx.x) * NORM_V, cnt = min(NORM_V, a.D - c);
            if (c < a.D) {
                f32x2 wp[N], sc[N], g[N];
                norm_weight<VEC>(has_post, a.w_post, c, cnt, wp);
                norm_weight<VEC>(has_scale, a.scale, c, cnt, sc);
                rg[i].get(xb, g);
                rr[i].get(rb, o[i]);
#pragma unroll
                for (int v = 0; v < N; ++v) {
                    f32x2 m = mul2(mul2(sc[v], wp[v]), k);
                    if (has_gate) m = mul2(m, sigmoid2(g[v]));
                    o[i][v] = fma2(m, f[i][v], o[i][v]);
                    s2 = fma2(o[i][v], o[i][v], s2);
                }
                if (out_r) norm_store<VEC>(a.r_out, rb, base + c, cnt, o[i]);
            }
        }
        if (!out_n) continue;
        ss[0] = sum2(s2);
        red.sum(ss);
        k = dup2(rsqrtf(ss[0] * inv_d + a.eps));
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int c = (i * blockDim.x + threadIdx.x) * NORM_V, cnt = min(NORM_V, a.D - c);
            if (c < a.D) {
                f32x2 wq[N];
                norm_weight<VEC>(has_pre, a.w_pre, c, cnt, wq);
#pragma unroll
                for (int v = 0; v < N; ++v) o[i][v] = mul2(o[i][v], mul2(k, wq[v]));
                norm_store<VEC>(a.n, xb, base + c, cnt, o[i]);
            }
        }
    }
}

// Rows of more than 4096 columns: a block takes a row in passes over its columns, each thread the
// same ones in every pass, with the row as floats in shared memory between them: f and the sum of
// its squares; o, which replaces f, r_out and the sum of o's squares; n.
constexpr int NORM_U = 4;  // pieces whose loads are in flight together
template <bool VEC>
__global__ void __launch_bounds__(NORM_WIDE, 4) block_norm_wide_kernel(NormArgs a) {
    constexpr int U = NORM_U, H = NORM_U / 2;
    extern __shared__ __align__(16) char smem[];
    __shared__ __align__(16) NormSums s_sum;
    ulonglong2* kept = reinterpret_cast<ulonglong2*>(smem);  // a piece each
    const bool rb = a.rb, fb = a.fb, xb = a.xb;
    const bool has_gate = a.gate, has_post = a.w_post, has_scale = a.scale;
    RowSum red{s_sum, 0};
    s_sum.clear();
    __syncthreads();
    const float inv_d = 1.f / (float)a.D;
    const int S = NORM_WIDE * NORM_V, first = threadIdx.x * NORM_V;
    for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const long long base = row * a.D;
        f32x2 s2 = dup2(0.f);
        float ss[1];
        for (int c0 = first; c0 < a.D; c0 += U * S) {
            NormRaw<VEC> rf[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int c = c0 + u * S;
                rf[u].clear();
                if (c < a.D) rf[u].load(a.f, fb, base + c, min(NORM_V, a.D - c));
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int c = c0 + u * S;
                f32x2 f[2];
                rf[u].get(fb, f);
                s2 = fma2(f[0], f[0], s2);
                s2 = fma2(f[1], f[1], s2);
                if (c < a.D) kept[c / NORM_V] = make_ulonglong2(f[0], f[1]);
            }
        }
        f32x2 k = dup2(1.f);
        if (has_post) {
            ss[0] = sum2(s2);
            red.sum(ss);
            k = dup2(rsqrtf(ss[0] * inv_d + a.eps));
        }
        s2 = dup2(0.f);
        for (int c0 = first; c0 < a.D; c0 += H * S) {
            NormRaw<VEC> rr[H], rg[H];
#pragma unroll
            for (int u = 0; u < H; ++u) {
                const int c = c0 + u * S, cnt = min(NORM_V, a.D - c);
                rr[u].clear();
                rg[u].clear();
                if (c < a.D) {
                    rr[u].load(a.r, rb, base + c, cnt);
                    if (has_gate) rg[u].load(a.gate, xb, base + c, cnt);
                }
            }
#pragma unroll
            for (int u = 0; u < H; ++u) {
                const int c = c0 + u * S, cnt = min(NORM_V, a.D - c);
                if (c >= a.D) continue;
                f32x2 wp[2], sc[2], g[2], o[2];
                norm_weight<VEC>(has_post, a.w_post, c, cnt, wp);
                norm_weight<VEC>(has_scale, a.scale, c, cnt, sc);
                rg[u].get(xb, g);
                rr[u].get(rb, o);
                const ulonglong2 f = kept[c / NORM_V];
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    f32x2 m = mul2(mul2(sc[v], wp[v]), k);
                    if (has_gate) m = mul2(m, sigmoid2(g[v]));
                    o[v] = fma2(m, v ? f.y : f.x, o[v]);
                    s2 = fma2(o[v], o[v], s2);
                }
                if (a.r_out) norm_store<VEC>(a.r_out, rb, base + c, cnt, o);
                kept[c / NORM_V] = make_ulonglong2(o[0], o[1]);
            }
        }
        if (!a.n) continue;
        ss[0] = sum2(s2);
        red.sum(ss);
        k = dup2(rsqrtf(ss[0] * inv_d + a.eps));
#pragma unroll 2
        for (int c = first; c < a.D; c += S) {
            const int cnt = min(NORM_V, a.D - c);
            f32x2 wq[2];
            norm_weight<VEC>(a.w_pre, a.w_pre, c, cnt, wq);
            const ulonglong2 o = kept[c / NORM_V];
            const f32x2 n[2] = {mul2(o.x, mul2(k, wq[0])), mul2(o.y, mul2(k, wq[1]))};
            norm_store<VEC>(a.n, xb, base + c, cnt, n);
        }
    }
}

template <int DT, bool ALL>
__global__ void __launch_bounds__(NORM_THREADS, 1) block_norm_bwd_kernel(NormArgs a) {
    constexpr int P = NORM_P, N = 2;
    __shared__ __align__(16) NormSums s_sum;
    const bool rb = DT & 1, fb = DT & 2, xb = DT & 4;
    const bool has_gate = ALL || a.gate, has_post = ALL || a.w_post, has_scale = ALL || a.scale,
               has_pre = ALL || a.w_pre, has_dn = ALL || a.dn, has_dr = ALL || a.dr_out,
               out_dr = ALL || a.dr, out_df = ALL || a.df, out_dg = ALL || a.dgate;
    RowSum red{s_sum, 0};
    s_sum.clear();
    __syncthreads();
    const f32x2 one = dup2(1.f), zero = dup2(0.f);
    f32x2 aw[P][N], as[P][N], aq[P][N];
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
        for (int v = 0; v < N; ++v) aw[i][v] = as[i][v] = aq[i][v] = zero;
    const float inv_d = 1.f / (float)a.D;
    NormRaw<true> rf[P], rr[P], rg[P], rn[P], rd[P];
    auto fetch = [&](long long row) {
        const long long base = row * a.D;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int c = (i * blockDim.x + threadIdx.x) * NORM_V, cnt = NORM_V;
            rf[i].clear();
            rr[i].clear();
            rg[i].clear();
            rn[i].clear();
            rd[i].clear();
            if (c < a.D && row < a.rows) {
                rf[i].load(a.f, fb, base + c, cnt);
                rr[i].load(a.r, rb, base + c, cnt);
                if (has_gate) rg[i].load(a.gate, xb, base + c, cnt);
                if (has_dn) rn[i].load(a.dn, xb, base + c, cnt);
                if (has_dr) rd[i].load(a.dr_out, rb, base + c, cnt);
            }
        }
    };
    fetch(blockIdx.x);
    // One reduction a row: the sum of the next row's f^2 goes with this row's.  What df needs of the
    // row, mean(q f^) = mean(do a) with a = scale sigmoid(gate) p, follows from the sums of m a, o a
    // and dr_out a, since do = dr_out + ro (m - o^ mean(m o^)).
    auto square = [&]() {
        f32x2 s2 = zero;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            f32x2 f[N];
            rf[i].get(fb, f);
#pragma unroll
            for (int v = 0; v < N; ++v) s2 = fma2(f[v], f[v], s2);
        }
        return sum2(s2);
    };
    float next[1] = {has_post ? square() : 0.f};
    if (has_post) red.sum(next);
    for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const long long base = row * a.D;
        const f32x2 rf1 = has_post ? dup2(rsqrtf(next[0] * inv_d + a.eps)) : one;
        f32x2 f[P][N], o[P][N], g[P][N], dn[P][N], dr[P][N];
        f32x2 so = zero, sm = zero, sma = zero, soa = zero, sda = zero;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            rf[i].get(fb, f[i]);
            rr[i].get(rb, o[i]);
            rg[i].get(xb, g[i]);
            rn[i].get(xb, dn[i]);
            rd[i].get(rb, dr[i]);
        }
        fetch(row + gridDim.x);
        // f becomes f^ (f itself without the norm), g the gate's sigmoid
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int c = (i * blockDim.x + threadIdx.x) * NORM_V, cnt = NORM_V;
            if (c >= a.D) continue;
            f32x2 wp[N], sc[N], wq[N];
            norm_weight<true>(has_post, a.w_post, c, cnt, wp);
            norm_weight<true>(has_scale, a.scale, c, cnt, sc);
            norm_weight<true>(has_pre, a.w_pre, c, cnt, wq);
#pragma unroll
            for (int v = 0; v < N; ++v) {
                f[i][v] = mul2(f[i][v], rf1);
                g[i][v] = has_gate ? sigmoid2(g[i][v]) : one;
                const f32x2 k = mul2(mul2(sc[v], g[i][v]), mul2(f[i][v], wp[v])), m = mul2(dn[i][v], wq[v]);
                o[i][v] = add2(k, o[i][v]);
                so = fma2(o[i][v], o[i][v], so);
                sm = fma2(o[i][v], m, sm);
                sma = fma2(m, k, sma);
                soa = fma2(o[i][v], k, soa);
                sda = fma2(dr[i][v], k, sda);
            }
        }
        f32x2 ro = zero, mo = zero, mf = zero;
        if (has_dn || has_post) {
            float st[6] = {sum2(so), sum2(sm), sum2(sma), sum2(soa), sum2(sda), has_post ? square() : 0.f};
            red.sum(st);
            next[0] = st[5];
            float q = 0.f, mean = 0.f;
            if (has_dn) {
                q = rsqrtf(st[0] * inv_d + a.eps);
                mean = st[1] * q * inv_d;  // mean(m o^)
            }
            ro = dup2(q);
            mo = dup2(-mean);
            if (has_post) mf = dup2(-(st[4] + q * (st[2] - q * mean * st[3])) * inv_d);
        }
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int c = (i * blockDim.x + threadIdx.x) * NORM_V, cnt = NORM_V;
            if (c >= a.D) continue;
            f32x2 wp[N], sc[N], wq[N], dg[N];
            norm_weight<true>(has_post, a.w_post, c, cnt, wp);
            norm_weight<true>(has_scale, a.scale, c, cnt, sc);
            norm_weight<true>(has_pre, a.w_pre, c, cnt, wq);
#pragma unroll
            for (int v = 0; v < N; ++v) {
                const f32x2 oh = mul2(o[i][v], ro);
                aq[i][v] = fma2(dn[i][v], oh, aq[i][v]);
                const f32x2 d = fma2(ro, fma2(dn[i][v], wq[v], mul2(oh, mo)), dr[i][v]);
                dr[i][v] = d;
                const f32x2 ds = mul2(d, g[i][v]);  // do sigmoid(gate)
                const f32x2 dsp = mul2(ds, mul2(f[i][v], wp[v]));
                as[i][v] = add2(as[i][v], dsp);
                dg[v] = mul2(mul2(dsp, sc[v]), fma2(g[i][v], dup2(-1.f), one));
                const f32x2 dp = mul2(ds, sc[v]);
                aw[i][v] = fma2(dp, f[i][v], aw[i][v]);
                o[i][v] = mul2(rf1, fma2(f[i][v], mf, mul2(dp, wp[v])));
            }
            if (out_dr) norm_store<true>(a.dr, rb, base + c, cnt, dr[i]);
            if (out_dg) norm_store<true>(a.dgate, xb, base + c, cnt, dg);
            if (out_df) norm_store<true>(a.df, fb, base + c, cnt, o[i]);
        }
    }
    float* part = a.part + (long long)blockIdx.x * 3 * a.D;
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int c = (i * blockDim.x + threadIdx.x) * NORM_V, cnt = NORM_V;
        if (c < a.D) {
            norm_store<true>(part, false, c, cnt, as[i]);
            norm_store<true>(part, false, (long long)a.D + c, cnt, aw[i]);
            norm_store<true>(part, false, 2LL * a.D + c, cnt, aq[i]);
        }
    }
}

// The gradient of rows of more than 4096 columns, and of odd widths, whose pieces' addresses and bounds
// do not fit the registers beside a row: two passes over a row's columns, the second of which finds
// the inputs in L2; the columns' sums are kept in shared memory, each by its thread.
template <bool VEC>
__global__ void __launch_bounds__(NORM_THREADS, 1) block_norm_bwd_wide_kernel(NormArgs a) {
    constexpr int U = 2;
    extern __shared__ __align__(16) char smem[];
    __shared__ __align__(16) NormSums s_sum;
    const int pieces = (a.D + NORM_V - 1) / NORM_V;
    ulonglong2* acc = reinterpret_cast<ulonglong2*>(smem);  // [3][pieces]: dscale, dw_post, dw_pre
    const bool rb = a.rb, fb = a.fb, xb = a.xb;
    const bool has_gate = a.gate, has_post = a.w_post, has_scale = a.scale, has_pre = a.w_pre;
    RowSum red{s_sum, 0};
    s_sum.clear();
    __syncthreads();
    const f32x2 one = dup2(1.f), zero = dup2(0.f);
    const float inv_d = 1.f / (float)a.D;
    const int S = blockDim.x * NORM_V, first = threadIdx.x * NORM_V;
    for (int p = threadIdx.x; p < pieces; p += blockDim.x)
        acc[p] = acc[pieces + p] = acc[2 * pieces + p] = make_ulonglong2(zero, zero);

    // the pieces at c0 + u*S of a row, and the next row's f where its squares are summed
    NormRaw<VEC> rf[U], rr[U], rg[U], rn[U], rd[U], rx[U];
    auto load = [&](long long base, long long ahead, int c0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = c0 + u * S, cnt = min(NORM_V, a.D - c);
            rf[u].clear();
            rr[u].clear();
            rg[u].clear();
            rn[u].clear();
            rd[u].clear();
            rx[u].clear();
            if (c < a.D) {
                if (base >= 0) {
                    rf[u].load(a.f, fb, base + c, cnt);
                    rr[u].load(a.r, rb, base + c, cnt);
                    if (has_gate) rg[u].load(a.gate, xb, base + c, cnt);
                    if (a.dn) rn[u].load(a.dn, xb, base + c, cnt);
                    if (a.dr_out) rd[u].load(a.dr_out, rb, base + c, cnt);
                }
                if (ahead >= 0) rx[u].load(a.f, fb, ahead + c, cnt);
            }
        }
    };
    auto ahead_of = [&](long long row) { return has_post && row < a.rows ? row * a.D : -1LL; };
    auto square = [&](f32x2 s2) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            f32x2 f[2];
            rx[u].get(fb, f);
            s2 = fma2(f[0], f[0], s2);
            s2 = fma2(f[1], f[1], s2);
        }
        return s2;
    };
    float next[1] = {0.f};
    if (has_post) {
        f32x2 s2 = zero;
        for (int c0 = first; c0 < a.D; c0 += U * S) {
            load(-1, ahead_of(blockIdx.x), c0);
            s2 = square(s2);
        }
        next[0] = sum2(s2);
        red.sum(next);
    }
    for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const long long base = row * a.D;
        const f32x2 rf1 = has_post ? dup2(rsqrtf(next[0] * inv_d + a.eps)) : one;
        // one piece: f becomes f^ (f itself without the norm), g the gate's sigmoid, o the output
        f32x2 f[2], o[2], g[2], dn[2], dr[2], wp[2], sc[2], wq[2];
        auto piece = [&](int u, int c, int cnt) {
            norm_weight<VEC>(has_post, a.w_post, c, cnt, wp);
            norm_weight<VEC>(has_scale, a.scale, c, cnt, sc);
            norm_weight<VEC>(has_pre, a.w_pre, c, cnt, wq);
            rf[u].get(fb, f);
            rr[u].get(rb, o);
            rg[u].get(xb, g);
            rn[u].get(xb, dn);
            rd[u].get(rb, dr);
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                f[v] = mul2(f[v], rf1);
                g[v] = has_gate ? sigmoid2(g[v]) : one;
            }
        };
        f32x2 so = zero, sm = zero, sma = zero, soa = zero, sda = zero, s2 = zero;
        if (a.dn || has_post) {
            for (int c0 = first; c0 < a.D; c0 += U * S) {
                load(base, ahead_of(row + gridDim.x), c0);
                s2 = square(s2);
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int c = c0 + u * S, cnt = min(NORM_V, a.D - c);
                    if (c >= a.D) continue;
                    piece(u, c, cnt);
#pragma unroll
                    for (int v = 0; v < 2; ++v) {
                        const f32x2 k = mul2(mul2(sc[v], g[v]), mul2(f[v], wp[v])), m = mul2(dn[v], wq[v]);
                        o[v] = add2(k, o[v]);
                        so = fma2(o[v], o[v], so);
                        sm = fma2(o[v], m, sm);
                        sma = fma2(m, k, sma);
                        soa = fma2(o[v], k, soa);
                        sda = fma2(dr[v], k, sda);
                    }
                }
            }
        }
        f32x2 ro = zero, mo = zero, mf = zero;
        if (a.dn || has_post) {
            float st[6] = {sum2(so), sum2(sm), sum2(sma), sum2(soa), sum2(sda), sum2(s2)};
            red.sum(st);
            next[0] = st[5];
            float q = 0.f, mean = 0.f;
            if (a.dn) {
                q = rsqrtf(st[0] * inv_d + a.eps);
                mean = st[1] * q * inv_d;  // mean(m o^)
            }
            ro = dup2(q);
            mo = dup2(-mean);
            if (has_post) mf = dup2(-(st[4] + q * (st[2] - q * mean * st[3])) * inv_d);
        }
        for (int c0 = first; c0 < a.D; c0 += U * S) {
            load(base, -1, c0);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int c = c0 + u * S, cnt = min(NORM_V, a.D - c);
                if (c >= a.D) continue;
                piece(u, c, cnt);
                ulonglong2* at = acc + c / NORM_V;
                const ulonglong2 q0 = at[0], q1 = at[pieces], q2 = at[2 * pieces];
                f32x2 as[2] = {q0.x, q0.y}, aw[2] = {q1.x, q1.y}, aq[2] = {q2.x, q2.y}, dg[2];
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    o[v] = fma2(mul2(sc[v], g[v]), mul2(f[v], wp[v]), o[v]);
                    const f32x2 oh = mul2(o[v], ro);
                    aq[v] = fma2(dn[v], oh, aq[v]);
                    const f32x2 d = fma2(ro, fma2(dn[v], wq[v], mul2(oh, mo)), dr[v]);
                    dr[v] = d;
                    const f32x2 ds = mul2(d, g[v]);  // do sigmoid(gate)
                    const f32x2 dsp = mul2(ds, mul2(f[v], wp[v]));
                    as[v] = add2(as[v], dsp);
                    dg[v] = mul2(mul2(dsp, sc[v]), fma2(g[v], dup2(-1.f), one));
                    const f32x2 dp = mul2(ds, sc[v]);
                    aw[v] = fma2(dp, f[v], aw[v]);
                    o[v] = mul2(rf1, fma2(f[v], mf, mul2(dp, wp[v])));
                }
                at[0] = make_ulonglong2(as[0], as[1]);
                at[pieces] = make_ulonglong2(aw[0], aw[1]);
                at[2 * pieces] = make_ulonglong2(aq[0], aq[1]);
                if (a.dr) norm_store<VEC>(a.dr, rb, base + c, cnt, dr);
                if (a.dgate) norm_store<VEC>(a.dgate, xb, base + c, cnt, dg);
                if (a.df) norm_store<VEC>(a.df, fb, base + c, cnt, o);
            }
        }
    }
    float* part = a.part + (long long)blockIdx.x * 3 * a.D;
    for (int p = threadIdx.x; p < pieces; p += blockDim.x)
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            const ulonglong2 q = acc[k * pieces + p];
            const f32x2 v[2] = {q.x, q.y};
            norm_store<VEC>(part, false, (long long)k * a.D + p * NORM_V, min(NORM_V, a.D - p * NORM_V), v);
        }
}

// out[k][c] = the row groups' shares in a fixed order, k: dscale, dw_post, dw_pre: eight interleaved
// segments of shares, then the segments.
constexpr int SUM_SEG = 8;
__global__ void __launch_bounds__(32 * SUM_SEG) norm_sum_kernel(const float* part, int shares,
                                                                int D, float* dscale,
                                                                float* dw_post, float* dw_pre) {
    __shared__ float s[SUM_SEG][32];
    const int lane = threadIdx.x & 31, seg = threadIdx.x >> 5;
    const long long e = (long long)blockIdx.x * 32 + lane, n = 3LL * D;
    float sum = 0.f;
    if (e < n) {
#pragma unroll 4
        for (int p = seg; p < shares; p += SUM_SEG) sum += part[p * n + e];
    }
    s[seg][lane] = sum;
    __syncthreads();
    if (seg == 0 && e < n) {
#pragma unroll
        for (int k = 1; k < SUM_SEG; ++k) sum += s[k][lane];
        float* out = e < D ? dscale : (e < 2 * D ? dw_post : dw_pre);
        if (out) out[e % D] = sum;
    }
}

}  // namespace ssm
}  // namespace sdm
