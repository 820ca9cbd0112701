// The norms around a block with its gate and residual scale, over rows of D values:
//   p = f rf w_post,  rf = (mean f^2 + eps)^-1/2      o = r + scale sigmoid(gate) p
//   r_out = o,        n = o ro w_pre,  ro = (mean o^2 + eps)^-1/2
// and its gradient, with dn w_pre = m, o^ = o ro, f^ = f rf:
//   do = dr_out + ro (m - o^ mean(m o^)),  dr = do
//   dp = do scale sigmoid(gate),  q = dp w_post,  df = rf (q - f^ mean(q f^))
//   dgate = do scale p s (1-s),  dscale = sum do s p,  dw_post = sum dp f^,  dw_pre = sum dn o^
//
// Bound by memory.  A block takes whole rows, each read once into registers (so r_out may be r)
// and normalised in place; the weights come from L1 after the first row.  The two sums of a row
// (four in the gradient, two of them together) are block reductions in fp32.  What hides the
// loads' latency: two blocks an SM that wait in turn, or (gradient, whose registers allow only
// one) the next row's loads issued ahead.
#pragma once

#include "ssm_util.cuh"

namespace sdm {
namespace ssm {

struct NormArgs {
    const void *r, *f, *gate, *dr_out, *dn;
    void *r_out, *n, *dr, *df, *dgate;  // r_out, n: forward
    const float *w_post, *scale, *w_pre;
    float* part;  // backward: [gridDim.x][3][D] (dscale, dw_post, dw_pre)
    long long rows;
    int D, rb, fb, xb;  // 1: bf16
    float eps;
};

// V values of a row as they are stored, in registers until they are used: a block's loads are all
// in flight before the first is waited for.
template <int V>
struct NormRaw {
    uint32_t x[V];
    SDM_DEV void clear() {
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = 0u;
    }
    SDM_DEV void load(const void* p, int is_bf16, long long at) {
        if constexpr (V == 4) {
            if (is_bf16) {
                const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const bf16*>(p) + at);
                x[0] = v.x, x[1] = v.y;
            } else {
                const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const float*>(p) + at);
                x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
            }
        } else {
            x[0] = is_bf16 ? static_cast<const uint16_t*>(p)[at] : static_cast<const uint32_t*>(p)[at];
        }
    }
    SDM_DEV void get(int is_bf16, float (&v)[V]) const {
        if constexpr (V == 4) {
            v[0] = is_bf16 ? bf16_lo(x[0]) : __uint_as_float(x[0]);
            v[1] = is_bf16 ? bf16_hi(x[0]) : __uint_as_float(x[1]);
            v[2] = is_bf16 ? bf16_lo(x[1]) : __uint_as_float(x[2]);
            v[3] = is_bf16 ? bf16_hi(x[1]) : __uint_as_float(x[3]);
        } else {
            v[0] = is_bf16 ? bf16_lo(x[0]) : __uint_as_float(x[0]);
        }
    }
};
template <int V>
SDM_DEV void norm_store(void* p, int is_bf16, long long at, const float (&v)[V]) {
    if (is_bf16) Vec<V>::store(static_cast<bf16*>(p) + at, v);
    else Vec<V>::store(static_cast<float*>(p) + at, v);
}
// V entries of a weight vector (1 where there is none), from L1 after the block's first row.
template <int V>
SDM_DEV void norm_weight(const float* w, int c, float (&v)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = 1.f;
    if (w) Vec<V>::load(w + c, v);
}

// Sums of K values over the block (every thread gets them).  The slot alternates from one
// reduction to the next, so that one barrier each is enough: a slot is written again only
// behind the barrier of the reduction after the one that read it.
template <int K>
SDM_DEV void block_sum(float (&v)[K], float (*s)[2][32], int& slot) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = warp_sum(v[k]);
    if (nw == 1) return;
    if (lane == 0) {
#pragma unroll
        for (int k = 0; k < K; ++k) s[slot][k][warp] = v[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = warp_sum(lane < nw ? s[slot][k][lane] : 0.f);
    slot ^= 1;
}

// Element i of thread t is column (i*blockDim + t)*V.
template <int V, int P>
__global__ void __launch_bounds__(512, P * V <= 8 ? 2 : 1) block_norm_kernel(NormArgs a) {
    __shared__ float s_sum[2][2][32];
    int slot = 0;
    const float inv_d = 1.f / (float)a.D;
    for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const long long base = row * a.D;
        NormRaw<V> rf[P], rr[P], rg[P];
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int c = (i * blockDim.x + threadIdx.x) * V;
            rf[i].clear();
            rr[i].clear();
            rg[i].clear();
            if (c < a.D) {
                rf[i].load(a.f, a.fb, base + c);
                rr[i].load(a.r, a.rb, base + c);
                if (a.gate) rg[i].load(a.gate, a.xb, base + c);
            }
        }
        float f[P][V], o[P][V];
        float ss[1] = {0.f};
#pragma unroll
        for (int i = 0; i < P; ++i) {
            rf[i].get(a.fb, f[i]);
#pragma unroll
            for (int v = 0; v < V; ++v) ss[0] = fmaf(f[i][v], f[i][v], ss[0]);
        }
        float k = 1.f;
        if (a.w_post) {
            block_sum<1>(ss, s_sum, slot);
            k = rsqrtf(ss[0] * inv_d + a.eps);
        }
        ss[0] = 0.f;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int c = (i * blockDim.x + threadIdx.x) * V;
            if (c < a.D) {
                float wp[V], sc[V], g[V];
                norm_weight<V>(a.w_post, c, wp);
                norm_weight<V>(a.scale, c, sc);
                rg[i].get(a.xb, g);
                rr[i].get(a.rb, o[i]);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    float m = sc[v] * wp[v] * k;
                    if (a.gate) m *= sigmoid(g[v]);
                    o[i][v] = fmaf(m, f[i][v], o[i][v]);
                    ss[0] = fmaf(o[i][v], o[i][v], ss[0]);
                }
                if (a.r_out) norm_store<V>(a.r_out, a.rb, base + c, o[i]);
            }
        }
        if (!a.n) continue;
        block_sum<1>(ss, s_sum, slot);
        const float ro = rsqrtf(ss[0] * inv_d + a.eps);
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int c = (i * blockDim.x + threadIdx.x) * V;
            if (c < a.D) {
                float wq[V];
                norm_weight<V>(a.w_pre, c, wq);
#pragma unroll
                for (int v = 0; v < V; ++v) o[i][v] *= ro * wq[v];
                norm_store<V>(a.n, a.xb, base + c, o[i]);
            }
        }
    }
}

// The next row's loads are issued before this row's arithmetic, so that one block an SM keeps
// memory busy.
template <int V, int P>
__global__ void __launch_bounds__(512, 1) block_norm_bwd_kernel(NormArgs a) {
    __shared__ float s_sum[2][2][32];
    int slot = 0;
    float aw[P][V], as[P][V], aq[P][V];
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
        for (int v = 0; v < V; ++v) aw[i][v] = as[i][v] = aq[i][v] = 0.f;
    const float inv_d = 1.f / (float)a.D;
    NormRaw<V> rf[P], rr[P], rg[P], rn[P], rd[P];
    auto fetch = [&](long long row) {
        const long long base = row * a.D;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int c = (i * blockDim.x + threadIdx.x) * V;
            rf[i].clear();
            rr[i].clear();
            rg[i].clear();
            rn[i].clear();
            rd[i].clear();
            if (c < a.D && row < a.rows) {
                rf[i].load(a.f, a.fb, base + c);
                rr[i].load(a.r, a.rb, base + c);
                if (a.gate) rg[i].load(a.gate, a.xb, base + c);
                if (a.dn) rn[i].load(a.dn, a.xb, base + c);
                if (a.dr_out) rd[i].load(a.dr_out, a.rb, base + c);
            }
        }
    };
    fetch(blockIdx.x);
    for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const long long base = row * a.D;
        float f[P][V], o[P][V], g[P][V], dn[P][V], dr[P][V];
        float ss[1] = {0.f};
#pragma unroll
        for (int i = 0; i < P; ++i) {
            rf[i].get(a.fb, f[i]);
            rr[i].get(a.rb, o[i]);
            rg[i].get(a.xb, g[i]);
            rn[i].get(a.xb, dn[i]);
            rd[i].get(a.rb, dr[i]);
#pragma unroll
            for (int v = 0; v < V; ++v) ss[0] = fmaf(f[i][v], f[i][v], ss[0]);
        }
        fetch(row + gridDim.x);
        float rf1 = 1.f;
        if (a.w_post) {
            block_sum<1>(ss, s_sum, slot);
            rf1 = rsqrtf(ss[0] * inv_d + a.eps);
        }
        // f becomes f^ (f itself without the norm), g the gate's sigmoid
        float s2[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int c = (i * blockDim.x + threadIdx.x) * V;
            if (c >= a.D) continue;
            float wp[V], sc[V], wq[V];
            norm_weight<V>(a.w_post, c, wp);
            norm_weight<V>(a.scale, c, sc);
            norm_weight<V>(a.w_pre, c, wq);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                f[i][v] *= rf1;
                g[i][v] = a.gate ? sigmoid(g[i][v]) : 1.f;
                o[i][v] = fmaf(sc[v] * g[i][v], f[i][v] * wp[v], o[i][v]);
                s2[0] = fmaf(o[i][v], o[i][v], s2[0]);
                s2[1] = fmaf(o[i][v] * wq[v], dn[i][v], s2[1]);
            }
        }
        float ro = 0.f, mo = 0.f;
        if (a.dn) {
            block_sum<2>(s2, s_sum, slot);
            ro = rsqrtf(s2[0] * inv_d + a.eps);
            mo = s2[1] * ro * inv_d;  // mean(m o^)
        }
        float sq[1] = {0.f};
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int c = (i * blockDim.x + threadIdx.x) * V;
            if (c >= a.D) continue;
            float wp[V], sc[V], wq[V], dg[V];
            norm_weight<V>(a.w_post, c, wp);
            norm_weight<V>(a.scale, c, sc);
            norm_weight<V>(a.w_pre, c, wq);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float oh = o[i][v] * ro;
                aq[i][v] = fmaf(dn[i][v], oh, aq[i][v]);
                const float d = fmaf(ro, fmaf(dn[i][v], wq[v], -oh * mo), dr[i][v]);
                dr[i][v] = d;
                const float p = f[i][v] * wp[v], dsp = d * p * g[i][v];
                as[i][v] += dsp;
                dg[v] = dsp * sc[v] * (1.f - g[i][v]);
                const float dp = d * sc[v] * g[i][v];
                aw[i][v] = fmaf(dp, f[i][v], aw[i][v]);
                o[i][v] = dp * wp[v];  // q
                sq[0] = fmaf(o[i][v], f[i][v], sq[0]);
            }
            if (a.dr) norm_store<V>(a.dr, a.rb, base + c, dr[i]);
            if (a.dgate) norm_store<V>(a.dgate, a.xb, base + c, dg);
        }
        float mf = 0.f;
        if (a.w_post) {
            block_sum<1>(sq, s_sum, slot);
            mf = sq[0] * inv_d;
        }
        if (a.df) {
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const int c = (i * blockDim.x + threadIdx.x) * V;
                if (c >= a.D) continue;
#pragma unroll
                for (int v = 0; v < V; ++v) o[i][v] = rf1 * (o[i][v] - f[i][v] * mf);
                norm_store<V>(a.df, a.fb, base + c, o[i]);
            }
        }
    }
    float* part = a.part + (long long)blockIdx.x * 3 * a.D;
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int c = (i * blockDim.x + threadIdx.x) * V;
        if (c < a.D) {
            Vec<V>::store(part + c, as[i]);
            if constexpr (V == 4) {
                Vec<V>::store(part + a.D + c, aw[i]);  // D is a multiple of 4
                Vec<V>::store(part + 2 * a.D + c, aq[i]);
            } else {
                part[a.D + c] = aw[i][0];
                part[2 * a.D + c] = aq[i][0];
            }
        }
    }
}

// out[k][c] = the blocks' shares in order, k: dscale, dw_post, dw_pre.  One warp row of 32
// columns per 8 segments of blocks, the segments added in order.
constexpr int SUM_SEG = 8;
__global__ void __launch_bounds__(32 * SUM_SEG) norm_sum_kernel(const float* part, int blocks,
                                                                int D, float* dscale,
                                                                float* dw_post, float* dw_pre) {
    __shared__ float s[SUM_SEG][32];
    const int lane = threadIdx.x & 31, seg = threadIdx.x >> 5;
    const long long e = (long long)blockIdx.x * 32 + lane, n = 3LL * D;
    const int per = (blocks + SUM_SEG - 1) / SUM_SEG;
    float sum = 0.f;
    if (e < n)
        for (int p = seg * per; p < min(blocks, (seg + 1) * per); ++p) sum += part[p * n + e];
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
