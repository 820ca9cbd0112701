// The norms around a block with its gate and residual scale, over rows of D values:
//   p = f rf w_post,  rf = (mean f^2 + eps)^-1/2      o = r + scale sigmoid(gate) p
//   r_out = o,        n = o ro w_pre,  ro = (mean o^2 + eps)^-1/2
// and its gradient, with dn w_pre = m, o^ = o ro, f^ = f rf:
//   do = dr_out + ro (m - o^ mean(m o^)),  dr = do
//   dp = do scale sigmoid(gate),  q = dp w_post,  df = rf (q - f^ mean(q f^))
//   dgate = do scale p s (1-s),  dscale = sum do s p,  dw_post = sum dp f^,  dw_pre = sum dn o^
//
// Bound by memory.  A block takes whole rows, each read once into registers (so r_out may be r)
// and normalised in place; the weights stay in registers over the block's rows.  The two sums
// of a row (four in the gradient, two of them together) are block reductions in fp32.
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

template <int V>
SDM_DEV void norm_load(const void* p, int is_bf16, long long at, float (&v)[V]) {
    if (is_bf16) Vec<V>::load(static_cast<const bf16*>(p) + at, v);
    else Vec<V>::load(static_cast<const float*>(p) + at, v);
}
template <int V>
SDM_DEV void norm_store(void* p, int is_bf16, long long at, const float (&v)[V]) {
    if (is_bf16) Vec<V>::store(static_cast<bf16*>(p) + at, v);
    else Vec<V>::store(static_cast<float*>(p) + at, v);
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
__global__ void __launch_bounds__(512) block_norm_kernel(NormArgs a) {
    __shared__ float s_sum[2][2][32];
    int slot = 0;
    float wp[P][V], sc[P][V], wq[P][V];
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int c = (i * blockDim.x + threadIdx.x) * V;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const bool in = c < a.D;
            wp[i][v] = in && a.w_post ? a.w_post[c + v] : 1.f;
            sc[i][v] = in && a.scale ? a.scale[c + v] : 1.f;
            wq[i][v] = in && a.w_pre ? a.w_pre[c + v] : 1.f;
        }
    }
    for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const long long base = row * a.D;
        float f[P][V], o[P][V], g[P][V];
        float ss[1] = {0.f};
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int c = (i * blockDim.x + threadIdx.x) * V;
            if (c < a.D) {
                norm_load<V>(a.f, a.fb, base + c, f[i]);
                norm_load<V>(a.r, a.rb, base + c, o[i]);
                if (a.gate) norm_load<V>(a.gate, a.xb, base + c, g[i]);
#pragma unroll
                for (int v = 0; v < V; ++v) ss[0] = fmaf(f[i][v], f[i][v], ss[0]);
            }
        }
        float rf = 1.f;
        if (a.w_post) {
            block_sum<1>(ss, s_sum, slot);
            rf = rsqrtf(ss[0] / (float)a.D + a.eps);
        }
        ss[0] = 0.f;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int c = (i * blockDim.x + threadIdx.x) * V;
            if (c < a.D) {
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    float k = sc[i][v] * wp[i][v] * rf;
                    if (a.gate) k *= sigmoid(g[i][v]);
                    o[i][v] = fmaf(k, f[i][v], o[i][v]);
                    ss[0] = fmaf(o[i][v], o[i][v], ss[0]);
                }
                if (a.r_out) norm_store<V>(a.r_out, a.rb, base + c, o[i]);
            }
        }
        if (!a.n) continue;
        block_sum<1>(ss, s_sum, slot);
        const float ro = rsqrtf(ss[0] / (float)a.D + a.eps);
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int c = (i * blockDim.x + threadIdx.x) * V;
            if (c < a.D) {
#pragma unroll
                for (int v = 0; v < V; ++v) o[i][v] *= ro * wq[i][v];
                norm_store<V>(a.n, a.xb, base + c, o[i]);
            }
        }
    }
}

template <int V, int P>
__global__ void __launch_bounds__(512) block_norm_bwd_kernel(NormArgs a) {
    __shared__ float s_sum[2][2][32];
    int slot = 0;
    float wp[P][V], sc[P][V], wq[P][V], aw[P][V], as[P][V], aq[P][V];
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int c = (i * blockDim.x + threadIdx.x) * V;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const bool in = c < a.D;
            wp[i][v] = in && a.w_post ? a.w_post[c + v] : 1.f;
            sc[i][v] = in && a.scale ? a.scale[c + v] : 1.f;
            wq[i][v] = in && a.w_pre ? a.w_pre[c + v] : 1.f;
            aw[i][v] = as[i][v] = aq[i][v] = 0.f;
        }
    }
    const float inv_d = 1.f / (float)a.D;
    for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const long long base = row * a.D;
        float f[P][V], o[P][V], g[P][V], dn[P][V], dr[P][V];
        float ss[1] = {0.f};
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int c = (i * blockDim.x + threadIdx.x) * V;
#pragma unroll
            for (int v = 0; v < V; ++v) f[i][v] = o[i][v] = g[i][v] = dn[i][v] = dr[i][v] = 0.f;
            if (c < a.D) {
                norm_load<V>(a.f, a.fb, base + c, f[i]);
                norm_load<V>(a.r, a.rb, base + c, o[i]);
                if (a.gate) norm_load<V>(a.gate, a.xb, base + c, g[i]);
                if (a.dn) norm_load<V>(a.dn, a.xb, base + c, dn[i]);
                if (a.dr_out) norm_load<V>(a.dr_out, a.rb, base + c, dr[i]);
#pragma unroll
                for (int v = 0; v < V; ++v) ss[0] = fmaf(f[i][v], f[i][v], ss[0]);
            }
        }
        float rf = 1.f;
        if (a.w_post) {
            block_sum<1>(ss, s_sum, slot);
            rf = rsqrtf(ss[0] * inv_d + a.eps);
        }
        // f becomes f^ (f itself without the norm), g the gate's sigmoid
        float s2[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < P; ++i)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                f[i][v] *= rf;
                g[i][v] = a.gate ? sigmoid(g[i][v]) : 1.f;
                o[i][v] = fmaf(sc[i][v] * g[i][v], f[i][v] * wp[i][v], o[i][v]);
                s2[0] = fmaf(o[i][v], o[i][v], s2[0]);
                s2[1] = fmaf(o[i][v] * wq[i][v], dn[i][v], s2[1]);
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
            float dg[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float oh = o[i][v] * ro;
                aq[i][v] = fmaf(dn[i][v], oh, aq[i][v]);
                const float d = fmaf(ro, fmaf(dn[i][v], wq[i][v], -oh * mo), dr[i][v]);
                dr[i][v] = d;
                const float p = f[i][v] * wp[i][v], dsp = d * p * g[i][v];
                as[i][v] += dsp;
                dg[v] = dsp * sc[i][v] * (1.f - g[i][v]);
                const float dp = d * sc[i][v] * g[i][v];
                aw[i][v] = fmaf(dp, f[i][v], aw[i][v]);
                o[i][v] = dp * wp[i][v];  // q
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
                for (int v = 0; v < V; ++v) o[i][v] = rf * (o[i][v] - f[i][v] * mf);
                norm_store<V>(a.df, a.fb, base + c, o[i]);
            }
        }
    }
    float* part = a.part + (long long)blockIdx.x * 3 * a.D;
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int c = (i * blockDim.x + threadIdx.x) * V;
        if (c < a.D) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                part[c + v] = as[i][v];
                part[a.D + c + v] = aw[i][v];
                part[2 * a.D + c + v] = aq[i][v];
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
