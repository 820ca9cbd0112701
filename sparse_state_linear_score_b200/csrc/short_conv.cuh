// Short causal convolution over the tokens, one filter of K <= 8 taps per channel:
//   p_t = bias + sum_{j<K} w[j] x_{t-K+1+j},  y_t = p_t or p_t sigmoid(p_t)
// with the K-1 inputs before the call in a state, and its gradient:
//   g_t  = dy_t act'(p_t),   dx_s = sum_j w[j] g_{s+K-1-j} (+ dstate_end where s is kept),
//   dw_j = sum_{b,t} g_t x_{t-K+1+j},  dbias = sum_{b,t} g_t
//
// Bound by memory: 2 reads or writes an element (forward), 3 (backward), about 2K + 5 (6K + 8)
// operations.  A warp walks a run of tokens of one sequence; its lanes hold 32 neighbouring
// channel vectors of the flattened (head, channel) axis, whose filters stay in registers, and
// the last K-1 tokens move through a register window, so each input is read from memory once
// (plus K-1 tokens where runs meet, which L2 holds).  The loads of the next tokens are issued
// before the current ones are used.
#pragma once

#include "ssm_util.cuh"

namespace sdm {
namespace ssm {

constexpr int CONV_WARPS = 4;
constexpr int CONV_MAXK = 8;
constexpr int CONV_RUN_MIN = 8;  // tokens of a run: at least the CONV_MAXK - 1 of its halo

template <typename T>
struct ConvArgs {
    View<const T> x;
    View<T> y;  // backward: dx
    View<const T> dy;
    const float* w;
    const float* bias;
    T* state;
    const int* lens;
    const float* dstate_end;
    float* dstate;
    float* part;  // backward: [gridDim.y][K + 1][C]
    int B, H, T_, d, K, act, fresh;
    int run, runs;  // tokens of a run, runs of a sequence
};

// Tokens t0-K+1 .. t0-1 of the sequence: from x, or before its start from the state.
template <typename T, int V, int K>
SDM_DEV void conv_load_window(const ConvArgs<T>& a, const T* x, const T* state, int t0, int len,
                              float (&win)[K][V]) {
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
        const int s = t0 - (K - 1) + j;
#pragma unroll
        for (int v = 0; v < V; ++v) win[j][v] = 0.f;
        if (s >= 0) {
            if (s < len) Vec<V>::load(x + s * a.x.st, win[j]);
        } else if (state) {
            Vec<V>::load(state + (long long)(s + K - 1) * a.d, win[j]);
        }
    }
}

template <typename T, int V, int K>
__global__ void __launch_bounds__(CONV_WARPS * 32) short_conv_kernel(ConvArgs<T> a) {
    constexpr int U = K <= 4 ? 8 : 4;  // tokens whose loads are in flight together
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int nv = a.d / V;
    const long long cv = (long long)blockIdx.x * 32 + lane;
    const long long rr = (long long)blockIdx.y * CONV_WARPS + warp;
    if (cv >= (long long)a.H * nv || rr >= (long long)a.B * a.runs) return;
    const int h = (int)(cv / nv), c = (int)(cv % nv) * V;
    const int b = (int)(rr / a.runs), run = (int)(rr % a.runs);
    const long long ch = (long long)h * a.d + c;
    const int len = clamp_len(a.lens, b, a.T_);
    const int t0 = run * a.run;
    if (t0 >= len && run > 0) return;
    const int t1 = min(t0 + a.run, len);
    const T* x = a.x.p + b * a.x.sb + h * a.x.sh + c;
    T* y = a.y.p + b * a.y.sb + h * a.y.sh + c;
    T* state = a.state ? a.state + ((long long)b * a.H + h) * (K - 1) * a.d + c : nullptr;

    float w[K][V], bias[V], win[K][V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int j = 0; j < K; ++j) w[j][v] = a.w[(ch + v) * K + j];
        bias[v] = a.bias ? a.bias[ch + v] : 0.f;
    }
    conv_load_window<T, V, K>(a, x, a.fresh ? nullptr : state, t0, len, win);

    // The sequence's first run also moves the state on: the K-1 inputs that end at len, from x
    // or, where the call is shorter, from the old state (which is in the window).
    if (run == 0 && state) {
        float keep[K][V];
#pragma unroll
        for (int k = 0; k < K - 1; ++k) {
            const int s = len - (K - 1) + k;
            if (s >= 0) {
                Vec<V>::load(x + s * a.x.st, keep[k]);
            } else {
#pragma unroll
                for (int q = 0; q < K - 1; ++q)
                    if (q == s + K - 1) {
#pragma unroll
                        for (int v = 0; v < V; ++v) keep[k][v] = win[q][v];
                    }
            }
        }
#pragma unroll
        for (int k = 0; k < K - 1; ++k) Vec<V>::store(state + (long long)k * a.d, keep[k]);
    }

    for (int t = t0; t < t1; t += U) {
        float in[U][V];
#pragma unroll
        for (int i = 0; i < U; ++i)
            if (t + i < t1) Vec<V>::load(x + (t + i) * a.x.st, in[i]);
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if (t + i < t1) {
                float p[V];
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    win[K - 1][v] = in[i][v];
                    p[v] = bias[v];
#pragma unroll
                    for (int j = 0; j < K; ++j) p[v] = fmaf(w[j][v], win[j][v], p[v]);
#pragma unroll
                    for (int j = 0; j < K - 1; ++j) win[j][v] = win[j + 1][v];
                    if (a.act) p[v] *= sigmoid(p[v]);
                }
                Vec<V>::store(y + (t + i) * a.y.st, p);
            }
        }
    }
}

// A warp takes every (gridDim.y * CONV_WARPS)-th run and sums its share of dw and dbias in
// registers; the block's warps are added in order in shared memory, the blocks in order by
// conv_sum_kernel.
template <typename T, int V, int K>
__global__ void __launch_bounds__(CONV_WARPS * 32) short_conv_bwd_kernel(ConvArgs<T> a) {
    constexpr int U = 4;
    __shared__ float s_part[CONV_WARPS][K + 1][V][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int nv = a.d / V;
    const long long C = (long long)a.H * a.d;
    const long long cv = (long long)blockIdx.x * 32 + lane;
    const bool live = cv < (long long)a.H * nv;
    const int h = live ? (int)(cv / nv) : 0, c = live ? (int)(cv % nv) * V : 0;
    const long long ch = (long long)h * a.d + c;

    float w[K][V], bias[V], dw[K][V], db[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int j = 0; j < K; ++j) {
            w[j][v] = a.w[(ch + v) * K + j];
            dw[j][v] = 0.f;
        }
        bias[v] = a.bias ? a.bias[ch + v] : 0.f;
        db[v] = 0.f;
    }
    const long long nruns = live ? (long long)a.B * a.runs : 0;
    for (long long rr = (long long)blockIdx.y * CONV_WARPS + warp; rr < nruns;
         rr += (long long)gridDim.y * CONV_WARPS) {
        const int b = (int)(rr / a.runs), run = (int)(rr % a.runs);
        const int len = clamp_len(a.lens, b, a.T_);
        const int t0 = run * a.run, t1 = min(t0 + a.run, a.T_);
        const T* x = a.x.p + b * a.x.sb + h * a.x.sh + c;
        const T* dy = a.dy.p + b * a.dy.sb + h * a.dy.sh + c;
        T* dx = a.y.p + b * a.y.sb + h * a.y.sh + c;
        const long long so = ((long long)b * a.H + h) * (K - 1) * a.d + c;
        const T* state = a.state && !a.fresh ? a.state + so : nullptr;
        float win[K][V], g[K][V];  // inputs and g of the last K tokens, oldest first
        conv_load_window<T, V, K>(a, x, state, t0, len, win);
#pragma unroll
        for (int j = 0; j < K; ++j)
#pragma unroll
            for (int v = 0; v < V; ++v) g[j][v] = 0.f;
        // Token t brings g_t and completes dx of token t-K+1; the run's last K-1 need the g of
        // tokens behind it.
        const int tend = t1 + K - 1, tload = min(tend, len);
        for (int t = t0; t < tend; t += U) {
            float xi[U][V], gi[U][V];
#pragma unroll
            for (int i = 0; i < U; ++i) {
#pragma unroll
                for (int v = 0; v < V; ++v) xi[i][v] = gi[i][v] = 0.f;
                if (t + i < tload) {
                    Vec<V>::load(x + (t + i) * a.x.st, xi[i]);
                    Vec<V>::load(dy + (t + i) * a.dy.st, gi[i]);
                }
            }
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int tt = t + i;
                if (tt >= tend) break;
                float out[V];
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    win[K - 1][v] = xi[i][v];
                    float gt = gi[i][v];
                    if (a.act) {
                        float p = bias[v];
#pragma unroll
                        for (int j = 0; j < K; ++j) p = fmaf(w[j][v], win[j][v], p);
                        const float sg = sigmoid(p);
                        gt *= sg * (1.f + p * (1.f - sg));
                    }
                    if (tt >= len) gt = 0.f;  // also where p is not finite
#pragma unroll
                    for (int j = 0; j < K - 1; ++j) g[j][v] = g[j + 1][v];
                    g[K - 1][v] = gt;
                    if (tt < t1 && tt < len) {
                        db[v] += gt;
#pragma unroll
                        for (int j = 0; j < K; ++j) dw[j][v] = fmaf(gt, win[j][v], dw[j][v]);
                    }
                    out[v] = 0.f;
#pragma unroll
                    for (int j = 0; j < K; ++j) out[v] = fmaf(w[j][v], g[K - 1 - j][v], out[v]);
#pragma unroll
                    for (int j = 0; j < K - 1; ++j) win[j][v] = win[j + 1][v];
                }
                const int s = tt - (K - 1);
                if (s < t0 && run > 0) continue;  // the run before has it
                const int kept = s - len + K - 1;  // its row in the state after the call
                if (a.dstate_end && kept >= 0 && kept < K - 1) {
                    float e[V];
                    Vec<V>::load(a.dstate_end + so + (long long)kept * a.d, e);
#pragma unroll
                    for (int v = 0; v < V; ++v) out[v] += e[v];
                }
                if (s >= len && s >= 0) {
#pragma unroll
                    for (int v = 0; v < V; ++v) out[v] = 0.f;
                }
                if (s >= 0) Vec<V>::store(dx + s * a.y.st, out);
                else if (a.dstate) Vec<V>::store(a.dstate + so + (long long)(s + K - 1) * a.d, out);
            }
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int j = 0; j < K; ++j) s_part[warp][j][v][lane] = dw[j][v];
        s_part[warp][K][v][lane] = db[v];
    }
    __syncthreads();
    for (int e = threadIdx.x; e < (K + 1) * V * 32; e += CONV_WARPS * 32) {
        const int l = e & 31, v = (e >> 5) % V, j = (e >> 5) / V;
        const long long q = (long long)blockIdx.x * 32 + l;
        if (q >= (long long)a.H * nv) continue;
        float sum = 0.f;
        for (int k = 0; k < CONV_WARPS; ++k) sum += s_part[k][j][v][l];
        const long long chan = (q / nv) * a.d + (q % nv) * V + v;
        a.part[((long long)blockIdx.y * (K + 1) + j) * C + chan] = sum;
    }
}

// dw[c][j] and dbias[c] from the blocks' shares, in order.
__global__ void __launch_bounds__(256) conv_sum_kernel(const float* part, int blocks, long long C,
                                                       int K, float* dw, float* dbias) {
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    if (i >= C * (K + 1)) return;
    const long long c = i % C;
    const int j = (int)(i / C);
    if (j == K && !dbias) return;
    float sum = 0.f;
    for (int p = 0; p < blocks; ++p) sum += part[((long long)p * (K + 1) + j) * C + c];
    if (j < K) dw[c * K + j] = sum;
    else dbias[c] = sum;
}

}  // namespace ssm
}  // namespace sdm
