// Short causal convolution over the tokens, one filter of K <= 8 taps per channel:
//   p_t = bias + sum_{j<K} w[j] x_{t-K+1+j},  y_t = p_t or p_t sigmoid(p_t)
// with the K-1 inputs before the call in a state, and its gradient:
//   g_t  = dy_t act'(p_t),   dx_s = sum_j w[j] g_{s+K-1-j} (+ dstate_end where s is kept),
//   dw_j = sum_{b,t} g_t x_{t-K+1+j},  dbias = sum_{b,t} g_t
//
// Bound by memory: 2 reads or writes an element (forward), 3 (gradient), about 2K + 5 (6K + 8)
// operations.  A warp walks a run of tokens of one sequence; its lanes hold 32 neighbouring vectors
// of the flattened (head, channel) axis, whose filters stay in registers, and the last K-1 tokens
// move through a register window, so each input is read from memory once (plus K-1 tokens where
// runs meet, which L2 holds).  Loads are issued as they are stored and converted only when used: a
// conversion behind a load waits for it (the gradient took 506 us so, 206 us without); through a
// ring in shared memory they take no registers meanwhile (forward, 8 x 16 x 2048 x 128: 34.7 us with
// eight tokens in registers, 31.6 us; eight taps 61 and 42 us).
// Measured, bf16, K = 4, inputs not in L2: forward 2 x 4 x 4096 x 128 7.1 us, 8 x 16 x 2048 x 128 31 us,
// 4.3 TB/s; gradient 8 x 16 x 8192 x 64 88 us, 4.3 TB/s, 55 % of the issue slots.
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

template <bool B>
struct Flag {
    static constexpr bool value = B;
};

// V channels of a token as pairs of floats (one channel: a pair with a zero).
template <int V>
struct Pairs {
    static constexpr int N = (V + 1) / 2;
    template <typename T>
    SDM_DEV static void load(const T* p, f32x2 (&v)[N]) {
        float x[V];
        Vec<V>::load(p, x);
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = pack2(x[2 * i], 2 * i + 1 < V ? x[2 * i + 1 < V ? 2 * i + 1 : 0] : 0.f);
    }
    template <typename T>
    SDM_DEV static void store(T* p, const f32x2 (&v)[N]) {
        float x[2 * N], y[V];
#pragma unroll
        for (int i = 0; i < N; ++i) unpack2(v[i], x[2 * i], x[2 * i + 1]);
#pragma unroll
        for (int i = 0; i < V; ++i) y[i] = x[i];
        Vec<V>::store(p, y);
    }
};

// The filters w[j] and biases of channels ch .. ch+V-1.
template <int V, int K>
SDM_DEV void conv_load_filter(const float* w, const float* bias, long long ch,
                              f32x2 (&wr)[K][Pairs<V>::N], f32x2 (&br)[Pairs<V>::N]) {
    float x[V * K];
    if constexpr (V == 4) {  // V*K floats from a multiple of 16 bytes
#pragma unroll
        for (int i = 0; i < V * K; i += 4) {
            const float4 q = *reinterpret_cast<const float4*>(w + ch * K + i);
            x[i] = q.x, x[i + 1] = q.y, x[i + 2] = q.z, x[i + 3] = q.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < V * K; ++i) x[i] = w[ch * K + i];
    }
#pragma unroll
    for (int p = 0; p < Pairs<V>::N; ++p) {
#pragma unroll
        for (int j = 0; j < K; ++j)
            wr[j][p] = pack2(x[2 * p * K + j], 2 * p + 1 < V ? x[(2 * p + 1) % V * K + j] : 0.f);
        br[p] = dup2(0.f);
    }
    if (bias) Pairs<V>::load(bias + ch, br);
}

// Tokens t0-K+1 .. t0-1 of the sequence: from x, or before its start from the state.
template <typename T, int V, int K>
SDM_DEV void conv_load_window(const ConvArgs<T>& a, const T* x, const T* state, int t0, int len,
                              f32x2 (&win)[K][Pairs<V>::N]) {
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
        const int s = t0 - (K - 1) + j;
#pragma unroll
        for (int p = 0; p < Pairs<V>::N; ++p) win[j][p] = dup2(0.f);
        if (s >= 0) {
            if (s < len) Pairs<V>::load(x + s * a.x.st, win[j]);
        } else if (state) {
            Pairs<V>::load(state + (long long)(s + K - 1) * a.d, win[j]);
        }
    }
}

// What a lane's loads pass through: a ring in shared memory that cp.async fills, three groups of four
// tokens ahead (whole vectors; each lane reads what it has copied itself), or registers, one group
// ahead.
constexpr int CONV_GRP = 4, CONV_RING = 4;
template <typename T, int V>
__host__ __device__ constexpr size_t conv_ring_bytes(int streams) {
    return V == 4 ? (size_t)CONV_WARPS * CONV_RING * CONV_GRP * streams * 32 * V * sizeof(T) : 0;
}

template <typename T, int V, int K>
__global__ void __launch_bounds__(CONV_WARPS * 32) short_conv_kernel(ConvArgs<T> a) {
    constexpr bool RING = V == 4;
    constexpr int U = RING ? CONV_GRP : 8, N = Pairs<V>::N;  // U tokens of a group
    extern __shared__ __align__(16) char smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int nv = a.d / V;
    const long long cv = (long long)blockIdx.x * 32 + lane;
    const long long rr = (long long)blockIdx.y * CONV_WARPS + warp;
    if (cv >= (long long)a.H * nv || rr >= (long long)a.B * a.runs) return;
    const int h = (int)(cv / nv), c = (int)(cv % nv) * V;
    const int b = (int)(rr / a.runs), run = (int)(rr % a.runs);
    const int len = clamp_len(a.lens, b, a.T_);
    const int t0 = run * a.run;
    if (t0 >= len && run > 0) return;
    const int t1 = min(t0 + a.run, len);
    const T* x = a.x.p + b * a.x.sb + h * a.x.sh + c;
    T* y = a.y.p + b * a.y.sb + h * a.y.sh + c;
    T* state = a.state ? a.state + ((long long)b * a.H + h) * (K - 1) * a.d + c : nullptr;

    Raw<T, V> in[U];
    T* ring = reinterpret_cast<T*>(smem) + (warp * CONV_RING * U * 32 + lane) * V;
    auto fetch = [&](int k, int t) {  // tokens t.. into group k of the ring, or into registers
        if constexpr (RING) {
#pragma unroll
            for (int i = 0; i < U; ++i)
                async_copy<V * sizeof(T)>(ring + (k % CONV_RING * U + i) * 32 * V, x + (t + i) * a.x.st,
                                          t + i < t1 ? V * (int)sizeof(T) : 0);
            async_commit();
        } else {
#pragma unroll
            for (int i = 0; i < U; ++i) {
                in[i].clear();
                if (t + i < t1) in[i].load(x + (t + i) * a.x.st);
            }
        }
    };
#pragma unroll
    for (int k = 0; k < (RING ? CONV_RING - 1 : 1); ++k) fetch(k, t0 + k * U);
    f32x2 w[K][N], bias[N], win[K][N];
    conv_load_filter<V, K>(a.w, a.bias, (long long)h * a.d + c, w, bias);
    conv_load_window<T, V, K>(a, x, a.fresh ? nullptr : state, t0, len, win);

    // The sequence's first run also moves the state on: the K-1 inputs that end at len, from x
    // or, where the call is shorter, from later rows of the old state, all read before any is
    // written.
    if (run == 0 && state) {
        f32x2 keep[K][N];
#pragma unroll
        for (int k = 0; k < K - 1; ++k) {
            const int s = len - (K - 1) + k;
#pragma unroll
            for (int p = 0; p < N; ++p) keep[k][p] = dup2(0.f);
            if (s >= 0) Pairs<V>::load(x + s * a.x.st, keep[k]);
            else if (!a.fresh) Pairs<V>::load(state + (long long)(len + k) * a.d, keep[k]);
        }
#pragma unroll
        for (int k = 0; k < K - 1; ++k) Pairs<V>::store(state + (long long)k * a.d, keep[k]);
    }

    auto walk = [&](auto act) {
        constexpr bool ACT = decltype(act)::value;
        for (int t = t0, k = 0; t < t1; t += U, ++k) {
            f32x2 cur[U][N];
            if constexpr (RING) {
                async_wait<CONV_RING - 2>();
#pragma unroll
                for (int i = 0; i < U; ++i) in[i].load(ring + (k % CONV_RING * U + i) * 32 * V);
            }
#pragma unroll
            for (int i = 0; i < U; ++i) in[i].pairs(cur[i]);
            if constexpr (RING) fetch(k + CONV_RING - 1, t + (CONV_RING - 1) * U);
            else fetch(k + 1, t + U);
#pragma unroll
            for (int i = 0; i < U; ++i) {
                f32x2 o[N];
#pragma unroll
                for (int p = 0; p < N; ++p) {
                    win[K - 1][p] = cur[i][p];
                    o[p] = bias[p];
#pragma unroll
                    for (int j = 0; j < K; ++j) o[p] = fma2(w[j][p], win[j][p], o[p]);
#pragma unroll
                    for (int j = 0; j < K - 1; ++j) win[j][p] = win[j + 1][p];
                    if (ACT) o[p] = silu2(o[p]);
                }
                if (t + i < t1) Pairs<V>::store(y + (t + i) * a.y.st, o);
            }
        }
    };
    if (a.act) walk(Flag<true>());
    else walk(Flag<false>());
}

// A warp takes every (gridDim.y * CONV_WARPS)-th run and sums its share of dw and dbias in
// registers; the block's warps are added in order in shared memory, the blocks in order by
// conv_sum_kernel.
template <typename T, int V, int K>
__global__ void __launch_bounds__(CONV_WARPS * 32, K <= 4 ? 3 : 1) short_conv_bwd_kernel(ConvArgs<T> a) {
    constexpr int U = CONV_GRP, N = Pairs<V>::N;
    constexpr bool RING = V == 4;
    extern __shared__ __align__(16) char smem[];
    __shared__ float s_part[CONV_WARPS][K + 1][2 * N][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int nv = a.d / V;
    const long long C = (long long)a.H * a.d;
    const long long cv = (long long)blockIdx.x * 32 + lane;
    const bool live = cv < (long long)a.H * nv;
    const int h = live ? (int)(cv / nv) : 0, c = live ? (int)(cv % nv) * V : 0;

    f32x2 w[K][N], bias[N], dw[K][N], db[N];
    conv_load_filter<V, K>(a.w, a.bias, (long long)h * a.d + c, w, bias);
#pragma unroll
    for (int p = 0; p < N; ++p) {
#pragma unroll
        for (int j = 0; j < K; ++j) dw[j][p] = dup2(0.f);
        db[p] = dup2(0.f);
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
        // Token t brings g_t and completes dx of token t-K+1; the run's last K-1 need the g of
        // tokens behind it.  Inputs and g of the last K tokens, oldest first:
        f32x2 win[K][N], g[K][N];
        Raw<T, V> xi[U], gi[U];
        T* ring = reinterpret_cast<T*>(smem) + (warp * CONV_RING * U * 2 * 32 + lane) * V;
        const int tend = t1 + K - 1, tload = min(tend, len);
        // tokens t.. into group k of the ring, or into registers; zero from tload on
        auto fetch = [&](int k, int t) {
            const T* xp = x + t * a.x.st;
            const T* gp = dy + t * a.dy.st;
            if constexpr (RING) {
                T* to = ring + k % CONV_RING * U * 2 * 32 * V;
#pragma unroll
                for (int i = 0; i < U; ++i) {
                    const int bytes = t + i < tload ? V * (int)sizeof(T) : 0;
                    async_copy<V * sizeof(T)>(to + 2 * i * 32 * V, xp + i * a.x.st, bytes);
                    async_copy<V * sizeof(T)>(to + (2 * i + 1) * 32 * V, gp + i * a.dy.st, bytes);
                }
                async_commit();
            } else {
#pragma unroll
                for (int i = 0; i < U; ++i) {
                    xi[i].clear();
                    gi[i].clear();
                    if (t + i < tload) {
                        xi[i].load(xp + i * a.x.st);
                        gi[i].load(gp + i * a.dy.st);
                    }
                }
            }
        };
        // U tokens; EDGE: some of them, or the tokens they complete, lie outside the run, behind
        // the sequence, before its start or in the state after the call.
        auto group = [&](int k, int t, auto edge, auto act) {
            constexpr bool EDGE = decltype(edge)::value, ACT = decltype(act)::value;
            f32x2 cx[U][N], cg[U][N], out[U][N];
            if constexpr (RING) {
                async_wait<CONV_RING - 2>();
                const T* from = ring + k % CONV_RING * U * 2 * 32 * V;
#pragma unroll
                for (int i = 0; i < U; ++i) {
                    xi[i].load(from + 2 * i * 32 * V);
                    gi[i].load(from + (2 * i + 1) * 32 * V);
                }
            }
#pragma unroll
            for (int i = 0; i < U; ++i) {
                xi[i].pairs(cx[i]);
                gi[i].pairs(cg[i]);
            }
            if constexpr (RING) fetch(k + CONV_RING - 1, t + (CONV_RING - 1) * U);
            else fetch(k + 1, t + U);
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const unsigned long long inside = !EDGE || t + i < len ? ~0ull : 0ull;
                const unsigned long long own = !EDGE || t + i < t1 ? ~0ull : 0ull;
#pragma unroll
                for (int p = 0; p < N; ++p) {
                    win[K - 1][p] = cx[i][p];
                    f32x2 gt = cg[i][p];
                    if (ACT) {
                        f32x2 q = bias[p];
#pragma unroll
                        for (int j = 0; j < K; ++j) q = fma2(w[j][p], win[j][p], q);
                        gt = mul2(gt, dsilu2(q));
                    }
                    if (EDGE) gt &= inside;  // also where q is not finite
#pragma unroll
                    for (int j = 0; j < K - 1; ++j) g[j][p] = g[j + 1][p];
                    g[K - 1][p] = gt;
                    if (EDGE) gt &= own;
                    db[p] = add2(db[p], gt);
#pragma unroll
                    for (int j = 0; j < K; ++j) dw[j][p] = fma2(gt, win[j][p], dw[j][p]);
                    out[i][p] = mul2(w[0][p], g[K - 1][p]);
#pragma unroll
                    for (int j = 1; j < K; ++j) out[i][p] = fma2(w[j][p], g[K - 1 - j][p], out[i][p]);
#pragma unroll
                    for (int j = 0; j < K - 1; ++j) win[j][p] = win[j + 1][p];
                }
            }
            T* op = dx + (t - (K - 1)) * a.y.st;
#pragma unroll
            for (int i = 0; i < U; ++i) {
                if (!EDGE) {
                    Pairs<V>::store(op + i * a.y.st, out[i]);
                    continue;
                }
                const int s = t + i - (K - 1);
                if (t + i >= tend || (s < t0 && run > 0)) continue;  // the run before has it
                if (s >= len) {  // zero, also where a filter is not finite
#pragma unroll
                    for (int p = 0; p < N; ++p) out[i][p] = dup2(0.f);
                }
                const int kept = s - len + K - 1;  // its row in the state after the call
                if (a.dstate_end && kept >= 0 && kept < K - 1) {
                    f32x2 e[N];
                    Pairs<V>::load(a.dstate_end + so + (long long)kept * a.d, e);
#pragma unroll
                    for (int p = 0; p < N; ++p) out[i][p] = add2(out[i][p], e[p]);
                }
                if (s >= 0) Pairs<V>::store(dx + s * a.y.st, out[i]);
                else if (a.dstate) Pairs<V>::store(a.dstate + so + (long long)(s + K - 1) * a.d, out[i]);
            }
        };
        if constexpr (RING) {
#pragma unroll
            for (int k = 0; k < CONV_RING - 1; ++k) fetch(k, t0 + k * U);
        } else {
            fetch(0, t0);
        }
        // a run behind the sequence multiplies its window by zeros only: zero too, so that what lies
        // before it (of an empty sequence, its state) reaches dw of no other sequence, finite or not
        const bool behind = t0 >= len;
        conv_load_window<T, V, K>(a, x, behind ? nullptr : state, t0, behind ? 0 : len, win);
#pragma unroll
        for (int j = 0; j < K; ++j)
#pragma unroll
            for (int p = 0; p < N; ++p) g[j][p] = dup2(0.f);
        const int inner = min(t1, len - (K - 1));  // tokens before it are in no state after the call
        auto walk = [&](auto act) {
            for (int t = t0, k = 0; t < tend; t += U, ++k) {
                if (t >= t0 + K - 1 && t + U <= inner) group(k, t, Flag<false>(), act);
                else group(k, t, Flag<true>(), act);
            }
        };
        if (a.act) walk(Flag<true>());
        else walk(Flag<false>());
        if (RING) async_wait<0>();  // the next run fills the ring from its start
    }
#pragma unroll
    for (int p = 0; p < N; ++p) {
        float lo, hi;
#pragma unroll
        for (int j = 0; j < K; ++j) {
            unpack2(dw[j][p], lo, hi);
            s_part[warp][j][2 * p][lane] = lo;
            s_part[warp][j][2 * p + 1][lane] = hi;
        }
        unpack2(db[p], lo, hi);
        s_part[warp][K][2 * p][lane] = lo;
        s_part[warp][K][2 * p + 1][lane] = hi;
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

// dw[c][j] and dbias[c] from the blocks' shares, in order: eight interleaved segments of blocks, then
// the segments.
constexpr int CSUM_SEG = 8;
__global__ void __launch_bounds__(32 * CSUM_SEG) conv_sum_kernel(const float* part, int blocks,
                                                                 long long C, int K, float* dw,
                                                                 float* dbias) {
    __shared__ float s[CSUM_SEG][32];
    const int lane = threadIdx.x & 31, seg = threadIdx.x >> 5;
    const long long i = (long long)blockIdx.x * 32 + lane, n = C * (K + 1);
    float sum = 0.f;
    if (i < n) {
#pragma unroll 4
        for (int p = seg; p < blocks; p += CSUM_SEG) sum += part[p * n + i];
    }
    s[seg][lane] = sum;
    __syncthreads();
    if (seg > 0 || i >= n) return;
#pragma unroll
    for (int k = 1; k < CSUM_SEG; ++k) sum += s[k][lane];
    const long long c = i % C;
    const int j = (int)(i / C);
    if (j < K) dw[c * K + j] = sum;
    else if (dbias) dbias[c] = sum;
}

}  // namespace ssm
}  // namespace sdm
