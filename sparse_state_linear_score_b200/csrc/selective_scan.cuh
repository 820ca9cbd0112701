// Selective state-space scan, D channels of N states (B and C shared by a group's channels):
//   s_t = softplus(delta_t + dt_bias),  h_t[n] = exp(s_t A[n]) h_{t-1}[n] + s_t B_t[n] u_t,
//   y_t = (sum_n C_t[n] h_t[n] + Dskip u_t) z_t sigmoid(z_t)
//
// Per token and channel: one exponential, one product and three multiply-adds a state, against
// four activations of memory traffic.  At N = 16 in bf16 that is bound by the exponential unit
// (16 a clock and SM: 148 SMs at 1.9 GHz make 4.5e12 a second), about three times above the
// memory's time.  So the states live in registers over the whole run, NPT a thread, LN
// neighbouring lanes a channel, and products and multiply-adds go two states at a time (f32x2).
//
// A warp works alone, on 32/LN channels of one sequence, in tiles of 16 tokens: cp.async brings the
// next three tiles' activations to shared memory; what a token needs once a channel (softplus,
// before; gate and rounding, after) is spread over all lanes, one token and channel each; between
// the two every lane walks the tile's tokens with its states.  One warp a block, so that the SMs
// get equal numbers of them.
//
// Where the channels alone do not fill the GPU the tokens are split into chunks: the decay over a
// chunk is exp(A sum s), so a chunk's effect on the state is its end state from zero and the sum
// of its steps.  The same walk computes those first (the exponentials once more),
// scan_carry_kernel chains them, and every chunk's outputs start from its true state.
#pragma once

#include "ssm_util.cuh"

namespace sdm {
namespace ssm {

constexpr int SCAN_TILE = 16;   // tokens staged and walked at a time
constexpr int SCAN_STAGES = 4;  // tiles in shared memory: one in use, three on their way
constexpr int SCAN_GRP = 8;     // tokens whose outputs are summed over a channel's lanes together
enum { SCAN_OUT = 0, SCAN_CHUNK = 1, SCAN_CHUNK_REV = 2 };  // what a walk computes

// A view and the bytes of an asynchronous copy that its rows' addresses allow (16, 8, 4, or 0:
// element by element).
template <typename T>
struct Rows {
    View<const T> v;
    int piece;
};

template <typename T>
struct ScanArgs {
    Rows<T> u, delta, z, Bm, Cm, dy;
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

// Copies W elements of each of TILE rows (tokens t.. of a sequence, zero from t1 on and behind
// `cols`) to s[TILE][W], by the warp.  Pieces of 16, 8 or 4 bytes go asynchronously.
template <typename T, int W, int TILE>
SDM_DEV void rows_to_smem(const T* p, long long stride, int piece, int t, int t1, int cols, T* s) {
    const int lane = threadIdx.x & 31;
    if (piece) {
        const int per = W * (int)sizeof(T) / piece;  // pieces of a row, a power of two
        const int sh = __ffs(per) - 1;
        for (int i = lane; i < TILE * per; i += 32) {
            const int r = i >> sh, k = i & (per - 1);
            int bytes = t + r < t1 ? cols * (int)sizeof(T) - k * piece : 0;
            bytes = bytes < 0 ? 0 : (bytes > piece ? piece : bytes);
            const char* src = reinterpret_cast<const char*>(p);
            if (bytes > 0) src = reinterpret_cast<const char*>(p + (t + r) * stride) + k * piece;
            const uint32_t dst = (uint32_t)__cvta_generic_to_shared(s + r * W) + k * piece;
            if (piece == 16)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                             "r"(bytes) : "memory");
            else if (piece == 8)
                asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src),
                             "r"(bytes) : "memory");
            else
                asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src),
                             "r"(bytes) : "memory");
        }
    } else {
        for (int i = lane; i < TILE * W; i += 32) {
            const int r = i / W, k = i % W;
            T v = T(0.f);
            if (t + r < t1 && k < cols) v = p[(t + r) * stride + k];
            s[i] = v;
        }
    }
}
SDM_DEV void async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
SDM_DEV void async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Rows of float as they are, rows of bf16 converted to floats in `f`; by the warp.
template <typename T, int COUNT>
SDM_DEV const float* rows_as_float(const T* s, float* f) {
    if constexpr (sizeof(T) == 4) {
        return reinterpret_cast<const float*>(s);
    } else {
#pragma unroll
        for (int i = (threadIdx.x & 31) * 4; i < COUNT; i += 128) {
            float v[4];
            Vec<4>::load(s + i, v);
            Vec<4>::store(f + i, v);
        }
        return f;
    }
}

// The states a lane holds: of the warp's channels the (lane / LN)-th, NPT states of it.
template <int NPT, int LN>
struct ScanLane {
    static constexpr int WCH = 32 / LN;
    int g, c0, cols, c, nl, n0, b;  // group, first channel and channels of the warp; own channel
    bool live;
    SDM_DEV ScanLane(int D, int G) {
        const int dg = D / G, tiles = (dg + WCH - 1) / WCH, lane = threadIdx.x & 31;
        g = blockIdx.x / tiles;
        const int first = (blockIdx.x % tiles) * WCH;
        c0 = g * dg + first;
        cols = min(WCH, dg - first);
        live = lane / LN < cols;
        c = c0 + (live ? lane / LN : 0);
        nl = lane % LN;
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

// A tile in shared memory: u, delta, z, dy [TILE][WCH] and B, C [TILE][NN] as they are stored.
template <typename T, int NN, int WCH, int MODE>
struct ScanStage {
    static constexpr int W = SCAN_TILE * WCH, SPARE = 16 / sizeof(T);
    T u[W], d[W], z[MODE == SCAN_CHUNK ? SPARE : W], dy[MODE == SCAN_CHUNK_REV ? W : SPARE];
    T B[SCAN_TILE * NN], C[SCAN_TILE * NN];
};
template <typename T, int NN, int WCH, int MODE>
struct ScanShared {
    ScanStage<T, NN, WCH, MODE> st[SCAN_STAGES];
    float B[SCAN_TILE * NN], C[SCAN_TILE * NN];  // the tile's, of bf16 rows
    float2 tok[SCAN_TILE * WCH];                 // a token's step and step * u
    float y[SCAN_TILE * WCH];                    // its sum C h, or (gradient) the gated dy
};

// The walk over a chunk.  SCAN_OUT: its outputs from the start state (and the end state where the
// sequence ends in it).  SCAN_CHUNK: its end state from zero and the sum of its steps;
// SCAN_CHUNK_REV: also what its outputs' gradients carry to the token before it,
// sum_t (prod_{s<=t} a_s) C_t dy_t.
template <typename T, int NPT, int LN, int MODE>
__global__ void __launch_bounds__(32) scan_walk_kernel(ScanArgs<T> a) {
    constexpr int NN = NPT * LN, NP = NPT / 2, WCH = 32 / LN, ITEMS = SCAN_TILE * WCH / 32;
    constexpr bool OUT = MODE == SCAN_OUT, REV = MODE == SCAN_CHUNK_REV;
    extern __shared__ __align__(16) char smem[];
    using Shared = ScanShared<T, NN, WCH, MODE>;
    Shared& sh = *reinterpret_cast<Shared*>(smem);
    const ScanLane<NPT, LN> L(a.D, a.G);
    const int lane = threadIdx.x;
    const int len = clamp_len(a.lens, L.b, a.T_);
    const int t0 = blockIdx.y * a.chunk, t1 = min(t0 + a.chunk, len);
    if (OUT && t0 >= len && blockIdx.y > 0) return;
    const bool gate = a.z.v.p && (OUT || REV);
    const T* up = a.u.v.p + L.b * a.u.v.sb + L.c0;
    const T* dp = a.delta.v.p + L.b * a.delta.v.sb + L.c0;
    const T* zp = gate ? a.z.v.p + L.b * a.z.v.sb + L.c0 : nullptr;
    const T* gp = REV ? a.dy.v.p + L.b * a.dy.v.sb + L.c0 : nullptr;
    const T* Bp = a.Bm.v.p + L.b * a.Bm.v.sb + L.g * a.Bm.v.sh;
    const T* Cp = a.Cm.v.p + L.b * a.Cm.v.sb + L.g * a.Cm.v.sh;
    auto fetch = [&](int tile) {
        const int t = t0 + tile * SCAN_TILE;
        if (t < t1) {
            auto& s = sh.st[tile % SCAN_STAGES];
            rows_to_smem<T, WCH, SCAN_TILE>(up, a.u.v.st, a.u.piece, t, t1, L.cols, s.u);
            rows_to_smem<T, WCH, SCAN_TILE>(dp, a.delta.v.st, a.delta.piece, t, t1, L.cols, s.d);
            if (gate) rows_to_smem<T, WCH, SCAN_TILE>(zp, a.z.v.st, a.z.piece, t, t1, L.cols, s.z);
            if (REV) rows_to_smem<T, WCH, SCAN_TILE>(gp, a.dy.v.st, a.dy.piece, t, t1, L.cols, s.dy);
            rows_to_smem<T, NN, SCAN_TILE>(Bp, a.Bm.v.st, a.Bm.piece, t, t1, a.N, s.B);
            if (OUT || REV)
                rows_to_smem<T, NN, SCAN_TILE>(Cp, a.Cm.v.st, a.Cm.piece, t, t1, a.N, s.C);
        }
        async_commit();
    };
#pragma unroll
    for (int i = 0; i < SCAN_STAGES - 1; ++i) fetch(i);

    float tmp[NPT];
    f32x2 A2[NP], h[NP], r[NP], P[NP];
    L.load(a.A + (long long)L.c * a.N, a.N, tmp);
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        A2[i] = pack2(tmp[2 * i] * kLog2e, tmp[2 * i + 1] * kLog2e);
        r[i] = pack2(0.f, 0.f);
        P[i] = pack2(1.f, 1.f);
    }
#pragma unroll
    for (int i = 0; i < NPT; ++i) tmp[i] = 0.f;
    const long long at = ((long long)L.b * a.nchunk + blockIdx.y) * a.D + L.c;
    float* state = OUT && a.state ? a.state + ((long long)L.b * a.D + L.c) * a.N : nullptr;
    if (OUT && a.nchunk > 1) L.load(a.E + at * a.N, a.N, tmp);
    else if (state && !a.fresh) L.load(state, a.N, tmp);
#pragma unroll
    for (int i = 0; i < NP; ++i) h[i] = pack2(tmp[2 * i], tmp[2 * i + 1]);

    // before and after the walk a lane looks after channel lane % WCH, every (32/WCH)-th token
    const int ic = lane % WCH, ig = L.c0 + (ic < L.cols ? ic : 0);
    const float bias = a.dt_bias ? a.dt_bias[ig] : 0.f;
    const float skip = OUT && a.Dskip ? a.Dskip[ig] : 0.f;
    T* yp = OUT ? a.y.p + L.b * a.y.sb + L.c0 + ic : nullptr;
    float steps = 0.f;
    const float2* tok = sh.tok + lane / LN;

    for (int tile = 0; t0 + tile * SCAN_TILE < t1; ++tile) {
        const int tt = t0 + tile * SCAN_TILE;
        async_wait<SCAN_STAGES - 2>();
        __syncwarp();
        fetch(tile + SCAN_STAGES - 1);  // into the stage that the tile before this one used
        const auto& s = sh.st[tile % SCAN_STAGES];
#pragma unroll
        for (int k = 0; k < ITEMS; ++k) {
            const int e = lane + 32 * k, t = tt + e / WCH;
            float step = ld(s.d + e) + bias;
            if (a.softplus) step = softplus(step);
            if (t >= t1) step = 0.f;  // behind the sequence: the state stays
            sh.tok[e] = make_float2(step, step * ld(s.u + e));
            if (!OUT) steps += step;
            if (REV) {
                float g = ld(s.dy + e);
                if (gate) {
                    const float z = ld(s.z + e);
                    g *= z * sigmoid(z);
                }
                sh.y[e] = g;
            }
        }
        const float* Bs = rows_as_float<T, SCAN_TILE * NN>(s.B, sh.B);
        const float* Cs = nullptr;
        if (OUT || REV) Cs = rows_as_float<T, SCAN_TILE * NN>(s.C, sh.C);
        __syncwarp();
#pragma unroll
        for (int gq = 0; gq < SCAN_TILE / SCAN_GRP; ++gq) {
            float y[SCAN_GRP];
#pragma unroll
            for (int i = 0; i < SCAN_GRP; ++i) {
                const int q = gq * SCAN_GRP + i;
                const float2 x = tok[q * WCH];
                const f32x2 d2 = pack2(x.x, x.x), e2 = pack2(x.y, x.y);
                const f32x2* Br = reinterpret_cast<const f32x2*>(Bs + q * NN + L.n0);
                const f32x2* Cr = reinterpret_cast<const f32x2*>(Cs + q * NN + L.n0);
                f32x2 acc = pack2(0.f, 0.f), g2;
                if (REV) {
                    const float g = sh.y[q * WCH + lane / LN];
                    g2 = pack2(g, g);
                }
#pragma unroll
                for (int p = 0; p < NP; ++p) {
                    const f32x2 dec = exp2_pair(mul2(d2, A2[p]));
                    h[p] = fma2(dec, h[p], mul2(e2, Br[p]));
                    if (OUT) acc = fma2(h[p], Cr[p], acc);
                    if (REV) {
                        P[p] = mul2(P[p], dec);
                        r[p] = fma2(P[p], mul2(g2, Cr[p]), r[p]);
                    }
                }
                if (OUT) {
                    float lo, hi;
                    unpack2(acc, lo, hi);
                    y[i] = lo + hi;
                }
            }
            if (OUT) {
                spread_sum<LN>(y, L.nl);
#pragma unroll
                for (int k = 0; k < SCAN_GRP / LN; ++k)
                    sh.y[(gq * SCAN_GRP + k * LN + L.nl) * WCH + lane / LN] = y[k];
            }
        }
        __syncwarp();
        if (OUT) {
#pragma unroll
            for (int k = 0; k < ITEMS; ++k) {
                const int e = lane + 32 * k, t = tt + e / WCH;
                float v = fmaf(skip, ld(s.u + e), sh.y[e]);
                if (gate) {
                    const float z = ld(s.z + e);
                    v *= z * sigmoid(z);
                }
                if (t < t1 && ic < L.cols) st(yp + t * a.y.st, v);
            }
        }
    }
    if (OUT) {
        if (state && t1 == len) {
#pragma unroll
            for (int i = 0; i < NP; ++i) unpack2(h[i], tmp[2 * i], tmp[2 * i + 1]);
            L.store(state, a.N, tmp);
        }
    } else {
#pragma unroll
        for (int i = 0; i < NP; ++i) unpack2(h[i], tmp[2 * i], tmp[2 * i + 1]);
        L.store(a.E + at * a.N, a.N, tmp);
        if (REV) {
#pragma unroll
            for (int i = 0; i < NP; ++i) unpack2(r[i], tmp[2 * i], tmp[2 * i + 1]);
            L.store(a.R + at * a.N, a.N, tmp);
        }
#pragma unroll
        for (int m = WCH; m < 32; m <<= 1) steps += __shfl_xor_sync(0xffffffffu, steps, m);
        if (lane < L.cols) a.S[((long long)L.b * a.nchunk + blockIdx.y) * a.D + L.c0 + lane] = steps;
    }
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
        float d = ld(a.delta.v.p + b * a.delta.v.sb + cc) + (a.dt_bias ? a.dt_bias[cc] : 0.f);
        if (a.softplus) d = softplus(d);
        const float u = ld(a.u.v.p + b * a.u.v.sb + cc);
        const T* Bp = a.Bm.v.p + b * a.Bm.v.sb + g * a.Bm.v.sh + n0;
        const T* Cp = a.Cm.v.p + b * a.Cm.v.sb + g * a.Cm.v.sh + n0;
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
            if (a.z.v.p) {
                const float z = ld(a.z.v.p + b * a.z.v.sb + cc);
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
