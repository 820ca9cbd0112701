// Gradient of the selective scan.  With dp_t = dy_t z sigmoid(z) (dy_t without a gate), tokens
// walked backwards and g the gradient that reaches h_t from the tokens behind it:
//   dh = C_t dp_t + g,   w = dh a_t,   q = w h_{t-1},   g <- w
//   dA += s_t q,   ds = sum_n (A q + dh B_t u_t),   du = Dskip dp_t + s_t sum_n dh B_t
//   dB_t += dh s_t u_t,   dC_t += dp_t h_t (over the group's channels)
//   ddelta = ds sigmoid(delta + dt_bias),  dz = dy_t y_t dsilu(z),  dDskip += dp_t u_t
//
// h_{t-1} is needed in reverse, and undoing h_t = a h_{t-1} + b divides by a small a; so it is
// computed again from states kept on the way.  The tokens are split into chunks of 64 whose start
// states and carries scan_chunk_kernel and scan_carry_kernel find, which also makes the chunks
// independent.  scan_bwd_kernel walks a chunk forward keeping every 8th state in shared memory, then
// takes its groups of 8 from the last: forward through the group with states and decays in
// registers, then back.  Four states a thread, so that a group's 8 x 4 states and decays fit.
//
// dB and dC sum over channels: over a warp's channels by shuffles that halve the number of values
// with each step, over the block's warps and then its channel tiles in shared memory, over blocks
// by scan_bc_sum_kernel, all in a fixed order.
#pragma once

#include "selective_scan.cuh"

namespace sdm {
namespace ssm {

constexpr int BWD_THREADS = 256;
constexpr int BWD_CHUNK = 64;
constexpr int BWD_NPT = 4;
constexpr int BWD_WARPS = BWD_THREADS / 32;

template <typename T>
struct ScanBwdArgs {
    ScanArgs<T> s;
    View<T> du, ddelta, dz;
    float* part_a;   // [B*nchunk][D][N]
    float* part_d;   // [B*nchunk][2][D]: dDskip, ddt_bias
    float* part_bc;  // [blocks of a group][B][T][G][2][N]
    float* dstate;
    int tiles, blocks;  // channel tiles of a block, blocks of a group
};

// Bytes of dynamic shared memory for NN = 4*LN states.
__host__ __device__ constexpr size_t bwd_smem(int NN) {
    const size_t bc = (size_t)BWD_CHUNK * 2 * NN * 4;             // B, C
    const size_t acc = bc;                                         // dB, dC
    const size_t red = (size_t)BWD_WARPS * SCAN_GRP * 2 * NN * 4;  // the warps' shares of a group
    const size_t ck = (size_t)(BWD_CHUNK / SCAN_GRP) * BWD_THREADS * 16;
    const size_t tok = (size_t)(BWD_THREADS / (NN / 4)) * SCAN_GRP * 16;
    return bc + acc + red + ck + tok;
}

template <typename T, int LN>
__global__ void __launch_bounds__(BWD_THREADS) scan_bwd_kernel(ScanBwdArgs<T> A) {
    constexpr int NPT = BWD_NPT, NN = NPT * LN, OWN = SCAN_GRP / (LN < SCAN_GRP ? LN : SCAN_GRP);
    constexpr int GL = LN < SCAN_GRP ? LN : SCAN_GRP;  // lanes that share a group's tokens
    constexpr int CH = BWD_THREADS / LN;               // channels of a tile
    constexpr int WCH = 32 / LN;                       // of them in a warp
    const ScanArgs<T>& a = A.s;
    extern __shared__ __align__(16) char smem[];
    float* s_bc = reinterpret_cast<float*>(smem);             // [CHUNK][2][NN]
    float* s_acc = s_bc + BWD_CHUNK * 2 * NN;                 // [CHUNK][2][NN]
    float* s_red = s_acc + BWD_CHUNK * 2 * NN;                // [WARPS][GRP][2][NN]
    float4* s_ck = reinterpret_cast<float4*>(s_red + BWD_WARPS * SCAN_GRP * 2 * NN);
    float4* s_tok = s_ck + (BWD_CHUNK / SCAN_GRP) * BWD_THREADS;  // [WARPS][GRP][WCH]

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int nl = tid % LN, n0 = nl * NPT, wch = lane / LN;
    const int tl = nl % GL;  // which of a group's tokens this lane looks after (lanes nl < GL)
    const int b = blockIdx.z, ck = blockIdx.y;
    const int g = blockIdx.x / A.blocks, blk = blockIdx.x % A.blocks;
    const int dg = a.D / a.G;
    const int len = clamp_len(a.lens, b, a.T_);
    const int t0 = ck * a.chunk, tend = min(t0 + a.chunk, a.T_), t1 = min(tend, len);
    const int groups = (tend - t0 + SCAN_GRP - 1) / SCAN_GRP;
    const long long pc = (long long)b * a.nchunk + ck;

    {  // the chunk's B and C, zero behind the sequence
        const T* Bp = a.Bm.v.p + b * a.Bm.v.sb + g * a.Bm.v.sh;
        const T* Cp = a.Cm.v.p + b * a.Cm.v.sb + g * a.Cm.v.sh;
        for (int e = tid; e < BWD_CHUNK * 2 * NN; e += BWD_THREADS) {
            const int t = t0 + e / (2 * NN), k = e % (2 * NN), n = k % NN;
            float v = 0.f;
            if (t < t1 && n < a.N) v = k < NN ? ld(Bp + t * a.Bm.v.st + n) : ld(Cp + t * a.Cm.v.st + n);
            s_bc[e] = v;
            s_acc[e] = 0.f;
        }
    }
    __syncthreads();

    for (int tile = 0; tile < A.tiles; ++tile) {
        const int cg = (blk * A.tiles + tile) * CH + tid / LN;
        if ((blk * A.tiles + tile) * CH >= dg) break;  // the same for the whole block
        const bool live = cg < dg;
        const int c = g * dg + (live ? cg : 0);
        const T* up = a.u.v.p + b * a.u.v.sb + c;
        const T* dp = a.delta.v.p + b * a.delta.v.sb + c;
        const T* zp = a.z.v.p ? a.z.v.p + b * a.z.v.sb + c : nullptr;
        const T* yp = a.dy.v.p + b * a.dy.v.sb + c;
        const float bias = a.dt_bias ? a.dt_bias[c] : 0.f;
        const float skip = a.Dskip ? a.Dskip[c] : 0.f;
        float A2[NPT], h[NPT], gr[NPT], dA[NPT];
#pragma unroll
        for (int k = 0; k < NPT; ++k) {
            const bool in = live && n0 + k < a.N;
            const long long cn = (long long)c * a.N + n0 + k;
            A2[k] = in ? a.A[cn] * kLog2e : 0.f;
            h[k] = gr[k] = dA[k] = 0.f;
            if (in) {
                const long long bcn = (long long)b * a.D * a.N + cn;
                if (a.nchunk > 1) {
                    h[k] = a.E[pc * a.D * a.N + cn];
                    gr[k] = a.R[pc * a.D * a.N + cn];
                } else {
                    if (a.state && !a.fresh) h[k] = a.state[bcn];
                    if (a.dstate_end) gr[k] = a.dstate_end[bcn];
                }
            }
        }
        float dD = 0.f, dbias = 0.f;
        float4* tok = s_tok + warp * SCAN_GRP * WCH;

        // forward: the state before every group
        for (int q = 0; q < groups; ++q) {
            s_ck[q * BWD_THREADS + tid] = make_float4(h[0], h[1], h[2], h[3]);
            if (q + 1 == groups) break;
            const int tg = t0 + q * SCAN_GRP;
            __syncwarp();
            if (nl < GL) {
#pragma unroll
                for (int k = 0; k < OWN; ++k) {
                    const int i = k * GL + tl, t = tg + i;
                    float dt = 0.f, dtu = 0.f;
                    if (t < t1 && live) {
                        const float d = ld(dp + t * a.delta.v.st) + bias;
                        dt = a.softplus ? softplus(d) : d;
                        dtu = dt * ld(up + t * a.u.v.st);
                    }
                    tok[i * WCH + wch] = make_float4(dt, dtu, 0.f, 0.f);
                }
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < SCAN_GRP; ++i) {
                const float4 x = tok[i * WCH + wch];
                const float* Br = s_bc + (q * SCAN_GRP + i) * 2 * NN + n0;
#pragma unroll
                for (int k = 0; k < NPT; ++k)
                    h[k] = fmaf(exp2_fast(x.x * A2[k]), h[k], x.y * Br[k]);
            }
        }

        // backward, group by group
        for (int q = groups - 1; q >= 0; --q) {
            const int tg = t0 + q * SCAN_GRP;
            float u[OWN], dt[OWN], raw[OWN], z[OWN], dy[OWN];
            __syncwarp();
#pragma unroll
            for (int k = 0; k < OWN; ++k) {
                const int i = k * GL + tl, t = tg + i;
                u[k] = dt[k] = raw[k] = z[k] = dy[k] = 0.f;
                float gy = 0.f;
                if (t < t1 && live && nl < GL) {
                    u[k] = ld(up + t * a.u.v.st);
                    raw[k] = ld(dp + t * a.delta.v.st) + bias;
                    dt[k] = a.softplus ? softplus(raw[k]) : raw[k];
                    dy[k] = gy = ld(yp + t * a.dy.v.st);
                    if (zp) {
                        z[k] = ld(zp + t * a.z.v.st);
                        gy *= z[k] * sigmoid(z[k]);
                    }
                }
                if (nl < GL) tok[i * WCH + wch] = make_float4(dt[k], dt[k] * u[k], gy, 0.f);
            }
            __syncwarp();
            const float4 h0 = s_ck[q * BWD_THREADS + tid];
            h[0] = h0.x, h[1] = h0.y, h[2] = h0.z, h[3] = h0.w;
            float hp[SCAN_GRP][NPT], dec[SCAN_GRP][NPT];
            float yh[SCAN_GRP], sA[SCAN_GRP], sB[SCAN_GRP];
#pragma unroll
            for (int i = 0; i < SCAN_GRP; ++i) {
                const float4 x = tok[i * WCH + wch];
                const float* Br = s_bc + (q * SCAN_GRP + i) * 2 * NN + n0;
                yh[i] = 0.f;
#pragma unroll
                for (int k = 0; k < NPT; ++k) {
                    hp[i][k] = h[k];
                    dec[i][k] = exp2_fast(x.x * A2[k]);
                    h[k] = fmaf(dec[i][k], h[k], x.y * Br[k]);
                    yh[i] = fmaf(Br[NN + k], h[k], yh[i]);
                }
            }
#pragma unroll
            for (int i = SCAN_GRP - 1; i >= 0; --i) {
                const float4 x = tok[i * WCH + wch];
                const float* Br = s_bc + (q * SCAN_GRP + i) * 2 * NN + n0;
                float v[2 * NPT];
                sA[i] = sB[i] = 0.f;
#pragma unroll
                for (int k = 0; k < NPT; ++k) {
                    const float dh = fmaf(Br[NN + k], x.z, gr[k]);
                    gr[k] = dh * dec[i][k];
                    const float qq = gr[k] * hp[i][k];
                    dA[k] = fmaf(x.x, qq, dA[k]);
                    sA[i] = fmaf(A2[k], qq, sA[i]);
                    sB[i] = fmaf(dh, Br[k], sB[i]);
                    v[k] = dh * x.y;
                    v[NPT + k] = x.z * (i + 1 < SCAN_GRP ? hp[i + 1 < SCAN_GRP ? i + 1 : i][k] : h[k]);
                }
                // over the warp's channels; a lane keeps the values whose index has its bits
                int cnt = 2 * NPT, base = 0;
#pragma unroll
                for (int m = LN; m < 32; m <<= 1) {
                    if (cnt > 1) {
                        cnt >>= 1;
                        const bool upper = lane & m;
                        if (upper) base += cnt;
#pragma unroll
                        for (int k = 0; k < NPT; ++k)
                            if (k < cnt) {
                                const float mine = upper ? v[cnt + k] : v[k];
                                const float other = upper ? v[k] : v[cnt + k];
                                v[k] = mine + __shfl_xor_sync(0xffffffffu, other, m);
                            }
                    } else {
                        v[0] += __shfl_xor_sync(0xffffffffu, v[0], m);
                    }
                }
                constexpr int KEEP = WCH >= 2 * NPT ? 1 : 2 * NPT / WCH;
                float* red = s_red + (warp * SCAN_GRP + i) * 2 * NN;
                if (wch < 2 * NPT) {
#pragma unroll
                    for (int k = 0; k < KEEP; ++k) {
                        const int e = base + k;  // dB of states 0..3, dC of states 0..3
                        red[(e / NPT) * NN + n0 + e % NPT] = v[k];
                    }
                }
            }
            __syncthreads();
            for (int e = tid; e < SCAN_GRP * 2 * NN; e += BWD_THREADS) {
                float sum = 0.f;
#pragma unroll
                for (int w = 0; w < BWD_WARPS; ++w) sum += s_red[w * SCAN_GRP * 2 * NN + e];
                s_acc[q * SCAN_GRP * 2 * NN + e] += sum;
            }
            // over the channel's lanes; lane tl ends with its own tokens
            if (LN > SCAN_GRP) {
#pragma unroll
                for (int m = SCAN_GRP; m < LN; m <<= 1)
#pragma unroll
                    for (int i = 0; i < SCAN_GRP; ++i) {
                        yh[i] += __shfl_xor_sync(0xffffffffu, yh[i], m);
                        sA[i] += __shfl_xor_sync(0xffffffffu, sA[i], m);
                        sB[i] += __shfl_xor_sync(0xffffffffu, sB[i], m);
                    }
            }
            spread_sum<GL>(yh, tl);
            spread_sum<GL>(sA, tl);
            spread_sum<GL>(sB, tl);
#pragma unroll
            for (int k = 0; k < OWN; ++k) {
                const int t = tg + k * GL + tl;
                if (t >= tend || !live || nl >= GL) continue;
                float vdu = 0.f, vdd = 0.f, vdz = 0.f;
                if (t < t1) {
                    float gy = dy[k];
                    if (zp) {
                        const float sg = sigmoid(z[k]);
                        const float y = fmaf(skip, u[k], yh[k]);
                        vdz = dy[k] * y * (sg * (1.f + z[k] * (1.f - sg)));
                        gy *= z[k] * sg;
                    }
                    vdu = fmaf(skip, gy, dt[k] * sB[k]);
                    vdd = fmaf(sA[k], 0.69314718055994530942f, sB[k] * u[k]);
                    if (a.softplus) vdd *= sigmoid(raw[k]);
                    dD = fmaf(gy, u[k], dD);
                    dbias += vdd;
                }
                st(A.du.p + b * A.du.sb + t * A.du.st + c, vdu);
                st(A.ddelta.p + b * A.ddelta.sb + t * A.ddelta.st + c, vdd);
                if (zp) st(A.dz.p + b * A.dz.sb + t * A.dz.st + c, vdz);
            }
            __syncthreads();  // s_red is written again
        }

#pragma unroll
        for (int m = 1; m < LN; m <<= 1) {
            dD += __shfl_xor_sync(0xffffffffu, dD, m);
            dbias += __shfl_xor_sync(0xffffffffu, dbias, m);
        }
        if (live) {
#pragma unroll
            for (int k = 0; k < NPT; ++k)
                if (n0 + k < a.N) {
                    const long long cn = (long long)c * a.N + n0 + k;
                    A.part_a[pc * a.D * a.N + cn] = dA[k];
                    if (ck == 0 && A.dstate) A.dstate[(long long)b * a.D * a.N + cn] = gr[k];
                }
            if (nl == 0) {
                A.part_d[pc * 2 * a.D + c] = dD;
                A.part_d[(pc * 2 + 1) * a.D + c] = dbias;
            }
        }
    }
    __syncthreads();
    for (int e = tid; e < (tend - t0) * 2 * NN; e += BWD_THREADS) {
        const int t = t0 + e / (2 * NN), k = e % (2 * NN), n = k % NN;
        if (n < a.N)
            A.part_bc[(((((long long)blk * a.B + b) * a.T_ + t) * a.G + g) * 2 + k / NN) * a.N + n] =
                s_acc[e];
    }
}

// dB and dC from the blocks' shares, in order.
template <typename T>
__global__ void __launch_bounds__(256) scan_bc_sum_kernel(const float* part, int blocks,
                                                          long long btg, int N, T* dB, T* dC) {
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x, n = btg * 2 * N;
    if (i >= n) return;
    float sum = 0.f;
    for (int p = 0; p < blocks; ++p) sum += part[p * n + i];
    const long long row = i / (2 * N);
    const int k = (int)(i % (2 * N));
    if (k < N) st(dB + row * N + k, sum);
    else st(dC + row * N + (k - N), sum);
}

// out[e] = sum over p of part[p][e] for e < n, in a fixed order: 8 interleaved segments of p, then
// the segments.  Columns [0, na) are dA, then D of dDskip, then D of ddt_bias.
constexpr int DSUM_SEG = 8;
__global__ void __launch_bounds__(32 * DSUM_SEG) scan_param_sum_kernel(
    const float* part_a, const float* part_d, long long P, long long na, int D, float* dA,
    float* dDskip, float* ddt_bias) {
    __shared__ float s[DSUM_SEG][32];
    const int lane = threadIdx.x & 31, seg = threadIdx.x >> 5;
    const long long e = (long long)blockIdx.x * 32 + lane;
    const bool in = e < na + 2LL * D;
    const float* src = e < na ? part_a + e : part_d + (e - na);
    const long long step = e < na ? na : 2LL * D;
    float sum = 0.f;
    if (in)
#pragma unroll 4
        for (long long p = seg; p < P; p += DSUM_SEG) sum += src[p * step];
    s[seg][lane] = sum;
    __syncthreads();
    if (seg == 0 && in) {
#pragma unroll
        for (int k = 1; k < DSUM_SEG; ++k) sum += s[k][lane];
        if (e < na) dA[e] = sum;
        else if (e < na + D) {
            if (dDskip) dDskip[e - na] = sum;
        } else if (ddt_bias) {
            ddt_bias[e - na - D] = sum;
        }
    }
}

}  // namespace ssm
}  // namespace sdm
