// Gradient of the selective scan.  With dp_t = dy_t z sigmoid(z) (dy_t without a gate), tokens
// walked backwards and g the gradient that reaches h_t from the tokens behind it:
//   dh = C_t dp_t + g,   w = dh a_t,   q = w h_{t-1},   g <- w
//   dA += s_t q,   ds = sum_n (A q + dh B_t u_t),   du = Dskip dp_t + s_t sum_n dh B_t
//   dB_t += dh s_t u_t,   dC_t += dp_t h_t (over the group's channels)
//   ddelta = ds sigmoid(delta + dt_bias),  dz = dy_t y_t dsilu(z),  dDskip += dp_t u_t
//
// h_{t-1} is needed in reverse, and undoing h_t = a h_{t-1} + b divides by a small a; so it is
// computed again from states kept on the way.  The tokens are split into chunks of 32 whose start
// states and carries the SCAN_CHUNK_REV walk and scan_carry_kernel find, which also makes the chunks
// independent.  A warp takes the channel tiles of a chunk one after another: it walks a tile's 32
// tokens forward keeping every 8th state in shared memory, then takes the groups of 8 from the
// last: forward through the group with states and decays in registers, then back.  Four states a
// lane, so that a group's 8 x 4 states and decays fit.  The next tile's rows are on their way
// (cp.async) meanwhile.
//
// Tokens behind the sequence have a step and inputs of zero, which leave the sums as they are only
// while the states and what comes to them are finite (an empty sequence's need not be), so their
// outputs, and dA of a chunk without tokens, are written as zero.
//
// dB and dC sum over channels: over a warp's channels by shuffles that halve the number of values
// with each step, over its tiles and then the block's warps in shared memory, over blocks by
// scan_bc_sum_kernel, all in a fixed order.
//
// Bound by issue and shared memory: about 155 instructions and 37 shared-memory cycles a token and
// eight channels of 16 states.  2 sequences of 2048 tokens, 2048 channels, bf16: 266 us (issue 58 %,
// shared memory 53 %), with the walks, carries and sums 363 us; three passes over the exponentials
// alone are 90 us.  Three blocks live on an SM in bf16 with 9 to 32 states, in the other forms two (of
// fp32 with up to 8 states one), by their shared memory; all are compiled for three, 168 registers,
// and spill 20 to 128 bytes a thread.
#pragma once

#include "selective_scan.cuh"

namespace sdm {
namespace ssm {

constexpr int BWD_WARPS = 4;
constexpr int BWD_CHUNK = 32;
constexpr int BWD_NPT = 4;

template <typename T>
struct ScanBwdArgs {
    ScanArgs<T> s;
    View<T> du, ddelta, dz;
    float* part_a;   // [B*nchunk][D][N]
    float* part_d;   // [B*nchunk][2][D]: dDskip, ddt_bias
    float* part_bc;  // [blocks of a group][B][T][G][2][N]
    float* dstate;
    int tiles, blocks;  // channel tiles of a warp, blocks of a group
};

template <typename T, int LN>
struct BwdShared {
    static constexpr int NN = BWD_NPT * LN, WCH = 32 / LN, W = BWD_CHUNK * WCH;
    struct Warp {
        T u[2][W], d[2][W], z[2][W], dy[2][W];
        float2 tok[W];              // a token's step and step * u
        float g[W];                 // its gated dy
        float yh[W], sA[W], sB[W];  // its sums of C h, A2 q and dh B
        float4 ck[BWD_CHUNK / SCAN_GRP][32];
        float acc[BWD_CHUNK * 2 * NN];  // dB and dC over the warp's tiles
    };
    T B[BWD_CHUNK * NN], C[BWD_CHUNK * NN];
    Warp w[BWD_WARPS];
};

// Four consecutive values from shared memory as two pairs.
SDM_DEV void quad(const float* p, f32x2 (&v)[2]) {
    const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(p);
    v[0] = x.x, v[1] = x.y;
}
SDM_DEV void quad(const bf16* p, f32x2 (&v)[2]) {
    const uint2 x = *reinterpret_cast<const uint2*>(p);
    v[0] = pack2(bf16_lo(x.x), bf16_hi(x.x)), v[1] = pack2(bf16_lo(x.y), bf16_hi(x.y));
}

template <typename T, int LN>
__global__ void __launch_bounds__(BWD_WARPS * 32, 3) scan_bwd_kernel(ScanBwdArgs<T> A) {
    constexpr int NPT = BWD_NPT, NN = NPT * LN, WCH = 32 / LN;
    constexpr int GL = LN < SCAN_GRP ? LN : SCAN_GRP;  // lanes that share a group's sums
    constexpr int OWN = SCAN_GRP / GL, PAIRS = BWD_CHUNK * WCH / 64, GROUPS = BWD_CHUNK / SCAN_GRP;
    const ScanArgs<T>& a = A.s;
    extern __shared__ __align__(16) char smem[];
    BwdShared<T, LN>& sh = *reinterpret_cast<BwdShared<T, LN>*>(smem);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    auto& w = sh.w[warp];
    const int nl = lane % LN, n0 = nl * NPT, wch = lane / LN;
    const int b = blockIdx.z, chunk = blockIdx.y;
    const int g = blockIdx.x / A.blocks, blk = blockIdx.x % A.blocks;
    const int dg = a.D / a.G;
    const int len = clamp_len(a.lens, b, a.T_);
    const int t0 = chunk * BWD_CHUNK, tend = min(t0 + BWD_CHUNK, a.T_), t1 = min(tend, len);
    const long long pc = (long long)b * a.nchunk + chunk;

    // the warp's tiles: every BWD_WARPS-th of the block's, which follow those of the blocks before
    const int all = (dg + WCH - 1) / WCH;
    auto tile_at = [&](int k) { return (blk * A.tiles + k) * BWD_WARPS + warp; };
    auto fetch = [&](int k) {
        const int tile = tile_at(k);
        if (k < A.tiles && tile < all && t1 > t0) {
            const int c0 = g * dg + tile * WCH, cols = min(WCH, dg - tile * WCH), p = k & 1;
            constexpr bool ODD = sizeof(T) == 2;
            RowCopy<T, WCH, BWD_CHUNK, ODD> ru, rd, ry, rz;
            ru.init(a.u, b * a.u.v.sb + c0, t0, cols);
            ru.fetch(0, t1 - t0, w.u[p]);
            rd.init(a.delta, b * a.delta.v.sb + c0, t0, cols);
            rd.fetch(0, t1 - t0, w.d[p]);
            ry.init(a.dy, b * a.dy.v.sb + c0, t0, cols);
            ry.fetch(0, t1 - t0, w.dy[p]);
            rz.held_for = nullptr;
            if (a.z.v.p) {
                rz.init(a.z, b * a.z.v.sb + c0, t0, cols);
                rz.fetch(0, t1 - t0, w.z[p]);
            }
            ru.flush();  // rows at odd addresses: all loaded, then all stored
            rd.flush();
            ry.flush();
            rz.flush();
        }
        async_commit();
    };
    fetch(0);
    {  // the chunk's B and C, zero behind the sequence
        const T* Bp = a.Bm.v.p + b * a.Bm.v.sb + g * a.Bm.v.sh;
        const T* Cp = a.Cm.v.p + b * a.Cm.v.sb + g * a.Cm.v.sh;
        for (int e = tid; e < BWD_CHUNK * NN; e += BWD_WARPS * 32) {
            const int t = t0 + e / NN, n = e % NN;
            const bool in = t < t1 && n < a.N;
            sh.B[e] = in ? Bp[t * a.Bm.v.st + n] : T(0.f);
            sh.C[e] = in ? Cp[t * a.Cm.v.st + n] : T(0.f);
        }
        for (int e = lane; e < BWD_CHUNK * 2 * NN; e += 32) w.acc[e] = 0.f;
    }
    __syncthreads();

    const f32x2 one = dup2(1.f), zero = dup2(0.f);
    const unsigned long long m_sp = a.softplus ? ~0ull : 0ull;
    const bool gate = a.z.v.p;
    const int ic = 2 * (lane % (WCH / 2));  // before and after the walk: a pair of channels
    const T* Bs = sh.B + n0;
    const T* Cs = sh.C + n0;
    for (int k = 0; k < A.tiles; ++k) {
        const int tile = tile_at(k);
        if (tile >= all) break;
        const int c0 = g * dg + tile * WCH, cols = min(WCH, dg - tile * WCH), p = k & 1;
        const int c = c0 + (wch < cols ? wch : 0);
        fetch(k + 1);
        f32x2 A2[2], h[2], gr[2], dA[2];
        {
            float av[NPT], hv[NPT], gv[NPT];
#pragma unroll
            for (int i = 0; i < NPT; ++i) {
                const bool in = wch < cols && n0 + i < a.N;
                const long long cn = (long long)c * a.N + n0 + i;
                const long long bcn = (long long)b * a.D * a.N + cn;
                av[i] = hv[i] = gv[i] = 0.f;
                if (in) {
                    av[i] = a.A[cn];
                    if (a.nchunk > 1) {
                        hv[i] = a.E[pc * a.D * a.N + cn];
                        gv[i] = a.R[pc * a.D * a.N + cn];
                    } else {
                        if (a.state && !a.fresh) hv[i] = a.state[bcn];
                        if (a.dstate_end) gv[i] = a.dstate_end[bcn];
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                A2[i] = pack2(decay_rate(av[2 * i]), decay_rate(av[2 * i + 1]));
                h[i] = pack2(hv[2 * i], hv[2 * i + 1]);
                gr[i] = pack2(gv[2 * i], gv[2 * i + 1]);
                dA[i] = zero;
            }
        }
        const int j0 = c0 + (ic < cols ? ic : 0), j1 = c0 + (ic + 1 < cols ? ic + 1 : 0);
        const f32x2 bias = a.dt_bias ? pack2(a.dt_bias[j0], a.dt_bias[j1]) : zero;
        const f32x2 skip = a.Dskip ? pack2(a.Dskip[j0], a.Dskip[j1]) : zero;
        async_wait<1>();
        __syncwarp();
        auto inside = [&](int e) { return t0 + e / WCH < t1 ? ~0ull : 0ull; };
#pragma unroll
        for (int q = 0; q < PAIRS; ++q) {
            const int e = 2 * (lane + 32 * q);
            float d[2], u[2], gy[2], z[2];
            Vec<2>::load(w.d[p] + e, d);
            Vec<2>::load(w.u[p] + e, u);
            Vec<2>::load(w.dy[p] + e, gy);
            f32x2 s2 = add2(pack2(d[0], d[1]), bias), g2 = pack2(gy[0], gy[1]);
            s2 = (softplus2(s2) & m_sp) | (s2 & ~m_sp);
            if (gate) {
                Vec<2>::load(w.z[p] + e, z);
                g2 = mul2(g2, silu2(pack2(z[0], z[1])));
            }
            s2 &= inside(e);
            g2 &= inside(e);
            const f32x2 su = mul2(s2, pack2(u[0], u[1])) & inside(e);
            float x0, x1, y0, y1;
            unpack2(s2, x0, x1);
            unpack2(su, y0, y1);
            *reinterpret_cast<float4*>(w.tok + e) = make_float4(x0, y0, x1, y1);
            *reinterpret_cast<f32x2*>(w.g + e) = g2;
        }
        __syncwarp();

        // forward: the state before every group but the last, which stays in h
#pragma unroll 1
        for (int q = 0; q < GROUPS - 1; ++q) {
            float4 c4;
            unpack2(h[0], c4.x, c4.y);
            unpack2(h[1], c4.z, c4.w);
            w.ck[q][lane] = c4;
#pragma unroll
            for (int i = 0; i < SCAN_GRP; ++i) {
                const float2 x = w.tok[(q * SCAN_GRP + i) * WCH + wch];
                const f32x2 d2 = dup2(x.x), e2 = dup2(x.y);
                f32x2 Bv[2];
                quad(Bs + (q * SCAN_GRP + i) * NN, Bv);
#pragma unroll
                for (int r = 0; r < 2; ++r)
                    h[r] = fma2(exp2_pair(mul2(d2, A2[r])), h[r], mul2(e2, Bv[r]));
            }
        }

        // backward, group by group
#pragma unroll 1
        for (int q = GROUPS - 1; q >= 0; --q) {
            if (q < GROUPS - 1) {
                const float4 c4 = w.ck[q][lane];
                h[0] = pack2(c4.x, c4.y);
                h[1] = pack2(c4.z, c4.w);
            }
            f32x2 hp[SCAN_GRP][2], dec[SCAN_GRP][2];
            float yh[SCAN_GRP], sA[SCAN_GRP], sB[SCAN_GRP];
#pragma unroll
            for (int i = 0; i < SCAN_GRP; ++i) {
                const float2 x = w.tok[(q * SCAN_GRP + i) * WCH + wch];
                const f32x2 d2 = dup2(x.x), e2 = dup2(x.y);
                f32x2 Bv[2], Cv[2], y2 = zero;
                quad(Bs + (q * SCAN_GRP + i) * NN, Bv);
                quad(Cs + (q * SCAN_GRP + i) * NN, Cv);
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    hp[i][r] = h[r];
                    dec[i][r] = exp2_pair(mul2(d2, A2[r]));
                    h[r] = fma2(dec[i][r], h[r], mul2(e2, Bv[r]));
                    y2 = fma2(h[r], Cv[r], y2);
                }
                float lo, hi;
                unpack2(y2, lo, hi);
                yh[i] = lo + hi;
            }
#pragma unroll
            for (int i = SCAN_GRP - 1; i >= 0; --i) {
                const int e = (q * SCAN_GRP + i) * WCH + wch;
                const float2 x = w.tok[e];
                const f32x2 d2 = dup2(x.x), e2 = dup2(x.y), g2 = dup2(w.g[e]);
                f32x2 Bv[2], Cv[2], sA2 = zero, sB2 = zero;
                quad(Bs + (q * SCAN_GRP + i) * NN, Bv);
                quad(Cs + (q * SCAN_GRP + i) * NN, Cv);
                float v[2 * NPT], lo, hi;
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const f32x2 dh = fma2(Cv[r], g2, gr[r]);
                    gr[r] = mul2(dh, dec[i][r]);
                    const f32x2 qq = mul2(gr[r], hp[i][r]);
                    dA[r] = fma2(d2, qq, dA[r]);
                    sA2 = fma2(A2[r], qq, sA2);
                    sB2 = fma2(dh, Bv[r], sB2);
                    unpack2(mul2(dh, e2), v[2 * r], v[2 * r + 1]);
                    const f32x2 ht = i + 1 < SCAN_GRP ? hp[i + 1 < SCAN_GRP ? i + 1 : i][r] : h[r];
                    unpack2(mul2(g2, ht), v[NPT + 2 * r], v[NPT + 2 * r + 1]);
                }
                unpack2(sA2, lo, hi);
                sA[i] = lo + hi;
                unpack2(sB2, lo, hi);
                sB[i] = lo + hi;
                // over the warp's channels; a lane keeps the values whose index has its bits
                int cnt = 2 * NPT, base = 0;
#pragma unroll
                for (int m = LN; m < 32; m <<= 1) {
                    if (cnt > 1) {
                        cnt >>= 1;
                        const bool upper = lane & m;
                        if (upper) base += cnt;
#pragma unroll
                        for (int r = 0; r < NPT; ++r)
                            if (r < cnt) {
                                const float mine = upper ? v[cnt + r] : v[r];
                                const float other = upper ? v[r] : v[cnt + r];
                                v[r] = mine + __shfl_xor_sync(0xffffffffu, other, m);
                            }
                    } else {
                        v[0] += __shfl_xor_sync(0xffffffffu, v[0], m);
                    }
                }
                constexpr int KEEP = WCH >= 2 * NPT ? 1 : 2 * NPT / WCH;
                if (wch < 2 * NPT) {
                    float* acc = w.acc + (q * SCAN_GRP + i) * 2 * NN + n0;
#pragma unroll
                    for (int r = 0; r < KEEP; ++r) {  // dB of states 0..3, dC of states 0..3
                        const int e8 = base + r;
                        acc[(e8 / NPT) * NN + e8 % NPT] += v[r];
                    }
                }
            }
            // over the channel's lanes; lane nl ends with tokens k*GL + nl
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
            spread_sum<GL>(yh, nl);
            spread_sum<GL>(sA, nl);
            spread_sum<GL>(sB, nl);
            if (nl < GL) {
#pragma unroll
                for (int i = 0; i < OWN; ++i) {
                    const int e = (q * SCAN_GRP + i * GL + nl) * WCH + wch;
                    w.yh[e] = yh[i];
                    w.sA[e] = sA[i];
                    w.sB[e] = sB[i];
                }
            }
        }
        __syncwarp();

        f32x2 dD = zero, dbias = zero;
        T* du = A.du.p + b * A.du.sb + c0 + ic;
        T* dd = A.ddelta.p + b * A.ddelta.sb + c0 + ic;
        T* dz = gate ? A.dz.p + b * A.dz.sb + c0 + ic : nullptr;
        const bool pair = ic + 1 < cols && A.du.st % 2 == 0 && A.ddelta.st % 2 == 0 &&
                          (((uintptr_t)du | (uintptr_t)dd) % (2 * sizeof(T))) == 0 &&
                          (!gate || (A.dz.st % 2 == 0 && (uintptr_t)dz % (2 * sizeof(T)) == 0));
        auto put = [&](T* at, f32x2 v) {
            float x[2];
            unpack2(v, x[0], x[1]);
            if (pair) {
                Vec<2>::store(at, x);
            } else {
                if (ic < cols) st(at, x[0]);
                if (ic + 1 < cols) st(at + 1, x[1]);
            }
        };
#pragma unroll
        for (int q = 0; q < PAIRS; ++q) {
            const int e = 2 * (lane + 32 * q), t = t0 + e / WCH;
            float d[2], u[2], y[2], z[2];
            Vec<2>::load(w.d[p] + e, d);
            Vec<2>::load(w.u[p] + e, u);
            Vec<2>::load(w.dy[p] + e, y);
            const f32x2 u2 = pack2(u[0], u[1]) & inside(e), dy2 = pack2(y[0], y[1]) & inside(e);
            const f32x2 sA2 = *reinterpret_cast<const f32x2*>(w.sA + e);
            const f32x2 sB2 = *reinterpret_cast<const f32x2*>(w.sB + e);
            const f32x2 g2 = *reinterpret_cast<const f32x2*>(w.g + e);
            const float4 x = *reinterpret_cast<const float4*>(w.tok + e);
            const f32x2 vdu = fma2(skip, g2, mul2(pack2(x.x, x.z), sB2));
            f32x2 vdd = fma2(sB2, u2, mul2(sA2, dup2(0.69314718055994530942f)));
            const f32x2 raw = add2(pack2(d[0], d[1]), bias);
            const f32x2 sg = mul2(vdd, rcp_pair(add2(exp2_pair(mul2(raw, dup2(-kLog2e))), one)));
            vdd = ((sg & m_sp) | (vdd & ~m_sp)) & inside(e);
            dD = fma2(g2, u2, dD);
            dbias = add2(dbias, vdd);
            if (t < tend) {
                put(du + t * A.du.st, vdu & inside(e));
                put(dd + t * A.ddelta.st, vdd);
                if (gate) {
                    Vec<2>::load(w.z[p] + e, z);
                    const f32x2 y2 = fma2(skip, u2, *reinterpret_cast<const f32x2*>(w.yh + e));
                    const f32x2 vdz = mul2(mul2(dy2, y2), dsilu2(pack2(z[0], z[1])));
                    put(dz + t * A.dz.st, vdz & inside(e));
                }
            }
        }
        float s0, s1, r0, r1;
        unpack2(dD, s0, s1);
        unpack2(dbias, r0, r1);
#pragma unroll
        for (int m = WCH / 2; m < 32; m <<= 1) {
            s0 += __shfl_xor_sync(0xffffffffu, s0, m);
            s1 += __shfl_xor_sync(0xffffffffu, s1, m);
            r0 += __shfl_xor_sync(0xffffffffu, r0, m);
            r1 += __shfl_xor_sync(0xffffffffu, r1, m);
        }
        if (lane < WCH / 2) {
            float* pd = A.part_d + pc * 2 * a.D + c0 + ic;
            if (ic < cols) pd[0] = s0, pd[a.D] = r0;
            if (ic + 1 < cols) pd[1] = s1, pd[a.D + 1] = r1;
        }
        float dv[NPT], gv[NPT];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            unpack2(dA[i], dv[2 * i], dv[2 * i + 1]);
            unpack2(gr[i], gv[2 * i], gv[2 * i + 1]);
        }
        if (wch < cols) {
#pragma unroll
            for (int i = 0; i < NPT; ++i)
                if (n0 + i < a.N) {
                    const long long cn = (long long)c * a.N + n0 + i;
                    A.part_a[pc * a.D * a.N + cn] = t1 > t0 ? dv[i] : 0.f;
                    if (chunk == 0 && A.dstate) A.dstate[(long long)b * a.D * a.N + cn] = gv[i];
                }
        }
        __syncwarp();  // the tile's rows and words are written again
    }
    async_wait<0>();
    __syncthreads();
    for (int e = tid; e < (tend - t0) * 2 * NN; e += BWD_WARPS * 32) {
        const int t = t0 + e / (2 * NN), k = e % (2 * NN), n = k % NN;
        if (n < a.N) {
            float sum = 0.f;
#pragma unroll
            for (int q = 0; q < BWD_WARPS; ++q) sum += sh.w[q].acc[e];
            A.part_bc[(((((long long)blk * a.B + b) * a.T_ + t) * a.G + g) * 2 + k / NN) * a.N + n] =
                t < t1 ? sum : 0.f;
        }
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
