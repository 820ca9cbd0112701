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
// A warp works alone, on 32/LN channels of one sequence, in tiles of 16 or 32 tokens: cp.async brings the
// next tiles' activations to shared memory; what a token needs once a channel (softplus, before;
// gate and rounding, after) is spread over all lanes, by token and channel pair; between the two
// every lane walks the tile's tokens with its states.  One warp a block, so that the SMs get equal
// numbers of them.
//
// Where the channels alone do not fill the GPU the tokens are split into chunks: the decay over a
// chunk is exp(A sum s), so a chunk's effect on the state is its end state from zero and the sum
// of its steps.  The same walk computes those first (the exponentials once more),
// scan_carry_kernel chains them, and every chunk's outputs start from its true state.
//
// Measured, 16 states: 2 sequences of 4096 tokens, 4096 channels, bf16, 274 us (119 us of
// exponentials; issue 60 %, exponential unit 54 %, shared memory 57 %, 1.7 warps a sub-partition);
// one of 16384 tokens, 512 channels, fp32, 114 us in 37 chunks.
#pragma once

#include "ssm_util.cuh"

namespace sdm {
namespace ssm {

// Tokens staged and walked at a time, and tiles in shared memory: three in use, the others on their
// way.  Longer tiles pay where a sub-partition has a warp or two of four states a lane (bf16, 1024
// tokens of 4096 channels: 61 us in tiles of 32, 71 us in tiles of 16; two sequences 86 and 92 us);
// with eight states a lane they do not fit its registers (133 and 197 us), and rows of fp32 are kept
// to what lets eight warps live on an SM.
template <typename T, int NPT>
struct ScanTile {
    static constexpr int TILE = NPT <= 4 && sizeof(T) == 2 ? 32 : 16;
    static constexpr int STAGES = TILE == 32 || (NPT > 4 && sizeof(T) == 4) ? 4 : 6;
};
constexpr int SCAN_ROUND = 32;  // chunks are whole tiles of either
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
    int run;            // tokens of a walk: its chunk, or (SCAN_CHUNK_REV) several
};

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

// Copies W elements of each of TILE rows of a view (tokens t.., zero from t1 on and behind
// `cols`) to shared memory, by the warp, tile after tile.  Where the rows allow whole pieces of
// PIECE bytes a lane copies the same pieces of every tile and keeps their address, so that a piece
// costs a comparison, an addition and the copy.  Rows of bf16 at odd addresses (an odd width or
// stride) cannot go asynchronously: with HOLD a lane loads its elements of a tile to registers and
// stores them when the next tile is fetched, so that it does not wait for them either.
template <typename T, int W, int TILE, bool HOLD = false>
struct RowCopy {
    static constexpr int HELD = HOLD ? (TILE * W + 31) / 32 : 1;
    T held[HELD];
    T* held_for;
    static constexpr int ROW = W * (int)sizeof(T), PIECE = ROW < 16 ? ROW : 16, PER = ROW / PIECE;
    static constexpr int ITER = (TILE * PER + 31) / 32, RSTEP = 32 / PER;  // rows between a lane's pieces
    static_assert(PER <= 32 && (PER & (PER - 1)) == 0, "pieces of a row");
    const T* p;           // element (t0, 0)
    const char* next;     // the lane's first piece of the next tile
    long long stride;
    int piece, cols, bytes;
    SDM_DEV void init(const Rows<T>& r, long long at, int t0, int columns) {
        const int lane = threadIdx.x & 31;
        stride = r.v.st;
        p = r.v.p + at + t0 * stride;
        piece = r.piece;
        cols = columns;
        held_for = nullptr;
        const int k = lane % PER * PIECE;
        next = reinterpret_cast<const char*>(p + lane / PER * stride) + k;
        bytes = lane < TILE * PER ? min(max(cols * (int)sizeof(T) - k, 0), PIECE) : 0;
    }
    // Rows that allow smaller pieces only (or, of bf16 at odd addresses, none).
    template <int BYTES>
    SDM_DEV void small(int first, int left, T* s) const {
        constexpr int E = BYTES / (int)sizeof(T);
        if constexpr (BYTES < PIECE) {
            for (int i = threadIdx.x & 31; i < TILE * W / E; i += 32) {
                const int r = i * E / W, k = i * E % W;
                const int n = r < left ? min(max((cols - k) * (int)sizeof(T), 0), BYTES) : 0;
                async_copy<BYTES>(s + i * E, n ? p + (first + r) * stride + k : p, n);
            }
        }
    }
    // The tile that starts `first` tokens behind t0; `left` tokens remain from there.
    SDM_DEV void fetch(int first, int left, T* s) {
        if (piece >= PIECE) {
            const int lane = threadIdx.x & 31;
            char* dst = reinterpret_cast<char*>(s) + lane * PIECE;
            if (TILE * PER >= 32 || lane < TILE * PER) {
#pragma unroll
                for (int i = 0; i < ITER; ++i)
                    async_copy<PIECE>(dst + i * 32 * PIECE, next + i * RSTEP * stride * (long long)sizeof(T),
                                      lane / PER + i * RSTEP < left ? bytes : 0);
            }
            next += TILE * stride * (long long)sizeof(T);
        } else if (piece == 8) {
            small<8>(first, left, s);
        } else if (piece == 4) {
            small<4>(first, left, s);
        } else if (HOLD) {
            load(first, left);
            held_for = s;
        }
    }
    SDM_DEV void load(int first, int left) {
#pragma unroll
        for (int j = 0; j < HELD; ++j) {
            const int i = (threadIdx.x & 31) + 32 * j, r = i / W, k = i % W;
            held[j] = T(0.f);
            if (i < TILE * W && r < left && k < cols) held[j] = p[(first + r) * stride + k];
        }
    }
    // Stores what is held.
    SDM_DEV void flush() {
        if constexpr (HOLD) {
            if (!held_for) return;
#pragma unroll
            for (int j = 0; j < HELD; ++j) {
                const int i = (threadIdx.x & 31) + 32 * j;
                if (i < TILE * W) held_for[i] = held[j];
            }
            held_for = nullptr;
        }
    }
};

// N consecutive values from shared memory.
template <int N>
SDM_DEV void row_floats(const bf16* p, float (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
        float x[4];
        Vec<4>::load(p + i, x);
        v[i] = x[0], v[i + 1] = x[1], v[i + 2] = x[2], v[i + 3] = x[3];
    }
}
template <int N>
SDM_DEV void row_floats(const float* p, float (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
        const float4 x = *reinterpret_cast<const float4*>(p + i);
        v[i] = x.x, v[i + 1] = x.y, v[i + 2] = x.z, v[i + 3] = x.w;
    }
}

// Sum of a channel's LN neighbouring shares.
template <int LN>
SDM_DEV float share_sum(const float* p) {
    if constexpr (LN == 1) {
        return p[0];
    } else if constexpr (LN == 2) {
        const float2 v = *reinterpret_cast<const float2*>(p);
        return v.x + v.y;
    } else {
        float s = 0.f;
#pragma unroll
        for (int l = 0; l < LN; l += 4) {
            const float4 v = *reinterpret_cast<const float4*>(p + l);
            s += (v.x + v.y) + (v.z + v.w);
        }
        return s;
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
            for (int i = 0; i < NPT; i += 4) {
                float x[4] = {0.f, 0.f, 0.f, 0.f};
                if (live && n0 + i < N) Vec<4>::load(p + n0 + i, x);
#pragma unroll
                for (int k = 0; k < 4; ++k) v[i + k] = x[k];
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
            for (int i = 0; i < NPT; i += 4) {
                const float x[4] = {v[i], v[i + 1], v[i + 2], v[i + 3]};
                if (n0 + i < N) Vec<4>::store(p + n0 + i, x);
            }
        } else {
#pragma unroll
            for (int i = 0; i < NPT; ++i)
                if (n0 + i < N) p[n0 + i] = v[i];
        }
    }
};

// A tile in shared memory: u, delta, z, dy [TILE][WCH] and B, C [TILE][NN] as they are stored.
template <typename T, int NN, int WCH, int MODE, int TILE>
struct ScanStage {
    static constexpr int W = TILE * WCH, SPARE = 16 / sizeof(T);
    T u[W], d[W], z[MODE == SCAN_CHUNK ? SPARE : W], dy[MODE == SCAN_CHUNK_REV ? W : SPARE];
    T B[TILE * NN], C[TILE * NN];
};
template <typename T, int NPT, int LN, int MODE>
struct ScanShared {
    static constexpr int NN = NPT * LN, WCH = 32 / LN, TILE = ScanTile<T, NPT>::TILE;
    static constexpr int WIDE = sizeof(T) == 2 && NPT > 4 ? TILE * NN : 4;
    ScanStage<T, NN, WCH, MODE, TILE> st[ScanTile<T, NPT>::STAGES];
    float B[WIDE], C[MODE == SCAN_CHUNK ? 4 : WIDE];   // the tile's rows, of bf16
    float2 tok[TILE * WCH];                            // a token's step and step * u
    float g[MODE == SCAN_CHUNK_REV ? TILE * WCH : 4];  // its gated dy
    float y[MODE == SCAN_OUT ? TILE * 32 : 4];         // each lane's share of its sum C h
};

// The walk over a chunk.  SCAN_OUT: its outputs from the start state (and the end state where the
// sequence ends in it).  SCAN_CHUNK: its end state from zero and the sum of its steps;
// SCAN_CHUNK_REV: also what its outputs' gradients carry to the token before it,
// sum_t (prod_{s<=t} a_s) C_t dy_t.
//
// Three things overlap in an iteration, so that the few warps that there are keep the units busy:
// the walk of tile i, the steps of tile i+1 (with its rows of B and C as floats) and the outputs of
// tile i-1.  What they read from shared memory is loaded first, what they write is stored last, and
// nothing in between branches (the flags are masks, the tiles before the first and behind the last
// are computed from what lies there and dropped), so the compiler mixes their arithmetic.
// Shared memory gives the registers 128 bytes a clock, broadcast or not, which is why a token's
// step and input are two words and not two pairs, and why four states a lane read B and C as bf16
// (where they are) and convert them in registers (1024 tokens of 4096 channels, two sequences: 80
// us, as floats 84 us); eight states a lane, which read them half as often, take them as floats that
// are converted once (130 us, as bf16 138 us).  Two warps live on a sub-partition: more registers
// do better than a third.  ODD: some rows are of bf16 at odd addresses.
template <typename T, int NPT, int LN, int MODE, bool ODD>
__global__ void __launch_bounds__(32, 8) scan_walk_kernel(ScanArgs<T> a) {
    constexpr int NN = NPT * LN, NP = NPT / 2, WCH = 32 / LN;
    constexpr int TILE = ScanTile<T, NPT>::TILE, STAGES = ScanTile<T, NPT>::STAGES;
    constexpr int PAIRS = TILE * WCH / 64;  // of (token, channel pair) a lane
    constexpr int SB = NP >= 4 ? 4 : 8;      // tokens whose decays are computed ahead
    constexpr bool OUT = MODE == SCAN_OUT, REV = MODE == SCAN_CHUNK_REV, WIDE = sizeof(T) == 2 && NPT > 4;
    extern __shared__ __align__(16) char smem[];
    using Shared = ScanShared<T, NPT, LN, MODE>;
    Shared& sh = *reinterpret_cast<Shared*>(smem);
    const ScanLane<NPT, LN> L(a.D, a.G);
    const int lane = threadIdx.x;
    const int len = clamp_len(a.lens, L.b, a.T_);
    const int t0 = blockIdx.y * a.run, t1 = min(t0 + a.run, len);
    if (OUT && t0 >= len && blockIdx.y > 0) return;
    const bool gate = a.z.v.p && (OUT || REV);
    RowCopy<T, WCH, TILE, ODD> cu, cd, cz, cg;
    RowCopy<T, NN, TILE, ODD> cB, cC;
    cu.init(a.u, L.b * a.u.v.sb + L.c0, t0, L.cols);
    cd.init(a.delta, L.b * a.delta.v.sb + L.c0, t0, L.cols);
    if (gate) cz.init(a.z, L.b * a.z.v.sb + L.c0, t0, L.cols);
    if (REV) cg.init(a.dy, L.b * a.dy.v.sb + L.c0, t0, L.cols);
    cB.init(a.Bm, L.b * a.Bm.v.sb + L.g * a.Bm.v.sh, t0, a.N);
    if (OUT || REV) cC.init(a.Cm, L.b * a.Cm.v.sb + L.g * a.Cm.v.sh, t0, a.N);
    auto fetch = [&](int tile) {
        const int first = tile * TILE, left = t1 - t0 - first;
        if (ODD) {  // the tile before it
            cu.flush();
            cd.flush();
            if (gate) cz.flush();
            if (REV) cg.flush();
            cB.flush();
            if (OUT || REV) cC.flush();
        }
        if (left > 0) {
            auto& s = sh.st[tile % STAGES];
            cu.fetch(first, left, s.u);
            cd.fetch(first, left, s.d);
            if (gate) cz.fetch(first, left, s.z);
            if (REV) cg.fetch(first, left, s.dy);
            cB.fetch(first, left, s.B);
            if (OUT || REV) cC.fetch(first, left, s.C);
        }
        async_commit();
    };
#pragma unroll 1
    for (int i = 0; i < STAGES - 1; ++i) fetch(i);

    float tmp[NPT], A2[NPT];
    f32x2 h[NP], r[NP], P[NP];
    L.load(a.A + (long long)L.c * a.N, a.N, A2);
#pragma unroll
    for (int i = 0; i < NPT; ++i) {
        A2[i] = decay_rate(A2[i]);
        tmp[i] = 0.f;
    }
    const long long at = ((long long)L.b * a.nchunk + blockIdx.y) * a.D + L.c;
    float* state = OUT && a.state ? a.state + ((long long)L.b * a.D + L.c) * a.N : nullptr;
    if (OUT && a.nchunk > 1) L.load(a.E + at * a.N, a.N, tmp);
    else if (state && !a.fresh) L.load(state, a.N, tmp);
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        h[i] = pack2(tmp[2 * i], tmp[2 * i + 1]);
        r[i] = dup2(0.f);
        P[i] = dup2(1.f);
    }

    // before and after the walk a lane looks after two channels, of every (64/WCH)-th token
    const int ic = 2 * (lane % (WCH / 2));
    const int i0 = L.c0 + (ic < L.cols ? ic : 0), i1 = L.c0 + (ic + 1 < L.cols ? ic + 1 : 0);
    const f32x2 bias = a.dt_bias ? pack2(a.dt_bias[i0], a.dt_bias[i1]) : dup2(0.f);
    const f32x2 skip = OUT && a.Dskip ? pack2(a.Dskip[i0], a.Dskip[i1]) : dup2(0.f);
    T* yp = OUT ? a.y.p + L.b * a.y.sb + L.c0 + ic : nullptr;
    const bool pair = OUT && ic + 1 < L.cols && ((uintptr_t)yp % (2 * sizeof(T))) == 0 && a.y.st % 2 == 0;
    f32x2 steps = dup2(0.f), ahead = dup2(0.f);  // of the chunk so far, of the next tile
    const unsigned long long m_sp = a.softplus ? ~0ull : 0ull, m_z = gate ? ~0ull : 0ull;
    const float2* tok = sh.tok + lane / LN;

    // the steps of a tile: its rows, then its words for the walk
    f32x2 st2[PAIRS], su2[PAIRS], g2[PAIRS];
    auto tile_steps = [&](int tile) {
        const auto& s = sh.st[tile % STAGES];
        if (!OUT) {
            steps = add2(steps, ahead);
            ahead = dup2(0.f);
        }
#pragma unroll
        for (int k = 0; k < PAIRS; ++k) {
            const int e = 2 * (lane + 32 * k);
            float d[2], u[2], g[2], z[2];
            Vec<2>::load(s.d + e, d);
            Vec<2>::load(s.u + e, u);
            if (REV) Vec<2>::load(s.dy + e, g);
            if (REV) Vec<2>::load(s.z + e, z);
            st2[k] = add2(pack2(d[0], d[1]), bias);
            const f32x2 sp = softplus2(st2[k]);
            st2[k] = (sp & m_sp) | (st2[k] & ~m_sp);
            st2[k] &= t0 + tile * TILE + e / WCH < t1 ? ~0ull : 0ull;  // else the state stays
            su2[k] = mul2(st2[k], pack2(u[0], u[1]));
            if (!OUT) ahead = add2(ahead, st2[k]);
            if (REV) {
                g2[k] = pack2(g[0], g[1]);
                const f32x2 gz = mul2(g2[k], silu2(pack2(z[0], z[1])));
                g2[k] = (gz & m_z) | (g2[k] & ~m_z);
            }
        }
    };
    auto put_steps = [&]() {
#pragma unroll
        for (int k = 0; k < PAIRS; ++k) {
            const int e = 2 * (lane + 32 * k);
            float s0, s1, w0, w1;
            unpack2(st2[k], s0, s1);
            unpack2(su2[k], w0, w1);
            *reinterpret_cast<float4*>(sh.tok + e) = make_float4(s0, w0, s1, w1);
            if (REV) *reinterpret_cast<f32x2*>(sh.g + e) = g2[k];
        }
    };
    // the outputs of a tile whose sums are in sh.y
    f32x2 o2[PAIRS];
    auto tile_outputs = [&](int tile) {
        const auto& s = sh.st[tile % STAGES];
#pragma unroll
        for (int k = 0; k < PAIRS; ++k) {
            const int e = 2 * (lane + 32 * k);
            float u[2], z[2];
            const f32x2 y = pack2(share_sum<LN>(sh.y + e * LN), share_sum<LN>(sh.y + (e + 1) * LN));
            Vec<2>::load(s.u + e, u);
            Vec<2>::load(s.z + e, z);
            o2[k] = fma2(skip, pack2(u[0], u[1]), y);
            const f32x2 oz = mul2(o2[k], silu2(pack2(z[0], z[1])));
            o2[k] = (oz & m_z) | (o2[k] & ~m_z);
        }
    };
    auto put_outputs = [&](int tile) {
#pragma unroll
        for (int k = 0; k < PAIRS; ++k) {
            const int t = t0 + tile * TILE + 2 * (lane + 32 * k) / WCH;
            if (t >= t0 && t < t1) {
                float y[2];
                unpack2(o2[k], y[0], y[1]);
                T* o = yp + t * a.y.st;
                if (pair) {
                    Vec<2>::store(o, y);
                } else {
                    if (ic < L.cols) st(o, y[0]);
                    if (ic + 1 < L.cols) st(o + 1, y[1]);
                }
            }
        }
    };

    // where the walk finds a tile's rows of B and C
    auto rows_B = [&](int tile) {
        if constexpr (WIDE) return static_cast<const float*>(sh.B);
        else return static_cast<const T*>(sh.st[tile % STAGES].B);
    };
    auto rows_C = [&](int tile) {
        if constexpr (WIDE) return static_cast<const float*>(sh.C);
        else return static_cast<const T*>(sh.st[tile % STAGES].C);
    };
    // a tile's rows of B and C, of bf16, as floats
    constexpr int RW = WIDE ? (TILE * NN + 255) / 256 : 0;
    float wB[RW + 1][8], wC[RW + 1][8];
    auto wide_rows = [&](int tile) {
        if constexpr (WIDE) {
            const auto& s = sh.st[tile % STAGES];
#pragma unroll
            for (int k = 0; k < RW; ++k) {
                const int e = (lane + 32 * k) * 8 % (TILE * NN);  // a small tile: some twice
                Vec<8>::load(s.B + e, wB[k]);
                if (OUT || REV) Vec<8>::load(s.C + e, wC[k]);
            }
        }
    };
    auto put_rows = [&]() {
#pragma unroll
        for (int k = 0; k < RW; ++k) {
            const int e = (lane + 32 * k) * 8 % (TILE * NN);
#pragma unroll
            for (int i = 0; i < 8; i += 4) {
                *reinterpret_cast<float4*>(sh.B + e + i) =
                    make_float4(wB[k][i], wB[k][i + 1], wB[k][i + 2], wB[k][i + 3]);
                if (OUT || REV)
                    *reinterpret_cast<float4*>(sh.C + e + i) =
                        make_float4(wC[k][i], wC[k][i + 1], wC[k][i + 2], wC[k][i + 3]);
            }
        }
    };

    // what a chunk leaves; the next starts from zero
    auto emit = [&](int chunk) {
        const long long to = ((long long)L.b * a.nchunk + chunk) * a.D + L.c;
        float v[NPT];
#pragma unroll
        for (int i = 0; i < NP; ++i) unpack2(h[i], v[2 * i], v[2 * i + 1]);
        L.store(a.E + to * a.N, a.N, v);
        if (REV) {
#pragma unroll
            for (int i = 0; i < NP; ++i) unpack2(r[i], v[2 * i], v[2 * i + 1]);
            L.store(a.R + to * a.N, a.N, v);
        }
        float s0, s1;
        unpack2(steps, s0, s1);
#pragma unroll
        for (int m = WCH / 2; m < 32; m <<= 1) {
            s0 += __shfl_xor_sync(0xffffffffu, s0, m);
            s1 += __shfl_xor_sync(0xffffffffu, s1, m);
        }
        if (lane < WCH / 2) {
            float* S = a.S + ((long long)L.b * a.nchunk + chunk) * a.D + L.c0;
            if (ic < L.cols) S[ic] = s0;
            if (ic + 1 < L.cols) S[ic + 1] = s1;
        }
        steps = dup2(0.f);
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            h[i] = r[i] = dup2(0.f);
            P[i] = dup2(1.f);
        }
    };

    const int tiles = max(0, (t1 - t0 + TILE - 1) / TILE);
    if (tiles > 0) {
        async_wait<STAGES - 2>();
        __syncwarp();
        tile_steps(0);
        wide_rows(0);
        put_steps();
        put_rows();
        async_wait<STAGES - 3>();
        __syncwarp();
    }
    for (int tile = 0; tile < tiles; ++tile) {
        if (OUT) tile_outputs(tile + STAGES - 1);  // of the tile before this one
        tile_steps(tile + 1);  // adds this tile's steps to the chunk's
        wide_rows(tile + 1);
        const auto* Bs = rows_B(tile) + L.n0;
        const auto* Cs = rows_C(tile) + L.n0;
        float y[TILE];
#pragma unroll
        for (int q0 = 0; q0 < TILE; q0 += SB) {
            f32x2 dec[SB][NP], in[SB][NP];
#pragma unroll
            for (int i = 0; i < SB; ++i) {
                const float2 x = tok[(q0 + i) * WCH];
                float B[NPT];
                row_floats<NPT>(Bs + (q0 + i) * NN, B);
#pragma unroll
                for (int p = 0; p < NP; ++p) {
                    dec[i][p] = exp2_pair(mul2(dup2(x.x), pack2(A2[2 * p], A2[2 * p + 1])));
                    in[i][p] = mul2(dup2(x.y), pack2(B[2 * p], B[2 * p + 1]));
                }
            }
#pragma unroll
            for (int i = 0; i < SB; ++i) {
                float C[NPT], g = 0.f;
                if (OUT || REV) row_floats<NPT>(Cs + (q0 + i) * NN, C);
                if (REV) g = sh.g[(q0 + i) * WCH + lane / LN];
                f32x2 acc = dup2(0.f);
#pragma unroll
                for (int p = 0; p < NP; ++p) {
                    h[p] = fma2(dec[i][p], h[p], in[i][p]);
                    if (OUT) {
                        const f32x2 c2 = pack2(C[2 * p], C[2 * p + 1]);
                        acc = p == 0 ? mul2(h[p], c2) : fma2(h[p], c2, acc);
                    }
                    if (REV) {
                        P[p] = mul2(P[p], dec[i][p]);
                        r[p] = fma2(P[p], pack2(g * C[2 * p], g * C[2 * p + 1]), r[p]);
                    }
                }
                if (OUT) {
                    float lo, hi;
                    unpack2(acc, lo, hi);
                    y[q0 + i] = lo + hi;
                }
            }
        }
        __syncwarp();  // the tile's words and the outputs' stage have been read
        if (OUT) {
#pragma unroll
            for (int q = 0; q < TILE; ++q) sh.y[q * 32 + lane] = y[q];
            put_outputs(tile - 1);
        }
        put_steps();
        put_rows();
        if (!OUT && (tile + 1) * TILE % a.chunk == 0)
            emit(blockIdx.y * (a.run / a.chunk) + (tile + 1) * TILE / a.chunk - 1);
        fetch(tile + STAGES - 1);  // into the stage of the tile before this one
        async_wait<STAGES - 3>();  // the tile after the next is there
        __syncwarp();
    }
    if (OUT && tiles > 0) {
        tile_outputs(tiles - 1);
        put_outputs(tiles - 1);
    }
    if (!OUT) {  // the chunks that end behind the last whole one, the empty ones among them
        const int first = blockIdx.y * (a.run / a.chunk) + tiles * TILE / a.chunk;
        const int last = min((int)(blockIdx.y + 1) * (a.run / a.chunk), a.nchunk);
        for (int k = first; k < last; ++k) emit(k);
    }
    if (OUT) {
        if (state && t1 == len) {
#pragma unroll
            for (int i = 0; i < NP; ++i) unpack2(h[i], tmp[2 * i], tmp[2 * i + 1]);
            L.store(state, a.N, tmp);
        }
    }
}

// Chains the chunks: E[k] becomes the state that chunk k starts from and, in the gradient (the
// grid's second row), R[k] the carry that reaches its last token.  One thread a state; the loads of
// SCAN_AHEAD chunks are in flight together.  Both directions of 2 x 64 chunks of 2048 x 16 states,
// 34 MB read and 34 MB written, take 20 us: 3.4 TB/s, half of the copy rate, bound by the latency of a
// thread's chunks in turn.
constexpr int SCAN_AHEAD = 8;
template <typename T>
__global__ void __launch_bounds__(256) scan_carry_kernel(ScanArgs<T> a) {
    const bool rev = blockIdx.y;
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    const long long dn = (long long)a.D * a.N;
    if (i >= a.B * dn) return;
    const long long b = i / dn, cn = i % dn;
    const float A2 = decay_rate(a.A[cn]);
    const long long last = a.nchunk - 1;
    const long long step = rev ? -1 : 1;
    float* E = (rev ? a.R : a.E) + (b * a.nchunk + (rev ? last : 0)) * dn + cn;
    const float* S = a.S + (b * a.nchunk + (rev ? last : 0)) * a.D + cn / a.N;
    float h = 0.f;
    if (rev) {
        if (a.dstate_end) h = a.dstate_end[i];
    } else if (a.state && !a.fresh) {
        h = a.state[i];
    }
    float e[SCAN_AHEAD], s[SCAN_AHEAD];
    auto fetch = [&](long long k) {
#pragma unroll
        for (int q = 0; q < SCAN_AHEAD; ++q)
            if (k + q < last) {  // the last chunk's effect is not needed
                e[q] = E[(k + q) * step * dn];
                s[q] = S[(k + q) * step * a.D];
            }
    };
    fetch(0);
    for (long long k = 0; k <= last; k += SCAN_AHEAD) {
        float ce[SCAN_AHEAD], cs[SCAN_AHEAD];
#pragma unroll
        for (int q = 0; q < SCAN_AHEAD; ++q) ce[q] = e[q], cs[q] = s[q];
        fetch(k + SCAN_AHEAD);
#pragma unroll
        for (int q = 0; q < SCAN_AHEAD; ++q)
            if (k + q <= last) {
                E[(k + q) * step * dn] = h;
                if (k + q < last) h = fmaf(exp2_fast(cs[q] * A2), h, ce[q]);
            }
    }
}

// One token a sequence: bound by the state, read and written once (8 N bytes a channel against 8 of
// activations in bf16; 64 sequences of 4096 channels of 16 states, 36 MB, take 13.4 us with cold
// caches, 2.7 TB/s, of which about 3 us are the launch).  Four states a thread, so that a warp's
// state accesses are whole contiguous lines, of NB sequences, whose loads are all in flight before
// the first is used and share the channel's A, bias and addresses.  vec: B and C can be read four at
// a time.
template <typename T, int LN, int NB>
__global__ void __launch_bounds__(256) scan_step_kernel(ScanArgs<T> a, bool vec) {
    const int nl = threadIdx.x % LN, n0 = nl * 4;
    const int c = blockIdx.x * (256 / LN) + threadIdx.x / LN, b0 = blockIdx.y * NB;
    const int cc = c < a.D ? c : 0, g = cc / (a.D / a.G), left = c < a.D ? a.N - n0 : 0;
    const bool four = a.N % 4 == 0;
    f32x2 A2[2], h[NB][2];
    T u[NB], d[NB], z[NB];
    Raw<T, 4> Bv[NB], Cv[NB];
    bool on[NB];
    auto load4 = [&](const float* p, f32x2 (&v)[2]) {
        v[0] = v[1] = dup2(0.f);
        if (four) {
            if (left > 0) {
                const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(p);
                v[0] = x.x, v[1] = x.y;
            }
        } else {
            v[0] = pack2(left > 0 ? p[0] : 0.f, left > 1 ? p[1] : 0.f);
            v[1] = pack2(left > 2 ? p[2] : 0.f, left > 3 ? p[3] : 0.f);
        }
    };
    float* state = a.state ? a.state + ((long long)b0 * a.D + cc) * a.N + n0 : nullptr;
    const long long sb = (long long)a.D * a.N;
#pragma unroll
    for (int j = 0; j < NB; ++j) {
        const int b = b0 + j;
        on[j] = b < a.B && clamp_len(a.lens, b, 1) > 0;
        h[j][0] = h[j][1] = dup2(0.f);
        if (b < a.B && state && !a.fresh) load4(state + j * sb, h[j]);
        u[j] = d[j] = z[j] = T(0.f);
        Bv[j].clear();
        Cv[j].clear();
        if (on[j]) {
            u[j] = a.u.v.p[b * a.u.v.sb + cc];
            d[j] = a.delta.v.p[b * a.delta.v.sb + cc];
            if (a.z.v.p) z[j] = a.z.v.p[b * a.z.v.sb + cc];
            const T* Bp = a.Bm.v.p + b * a.Bm.v.sb + g * a.Bm.v.sh + n0;
            const T* Cp = a.Cm.v.p + b * a.Cm.v.sb + g * a.Cm.v.sh + n0;
            if (vec) {
                if (left > 0) {
                    Bv[j].load(Bp);
                    Cv[j].load(Cp);
                }
            } else {
                Bv[j].load(Bp, left);
                Cv[j].load(Cp, left);
            }
        }
    }
    load4(a.A + (long long)cc * a.N + n0, A2);
    const float bias = a.dt_bias ? a.dt_bias[cc] : 0.f, skip = a.Dskip ? a.Dskip[cc] : 0.f;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        float lo, hi;
        unpack2(A2[r], lo, hi);
        A2[r] = pack2(decay_rate(lo), decay_rate(hi));
    }
#pragma unroll
    for (int j = 0; j < NB; ++j) {
        const int b = b0 + j;
        if (b >= a.B) break;
        float s = ld(&d[j]) + bias;
        if (a.softplus) s = softplus(s);
        const float su = s * ld(&u[j]);
        f32x2 Bf[2], Cf[2], acc = dup2(0.f);
        Bv[j].pairs(Bf);
        Cv[j].pairs(Cf);
        if (on[j]) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                h[j][r] = fma2(exp2_pair(mul2(dup2(s), A2[r])), h[j][r], mul2(dup2(su), Bf[r]));
                acc = fma2(h[j][r], Cf[r], acc);
            }
        }
        float lo, hi;
        unpack2(acc, lo, hi);
        float y = lo + hi;
#pragma unroll
        for (int m = 1; m < LN; m <<= 1) y += __shfl_xor_sync(0xffffffffu, y, m);
        if (nl == 0 && c < a.D && on[j]) {
            y = fmaf(skip, ld(&u[j]), y);
            if (a.z.v.p) {
                const float zf = ld(&z[j]);
                y *= zf * sigmoid(zf);
            }
            st(a.y.p + b * a.y.sb + cc, y);
        }
        if (state && left > 0 && (on[j] || a.fresh)) {
            float* to = state + j * sb;
            if (four) {
                ulonglong2 x;
                x.x = h[j][0], x.y = h[j][1];
                *reinterpret_cast<ulonglong2*>(to) = x;
            } else {
                float v[4];
                unpack2(h[j][0], v[0], v[1]);
                unpack2(h[j][1], v[2], v[3]);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (k < left) to[k] = v[k];
            }
        }
    }
}

}  // namespace ssm
}  // namespace sdm
