// C ABI of the state-space block's operators (declared in include/sdm.h): host-side validation,
// workspace layout and launches of the short convolution, the selective scan and the block norms.
#include <stdint.h>

#include <algorithm>

#include "../../include/sdm.h"
#include "block_norm.cuh"
#include "selective_scan.cuh"
#include "selective_scan_bwd.cuh"
#include "short_conv.cuh"

using namespace sdm::ssm;

namespace {

constexpr int kSms = 148;
constexpr int kMaxGrid = 65535;  // of a grid's second and third axis
constexpr int kScanMaxT = kMaxGrid * BWD_CHUNK;  // the gradient's chunks are a grid's second axis

size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }
long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }

bool aligned(const void* p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

size_t elem_bytes(int32_t dtype) { return dtype == SDM_BF16 ? 2 : 4; }

bool known(int32_t dtype) { return dtype == SDM_F32 || dtype == SDM_BF16; }

sdm_status launched() { return cudaGetLastError() == cudaSuccess ? SDM_OK : SDM_ERR_CUDA; }

// A required input view; without tokens its data is not looked at.
sdm_status check_in(const sdm_view* v, int32_t dtype, int64_t T) {
    if (!v || (!v->data && T > 0)) return SDM_ERR_ARG;
    if (v->sb < 0 || v->sh < 0 || v->st < 0) return SDM_ERR_ARG;
    return aligned(v->data, elem_bytes(dtype)) ? SDM_OK : SDM_ERR_ALIGN;
}

// An output view of rows of `row` elements: its rows may not overlap.  The axes of more than one
// entry, from the smallest stride up, have to nest: each stride clears what lies inside it.
sdm_status check_out(const sdm_view* v, int32_t dtype, int64_t nb, int64_t nh, int64_t nt,
                     int64_t row) {
    const sdm_status e = check_in(v, dtype, nt);
    if (e) return e;
    struct Axis {
        int64_t stride, n;
    } ax[3] = {{v->sb, nb}, {v->sh, nh}, {v->st, nt}};
    std::sort(ax, ax + 3, [](const Axis& a, const Axis& b) { return a.stride < b.stride; });
    __int128 span = row;
    for (const Axis& x : ax) {
        if (x.n <= 1) continue;
        if (x.stride < span) return SDM_ERR_ARG;
        span += (__int128)x.stride * (x.n - 1);
    }
    return SDM_OK;
}

bool same_data(const sdm_view* a, const sdm_view* b, int64_t T) {
    return a && T > 0 && a->data == b->data;
}

template <typename T>
View<T> view(const sdm_view* v) {
    if (!v) return View<T>{nullptr, 0, 0, 0};
    return View<T>{static_cast<T*>(v->data), v->sb, v->sh, v->st};
}

// Four elements at a time where the rows allow it.
bool vec4_ok(const sdm_view* v, int32_t dtype) {
    return !v || (aligned(v->data, 4 * elem_bytes(dtype)) && v->sb % 4 == 0 && v->sh % 4 == 0 &&
                  v->st % 4 == 0);
}

// Dynamic shared memory beyond what a kernel gets unasked: 48 KB, of which these kernels' own arrays
// take 20 KB at most.  `most` is what any call of the kernel takes: the limit is the kernel's, and
// another host thread that set it to less would make this call's launch fail.
template <typename K>
bool allow_smem(K kernel, size_t bytes, size_t most) {
    if (bytes <= 28 * 1024) return true;
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most) ==
           cudaSuccess;
}

// ---- short convolution ---------------------------------------------------------------------
sdm_status check_conv(const sdm_conv_dims* d) {
    if (!d) return SDM_ERR_ARG;
    if (!known(d->x_dtype)) return SDM_ERR_DTYPE;
    if (d->act != SDM_ACT_NONE && d->act != SDM_ACT_SILU) return SDM_ERR_ARG;
    if (d->fresh != 0 && d->fresh != 1) return SDM_ERR_ARG;
    if (d->B < 1 || d->H < 1 || d->d < 1 || d->T < 0 || d->T > (1 << 30)) return SDM_ERR_SHAPE;
    if ((long long)d->B * d->H > kMaxGrid) return SDM_ERR_SHAPE;
    if (d->K < 1 || d->K > CONV_MAXK) return SDM_ERR_SHAPE;
    return SDM_OK;
}

struct ConvPlan {
    int run, runs;
    unsigned gx, gy;
};

// Tokens of a run: eight; twelve, what the ring holds at once, where that leaves 12 warps an SM; more,
// since a run reads K-1 tokens of its neighbour, as long as there are 24 warps an SM, or 48 where the
// sequences have lengths and runs behind them end at once.  (bf16, K = 4: 2 x 4 x 512 x 128 4.4 us
// in runs of 8, 4.7 us of 12; 2 x 4 x 4096 x 128 8.4 us in runs of 8, 7.1 us of 12, 8.9 us of 32;
// 8 x 16 x 2048 x 128 31 us in runs of 64, 34.7 and 33.5 us of 32 and 128; 8 x 16 x 8192 x 64 55 us in
// runs of 128, 57 us of 64, half of it padding 40 and 35 us.)
ConvPlan conv_plan(const sdm_conv_dims* d, int V, bool lens) {
    ConvPlan p;
    p.gx = (unsigned)ceil_div((long long)d->H * (d->d / V), 32);
    auto warps = [&](int run) { return (long long)p.gx * d->B * ceil_div(d->T, run); };
    p.run = V == 4 && warps(CONV_GRP * (CONV_RING - 1)) >= kSms * 12 ? CONV_GRP * (CONV_RING - 1)
                                                                     : CONV_RUN_MIN;
    for (int next = V == 4 ? 32 : 16; next <= 256 && warps(next) >= kSms * (lens ? 48 : 24); next *= 2)
        p.run = next;
    while (ceil_div((long long)d->B * ceil_div(d->T, p.run), CONV_WARPS) > kMaxGrid) p.run *= 2;
    p.runs = (int)std::max(1LL, ceil_div(d->T, p.run));
    p.gy = (unsigned)ceil_div((long long)d->B * p.runs, CONV_WARPS);
    return p;
}

// The gradient: runs of 128 tokens (the headline shape takes 88 us, in runs of 64 110 us), shorter
// ones where those leave SMs without three warps a sub-partition; four blocks an SM, three of them at
// a time, whose shares of dw are added afterwards.
ConvPlan conv_bwd_plan(const sdm_conv_dims* d, int V) {
    ConvPlan p;
    p.gx = (unsigned)ceil_div((long long)d->H * (d->d / V), 32);
    p.run = 128;
    while (p.run > 16 && (long long)p.gx * d->B * ceil_div(d->T, p.run) < kSms * 12) p.run /= 2;
    p.runs = (int)std::max(1LL, ceil_div(d->T, p.run));
    const long long need = ceil_div((long long)d->B * p.runs, CONV_WARPS);
    p.gy = (unsigned)std::max(1LL, std::min(need, 4LL * kSms / p.gx));
    return p;
}

template <typename T, int V, int K>
sdm_status launch_conv(const ConvArgs<T>& a, const ConvPlan& p, bool bwd, cudaStream_t s) {
    const dim3 grid(p.gx, p.gy);
    if (bwd) {
        constexpr size_t ring = conv_ring_bytes<T, V>(2);
        if (!allow_smem(short_conv_bwd_kernel<T, V, K>, ring, ring)) return SDM_ERR_CUDA;
        short_conv_bwd_kernel<T, V, K><<<grid, CONV_WARPS * 32, ring, s>>>(a);
    } else {
        short_conv_kernel<T, V, K><<<grid, CONV_WARPS * 32, conv_ring_bytes<T, V>(1), s>>>(a);
    }
    return launched();
}

template <typename T, int V>
sdm_status launch_conv_k(const ConvArgs<T>& a, const ConvPlan& p, bool bwd, cudaStream_t s) {
    switch (a.K) {
        case 1: return launch_conv<T, V, 1>(a, p, bwd, s);
        case 2: return launch_conv<T, V, 2>(a, p, bwd, s);
        case 3: return launch_conv<T, V, 3>(a, p, bwd, s);
        case 4: return launch_conv<T, V, 4>(a, p, bwd, s);
        case 5: return launch_conv<T, V, 5>(a, p, bwd, s);
        case 6: return launch_conv<T, V, 6>(a, p, bwd, s);
        case 7: return launch_conv<T, V, 7>(a, p, bwd, s);
        default: return launch_conv<T, V, 8>(a, p, bwd, s);
    }
}

template <typename T>
ConvArgs<T> conv_args(const sdm_conv_dims* d, const sdm_view* x, const float* w, const float* bias,
                      const void* state, const int32_t* lens) {
    ConvArgs<T> a{};
    a.x = view<const T>(x);
    a.w = w;
    a.bias = bias;
    a.state = d->K > 1 ? static_cast<T*>(const_cast<void*>(state)) : nullptr;
    a.lens = lens;
    a.B = d->B, a.H = d->H, a.T_ = d->T, a.d = d->d, a.K = d->K, a.act = d->act, a.fresh = d->fresh;
    return a;
}

template <typename T>
sdm_status run_conv(const sdm_conv_dims* d, const sdm_view* x, const float* w, const float* bias,
                    void* state, const int32_t* lens, const sdm_view* y, cudaStream_t s) {
    ConvArgs<T> a = conv_args<T>(d, x, w, bias, state, lens);
    a.y = view<T>(y);
    const bool v4 = d->d % 4 == 0 && vec4_ok(x, d->x_dtype) && vec4_ok(y, d->x_dtype);
    const ConvPlan p = conv_plan(d, v4 ? 4 : 1, lens != nullptr);
    a.run = p.run, a.runs = p.runs;
    return v4 ? launch_conv_k<T, 4>(a, p, false, s) : launch_conv_k<T, 1>(a, p, false, s);
}

template <typename T>
sdm_status run_conv_bwd(const sdm_conv_dims* d, const sdm_view* x, const float* w,
                        const float* bias, const void* state, const int32_t* lens,
                        const sdm_view* dy, const float* dstate_end, const sdm_view* dx, float* dw,
                        float* dbias, float* dstate, void* ws, cudaStream_t s) {
    ConvArgs<T> a = conv_args<T>(d, x, w, bias, state, lens);
    a.y = view<T>(dx);
    a.dy = view<const T>(dy);
    a.dstate_end = d->K > 1 ? dstate_end : nullptr;
    a.dstate = d->K > 1 ? dstate : nullptr;
    a.part = static_cast<float*>(ws);
    const bool v4 = d->d % 4 == 0 && vec4_ok(x, d->x_dtype) && vec4_ok(dy, d->x_dtype) &&
                    vec4_ok(dx, d->x_dtype);
    const ConvPlan p = conv_bwd_plan(d, v4 ? 4 : 1);
    a.run = p.run, a.runs = p.runs;
    const sdm_status e = v4 ? launch_conv_k<T, 4>(a, p, true, s) : launch_conv_k<T, 1>(a, p, true, s);
    if (e) return e;
    const long long C = (long long)d->H * d->d;
    conv_sum_kernel<<<(unsigned)ceil_div(C * (d->K + 1), 32), 32 * CSUM_SEG, 0, s>>>(
        a.part, (int)p.gy, C, d->K, dw, dbias);
    return launched();
}

// ---- selective scan ------------------------------------------------------------------------
sdm_status check_scan(const sdm_scan_dims* d) {
    if (!d) return SDM_ERR_ARG;
    if (!known(d->x_dtype)) return SDM_ERR_DTYPE;
    if (d->softplus != 0 && d->softplus != 1) return SDM_ERR_ARG;
    if (d->fresh != 0 && d->fresh != 1) return SDM_ERR_ARG;
    if (d->B < 1 || d->D < 1 || d->G < 1 || d->T < 0 || d->T > kScanMaxT) return SDM_ERR_SHAPE;
    if (d->N < 1 || d->N > 64 || d->D % d->G != 0) return SDM_ERR_SHAPE;
    if ((long long)d->B * d->G > kMaxGrid) return SDM_ERR_SHAPE;
    return SDM_OK;
}

int pad_states(int N) { return N <= 8 ? 8 : (N <= 16 ? 16 : (N <= 32 ? 32 : 64)); }

struct ScanPlan {
    int NN, LN;         // states with padding, lanes of a channel
    int chunk, nchunk;  // tokens of a chunk
    size_t off_S, total;
};

long long scan_warps(const sdm_scan_dims* d, int LN) {
    return (long long)d->B * d->G * ceil_div(d->D / d->G, 32 / LN);
}

// Warps of a walk that live on an SM: eight by their registers, fewer where their tiles are large.
template <typename T, int NPT>
long long walk_warps(int LN) {
    constexpr int TILE = ScanTile<T, NPT>::TILE, STAGES = ScanTile<T, NPT>::STAGES;
    const size_t es = sizeof(T), ch = 32 / LN, NN = NPT * LN;
    const size_t rows = TILE * (3 * ch + 2 * NN) * es + 16;
    const size_t smem = STAGES * rows + (es == 2 && NPT > 4 ? 2 * TILE * NN * 4 : 0) + TILE * (ch * 8 + 128) + 64;
    return std::min<long long>(8, 227 * 1024 / (smem + 1024));
}
long long walk_warps(const sdm_scan_dims* d, int NPT, int LN) {
    if (d->x_dtype == SDM_BF16) return NPT == 4 ? walk_warps<bf16, 4>(LN) : walk_warps<bf16, 8>(LN);
    return NPT == 4 ? walk_warps<float, 4>(LN) : walk_warps<float, 8>(LN);
}

// Eight states a lane where that makes four warps an SM, else four: eight warps of either live on an
// SM.  (16 states, bf16, 1024 tokens of 4096 channels: 2 sequences take 95 us in 512 warps of eight
// a lane and 80 us in 1024 of four, 3 sequences 131 and 139 us, 4 sequences 132 and 169 us; sixteen
// a lane in one warp of 32 channels 216 us.)  While that leaves half of the SMs' sub-partitions
// without a warp, chunks of the tokens, eight states a lane: a second pass over the exponentials
// costs more than it gains above that (at 512 warps 68 us against 61 us).
ScanPlan scan_plan(const sdm_scan_dims* d) {
    ScanPlan p{};
    p.NN = pad_states(d->N);
    const int eight = p.NN / 8, four = std::min(2 * eight, 8);  // lanes of a channel
    p.chunk = std::max(1, d->T);
    p.nchunk = 1;
    p.LN = scan_warps(d, eight) < 4 * kSms ? four : eight;
    if (scan_warps(d, p.LN) <= 2 * kSms) {
        const long long want = std::min(ceil_div(d->T, 64), walk_warps(d, 8, eight) * kSms /
                                                                scan_warps(d, eight));
        if (want > 1) {
            p.LN = eight;
            p.chunk = (int)(ceil_div(ceil_div(d->T, want), SCAN_ROUND) * SCAN_ROUND);
            p.nchunk = (int)ceil_div(d->T, p.chunk);
        }
    }
    const size_t bc = (size_t)d->B * p.nchunk * d->D;
    if (p.nchunk > 1) {
        p.off_S = up256(bc * d->N * 4);
        p.total = up256(p.off_S + bc * 4);
    }
    return p;
}

// Bytes that one asynchronous copy may move of a view's rows of `row` bytes which also start at
// multiples of `step` bytes: 16, 8, 4, or 0 where nothing is aligned enough.
int copy_piece(const sdm_view* v, size_t es, size_t row, size_t step) {
    const uint64_t bits = (uint64_t)(uintptr_t)v->data | (uint64_t)v->sb * es | (uint64_t)v->sh * es |
                          (uint64_t)v->st * es | row | step;
    return bits % 16 == 0 ? 16 : (bits % 8 == 0 ? 8 : (bits % 4 == 0 ? 4 : 0));
}

template <typename T>
Rows<T> rows(const sdm_view* v) {
    return Rows<T>{view<const T>(v), 0};
}

// The pieces of a walk whose warps take `ch` channels: rows of ch elements in shared memory, that
// start at multiples of them within a group; B and C rows of NN.
template <typename T>
void set_pieces(ScanArgs<T>& a, const sdm_view* const (&v)[6], int ch, int NN) {
    Rows<T>* r[6] = {&a.u, &a.delta, &a.z, &a.dy, &a.Bm, &a.Cm};
    for (int i = 0; i < 6; ++i) {
        if (!v[i]) continue;
        const size_t row = (size_t)(i < 4 ? ch : NN) * sizeof(T);
        const size_t step = i < 4 ? (size_t)(a.G > 1 ? a.D / a.G : 0) * sizeof(T) : 0;
        r[i]->piece = copy_piece(v[i], sizeof(T), row, step);
    }
}

template <typename T>
ScanArgs<T> scan_args(const sdm_scan_dims* d, const sdm_view* u, const sdm_view* delta,
                      const float* A, const sdm_view* Bm, const sdm_view* Cm, const float* Dskip,
                      const sdm_view* z, const float* dt_bias, const float* state,
                      const int32_t* lens) {
    ScanArgs<T> a{};
    a.u = rows<T>(u), a.delta = rows<T>(delta), a.z = rows<T>(z);
    a.Bm = rows<T>(Bm), a.Cm = rows<T>(Cm);
    a.A = A, a.Dskip = Dskip, a.dt_bias = dt_bias;
    a.state = const_cast<float*>(state);
    a.lens = lens;
    a.B = d->B, a.T_ = d->T, a.D = d->D, a.N = d->N, a.G = d->G;
    a.softplus = d->softplus, a.fresh = d->fresh;
    return a;
}

template <typename T, int NPT, int LN, int MODE, bool ODD>
sdm_status launch_walk_t(const ScanArgs<T>& a, int runs, cudaStream_t s) {
    constexpr int WCH = 32 / LN;
    constexpr size_t smem = sizeof(ScanShared<T, NPT, LN, MODE>);
    if (!allow_smem(scan_walk_kernel<T, NPT, LN, MODE, ODD>, smem, smem)) return SDM_ERR_CUDA;
    const unsigned gx = (unsigned)(a.G * ceil_div(a.D / a.G, WCH));
    scan_walk_kernel<T, NPT, LN, MODE, ODD><<<dim3(gx, runs, a.B), 32, smem, s>>>(a);
    return launched();
}

template <typename T, int NPT, int LN, int MODE>
sdm_status launch_walk(const ScanArgs<T>& a, int runs, cudaStream_t s) {
    if constexpr (sizeof(T) == 2) {
        const bool odd = !a.u.piece || !a.delta.piece || (a.z.v.p && !a.z.piece) || !a.Bm.piece ||
                         !a.Cm.piece || (MODE == SCAN_CHUNK_REV && !a.dy.piece);
        if (odd) return launch_walk_t<T, NPT, LN, MODE, true>(a, runs, s);
    }
    return launch_walk_t<T, NPT, LN, MODE, false>(a, runs, s);
}

template <typename T, int NPT, int LN>
sdm_status launch_scan_t(ScanArgs<T> a, const sdm_view* const (&v)[6], cudaStream_t s) {
    set_pieces(a, v, 32 / LN, NPT * LN);
    if constexpr (NPT == 8) {  // four states a lane are not split over time
        if (a.nchunk > 1) {
            const sdm_status e = launch_walk<T, NPT, LN, SCAN_CHUNK>(a, a.nchunk - 1, s);
            if (e) return e;
            const long long n = (long long)a.B * a.D * a.N;
            scan_carry_kernel<T><<<(unsigned)ceil_div(n, 256), 256, 0, s>>>(a);
        }
    }
    return launch_walk<T, NPT, LN, SCAN_OUT>(a, a.nchunk, s);
}

// Four sequences a thread where that leaves four blocks an SM (64 sequences of 4096 channels of 16
// states, caches cold: 13.4 us, one a thread 16.0 us), else one.
template <typename T, int LN>
void launch_step_n(const ScanArgs<T>& a, bool vec, cudaStream_t s) {
    const unsigned gx = (unsigned)ceil_div(a.D, 256 / LN);
    if ((long long)gx * ceil_div(a.B, 4) >= 4 * kSms)
        scan_step_kernel<T, LN, 4><<<dim3(gx, (unsigned)ceil_div(a.B, 4)), 256, 0, s>>>(a, vec);
    else
        scan_step_kernel<T, LN, 1><<<dim3(gx, a.B), 256, 0, s>>>(a, vec);
}

template <typename T>
void launch_step(const ScanArgs<T>& a, const sdm_view* const (&v)[6], int NN, cudaStream_t s) {
    const int32_t dt = sizeof(T) == 2 ? SDM_BF16 : SDM_F32;
    const bool vec = a.N % 4 == 0 && vec4_ok(v[4], dt) && vec4_ok(v[5], dt);
    if (NN == 8) launch_step_n<T, 2>(a, vec, s);
    else if (NN == 16) launch_step_n<T, 4>(a, vec, s);
    else if (NN == 32) launch_step_n<T, 8>(a, vec, s);
    else launch_step_n<T, 16>(a, vec, s);
}

template <typename T>
sdm_status run_scan(const sdm_scan_dims* d, ScanArgs<T> a, const sdm_view* const (&v)[6],
                    const sdm_view* y, void* ws, cudaStream_t s) {
    a.y = view<T>(y);
    if (d->T == 1) {
        launch_step<T>(a, v, pad_states(d->N), s);
        return launched();
    }
    const ScanPlan p = scan_plan(d);
    a.chunk = a.run = p.chunk, a.nchunk = p.nchunk;
    a.E = static_cast<float*>(ws);
    a.S = reinterpret_cast<float*>(static_cast<char*>(ws) + p.off_S);
    if (p.LN * 8 == p.NN) {  // eight states a lane
        switch (p.LN) {
            case 1: return launch_scan_t<T, 8, 1>(a, v, s);
            case 2: return launch_scan_t<T, 8, 2>(a, v, s);
            case 4: return launch_scan_t<T, 8, 4>(a, v, s);
            default: return launch_scan_t<T, 8, 8>(a, v, s);
        }
    }
    switch (p.LN) {
        case 2: return launch_scan_t<T, 4, 2>(a, v, s);
        case 4: return launch_scan_t<T, 4, 4>(a, v, s);
        default: return launch_scan_t<T, 4, 8>(a, v, s);
    }
}

struct ScanBwdPlan {
    int NN, nchunk, tiles, blocks;
    size_t off_R, off_S, off_a, off_d, off_bc, total;
};

ScanBwdPlan scan_bwd_plan(const sdm_scan_dims* d) {
    ScanBwdPlan p{};
    p.NN = pad_states(d->N);
    p.nchunk = (int)std::max(1LL, ceil_div(d->T, BWD_CHUNK));
    // A block's channels go by turns of its warps: more turns, fewer shares of dB and dC to write and
    // add; fewer turns, more blocks to even the SMs' work out.  Fourteen blocks an SM, of which
    // three run at a time, did best (bf16, 16 states, the only form compared: 2 sequences of 2048
    // tokens, 2048 channels: 361 us in 2048 blocks, 368 us in 896, 390 us in 384, 407 us in 8192).
    const int ch = BWD_WARPS * 32 / (p.NN / 4), all = (int)ceil_div(d->D / d->G, ch);
    const long long rest = (long long)d->B * p.nchunk * d->G;
    const long long want = std::max(1LL, std::min<long long>(all, 14 * kSms / rest));
    p.tiles = (int)ceil_div(all, want);
    p.blocks = (int)ceil_div(all, p.tiles);
    const size_t bk = (size_t)d->B * p.nchunk, states = bk * d->D * d->N * 4;
    size_t o = 0;
    if (p.nchunk > 1) {
        o = up256(o + states);
        p.off_R = o, o = up256(o + states);
        p.off_S = o, o = up256(o + bk * d->D * 4);
    }
    p.off_a = o, o = up256(o + states);
    p.off_d = o, o = up256(o + bk * d->D * 8);
    p.off_bc = o, o = up256(o + (size_t)p.blocks * d->B * d->T * d->G * 2 * d->N * 4);
    p.total = o;
    return p;
}

template <typename T, int LN>
sdm_status launch_scan_bwd_t(const ScanBwdArgs<T>& A, const ScanBwdPlan& p,
                             const sdm_view* const (&v)[6], cudaStream_t s) {
    ScanArgs<T> a = A.s;
    constexpr int NN = LN * BWD_NPT, CLN = NN / 8;
    if (p.nchunk > 1) {
        set_pieces(a, v, 32 / CLN, NN);
        // a walk over several chunks keeps its tiles coming; runs for 16 warps an SM
        const long long warps = (long long)a.B * a.G * ceil_div(a.D / a.G, 32 / CLN);
        const long long runs = std::min<long long>(p.nchunk, ceil_div(16 * kSms, warps));
        a.run = (int)ceil_div(p.nchunk, runs) * BWD_CHUNK;
        const sdm_status e =
            launch_walk<T, 8, CLN, SCAN_CHUNK_REV>(a, (int)ceil_div(p.nchunk, a.run / BWD_CHUNK), s);
        if (e) return e;
        const unsigned n = (unsigned)ceil_div((long long)a.B * a.D * a.N, 256);
        scan_carry_kernel<T><<<dim3(n, 2), 256, 0, s>>>(a);
    }
    ScanBwdArgs<T> B = A;
    set_pieces(B.s, v, 32 / LN, NN);
    constexpr size_t smem = sizeof(BwdShared<T, LN>);
    if (!allow_smem(scan_bwd_kernel<T, LN>, smem, smem)) return SDM_ERR_CUDA;
    scan_bwd_kernel<T, LN>
        <<<dim3((unsigned)(a.G * p.blocks), p.nchunk, a.B), BWD_WARPS * 32, smem, s>>>(B);
    return launched();
}

template <typename T>
sdm_status run_scan_bwd(const sdm_scan_dims* d, ScanArgs<T> a, const sdm_view* const (&v)[6],
                        const float* dstate_end, const sdm_view* du, const sdm_view* ddelta,
                        float* dA, void* dB, void* dC, float* dDskip, const sdm_view* dz,
                        float* ddt_bias, float* dstate, void* ws, cudaStream_t s) {
    const ScanBwdPlan p = scan_bwd_plan(d);
    char* base = static_cast<char*>(ws);
    a.dy = rows<T>(v[3]);
    a.dstate_end = dstate_end;
    a.chunk = BWD_CHUNK, a.nchunk = p.nchunk;
    a.E = reinterpret_cast<float*>(base);
    a.R = reinterpret_cast<float*>(base + p.off_R);
    a.S = reinterpret_cast<float*>(base + p.off_S);
    ScanBwdArgs<T> A{};
    A.s = a;
    A.du = view<T>(du), A.ddelta = view<T>(ddelta), A.dz = view<T>(dz);
    A.part_a = reinterpret_cast<float*>(base + p.off_a);
    A.part_d = reinterpret_cast<float*>(base + p.off_d);
    A.part_bc = reinterpret_cast<float*>(base + p.off_bc);
    A.dstate = dstate;
    A.tiles = p.tiles, A.blocks = p.blocks;
    sdm_status e;
    if (p.NN == 8) e = launch_scan_bwd_t<T, 2>(A, p, v, s);
    else if (p.NN == 16) e = launch_scan_bwd_t<T, 4>(A, p, v, s);
    else if (p.NN == 32) e = launch_scan_bwd_t<T, 8>(A, p, v, s);
    else e = launch_scan_bwd_t<T, 16>(A, p, v, s);
    if (e) return e;
    const long long btg = (long long)d->B * d->T * d->G;
    if (btg > 0)
        scan_bc_sum_kernel<T><<<(unsigned)ceil_div(btg * 2 * d->N, 256), 256, 0, s>>>(
            A.part_bc, p.blocks, btg, d->N, static_cast<T*>(dB), static_cast<T*>(dC));
    const long long na = (long long)d->D * d->N;
    scan_param_sum_kernel<<<(unsigned)ceil_div(na + 2LL * d->D, 32), 32 * DSUM_SEG, 0, s>>>(
        A.part_a, A.part_d, (long long)d->B * p.nchunk, na, d->D, dA, dDskip, ddt_bias);
    return launched();
}

sdm_status check_scan_in(const sdm_scan_dims* d, const sdm_view* u, const sdm_view* delta,
                         const float* A, const sdm_view* Bm, const sdm_view* Cm,
                         const float* Dskip, const sdm_view* z, const float* dt_bias,
                         const float* state, const int32_t* lens) {
    sdm_status e = check_scan(d);
    if (e) return e;
    if ((e = check_in(u, d->x_dtype, d->T)) || (e = check_in(delta, d->x_dtype, d->T)) ||
        (e = check_in(Bm, d->x_dtype, d->T)) || (e = check_in(Cm, d->x_dtype, d->T)))
        return e;
    if (z && (e = check_in(z, d->x_dtype, d->T))) return e;
    if (!A) return SDM_ERR_ARG;
    if (!aligned(A, 16) || !aligned(Dskip, 16) || !aligned(dt_bias, 16) || !aligned(state, 16) ||
        !aligned(lens, 4))
        return SDM_ERR_ALIGN;
    return SDM_OK;
}

// ---- block norms ---------------------------------------------------------------------------

constexpr int kNormMaxD = 16384;

sdm_status check_norm(const sdm_norm_dims* d) {
    if (!d) return SDM_ERR_ARG;
    if (!known(d->r_dtype) || !known(d->f_dtype) || !known(d->x_dtype)) return SDM_ERR_DTYPE;
    if (d->rows < 0 || d->D < 1 || d->D > kNormMaxD) return SDM_ERR_SHAPE;
    if (!(d->eps >= 0.f)) return SDM_ERR_ARG;
    return SDM_OK;
}

NormArgs norm_args(const sdm_norm_dims* d, const void* r, const void* f, const float* w_post,
                   const void* gate, const float* scale, const float* w_pre) {
    NormArgs a{};
    a.r = r, a.f = f, a.gate = gate;
    a.w_post = w_post, a.scale = scale, a.w_pre = w_pre;
    a.rows = d->rows, a.D = d->D, a.eps = d->eps;
    a.rb = d->r_dtype == SDM_BF16, a.fb = d->f_dtype == SDM_BF16, a.xb = d->x_dtype == SDM_BF16;
    return a;
}

struct NormPlan {
    unsigned threads, blocks;  // a row's block, blocks that take rows in turn
    size_t smem;
};

size_t norm_smem(int D, bool bwd) { return (size_t)ceil_div(D, 4) * 16 * (bwd ? 3 : 1); }  // in passes

bool norm_in_passes(int D, bool bwd) { return D > NORM_COLS || (bwd && D % 4 != 0); }

// Eight values a thread.  The forward pass keeps 1024 threads of blocks an SM (16 blocks at most), the
// gradient 512, so that few shares of its sums are written.  In passes: up to 256 threads, and a row
// of floats in shared memory, the gradient three of them; 512 threads where only one block's fit an SM.
NormPlan norm_plan(const sdm_norm_dims* d, bool bwd) {
    NormPlan p{};
    const bool passes = norm_in_passes(d->D, bwd);
    const int most = passes ? NORM_WIDE : NORM_THREADS;
    p.threads = (unsigned)std::min<long long>(most, ceil_div(ceil_div(d->D, 8), 32) * 32);
    long long per_sm = std::min<long long>(16, (bwd ? 512 : 1024) / p.threads);
    if (passes) {
        p.smem = norm_smem(d->D, bwd);
        per_sm = std::min<long long>(per_sm, 220 * 1024 / (p.smem + 3 * 1024));
        if (bwd && per_sm == 1) p.threads = NORM_THREADS;
    }
    p.blocks = (unsigned)std::min<long long>(d->rows, kSms * per_sm);
    return p;
}

template <bool VEC>
sdm_status launch_norm_wide(const NormArgs& a, bool bwd, const NormPlan& p, cudaStream_t s) {
    auto kernel = bwd ? block_norm_bwd_wide_kernel<VEC> : block_norm_wide_kernel<VEC>;
    if (!allow_smem(kernel, p.smem, norm_smem(kNormMaxD, bwd))) return SDM_ERR_CUDA;
    kernel<<<p.blocks, p.threads, p.smem, s>>>(a);
    return launched();
}

template <int DT>
sdm_status launch_norm_typed(const NormArgs& a, bool bwd, const NormPlan& p, cudaStream_t s) {
    const bool all = a.gate && a.w_post && a.scale && a.w_pre &&
                     (bwd ? a.dr_out && a.dn && a.dr && a.df && a.dgate : a.r_out && a.n);
    auto kernel = bwd ? (all ? block_norm_bwd_kernel<DT, true> : block_norm_bwd_kernel<DT, false>)
                      : (all ? block_norm_kernel<true, DT, true> : block_norm_kernel<true, DT, false>);
    kernel<<<p.blocks, p.threads, 0, s>>>(a);
    return launched();
}

// Rows of whole pieces that fit a block's registers are compiled for their types; the others look the
// types up.
sdm_status launch_norm_any(const NormArgs& a, bool bwd, const NormPlan& p, cudaStream_t s) {
    if (norm_in_passes(a.D, bwd))
        return a.D % 4 ? launch_norm_wide<false>(a, bwd, p, s) : launch_norm_wide<true>(a, bwd, p, s);
    if (a.D % 4) {
        block_norm_kernel<false, -1, false><<<p.blocks, p.threads, 0, s>>>(a);
        return launched();
    }
    switch (a.rb | a.fb << 1 | a.xb << 2) {
        case 0: return launch_norm_typed<0>(a, bwd, p, s);
        case 1: return launch_norm_typed<1>(a, bwd, p, s);
        case 2: return launch_norm_typed<2>(a, bwd, p, s);
        case 3: return launch_norm_typed<3>(a, bwd, p, s);
        case 4: return launch_norm_typed<4>(a, bwd, p, s);
        case 5: return launch_norm_typed<5>(a, bwd, p, s);
        case 6: return launch_norm_typed<6>(a, bwd, p, s);
        default: return launch_norm_typed<7>(a, bwd, p, s);
    }
}

}  // namespace

extern "C" {

sdm_status sdm_short_conv(const sdm_conv_dims* dims, const sdm_view* x, const float* w,
                          const float* bias, void* state, const int32_t* lens, const sdm_view* y,
                          sdm_stream_t stream) {
    sdm_status e = check_conv(dims);
    if (e) return e;
    if ((e = check_in(x, dims->x_dtype, dims->T))) return e;
    if ((e = check_out(y, dims->x_dtype, dims->B, dims->H, dims->T, dims->d))) return e;
    if (!w || same_data(x, y, dims->T)) return SDM_ERR_ARG;
    if (!aligned(w, 16) || !aligned(bias, 16) || !aligned(state, 16) || !aligned(lens, 4))
        return SDM_ERR_ALIGN;
    if (dims->x_dtype == SDM_BF16) return run_conv<bf16>(dims, x, w, bias, state, lens, y, stream);
    return run_conv<float>(dims, x, w, bias, state, lens, y, stream);
}

size_t sdm_short_conv_backward_workspace_bytes(const sdm_conv_dims* dims) {
    if (check_conv(dims) != SDM_OK) return 0;
    const unsigned gy = std::max(conv_bwd_plan(dims, 1).gy,
                                 dims->d % 4 == 0 ? conv_bwd_plan(dims, 4).gy : 0u);
    return up256((size_t)gy * (dims->K + 1) * dims->H * dims->d * 4);
}

sdm_status sdm_short_conv_backward(const sdm_conv_dims* dims, const sdm_view* x, const float* w,
                                   const float* bias, const void* state, const int32_t* lens,
                                   const sdm_view* dy, const float* dstate_end,
                                   const sdm_view* dx, float* dw, float* dbias, float* dstate,
                                   void* ws, size_t ws_bytes, sdm_stream_t stream) {
    sdm_status e = check_conv(dims);
    if (e) return e;
    if ((e = check_in(x, dims->x_dtype, dims->T)) || (e = check_in(dy, dims->x_dtype, dims->T))) return e;
    if ((e = check_out(dx, dims->x_dtype, dims->B, dims->H, dims->T, dims->d))) return e;
    if (!w || !dw || same_data(x, dx, dims->T) || same_data(dy, dx, dims->T)) return SDM_ERR_ARG;
    if (!aligned(w, 16) || !aligned(bias, 16) || !aligned(state, 16) || !aligned(lens, 4) ||
        !aligned(dstate_end, 16) || !aligned(dw, 16) || !aligned(dbias, 16) || !aligned(dstate, 16))
        return SDM_ERR_ALIGN;
    if (!ws || ws_bytes < sdm_short_conv_backward_workspace_bytes(dims)) return SDM_ERR_WORKSPACE;
    if (!aligned(ws, 16)) return SDM_ERR_ALIGN;
    if (dims->x_dtype == SDM_BF16)
        return run_conv_bwd<bf16>(dims, x, w, bias, state, lens, dy, dstate_end, dx, dw, dbias,
                                  dstate, ws, stream);
    return run_conv_bwd<float>(dims, x, w, bias, state, lens, dy, dstate_end, dx, dw, dbias, dstate,
                               ws, stream);
}

size_t sdm_selective_scan_workspace_bytes(const sdm_scan_dims* dims) {
    if (check_scan(dims) != SDM_OK || dims->T <= 1) return 0;
    return scan_plan(dims).total;
}

sdm_status sdm_selective_scan(const sdm_scan_dims* dims, const sdm_view* u, const sdm_view* delta,
                              const float* A, const sdm_view* Bm, const sdm_view* Cm,
                              const float* Dskip, const sdm_view* z, const float* dt_bias,
                              float* state, const int32_t* lens, const sdm_view* y, void* ws,
                              size_t ws_bytes, sdm_stream_t stream) {
    sdm_status e = check_scan_in(dims, u, delta, A, Bm, Cm, Dskip, z, dt_bias, state, lens);
    if (e) return e;
    if ((e = check_out(y, dims->x_dtype, dims->B, 1, dims->T, dims->D))) return e;
    for (const sdm_view* in : {u, delta, z, Bm, Cm})
        if (same_data(in, y, dims->T)) return SDM_ERR_ARG;
    const size_t need = sdm_selective_scan_workspace_bytes(dims);
    if (need && (!ws || ws_bytes < need)) return SDM_ERR_WORKSPACE;
    if (!aligned(ws, 16)) return SDM_ERR_ALIGN;
    const sdm_view* const v[6] = {u, delta, z, nullptr, Bm, Cm};
    if (dims->x_dtype == SDM_BF16)
        return run_scan<bf16>(dims, scan_args<bf16>(dims, u, delta, A, Bm, Cm, Dskip, z, dt_bias,
                                                    state, lens), v, y, ws, stream);
    return run_scan<float>(dims, scan_args<float>(dims, u, delta, A, Bm, Cm, Dskip, z, dt_bias,
                                                  state, lens), v, y, ws, stream);
}

size_t sdm_selective_scan_backward_workspace_bytes(const sdm_scan_dims* dims) {
    if (check_scan(dims) != SDM_OK) return 0;
    return scan_bwd_plan(dims).total;
}

sdm_status sdm_selective_scan_backward(
    const sdm_scan_dims* dims, const sdm_view* u, const sdm_view* delta, const float* A,
    const sdm_view* Bm, const sdm_view* Cm, const float* Dskip, const sdm_view* z,
    const float* dt_bias, const float* state, const int32_t* lens, const sdm_view* dy,
    const float* dstate_end, const sdm_view* du, const sdm_view* ddelta, float* dA, void* dB,
    void* dC, float* dDskip, const sdm_view* dz, float* ddt_bias, float* dstate, void* ws,
    size_t ws_bytes, sdm_stream_t stream) {
    sdm_status e = check_scan_in(dims, u, delta, A, Bm, Cm, Dskip, z, dt_bias, state, lens);
    if (e) return e;
    if ((e = check_in(dy, dims->x_dtype, dims->T))) return e;
    if ((z != nullptr) != (dz != nullptr) || !dA) return SDM_ERR_ARG;
    if (dims->T > 0 && (!dB || !dC)) return SDM_ERR_ARG;
    const sdm_view* outs[3] = {du, ddelta, dz};
    for (int i = 0; i < 3; ++i) {
        if (i == 2 && !dz) break;
        if ((e = check_out(outs[i], dims->x_dtype, dims->B, 1, dims->T, dims->D))) return e;
        for (const sdm_view* in : {u, delta, z, Bm, Cm, dy})
            if (same_data(in, outs[i], dims->T)) return SDM_ERR_ARG;
        for (int j = 0; j < i; ++j)
            if (same_data(outs[j], outs[i], dims->T)) return SDM_ERR_ARG;
    }
    if (!aligned(dstate_end, 16) || !aligned(dA, 16) || !aligned(dB, 16) || !aligned(dC, 16) ||
        !aligned(dDskip, 16) || !aligned(ddt_bias, 16) || !aligned(dstate, 16))
        return SDM_ERR_ALIGN;
    if (!ws || ws_bytes < sdm_selective_scan_backward_workspace_bytes(dims))
        return SDM_ERR_WORKSPACE;
    if (!aligned(ws, 16)) return SDM_ERR_ALIGN;
    const sdm_view* const v[6] = {u, delta, z, dy, Bm, Cm};
    if (dims->x_dtype == SDM_BF16)
        return run_scan_bwd<bf16>(dims, scan_args<bf16>(dims, u, delta, A, Bm, Cm, Dskip, z,
                                                        dt_bias, state, lens),
                                  v, dstate_end, du, ddelta, dA, dB, dC, dDskip, dz, ddt_bias,
                                  dstate, ws, stream);
    return run_scan_bwd<float>(dims, scan_args<float>(dims, u, delta, A, Bm, Cm, Dskip, z, dt_bias,
                                                      state, lens),
                               v, dstate_end, du, ddelta, dA, dB, dC, dDskip, dz, ddt_bias, dstate,
                               ws, stream);
}

sdm_status sdm_block_norm(const sdm_norm_dims* dims, const void* r, const void* f,
                          const float* w_post, const void* gate, const float* scale,
                          const float* w_pre, void* r_out, void* n, sdm_stream_t stream) {
    sdm_status e = check_norm(dims);
    if (e) return e;
    if (dims->rows > 0 && (!r || !f || (!r_out && !n))) return SDM_ERR_ARG;
    if (!aligned(r, 16) || !aligned(f, 16) || !aligned(w_post, 16) || !aligned(gate, 16) ||
        !aligned(scale, 16) || !aligned(w_pre, 16) || !aligned(r_out, 16) || !aligned(n, 16))
        return SDM_ERR_ALIGN;
    if (dims->rows == 0) return SDM_OK;
    NormArgs a = norm_args(dims, r, f, w_post, gate, scale, w_pre);
    a.r_out = r_out, a.n = n;
    return launch_norm_any(a, false, norm_plan(dims, false), stream);
}

size_t sdm_block_norm_backward_workspace_bytes(const sdm_norm_dims* dims) {
    if (check_norm(dims) != SDM_OK) return 0;
    return up256(std::max<size_t>(1, norm_plan(dims, true).blocks) * 3 * dims->D * 4);
}

sdm_status sdm_block_norm_backward(const sdm_norm_dims* dims, const void* r, const void* f,
                                   const float* w_post, const void* gate, const float* scale,
                                   const float* w_pre, const void* dr_out, const void* dn,
                                   void* dr, void* df, void* dgate, float* dscale, float* dw_post,
                                   float* dw_pre, void* ws, size_t ws_bytes, sdm_stream_t stream) {
    sdm_status e = check_norm(dims);
    if (e) return e;
    if (dims->rows > 0 && (!r || !f)) return SDM_ERR_ARG;
    if ((dgate && !gate) || (dw_post && !w_post)) return SDM_ERR_ARG;
    const void* ptrs[] = {r, f, w_post, gate, scale, w_pre, dr_out, dn, dr, df, dgate, dscale,
                          dw_post, dw_pre};
    for (const void* p : ptrs)
        if (!aligned(p, 16)) return SDM_ERR_ALIGN;
    if (!ws || ws_bytes < sdm_block_norm_backward_workspace_bytes(dims)) return SDM_ERR_WORKSPACE;
    if (!aligned(ws, 16)) return SDM_ERR_ALIGN;
    NormArgs a = norm_args(dims, r, f, w_post, gate, scale, w_pre);
    a.dr_out = dr_out, a.dn = dn;
    a.dr = dr, a.df = df, a.dgate = dgate;
    a.part = static_cast<float*>(ws);
    const NormPlan p = norm_plan(dims, true);
    if (dims->rows > 0 && (e = launch_norm_any(a, true, p, stream))) return e;
    norm_sum_kernel<<<(unsigned)ceil_div(3LL * dims->D, 32), 32 * SUM_SEG, 0, stream>>>(
        a.part, (int)p.blocks, dims->D, dscale, dw_post, dw_pre);
    return launched();
}

}  // extern "C"
