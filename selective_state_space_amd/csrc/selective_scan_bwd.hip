// Gradients of the per-channel selective scan.  With a_t = exp(d_t A), the
// states h_t of the forward, dyp = dy silu(z) (dy without a gate) and g the
// adjoint of the state, g_T = dfinal and from the last token to the first
//
//     g      = (carried) + dyp_t C_t
//     dC_t   = sum_c dyp h_t        dB_t = sum_c g d x
//     gB     = sum_n g B_t          q = a_t g h_{t-1}   (per c, n)
//     dx_t   = d gB + D dyp         dd_t = x gB + sum_n q A
//     dA    += d q                  (carried) = a_t g
//
// and ddt = dd sigmoid(dt + bias) under softplus, dbias = sum ddt, dD = sum
// dyp x, dz = dy (sum_n h C + D x) silu'(z).
//
// The states are not kept by the forward: a first pass scans again and writes
// the state before every 16th token; the reverse pass then recomputes a
// tile's 16 states into registers (4 per lane and token) and walks them
// backwards, so every h_{t-1} is exact, never divided out.  Sums over n are
// made on the S lanes of a channel.  Sums over channels (dB, dC: 2 KS values
// per lane and token) pass through LDS, where each lane adds up a share of the
// wavefront's; the wavefronts are joined there too, and channel blocks by a
// last kernel.  Every sum has a fixed order.  (4 x 2048 tokens of 2048 channels,
// N 16: the reverse pass takes 277 us, with the values swapped between lanes
// 284, with matrix instructions that add them up 459.)
//
// With several segments per sequence (few rows, see plan() below)
// the first pass starts each segment from zero and the reverse pass adds the
// decayed entry state to its checkpoints; the adjoints entering the segments
// come from a reverse pass without outputs and a chain over segments.

#include <type_traits>

#include "selective_scan.h"

namespace ssd {

namespace {

constexpr int TB = 16;   // tokens of a backward tile, and between checkpoints

template <int N, int KS>
struct BTile {
    typedef SelSplit<N, KS> Sp;
    static constexpr int VPR = Sp::CB / 4;                       // 4-channel vectors of a row
    static constexpr int ITEMS = TB * VPR;                       // (token, vector) pairs
    static constexpr int NI = (ITEMS + 255) / 256;               // of them per thread
    static constexpr int ROWS = ITEMS < 256 ? ITEMS / VPR : 256 / VPR;
    static constexpr int BC = TB * N / 4;                        // 4-element vectors of B (or C)
};

// The adjoint leaving a segment at its first token, started from zero after
// its last one (segments 1 .. nseg-1; block blk of theirs).
template <int N, int KS, typename Tio, bool GATE, bool RAG>
__device__ __forceinline__ void sel_adj(
    const Tio *__restrict__ dt, const float *__restrict__ A, const Tio *__restrict__ C,
    const Tio *__restrict__ z, const float *__restrict__ dt_bias, const float *__restrict__ dy,
    float *__restrict__ adj, const SelGeom &g, uint32_t blk) {
    typedef SelSplit<N, KS> Sp;
    typedef BTile<N, KS> Bt;
    constexpr int S = Sp::S, CPW = Sp::CPW, CB = Sp::CB;
    constexpr int VPR = Bt::VPR, NI = Bt::NI, ITEMS = Bt::ITEMS, BC = Bt::BC;
    __shared__ __align__(16) float sdy[2][TB][CB];   // d, dyp
    __shared__ __align__(16) float sc[TB][N];
    const int tid = threadIdx.x;
    const uint32_t cb = blk % (uint32_t)g.ncb;
    const uint32_t rest = blk / (uint32_t)g.ncb;
    const int64_t b = rest / (uint32_t)(g.nseg - 1);
    const int32_t seg = 1 + rest % (uint32_t)(g.nseg - 1);
    const int64_t t0 = seg * g.seg_len, t1 = min(g.T, t0 + g.seg_len);
    const int sv = tid % VPR;
    const int32_t ch0 = cb * CB + 4 * sv;
    const int chn = min(4, g.Dm - ch0);
    float bias[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) bias[i] = dt_bias && i < chn ? dt_bias[ch0 + i] : 0.f;
    const int lane = tid & 63, wave = tid >> 6;
    const int s = lane % S, cl = wave * CPW + lane / S;
    const int32_t c = cb * CB + cl;
    float a2[KS] = {}, car[KS] = {};
    if (c < g.Dm) {
        load_ks(A + (int64_t)c * N + KS * s, a2);
#pragma unroll
        for (int i = 0; i < KS; ++i) a2[i] = rate2(a2[i]);
    }
    const int64_t ntile = (t1 - t0 + TB - 1) / TB;
    for (int64_t k = ntile - 1; k >= 0; --k) {
        const int64_t tb = t0 + k * TB;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int e = tid + 256 * i, r = e / VPR;
            const int64_t t = tb + r;
            if (e < ITEMS) {
                float d[4] = {}, p[4] = {};
                if (t < t1 && chn > 0) {
                    const int64_t o = (b * g.T + t) * g.Dm + ch0;
                    const float4 dv = widen4(load_raw<RAG>(dt + o, chn));
                    const float4 yv = widen4(load_raw<RAG>(dy + o, chn));
                    float4 zv = make_float4(0.f, 0.f, 0.f, 0.f);
                    if constexpr (GATE) zv = widen4(load_raw<RAG>(z + o, chn));
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float rw = (&dv.x)[j] + bias[j];
                        d[j] = g.softplus ? softplus_f(rw) : rw;
                        p[j] = (&yv.x)[j];
                        if constexpr (GATE) p[j] *= fast_silu((&zv.x)[j]);
                    }
                }
                *reinterpret_cast<float4 *>(&sdy[0][r][4 * sv]) =
                    make_float4(d[0], d[1], d[2], d[3]);
                *reinterpret_cast<float4 *>(&sdy[1][r][4 * sv]) =
                    make_float4(p[0], p[1], p[2], p[3]);
            }
        }
        for (int e = tid; e < BC; e += 256) {
            const int64_t t = tb + e / (N / 4);
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (t < t1) v = widen4(load_raw<false>(C + (b * g.T + t) * N + 4 * (e % (N / 4)), 4));
            reinterpret_cast<float4 *>(&sc[0][0])[e] = v;
        }
        lds_barrier();
#pragma unroll
        for (int t = TB - 1; t >= 0; --t) {
            const float2 w = make_float2(sdy[0][t][cl], sdy[1][t][cl]);
            float cv[KS];
            load_ks(&sc[t][KS * s], cv);
#pragma unroll
            for (int i = 0; i < KS; ++i)
                car[i] = fast_exp2(w.x * a2[i]) * fmaf(w.y, cv[i], car[i]);
        }
        lds_barrier();
    }
    if (c < g.Dm)
        store_ks(adj + (((b * g.nseg) + seg) * g.Dm + c) * N + KS * s, car);
}

// Both passes over the segments in one launch, as neither needs the other: the
// first `scans` blocks checkpoint the states, the rest form the adjoints (all
// gradients of 2 x 333 tokens, 777 channels, N 32: 47 us, in two launches 53;
// 4 x 2048 x 2048, N 16: 365 us, 372).
template <int N, int KS, typename Tio, bool GATE, bool RAG>
__global__ __launch_bounds__(256) void sel_ends_kernel(
    const Tio *__restrict__ x, const Tio *__restrict__ dt, const float *__restrict__ A,
    const Tio *__restrict__ B, const Tio *__restrict__ C, const Tio *__restrict__ z,
    const float *__restrict__ dt_bias, const float *__restrict__ dy, float *__restrict__ hseg,
    float *__restrict__ dsum, float *__restrict__ ckpt, float *__restrict__ cumd,
    float *__restrict__ adj, uint32_t scans, SelGeom g) {
    if (blockIdx.x < scans)
        sel_scan<N, KS, Tio, float, false, RAG, SCAN_CKPT>(
            x, dt, A, B, nullptr, nullptr, nullptr, dt_bias, nullptr, nullptr, nullptr, hseg, dsum,
            ckpt, cumd, g, blockIdx.x);
    else
        sel_adj<N, KS, Tio, GATE, RAG>(dt, A, C, z, dt_bias, dy, adj, g, blockIdx.x - scans);
}

// Both chains over the segments: the states entering each (hseg, in place of
// the end states) and the adjoints entering each from the right (adj).
__global__ __launch_bounds__(256) void sel_chain_bwd_kernel(
    float *__restrict__ hseg, float *__restrict__ adj, const float *__restrict__ dsum,
    const float *__restrict__ A, const float *__restrict__ init,
    const float *__restrict__ dfinal, int64_t total, int32_t Dm, int32_t N, int32_t nseg) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;   // (b, c, n)
    if (i >= total) return;
    const int64_t per = (int64_t)Dm * N;
    const int64_t b = i / per, cn = i % per;
    const float a2 = rate2(A[cn]);
    const float *q = dsum + b * nseg * Dm + cn / N;
    float *p = hseg + b * nseg * per + cn;
    float h = init ? init[i] : 0.f;
    // 8 segments' values in flight at a time
    for (int32_t k0 = 0; k0 < nseg; k0 += 8) {
        float e[8], d[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int32_t k = k0 + j;
            e[j] = k < nseg ? p[k * per] : 0.f;
            d[j] = k < nseg ? q[(int64_t)k * Dm] : 0.f;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (k0 + j < nseg) p[(k0 + j) * per] = h;
            h = fmaf(fast_exp2(d[j] * a2), h, e[j]);
        }
    }
    p = adj + b * nseg * per + cn;
    float r = dfinal ? dfinal[i] : 0.f;
    for (int32_t k0 = nseg - 1; k0 >= 0; k0 -= 8) {
        float e[8], d[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int32_t k = k0 - j;
            e[j] = k > 0 ? p[k * per] : 0.f;
            d[j] = k >= 0 ? q[(int64_t)k * Dm] : 0.f;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (k0 - j >= 0) p[(k0 - j) * per] = r;
            r = fmaf(fast_exp2(d[j] * a2), r, e[j]);
        }
    }
}

template <int N, int KS, typename Tio, bool GATE, bool RAG>
__global__ __launch_bounds__(256, 2) void sel_bwd_kernel(
    const Tio *__restrict__ x, const Tio *__restrict__ dt, const float *__restrict__ A,
    const Tio *__restrict__ B, const Tio *__restrict__ C, const float *__restrict__ D,
    const Tio *__restrict__ z, const float *__restrict__ dt_bias, const float *__restrict__ dy,
    const float *__restrict__ right, const float *__restrict__ ckpt,
    const float *__restrict__ cumd, const float *__restrict__ hseg, float *__restrict__ dx,
    float *__restrict__ ddt, float *__restrict__ dz, float *__restrict__ dinit,
    float *__restrict__ pbc, float *__restrict__ pA, float *__restrict__ pD,
    float *__restrict__ pbias, SelGeom g) {
    typedef SelSplit<N, KS> Sp;
    typedef BTile<N, KS> Bt;
    constexpr int S = Sp::S, CPW = Sp::CPW, CB = Sp::CB;
    constexpr int VPR = Bt::VPR, NI = Bt::NI, ITEMS = Bt::ITEMS;
    constexpr int BC = Bt::BC, NBC = (BC + 255) / 256, ROWS = Bt::ROWS;
    __shared__ __align__(16) float sdu[2][TB][CB];        // d, d x
    __shared__ __align__(16) float sdy[TB][CB];           // dyp
    __shared__ __align__(16) float sbc[2][TB][N];
    __shared__ __align__(16) float sgd[2][TB][Sp::ROW];   // gB, sum q a2
    __shared__ __align__(16) float sy[GATE ? TB : 1][GATE ? Sp::ROW : 4];
    __shared__ __align__(16) float sdbc[4][TB][2 * N];
    __shared__ __align__(16) float ssp[TB][CB];                        // softplus'
    __shared__ __align__(16) float ssz[GATE ? TB : 1][GATE ? CB : 4];   // sigmoid(z)
    // the products summed over a wavefront's channels: RT tokens of [channel][dB, dC]
    constexpr int RT = N <= 16 ? 2 : 1;
    constexpr int RV = N <= 32 ? 1 : 2;                       // values per summing lane
    constexpr int RC = N == 8 ? CPW / 2 : CPW;                // channels it sums
    constexpr int RP = CPW * 2 * N + 32;                      // (+ 32: tokens on other banks)
    __shared__ __align__(16) float sred[4][RT][RP];
    const int tid = threadIdx.x;
    const uint32_t cb = blockIdx.x % (uint32_t)g.ncb;
    const uint32_t rest = blockIdx.x / (uint32_t)g.ncb;   // (b, segment)
    const int64_t b = rest / (uint32_t)g.nseg;
    const int32_t seg = rest % (uint32_t)g.nseg;
    const int64_t t0 = seg * g.seg_len, t1 = min(g.T, t0 + g.seg_len);
    const int64_t ntile = (t1 - t0 + TB - 1) / TB;

    // (staging may need half of the threads: odd and even workgroups take
    // different halves, so that every SIMD has its share)
    const int st = ITEMS < 256 ? tid ^ (int)((blockIdx.x & 1) << 7) : tid;
    const int sv = st % VPR;
    const int32_t ch0 = cb * CB + 4 * sv;
    const int chn = min(4, g.Dm - ch0);
    float bias[4], Dv[4], accD[4] = {}, accb[4] = {};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        bias[i] = dt_bias && i < chn ? dt_bias[ch0 + i] : 0.f;
        Dv[i] = i < chn ? D[ch0 + i] : 0.f;
    }
    const int lane = tid & 63, wave = tid >> 6;
    const int s = lane % S, cl = wave * CPW + lane / S;
    const int32_t c = cb * CB + cl;
    float a2[KS] = {}, car[KS] = {}, dA[KS] = {}, hs[KS] = {};
    if (c < g.Dm) {
        load_ks(A + (int64_t)c * N + KS * s, a2);
#pragma unroll
        for (int i = 0; i < KS; ++i) a2[i] = rate2(a2[i]);
        const int64_t u = ((int64_t)rest * g.Dm + c) * N + KS * s;
        if (right) load_ks(right + u, car);   // [Bt][nseg][Dm][N]: with one segment dfinal
        if (g.nseg > 1) load_ks(hseg + u, hs);
    }
    struct Tok {
        Raw4<Tio> x, dt, z;
        Raw4<float> dy;
    };
    // (rows of an odd width are not aligned to a lane's vector: RAG takes them
    // through plain loads and bounds its last channels by hand)
    const int64_t row0 = b * g.T;
    const uint32_t off = chn > 0 ? (uint32_t)(st / VPR) * g.Dm + ch0 : kNoOffset / 4;
    const uint32_t item = (256 / VPR) * (uint32_t)g.Dm;   // elements between a thread's items
    auto left = [&](int64_t tb) { return tb >= t0 ? min(t1 - tb, (int64_t)TB) : (int64_t)0; };
    auto load_one = [&](auto *p, int64_t tb, int i) {
        typedef typename std::remove_cv<typename std::remove_pointer<decltype(p)>::type>::type T;
        if constexpr (RAG) {
            Raw4<T> r;
            zero_raw(r);
            const int64_t row = (st + 256 * i) / VPR;
            if (st + 256 * i < ITEMS && row < left(tb) && chn > 0)
                r = load_raw<true>(p + (row0 + tb + row) * g.Dm + ch0, chn);
            return r;
        } else {
            return load_buf(tile_rsrc(p, row0 + tb, left(tb), g.Dm),
                            (off + i * item) * (uint32_t)sizeof(T), T());
        }
    };
    auto store_one = [&](float *p, int64_t tb, int i, float4 v) {
        if constexpr (RAG) {
            const int64_t row = (st + 256 * i) / VPR;
            if (row < left(tb) && chn > 0)
                store4<true>(p + (row0 + tb + row) * g.Dm + ch0, v, chn);
        } else {
            store_buf(tile_rsrc(p, row0 + tb, left(tb), g.Dm), (off + i * item) * 4u, v, 0.f);
        }
    };
    auto load_tok = [&](int64_t tb, int i) {
        Tok r;
        r.x = load_one(x, tb, i);
        r.dt = load_one(dt, tb, i);
        r.dy = load_one(dy, tb, i);
        if constexpr (GATE) r.z = load_one(z, tb, i);
        return r;
    };
    // vectors e of the tile's B (from the first thread up) and C (from the last down)
    auto load_bc = [&](const Tio *p, int64_t tb, int e) {
        return load_buf(tile_rsrc(p, row0 + tb, left(tb), N),
                        e < BC ? (uint32_t)e * 4 * sizeof(Tio) : kNoOffset, Tio());
    };
    const uint32_t coff = c < g.Dm ? (uint32_t)c * N + KS * s : kNoOffset / 4;
    auto load_h0 = [&](int64_t tb, float (&h)[KS]) {
        const int64_t u = uniform64((b * ((g.T + 15) >> 4) + (tb >> 4)) * g.Dm);
        const uint32_t bytes =
            __builtin_amdgcn_readfirstlane(tb >= t0 ? (uint32_t)g.Dm * 4u : 0u);
        load_buf_ks(make_rsrc(ckpt + u * N, bytes * N), coff * 4u, h);
        if (g.nseg > 1) {
            const float cd = __uint_as_float(
                __builtin_amdgcn_raw_buffer_load_b32(make_rsrc(cumd + u, bytes), c * 4u, 0, 0));
#pragma unroll
            for (int i = 0; i < KS; ++i) h[i] = fmaf(fast_exp2(cd * a2[i]), hs[i], h[i]);
        }
    };

    int64_t tb = t0 + (ntile - 1) * TB;
    Tok tok[NI];
    Raw4<Tio> rb[NBC], rc[NBC];
#pragma unroll
    for (int i = 0; i < NI; ++i) tok[i] = load_tok(tb, i);
#pragma unroll
    for (int k = 0; k < NBC; ++k) {
        rb[k] = load_bc(B, tb, tid + 256 * k);
        rc[k] = load_bc(C, tb, 255 - tid + 256 * k);
    }
    float h0[KS];
    load_h0(tb, h0);

    for (; tb >= t0; tb -= TB) {
        // stage
        float dkeep[NI][4];
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int e = st + 256 * i, r = e / VPR;
            if (e < ITEMS) {
                const float4 xv = widen4(tok[i].x), dv = widen4(tok[i].dt), yv = tok[i].dy.v;
                const float4 zv = widen4(tok[i].z);
                float u[4], p[4], sp[4], sz[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float rw = (&dv.x)[j] + bias[j];
                    sp[j] = 1.f;
                    float d = g.softplus ? softplus_f(rw, sp[j]) : rw;
                    if (tb + TB > t1 && tb + r >= t1) d = 0.f;
                    dkeep[i][j] = d;
                    u[j] = d * (&xv.x)[j];
                    p[j] = (&yv.x)[j];
                    if constexpr (GATE) {
                        sz[j] = sigmoid_f((&zv.x)[j]);
                        p[j] *= (&zv.x)[j] * sz[j];
                    }
                }
                *reinterpret_cast<float4 *>(&ssp[r][4 * sv]) =
                    make_float4(sp[0], sp[1], sp[2], sp[3]);
                if constexpr (GATE)
                    *reinterpret_cast<float4 *>(&ssz[r][4 * sv]) =
                        make_float4(sz[0], sz[1], sz[2], sz[3]);
                *reinterpret_cast<float4 *>(&sdu[0][r][4 * sv]) =
                    make_float4(dkeep[i][0], dkeep[i][1], dkeep[i][2], dkeep[i][3]);
                *reinterpret_cast<float4 *>(&sdu[1][r][4 * sv]) =
                    make_float4(u[0], u[1], u[2], u[3]);
                *reinterpret_cast<float4 *>(&sdy[r][4 * sv]) = make_float4(p[0], p[1], p[2], p[3]);
            }
        }
#pragma unroll
        for (int k = 0; k < NBC; ++k) {
            const int eb = tid + 256 * k, ec = 255 - tid + 256 * k;
            if (eb < BC) reinterpret_cast<float4 *>(&sbc[0][0][0])[eb] = widen4(rb[k]);
            if (ec < BC) reinterpret_cast<float4 *>(&sbc[1][0][0])[ec] = widen4(rc[k]);
        }
        // the previous tile's loads, in flight during this one's arithmetic
        const int64_t tp = tb - TB;
        Tok ntok[NI];
#pragma unroll
        for (int i = 0; i < NI; ++i) ntok[i] = load_tok(tp, i);
#pragma unroll
        for (int k = 0; k < NBC; ++k) {
            rb[k] = load_bc(B, tp, tid + 256 * k);
            rc[k] = load_bc(C, tp, 255 - tid + 256 * k);
        }
        lds_barrier();

        // the tile's states; a token's operands are loaded two tokens ahead and
        // its exponentials taken one ahead, and no earlier (registers)
        struct Op {
            float2 w;
            float p, bv[KS], cv[KS];
        };
        float H[TB][KS];
        {
            auto load_op = [&](int t, Op &o) {
                o.w = make_float2(sdu[0][t][cl], sdu[1][t][cl]);
                load_ks(&sbc[0][t][KS * s], o.bv);
                if constexpr (GATE) load_ks(&sbc[1][t][KS * s], o.cv);
            };
            Op op[2];
            float a[KS], an[KS];
            load_op(0, op[0]);
            load_op(1, op[1]);
#pragma unroll
            for (int i = 0; i < KS; ++i) a[i] = fast_exp2(op[0].w.x * a2[i]);
#pragma unroll
            for (int tq = 0; tq < TB; tq += S) {
                float y[S];
#pragma unroll
                for (int k = 0; k < S; ++k) {
                    const int t = tq + k;
                    const Op cur = op[t & 1];
                    if (t + 2 < TB) load_op(t + 2, op[t & 1]);
                    if (t + 1 < TB) {
#pragma unroll
                        for (int i = 0; i < KS; ++i)
                            an[i] = fast_exp2(op[(t + 1) & 1].w.x * a2[i]);
                    }
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int i = 0; i < KS; ++i)
                        H[t][i] = fmaf(a[i], t ? H[t ? t - 1 : 0][i] : h0[i], cur.w.y * cur.bv[i]);
                    if constexpr (GATE) {
                        y[k] = H[t][0] * cur.cv[0];
#pragma unroll
                        for (int i = 1; i < KS; ++i) y[k] = fmaf(H[t][i], cur.cv[i], y[k]);
                    }
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int i = 0; i < KS; ++i) a[i] = an[i];
                }
                if constexpr (GATE) sy[tq + s][cl] = lane_sums<S>(y, s);
            }
        }
        // and backwards (the operands are read from LDS again: kept in
        // registers from the first walk they would halve the wavefronts)
        float dAt[KS] = {};
        int cr = cl, sr = KS * s;
        asm volatile("" : "+v"(cr), "+v"(sr));
        // Sums over the wavefront's channels (dB, dC) through LDS: every lane
        // writes its 2 KS products, then adds up one value (RV of them) of one
        // token over the channels.  The values are read after a batch of RT
        // tokens and added during the next.
        const int wl = lane / S;   // channel in the wavefront
        // (every other channel, or pair for N 8, has dB and dC exchanged in its
        // row: the lanes that write together then meet different banks)
        const int wx = N == 16 ? (wl & 1) * N : (N == 8 ? (wl >> 1 & 1) * N : 0);
        const int rj = RV * lane % (2 * N), rt = RV * lane / (2 * N) % RT;   // value, token
        const int rc = N == 8 ? lane >> 5 : 0;                          // half of the channels
        float rr[RC][RV];
        auto red_read = [&] {
#pragma unroll
            for (int i = 0; i < RC; ++i) {
                const int x = N == 16 ? (i & 1) * N : (N == 8 ? (i >> 1 & 1) * N : 0);
                const float *p = &sred[wave][rt][(rc * RC + i) * 2 * N + (rj ^ x)];
                if constexpr (RV == 1)
                    rr[i][0] = *p;
                else
                    load_ks(p, rr[i]);
            }
        };
        auto red_add = [&](int t) {   // of the batch whose first token is t
            float o[RV];
#pragma unroll
            for (int q = 0; q < RV; ++q) {
#pragma unroll
                for (int w = 1; w < RC; w *= 2)
#pragma unroll
                    for (int i = 0; i + w < RC; i += 2 * w) rr[i][q] += rr[i + w][q];
                o[q] = rr[0][q];
                if constexpr (N == 8) o[q] += __shfl_xor(o[q], 32, 64);
            }
            if constexpr (RV == 1)
                sdbc[wave][t + rt][rj] = o[0];
            else
                store_ks(&sdbc[wave][t + rt][rj], o);
        };
        {
            auto load_op = [&](int t, Op &o) {
                o.w = make_float2(sdu[0][t][cr], sdu[1][t][cr]);
                o.p = sdy[t][cr];
                load_ks(&sbc[0][t][sr], o.bv);
                load_ks(&sbc[1][t][sr], o.cv);
            };
            Op op[2];
            float a[KS], an[KS];
            load_op(TB - 1, op[1]);
            load_op(TB - 2, op[0]);
#pragma unroll
            for (int i = 0; i < KS; ++i) a[i] = fast_exp2(op[1].w.x * a2[i]);
#pragma unroll
            for (int tq = TB - S; tq >= 0; tq -= S) {
                float pg[S], pq[S];
#pragma unroll
                for (int k = S - 1; k >= 0; --k) {
                    const int t = tq + k;
                    const Op cur = op[t & 1];
                    if (t > 1) load_op(t - 2, op[t & 1]);
                    if (t > 0) {
#pragma unroll
                        for (int i = 0; i < KS; ++i)
                            an[i] = fast_exp2(op[(t - 1) & 1].w.x * a2[i]);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                    float vb[KS], vc[KS], g1, q1;
#pragma unroll
                    for (int i = 0; i < KS; ++i) {
                        const float gi = fmaf(cur.p, cur.cv[i], car[i]);
                        vb[i] = gi * cur.w.y;
                        vc[i] = cur.p * H[t][i];
                        g1 = i ? fmaf(gi, cur.bv[i], g1) : gi * cur.bv[i];
                        car[i] = gi * a[i];
                        const float q = car[i] * (t ? H[t ? t - 1 : 0][i] : h0[i]);
                        q1 = i ? fmaf(q, a2[i], q1) : q * a2[i];
                        dAt[i] = fmaf(q, cur.w.x, dAt[i]);
                    }
                    pg[k] = g1;
                    pq[k] = q1;
                    // (pinned here: else the sums are put off and hold their terms in registers)
#pragma unroll
                    for (int i = 0; i < KS; ++i) asm volatile("" : "+v"(dAt[i]), "+v"(car[i]));
                    asm volatile("" : "+v"(pg[k]), "+v"(pq[k]));
                    if (RT == 1 ? t < TB - 1 : t % 2 == 1 && t < TB - 2) red_add(t + 1);
                    float *to = &sred[wave][RT == 1 ? 0 : t % 2][wl * 2 * N + KS * s];
                    store_ks(to + wx, vb);
                    store_ks(to + (wx ^ N), vc);
                    if (t % RT == 0) red_read();
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int i = 0; i < KS; ++i) a[i] = an[i];
                }
                sgd[0][tq + s][cl] = lane_sums<S>(pg, s);
                sgd[1][tq + s][cl] = lane_sums<S>(pq, s);
            }
        }
        red_add(0);
#pragma unroll
        for (int i = 0; i < KS; ++i) dA[i] += dAt[i];
        load_h0(tp, h0);
        lds_barrier();

        // per-channel outputs
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int e = st + 256 * i, r = e / VPR;
            const int64_t t = tb + r;
            if (e < ITEMS && t < t1 && chn > 0) {
                const float4 xv = widen4(tok[i].x), yv = tok[i].dy.v;
                const float4 zv = widen4(tok[i].z);
                const float4 gb = *reinterpret_cast<const float4 *>(&sgd[0][r][4 * sv]);
                const float4 qa = *reinterpret_cast<const float4 *>(&sgd[1][r][4 * sv]);
                const float4 sp = *reinterpret_cast<const float4 *>(&ssp[r][4 * sv]);
                const float4 pv = *reinterpret_cast<const float4 *>(&sdy[r][4 * sv]);
                float4 ys = make_float4(0.f, 0.f, 0.f, 0.f), sz = ys;
                if constexpr (GATE) {
                    ys = *reinterpret_cast<const float4 *>(&sy[r][4 * sv]);
                    sz = *reinterpret_cast<const float4 *>(&ssz[r][4 * sv]);
                }
                float ox[4], od[4], oz[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float xj = (&xv.x)[j], p = (&pv.x)[j];
                    if constexpr (GATE) {
                        // silu' = s (1 + z (1 - s))
                        const float s = (&sz.x)[j], zj = (&zv.x)[j];
                        oz[j] = (&yv.x)[j] * ((&ys.x)[j] + Dv[j] * xj) *
                                (s * fmaf(zj, 1.f - s, 1.f));
                    }
                    ox[j] = fmaf(dkeep[i][j], (&gb.x)[j], Dv[j] * p);
                    od[j] = fmaf(xj, (&gb.x)[j], (&qa.x)[j] * kLn2) * (&sp.x)[j];
                    accD[j] = fmaf(p, xj, accD[j]);
                    accb[j] += od[j];
                }
                store_one(dx, tb, i, make_float4(ox[0], ox[1], ox[2], ox[3]));
                store_one(ddt, tb, i, make_float4(od[0], od[1], od[2], od[3]));
                if constexpr (GATE) store_one(dz, tb, i, make_float4(oz[0], oz[1], oz[2], oz[3]));
            }
        }
        // dB and dC of this channel block
        const auto rp = tile_rsrc(pbc, ((int64_t)cb * g.Bt + b) * g.T + tb, left(tb), 2 * N);
        for (int e = tid; e < TB * N / 2; e += 256) {
            const int r = e / (N / 2), o = 4 * (e % (N / 2));
            float4 v[4];
#pragma unroll
            for (int w = 0; w < 4; ++w) v[w] = *reinterpret_cast<const float4 *>(&sdbc[w][r][o]);
            float4 q;
            q.x = (v[0].x + v[1].x) + (v[2].x + v[3].x);
            q.y = (v[0].y + v[1].y) + (v[2].y + v[3].y);
            q.z = (v[0].z + v[1].z) + (v[2].z + v[3].z);
            q.w = (v[0].w + v[1].w) + (v[2].w + v[3].w);
            store_buf(rp, (uint32_t)e * 16u, q, 0.f);
        }
#pragma unroll
        for (int i = 0; i < NI; ++i) tok[i] = ntok[i];
    }

    if (c < g.Dm) {
        store_ks(pA + ((int64_t)rest * g.Dm + c) * N + KS * s, dA);
        if (dinit && seg == 0) store_ks(dinit + (b * g.Dm + c) * N + KS * s, car);
    }
    // sums over this block's token rows
    __syncthreads();
    float(*red)[CB] = reinterpret_cast<float(*)[CB]>(&sdu[0][0][0]);   // [2 ROWS][CB]
    if (st < ROWS * VPR) {
        const int r = st / VPR;
        *reinterpret_cast<float4 *>(&red[r][4 * sv]) =
            make_float4(accD[0], accD[1], accD[2], accD[3]);
        *reinterpret_cast<float4 *>(&red[ROWS + r][4 * sv]) =
            make_float4(accb[0], accb[1], accb[2], accb[3]);
    }
    __syncthreads();
    for (int e = tid; e < 2 * CB; e += 256) {
        const int q = e / CB, o = e % CB;
        const int32_t co = cb * CB + o;
        if (co < g.Dm) {
            float v = 0.f;
#pragma unroll
            for (int r = 0; r < ROWS; ++r) v += red[q * ROWS + r][o];
            (q ? pbias : pD)[(int64_t)rest * g.Dm + co] = v;
        }
    }
}

// out = sum over the partials, in order and in double.  A workgroup owns 64
// outputs; its 4 wavefronts take every fourth partial.
struct SumJob {
    const float *part;
    int64_t count, np;       // outputs, partials ([np][count])
    float *out0, *out1;      // out1: the second half of every row of 2 half elements
    int32_t half;            // 0: one output array
    uint32_t blocks;
};
struct SumJobs {
    SumJob j[4];
};
__global__ __launch_bounds__(256) void sel_sum_kernel(SumJobs jobs) {
    __shared__ double red[4][64];
    uint32_t blk = blockIdx.x;
    int k = 0;
    while (k < 3 && blk >= jobs.j[k].blocks) blk -= jobs.j[k++].blocks;
    const SumJob &j = jobs.j[k];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t i = (int64_t)blk * 64 + lane;
    double v = 0.0;
    if (i < j.count) {
#pragma unroll 8
        for (int64_t p = wave; p < j.np; p += 4) v += (double)j.part[p * j.count + i];
    }
    red[wave][lane] = v;
    __syncthreads();
    if (wave == 0 && i < j.count) {
        const float r = (float)((red[0][lane] + red[1][lane]) + (red[2][lane] + red[3][lane]));
        if (j.half) {
            const int64_t row = i / (2 * j.half);
            const int32_t o = (int32_t)(i - row * 2 * j.half);
            if (o < j.half)
                j.out0[row * j.half + o] = r;
            else
                j.out1[row * j.half + o - j.half] = r;
        } else if (j.out0) {
            j.out0[i] = r;
        }
    }
}

// How a launch is cut.  Times are counted in tiles of the reverse pass (8.6 us
// for 512 workgroups of 4 states per lane, which fill the chip: it keeps 16
// tokens' states in registers):
//   * the reverse pass takes its rounds of 512 workgroups times a segment's
//     tiles, and half a tile for first loads and last sums;
//   * the first pass, and with segments the adjoints', take 0.24 of that per
//     tile, less where more workgroups hide their waits (58 us with 2048, 75
//     with 512);
//   * 2 states per lane take 0.62 of 4.
// The cheapest is taken (8 x 1024 tokens, 5120 channels: 934 us whole, 851 us
// in 4 segments; 16 x 512 x 2048: 320 us whole, 361 in 4; 4 x 2048 x 2048: 883
// whole, 390 in 4, 374 in 16).
// (N 8 with 4 states per lane would spill registers in every form.  Of the 4-state
// forms kept, those with float32 io, a gate and an odd width spill 2 or 10 registers;
// they still beat 2 states: 4 x 2048 tokens of 2047 channels, N 16, 456 us against
// 510, 4 x 1024 of 1023, N 32, 196 against 256.)
constexpr int bwd_most_ks(int N) { return N == 8 ? 2 : 4; }
struct BwdPlan {
    int ks;
    int64_t nseg, seg_len, ncb;
    // float offsets into the workspace.  (pbc, a partial dB and dC of every channel
    // block, grows with N^2: Dm N^2 / 128 bytes a token, 4 x 2048 tokens of 2048
    // channels with N 64 0.54 GB of 0.81 GB.)
    size_t ckpt, cumd, hseg, adj, dsum, pbc, pA, pD, pbias, total;
};
BwdPlan plan(const SelArgs &a) {
    BwdPlan p;
    const int64_t tiles = cdiv64(a.T > 0 ? a.T : 1, TB);
    double best = 0.0;
    p.ks = 0;
    for (int ks = bwd_most_ks(a.N); ks >= (a.N < 64 ? 2 : 4); ks -= 2) {
        const int64_t ncb = chan_blocks(a, ks);
        for (int64_t n = 1; n <= 64 && n <= tiles; ++n) {
            const int64_t seg = cdiv64(tiles, n), nseg = cdiv64(tiles, seg);
            const double blocks = (double)(a.Bt * ncb * nseg), len = (double)seg;
            const double rounds = (double)cdiv64(a.Bt * ncb * nseg, 512);
            const double work = blocks * len / 512.0, least = 0.75 * len;
            const double passes = 2.0 - 1.0 / (double)nseg;
            const double cost =
                (ks == 2 ? 0.62 : 1.0) *
                    (rounds * (len + 0.5) +
                     0.24 * passes * (work > least ? work : least) *
                         (0.8 + 240.0 / (blocks > 256.0 ? blocks : 256.0))) +
                (nseg > 1 ? 0.5 + 0.01 * (double)nseg : 0.0);
            if (p.ks == 0 || cost < best) {
                best = cost;
                p.ks = ks;
                p.ncb = ncb;
                p.nseg = nseg;
                p.seg_len = seg * TB;
            }
        }
    }
    const int64_t ncb = p.ncb;
    const size_t st = (size_t)a.Bt * a.Dm * a.N, ch = (size_t)a.Bt * a.Dm;
    const size_t nt = (size_t)cdiv64(a.T, TB), ns = p.nseg;
    size_t o = 0;
    auto take = [&](size_t n) {
        const size_t at = o;
        o += (n + 63) & ~size_t(63);
        return at;
    };
    p.ckpt = take(st * nt);
    p.cumd = take(ns > 1 ? ch * nt : 0);
    p.hseg = take(ns > 1 ? st * ns : 0);
    p.adj = take(ns > 1 ? st * ns : 0);
    p.dsum = take(ns > 1 ? ch * ns : 0);
    p.pbc = take((size_t)ncb * a.Bt * a.T * 2 * a.N);
    p.pA = take(st * ns);
    p.pD = take(ch * ns);
    p.pbias = take(ch * ns);
    p.total = o;
    return p;
}

}  // namespace

bool selective_scan_bwd_fits(const SelArgs &a) {
    if (a.Bt == 0) return true;
    if ((double)a.Bt * (double)chan_blocks(a, 2) > (double)kMaxBlocks) return false;
    const BwdPlan p = plan(a);
    // the widest of the passes, the chain over segments and the last sums
    const double sums = ((double)a.Bt * (double)a.T * 2.0 + (double)a.Dm) * a.N / 64.0 +
                        (double)a.Dm / 32.0 + 4.0;
    return (double)a.Bt * (2.0 * (double)p.nseg - 1.0) * (double)p.ncb <= (double)kMaxBlocks &&
           (double)a.Bt * (double)a.Dm * (double)a.N <= 256.0 * (double)kMaxBlocks &&
           sums <= (double)kMaxBlocks;
}

SelLayout selective_scan_bwd_layout(const SelArgs &a) {
    const BwdPlan p = plan(a);
    return SelLayout{p.ks, p.nseg};
}

size_t selective_scan_bwd_workspace(const SelArgs &a) {
    return a.Bt > 0 ? plan(a).total * sizeof(float) : 0;
}

hipError_t launch_selective_scan_bwd(const SelArgs &a, hipStream_t st) {
    const BwdPlan p = plan(a);
    float *ws = static_cast<float *>(a.ws);
    SelGeom g;
    g.T = a.T;
    g.Bt = a.Bt;
    g.Dm = (int32_t)a.Dm;
    g.ncb = (int32_t)p.ncb;
    g.nseg = (int32_t)p.nseg;
    g.seg_len = p.seg_len;
    g.softplus = a.softplus ? 1 : 0;
    const bool rag = a.Dm % 4 != 0, split = p.nseg > 1;
    const int64_t rows = a.Bt * p.nseg;
    hipError_t e;
    if (a.Bt > 0) {
        // f(N, KS, io type, RAG)
        auto each = [&](auto f) {
            by_state(a, [&](auto n, auto io) {
                by_flag(rag, [&](auto r) {
                    constexpr int N = decltype(n)::value;
                    if constexpr (N < 64 && bwd_most_ks(N) > 2)
                        if (p.ks == 2) return f(n, std::integral_constant<int, 2>(), io, r);
                    f(n, std::integral_constant<int, bwd_most_ks(N)>(), io, r);
                });
            });
        };
        const uint32_t scans = (uint32_t)(rows * g.ncb);
        if (!split) {
            each([&](auto n, auto ks, auto io, auto r) {
                typedef decltype(io) Tio;
                sel_scan_kernel<decltype(n)::value, decltype(ks)::value, Tio, float, false,
                                decltype(r)::value, SCAN_CKPT><<<dim3(scans), 256, 0, st>>>(
                    (const Tio *)a.x, (const Tio *)a.dt, a.A, (const Tio *)a.B, nullptr, nullptr,
                    nullptr, a.dt_bias, a.init, nullptr, nullptr, ws + p.hseg, ws + p.dsum,
                    ws + p.ckpt, ws + p.cumd, g);
            });
            if ((e = hipGetLastError()) != hipSuccess) return e;
        } else {
            each([&](auto n, auto ks, auto io, auto r) {
                typedef decltype(io) Tio;
                by_flag(a.z != nullptr, [&](auto gate) {
                    sel_ends_kernel<decltype(n)::value, decltype(ks)::value, Tio,
                                    decltype(gate)::value, decltype(r)::value>
                        <<<dim3(scans + (uint32_t)(a.Bt * (p.nseg - 1) * g.ncb)), 256, 0, st>>>(
                            (const Tio *)a.x, (const Tio *)a.dt, a.A, (const Tio *)a.B,
                            (const Tio *)a.C, (const Tio *)a.z, a.dt_bias, a.dy, ws + p.hseg,
                            ws + p.dsum, ws + p.ckpt, ws + p.cumd, ws + p.adj, scans, g);
                });
            });
            if ((e = hipGetLastError()) != hipSuccess) return e;
            const int64_t total = a.Bt * a.Dm * a.N;
            sel_chain_bwd_kernel<<<dim3((uint32_t)cdiv64(total, 256)), 256, 0, st>>>(
                ws + p.hseg, ws + p.adj, ws + p.dsum, a.A, a.init, a.dfinal, total,
                (int32_t)a.Dm, (int32_t)a.N, (int32_t)p.nseg);
            if ((e = hipGetLastError()) != hipSuccess) return e;
        }
        each([&](auto n, auto ks, auto io, auto r) {
            typedef decltype(io) Tio;
            by_flag(a.z != nullptr, [&](auto gate) {
                sel_bwd_kernel<decltype(n)::value, decltype(ks)::value, Tio,
                               decltype(gate)::value, decltype(r)::value>
                    <<<dim3((uint32_t)(rows * g.ncb)), 256, 0, st>>>(
                        (const Tio *)a.x, (const Tio *)a.dt, a.A, (const Tio *)a.B,
                        (const Tio *)a.C, a.D, (const Tio *)a.z, a.dt_bias, a.dy,
                        split ? ws + p.adj : a.dfinal, ws + p.ckpt, ws + p.cumd, ws + p.hseg,
                        a.dx, a.ddt, a.dz, a.dinit, ws + p.pbc, ws + p.pA, ws + p.pD,
                        ws + p.pbias, g);
            });
        });
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    SumJobs jobs;
    auto job = [&](const float *part, int64_t count, int64_t np, float *o0, float *o1, int half) {
        return SumJob{part, count, np, o0, o1, half, (uint32_t)cdiv64(count, 64)};
    };
    jobs.j[0] = job(ws + p.pbc, a.Bt * a.T * 2 * a.N, p.ncb, a.dB, a.dC, a.N);
    jobs.j[1] = job(ws + p.pA, a.Dm * a.N, rows, a.dA, nullptr, 0);
    jobs.j[2] = job(ws + p.pD, a.Dm, rows, a.dD, nullptr, 0);
    jobs.j[3] = job(ws + p.pbias, a.Dm, rows, a.dbias, nullptr, 0);
    uint32_t blocks = 0;
    for (const SumJob &j : jobs.j) blocks += j.blocks;
    sel_sum_kernel<<<dim3(blocks), 256, 0, st>>>(jobs);
    return hipGetLastError();
}

}  // namespace ssd
