// Shared by the forward, step and backward kernels of the per-channel
// selective scan (gfx950 only).
//
// Work split: a channel's N states lie on S = N/KS neighbouring lanes, KS (4 or
// 2) per lane, so a wavefront holds 64/S channels and a workgroup of 4
// wavefronts CB = 256/S.  Token tiles pass through LDS: lanes load 4 channels
// of a token, d = softplus(dt + bias) and u = d x are formed once per (token,
// channel), and the scanning lanes then read (d, u) of their channel and their
// KS elements of B and C.
#pragma once

#include <type_traits>

#include "layer_launch.h"
#include "ssd_device.h"

namespace ssd {

template <int N, int KS = 4>
struct SelSplit {
    static constexpr int S = N / KS;       // lanes of a channel
    static constexpr int CPW = 64 / S;     // channels of a wavefront
    static constexpr int CB = 4 * CPW;     // channels of a workgroup
    static constexpr int TL = 1024 / CB;   // tokens of a tile: 4 elements per thread
    static constexpr int VPR = CB / 4;     // 4-channel vectors of a tile's row
    // Row of an LDS array that a channel's lanes write as S tokens at once: rows
    // are moved on by 32 / S banks, so that they do not meet in one (conflict
    // cycles of 8 x 4096 tokens, 5120 channels: 13 million, 47 without; 705 us, 718)
    static constexpr int ROW = CB + (S <= 2 ? 16 : (S == 4 ? 8 : 4));
    static constexpr int BC = TL * N / 4;  // 4-element vectors of a tile's B (or C)
    static constexpr int NBC = (BC + 255) / 256;   // of them per thread
};

constexpr float kLn2 = 0.69314718055994531f;

// 4 consecutive stored elements; n (<= 4) of them exist.  Rows of an odd
// width start at any element, so only element alignment is assumed.
template <typename Tio>
struct Raw4;
template <>
struct Raw4<float> {
    typedef float type __attribute__((ext_vector_type(4), aligned(4)));
    float4 v;
};
template <>
struct Raw4<uint16_t> {
    typedef uint32_t type __attribute__((ext_vector_type(2), aligned(2)));
    uint2 v;
};
__device__ __forceinline__ void zero_raw(Raw4<float> &r) { r.v = make_float4(0.f, 0.f, 0.f, 0.f); }
__device__ __forceinline__ void zero_raw(Raw4<uint16_t> &r) { r.v = make_uint2(0u, 0u); }
template <bool RAG>
__device__ __forceinline__ Raw4<float> load_raw(const float *p, int n) {
    Raw4<float> r;
    if (!RAG || n >= 4) {
        const auto w = *reinterpret_cast<const Raw4<float>::type *>(p);
        r.v = make_float4(w[0], w[1], w[2], w[3]);
    } else {
        r.v.x = n > 0 ? p[0] : 0.f;
        r.v.y = n > 1 ? p[1] : 0.f;
        r.v.z = n > 2 ? p[2] : 0.f;
        r.v.w = 0.f;
    }
    return r;
}
template <bool RAG>
__device__ __forceinline__ Raw4<uint16_t> load_raw(const uint16_t *p, int n) {
    Raw4<uint16_t> r;
    if (!RAG || n >= 4) {
        const auto w = *reinterpret_cast<const Raw4<uint16_t>::type *>(p);
        r.v = make_uint2(w[0], w[1]);
    } else {
        const uint32_t e0 = n > 0 ? p[0] : 0u, e1 = n > 1 ? p[1] : 0u, e2 = n > 2 ? p[2] : 0u;
        r.v = make_uint2(e0 | e1 << 16, e2);
    }
    return r;
}
__device__ __forceinline__ float4 widen4(const Raw4<float> &r) { return r.v; }
__device__ __forceinline__ float4 widen4(const Raw4<uint16_t> &r) {
    return make_float4(bf16_lo(r.v.x), bf16_hi(r.v.x), bf16_lo(r.v.y), bf16_hi(r.v.y));
}
template <bool RAG>
__device__ __forceinline__ void store4(float *p, float4 v, int n) {
    if (!RAG || n >= 4) {
        typedef Raw4<float>::type W;
        const W w = {v.x, v.y, v.z, v.w};
        *reinterpret_cast<W *>(p) = w;
    } else {
        if (n > 0) p[0] = v.x;
        if (n > 1) p[1] = v.y;
        if (n > 2) p[2] = v.z;
    }
}
template <bool RAG>
__device__ __forceinline__ void store4(uint16_t *p, float4 v, int n) {
    const uint32_t lo = pack_bf16x2(v.x, v.y), hi = pack_bf16x2(v.z, v.w);
    if (!RAG || n >= 4) {
        typedef Raw4<uint16_t>::type W;
        const W w = {lo, hi};
        *reinterpret_cast<W *>(p) = w;
    } else {
        if (n > 0) p[0] = (uint16_t)(lo & 0xffffu);
        if (n > 1) p[1] = (uint16_t)(lo >> 16);
        if (n > 2) p[2] = (uint16_t)(hi & 0xffffu);
    }
}

// d = log(1 + e^r) = max(r, 0) + log(1 + e^-|r|); above 20 that is r in
// float32.  e^-|r| as a power of two (of hi, with the rest of the argument put
// back to first order), and log(1 + e) with the rounding of 1 + e put back, so
// small results keep their relative accuracy.  |r| is held to 126, where e^-|r|
// is 0 next to anything: hi stays finite up to r = +-inf.  The minimum and the
// maximum let NaN through.  w = 1 + e, for the derivative below.
__device__ __forceinline__ float softplus_f(float r, float &e, float &w) {
    const float q = -__builtin_elementwise_minimum(fabsf(r), 126.f), hi = q * kLog2e;
    e = fast_exp2(hi);
    e = fmaf(e, fmaf(hi, -kLn2, q), e);
    w = 1.f + e;
    return __builtin_elementwise_maximum(r, 0.f) +
           fmaf(__builtin_amdgcn_logf(w), kLn2, e - (w - 1.f));
}
__device__ __forceinline__ float softplus_f(float r) {
    float e, w;
    return softplus_f(r, e, w);
}
// d and its derivative sigmoid(r)
__device__ __forceinline__ float softplus_f(float r, float &slope) {
    float e, w;
    const float d = softplus_f(r, e, w);
    slope = (r < 0.f ? e : 1.f) * __builtin_amdgcn_rcpf(w);
    return d;
}
__device__ __forceinline__ float sigmoid_f(float v) {
    return __builtin_amdgcn_rcpf(1.f + fast_exp2(-kLog2e * v));
}

// A rate for exponentials to base 2.  Held where the product is finite (-2^127), so
// that a step of d = 0 leaves the state as it is at any rate; NaN passes.
__device__ __forceinline__ float rate2(float A) {
    return __builtin_elementwise_maximum(A, -0x1p127f) * kLog2e;
}

// Sum over the S lanes of a channel, in every one of them.
template <int S>
__device__ __forceinline__ float chan_sum(float v) {
    v += dpp_mov<0xB1>(v);                            // quad_perm [1,0,3,2]
    if constexpr (S >= 4) v += dpp_mov<0x4E>(v);      // quad_perm [2,3,0,1]
    if constexpr (S >= 8) v += dpp_mov<0x141>(v);     // row_half_mirror
    if constexpr (S >= 16) v += dpp_mov<0x140>(v);    // row_mirror
    return v;
}

// Sums over the S lanes of a channel of S values per lane (one per token):
// lane s receives the sum of p[s].  Each step pairs lanes by a mirror or a
// swap, keeps half of the values and hands the partner the other half: S - 1
// additions for S sums, where S separate butterflies take S log2 S.
template <int S>
__device__ __forceinline__ float lane_sums(float (&p)[S], int s) {
    if constexpr (S == 16) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float keep = s & 8 ? p[i + 8] : p[i], send = s & 8 ? p[i] : p[i + 8];
            p[i] = keep + dpp_mov<0x140>(send);   // row_mirror: lane 15 - s
        }
    }
    if constexpr (S >= 8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float keep = s & 4 ? p[i + 4] : p[i], send = s & 4 ? p[i] : p[i + 4];
            p[i] = keep + dpp_mov<0x141>(send);   // row_half_mirror: lane 7 - s
        }
    }
    if constexpr (S >= 4) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float keep = s & 2 ? p[i + 2] : p[i], send = s & 2 ? p[i] : p[i + 2];
            p[i] = keep + dpp_mov<0x4E>(send);    // lane s ^ 2
        }
    }
    const float keep = s & 1 ? p[1] : p[0], send = s & 1 ? p[0] : p[1];
    return keep + dpp_mov<0xB1>(send);            // lane s ^ 1
}

// KS consecutive floats of LDS or global memory (aligned)
template <int KS>
__device__ __forceinline__ void load_ks(const float *p, float (&v)[KS]) {
    if constexpr (KS == 4) {
        const float4 w = *reinterpret_cast<const float4 *>(p);
        v[0] = w.x;
        v[1] = w.y;
        v[2] = w.z;
        v[3] = w.w;
    } else {
        const float2 w = *reinterpret_cast<const float2 *>(p);
        v[0] = w.x;
        v[1] = w.y;
    }
}
template <int KS>
__device__ __forceinline__ void store_ks(float *p, const float (&v)[KS]) {
    if constexpr (KS == 4)
        *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
    else
        *reinterpret_cast<float2 *>(p) = make_float2(v[0], v[1]);
}

// A value that every lane holds alike, in scalar registers: a resource built
// from vector registers would be read lane by lane in a loop.
__device__ __forceinline__ int64_t uniform64(int64_t v) {
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)((uint64_t)v >> 32));
    return (int64_t)((uint64_t)hi << 32 | lo);
}

// Rows of a token tile through a buffer resource: row r, byte v within it at
// offset r * width + v from the tile's first row, rows past the last token
// read as zero and are not written (the buffer range check).
template <typename T>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t tile_rsrc(T *base, int64_t row, int64_t rows,
                                                            int32_t width) {
    const int64_t left = rows < 64 ? (rows > 0 ? rows : 0) : 64;
    return make_rsrc(base + uniform64(row * width),
                     __builtin_amdgcn_readfirstlane(
                         (uint32_t)(left * width * (int64_t)sizeof(T))));
}
constexpr uint32_t kNoOffset = 0x80000000u;   // past every tile
__device__ __forceinline__ Raw4<float> load_buf(__amdgpu_buffer_rsrc_t r, uint32_t off, float) {
    const auto v = __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0);
    Raw4<float> o;
    o.v = make_float4(__uint_as_float(v[0]), __uint_as_float(v[1]), __uint_as_float(v[2]),
                      __uint_as_float(v[3]));
    return o;
}
__device__ __forceinline__ Raw4<uint16_t> load_buf(__amdgpu_buffer_rsrc_t r, uint32_t off,
                                                   uint16_t) {
    const auto v = __builtin_amdgcn_raw_buffer_load_b64(r, off, 0, 0);
    Raw4<uint16_t> o;
    o.v = make_uint2(v[0], v[1]);
    return o;
}
__device__ __forceinline__ void store_buf(__amdgpu_buffer_rsrc_t r, uint32_t off, float4 v,
                                          float) {
    const u32x4 w = {__float_as_uint(v.x), __float_as_uint(v.y), __float_as_uint(v.z),
                     __float_as_uint(v.w)};
    __builtin_amdgcn_raw_buffer_store_b128(w, r, off, 0, 0);
}
__device__ __forceinline__ void store_buf(__amdgpu_buffer_rsrc_t r, uint32_t off, float4 v,
                                          uint16_t) {
    const u32x2 w = {pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w)};
    __builtin_amdgcn_raw_buffer_store_b64(w, r, off, 0, 0);
}

// KS floats at byte offset off (zero past the resource)
template <int KS>
__device__ __forceinline__ void load_buf_ks(__amdgpu_buffer_rsrc_t r, uint32_t off,
                                            float (&v)[KS]) {
    if constexpr (KS == 4) {
        const auto w = __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(w[i]);
    } else {
        const auto w = __builtin_amdgcn_raw_buffer_load_b64(r, off, 0, 0);
        v[0] = __uint_as_float(w[0]);
        v[1] = __uint_as_float(w[1]);
    }
}

struct SelGeom {
    int64_t T, Bt;
    int32_t Dm, ncb;      // channels, channel blocks
    int32_t nseg;         // segments of a sequence
    int64_t seg_len;      // its tokens: a multiple of the tile, in the gradients of 16
    int32_t softplus;
};

// One segment of one sequence, CB channels (block blk of the launch's).
//   SCAN_OUT   write y, and the last segment the final state;
//   SCAN_END   write the segment's end state, started from zero, and its sum of
//              d (every segment but the last);
//   SCAN_CKPT  write the state before every 16th token and, with several
//              segments (each then started from zero), the sum of d up to it,
//              the end states and sums of d.
enum ScanMode { SCAN_OUT, SCAN_END, SCAN_CKPT };
template <int N, int KS, typename Tio, typename Ty, bool GATE, bool RAG, ScanMode MODE>
__device__ __forceinline__ void sel_scan(
    const Tio *__restrict__ x, const Tio *__restrict__ dt, const float *__restrict__ A,
    const Tio *__restrict__ B, const Tio *__restrict__ C, const float *__restrict__ D,
    const Tio *__restrict__ z, const float *__restrict__ dt_bias, const float *start,
    const int32_t *__restrict__ lens, Ty *__restrict__ y, float *fin, float *__restrict__ dsum,
    float *__restrict__ ckpt, float *__restrict__ cumd, SelGeom g, uint32_t blk) {
    constexpr bool OUT = MODE == SCAN_OUT;
    typedef SelSplit<N, KS> Sp;
    constexpr int S = Sp::S, CPW = Sp::CPW, CB = Sp::CB, TL = Sp::TL, VPR = Sp::VPR;
    constexpr int BC = Sp::BC, NBC = Sp::NBC;
    __shared__ __align__(16) float2 sdu[TL][CB];
    __shared__ __align__(16) float sbc[2][TL][N];
    __shared__ __align__(16) float sy[OUT ? TL : 1][OUT ? Sp::ROW : 4];

    const int tid = threadIdx.x;
    const uint32_t cb = blk % (uint32_t)g.ncb;
    const uint32_t rest = blk / (uint32_t)g.ncb;
    const uint32_t nsg = MODE == SCAN_END ? g.nseg - 1 : g.nseg;
    const int64_t b = rest / nsg;
    const int32_t seg = rest % nsg;
    const int64_t t0 = seg * g.seg_len;
    const int64_t t1 = min(g.T, t0 + g.seg_len);
    const int64_t len = lens ? min((int64_t)max(lens[b], 0), g.T) : g.T;
    const int64_t te = min(t1, max(len, t0));         // tokens scanned: t0 .. te

    // staging role: token row sr of the tile, channels sc .. sc + 3
    const int sr = tid / VPR, sv = tid % VPR;
    const int32_t sc = cb * CB + 4 * sv;
    const int scn = min(4, g.Dm - sc);                // how many exist (may be <= 0)
    float bias[4], Dv[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        bias[i] = dt_bias && i < scn ? dt_bias[sc + i] : 0.f;
        Dv[i] = OUT && i < scn ? D[sc + i] : 0.f;
    }
    const int64_t row0 = b * g.T;
    // (rows of an odd width are not aligned to a lane's vector: RAG takes them
    // through plain loads and bounds its last channels by hand)
    const uint32_t off = scn > 0 ? ((uint32_t)sr * g.Dm + sc) : kNoOffset / sizeof(Tio);
    auto load_tok = [&](const Tio *p, int64_t tb) {
        if constexpr (RAG) {
            Raw4<Tio> r;
            zero_raw(r);
            if (tb + sr < te && scn > 0)
                r = load_raw<true>(p + (row0 + tb + sr) * g.Dm + sc, scn);
            return r;
        } else {
            return load_buf(tile_rsrc(p, row0 + tb, te - tb, g.Dm), off * sizeof(Tio), Tio());
        }
    };
    auto store_tok = [&](int64_t tb, float4 v) {
        if constexpr (RAG) {
            if (tb + sr < te && scn > 0)
                store4<true>(y + (row0 + tb + sr) * g.Dm + sc, v, scn);
        } else {
            store_buf(tile_rsrc(y, row0 + tb, te - tb, g.Dm),
                      scn > 0 ? off * (uint32_t)sizeof(Ty) : kNoOffset, v, Ty());
        }
    };
    // vectors e of the tile's B (from the first thread up) and C (from the last down)
    auto load_bc = [&](const Tio *p, int64_t tb, int e) {
        return load_buf(tile_rsrc(p, row0 + tb, min(te - tb, (int64_t)TL), N),
                        e < BC ? (uint32_t)e * 4 * sizeof(Tio) : kNoOffset, Tio());
    };

    // scanning role: KS states of one channel
    const int lane = tid & 63, wave = tid >> 6;
    const int s = lane % S, cl = wave * CPW + lane / S;
    const int32_t c = cb * CB + cl;
    float a2[KS], h[KS], ds = 0.f;
#pragma unroll
    for (int i = 0; i < KS; ++i) a2[i] = h[i] = 0.f;
    if (c < g.Dm) {
        load_ks(A + (int64_t)c * N + KS * s, a2);
#pragma unroll
        for (int i = 0; i < KS; ++i) a2[i] = rate2(a2[i]);
        if (start)   // [Bt][nseg][Dm][N]: with one segment the initial state
            load_ks(start + (((b * g.nseg) + seg) * g.Dm + c) * N + KS * s, h);
    }

    Raw4<Tio> rx = load_tok(x, t0), rd = load_tok(dt, t0), rz, rb[NBC], rc[NBC];
    if constexpr (GATE && OUT) rz = load_tok(z, t0);
#pragma unroll
    for (int k = 0; k < NBC; ++k) {
        rb[k] = load_bc(B, t0, tid + 256 * k);
        if constexpr (OUT) rc[k] = load_bc(C, t0, 255 - tid + 256 * k);
    }

    for (int64_t tb = t0; tb < te; tb += TL) {
        // stage the tile
        const float4 xv = widen4(rx), dv = widen4(rd);
        const float *xp = &xv.x, *dp = &dv.x;
        float d[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float r = dp[i] + bias[i];
            d[i] = g.softplus ? softplus_f(r) : r;
        }
        if (tb + TL > te) {   // (tokens past the end leave the state as it is)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (tb + sr >= te) d[i] = 0.f;
        }
        float4 *du = reinterpret_cast<float4 *>(&sdu[sr][4 * sv]);
        du[0] = make_float4(d[0], d[0] * xp[0], d[1], d[1] * xp[1]);
        du[1] = make_float4(d[2], d[2] * xp[2], d[3], d[3] * xp[3]);
#pragma unroll
        for (int k = 0; k < NBC; ++k) {
            const int eb = tid + 256 * k, ec = 255 - tid + 256 * k;
            if (eb < BC) reinterpret_cast<float4 *>(&sbc[0][0][0])[eb] = widen4(rb[k]);
            if (OUT && ec < BC) reinterpret_cast<float4 *>(&sbc[1][0][0])[ec] = widen4(rc[k]);
        }
        // the next tile's loads, in flight during the scan
        const int64_t tn = tb + TL;
        const Raw4<Tio> nx = load_tok(x, tn), nd = load_tok(dt, tn);
        Raw4<Tio> nz;
        if constexpr (GATE && OUT) nz = load_tok(z, tn);
#pragma unroll
        for (int k = 0; k < NBC; ++k) {
            rb[k] = load_bc(B, tn, tid + 256 * k);
            if constexpr (OUT) rc[k] = load_bc(C, tn, 255 - tid + 256 * k);
        }
        lds_barrier();

        // scan the tile
        constexpr int U = TL < 32 ? TL : 32;   // tokens unrolled
#pragma unroll 1
        for (int tq = 0; tq < TL && tb + tq < te; tq += U) {
#pragma unroll
            for (int k0 = 0; k0 < U; k0 += S) {
                float p[S];
#pragma unroll
                for (int k = 0; k < S; ++k) {
                    const int t = tq + k0 + k;
                    if constexpr (MODE == SCAN_CKPT) {
                        if ((k0 + k) % 8 == 0 && ((tb + t) & 15) == 0 && tb + t < te && c < g.Dm) {
                            const int64_t u =
                                (b * ((g.T + 15) >> 4) + ((tb + t) >> 4)) * g.Dm + c;
                            store_ks(ckpt + u * N + KS * s, h);
                            if (g.nseg > 1 && s == 0) cumd[u] = ds;
                        }
                    }
                    const float2 w = sdu[t][cl];
                    float bv[KS];
                    load_ks(&sbc[0][t][KS * s], bv);
#pragma unroll
                    for (int i = 0; i < KS; ++i)
                        h[i] = fmaf(fast_exp2(w.x * a2[i]), h[i], w.y * bv[i]);
                    if constexpr (OUT) {
                        float cv[KS];
                        load_ks(&sbc[1][t][KS * s], cv);
                        p[k] = h[0] * cv[0];
#pragma unroll
                        for (int i = 1; i < KS; ++i) p[k] = fmaf(h[i], cv[i], p[k]);
                    } else {
                        ds += w.x;
                    }
                }
                if constexpr (OUT) sy[tq + k0 + s][cl] = lane_sums<S>(p, s);
            }
        }
        lds_barrier();

        if constexpr (OUT) {
            const float4 yv = *reinterpret_cast<const float4 *>(&sy[sr][4 * sv]);
            const float *yp = &yv.x;
            float o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = yp[i] + Dv[i] * xp[i];
            if constexpr (GATE) {
                const float4 zv = widen4(rz);
                const float *zp = &zv.x;
#pragma unroll
                for (int i = 0; i < 4; ++i) o[i] *= fast_silu(zp[i]);
            }
            store_tok(tb, make_float4(o[0], o[1], o[2], o[3]));
            if constexpr (GATE) rz = nz;
        }
        rx = nx;
        rd = nd;
    }

    if constexpr (OUT) {
        // padded tokens
        if (scn > 0)
            for (int64_t t = te + sr; t < t1; t += TL)
                store4<RAG>(y + (row0 + t) * g.Dm + sc, make_float4(0.f, 0.f, 0.f, 0.f), scn);
        if (fin && seg == g.nseg - 1 && c < g.Dm)
            store_ks(fin + (b * g.Dm + c) * N + KS * s, h);
    } else if (c < g.Dm && g.nseg > 1) {
        const int64_t u = (b * g.nseg + seg) * g.Dm + c;
        store_ks(fin + u * N + KS * s, h);
        if (s == 0) dsum[u] = ds;
    }
}
template <int N, int KS, typename Tio, typename Ty, bool GATE, bool RAG, ScanMode MODE>
__global__ __launch_bounds__(256) void sel_scan_kernel(
    const Tio *__restrict__ x, const Tio *__restrict__ dt, const float *__restrict__ A,
    const Tio *__restrict__ B, const Tio *__restrict__ C, const float *__restrict__ D,
    const Tio *__restrict__ z, const float *__restrict__ dt_bias, const float *start,
    const int32_t *__restrict__ lens, Ty *__restrict__ y, float *fin, float *__restrict__ dsum,
    float *__restrict__ ckpt, float *__restrict__ cumd, SelGeom g) {
    sel_scan<N, KS, Tio, Ty, GATE, RAG, MODE>(x, dt, A, B, C, D, z, dt_bias, start, lens, y, fin,
                                              dsum, ckpt, cumd, g, blockIdx.x);
}

// f(integral_constant<N>, io type)
template <typename F>
void by_state(const SelArgs &a, F f) {
    auto g = [&](auto n) {
        if (a.bf16)
            f(n, uint16_t());
        else
            f(n, float());
    };
    if (a.N == 8) g(std::integral_constant<int, 8>());
    if (a.N == 16) g(std::integral_constant<int, 16>());
    if (a.N == 32) g(std::integral_constant<int, 32>());
    if (a.N == 64) g(std::integral_constant<int, 64>());
}
template <typename F>
void by_flag(bool v, F f) {
    if (v)
        f(std::true_type());
    else
        f(std::false_type());
}

inline int64_t cdiv64(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int64_t chan_blocks(const SelArgs &a, int ks = 4) {
    return cdiv64(a.Dm, 256 * ks / a.N);
}

}  // namespace ssd
