// Shared by the forward, step and backward kernels of the per-channel
// selective scan (gfx950 only).
//
// Work split: a channel's N states lie on S = N/4 neighbouring lanes, 4 per
// lane, so a wavefront holds 64/S channels and a workgroup of 4 wavefronts CB
// = 256/S.  Token tiles pass through LDS: 16-byte row segments are loaded,
// d = softplus(dt + bias) and u = d x formed once per (token, channel), and
// the scanning lanes then read (d, u) of their channel and their 4 elements
// of B and C.
#pragma once

#include <type_traits>

#include "layer_launch.h"
#include "ssd_device.h"

namespace ssd {

template <int N>
struct SelSplit {
    static constexpr int S = N / 4;        // lanes of a channel
    static constexpr int CPW = 64 / S;     // channels of a wavefront
    static constexpr int CB = 4 * CPW;     // channels of a workgroup
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

// log(1 + e^r), r above 20 unchanged.  e^r as a power of two with the
// argument's rounding put back; log(1 + e) with the rounding of 1 + e put
// back, so small results keep their relative accuracy.
__device__ __forceinline__ float softplus_f(float r) {
    if (r > 20.f) return r;
    r = r < -150.f ? -150.f : r;   // (e^r is 0 in float32; -inf stays out of the products)
    constexpr float kLog2eLo = 1.9259629911266175e-8f;   // log2(e) - (float)log2(e)
    const float hi = r * kLog2e;
    const float lo = fmaf(r, kLog2eLo, fmaf(r, kLog2e, -hi));
    float e = fast_exp2(hi);
    e = fmaf(e, lo * kLn2, e);
    const float w = 1.f + e;
    return fmaf(__builtin_amdgcn_logf(w), kLn2, (e - (w - 1.f)) * __builtin_amdgcn_rcpf(w));
}
__device__ __forceinline__ float sigmoid_f(float v) {
    return __builtin_amdgcn_rcpf(1.f + fast_exp2(-kLog2e * v));
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

// Tokens of a tile: N * CB = 1024 elements, 4 per thread.
template <int N>
struct Tile {
    static constexpr int TL = N;
    static constexpr int VPR = SelSplit<N>::CB / 4;              // 4-channel vectors of a row
    static constexpr int NBC = (2 * TL * N / 4 + 255) / 256;     // B, C vectors per thread
};

struct SelGeom {
    int64_t T, Bt;
    int32_t Dm, ncb;      // channels, channel blocks
    int32_t nseg;         // segments of a sequence
    int64_t seg_len;      // tokens of a segment (a multiple of the tile)
    int32_t softplus;
};

// One segment of one sequence, CB channels.
//   SCAN_OUT   write y, and the last segment the final state;
//   SCAN_END   write the segment's end state, started from zero, and its sum of
//              d (every segment but the last);
//   SCAN_CKPT  write the state before every 16th token and, with several
//              segments (each then started from zero), the sum of d up to it,
//              the end states and sums of d.
enum ScanMode { SCAN_OUT, SCAN_END, SCAN_CKPT };
template <int N, typename Tio, typename Ty, bool GATE, bool RAG, ScanMode MODE>
__global__ __launch_bounds__(256) void sel_scan_kernel(
    const Tio *__restrict__ x, const Tio *__restrict__ dt, const float *__restrict__ A,
    const Tio *__restrict__ B, const Tio *__restrict__ C, const float *__restrict__ D,
    const Tio *__restrict__ z, const float *__restrict__ dt_bias, const float *start,
    const int32_t *__restrict__ lens, Ty *__restrict__ y, float *fin, float *__restrict__ dsum,
    float *__restrict__ ckpt, float *__restrict__ cumd, SelGeom g) {
    constexpr bool OUT = MODE == SCAN_OUT;
    constexpr int S = SelSplit<N>::S, CPW = SelSplit<N>::CPW, CB = SelSplit<N>::CB;
    constexpr int TL = Tile<N>::TL, VPR = Tile<N>::VPR, NBC = Tile<N>::NBC;
    __shared__ __align__(16) float2 sdu[TL][CB];
    __shared__ __align__(16) float sbc[2][TL][N];
    __shared__ __align__(16) float sy[OUT ? TL : 1][OUT ? CB : 4];

    const int tid = threadIdx.x;
    const uint32_t cb = blockIdx.x % (uint32_t)g.ncb;
    const uint32_t rest = blockIdx.x / (uint32_t)g.ncb;
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
    auto load_tok = [&](const Tio *p, int64_t t) {
        Raw4<Tio> r;
        zero_raw(r);
        if (t < te && scn > 0) r = load_raw<RAG>(p + (row0 + t) * g.Dm + sc, scn);
        return r;
    };
    auto load_bc = [&](int64_t tb, int k) {           // vector k of this thread's B, C share
        const int e = tid + 256 * k;
        Raw4<Tio> r;
        zero_raw(r);
        if (e < 2 * TL * N / 4) {
            const int q = e / (TL * N / 4), o = e % (TL * N / 4);
            const int64_t t = tb + o / (N / 4);
            if (t < te && (OUT || q == 0))
                r = load_raw<false>((q ? C : B) + (row0 + t) * N + 4 * (o % (N / 4)), 4);
        }
        return r;
    };

    // scanning role: 4 states of one channel
    const int lane = tid & 63, wave = tid >> 6;
    const int s = lane % S, cl = wave * CPW + lane / S;
    const int32_t c = cb * CB + cl;
    float a2[4], h[4], ds = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) a2[i] = h[i] = 0.f;
    if (c < g.Dm) {
        const float4 av = *reinterpret_cast<const float4 *>(A + (int64_t)c * N + 4 * s);
        a2[0] = av.x * kLog2e;
        a2[1] = av.y * kLog2e;
        a2[2] = av.z * kLog2e;
        a2[3] = av.w * kLog2e;
        if (start) {   // [Bt][nseg][Dm][N]: with one segment the initial state
            const float4 hv = *reinterpret_cast<const float4 *>(
                start + (((b * g.nseg) + seg) * g.Dm + c) * N + 4 * s);
            h[0] = hv.x;
            h[1] = hv.y;
            h[2] = hv.z;
            h[3] = hv.w;
        }
    }

    Raw4<Tio> rx = load_tok(x, t0 + sr), rd = load_tok(dt, t0 + sr), rz, rbc[NBC];
    if constexpr (GATE && OUT) rz = load_tok(z, t0 + sr);
#pragma unroll
    for (int k = 0; k < NBC; ++k) rbc[k] = load_bc(t0, k);

    for (int64_t tb = t0; tb < te; tb += TL) {
        // stage the tile
        const float4 xv = widen4(rx), dv = widen4(rd);
        const float *xp = &xv.x, *dp = &dv.x;
        float d[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float r = dp[i] + bias[i];
            d[i] = g.softplus ? softplus_f(r) : r;
            if (tb + sr >= te) d[i] = 0.f;
        }
        float4 *du = reinterpret_cast<float4 *>(&sdu[sr][4 * sv]);
        du[0] = make_float4(d[0], d[0] * xp[0], d[1], d[1] * xp[1]);
        du[1] = make_float4(d[2], d[2] * xp[2], d[3], d[3] * xp[3]);
#pragma unroll
        for (int k = 0; k < NBC; ++k) {
            const int e = tid + 256 * k;
            if (e < 2 * TL * N / 4)
                reinterpret_cast<float4 *>(&sbc[0][0][0])[e] = widen4(rbc[k]);
        }
        // the next tile's loads, in flight during the scan
        const int64_t tn = tb + TL;
        const Raw4<Tio> nx = load_tok(x, tn + sr), nd = load_tok(dt, tn + sr);
        Raw4<Tio> nz, nbc[NBC];
        if constexpr (GATE && OUT) nz = load_tok(z, tn + sr);
#pragma unroll
        for (int k = 0; k < NBC; ++k) nbc[k] = load_bc(tn, k);
        lds_barrier();

        // scan the tile
#pragma unroll 1
        for (int tq = 0; tq < TL; tq += 8) {
            if constexpr (MODE == SCAN_CKPT) {
                const int64_t t = tb + tq;
                if ((t & 15) == 0 && t < te && c < g.Dm) {
                    const int64_t u = (b * ((g.T + 15) >> 4) + (t >> 4)) * g.Dm + c;
                    *reinterpret_cast<float4 *>(ckpt + u * N + 4 * s) =
                        make_float4(h[0], h[1], h[2], h[3]);
                    if (g.nseg > 1 && s == 0) cumd[u] = ds;
                }
            }
            float keep = 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int t = tq + k;
                const float2 w = sdu[t][cl];
                const float4 bv = *reinterpret_cast<const float4 *>(&sbc[0][t][4 * s]);
                h[0] = fmaf(fast_exp2(w.x * a2[0]), h[0], w.y * bv.x);
                h[1] = fmaf(fast_exp2(w.x * a2[1]), h[1], w.y * bv.y);
                h[2] = fmaf(fast_exp2(w.x * a2[2]), h[2], w.y * bv.z);
                h[3] = fmaf(fast_exp2(w.x * a2[3]), h[3], w.y * bv.w);
                if constexpr (OUT) {
                    const float4 cv = *reinterpret_cast<const float4 *>(&sbc[1][t][4 * s]);
                    float p = h[0] * cv.x + h[1] * cv.y + h[2] * cv.z + h[3] * cv.w;
                    p = chan_sum<S>(p);
                    // lane s of a channel keeps token s of every S
                    if (S >= 8 ? s == t % S : s == k % S) keep = p;
                    if constexpr (S <= 8) {
                        if ((k + 1) % S == 0) sy[t - (S - 1) + s][cl] = keep;
                    } else if (k == 7 && (s >> 3) == ((tq >> 3) & 1)) {
                        sy[(tq & ~(S - 1)) + s][cl] = keep;
                    }
                } else {
                    ds += w.x;
                }
            }
        }
        lds_barrier();

        if constexpr (OUT) {
            const int64_t t = tb + sr;
            if (t < te && scn > 0) {
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
                store4<RAG>(y + (row0 + t) * g.Dm + sc, make_float4(o[0], o[1], o[2], o[3]), scn);
            }
            if constexpr (GATE) rz = nz;
        }
        rx = nx;
        rd = nd;
#pragma unroll
        for (int k = 0; k < NBC; ++k) rbc[k] = nbc[k];
    }

    if constexpr (OUT) {
        // padded tokens
        if (scn > 0)
            for (int64_t t = te + sr; t < t1; t += TL)
                store4<RAG>(y + (row0 + t) * g.Dm + sc, make_float4(0.f, 0.f, 0.f, 0.f), scn);
        if (fin && seg == g.nseg - 1 && c < g.Dm)
            *reinterpret_cast<float4 *>(fin + (b * g.Dm + c) * N + 4 * s) =
                make_float4(h[0], h[1], h[2], h[3]);
    } else if (c < g.Dm && g.nseg > 1) {
        const int64_t u = (b * g.nseg + seg) * g.Dm + c;
        *reinterpret_cast<float4 *>(fin + u * N + 4 * s) = make_float4(h[0], h[1], h[2], h[3]);
        if (s == 0) dsum[u] = ds;
    }
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
inline int64_t chan_blocks(const SelArgs &a) { return cdiv64(a.Dm, 1024 / a.N); }

}  // namespace ssd
