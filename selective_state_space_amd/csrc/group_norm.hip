// Group norm behind a mixer, channels last: each token's groups of S consecutive
// channels on their own (so that it is causal),
//     u = x, or x silu(z);   n = (u - mean) rstd w + b   (rms: mean = 0),
//     y = n, silu(n) or n silu(z),
// and its gradients.  silu(z) = z sigmoid(z).
//
// With c = (u - mean) rstd the normalised u and d the gradient of c,
//     du = rstd (d - mean(d) - c mean(d c))      (rms: without mean(d)).
//
// Everything is read once and written once, and memory bounds it: 8 x 4096 tokens of
// 5120 channels, 40 groups, bf16, gated, 210 us (4.8 TB/s, a copy's rate); gradients of
// 4 x 2048 x 2048, one group, gated in front, 45 us (3.7 TB/s, 4 us of them the weights'
// sums); a token for each of 5 sequences, 2100 channels, 3.7.  A row (a
// token's group) lies in the registers of TPR lanes, VPT accesses of VEC channels
// each, so that mean and variance are formed in two passes over registers: the
// variance of a row whose mean is large loses nothing to cancellation.  A lane
// keeps its channels for a run of tokens: their weights are loaded once, and their
// gradients summed in registers.

#include "block_launch.h"
#include "layer_launch.h"
#include "ssd_device.h"

#include "../../include/ssd.h"

namespace ssd {

namespace {

// sigmoid(z) on the transcendental unit
__device__ __forceinline__ float sigm(float z) {
    return __builtin_amdgcn_rcpf(1.f + fast_exp2(-kLog2e * z));
}

template <int VEC, typename T>
__device__ __forceinline__ void load_vec(float *v, const T *p) {
    if constexpr (VEC == 1) {
        v[0] = load1(p);
    } else if constexpr (sizeof(T) == 4) {
        const float4 f = *reinterpret_cast<const float4 *>(p);
        v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
    } else {
        const uint4 u = *reinterpret_cast<const uint4 *>(p);
        v[0] = bf16_lo(u.x), v[1] = bf16_hi(u.x), v[2] = bf16_lo(u.y), v[3] = bf16_hi(u.y);
        v[4] = bf16_lo(u.z), v[5] = bf16_hi(u.z), v[6] = bf16_lo(u.w), v[7] = bf16_hi(u.w);
    }
}
template <int VEC, typename T>
__device__ __forceinline__ void store_vec(T *p, const float *v) {
    if constexpr (sizeof(T) == 4) {
        if constexpr (VEC == 1) *p = v[0];
        else store_nt(p, make_float4(v[0], v[1], v[2], v[3]));
    } else {
        if constexpr (VEC == 1) *p = (uint16_t)f32_to_bf16_bits(v[0]);
        else
            store_nt(p, make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                   pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])));
    }
}

// Sums of NS values over the TPR lanes of a row, in every lane of it.  Rows of more
// than a wavefront pass through LDS; `turn` alternates its halves, so that one
// barrier a sum is enough.
template <int TPR, int NS>
__device__ __forceinline__ void row_sums(float *v, float *lds, int &turn) {
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        v[i] += dpp_mov<0xB1>(v[i]);                              // quad_perm [1,0,3,2]
        v[i] += dpp_mov<0x4E>(v[i]);                              // quad_perm [2,3,0,1]
        if constexpr (TPR >= 8) v[i] += dpp_mov<0x141>(v[i]);     // row_half_mirror
        if constexpr (TPR >= 16) v[i] += dpp_mov<0x140>(v[i]);    // row_mirror
        if constexpr (TPR >= 32) v[i] += __shfl_xor(v[i], 16, 64);
        if constexpr (TPR >= 64) v[i] += __shfl_xor(v[i], 32, 64);
    }
    if constexpr (TPR > 64) {
        constexpr int W = TPR / 64;
        float *p = lds + turn * W * 2;
        if ((threadIdx.x & 63) == 0)
#pragma unroll
            for (int i = 0; i < NS; ++i) p[i * W + (threadIdx.x >> 6)] = v[i];
        lds_barrier();
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < W; ++w) s += p[i * W + w];
            v[i] = s;
        }
        turn ^= 1;
    }
}

struct NormWork {
    NormArgs a;
    int64_t S;          // channels of a group
    int64_t tokens;     // Bt T
    int64_t run;        // tokens that a lane walks
    int64_t units;      // runs x groups
};

// A lane's place: its group's channels, and its run of tokens.
template <int VEC, int VPT, int TPR>
struct Place {
    int64_t c[VPT];        // first channel of each access
    bool in[VPT];
    int64_t t0, t1;        // tokens of the run (batch and time together)
    int64_t unit;
    __device__ __forceinline__ bool find(const NormWork &w) {
        constexpr int ROWS = (TPR > 256 ? TPR : 256) / TPR;
        unit = (int64_t)blockIdx.x * ROWS + threadIdx.x / TPR;
        if (unit >= w.units) return false;
        const int64_t g = unit % w.a.groups, run = unit / w.a.groups;
        t0 = run * w.run;
        t1 = t0 + w.run < w.tokens ? t0 + w.run : w.tokens;
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int64_t i = ((int64_t)k * TPR + threadIdx.x % TPR) * VEC;
            in[k] = i < w.S;
            c[k] = g * w.S + (in[k] ? i : 0);
        }
        return true;
    }
};

// whether token t of all is one that its sequence has
__device__ __forceinline__ bool live_token(const NormArgs &a, int64_t b, int64_t t) {
    return !a.lens || t < a.lens[b];
}

template <typename T, int VEC, int VPT, int TPR, int FORM>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256) void norm_fwd_kernel(const NormWork w) {
    constexpr bool Z = FORM == SSD_NORM_GATE || FORM == SSD_NORM_GATED_INPUT;
    __shared__ float lds[4 * (TPR > 64 ? TPR / 64 : 1)];
    int turn = 0;
    const NormArgs &a = w.a;
    Place<VEC, VPT, TPR> at;
    if (!at.find(w)) return;   // whole rows leave: TPR > 64 has one row a workgroup
    float wt[VPT][VEC], bs[VPT][VEC];
#pragma unroll
    for (int k = 0; k < VPT; ++k)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            wt[k][e] = a.weight ? a.weight[at.c[k] + e] : 1.f;
            bs[k][e] = a.bias ? a.bias[at.c[k] + e] : 0.f;
        }
    const float inv_s = 1.f / (float)w.S;
    for (int64_t tok = at.t0; tok < at.t1; ++tok) {
        const int64_t b = tok / a.T, t = tok - b * a.T;
        T *y = static_cast<T *>(a.y) + tok * a.C;
        if (!live_token(a, b, t)) {
            const float none[VEC] = {};
#pragma unroll
            for (int k = 0; k < VPT; ++k)
                if (at.in[k]) store_vec<VEC>(y + at.c[k], none);
            continue;
        }
        const T *x = static_cast<const T *>(a.x) + b * a.xb + t * a.xt;
        const T *z = static_cast<const T *>(a.z) + b * a.zb + t * a.zt;
        float u[VPT][VEC], gate[VPT][VEC];
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            load_vec<VEC>(u[k], x + at.c[k]);
            if constexpr (Z) load_vec<VEC>(gate[k], z + at.c[k]);
        }
        float s[1] = {0.f};
#pragma unroll
        for (int k = 0; k < VPT; ++k)
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                if constexpr (Z) gate[k][e] *= sigm(gate[k][e]);
                if constexpr (FORM == SSD_NORM_GATED_INPUT) u[k][e] *= gate[k][e];
                if (!at.in[k]) u[k][e] = 0.f;
                s[0] += u[k][e];
            }
        float mean = 0.f;
        if (!a.rms) {
            row_sums<TPR, 1>(s, lds, turn);
            mean = s[0] * inv_s;
        }
        s[0] = 0.f;
#pragma unroll
        for (int k = 0; k < VPT; ++k)
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                u[k][e] = at.in[k] ? u[k][e] - mean : 0.f;
                s[0] += u[k][e] * u[k][e];
            }
        row_sums<TPR, 1>(s, lds, turn);
        const float rstd = rsqrtf(s[0] * inv_s + a.eps);
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            float o[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float n = u[k][e] * rstd * wt[k][e] + bs[k][e];
                o[e] = FORM == SSD_NORM_SILU   ? n * sigm(n)
                       : FORM == SSD_NORM_GATE ? n * gate[k][e]
                                               : n;
            }
            if (at.in[k]) store_vec<VEC>(y + at.c[k], o);
        }
    }
}

template <typename T, int VEC, int VPT, int TPR, int FORM>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256) void norm_bwd_kernel(const NormWork w) {
    constexpr bool Z = FORM == SSD_NORM_GATE || FORM == SSD_NORM_GATED_INPUT;
    __shared__ float lds[4 * (TPR > 64 ? TPR / 64 : 1)];
    int turn = 0;
    const NormArgs &a = w.a;
    Place<VEC, VPT, TPR> at;
    if (!at.find(w)) return;
    float wt[VPT][VEC], bs[VPT][VEC], dw[VPT][VEC], db[VPT][VEC];
#pragma unroll
    for (int k = 0; k < VPT; ++k)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            wt[k][e] = a.weight ? a.weight[at.c[k] + e] : 1.f;
            bs[k][e] = a.bias ? a.bias[at.c[k] + e] : 0.f;
            dw[k][e] = db[k][e] = 0.f;
        }
    const float inv_s = 1.f / (float)w.S;
    for (int64_t tok = at.t0; tok < at.t1; ++tok) {
        const int64_t b = tok / a.T, t = tok - b * a.T;
        T *dx = static_cast<T *>(a.dx) + tok * a.C;
        T *dz = static_cast<T *>(a.dz) + tok * a.C;
        if (!live_token(a, b, t)) {
            const float none[VEC] = {};
#pragma unroll
            for (int k = 0; k < VPT; ++k)
                if (at.in[k]) {
                    store_vec<VEC>(dx + at.c[k], none);
                    if constexpr (Z) store_vec<VEC>(dz + at.c[k], none);
                }
            continue;
        }
        const T *x = static_cast<const T *>(a.x) + b * a.xb + t * a.xt;
        const T *z = static_cast<const T *>(a.z) + b * a.zb + t * a.zt;
        const T *dy = static_cast<const T *>(a.dy) + tok * a.C;
        // c: the input, then the normalised input; d: the output's gradient, then c's
        float xv[VPT][VEC], c[VPT][VEC], zv[VPT][VEC], d[VPT][VEC];
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            load_vec<VEC>(xv[k], x + at.c[k]);
            load_vec<VEC>(d[k], dy + at.c[k]);
            if constexpr (Z) load_vec<VEC>(zv[k], z + at.c[k]);
        }
        float s[2] = {0.f, 0.f};
#pragma unroll
        for (int k = 0; k < VPT; ++k)
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                c[k][e] = xv[k][e];
                if constexpr (FORM == SSD_NORM_GATED_INPUT) c[k][e] *= zv[k][e] * sigm(zv[k][e]);
                if (!at.in[k]) c[k][e] = d[k][e] = 0.f;
                s[0] += c[k][e];
            }
        float mean = 0.f;
        if (!a.rms) {
            row_sums<TPR, 1>(s, lds, turn);
            mean = s[0] * inv_s;
        }
        s[0] = 0.f;
#pragma unroll
        for (int k = 0; k < VPT; ++k)
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                c[k][e] = at.in[k] ? c[k][e] - mean : 0.f;
                s[0] += c[k][e] * c[k][e];
            }
        row_sums<TPR, 1>(s, lds, turn);
        const float rstd = rsqrtf(s[0] * inv_s + a.eps);
        s[0] = s[1] = 0.f;
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            float gz[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                c[k][e] *= rstd;
                const float n = c[k][e] * wt[k][e] + bs[k][e];
                if constexpr (FORM == SSD_NORM_SILU) {
                    const float g = sigm(n);
                    d[k][e] *= g * (1.f + n * (1.f - g));
                } else if constexpr (FORM == SSD_NORM_GATE) {
                    const float g = sigm(zv[k][e]);
                    gz[e] = d[k][e] * n * (g * (1.f + zv[k][e] * (1.f - g)));
                    d[k][e] *= zv[k][e] * g;
                }
                dw[k][e] += d[k][e] * c[k][e];
                db[k][e] += d[k][e];
                d[k][e] *= wt[k][e];
                s[0] += d[k][e];
                s[1] += d[k][e] * c[k][e];
            }
            if constexpr (FORM == SSD_NORM_GATE)
                if (at.in[k]) store_vec<VEC>(dz + at.c[k], gz);
        }
        row_sums<TPR, 2>(s, lds, turn);
        const float md = a.rms ? 0.f : s[0] * inv_s, mc = s[1] * inv_s;
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            float o[VEC], gz[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float du = rstd * (d[k][e] - md - c[k][e] * mc);
                if constexpr (FORM == SSD_NORM_GATED_INPUT) {
                    const float g = sigm(zv[k][e]);
                    gz[e] = du * xv[k][e] * (g * (1.f + zv[k][e] * (1.f - g)));
                    o[e] = du * (zv[k][e] * g);
                } else {
                    o[e] = du;
                }
            }
            if (at.in[k]) {
                store_vec<VEC>(dx + at.c[k], o);
                if constexpr (FORM == SSD_NORM_GATED_INPUT) store_vec<VEC>(dz + at.c[k], gz);
            }
        }
    }
    // the run's sums, [run][2][C]
    if (a.part) {
        float *p = a.part + at.unit / a.groups * 2 * a.C;
#pragma unroll
        for (int k = 0; k < VPT; ++k)
            if (at.in[k])
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    if (a.dweight) p[at.c[k] + e] = dw[k][e];
                    if (a.dbias) p[a.C + at.c[k] + e] = db[k][e];
                }
    }
}

// dweight and dbias: the runs' sums in order, in double.  A workgroup takes 16 channels:
// 16 lanes read them, 4 sets of lanes of each wavefront and 16 wavefronts share the runs.
__global__ __launch_bounds__(1024) void norm_sum_kernel(const float *__restrict__ part,
                                                        int64_t runs, int64_t C,
                                                        float *__restrict__ dweight,
                                                        float *__restrict__ dbias) {
    __shared__ double sums[64][17];
    float *out = blockIdx.y ? dbias : dweight;
    if (!out) return;
    const int i = threadIdx.x >> 4, m = threadIdx.x & 15;
    const int64_t c = (int64_t)blockIdx.x * 16 + m;
    const float *p = part + blockIdx.y * C + c;
    double s = 0.0;
    if (c < C)
#pragma unroll 4
        for (int64_t r = i; r < runs; r += 64) s += (double)p[r * 2 * C];
    sums[i][m] = s;
    __syncthreads();
    if (i == 0 && c < C) {
        for (int k = 1; k < 64; ++k) s += sums[k][m];
        out[c] = (float)s;
    }
}

// How rows lie on lanes: accesses of 16 bytes where groups, strides and starts allow
// them, else of single channels; on as few lanes as hold a row in one access each (8 x 4096
// tokens of 5120 channels, bf16, gated, groups of 16, 32, 64, 256 on 16, 16, 16, 64 lanes:
// 840, 430, 236, 247 us; on 4, 4, 8, 32: 236, 195, 195, 196), a wavefront in up to two (groups
// of 1024: 262 us on a workgroup, 205), a workgroup in up to 4 (4 x 2048 tokens of 2048
// channels, gradients, 4 accesses on a wavefront: 149 us, 1 on a workgroup: 54); what is
// longer on 1024 lanes (8 x 4096 x 5120, one group, float32 gradients: 713 us with 2
// accesses, 1905 with registers for 4).  Single channels are 2 or 4 bytes a lane and leave lanes
// idle (8 x 4096 tokens, bf16, gated, 40 groups of 129 on 256 lanes each: 1035 us, one of 5121:
// 444, where groups of 128 take 210; gradients of 4 x 2048: 313, 1007 and 87).
struct NormShape {
    int vec, vpt, tpr;
};
bool aligned16(const void *p) { return !(reinterpret_cast<uintptr_t>(p) & 15u); }
NormShape shape_of(const NormArgs &a) {
    const int e = a.bf16 ? 2 : 4, v = 16 / e;
    const int64_t S = a.C / a.groups;
    const bool wide = S % v == 0 && aligned16(a.x) && aligned16(a.z) && a.xb % v == 0 &&
                      a.xt % v == 0 && (!a.z || (a.zb % v == 0 && a.zt % v == 0));
    NormShape s;
    s.vec = wide ? v : 1;
    const int64_t n = S / s.vec;
    s.tpr = n <= 4 ? 4 : n <= 8 ? 8 : n <= 16 ? 16 : n <= 32 ? 32 : n <= 128 ? 64
            : n <= 1024 ? 256 : 1024;
    const int64_t vpt = (n + s.tpr - 1) / s.tpr;
    s.vpt = vpt <= 4 ? (int)vpt : 16;
    return s;
}
// the shape with strides that do, or do not, allow wide accesses
NormShape any_shape(NormArgs a, bool wide) {
    a.x = a.z = nullptr;
    a.xb = a.xt = a.zb = a.zt = wide ? 0 : 1;
    return shape_of(a);
}
// Tokens of a lane's run: long ones load weights and leave partial sums seldom, but leave
// CUs idle.  Forward, runs as long as leaves 1024 workgroups, up to 8 (4 x 2048 tokens of
// 2048 channels, gated, whole calls: runs of 1, 4, 8, 16: 35, 22, 22, 32 us); gradients, 512
// and 32 (runs of 4, 8, 16, 32: 59, 47, 47, 70 us).
int64_t run_of(const NormArgs &a, const NormShape &s, bool bwd) {
    const int64_t rows = s.tpr >= 256 ? 1 : 256 / s.tpr;
    const int64_t blocks = a.Bt * a.T * a.groups / rows;
    const int64_t run = blocks / (bwd ? 512 : 1024), most = bwd ? 32 : 8;
    return run < 1 ? 1 : run > most ? most : run;
}

NormWork work_of(const NormArgs &a, const NormShape &s, bool bwd) {
    NormWork w;
    w.a = a;
    w.S = a.C / a.groups;
    w.tokens = a.Bt * a.T;
    w.run = run_of(a, s, bwd);
    w.units = (w.tokens + w.run - 1) / w.run * a.groups;
    return w;
}

template <typename T, int VEC, int VPT, int TPR, bool BWD>
void launch_form(const NormWork &w, hipStream_t st) {
    constexpr int threads = TPR > 256 ? TPR : 256, rows = threads / TPR;
    const uint32_t blocks = (uint32_t)((w.units + rows - 1) / rows);
#define SSD_NORM_LAUNCH(FORM)                                                        \
    do {                                                                             \
        if constexpr (BWD)                                                           \
            norm_bwd_kernel<T, VEC, VPT, TPR, FORM><<<blocks, threads, 0, st>>>(w);  \
        else                                                                         \
            norm_fwd_kernel<T, VEC, VPT, TPR, FORM><<<blocks, threads, 0, st>>>(w);  \
    } while (0)
    switch (w.a.form) {
        case SSD_NORM_PLAIN: SSD_NORM_LAUNCH(SSD_NORM_PLAIN); break;
        case SSD_NORM_SILU: SSD_NORM_LAUNCH(SSD_NORM_SILU); break;
        case SSD_NORM_GATE: SSD_NORM_LAUNCH(SSD_NORM_GATE); break;
        default: SSD_NORM_LAUNCH(SSD_NORM_GATED_INPUT); break;
    }
#undef SSD_NORM_LAUNCH
}
template <typename T, int VEC, bool BWD>
void launch_shape(const NormWork &w, const NormShape &s, hipStream_t st) {
    if (s.tpr == 4)
        launch_form<T, VEC, 1, 4, BWD>(w, st);
    else if (s.tpr == 8)
        launch_form<T, VEC, 1, 8, BWD>(w, st);
    else if (s.tpr == 16)
        launch_form<T, VEC, 1, 16, BWD>(w, st);
    else if (s.tpr == 32)
        launch_form<T, VEC, 1, 32, BWD>(w, st);
    else if (s.tpr == 64)
        s.vpt == 1 ? launch_form<T, VEC, 1, 64, BWD>(w, st)
                   : launch_form<T, VEC, 2, 64, BWD>(w, st);
    else if (s.tpr == 256) {
        switch (s.vpt) {
            case 1: launch_form<T, VEC, 1, 256, BWD>(w, st); break;
            case 2: launch_form<T, VEC, 2, 256, BWD>(w, st); break;
            case 3: launch_form<T, VEC, 3, 256, BWD>(w, st); break;
            default: launch_form<T, VEC, 4, 256, BWD>(w, st); break;
        }
    } else if (s.vpt <= 2)
        launch_form<T, VEC, 2, 1024, BWD>(w, st);
    else if constexpr (VEC < 8) {   // (8 x 2 x 1024 channels are the most)
        if (s.vpt <= 4)
            launch_form<T, VEC, 4, 1024, BWD>(w, st);
        else if constexpr (VEC == 1)
            launch_form<T, 1, 16, 1024, BWD>(w, st);
    }
}
template <bool BWD>
void launch_type(const NormWork &w, const NormShape &s, hipStream_t st) {
    if (w.a.bf16)
        s.vec == 1 ? launch_shape<uint16_t, 1, BWD>(w, s, st)
                   : launch_shape<uint16_t, 8, BWD>(w, s, st);
    else
        s.vec == 1 ? launch_shape<float, 1, BWD>(w, s, st)
                   : launch_shape<float, 4, BWD>(w, s, st);
}

}  // namespace

bool norm_fits(const NormArgs &a) {
    if ((double)a.Bt * a.T * a.groups > 1e12) return false;
    // the most workgroups of any shape, forward, whose runs are the shorter ones
    for (int vec = 0; vec < 2; ++vec) {
        const NormShape s = any_shape(a, vec);
        const int64_t rows = s.tpr >= 256 ? 1 : 256 / s.tpr, threads = s.tpr > 256 ? s.tpr : 256;
        if ((work_of(a, s, false).units + rows - 1) / rows > kMaxBlocks * 256 / threads)
            return false;
    }
    return true;
}

size_t norm_bwd_workspace(const NormArgs &a) {
    if (a.Bt == 0 || a.T == 0) return 0;
    // the most runs of any shape that the strides may lead to
    int64_t most = 0;
    for (int vec = 0; vec < 2; ++vec) {
        const int64_t run = run_of(a, any_shape(a, vec), true), n = (a.Bt * a.T + run - 1) / run;
        most = n > most ? n : most;
    }
    return (size_t)most * 2 * a.C * 4;
}

hipError_t launch_norm_fwd(const NormArgs &a, hipStream_t st) {
    const NormShape s = shape_of(a);
    launch_type<false>(work_of(a, s, false), s, st);
    return hipGetLastError();
}

hipError_t launch_norm_bwd(const NormArgs &a, hipStream_t st) {
    NormArgs b = a;
    const bool sums = a.dweight || a.dbias;
    if (!sums) b.part = nullptr;
    int64_t runs = 0;
    if (a.Bt > 0 && a.T > 0) {
        const NormShape s = shape_of(b);
        const NormWork w = work_of(b, s, true);
        runs = w.units / a.groups;
        launch_type<true>(w, s, st);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (sums)
        norm_sum_kernel<<<dim3((uint32_t)((a.C + 15) / 16), 2), 1024, 0, st>>>(
            a.part, runs, a.C, a.dweight, a.dbias);
    return hipGetLastError();
}

}  // namespace ssd
