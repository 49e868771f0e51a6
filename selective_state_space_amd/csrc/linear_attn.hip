// Linear attention with a constant decay for each head, prompts and gradients:
//     S_t = e^r S_{t-1} + k_t (outer) v_t,     y_t = scale q_t S_t,     S [K][V].
//
// One recurrence serves all of it.  Over a chunk of L tokens with the state S
// before it,
//     y_i = inter e^{r (i+1-late)} q_i S + pair sum_{j<=i} e^{r (i-j)} (q_i.k_j) v_j
//     S  <- e^{r n} S + up sum_j e^{r (n-1-j+late)} k_j (outer) v_j
// (n the chunk's tokens), and the gradients are this with the operands changed
// round, two of them backwards in time:
//     dq   q:=dy k:=v  v:=k   state S^T    forwards   inter = pair = scale
//     dk   q:=v  k:=dy v:=q   state dS^T   backwards  pair = up = scale, late
//     dv   q:=k  k:=q  v:=dy  state dS     backwards  pair = up = scale, late
// (dS_t is the adjoint that reaches token t's update, e^r dS_t what it passes on:
// the state is used before its decay, hence late = 1).  So neither states nor
// adjoints go through memory except at the ends of segments.

#include "block_launch.h"
#include "layer_launch.h"
#include "ssd_device.h"

namespace ssd {

namespace {

// e^{r n}.  r log2(e) is held in two floats, and what the product with n loses is put
// back, so that far tokens' weights are as exact as near ones' (2^x alone would be
// off by half a step of x: 1.3e-6 of e^-30).  e^-1024 is 0: rates below it count as
// it, so that 0 tokens decay by 1 at any rate, -infinity included.
struct Rate {
    float hi, lo;
    __device__ __forceinline__ explicit Rate(float r) {
        r = r < -1024.f ? -1024.f : r;
        hi = r * kLog2e;
        lo = fmaf(r, kLog2e, -hi) + r * 1.9259630e-8f;   // (what log2(e) as a float lacks)
    }
    __device__ __forceinline__ float over(int n) const {
        const float x = (float)n, p = x * hi, e = fmaf(x, lo, fmaf(x, hi, -p));
        const float v = fast_exp2(p);
        return fmaf(v * 0.6931472f, e, v);
    }
};

// One recurrence over all sequences and heads.  The roles q, k and v may be any
// of the call's tensors; `group` marks those that have G heads, not H.
struct Job {
    const void *q, *k, *v;
    int64_t qb, qt, kb, kt, vb, vt;
    void *out;                  // [Bt, T, H, dv], token stride ot, batch stride ob
    int64_t ob, ot;
    const float *s0;            // start state, element (i, j) of (b, h) at
    float *s1;                  //   ((b H + h) K V) + i rs + j cs; s1 the end state
    int32_t rs, cs;
    int32_t dk, dv;             // the state's rows and columns
    float pair, up, inter;
    bool qgroup, kgroup, vgroup;
    bool reverse;               // late, and backwards in time
    bool wide;                  // out is float32 whatever the io dtype
};
constexpr int kMaxJobs = 3;
struct Jobs {
    Job job[kMaxJobs];
    const float *decay;
    const int32_t *lens;
    int64_t T, seg_tokens, seg_stride;   // seg_stride: elements between segments' states in s0, s1
    int32_t H, G, nseg, njobs, slices, state_size;
};

// Matrix operands.  A wavefront's operand register holds, for row (or column)
// lane % 16, kRun contraction indices from kRun (lane / 16); the accumulator of
// a 16 x 16 tile holds rows 4 (lane / 16) + 0..3 of column lane % 16.
template <typename T>
struct Mat;
template <>
struct Mat<uint16_t> {
    static constexpr int kChunk = 64;    // tokens of a chunk
    static constexpr int kDepth = 32;    // contraction indices of one operand
    static constexpr int kRun = 8;
    typedef bf16x8 Frag;
    // 4 consecutive rows (tokens) of one column: lanes 4 i + j of a 16-lane group
    // give the address of columns 4 j.. of row i, lane l receives column l
    static __device__ __forceinline__ u32x2 cols4(const uint16_t *p) {
        typedef short s16x4 __attribute__((ext_vector_type(4)));
        typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
        return __builtin_bit_cast(
            u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)const_cast<uint16_t *>(p)));
    }
    static __device__ __forceinline__ f32x4 mma(Frag a, Frag b, f32x4 c) {
        return mfma16x16x32(a, b, c);
    }
};
template <>
struct Mat<float> {
    static constexpr int kChunk = 32;
    static constexpr int kDepth = 16;
    static constexpr int kRun = 4;
    typedef f32x4 Frag;
    static __device__ __forceinline__ f32x4 mma(Frag a, Frag b, f32x4 c) {
#pragma unroll
        for (int r = 0; r < 4; ++r)
            c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[r], b[r], c, 0, 0, 0);
        return c;
    }
};

// Operands out of row-major tiles in LDS.  natural(): rows r0.. are the operand's
// rows, contraction along the tile's columns from c0.
template <typename T>
__device__ __forceinline__ typename Mat<T>::Frag natural(const T *tile, int stride, int r0, int c0,
                                                         int lane) {
    const T *p = tile + (r0 + (lane & 15)) * stride + c0 + Mat<T>::kRun * (lane >> 4);
    return *reinterpret_cast<const typename Mat<T>::Frag *>(p);
}
// across(): contraction along the tile's rows from r0; the operand's row m is
// column c0 + step * (m / 4) + m % 4.
template <int STEP>
__device__ __forceinline__ bf16x8 across(const uint16_t *tile, int stride, int r0, int c0,
                                         int lane) {
    const uint16_t *p = tile + (r0 + 8 * (lane >> 4) + ((lane & 15) >> 2)) * stride + c0 +
                        STEP * (lane & 3);
    const u32x2 lo = Mat<uint16_t>::cols4(p), hi = Mat<uint16_t>::cols4(p + 4 * stride);
    return as_bf16x8(make_uint4(lo[0], lo[1], hi[0], hi[1]));
}
template <int STEP>
__device__ __forceinline__ f32x4 across(const float *tile, int stride, int r0, int c0, int lane) {
    const int m = lane & 15;
    const float *p = tile + (r0 + 4 * (lane >> 4)) * stride + c0 + STEP * (m >> 2) + (m & 3);
    f32x4 v;
#pragma unroll
    for (int r = 0; r < 4; ++r) v[r] = p[r * stride];
    return v;
}

// The row of the state that accumulator row m of tile t holds: so chosen that the
// tiles of one contraction step hold kRun consecutive rows per lane, as natural()
// reads q.
template <typename T>
__device__ __forceinline__ int state_row(int t, int m) {
    if constexpr (sizeof(T) == 2) return 32 * (t >> 1) + 8 * (m >> 2) + 4 * (t & 1) + (m & 3);
    else return 16 * t + m;
}
// k across its tokens, as the operand whose rows are those of state tile t
template <typename T>
__device__ __forceinline__ typename Mat<T>::Frag state_cols(const T *tile, int stride, int r0,
                                                            int t, int lane) {
    if constexpr (sizeof(T) == 2)
        return across<8>(tile, stride, r0, 32 * (t >> 1) + 4 * (t & 1), lane);
    else
        return across<4>(tile, stride, r0, 16 * t, lane);
}

__device__ __forceinline__ float frag_at(bf16x8 f, int e) {
    return bf16_to_f32((uint16_t)f[e]);
}

// S += (k across) (w v): for bf16 the weighted v is split into three bf16 terms,
// v w = hi + mid + lo to 2^-24, so that the state keeps float32's precision at
// three matrix instructions for one; the single rounding that one term would take
// (2^-8 of each product) would stay in the state for as long as it lives.
template <int N>
struct Weighted {
    bf16x8 t[N];
};
__device__ __forceinline__ Weighted<3> weighted(bf16x8 v, const float *w) {
    Weighted<3> r;
    uint32_t hi[4], mid[4], lo[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        float a = frag_at(v, 2 * e) * w[2 * e], b = frag_at(v, 2 * e + 1) * w[2 * e + 1];
        hi[e] = pack_bf16x2(a, b);
        a -= bf16_lo(hi[e]);
        b -= bf16_hi(hi[e]);
        mid[e] = pack_bf16x2(a, b);
        lo[e] = pack_bf16x2(a - bf16_lo(mid[e]), b - bf16_hi(mid[e]));
    }
    r.t[0] = as_bf16x8(make_uint4(hi[0], hi[1], hi[2], hi[3]));
    r.t[1] = as_bf16x8(make_uint4(mid[0], mid[1], mid[2], mid[3]));
    r.t[2] = as_bf16x8(make_uint4(lo[0], lo[1], lo[2], lo[3]));
    return r;
}
__device__ __forceinline__ f32x4 weighted(f32x4 v, const float *w) {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] *= w[e];
    return v;
}
__device__ __forceinline__ f32x4 mma_weighted(bf16x8 a, const Weighted<3> &b, f32x4 c) {
    c = mfma16x16x32(a, b.t[2], c);
    c = mfma16x16x32(a, b.t[1], c);
    return mfma16x16x32(a, b.t[0], c);
}
__device__ __forceinline__ f32x4 mma_weighted(f32x4 a, f32x4 b, f32x4 c) {
    return Mat<float>::mma(a, b, c);
}

// The state as an operand of q S: rounded to bf16 for bf16 calls (2^-8 of each
// term, as y itself is rounded).
template <int NT>
__device__ __forceinline__ bf16x8 state_frag(const f32x4 (&s)[NT], int ks, uint16_t) {
    const f32x4 a = s[2 * ks], b = s[2 * ks + 1];
    return as_bf16x8(make_uint4(pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]),
                                pack_bf16x2(b[0], b[1]), pack_bf16x2(b[2], b[3])));
}
template <int NT>
__device__ __forceinline__ f32x4 state_frag(const f32x4 (&s)[NT], int ks, float) {
    return s[ks];
}

__device__ __forceinline__ void put4(uint16_t *p, f32x4 v) {
    *reinterpret_cast<uint2 *>(p) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
}
__device__ __forceinline__ void put4(float *p, f32x4 v) { *reinterpret_cast<f32x4 *>(p) = v; }

// A tile of tokens on its way from memory to LDS: 16-byte pieces, row by row.
template <typename T, int COLS>
struct Tile {
    static constexpr int kVec = 16 / sizeof(T);
    static constexpr int kPerRow = COLS / kVec;
    static constexpr int kPieces = Mat<T>::kChunk * kPerRow / 256;
    static constexpr int kStride = COLS + kVec;     // of a row in LDS
    static constexpr int kSize = Mat<T>::kChunk * kStride;
    uint4 v[kPieces];
    // rows [0, n) at base + row * stride, columns [0, cols); zeros elsewhere
    __device__ __forceinline__ void load(const T *base, int64_t stride, int n, int cols) {
#pragma unroll
        for (int p = 0; p < kPieces; ++p) {
            const int x = threadIdx.x + 256 * p, row = x / kPerRow, c = x % kPerRow * kVec;
            v[p] = make_uint4(0, 0, 0, 0);
            if (row < n && c < cols)
                v[p] = *reinterpret_cast<const uint4 *>(base + row * stride + c);
        }
    }
    __device__ __forceinline__ void keep(T *lds) const {
#pragma unroll
        for (int p = 0; p < kPieces; ++p) {
            const int x = threadIdx.x + 256 * p, row = x / kPerRow, c = x % kPerRow * kVec;
            *reinterpret_cast<uint4 *>(lds + row * kStride + c) = v[p];
        }
    }
};

// One workgroup walks the chunks of one segment of one sequence and head, for 64 NV
// columns of the state, which stay in accumulators; a wavefront owns 16 NV columns.
// OUT = false: only the state at the segment's end, from zero.
template <typename T, int KD, int NV, bool OUT>
__global__ __launch_bounds__(256) void attn_kernel(const Jobs a) {
    typedef Mat<T> M;
    typedef typename M::Frag Frag;
    constexpr int L = M::kChunk, LT = L / 16, VS = 64 * NV;
    constexpr int NT = KD / 16, KS = KD / M::kDepth, NB = L / M::kDepth;
    constexpr int PS = L + 16 / sizeof(T);
    typedef Tile<T, KD> KTile;
    typedef Tile<T, VS> VTile;
    __shared__ __align__(16) T ks[KTile::kSize];
    __shared__ __align__(16) T vs[VTile::kSize];
    __shared__ __align__(16) T qs[OUT ? KTile::kSize : 1];
    __shared__ __align__(16) T ps[OUT ? L * PS : 1];

    // consecutive ids share an XCD, and the tokens that they read
    uint32_t id = xcd_remap(blockIdx.x, gridDim.x);
    const int slice = id % a.slices;
    id /= a.slices;
    const Job &job = a.job[id % a.njobs];
    id /= a.njobs;
    const int nbh = gridDim.x / (a.slices * a.njobs * a.nseg);
    const int bh = id % nbh, seg = id / nbh;
    const int b = bh / a.H, h = bh % a.H, hg = h / (a.H / a.G);
    const int v0 = slice * VS;
    if (v0 >= job.dv) return;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int m = lane & 15, q4 = 4 * (lane >> 4);
    const int late = job.reverse ? 1 : 0;
    const Rate rate(a.decay[h]);

    const int64_t r0 = seg * a.seg_tokens;
    const int64_t r1 = a.T < r0 + a.seg_tokens ? a.T : r0 + a.seg_tokens;
    int64_t len = a.T;
    if (a.lens) {
        const int64_t n = a.lens[b];
        len = n < 0 ? 0 : n < len ? n : len;
    }
    // token r of the walk lies at first + r step
    const int64_t first = job.reverse ? len - 1 : 0, step = job.reverse ? -1 : 1;
    const T *qp = static_cast<const T *>(job.q) + b * job.qb + first * job.qt +
                  (job.qgroup ? hg : h) * job.dk;
    const T *kp = static_cast<const T *>(job.k) + b * job.kb + first * job.kt +
                  (job.kgroup ? hg : h) * job.dk;
    const T *vp = static_cast<const T *>(job.v) + b * job.vb + first * job.vt +
                  (job.vgroup ? hg : h) * job.dv + v0;
    const int64_t qst = step * job.qt, kst = step * job.kt, vst = step * job.vt;

    f32x4 s[NV][NT];
    const int64_t sbase = (int64_t)bh * a.state_size + seg * a.seg_stride;
    const bool given = OUT && job.s0;
#pragma unroll
    for (int nt = 0; nt < NV; ++nt)
#pragma unroll
        for (int t = 0; t < NT; ++t) s[nt][t] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (given) {
#pragma unroll
        for (int nt = 0; nt < NV; ++nt) {
            const int col = v0 + 16 * (NV * wave + nt) + m;
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int row = state_row<T>(t, q4 + r);
                    if (row < job.dk && col < job.dv)
                        s[nt][t][r] = job.s0[sbase + row * job.rs + col * job.cs];
                }
        }
    }

    float out_decay[LT], w[NB][M::kRun];
    if constexpr (OUT) {
#pragma unroll
        for (int it = 0; it < LT; ++it)
            out_decay[it] = job.inter * rate.over(16 * it + m + 1 - late);
        // (pairs of a later key stay zero: no tile above the diagonal is written)
        for (int x = threadIdx.x; x < L * PS; x += 256) ps[x] = 0;
    }
    auto weights = [&](int n) {   // of an update by n tokens
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int e = 0; e < M::kRun; ++e) {
                const int j = M::kDepth * nb + M::kRun * (lane >> 4) + e;
                w[nb][e] = j < n ? job.up * rate.over(n - 1 - j + late) : 0.f;
            }
    };
    weights(L);
    float turn = rate.over(L);

    auto tokens = [&](int64_t r) {   // of the chunk at r that the sequence has
        const int64_t n = (len < r1 ? len : r1) - r;
        return (int)(n < 0 ? 0 : n < L ? n : L);
    };
    KTile qt, kt;
    VTile vt;
    auto fetch = [&](int64_t r) {
        const int n = tokens(r);
        if constexpr (OUT) qt.load(qp + r * qst, qst, n, job.dk);
        kt.load(kp + r * kst, kst, n, job.dk);
        vt.load(vp + r * vst, vst, n, job.dv - v0);
    };
    auto put = [&](int64_t t, int col, f32x4 v) {   // 4 columns of the output at token t
        const int64_t at = b * job.ob + t * job.ot + (int64_t)h * job.dv + col;
        if (sizeof(T) == 4 || job.wide)
            put4(static_cast<float *>(job.out) + at, v);
        else
            put4(static_cast<uint16_t *>(job.out) + at, v);
    };

    bool live = given;
    fetch(r0);
    for (int64_t r = r0; r < r1; r += L) {
        const int n = tokens(r);
        const bool more = r + L < r1;
        const int rows = (int)(r1 - r < L ? r1 - r : L);
        lds_barrier();
        if constexpr (OUT) qt.keep(qs);
        kt.keep(ks);
        vt.keep(vs);
        if (more) fetch(r + L);
        lds_barrier();
        if constexpr (OUT) {
            // pairs: tiles (token i, key j <= i), shared by the wavefronts in turn
            int tile = 0;
#pragma unroll
            for (int it = 0; it < LT; ++it)
#pragma unroll
                for (int jt = 0; jt <= it; ++jt, ++tile) {
                    if ((tile & 3) != wave || 16 * it >= n) continue;
                    f32x4 p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int k = 0; k < KS; ++k)
                        p = M::mma(natural<T>(ks, KTile::kStride, 16 * jt, M::kDepth * k, lane),
                                   natural<T>(qs, KTile::kStride, 16 * it, M::kDepth * k, lane),
                                   p);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int gap = 16 * (it - jt) + m - (q4 + e);
                        p[e] = gap < 0 ? 0.f : p[e] * (job.pair * rate.over(gap));
                    }
                    put4(ps + (16 * it + m) * PS + 16 * jt + q4, p);
                }
            lds_barrier();
        }
        Frag vf[NB][NV];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int nt = 0; nt < NV; ++nt)
                vf[nb][nt] = across<4>(vs, VTile::kStride, M::kDepth * nb,
                                       16 * (NV * wave + nt), lane);
        if constexpr (OUT) {
            f32x4 o[LT][NV];
#pragma unroll
            for (int it = 0; it < LT; ++it)
#pragma unroll
                for (int nt = 0; nt < NV; ++nt) o[it][nt] = f32x4{0.f, 0.f, 0.f, 0.f};
            if (live) {
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    Frag sf[NV];
#pragma unroll
                    for (int nt = 0; nt < NV; ++nt) sf[nt] = state_frag(s[nt], k, T(0));
#pragma unroll
                    for (int it = 0; it < LT; ++it) {
                        const Frag qf = natural<T>(qs, KTile::kStride, 16 * it, M::kDepth * k,
                                                   lane);
#pragma unroll
                        for (int nt = 0; nt < NV; ++nt)
                            o[it][nt] = M::mma(sf[nt], qf, o[it][nt]);
                    }
                }
#pragma unroll
                for (int it = 0; it < LT; ++it)
#pragma unroll
                    for (int nt = 0; nt < NV; ++nt) o[it][nt] *= out_decay[it];
            }
#pragma unroll
            for (int it = 0; it < LT; ++it)
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                    if (M::kDepth * nb > 16 * it) continue;
                    const Frag pf = natural<T>(ps, PS, 16 * it, M::kDepth * nb, lane);
#pragma unroll
                    for (int nt = 0; nt < NV; ++nt) o[it][nt] = M::mma(vf[nb][nt], pf, o[it][nt]);
                }
#pragma unroll
            for (int it = 0; it < LT; ++it) {
                const int i = 16 * it + m;
                const int64_t t = i < n ? first + step * (r + i) : r + i;
#pragma unroll
                for (int nt = 0; nt < NV; ++nt) {
                    const int col = v0 + 16 * (NV * wave + nt) + q4;
                    if (i < rows && col < job.dv)
                        put(t, col, i < n ? o[it][nt] : f32x4{0.f, 0.f, 0.f, 0.f});
                }
            }
        }
        if (n > 0 && (more || job.s1)) {
            if (n < L) {
                weights(n);
                turn = rate.over(n);
            }
#pragma unroll
            for (int nt = 0; nt < NV; ++nt)
#pragma unroll
                for (int t = 0; t < NT; ++t) s[nt][t] *= turn;
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                decltype(weighted(Frag(), w[0])) wv[NV];
#pragma unroll
                for (int nt = 0; nt < NV; ++nt) wv[nt] = weighted(vf[nb][nt], w[nb]);
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const Frag kf = state_cols<T>(ks, KTile::kStride, M::kDepth * nb, t, lane);
#pragma unroll
                    for (int nt = 0; nt < NV; ++nt) s[nt][t] = mma_weighted(kf, wv[nt], s[nt][t]);
                }
            }
            live = true;
        }
    }
    if (job.s1) {
#pragma unroll
        for (int nt = 0; nt < NV; ++nt) {
            const int col = v0 + 16 * (NV * wave + nt) + m;
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int row = state_row<T>(t, q4 + e);
                    if (row < job.dk && col < job.dv)
                        job.s1[sbase + row * job.rs + col * job.cs] = s[nt][t][e];
                }
        }
    }
}

// The states before each segment from the segments' own ends (in place), and the
// state behind the last: four elements of one (b, h) per lane, segments in order.
struct Chain {
    float *seg;                // [nseg][Bt H][K V]
    const float *start;        // [Bt H][K V] or NULL
    float *end;                // [Bt H][K V] or NULL: then the last segment's end is not read
};
struct Chains {
    Chain c[2];
    const float *decay;
    const int32_t *lens;
    int64_t T, seg_tokens, seg_stride;
    int32_t H, nseg, state_size, blocks;   // blocks: workgroups per (b, h)
};
__global__ __launch_bounds__(256) void attn_chain_kernel(const Chains a) {
    const int bh = blockIdx.x / a.blocks;
    const int e = (blockIdx.x % a.blocks * 256 + threadIdx.x) * 4;
    if (e >= a.state_size) return;
    const Chain c = a.c[blockIdx.y];
    const Rate rate(a.decay[bh % a.H]);
    int64_t len = a.T;
    if (a.lens) {
        const int64_t n = a.lens[bh / a.H];
        len = n < 0 ? 0 : n < len ? n : len;
    }
    const int64_t at = (int64_t)bh * a.state_size + e;
    f32x4 cur = {0.f, 0.f, 0.f, 0.f};
    if (c.start) cur = *reinterpret_cast<const f32x4 *>(c.start + at);
    for (int sg = 0; sg < a.nseg; ++sg) {
        float *p = c.seg + sg * a.seg_stride + at;
        int64_t n = len - sg * a.seg_tokens;
        n = n < 0 ? 0 : n < a.seg_tokens ? n : a.seg_tokens;
        f32x4 own = {0.f, 0.f, 0.f, 0.f};
        if (sg + 1 < a.nseg || c.end) own = *reinterpret_cast<const f32x4 *>(p);
        *reinterpret_cast<f32x4 *>(p) = cur;
        const float d = rate.over((int)n);
        cur = d * cur + own;
    }
    if (c.end) *reinterpret_cast<f32x4 *>(c.end + at) = cur;
}

// Sums of float32 rows over the heads that share a key or value head, four columns a
// lane, heads in order.
template <typename T>
__global__ __launch_bounds__(256) void attn_share_kernel(const float *__restrict__ part,
                                                         T *__restrict__ out, int64_t n4, int dim4,
                                                         int G, int rep) {
    const int64_t x = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (x >= n4) return;
    const int64_t row = x / dim4;            // (token, group)
    const int c = (int)(x % dim4);
    const f32x4 *p = reinterpret_cast<const f32x4 *>(part) + row * rep * dim4 + c;
    f32x4 v = p[0];
    for (int i = 1; i < rep; ++i) v += p[(int64_t)i * dim4];
    put4(out + 4 * x, v);
}

int pad_dim(int d) { return d <= 64 ? 64 : d <= 128 ? 128 : 256; }

template <typename T, int KD, int NV>
void launch_jobs_t(const Jobs &j, bool out, uint32_t blocks, hipStream_t st) {
    if (out)
        attn_kernel<T, KD, NV, true><<<blocks, 256, 0, st>>>(j);
    else
        attn_kernel<T, KD, NV, false><<<blocks, 256, 0, st>>>(j);
}
template <typename T>
void launch_jobs_kd(int kd, int nv, const Jobs &j, bool out, uint32_t blocks, hipStream_t st) {
    if (kd == 64)
        nv == 2 ? launch_jobs_t<T, 64, 2>(j, out, blocks, st)
                : launch_jobs_t<T, 64, 1>(j, out, blocks, st);
    else if (kd == 128)
        nv == 2 ? launch_jobs_t<T, 128, 2>(j, out, blocks, st)
                : launch_jobs_t<T, 128, 1>(j, out, blocks, st);
    else
        launch_jobs_t<T, 256, 1>(j, out, blocks, st);
}

// Launches all jobs, those of one padded row count together.
hipError_t launch_jobs(const AttnArgs &a, const Jobs &all, bool out, int v_cols, hipStream_t st) {
    for (int kd = 64; kd <= 256; kd *= 2) {
        Jobs j = all;
        j.njobs = 0;
        int dv = 0;
        for (int i = 0; i < all.njobs; ++i)
            if (pad_dim(all.job[i].dk) == kd) {
                j.job[j.njobs++] = all.job[i];
                dv = all.job[i].dv > dv ? all.job[i].dv : dv;
            }
        if (!j.njobs) continue;
        const int nv = kd == 256 ? 1 : v_cols / 64;
        j.slices = (dv + 64 * nv - 1) / (64 * nv);
        const uint32_t blocks = (uint32_t)(a.Bt * a.H * j.njobs * j.slices * j.nseg);
        if (a.bf16)
            launch_jobs_kd<uint16_t>(kd, nv, j, out, blocks, st);
        else
            launch_jobs_kd<float>(kd, nv, j, out, blocks, st);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

Jobs jobs_of(const AttnArgs &a, const AttnLayout &l) {
    Jobs j{};
    j.decay = a.decay;
    j.lens = a.lens;
    j.T = a.T;
    j.seg_tokens = l.seg_tokens;
    j.H = (int32_t)a.H;
    j.G = (int32_t)a.G;
    j.nseg = (int32_t)l.segments;
    j.state_size = a.K * a.V;
    return j;
}

Job fwd_job(const AttnArgs &a) {
    Job j{};
    j.q = a.q;
    j.k = a.k;
    j.v = a.v;
    j.qb = a.qb, j.qt = a.qt, j.kb = a.kb, j.kt = a.kt, j.vb = a.vb, j.vt = a.vt;
    j.out = a.y;
    j.ot = a.H * a.V;
    j.ob = a.T * j.ot;
    j.s0 = a.init;
    j.s1 = a.fin;
    j.rs = a.V;
    j.cs = 1;
    j.dk = a.K;
    j.dv = a.V;
    j.kgroup = j.vgroup = true;
    j.pair = j.inter = a.scale;
    j.up = 1.f;
    return j;
}

size_t state_floats(const AttnArgs &a) { return (size_t)(a.Bt * a.H) * a.K * a.V; }

AttnLayout layout_of(const AttnArgs &a, int jobs) {
    AttnLayout l;
    l.v_cols = 64;
    const int64_t wide = a.K > a.V ? a.K : a.V;
    const int64_t groups = a.Bt * a.H * jobs * ((jobs > 1 ? wide : a.V) + 63) / 64;
    int64_t seg = groups ? (512 + groups - 1) / groups : 1;
    const int64_t most = a.T / 512;
    seg = seg < most ? seg : most;
    seg = seg < 1 ? 1 : seg;
    l.seg_tokens = (a.T + seg - 1) / seg;
    l.seg_tokens = (l.seg_tokens + 63) / 64 * 64;
    l.segments = l.seg_tokens ? (a.T + l.seg_tokens - 1) / l.seg_tokens : 1;
    if (l.segments < 1) l.segments = 1;
    return l;
}

hipError_t launch_chain(const AttnArgs &a, const AttnLayout &l, const Chain *c, int n,
                        hipStream_t st) {
    Chains x{};
    for (int i = 0; i < n; ++i) x.c[i] = c[i];
    x.decay = a.decay;
    x.lens = a.lens;
    x.T = a.T;
    x.seg_tokens = l.seg_tokens;
    x.seg_stride = (int64_t)state_floats(a);
    x.H = (int32_t)a.H;
    x.nseg = (int32_t)l.segments;
    x.state_size = a.K * a.V;
    x.blocks = (x.state_size + 1023) / 1024;
    attn_chain_kernel<<<dim3((uint32_t)(a.Bt * a.H * x.blocks), n), 256, 0, st>>>(x);
    return hipGetLastError();
}

template <typename T>
void launch_share_t(const float *part, void *out, int64_t rows, int dim, int64_t G, int rep,
                    hipStream_t st) {
    const int64_t n4 = rows * (dim / 4);
    attn_share_kernel<T><<<(uint32_t)((n4 + 255) / 256), 256, 0, st>>>(
        part, static_cast<T *>(out), n4, dim / 4, (int)G, rep);
}

}  // namespace

AttnLayout attn_layout(const AttnArgs &a) { return layout_of(a, 1); }
AttnLayout attn_bwd_layout(const AttnArgs &a) { return layout_of(a, 3); }

bool attn_fits(const AttnArgs &a) {
    const double heads = (double)a.Bt * (double)a.H, wide = a.K > a.V ? a.K : a.V;
    // the most workgroups of the recurrences (3 jobs, 4 slices; segments only while
    // there are fewer than 512), of the chains, and of the shared heads' sums
    return heads * 12 + 1024 <= (double)kMaxBlocks && heads * 64 <= (double)kMaxBlocks &&
           (double)a.Bt * a.T * a.G * (wide / 1024) + 1 <= (double)kMaxBlocks;
}

size_t attn_workspace(const AttnArgs &a) {
    const AttnLayout l = attn_layout(a);
    return l.segments > 1 ? l.segments * state_floats(a) * 4 : 0;
}

size_t attn_bwd_workspace(const AttnArgs &a) {
    const AttnLayout l = attn_bwd_layout(a);
    size_t n = l.segments > 1 ? 2 * l.segments * state_floats(a) * 4 : 0;
    if (a.G < a.H) n += (size_t)(a.Bt * a.T * a.H) * (a.K + a.V) * 4;
    return n;
}

hipError_t launch_attn_fwd(const AttnArgs &a, hipStream_t st) {
    const AttnLayout l = attn_layout(a);
    Jobs j = jobs_of(a, l);
    j.job[0] = fwd_job(a);
    j.njobs = 1;
    if (l.segments > 1) {
        float *seg = static_cast<float *>(a.ws);
        j.seg_stride = (int64_t)state_floats(a);
        Jobs s = j;
        s.job[0].s1 = seg;
        hipError_t e = launch_jobs(a, s, false, l.v_cols, st);
        if (e != hipSuccess) return e;
        const Chain c = {seg, a.init, a.fin};
        if ((e = launch_chain(a, l, &c, 1, st)) != hipSuccess) return e;
        j.job[0].s0 = seg;
        j.job[0].s1 = nullptr;
    }
    return launch_jobs(a, j, true, l.v_cols, st);
}

hipError_t launch_attn_bwd(const AttnArgs &a, hipStream_t st) {
    const AttnLayout l = attn_bwd_layout(a);
    const bool shared = a.G < a.H;
    const int64_t states = l.segments > 1 ? l.segments * (int64_t)state_floats(a) : 0;
    float *hseg = static_cast<float *>(a.ws), *dseg = hseg + states, *part = dseg + states;
    float *pk = part, *pv = part + a.Bt * a.T * a.H * a.K;
    const int64_t yt = a.H * a.V, yb = a.T * yt;

    Job dq{}, dk{}, dv{};
    dq.q = a.dy, dq.qb = yb, dq.qt = yt;
    dq.k = a.v, dq.kb = a.vb, dq.kt = a.vt, dq.kgroup = true;
    dq.v = a.k, dq.vb = a.kb, dq.vt = a.kt, dq.vgroup = true;
    dq.out = a.dq, dq.ot = a.H * a.K;
    dq.dk = a.V, dq.dv = a.K;
    dq.s0 = a.init, dq.rs = 1, dq.cs = a.V;
    dq.pair = dq.inter = a.scale, dq.up = 1.f;

    dk.q = a.v, dk.qb = a.vb, dk.qt = a.vt, dk.qgroup = true;
    dk.k = a.dy, dk.kb = yb, dk.kt = yt;
    dk.v = a.q, dk.vb = a.qb, dk.vt = a.qt;
    dk.out = shared ? (void *)pk : a.dk, dk.ot = a.H * a.K;
    dk.dk = a.V, dk.dv = a.K;
    dk.s0 = a.dfinal, dk.rs = 1, dk.cs = a.V;

    dv.q = a.k, dv.qb = a.kb, dv.qt = a.kt, dv.qgroup = true;
    dv.k = a.q, dv.kb = a.qb, dv.kt = a.qt;
    dv.v = a.dy, dv.vb = yb, dv.vt = yt;
    dv.out = shared ? (void *)pv : a.dv, dv.ot = a.H * a.V;
    dv.dk = a.K, dv.dv = a.V;
    dv.s0 = a.dfinal, dv.s1 = a.dinit, dv.rs = a.V, dv.cs = 1;
    for (Job *j : {&dk, &dv}) {
        j->pair = j->up = a.scale;
        j->inter = 1.f;
        j->reverse = true;
        j->wide = shared;
    }
    for (Job *j : {&dq, &dk, &dv}) j->ob = a.T * j->ot;

    Jobs j = jobs_of(a, l);
    hipError_t e;
    if (l.segments > 1) {
        j.seg_stride = (int64_t)state_floats(a);
        Jobs s = j;
        s.job[0] = fwd_job(a);
        s.job[0].s1 = hseg;
        s.job[1] = dv;
        s.job[1].s1 = dseg;
        s.njobs = 2;
        if ((e = launch_jobs(a, s, false, l.v_cols, st)) != hipSuccess) return e;
        const Chain c[2] = {{hseg, a.init, nullptr}, {dseg, a.dfinal, a.dinit}};
        if ((e = launch_chain(a, l, c, 2, st)) != hipSuccess) return e;
        dq.s0 = hseg;
        dk.s0 = dv.s0 = dseg;
        dv.s1 = nullptr;
    }
    j.job[0] = dq;
    j.job[1] = dk;
    j.job[2] = dv;
    j.njobs = 3;
    if ((e = launch_jobs(a, j, true, l.v_cols, st)) != hipSuccess || !shared ||
        a.T == 0)
        return e;
    const int rep = (int)(a.H / a.G);
    const int64_t rows = a.Bt * a.T * a.G;
    if (a.bf16) {
        launch_share_t<uint16_t>(pk, a.dk, rows, a.K, a.G, rep, st);
        launch_share_t<uint16_t>(pv, a.dv, rows, a.V, a.G, rep, st);
    } else {
        launch_share_t<float>(pk, a.dk, rows, a.K, a.G, rep, st);
        launch_share_t<float>(pv, a.dv, rows, a.V, a.G, rep, st);
    }
    return hipGetLastError();
}

// ---------------------------------------------------------------------------
namespace {

// One token: S <- e^r S + k (outer) v, y = scale q S, for states in a slot pool.
// The state goes through memory once in each direction, which bounds it.  A
// workgroup serves one (b, h): LPR lanes cover a row of the state with 16-byte
// accesses, so 256 / LPR rows are in flight per access, kBatch accesses before
// the first is used; a lane's four columns are summed over its rows in
// registers and over the workgroup's rows through LDS, in a fixed order.
template <typename T, int LPR>
__global__ __launch_bounds__(256) void attn_step_kernel(const AttnArgs a) {
    constexpr int RPI = 256 / LPR;     // rows per access of the workgroup
    constexpr int kBatch = 4;
    __shared__ __align__(16) float4 part[256];
    const int64_t bh = blockIdx.x;
    const int64_t b = bh / a.H;
    const int h = (int)(bh % a.H), hg = h / (int)(a.H / a.G);
    const int sub = threadIdx.x % LPR, rw = threadIdx.x / LPR;
    const int64_t slot = a.slots ? (int64_t)a.slots[b] : b;
    const int col = 4 * sub;
    T *y = static_cast<T *>(a.y) + bh * a.V + col;
    if (slot < 0 || slot >= a.nslots) {
        if (rw == 0 && col < a.V) put4(y, f32x4{0.f, 0.f, 0.f, 0.f});
        return;
    }
    const T *q = static_cast<const T *>(a.q) + b * a.qb + (int64_t)h * a.K;
    const T *k = static_cast<const T *>(a.k) + b * a.kb + (int64_t)hg * a.K;
    const T *v = static_cast<const T *>(a.v) + b * a.vb + (int64_t)hg * a.V;
    const float d = Rate(a.decay[h]).over(1);
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    if (col < a.V) {
        const float4 vv = load4(v + col);
        float *st = a.state + (slot * a.H + h) * (int64_t)(a.K * a.V) + col;
        for (int r0 = rw; r0 < a.K; r0 += kBatch * RPI) {
            float4 s[kBatch];
            float kk[kBatch], qq[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int row = r0 + i * RPI;
                s[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                kk[i] = qq[i] = 0.f;
                if (row < a.K) {
                    s[i] = load_nt(st + (int64_t)row * a.V);
                    kk[i] = load1(k + row);
                    qq[i] = load1(q + row);
                }
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int row = r0 + i * RPI;
                float4 n;
                n.x = d * s[i].x + kk[i] * vv.x;
                n.y = d * s[i].y + kk[i] * vv.y;
                n.z = d * s[i].z + kk[i] * vv.z;
                n.w = d * s[i].w + kk[i] * vv.w;
                sum.x += qq[i] * n.x;
                sum.y += qq[i] * n.y;
                sum.z += qq[i] * n.z;
                sum.w += qq[i] * n.w;
                if (row < a.K) store_nt(st + (int64_t)row * a.V, n);
            }
        }
    }
    part[threadIdx.x] = sum;
    __syncthreads();
    if (threadIdx.x < LPR && col < a.V) {
        float4 o = part[threadIdx.x];
#pragma unroll
        for (int i = 1; i < RPI; ++i) {
            const float4 p = part[threadIdx.x + i * LPR];
            o.x += p.x;
            o.y += p.y;
            o.z += p.z;
            o.w += p.w;
        }
        put4(y, f32x4{o.x * a.scale, o.y * a.scale, o.z * a.scale, o.w * a.scale});
    }
}

template <typename T>
void launch_step_t(const AttnArgs &a, hipStream_t st) {
    const uint32_t blocks = (uint32_t)(a.Bt * a.H);
    if (a.V <= 32)
        attn_step_kernel<T, 8><<<blocks, 256, 0, st>>>(a);
    else if (a.V <= 64)
        attn_step_kernel<T, 16><<<blocks, 256, 0, st>>>(a);
    else if (a.V <= 128)
        attn_step_kernel<T, 32><<<blocks, 256, 0, st>>>(a);
    else
        attn_step_kernel<T, 64><<<blocks, 256, 0, st>>>(a);
}

}  // namespace

hipError_t launch_attn_step(const AttnArgs &a, hipStream_t st) {
    if (a.bf16)
        launch_step_t<uint16_t>(a, st);
    else
        launch_step_t<float>(a, st);
    return hipGetLastError();
}

}  // namespace ssd
