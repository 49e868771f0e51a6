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
//
// Per 16 columns of a bf16 state of 128 rows a chunk of 32 tokens takes 44 matrix
// instructions of 16 x 16 x 32 and each wavefront 16 more for the pairs; bytes bound it
// below (8 x 4096 tokens of 40 heads of 128: 1.34 GB, 280 us at a copy's rate).  Reached:
// 414 us there (3.3 TB/s; matrix instructions 28% of the cycles, vector ones 41%), 128
// sequences and heads of 4096 tokens 181 (3.0 TB/s), 1 x 65536 tokens of 16 heads, in two
// passes, 454; gradients of 4 x 2048 tokens of 16 heads 131 (235 MB, 49 at a copy's rate).
// What bounds it is that a wavefront's chunk is a chain (operands out of LDS, products,
// splitting, products): with two wavefronts a SIMD the time of a chunk, 4500 cycles in those
// gradients, is about the sum of what both issue (350 vector instructions of 4 cycles, 60
// matrix ones of 16).  The long one's outputs pass comes near a copy's rate as well (4.8 TB/s):
// its two slices of 64 columns read q and k 1.6 times.  Tried with bf16 and slower, while
// operands were one term and 8 x 4096 took 390: chunks of 64 tokens through registers (636),
// eight wavefronts of 16 columns (405), pairs shared through LDS behind a second barrier
// (437), interleaving by hand (425 of 422 then), three workgroups a CU (1140, spills); since,
// for 121 in the gradients: the terms' difference by matrix instructions (118 to 120, but 188
// for 129 with 128 columns), by dot products (126), accumulators of its own for lo (129).
// None of it was tried with float32.

#include <float.h>

#include "block_launch.h"
#include "layer_launch.h"
#include "ssd_device.h"

namespace ssd {

namespace {

// Rates below -1024 count as it: e^-1024 is 0, and 0 tokens decay by 1 at any rate,
// -infinity included.
__device__ __forceinline__ float least_rate(float r) { return r < -1024.f ? -1024.f : r; }

// e^{r n}.  r log2(e) is held in two floats, and what the product with n loses is put
// back, so that far tokens' weights are as exact as near ones' (2^x alone would be
// off by half a step of x: 1.3e-6 of e^-30).
struct Rate {
    float hi, lo;
    __device__ __forceinline__ explicit Rate(float r) {
        r = least_rate(r);
        hi = r * kLog2e;
        lo = fmaf(r, kLog2e, -hi) + r * 1.9259630e-8f;   // (what log2(e) as a float lacks)
    }
    __device__ __forceinline__ float over(int n) const {
        const float x = (float)n, p = x * hi, e = fmaf(x, lo, fmaf(x, hi, -p));
        const float v = fast_exp2(p);
        return fmaf(v * 0.6931472f, e, v);
    }
};

// The factors by which one state is multiplied over and over, e^{r n} each time.  One float
// for all of them would be off by the same 2^-25 every time, which adds up: over 65536 tokens
// at r = -3e-6 the start state would weigh 5.7e-5 too much.  So what each factor leaves is
// put into the next one, and the product of any number of them is off by half a step.  (The
// exponential is taken in double, once a walk.)
struct Turn {
    float whole, less, by, left;   // e^{r n} as a float, what it lacks, 1 / whole; still owed
    __device__ __forceinline__ Turn(float r, int64_t n) {
        const double e = exp((double)least_rate(r) * (double)n);
        whole = (float)e;
        const bool held = whole > 0x1p-100f && whole < 0x1p100f;   // (else all is forgotten)
        by = held ? 1.f / whole : 0.f;
        less = held ? (float)(e - (double)whole) * by : 0.f;
        left = 0.f;
    }
    __device__ __forceinline__ float next() {
        left += less;
        const float f = fmaf(whole, left, whole);
        left -= (f - whole) * by;
        return f;
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
    bool wide;                  // out is float32 whatever the io dtype (kOutWide)
};
constexpr int kMaxJobs = 3;
struct Jobs {
    Job job[kMaxJobs];
    const float *decay;
    const int32_t *lens;
    int64_t T, seg_tokens, seg_stride;   // seg_stride: elements between segments' states in s0, s1
    int32_t H, G, nseg, njobs, slices, state_size;
};

constexpr int kChunk = 32;   // tokens of a chunk

// Matrix operands.  A wavefront's operand register holds, for row (or column)
// lane % 16, kRun contraction indices from kRun (lane / 16); the accumulator of
// a 16 x 16 tile holds rows 4 (lane / 16) + 0..3 of column lane % 16.
template <typename T>
struct Mat;
template <>
struct Mat<uint16_t> {
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

// A tile of tokens in LDS: rows of COLS elements without a gap, their 16-byte pieces
// in an order of the row's own (piece p at p ^ order(row)), so chosen that both ways of
// reading below find their 16 lanes on 16 different banks' groups.  (Rows one piece
// longer instead cost 5.0e7 conflict cycles of 9.0e7 in all, at 8 x 4096 tokens of 40
// heads of 128.)
template <typename T, int COLS>
struct Lds {
    static constexpr int kVec = 16 / sizeof(T);
    static constexpr int kPerRow = COLS / kVec;
    static constexpr int kSize = kChunk * COLS;
    static __device__ __forceinline__ int order(int row) {
        if constexpr (sizeof(T) == 4) return row & 15;
        else if constexpr (kPerRow == 8) return (row << 1 & 4) | (row >> 2 & 3);
        else return (row << 2 & 12) | (row >> 2 & 3);
    }
};

// Operands out of such tiles.  natural(): row `row` for the operand's row lane % 16,
// contraction along the tile's columns from c0 (a multiple of kDepth).
template <typename T, int COLS>
__device__ __forceinline__ typename Mat<T>::Frag natural(const T *tile, int row, int c0, int lane) {
    typedef Lds<T, COLS> S;
    const int piece = (lane >> 4) ^ S::order(row) ^ (c0 / S::kVec);
    return *reinterpret_cast<const typename Mat<T>::Frag *>(tile + row * COLS + piece * S::kVec);
}
// across(): contraction along the tile's rows from r0; the operand's row m is column
// c0 + STEP (m / 4) + m % 4.
template <int COLS, int STEP>
__device__ __forceinline__ bf16x8 across(const uint16_t *tile, int r0, int c0, int lane) {
    typedef Lds<uint16_t, COLS> S;
    const int row = 8 * (lane >> 4) + (lane >> 2 & 3), c = c0 + STEP * (lane & 3);
    auto at = [&](int r) {
        return tile + (r0 + r) * COLS + ((c >> 3) ^ S::order(r)) * 8 + (c & 4);
    };
    const u32x2 lo = Mat<uint16_t>::cols4(at(row)), hi = Mat<uint16_t>::cols4(at(row + 4));
    return as_bf16x8(make_uint4(lo[0], lo[1], hi[0], hi[1]));
}
template <int COLS, int STEP>
__device__ __forceinline__ f32x4 across(const float *tile, int r0, int c0, int lane) {
    typedef Lds<float, COLS> S;
    const int m = lane & 15, c = c0 + STEP * (m >> 2) + (m & 3);
    f32x4 v;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int row = r0 + 4 * (lane >> 4) + e;
        v[e] = tile[row * COLS + ((c >> 2) ^ S::order(row)) * 4 + (c & 3)];
    }
    return v;
}

// Single elements of such tiles: the product of two rows, four columns of one.
template <typename T, int COLS>
__device__ __forceinline__ f32x4 row4(const T *tile, int row, int c) {
    typedef Lds<T, COLS> S;
    const T *p = tile + row * COLS + ((c / S::kVec) ^ S::order(row)) * S::kVec + c % S::kVec;
    if constexpr (sizeof(T) == 4) {
        return *reinterpret_cast<const f32x4 *>(p);
    } else {
        const u32x2 u = *reinterpret_cast<const u32x2 *>(p);
        return f32x4{bf16_lo(u[0]), bf16_hi(u[0]), bf16_lo(u[1]), bf16_hi(u[1])};
    }
}
template <typename T, int COLS>
__device__ __forceinline__ float dot_rows(const T *a, int i, const T *b, int j) {
    float s = 0.f;
#pragma unroll 1
    for (int c = 0; c < COLS; c += 4) {
        const f32x4 x = row4<T, COLS>(a, i, c), y = row4<T, COLS>(b, j, c);
        for (int e = 0; e < 4; ++e) s = fmaf(x[e], y[e], s);
    }
    return s;
}

// What accumulator row m of tile t stands for where the accumulators become an operand
// themselves (the state's rows; the keys of a chunk's pairs): so chosen that the tiles
// of one contraction step hold kRun consecutive ones per lane, as the other operand
// has them.
template <typename T>
__device__ __forceinline__ int tile_row(int t, int m) {
    if constexpr (sizeof(T) == 2) return 32 * (t >> 1) + 8 * (m >> 2) + 4 * (t & 1) + (m & 3);
    else return 16 * t + m;
}
// k across its tokens, as the operand whose rows are those of state tile t
template <typename T, int COLS>
__device__ __forceinline__ typename Mat<T>::Frag state_cols(const T *tile, int r0, int t,
                                                            int lane) {
    if constexpr (sizeof(T) == 2)
        return across<COLS, 8>(tile, r0, 32 * (t >> 1) + 4 * (t & 1), lane);
    else
        return across<COLS, 4>(tile, r0, 16 * t, lane);
}

__device__ __forceinline__ float frag_at(bf16x8 f, int e) {
    return bf16_to_f32((uint16_t)f[e]);
}

// S += (k across) (w v): for bf16 the weighted v is split into three bf16 terms,
// v w = hi + mid + lo to 2^-22, so that the state keeps float32's precision at
// three matrix instructions for one; the single rounding that one term would take
// (2^-8 of each product) would stay in the state for as long as it lives.  hi and
// mid are cut, not rounded (their packing is one byte permutation), lo is rounded.
template <int N>
struct Weighted {
    bf16x8 t[N];
};
__device__ __forceinline__ Weighted<3> weighted(bf16x8 v, const float *w) {
    Weighted<3> r;
    uint32_t hi[4], mid[4], lo[4];
    auto top = [](float f) { return __uint_as_float(__float_as_uint(f) & 0xffff0000u); };
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        float a = frag_at(v, 2 * e) * w[2 * e], b = frag_at(v, 2 * e + 1) * w[2 * e + 1];
        hi[e] = pair_hi(__float_as_uint(a), __float_as_uint(b));
        a -= top(a);
        b -= top(b);
        mid[e] = pair_hi(__float_as_uint(a), __float_as_uint(b));
        lo[e] = pack_bf16x2(a - top(a), b - top(b));
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

// Accumulators as an operand (the state against q, the pairs' weights against the values):
// for bf16 two terms, hi cut and lo rounded, which leave at most 2^-15 of each element, so that an
// output is rounded to bf16 once, where it is stored.  (One term, 2^-8 of each element twice
// over, was 0.0023 of the outputs' norm off where that one rounding is 0.0017, at, us with one
// term and with two: 8 x 4096 tokens of 40 heads of 128 396 and 436, 1 x 65536 of 16 406 and
// 438, gradients of 4 x 2048 of 16 100 and 121.)
struct Halves {
    bf16x8 hi, lo;
};
template <int NT>
__device__ __forceinline__ Halves tile_frag(const f32x4 (&s)[NT], int k, uint16_t) {
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const f32x4 t = s[2 * k + (i >> 1)];
        const float a = t[2 * i & 3], b = t[(2 * i & 3) + 1];
        hi[i] = pair_hi(__float_as_uint(a), __float_as_uint(b));
        lo[i] = pack_bf16x2(a - bf16_hi(__float_as_uint(a)), b - bf16_hi(__float_as_uint(b)));
    }
    return {as_bf16x8(make_uint4(hi[0], hi[1], hi[2], hi[3])),
            as_bf16x8(make_uint4(lo[0], lo[1], lo[2], lo[3]))};
}
template <int NT>
__device__ __forceinline__ f32x4 tile_frag(const f32x4 (&s)[NT], int k, float) {
    return s[k];
}
__device__ __forceinline__ f32x4 mma_halves(const Halves &a, bf16x8 b, f32x4 c) {
    return mfma16x16x32(a.hi, b, mfma16x16x32(a.lo, b, c));
}
__device__ __forceinline__ f32x4 mma_halves(bf16x8 a, const Halves &b, f32x4 c) {
    return mfma16x16x32(a, b.hi, mfma16x16x32(a, b.lo, c));
}
__device__ __forceinline__ f32x4 mma_halves(f32x4 a, f32x4 b, f32x4 c) {
    return Mat<float>::mma(a, b, c);
}

__device__ __forceinline__ f32x4 f4(const float *v) { return f32x4{v[0], v[1], v[2], v[3]}; }

__device__ __forceinline__ void put4(uint16_t *p, f32x4 v) {
    *reinterpret_cast<uint2 *>(p) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
}
__device__ __forceinline__ void put4(float *p, f32x4 v) { *reinterpret_cast<f32x4 *>(p) = v; }

// A chunk's rows of one tensor, loaded from memory into LDS directly, 16 bytes a lane
// (a wavefront's 64 pieces lie in LDS as its lanes do, so the order within a row is
// made by which piece a lane loads).  Rows past the chunk's tokens and columns past
// the tensor's arrive as zeros: their lanes' offsets lie outside the buffer.
template <typename T, int COLS>
struct Tile {
    typedef Lds<T, COLS> S;
    static constexpr int kVec = S::kVec, kPerRow = S::kPerRow, kSize = S::kSize;
    static constexpr int kPieces = kChunk * kPerRow / 256;    // loads of a lane
    static_assert(kChunk * kPerRow % 256 == 0, "whole wavefronts");
    static constexpr uint32_t kNowhere = 0xffffffffu;
    const T *base;        // of the next chunk to be loaded
    int64_t turn;         // elements from one chunk to the next
    uint32_t at[kPieces]; // byte offsets of this lane's pieces
    static __device__ __forceinline__ int row(int p) { return (threadIdx.x + 256 * p) / kPerRow; }
    // p: the walk's first token; step +1 or -1 tokens of `stride` elements
    __device__ __forceinline__ void start(const T *p, int64_t stride, bool reverse, int cols) {
        base = reverse ? p - (kChunk - 1) * stride : p;
        turn = reverse ? -kChunk * stride : kChunk * stride;
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int r = reverse ? kChunk - 1 - row(i) : row(i);
            const int col = ((threadIdx.x + 256 * i) % kPerRow ^ S::order(row(i))) * kVec;
            at[i] = col < cols ? (uint32_t)((r * (uint64_t)stride + col) * sizeof(T)) : kNowhere;
        }
    }
    // rows [0, n) of the next chunk
    __device__ __forceinline__ void load(T *lds, int n, int wave) {
#ifdef __HIP_DEVICE_COMPILE__   // (16 bytes a lane are gfx950's: not known to the host's pass)
        typedef __attribute__((address_space(3))) T lds_t;
        const __amdgpu_buffer_rsrc_t rs = make_rsrc(base, 0xfffffff0u);
        base += turn;
#pragma unroll
        for (int i = 0; i < kPieces; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                rs, (lds_t *)(lds + (256 * i + 64 * wave) * kVec), 16,
                row(i) < n ? at[i] : kNowhere, 0, 0, 0);
#endif
    }
};

// at most N of the wavefront's vector memory accesses are still on their way
template <int N>
__device__ __forceinline__ void wait_vmcnt() {
    static_assert(N < 64, "");
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

template <bool B>
struct Const {
    static constexpr bool value = B;
};

// One workgroup walks the chunks of one segment of one sequence and head, for 16 NV
// columns of the state per wavefront, which stay in accumulators.  OUT = false:
// only the state at the segment's end, from zero.
//
// A chunk's tiles are loaded into LDS kAhead chunks before the walk comes to it, so
// that a load has kAhead chunks' time; one barrier a chunk lets the buffers turn.  Each
// wavefront forms the chunk's pairs for itself (16 of its 60 matrix instructions with 16
// columns, of 104 with 32): shared through LDS they need a second barrier, and a wait for it.
// Whole chunks run through one block of code whose only branch is the one for tokens that
// are not finite, in which matrix and vector instructions interleave.
enum Mode { kStateOnly, kOut, kOutWide };

template <typename T, int KD, int NV, int MODE>
__global__ __launch_bounds__(256, 2) void attn_kernel(const Jobs a) {
    typedef Mat<T> M;
    typedef typename M::Frag Frag;
    constexpr bool OUT = MODE != kStateOnly;
    constexpr int L = kChunk, LT = L / 16, VS = 64 * NV;
    constexpr int NT = KD / 16, KS = KD / M::kDepth, NB = L / M::kDepth;
    constexpr uint32_t kNowhere = 0xffffffffu;
    typedef Tile<T, KD> KTile;
    typedef Tile<T, VS> VTile;
    // (three buffers of 256 columns leave a CU one workgroup, or do not fit)
    constexpr int kAhead = KD == 256 ? 1 : 2, NBUF = kAhead + 1;
    // (separate variables: so the compiler sees that reads of one buffer need not wait for
    // loads into another)
    constexpr int kK = OUT ? KTile::kSize : 0, kV = kK + KTile::kSize, kAll = kV + VTile::kSize;
    __shared__ __align__(16) T tiles0[kAll];
    __shared__ __align__(16) T tiles1[kAll];
    __shared__ __align__(16) T tiles2[NBUF == 3 ? kAll : 8];
    auto tiles = [&](int buf) -> T * { return buf == 0 ? tiles0 : buf == 1 ? tiles1 : tiles2; };
    __shared__ __align__(16) float ws[2][L];    // weights of a whole and of a cut chunk

    // consecutive ids share an XCD, and the tokens that they read
    uint32_t id = xcd_remap(blockIdx.x, gridDim.x);
    const int slice = id % a.slices;
    id /= a.slices;
    const Job job = a.job[id % a.njobs];
    id /= a.njobs;
    const int nbh = gridDim.x / (a.slices * a.njobs * a.nseg);
    const int bh = id % nbh, seg = id / nbh;
    const int b = bh / a.H, h = bh % a.H, hg = h / (a.H / a.G);
    const int v0 = slice * VS;
    if (v0 >= job.dv) return;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
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
    const int64_t t0 = first + step * r0;
    KTile qt, kt;
    VTile vt;
    if constexpr (OUT)
        qt.start(static_cast<const T *>(job.q) + b * job.qb + t0 * job.qt +
                     (job.qgroup ? hg : h) * job.dk, job.qt, job.reverse, job.dk);
    kt.start(static_cast<const T *>(job.k) + b * job.kb + t0 * job.kt +
                 (job.kgroup ? hg : h) * job.dk, job.kt, job.reverse, job.dk);
    vt.start(static_cast<const T *>(job.v) + b * job.vb + t0 * job.vt +
                 (job.vgroup ? hg : h) * job.dv + v0, job.vt, job.reverse, job.dv - v0);
    // the sequence's tokens in this segment: whole chunks and a cut one
    const int64_t own = (len < r1 ? len : r1) - r0;
    const int tokens = own < 0 ? 0 : (int)own, whole = tokens / L, cut = tokens % L;
    int left = tokens;   // not yet on their way
    auto fetch = [&](int buf) {
        const int n = left < L ? left : L;
        T *to = tiles(buf);
        if constexpr (OUT) qt.load(to, n, wave);
        kt.load(to + kK, n, wave);
        vt.load(to + kV, n, wave);
        left -= n;
    };

    const int vcol = v0 + 16 * NV * wave;    // the wavefront's first column
    f32x4 s[NV][NT];
    const int64_t sbase = (int64_t)bh * a.state_size + seg * a.seg_stride;
    // byte offset of element e of tile t in a state
    auto place = [&](int v, int t, int e) {
        const int row = tile_row<T>(t, q4 + e), col = vcol + 16 * v + m;
        return row < job.dk && col < job.dv ? 4u * (row * job.rs + col * job.cs) : kNowhere;
    };
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int t = 0; t < NT; ++t) s[v][t] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (OUT && job.s0) {
        const __amdgpu_buffer_rsrc_t rs = make_rsrc(job.s0 + sbase, 4 * a.state_size);
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    s[v][t][e] = __uint_as_float(
                        __builtin_amdgcn_raw_buffer_load_b32(rs, place(v, t, e), 0, 0));
    }

    // outputs: a lane has 4 columns of one token of each tile
    const bool wide = sizeof(T) == 4 || (MODE == kOutWide && job.wide);
    const uint32_t osize = wide ? 4 : 2;
    char *out = static_cast<char *>(job.out) +
                (b * job.ob + (t0 - (job.reverse ? L - 1 : 0)) * job.ot + (int64_t)h * job.dv +
                 vcol) * (int64_t)osize;      // of the chunk's lowest token
    const int64_t out_turn = step * L * job.ot * (int64_t)osize;
    uint32_t out_at[NV][LT];
    float out_decay[LT], pair_decay[LT][LT][4];
    if constexpr (OUT) {
#pragma unroll
        for (int it = 0; it < LT; ++it) {
            out_decay[it] = job.inter * rate.over(16 * it + m + 1 - late);
            const int i = job.reverse ? L - 1 - 16 * it - m : 16 * it + m;
#pragma unroll
            for (int v = 0; v < NV; ++v)
                out_at[v][it] = vcol + 16 * v + q4 < job.dv
                                    ? (uint32_t)(i * job.ot + 16 * v + q4) * osize : kNowhere;
        }
#pragma unroll
        for (int it = 0; it < LT; ++it)
#pragma unroll
            for (int jt = 0; jt < LT; ++jt)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int gap = 16 * it + m - tile_row<T>(jt, q4 + e);
                    pair_decay[it][jt][e] = gap < 0 ? 0.f : job.pair * rate.over(gap);
                }
    }
    auto put = [&](const __amdgpu_buffer_rsrc_t &rs, uint32_t at, f32x4 v) {
        if (wide)
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), rs, at, 0, 0);
        else
            __builtin_amdgcn_raw_buffer_store_b64(
                u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])}, rs, at, 0, 0);
    };
    if (threadIdx.x < 2 * L) {
        const int j = threadIdx.x % L, n = threadIdx.x < L ? L : cut;
        ws[threadIdx.x / L][j] = j < n ? job.up * rate.over(n - 1 - j + late) : 0.f;
    }
    Turn turns(a.decay[h], L);

    // The next chunk's tiles have arrived, for all wavefronts, and this one's are free.
    // Behind the next one's loads at least the later chunks' loads and this chunk's stores
    // have been issued, and may still be on their way.
    auto turn_buffers = [&](bool stored) {
        constexpr int loads = (OUT ? KTile::kPieces : 0) + KTile::kPieces + VTile::kPieces;
        constexpr int later = (kAhead - 1) * loads, stores = OUT ? NV * LT : 0;
        __builtin_amdgcn_sched_barrier(0);
        if (stored) wait_vmcnt<later + stores>();
        else wait_vmcnt<later>();
        lds_barrier();
    };
    // one chunk, whole or (the last) cut
    auto chunk = [&](int buf, auto flag) {
        constexpr bool WHOLE = decltype(flag)::value;
        if constexpr (WHOLE) {
            fetch(buf + kAhead < NBUF ? buf + kAhead : buf + kAhead - NBUF);
            __builtin_amdgcn_sched_barrier(0);   // (left alone, the loads sink to the chunk's end)
        }
        const T *qc = tiles(buf), *kc = qc + kK, *vc = qc + kV;
        Frag vf[NV][NB];
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
                vf[v][nb] = across<VS, 4>(vc, M::kDepth * nb, 16 * (NV * wave + v), lane);
        if constexpr (OUT) {
            f32x4 o[NV][LT], y[NV][LT];   // of the state, and with the chunk's own tokens
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int it = 0; it < LT; ++it) o[v][it] = f32x4{0.f, 0.f, 0.f, 0.f};
            f32x4 p[LT][LT];    // weights of pairs: query tile, key tile
#pragma unroll
            for (int it = 0; it < LT; ++it)
#pragma unroll
                for (int jt = 0; jt < LT; ++jt) p[it][jt] = f32x4{0.f, 0.f, 0.f, 0.f};
            // (a step's operands are read one step ahead: left alone, the reads sink to where
            // they are used, 126 us for 121 in gradients of 4 x 2048 tokens of 16 heads of 128)
            Frag qs[2][LT], ks[2][LT];
            auto read = [&](int k) {
#pragma unroll
                for (int it = 0; it < LT; ++it) {
                    qs[k & 1][it] = natural<T, KD>(qc, 16 * it + m, M::kDepth * k, lane);
                    ks[k & 1][it] = natural<T, KD>(kc, tile_row<T>(it, m), M::kDepth * k, lane);
                }
                __builtin_amdgcn_sched_barrier(0);
            };
            read(0);
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                if (k + 1 < KS) read(k + 1);
                const Frag(&qf)[LT] = qs[k & 1], (&kf)[LT] = ks[k & 1];
#pragma unroll
                for (int it = 0; it < LT; ++it)
#pragma unroll
                    for (int jt = 0; jt < LT; ++jt)
                        if (sizeof(T) == 2 || jt <= it)
                            p[it][jt] = M::mma(kf[jt], qf[it], p[it][jt]);
#pragma unroll
                for (int v = 0; v < NV; ++v) {
                    const auto sf = tile_frag(s[v], k, T(0));
#pragma unroll
                    for (int it = 0; it < LT; ++it) o[v][it] = mma_halves(sf, qf[it], o[v][it]);
                }
            }
#pragma unroll
            for (int it = 0; it < LT; ++it) {
#pragma unroll
                for (int jt = 0; jt < LT; ++jt) p[it][jt] *= f4(pair_decay[it][jt]);
#pragma unroll
                for (int v = 0; v < NV; ++v) {
                    o[v][it] *= out_decay[it];
                    y[v][it] = o[v][it];
                }
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                    if (M::kDepth * nb > 16 * it) continue;
                    const auto pf = tile_frag(p[it], nb, T(0));
#pragma unroll
                    for (int v = 0; v < NV; ++v) y[v][it] = mma_halves(vf[v][nb], pf, y[v][it]);
                }
            }
            // A token's masked pairs are weights of 0, which an infinity or a NaN in a later
            // key or value turns into NaN: of the tokens that share a contraction with it
            // the first has it masked, and shows it.
            float bad = 0.f;
#pragma unroll
            for (int it = 0; it < LT; it += M::kDepth / 16)
#pragma unroll
                for (int v = 0; v < NV; ++v)
#pragma unroll
                    for (int e = 0; e < 4; ++e) bad = fmaf(y[v][it][e], 0.f, bad);
            if (__builtin_expect(__ballot(!(bad == 0.f)) != 0, 0)) {
                bool lost = false;     // what the state alone does not make of it
#pragma unroll
                for (int it = 0; it < LT; ++it)
#pragma unroll
                    for (int v = 0; v < NV; ++v)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            lost |= !(y[v][it][e] * 0.f == 0.f) && o[v][it][e] * 0.f == 0.f;
                if (__ballot(lost)) {
#pragma unroll
                    for (int it = 0; it < LT; ++it) {
#pragma unroll
                        for (int v = 0; v < NV; ++v) y[v][it] = o[v][it];
                        const int i = 16 * it + m;
#pragma unroll 1
                        for (int j = 0; j <= i; ++j) {
                            const float w =
                                dot_rows<T, KD>(qc, i, kc, j) * job.pair * rate.over(i - j);
#pragma unroll
                            for (int v = 0; v < NV; ++v)
                                y[v][it] += w * row4<T, VS>(vc, j, 16 * (NV * wave + v) + q4);
                        }
                    }
                }
            }
            const __amdgpu_buffer_rsrc_t rs = make_rsrc(out, 0xfffffff0u);
#pragma unroll
            for (int it = 0; it < LT; ++it)
#pragma unroll
                for (int v = 0; v < NV; ++v)
                    put(rs, WHOLE || 16 * it + m < cut ? out_at[v][it] : kNowhere, y[v][it]);
            out += out_turn;
        }
        if (WHOLE || job.s1) {
            const float turn = WHOLE ? turns.next() : rate.over(cut);
            const float *w = ws[!WHOLE] + M::kRun * (lane >> 4);
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int t = 0; t < NT; ++t) s[v][t] *= turn;
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                decltype(weighted(Frag(), w)) wv[NV];
#pragma unroll
                for (int v = 0; v < NV; ++v) wv[v] = weighted(vf[v][nb], w + M::kDepth * nb);
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const Frag kf = state_cols<T, KD>(kc, M::kDepth * nb, t, lane);
#pragma unroll
                    for (int v = 0; v < NV; ++v) s[v][t] = mma_weighted(kf, wv[v], s[v][t]);
                }
            }
        }
        if constexpr (WHOLE) {
            turn_buffers(true);
        }
    };
    if (tokens > 0) {
        // (chunks past the last read as zeros)
#pragma unroll
        for (int i = 0; i < kAhead; ++i) fetch(i);
        turn_buffers(false);
        int c = 0;
        for (; c + NBUF <= whole; c += NBUF)
#pragma unroll
            for (int i = 0; i < NBUF; ++i) chunk(i, Const<true>());
        int buf = 0;
        for (; c < whole; ++c, ++buf) chunk(buf, Const<true>());
        if (cut) chunk(buf, Const<false>());
    }
    if constexpr (OUT)   // zeros behind the sequence
        for (int64_t t = r0 + tokens; t < r1; t += L) {
            const __amdgpu_buffer_rsrc_t rs = make_rsrc(
                static_cast<char *>(job.out) +
                    (b * job.ob + t * job.ot + (int64_t)h * job.dv + vcol) * (int64_t)osize,
                0xfffffff0u);
#pragma unroll
            for (int it = 0; it < LT; ++it)
#pragma unroll
                for (int v = 0; v < NV; ++v)
                    put(rs, t + 16 * it + m < r1 && out_at[v][it] != kNowhere
                                ? (uint32_t)((16 * it + m) * job.ot + 16 * v + q4) * osize
                                : kNowhere,
                        f32x4{0.f, 0.f, 0.f, 0.f});
        }
    // (with outputs, s1 is the state behind the last segment)
    if (job.s1 && (!OUT || seg == a.nseg - 1)) {
        const __amdgpu_buffer_rsrc_t rs = make_rsrc(
            job.s1 + (OUT ? (int64_t)bh * a.state_size : sbase), 4 * a.state_size);
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(s[v][t][e]), rs,
                                                          place(v, t, e), 0, 0);
    }
}

// The states before each segment from the segments' own ends (in place; the last one's
// end is not among them): four elements of one (b, h) per lane, segments in order.
struct Chain {
    float *seg;                // [nseg][Bt H][K V]
    const float *start;        // [Bt H][K V] or NULL
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
    Turn turns(a.decay[bh % a.H], a.seg_tokens);
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
        if (sg + 1 < a.nseg) own = *reinterpret_cast<const f32x4 *>(p);
        *reinterpret_cast<f32x4 *>(p) = cur;
        cur = (n == a.seg_tokens ? turns.next() : rate.over((int)n)) * cur + own;
    }
}

// Sums of float32 rows over the heads that share a key or value head, four columns a
// lane, heads in order; dk and dv in one launch.
struct Share {
    const float *part[2];
    void *out[2];
    int64_t n4[2];
    int32_t dim4[2];
    int32_t rep;
};
template <typename T>
__global__ __launch_bounds__(256) void attn_share_kernel(const Share a) {
    const int w = blockIdx.y, dim4 = a.dim4[w];
    for (int64_t x = (int64_t)blockIdx.x * 256 + threadIdx.x; x < a.n4[w];
         x += (int64_t)gridDim.x * 256) {
        const int64_t row = x / dim4;            // (token, group)
        const f32x4 *p =
            reinterpret_cast<const f32x4 *>(a.part[w]) + row * a.rep * dim4 + x % dim4;
        f32x4 v = p[0];
        for (int i = 1; i < a.rep; ++i) v += p[(int64_t)i * dim4];
        put4(static_cast<T *>(a.out[w]) + 4 * x, v);
    }
}

int pad_dim(int d) { return d <= 64 ? 64 : d <= 128 ? 128 : 256; }

template <typename T, int KD>
void launch_jobs_t(const Jobs &j, Mode mode, uint32_t blocks, hipStream_t st) {
    if (mode == kStateOnly)
        attn_kernel<T, KD, 1, kStateOnly><<<blocks, 256, 0, st>>>(j);
    else if (mode == kOut || sizeof(T) == 4)
        attn_kernel<T, KD, 1, kOut><<<blocks, 256, 0, st>>>(j);
    else if constexpr (sizeof(T) == 2)
        attn_kernel<T, KD, 1, kOutWide><<<blocks, 256, 0, st>>>(j);
}
// (sequences are not cut where 128 columns are taken, nor are those taken by bf16's shared
// heads: layout_of)
template <typename T>
void launch_jobs_kd(int kd, int cols, const Jobs &j, Mode mode, uint32_t blocks, hipStream_t st) {
    if (kd == 256)
        launch_jobs_t<T, 256>(j, mode, blocks, st);
    else if (kd == 128)
        cols == 128 ? attn_kernel<T, 128, 2, kOut><<<blocks, 256, 0, st>>>(j)
                    : launch_jobs_t<T, 128>(j, mode, blocks, st);
    else
        cols == 128 ? attn_kernel<T, 64, 2, kOut><<<blocks, 256, 0, st>>>(j)
                    : launch_jobs_t<T, 64>(j, mode, blocks, st);
}

// Launches all jobs, those of one padded row count together; all of them where they do not
// fill the chip, since then the launches' times add up and the padding costs nothing
// (gradients of 2 x 333 tokens, 6 heads of 64 and 96, float32: 95 us in two launches).
hipError_t launch_jobs(const AttnArgs &a, const Jobs &all, bool out, int v_cols, hipStream_t st) {
    int widest = 0, most = 0;
    for (int i = 0; i < all.njobs; ++i) {
        widest = all.job[i].dk > widest ? all.job[i].dk : widest;
        most = all.job[i].dv > most ? all.job[i].dv : most;
    }
    const bool together = a.Bt * a.H * all.njobs * all.nseg * ((most + 63) / 64) <= 256;
    for (int kd = 64; kd <= 256; kd *= 2) {
        Jobs j = all;
        j.njobs = 0;
        int dv = 0;
        Mode mode = out ? kOut : kStateOnly;
        for (int i = 0; i < all.njobs; ++i)
            if (pad_dim(together ? widest : all.job[i].dk) == kd) {
                j.job[j.njobs++] = all.job[i];
                dv = all.job[i].dv > dv ? all.job[i].dv : dv;
                if (out && all.job[i].wide) mode = kOutWide;
            }
        if (!j.njobs) continue;
        const int cols = kd == 256 ? 64 : v_cols;
        j.slices = (dv + cols - 1) / cols;
        const uint32_t blocks = (uint32_t)(a.Bt * a.H * j.njobs * j.slices * j.nseg);
        if (a.bf16)
            launch_jobs_kd<uint16_t>(kd, cols, j, mode, blocks, st);
        else
            launch_jobs_kd<float>(kd, cols, j, mode, blocks, st);
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

// 64 or 128 columns a workgroup: 128 form the pairs half as often, 64 make twice the
// workgroups.  (us with 64 and 128, bf16, heads of 128, by sequences times heads.)  64 up to
// 128 of those (4096 tokens of 128: 180, 254; 2048 of 132: 126, 126), 128 above (2048 tokens of
// 160: 132, 126; 192: 135, 129; 224: 145, 144; 4096 of 192: 267, 253; float32, 1024 of 160:
// 327, 241), in bf16 also where the chip holds them twice over and more (4096 of 260: 393, 379;
// 320: 464, 410; 512: 614, 521; 1024: 1219, 1028; 1024 of 260: 109, 110; 512: 161, 139), with
// 64 state rows, whose pairs cost less, from 384 on (2048 of 320: 159, 166; 448: 202, 181).
// States of more than 128 rows have registers for 64 only; bf16 gradients take them too (192
// workgroups of the three recurrences: 122, 122; 216: 127, 124; float32, 192: 323, 229).
// Segments, three or more, where at most half the CUs would have a workgroup, though keys
// and values are read and the states formed twice.  bf16: up to two workgroups a CU, of 256
// tokens or more (1 x 65536 tokens of 16 heads: 1, 4, 8, 16, 32 segments 2412, 892, 532,
// 452, 456 us; 1 x 2048: 1, 4, 8, 16: 81, 45, 35, 38; 1 x 512 of 8 heads, 1 and 2: 24 and 28;
// 4 sequences of 32 heads, 256 workgroups, 1, 2, 4: 180, 205, 221; gradients of 4 x 2048 tokens
// of 16 heads, 384 workgroups, 1 to 4: 121, 137, 151, 147, of 2 x 4096 153, 168, 168, 146).
// float32, whose matrix instructions take 16 times as long: 64 tokens (2 x 256 of 4 heads, 1,
// 2, 4 segments: 45, 42, 28; 2 x 160 of 6 heads of 64, 1 and 2: 17 and 20), and one workgroup
// a CU, since LDS holds no more, unless that makes fewer than three (1 x 2048 of 16 heads, 8
// and 16: 77 and 84; gradients, 1, 4, 5: 322, 221, 184).
AttnLayout layout_of(const AttnArgs &a, int jobs) {
    AttnLayout l;
    const int64_t wide = jobs > 1 && a.K > a.V ? a.K : a.V;
    const int64_t rows = a.Bt * a.H * jobs, half = rows * ((wide + 127) / 128);
    const int64_t narrow = jobs > 1 && a.V < a.K ? a.V : a.K;    // the fewest state rows
    const bool many = a.bf16 && half > (a.K > 64 ? 256 : 384);
    l.v_cols = wide > 64 && narrow <= 128 && half > 128 && (half <= 256 || many) &&
                       !(a.bf16 && jobs > 1) ? 128 : 64;
    const int64_t groups = rows * ((wide + l.v_cols - 1) / l.v_cols);
    const int64_t most = a.T / (a.bf16 ? 256 : 64);
    int64_t seg = groups > 0 && groups <= 128 ? 512 / groups : 1;
    if (!a.bf16 && seg >= 6) seg /= 2;
    seg = seg < most ? seg : most;
    seg = seg < 3 ? 1 : seg;
    l.seg_tokens = ((a.T + seg - 1) / seg + kChunk - 1) / kChunk * kChunk;
    l.segments = l.seg_tokens ? (a.T + l.seg_tokens - 1) / l.seg_tokens : 1;
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

}  // namespace

AttnLayout attn_layout(const AttnArgs &a) { return layout_of(a, 1); }
AttnLayout attn_bwd_layout(const AttnArgs &a) { return layout_of(a, 3); }

bool attn_fits(const AttnArgs &a) {
    const double heads = (double)a.Bt * (double)a.H;
    // the most workgroups of the recurrences (3 jobs, 4 slices; segments, and the chains
    // between them, are taken for at most 128 workgroups), and sizes that 64 bits hold
    return heads * 12 <= (double)kMaxBlocks && heads * (double)a.T <= 0x1p40;
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
        --s.nseg;
        hipError_t e = launch_jobs(a, s, false, l.v_cols, st);
        if (e != hipSuccess) return e;
        const Chain c = {seg, a.init};
        if ((e = launch_chain(a, l, &c, 1, st)) != hipSuccess) return e;
        j.job[0].s0 = seg;
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
        --s.nseg;
        if ((e = launch_jobs(a, s, false, l.v_cols, st)) != hipSuccess) return e;
        const Chain c[2] = {{hseg, a.init}, {dseg, a.dfinal}};
        if ((e = launch_chain(a, l, c, 2, st)) != hipSuccess) return e;
        dq.s0 = hseg;
        dk.s0 = dv.s0 = dseg;
    }
    j.job[0] = dq;
    j.job[1] = dk;
    j.job[2] = dv;
    j.njobs = 3;
    if ((e = launch_jobs(a, j, true, l.v_cols, st)) != hipSuccess || !shared ||
        a.T == 0)
        return e;
    Share x;
    const int64_t rows = a.Bt * a.T * a.G;
    x.part[0] = pk, x.out[0] = a.dk, x.dim4[0] = a.K / 4;
    x.part[1] = pv, x.out[1] = a.dv, x.dim4[1] = a.V / 4;
    x.rep = (int32_t)(a.H / a.G);
    for (int i = 0; i < 2; ++i) x.n4[i] = rows * x.dim4[i];
    const int64_t n4 = x.n4[0] > x.n4[1] ? x.n4[0] : x.n4[1];
    const int64_t most = int64_t(1) << 20, blocks = (n4 + 255) / 256;
    const dim3 grid((uint32_t)(blocks < most ? blocks : most), 2);
    if (a.bf16)
        attn_share_kernel<uint16_t><<<grid, 256, 0, st>>>(x);
    else
        attn_share_kernel<float><<<grid, 256, 0, st>>>(x);
    return hipGetLastError();
}

// ---------------------------------------------------------------------------
namespace {

// One token: S <- e^r S + k (outer) v, y = scale q S, for states in a slot pool.
// The state goes through memory once in each direction, which bounds it.  A
// workgroup serves one (b, h): LPR lanes cover a row of the state with 16-byte
// accesses, so 256 / LPR rows are in flight per access, kBatch accesses before
// the first is used; a lane's four columns are summed over its rows in
// registers and over the workgroup's rows through LDS, in a fixed order.  e^r is two floats:
// one alone is off by the same 2^-25 for every token that a state lives through.  (256 sequences
// of 32 heads of 128 x 128: 206 us, 5.2 TB/s; kBatch 2, 8, 16: 209, 200, 228, and with 64 x
// 64 states 103, 103, 105, 162 for 2, 4, 8, 16.)
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
    const double e = exp((double)least_rate(a.decay[h]));
    const float d = (float)e, less = (float)(e - (double)d);
    // (an infinity times what d lacks would be one of either sign, or NaN)
    auto decayed = [&](float s, float add) {
        return fmaf(s, d, fmaf(fminf(fmaxf(s, -FLT_MAX), FLT_MAX), less, add));
    };
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
                n.x = decayed(s[i].x, kk[i] * vv.x);
                n.y = decayed(s[i].y, kk[i] * vv.y);
                n.z = decayed(s[i].z, kk[i] * vv.z);
                n.w = decayed(s[i].w, kk[i] * vv.w);
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
