// Projections with 4-bit weights.  Per output row and group of consecutive inputs,
//     scale = bf16(max|w| / 7),   code = round(w / scale) + 8   (1 to 15),
//     w = (code - 8) scale,       y = x w^T + bias,
// two codes to a byte, the even input in the low half.
//
// The codes bound a few rows' product, x's reading many rows' (the figures are at the
// kernels).  Packing 10576 x 2560 bf16 weights takes 22 us in a profile and unpacking them
// 11, 30.8 together (137 MB, 4.45 TB/s).

#include "block_launch.h"
#include "layer_launch.h"
#include "ssd_device.h"

namespace ssd {

namespace {

constexpr float kTiny = 0x1p-100f;    // groups below it are stored as zeros
constexpr uint32_t kInf = 0x7f800000u;

// w / s rounded to a whole number, ties to even.  The float quotient may lie on the
// other side of a border; w - k s is exact in sign (k s has at most 11 significant
// bits), so it says whether the next number is nearer.
__device__ __forceinline__ int nearest(float w, float s, float inv) {
    float k = rintf(w * inv);
    const float r = fmaf(-k, s, w), half = 0.5f * s;
    const bool odd = (int)k & 1;
    if (r > half || (r == half && odd)) k += 1.f;
    else if (r < -half || (r == -half && odd)) k -= 1.f;
    return (int)k;
}

// The largest of 16 lanes' magnitudes as bit patterns: infinity and NaN stay above
// every finite value.
__device__ __forceinline__ uint32_t max16(uint32_t m) {
    auto step = [&](uint32_t o) { m = m > o ? m : o; };
    step(__builtin_amdgcn_update_dpp(0, m, 0xB1, 0xf, 0xf, false));    // quad_perm [1,0,3,2]
    step(__builtin_amdgcn_update_dpp(0, m, 0x4E, 0xf, 0xf, false));    // quad_perm [2,3,0,1]
    step(__builtin_amdgcn_update_dpp(0, m, 0x141, 0xf, 0xf, false));   // row_half_mirror
    step(__builtin_amdgcn_update_dpp(0, m, 0x140, 0xf, 0xf, false));   // row_mirror
    return m;
}

// 16 lanes hold a group, GROUP / 16 consecutive inputs each.
template <typename T, int GROUP>
__global__ __launch_bounds__(256) void w4_quantize_kernel(const T *__restrict__ weight,
                                                          uint8_t *__restrict__ codes,
                                                          uint16_t *__restrict__ scales,
                                                          int64_t groups) {
    constexpr int E = GROUP / 16;
    const int64_t g = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);
    const bool in = g < groups;
    const int64_t at = (in ? g : 0) * GROUP + (threadIdx.x & 15) * E;
    float w[E];
#pragma unroll
    for (int i = 0; i < E; i += 4) {
        const float4 v = load4(weight + at + i);
        w[i] = v.x, w[i + 1] = v.y, w[i + 2] = v.z, w[i + 3] = v.w;
    }
    uint32_t mb = 0;
#pragma unroll
    for (int i = 0; i < E; ++i) mb = max(mb, __float_as_uint(fabsf(w[i])));
    mb = max16(mb);
    const float most = __uint_as_float(mb);
    uint32_t sb = 0, code = 0x88888888u;    // zeros
    if (mb >= kInf) {                       // an infinity or NaN in the group: NaN on reading
        sb = 0x7fc0u;
    } else if (most >= kTiny) {
        sb = f32_to_bf16_bits(most / 7.f);
        const float s = bf16_to_f32((uint16_t)sb), inv = 1.f / s;
        code = 0;
#pragma unroll
        for (int i = 0; i < E; ++i) code |= (uint32_t)(nearest(w[i], s, inv) + 8) << (4 * i);
    }
    if (!in) return;
    if constexpr (E == 4) *reinterpret_cast<uint16_t *>(codes + at / 2) = (uint16_t)code;
    else *reinterpret_cast<uint32_t *>(codes + at / 2) = code;
    if ((threadIdx.x & 15) == 0) scales[g] = (uint16_t)sb;
}

// 8 weights a lane.
template <typename T>
__global__ __launch_bounds__(256) void w4_dequantize_kernel(const uint8_t *__restrict__ codes,
                                                            const uint16_t *__restrict__ scales,
                                                            T *__restrict__ out, int64_t n8,
                                                            int per_group) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n8) return;
    const uint32_t w = reinterpret_cast<const uint32_t *>(codes)[i];
    const float s = bf16_to_f32(scales[i / per_group]);
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = (float)((int)(w >> (4 * e) & 15u) - 8) * s;
    if constexpr (sizeof(T) == 4) {
        store_nt(out + 8 * i, make_float4(v[0], v[1], v[2], v[3]));
        store_nt(out + 8 * i + 4, make_float4(v[4], v[5], v[6], v[7]));
    } else {
        store_nt(out + 8 * i, make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                         pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])));
    }
}

// Products of up to 16 RT rows on matrix instructions: rows of x as the one operand,
// 16 outputs' weights as the other.
//
// A lane's 8 codes become 8 bf16 by bit operations alone: a code in bits 3 to 6 of a
// bf16 16.0 reads 16 + code, exactly, so four words of pairs (i, i + 4) take four
// shifts and four and-ors; x comes in the same order.  What is 24 too much in each is
// taken off once a group: acc - 24 sum(x), the sum from a matrix instruction against
// ones, before the group's scale.  float32 rows are three bf16 rows (hi, mid, lo to
// 2^-24), so the products are exact for both types; for them 24 is taken off each
// weight at once, since sums five times as high would round five times as coarsely.
//
// A wavefront takes NT tiles of 16 outputs over its share of the inputs, 64 at a time;
// the shares of a workgroup's wavefronts are added through LDS, in order.  Rows and codes
// are loaded into the wavefront's own part of LDS, whole lines at a time and three steps
// ahead (64 rows, 5120 inputs, 2560 outputs: 13 us; one step ahead, 22 where three took 14):
// read straight into operands, 16 rows 16 bytes at a time, they came at 11 bytes a cycle and CU
// (26 us).  What bounds it is latency: a wavefront's share is a chain of steps (20 of 5120
// inputs), each a trip to L2 or memory that three steps cover in part.  x is read once for
// every 16 or 32 outputs (48 rows of 5120 for 2560: 39 MB in some 8 us, far below what the L2
// caches give); the codes' 6.6 MB alone would take 1.5.
//
// 8 inputs of one row: as they lie in LDS, and as operands in the codes' order (0 4 1 5 2 6 3 7).
template <typename T>
struct Rows;
template <>
struct Rows<uint16_t> {
    static constexpr int kTerms = 1;
    struct Raw {
        uint4 v;
        __device__ __forceinline__ void read(const uint16_t *row, int piece, int order) {
            const u32x4 f = *reinterpret_cast<const u32x4 *>(row + (piece ^ order) * 8);
            v = make_uint4(f[0], f[1], f[2], f[3]);
        }
        __device__ __forceinline__ void terms(bf16x8 *t) const {
            t[0] = as_bf16x8(make_uint4(pair_lo(v.x, v.z), pair_hi(v.x, v.z), pair_lo(v.y, v.w),
                                        pair_hi(v.y, v.w)));
        }
    };
};
template <>
struct Rows<float> {
    static constexpr int kTerms = 3;
    struct Raw {
        f32x4 a, b;
        __device__ __forceinline__ void read(const float *row, int piece, int order) {
            a = *reinterpret_cast<const f32x4 *>(row + (2 * piece ^ order) * 4);
            b = *reinterpret_cast<const f32x4 *>(row + ((2 * piece + 1) ^ order) * 4);
        }
        __device__ __forceinline__ void terms(bf16x8 *t) const {
            float lo[4] = {a[0], a[1], a[2], a[3]}, hi[4] = {b[0], b[1], b[2], b[3]};
#pragma unroll
            for (int e = 0; e < 3; ++e) {
                uint32_t w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    w[i] = pack_bf16x2(lo[i], hi[i]);
                    lo[i] -= bf16_lo(w[i]);
                    hi[i] -= bf16_hi(w[i]);
                }
                t[e] = as_bf16x8(make_uint4(w[0], w[1], w[2], w[3]));
            }
        }
    };
};

// 8 codes as 16 + code, in the order 0 4 1 5 2 6 3 7
__device__ __forceinline__ bf16x8 codes_frag(uint32_t w) {
    constexpr uint32_t kMask = 0x00780078u, k16 = 0x41804180u;
    return as_bf16x8(make_uint4((w << 3 & kMask) | k16, (w >> 1 & kMask) | k16,
                                (w >> 5 & kMask) | k16, (w >> 9 & kMask) | k16));
}

// the codes less 8, exactly
__device__ __forceinline__ bf16x8 weights_frag(uint32_t w) {
    uint4 c = __builtin_bit_cast(uint4, codes_frag(w));
    for (uint32_t *p : {&c.x, &c.y, &c.z, &c.w})
        *p = pack_bf16x2(bf16_lo(*p) - 24.f, bf16_hi(*p) - 24.f);
    return as_bf16x8(c);
}

template <typename T, int RT, int NT>
__global__ __launch_bounds__(256) void w4_linear_kernel(const W4Args a) {
    typedef Rows<T> R;
    constexpr int STEP = 64;           // inputs at a time
    constexpr int kVec = 16 / sizeof(T), kPerRow = STEP / kVec;      // 16-byte pieces of a row
    constexpr int kXLoads = 16 * RT * kPerRow / 64;                  // loads of a lane
    constexpr int kX = 16 * RT * STEP * sizeof(T), kAll = kX + 1024; // bytes
    constexpr bool kExact = sizeof(T) == 4;
    constexpr uint32_t kNowhere = 0xffffffffu;
    static_assert(NT <= 2, "a load of codes holds two tiles");
    static_assert(3 * (kXLoads + 1 + NT) < 64, "loads that a wait can count");
    // (separate variables, read by whole vectors: so the compiler sees that reads of one need
    // not wait for loads into another)
    __shared__ __align__(16) char buf0[4 * kAll];
    __shared__ __align__(16) char buf1[4 * kAll];
    __shared__ __align__(16) char buf2[4 * kAll];
    __shared__ __align__(16) char buf3[4 * kAll];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int m = lane & 15, q = lane >> 4;
    const int64_t o0 = (int64_t)blockIdx.x * (16 * NT);
    const int64_t row0 = (int64_t)blockIdx.y * (16 * RT);
    const int inputs = (int)a.inputs, steps = inputs / STEP;
    const int s0 = steps * wave / 4, s1 = steps * (wave + 1) / 4;
    const int per_group = a.group / STEP, groups = inputs / a.group;

    // lane offsets from the step's first input; a row's pieces lie in LDS in an order of its
    // own, so that 16 rows' same piece is on 16 banks' groups
    auto order = [](int row) { return sizeof(T) == 2 ? row >> 1 & 7 : row & 15; };
    const char *codes = reinterpret_cast<const char *>(a.codes) + o0 * (a.inputs / 2);
    const char *x = reinterpret_cast<const char *>(static_cast<const T *>(a.x) + row0 * a.xs);
    const uint16_t *scales = a.scales + o0 * groups;
    const int64_t last = a.outputs - 1 - o0;
    auto output = [&](int i) { return i < last ? (uint32_t)i : (uint32_t)last; };
    uint32_t xat[kXLoads], cat, sat[NT];
#pragma unroll
    for (int i = 0; i < kXLoads; ++i) {
        const int p = lane + 64 * i, row = p / kPerRow;
        const int col = (p % kPerRow ^ order(row & 15)) * kVec;
        xat[i] = row0 + row < a.rows ? (uint32_t)((row * (uint64_t)a.xs + col) * sizeof(T))
                                     : kNowhere;
    }
    cat = lane < 32 * NT ? output(lane >> 1) * (uint32_t)(inputs / 2) + 16 * (lane & 1) : kNowhere;
#pragma unroll
    for (int t = 0; t < NT; ++t) sat[t] = output(16 * t + m) * (uint32_t)groups * 2;
    auto load = [&](char *buf, uint32_t (&sc)[NT], int step) {
        // (past the share nothing is read and zeros arrive, without a branch: at one the
        // compiler would wait for every load on its way)
        const uint32_t bytes = step < s1 ? 0xfffffff0u : 0u;
        const __amdgpu_buffer_rsrc_t rs = make_rsrc(scales + step / per_group, bytes);
#pragma unroll
        for (int t = 0; t < NT; ++t)
            sc[t] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(rs, sat[t], 0, 0);
#ifdef __HIP_DEVICE_COMPILE__   // (16 bytes a lane are gfx950's: not known to the host's pass)
        typedef __attribute__((address_space(3))) char lds_t;
        const __amdgpu_buffer_rsrc_t rx = make_rsrc(x + (int64_t)step * (STEP * sizeof(T)), bytes);
        const __amdgpu_buffer_rsrc_t rc = make_rsrc(codes + (int64_t)step * (STEP / 2), bytes);
#pragma unroll
        for (int i = 0; i < kXLoads; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (lds_t *)(buf + i * 1024), 16, xat[i], 0,
                                                     0, 0);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rc, (lds_t *)(buf + kX), 16, cat, 0, 0, 0);
#endif
        __builtin_amdgcn_sched_barrier(0);   // (left alone, loads sink to where they are used)
    };
    f32x4 y[RT][NT];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int t = 0; t < NT; ++t) y[r][t] = f32x4{0.f, 0.f, 0.f, 0.f};
    const uint32_t one = 0x3f803f80u;
    const bf16x8 ones = as_bf16x8(make_uint4(one, one, one, one));
    auto multiply = [&](const char *buf, const uint32_t (&sc)[NT]) {
        // this step's loads are through, three later steps' may be on their way (the wait is
        // the kernel's own: the compiler takes a load into LDS for one lane's 16 bytes)
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(3 * (kXLoads + 1 + NT)) : "memory");
        // a lane has 16 consecutive inputs, in two contraction steps
        uint32_t w[NT][2];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const u32x2 v = *reinterpret_cast<const u32x2 *>(buf + kX + (16 * t + m) * 32 + 8 * q);
            w[t][0] = v[0], w[t][1] = v[1];
        }
        f32x4 sum[RT], acc[RT][NT];
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            sum[r] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int t = 0; t < NT; ++t) acc[r][t] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            bf16x8 wf[NT];
#pragma unroll
            for (int t = 0; t < NT; ++t)
                wf[t] = kExact ? weights_frag(w[t][i]) : codes_frag(w[t][i]);
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                typename R::Raw raw;
                raw.read(reinterpret_cast<const T *>(buf) + (16 * r + m) * STEP, 2 * q + i,
                         order(m));
                bf16x8 xf[R::kTerms];
                raw.terms(xf);
#pragma unroll
                for (int e = R::kTerms - 1; e >= 0; --e) {
                    if (!kExact) sum[r] = mfma16x16x32(xf[e], ones, sum[r]);
#pragma unroll
                    for (int t = 0; t < NT; ++t)
                        acc[r][t] = mfma16x16x32(xf[e], wf[t], acc[r][t]);
                }
            }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const float s = __uint_as_float(sc[t] << 16);
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    y[r][t][e] = fmaf(s, kExact ? acc[r][t][e]
                                                : fmaf(-24.f, sum[r][e], acc[r][t][e]),
                                      y[r][t][e]);
        }
        // (a buffer is loaded again only once it has been read)
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    };
    const int own = wave * kAll;
    uint32_t sc0[NT], sc1[NT], sc2[NT], sc3[NT];
    load(buf0 + own, sc0, s0);
    load(buf1 + own, sc1, s0 + 1);
    load(buf2 + own, sc2, s0 + 2);
    for (int st = s0; st < s1; st += 4) {
        load(buf3 + own, sc3, st + 3);
        multiply(buf0 + own, sc0);
        load(buf0 + own, sc0, st + 4);
        multiply(buf1 + own, sc1);
        load(buf1 + own, sc1, st + 5);
        multiply(buf2 + own, sc2);
        load(buf2 + own, sc2, st + 6);
        multiply(buf3 + own, sc3);
    }
    // buf0 is free once all wavefronts are through and nothing is on its way into it (loads
    // past the share write their zeros too; a barrier alone does not wait for them)
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    f32x4 *part = reinterpret_cast<f32x4 *>(buf0);
    if (wave > 0)
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int t = 0; t < NT; ++t)
                part[(((wave - 1) * RT + r) * NT + t) * 64 + lane] = y[r][t];
    __syncthreads();
    if (wave > 0) return;
    for (int v = 0; v < 3; ++v)
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int t = 0; t < NT; ++t) y[r][t] += part[((v * RT + r) * NT + t) * 64 + lane];
    // accumulator element e of lane (m, q): row 4 q + e, output m
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int64_t o = o0 + 16 * t + m;
        if (o >= a.outputs) continue;
        const float b = a.bias ? a.bias[o] : 0.f;
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int64_t row = row0 + 16 * r + 4 * q + e;
                if (row < a.rows)
                    store_y1(a.y, row * a.outputs + o, y[r][t][e] + b, sizeof(T) == 2);
            }
    }
}

// Products of RN rows (1 or 2) on the vector units, which need fewer steps than a
// matrix instruction whose 16 rows are mostly empty.  The rows lie in LDS, bf16 ones in
// the codes' order, so that two products take one instruction; a lane reads 16 codes
// at a time (8 bytes, of one group), all of a slab's before the first is used, and
// its partial sums of 24 x are taken off as above (float32 rows take codes one at a time: 2
// rows, whole calls, 11.9 us for bf16's 9.6).  10576 x 2560, one row: 7.1 us in a
// profile, of which 14.4 MB would take 3.0 at a copy's rate (661 workgroups of one slab
// each: the start of the launch and one trip to memory and back).
constexpr int kSlab = 4096;     // inputs that LDS holds at a time
template <typename T>
struct Piece;    // 16 inputs of a row in LDS
template <>
struct Piece<uint16_t> {
    uint4 v[2];
    // the 16 inputs at p, rearranged
    __device__ __forceinline__ void fill(const uint16_t *p) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint4 a = *reinterpret_cast<const uint4 *>(p + 8 * i);
            v[i] = make_uint4(pair_lo(a.x, a.z), pair_hi(a.x, a.z), pair_lo(a.y, a.w),
                              pair_hi(a.y, a.w));
        }
    }
    // what dot() gives too much
    __device__ __forceinline__ float excess() const {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            for (const uint32_t w : {v[i].x, v[i].y, v[i].z, v[i].w}) s += bf16_lo(w) + bf16_hi(w);
        return 24.f * s;
    }
    // sum of (16 + code) x
    __device__ __forceinline__ float dot(uint2 w) const {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint4 c = __builtin_bit_cast(uint4, codes_frag(i ? w.y : w.x));
            s = dot2(c.x, v[i].x, s);
            s = dot2(c.y, v[i].y, s);
            s = dot2(c.z, v[i].z, s);
            s = dot2(c.w, v[i].w, s);
        }
        return s;
    }
    static __device__ __forceinline__ float dot2(uint32_t a, uint32_t b, float c) {
#ifdef __HIP_DEVICE_COMPILE__   // (gfx950's, not known to the host's pass)
        return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2_t, a),
                                               __builtin_bit_cast(bf16x2_t, b), c, false);
#else
        return c;
#endif
    }
};
template <>
struct Piece<float> {
    float4 v[4];
    __device__ __forceinline__ void fill(const float *p) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = *reinterpret_cast<const float4 *>(p + 4 * i);
    }
    __device__ __forceinline__ float excess() const { return 0.f; }
    __device__ __forceinline__ float dot(uint2 w) const {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t c = (i < 2 ? w.x : w.y) >> (16 * (i & 1));
            auto value = [&](int e) { return (float)(int)((c >> (4 * e) & 15u) - 8u); };
            s = fmaf(value(0), v[i].x, s);
            s = fmaf(value(1), v[i].y, s);
            s = fmaf(value(2), v[i].z, s);
            s = fmaf(value(3), v[i].w, s);
        }
        return s;
    }
};

template <typename T, int RN, int OPW>
__global__ __launch_bounds__(256) void w4_rows_kernel(const W4Args a) {
    constexpr int kPieces = kSlab / 16, kIter = kSlab / 1024;
    __shared__ __align__(16) Piece<T> xs[RN][kPieces];
    __shared__ float sums[RN][kPieces];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int64_t o0 = ((int64_t)blockIdx.x * 4 + wave) * OPW;
    const int64_t bytes = a.inputs / 2, groups = a.inputs / a.group;
    const int shift = a.group == 64 ? 2 : 3;       // pieces of a group
    const T *x = static_cast<const T *>(a.x);
    float y[RN][OPW];
#pragma unroll
    for (int r = 0; r < RN; ++r)
#pragma unroll
        for (int o = 0; o < OPW; ++o) y[r][o] = 0.f;
    for (int64_t k0 = 0; k0 < a.inputs; k0 += kSlab) {
        const int pieces = (int)((a.inputs - k0 < kSlab ? a.inputs - k0 : kSlab) / 16);
        // codes and scales of the slab, on their way while the rows are brought in
        uint2 w[OPW][kIter];
        uint16_t s[OPW][kIter];
#pragma unroll
        for (int o = 0; o < OPW; ++o) {
            const int64_t out = o0 + o < a.outputs ? o0 + o : a.outputs - 1;
            const uint2 *c = reinterpret_cast<const uint2 *>(a.codes + out * bytes) + k0 / 16;
            const uint16_t *g = a.scales + out * groups + k0 / a.group;
#pragma unroll
            for (int i = 0; i < kIter; ++i) {
                const int p = lane + 64 * i;
                if (p < pieces) {
                    w[o][i] = c[p];
                    s[o][i] = g[p >> shift];
                }
            }
        }
        if (k0) __syncthreads();
#pragma unroll
        for (int r = 0; r < RN; ++r)
            for (int p = threadIdx.x; p < pieces; p += 256) {
                Piece<T> v;
                v.fill(x + r * a.xs + k0 + 16 * p);
                xs[r][p] = v;
                sums[r][p] = v.excess();
            }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kIter; ++i) {
            const int p = lane + 64 * i;
            if (p >= pieces) continue;
#pragma unroll
            for (int r = 0; r < RN; ++r) {
                const Piece<T> v = xs[r][p];
                const float off = sums[r][p];
#pragma unroll
                for (int o = 0; o < OPW; ++o)
                    y[r][o] = fmaf(bf16_to_f32(s[o][i]), v.dot(w[o][i]) - off, y[r][o]);
            }
        }
    }
#pragma unroll
    for (int r = 0; r < RN; ++r) {
#pragma unroll
        for (int o = 0; o < OPW; ++o) {
            float v = group_sum<16>(y[r][o]);
            v += __shfl_xor(v, 16, 64);
            v += __shfl_xor(v, 32, 64);
            if (lane == 0 && o0 + o < a.outputs)
                store_y1(a.y, r * a.outputs + o0 + o, v + (a.bias ? a.bias[o0 + o] : 0.f),
                         sizeof(T) == 2);
        }
    }
}

// One or two tiles of outputs (16 or 32): two halve the reading of x, but also the workgroups,
// so they are taken where one each would be more than a workgroup a CU (rows x inputs x
// outputs, us with one and two tiles of outputs; bf16: 64 x 8192 x 1024, 128 workgroups of
// one: 10.7, 14.4; 32 x 5120 x 2560, 160: 9.9, 13.0; 64 x 5120 x 2560, 320: 13.8, 13.0; 32 x 5120
// x 5120, 320: 14.1, 13.1; 3 x 1664 x 32768, 2048: 15.6, 12.6; 64 x 1664 x 32768, 4096: 47.7,
// 37.1; float32: 64 x 8192 x 1024, 256: 19.0, 23.8; 16 x 5120 x 2560, 160: 13.0, 16.4; 32 x
// 5120 x 2560, 320: 19.1, 16.7; 64 x 1664 x 32768, 8192: 112.5, 78.3).
template <typename T, int RT>
void launch_tiles(const W4Args &a, hipStream_t st) {
    const int64_t tiles = (a.outputs + 15) / 16, parts = (a.rows + 16 * RT - 1) / (16 * RT);
    if (tiles * parts <= 256)
        w4_linear_kernel<T, RT, 1>
            <<<dim3((uint32_t)tiles, (uint32_t)parts), 256, 0, st>>>(a);
    else
        w4_linear_kernel<T, RT, 2>
            <<<dim3((uint32_t)((tiles + 1) / 2), (uint32_t)parts), 256, 0, st>>>(a);
}
template <typename T, int RN, int OPW>
void launch_rows(const W4Args &a, hipStream_t st) {
    const uint32_t blocks = (uint32_t)((a.outputs + 4 * OPW - 1) / (4 * OPW));
    w4_rows_kernel<T, RN, OPW><<<blocks, 256, 0, st>>>(a);
}
// Up to two rows on the vector units (10576 x 2560 outputs, whole calls: 8.0 and 8.8 us, on
// matrix instructions 9.5 and 9.6; with 4 rows 12.2 and 9.9).  A wavefront there takes four
// outputs where that leaves two workgroups a CU, else two (6592 x 8192: 9.5 us, with four
// 12.2).
// More rows in tiles of 16 rows, one or two a workgroup (bf16; rows x inputs x outputs, us with
// one and two tiles of rows): two halve the reading of codes and fill what they read of x (20
// x 1664 x 32768: 22.6, 19.8; 64 x 2560 x 10576: 25.5, 21.0; 128 x 5120 x 5120: 31.6, 28.6; with
// a fifth, seventh or ninth tile half of whose pair stays empty too: 80 x 2560 x 10576: 28.8,
// 25.9; 112: 38.0, 36.1; 144: 44.5, 41.6; x 5120 x 2560: 14.3, 13.6; 19.8, 18.0; 20.0, 19.1),
// unless that is one of four (48 x 5120 x 2560: 10.3, 13.0; x 2560 x 10576: 20.0, 19.8; x 5120 x
// 5120: 14.9, 17.9) or CUs would idle (32 x 8192 x 1024, 128 workgroups of one: 10.7, 13.0).
// float32 always in single ones: three terms of two tiles leave a CU one workgroup (32 x 1664 x
// 32768: 40.7, 48.0).
template <typename T>
void launch_linear(const W4Args &a, hipStream_t st) {
    if (a.rows <= 2) {
        const bool four = a.outputs >= 16 * 512;
        if (a.rows == 1)
            four ? launch_rows<T, 1, 4>(a, st) : launch_rows<T, 1, 2>(a, st);
        else
            four ? launch_rows<T, 2, 4>(a, st) : launch_rows<T, 2, 2>(a, st);
        return;
    }
    const int64_t rows16 = (a.rows + 15) / 16, blocks = (a.outputs + 15) / 16 * rows16;
    if (sizeof(T) == 4 || rows16 == 1 || rows16 == 3 || blocks <= 256)
        launch_tiles<T, 1>(a, st);
    else if constexpr (sizeof(T) == 2)
        launch_tiles<T, 2>(a, st);
}

}  // namespace

bool w4_fits(const W4Args &a) {
    const double n = (double)a.inputs * (double)a.outputs;
    // (grid.y holds 65535 blocks of 16 rows)
    return n / 1024 + 1 <= (double)kMaxBlocks &&
           ((double)a.outputs / 16 + 1) * ((double)a.rows / 16 + 1) <= (double)kMaxBlocks &&
           a.rows <= int64_t(65535) * 16;
}

hipError_t launch_w4_quantize(const W4Args &a, hipStream_t st) {
    const int64_t groups = a.outputs * (a.inputs / a.group);
    const uint32_t blocks = (uint32_t)((groups + 15) / 16);
#define SSD_W4_QUANT(T, GROUP)                                                                \
    w4_quantize_kernel<T, GROUP><<<blocks, 256, 0, st>>>(static_cast<const T *>(a.weight), \
                                                         a.wcodes, a.wscales, groups)
    if (a.bf16)
        a.group == 64 ? SSD_W4_QUANT(uint16_t, 64) : SSD_W4_QUANT(uint16_t, 128);
    else
        a.group == 64 ? SSD_W4_QUANT(float, 64) : SSD_W4_QUANT(float, 128);
#undef SSD_W4_QUANT
    return hipGetLastError();
}

hipError_t launch_w4_dequantize(const W4Args &a, hipStream_t st) {
    const int64_t n8 = a.outputs * (a.inputs / 8);
    const uint32_t blocks = (uint32_t)((n8 + 255) / 256);
    if (a.bf16)
        w4_dequantize_kernel<uint16_t><<<blocks, 256, 0, st>>>(
            a.codes, a.scales, static_cast<uint16_t *>(a.out), n8, a.group / 8);
    else
        w4_dequantize_kernel<float><<<blocks, 256, 0, st>>>(
            a.codes, a.scales, static_cast<float *>(a.out), n8, a.group / 8);
    return hipGetLastError();
}

hipError_t launch_w4_linear(const W4Args &a, hipStream_t st) {
    if (a.bf16)
        launch_linear<uint16_t>(a, st);
    else
        launch_linear<float>(a, st);
    return hipGetLastError();
}

}  // namespace ssd
