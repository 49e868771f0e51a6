// Recurrent states in a slot pool at 8 bits per element: one scale per block
// of 64 consecutive elements, codes int8 or fp8 (e4m3),
//     scale = max|v| / q,   code = round(v q / max|v|),   value = code scale.
//
// Both directions move each element once and are bound by memory.  A lane
// holds 4 consecutive elements (16 bytes of the state, 4 of codes), 16 lanes
// hold a block, whose maximum is formed by DPP moves; a lane serves kIter
// such groups, all loaded before any is used.  (64 states of 655360 elements,
// int8: write 35 us, 6.0 TB/s; read 31 us, 6.8 TB/s, part of it from the
// memory-side cache.)

#include "layer_launch.h"
#include "ssd_device.h"

namespace ssd {

namespace {

constexpr int kIter = 4;                  // groups of 4 elements per lane
constexpr int kSpan = 256 * 4 * kIter;    // elements of a workgroup
constexpr float kTiny = 0x1p-100f;        // blocks below it are stored as zeros
constexpr uint32_t kInf = 0x7f800000u;

// The largest |v| of 16 lanes as its bit pattern, in every lane: as unsigned
// integers magnitudes order like the floats, infinity above every finite
// value and NaN above infinity.
__device__ __forceinline__ uint32_t block_amax(uint32_t m) {
    auto step = [&](uint32_t o) { m = m > o ? m : o; };
    step(__builtin_amdgcn_update_dpp(0, m, 0xB1, 0xf, 0xf, false));    // quad_perm [1,0,3,2]
    step(__builtin_amdgcn_update_dpp(0, m, 0x4E, 0xf, 0xf, false));    // quad_perm [2,3,0,1]
    step(__builtin_amdgcn_update_dpp(0, m, 0x141, 0xf, 0xf, false));   // row_half_mirror
    step(__builtin_amdgcn_update_dpp(0, m, 0x140, 0xf, 0xf, false));   // row_mirror
    return m;
}

// v q / amax rounded to a multiple of 2^-shift, ties to even.  The float
// quotient v * inv carries up to 2^-23 of itself; where that could cross the
// border between two codes (a few elements in ten thousand), the quotient is
// taken again in double, so the nearest code is always found.
template <typename Shift>
__device__ __forceinline__ float nearest_code(float v, float inv, float amax, float q,
                                              float margin, Shift shift) {
    const float r = v * inv;
    const int s = shift(r);
    const float u = ldexpf(r, s);
    float k = rintf(u);
    if (fabsf(fabsf(u - k) - 0.5f) < margin) {
        const double d = (double)v * (double)q / (double)amax;
        k = (float)rint(ldexp(d, s));
    }
    return ldexpf(k, -s);
}

template <bool FP8>
__device__ __forceinline__ uint32_t encode4(float4 v, float inv, float amax) {
    if constexpr (FP8) {
        // e4m3 keeps 4 significant bits, and steps of 2^-9 below 2^-6; the
        // multiples convert exactly.  Units are below 16: margin 16 * 2^-23 twice.
        auto code = [&](float x) {
            return nearest_code(x, inv, amax, 448.f, 0x1p-18f, [](float r) {
                return 4 - max(__builtin_amdgcn_frexp_expf(r), -5);
            });
        };
        uint32_t w = __builtin_amdgcn_cvt_pk_fp8_f32(code(v.x), code(v.y), 0, false);
        return __builtin_amdgcn_cvt_pk_fp8_f32(code(v.z), code(v.w), w, true);
    } else {
        // units up to 127: margin 128 * 2^-23 twice
        auto code = [&](float x) {
            return (uint32_t)(int)nearest_code(x, inv, amax, 127.f, 0x1p-15f,
                                               [](float) { return 0; }) & 0xffu;
        };
        return code(v.x) | code(v.y) << 8 | code(v.z) << 16 | code(v.w) << 24;
    }
}

template <bool FP8>
__global__ __launch_bounds__(256) void cache_write_kernel(const float *__restrict__ state,
                                                          const int32_t *__restrict__ slots,
                                                          uint8_t *__restrict__ codes,
                                                          float *__restrict__ scales,
                                                          int64_t size, int64_t nslots,
                                                          uint32_t blk) {
    const int64_t i = blockIdx.x / blk;
    const int64_t e0 = (int64_t)(blockIdx.x - (uint32_t)i * blk) * kSpan + threadIdx.x * 4;
    const int64_t slot = slots ? (int64_t)slots[i] : i;
    if (slot < 0 || slot >= nslots) return;
    const float *src = state + i * size;
    float4 v[kIter];
#pragma unroll
    for (int k = 0; k < kIter; ++k) {
        const int64_t e = e0 + k * 1024;
        v[k] = e < size ? load_nt(src + e) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    const int64_t nblk = (size + 63) / 64;
#pragma unroll
    for (int k = 0; k < kIter; ++k) {
        const int64_t e = e0 + k * 1024;
        const uint32_t m01 = max(__float_as_uint(fabsf(v[k].x)), __float_as_uint(fabsf(v[k].y)));
        const uint32_t m23 = max(__float_as_uint(fabsf(v[k].z)), __float_as_uint(fabsf(v[k].w)));
        const uint32_t mb = block_amax(max(m01, m23));
        const float amax = __uint_as_float(mb);
        constexpr float q = FP8 ? 448.f : 127.f;
        float scale;
        uint32_t w = 0;
        if (mb >= kInf) {               // an infinity or NaN in the block: NaN on reading
            scale = __uint_as_float(0x7fc00000u);
        } else if (amax < kTiny) {
            scale = 0.f;
        } else {
            scale = amax / q;
            // (at the top of the range the rounded quotient may read back as infinity)
            if (scale * q >= __uint_as_float(kInf))
                scale = __uint_as_float(__float_as_uint(scale) - 1u);
            w = encode4<FP8>(v[k], q / amax, amax);
        }
        if (e < size) {
            *reinterpret_cast<uint32_t *>(codes + slot * size + e) = w;
            if ((threadIdx.x & 15) == 0) scales[slot * nblk + (e >> 6)] = scale;
        }
    }
}

template <bool FP8>
__global__ __launch_bounds__(256) void cache_read_kernel(const uint8_t *__restrict__ codes,
                                                         const float *__restrict__ scales,
                                                         const int32_t *__restrict__ slots,
                                                         float *__restrict__ state, int64_t size,
                                                         int64_t nslots, uint32_t blk) {
    const int64_t i = blockIdx.x / blk;
    const int64_t e0 = (int64_t)(blockIdx.x - (uint32_t)i * blk) * kSpan + threadIdx.x * 4;
    const int64_t slot = slots ? (int64_t)slots[i] : i;
    const bool live = slot >= 0 && slot < nslots;
    const int64_t nblk = (size + 63) / 64;
    uint32_t w[kIter];
    float sc[kIter];
#pragma unroll
    for (int k = 0; k < kIter; ++k) {
        const int64_t e = e0 + k * 1024;
        const bool in = live && e < size;
        w[k] = in ? *reinterpret_cast<const uint32_t *>(codes + slot * size + e) : 0u;
        sc[k] = in ? scales[slot * nblk + (e >> 6)] : 0.f;
    }
#pragma unroll
    for (int k = 0; k < kIter; ++k) {
        const int64_t e = e0 + k * 1024;
        float4 v;
        if constexpr (FP8) {
            const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(w[k], false);
            const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8(w[k], true);
            v = make_float4(lo[0], lo[1], hi[0], hi[1]);
        } else {
            v = make_float4((float)(int8_t)(w[k] & 0xffu), (float)(int8_t)(w[k] >> 8 & 0xffu),
                            (float)(int8_t)(w[k] >> 16 & 0xffu), (float)(int8_t)(w[k] >> 24));
        }
        v.x *= sc[k];
        v.y *= sc[k];
        v.z *= sc[k];
        v.w *= sc[k];
        if (e < size) *reinterpret_cast<float4 *>(state + i * size + e) = v;
    }
}

uint32_t blocks_per_state(const CacheArgs &a) { return (uint32_t)((a.size + kSpan - 1) / kSpan); }

}  // namespace

bool cache_fits(const CacheArgs &a) {
    return (double)a.n * (double)((a.size + kSpan - 1) / kSpan) <= (double)kMaxBlocks;
}

hipError_t launch_cache_write(const CacheArgs &a, hipStream_t st) {
    const uint32_t blk = blocks_per_state(a);
    const dim3 grid((uint32_t)(a.n * blk));
    if (a.fp8)
        cache_write_kernel<true><<<grid, 256, 0, st>>>(a.src, a.slots, (uint8_t *)a.codes,
                                                       a.scales, a.size, a.nslots, blk);
    else
        cache_write_kernel<false><<<grid, 256, 0, st>>>(a.src, a.slots, (uint8_t *)a.codes,
                                                        a.scales, a.size, a.nslots, blk);
    return hipGetLastError();
}

hipError_t launch_cache_read(const CacheArgs &a, hipStream_t st) {
    const uint32_t blk = blocks_per_state(a);
    const dim3 grid((uint32_t)(a.n * blk));
    if (a.fp8)
        cache_read_kernel<true><<<grid, 256, 0, st>>>((const uint8_t *)a.codes, a.scales, a.slots,
                                                      a.dst, a.size, a.nslots, blk);
    else
        cache_read_kernel<false><<<grid, 256, 0, st>>>((const uint8_t *)a.codes, a.scales,
                                                       a.slots, a.dst, a.size, a.nslots, blk);
    return hipGetLastError();
}

}  // namespace ssd
