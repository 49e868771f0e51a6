// Projections with 4-bit weights.  Per output row and group of consecutive inputs,
//     scale = bf16(max|w| / 7),   code = round(w / scale) + 8   (1 to 15),
//     w = (code - 8) scale,       y = x w^T + bias,
// two codes to a byte, the even input in the low half.

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

// One wavefront per (output, row).
template <typename T>
__global__ __launch_bounds__(256) void w4_linear_kernel(const W4Args a) {
    const int64_t o = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    const int lane = threadIdx.x & 63;
    if (o >= a.outputs) return;
    const uint32_t *codes = reinterpret_cast<const uint32_t *>(a.codes + o * (a.inputs / 2));
    const uint16_t *scales = a.scales + o * (a.inputs / a.group);
    for (int64_t r = 0; r < a.rows; ++r) {
        const T *x = static_cast<const T *>(a.x) + r * a.xs;
        float sum = 0.f;
        for (int64_t k = lane * 8; k < a.inputs; k += 512) {
            const uint32_t w = codes[k >> 3];
            float p = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) p += (float)((int)(w >> (4 * e) & 15u) - 8) * load1(x + k + e);
            sum += p * bf16_to_f32(scales[k / a.group]);
        }
        sum = group_sum<16>(sum);
        sum += __shfl_xor(sum, 16, 64);
        sum += __shfl_xor(sum, 32, 64);
        if (lane == 0)
            store_y1(a.y, r * a.outputs + o, sum + (a.bias ? a.bias[o] : 0.f), sizeof(T) == 2);
    }
}

}  // namespace

bool w4_fits(const W4Args &a) {
    const double n = (double)a.inputs * (double)a.outputs;
    return n / 1024 + 1 <= (double)kMaxBlocks && (double)a.outputs / 4 + 1 <= (double)kMaxBlocks;
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
    const uint32_t blocks = (uint32_t)((a.outputs + 3) / 4);
    if (a.bf16)
        w4_linear_kernel<uint16_t><<<blocks, 256, 0, st>>>(a);
    else
        w4_linear_kernel<float><<<blocks, 256, 0, st>>>(a);
    return hipGetLastError();
}

}  // namespace ssd
