// Host-side launchers of the further operators of a layer: linear attention with
// a decay for each head, the group norm behind a mixer, and projections with
// 4-bit weights (internal to libssd.so).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace ssd {

struct AttnArgs {
    const void *q, *k, *v;     // [Bt, T, H, K], [Bt, T, G, K], [Bt, T, G, V] at the strides below
    int64_t qb, qt, kb, kt, vb, vt;   // batch and token strides, in elements
    const float *decay;        // [H]
    const float *init;         // [Bt, H, K, V] or NULL
    const int32_t *lens;       // [Bt] or NULL
    void *y;                   // dense [Bt, T, H, V] io dtype (fwd, step)
    float *fin;                // [Bt, H, K, V] or NULL (fwd)
    float *state;              // [nslots, H, K, V] (step)
    const int32_t *slots;      // [Bt] or NULL (step)
    int64_t nslots;
    const void *dy;            // dense [Bt, T, H, V] io dtype (bwd)
    const float *dfinal;       // [Bt, H, K, V] or NULL (bwd)
    void *dq, *dk, *dv;        // dense [Bt, T, H, K], [Bt, T, G, K], [Bt, T, G, V] io dtype (bwd)
    float *dinit;              // [Bt, H, K, V] or NULL (bwd)
    void *ws;
    int64_t Bt, T, H, G;
    int K, V;
    float scale;
    bool bf16;
};
// How a call is laid over the chip: segments that a sequence is cut into over
// time, their tokens, and the channels of v that a workgroup takes.
struct AttnLayout {
    int64_t segments, seg_tokens;
    int v_cols;
};
bool attn_fits(const AttnArgs &a);   // false: more workgroups than one launch holds
AttnLayout attn_layout(const AttnArgs &a);
AttnLayout attn_bwd_layout(const AttnArgs &a);
size_t attn_workspace(const AttnArgs &a);
size_t attn_bwd_workspace(const AttnArgs &a);
hipError_t launch_attn_fwd(const AttnArgs &a, hipStream_t st);
hipError_t launch_attn_step(const AttnArgs &a, hipStream_t st);
hipError_t launch_attn_bwd(const AttnArgs &a, hipStream_t st);

struct NormArgs {
    const void *x, *z;         // [Bt, T, C] io dtype at the strides below; z NULL without a gate
    int64_t xb, xt, zb, zt;    // batch and token strides, in elements
    const float *weight, *bias;       // [C] or NULL
    const int32_t *lens;       // [Bt] or NULL
    void *y;                   // dense [Bt, T, C] io dtype (fwd)
    const void *dy;            // dense [Bt, T, C] io dtype (bwd)
    void *dx, *dz;             // dense [Bt, T, C] io dtype (bwd); dz NULL without a gate
    float *dweight, *dbias;    // [C] or NULL (bwd)
    float *part;               // bwd workspace
    int64_t Bt, T, C, groups;
    float eps;
    int form;                  // ssd_norm_form
    bool rms, bf16;
};
bool norm_fits(const NormArgs &a);
size_t norm_bwd_workspace(const NormArgs &a);
hipError_t launch_norm_fwd(const NormArgs &a, hipStream_t st);
hipError_t launch_norm_bwd(const NormArgs &a, hipStream_t st);

struct W4Args {
    int64_t rows, inputs, outputs;
    int group;                 // inputs that share a scale: 64 or 128
    const uint8_t *codes;      // [outputs, inputs / 2]
    const uint16_t *scales;    // [outputs, inputs / group] bf16
    const void *x;             // [rows, inputs] io dtype at stride xs
    int64_t xs;
    const float *bias;         // [outputs] or NULL
    void *y;                   // dense [rows, outputs] io dtype
    const void *weight;        // [outputs, inputs] io dtype (quantize)
    uint8_t *wcodes;           // (quantize)
    uint16_t *wscales;
    void *out;                 // [outputs, inputs] io dtype (dequantize)
    bool bf16;
};
bool w4_fits(const W4Args &a);
hipError_t launch_w4_quantize(const W4Args &a, hipStream_t st);
hipError_t launch_w4_dequantize(const W4Args &a, hipStream_t st);
hipError_t launch_w4_linear(const W4Args &a, hipStream_t st);

}  // namespace ssd
