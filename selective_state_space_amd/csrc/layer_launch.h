// Host-side launchers of the operators around the layer scan: the short causal
// convolution, the per-channel selective scan and the 8-bit state cache
// (internal to libssd.so).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace ssd {

// Workgroups of 256 threads that one launch holds (fewer than 2^32 threads).
constexpr int64_t kMaxBlocks = (int64_t(1) << 24) - 1;

struct ConvArgs {
    const void *x;             // io dtype, rows at the strides below
    const float *weight;       // [C, W]
    const float *bias;         // [C] or NULL
    const void *init;          // [Bt, W-1, C] io dtype or NULL (fwd, bwd)
    const int32_t *lens;       // [Bt] or NULL (fwd)
    void *y[3];                // dense [Bt, T, ch[i]] io dtype (fwd, step)
    void *fin;                 // [Bt, W-1, C] io dtype or NULL (fwd)
    const int32_t *slots;      // [Bt] or NULL (step)
    void *state;               // [nslots, W-1, C] io dtype (step)
    int64_t nslots;
    const float *dy[3];        // dense [Bt, T, ch[i]] float32 (bwd)
    const float *dfinal;       // [Bt, W-1, C] or NULL (bwd)
    float *dx, *dweight, *dbias, *dinit;   // bwd outputs; dbias, dinit may be NULL
    float *part;               // bwd workspace
    int64_t Bt, T, sxb, sxt;   // batch and token strides of x, in elements
    int64_t C;                 // channels: the sum of ch
    int64_t ch[3];
    int W;
    bool silu, bf16;
};
hipError_t launch_conv1d_fwd(const ConvArgs &a, hipStream_t st);
hipError_t launch_conv1d_step(const ConvArgs &a, hipStream_t st);
hipError_t launch_conv1d_bwd(const ConvArgs &a, hipStream_t st);
size_t conv1d_bwd_workspace(const ConvArgs &a);
struct ConvLayout {
    int64_t fwd_run, bwd_run;   // tokens of a lane
    int step_rows;              // sequences of a lane
};
ConvLayout conv1d_layout(const ConvArgs &a);
// false: more workgroups than one launch holds
bool conv1d_fits(const ConvArgs &a);

struct CacheArgs {
    int64_t n, size, nslots;
    const int32_t *slots;   // [n], or NULL: state i in slot i
    void *codes;            // [nslots, size] 8-bit
    float *scales;          // [nslots, ceil(size / 64)]
    const float *src;       // write: [n, size]
    float *dst;             // read: [n, size]
    bool fp8;               // e4m3 codes (else int8)
};
bool cache_fits(const CacheArgs &a);   // false: more workgroups than one launch holds
hipError_t launch_cache_write(const CacheArgs &a, hipStream_t st);
hipError_t launch_cache_read(const CacheArgs &a, hipStream_t st);

struct SelArgs {
    const void *x, *dt, *B, *C, *z;   // [Bt, T, Dm] (B, C: [Bt, T, N]) io dtype; z NULL = no gate
    const float *A, *D;               // [Dm, N], [Dm]
    const float *dt_bias;             // [Dm] or NULL
    const float *init;                // [Bt, Dm, N] or NULL
    const int32_t *lens;              // [Bt] or NULL (fwd)
    void *y;                          // [Bt, T, Dm] float32, or io dtype with ybf (fwd, step)
    float *fin;                       // [Bt, Dm, N] or NULL (fwd)
    float *state;                     // [nslots, Dm, N] (step)
    const int32_t *slots;             // [Bt] or NULL (step)
    int64_t nslots;
    const float *dy, *dfinal;         // bwd
    float *dx, *ddt, *dA, *dB, *dC, *dD, *dbias, *dz, *dinit;   // bwd; dbias, dz, dinit may be NULL
    void *ws;
    int64_t Bt, T, Dm;
    int N;
    bool softplus, bf16, ybf;
};
// false: more workgroups than one launch holds
bool selective_scan_fits(const SelArgs &a);
bool selective_step_fits(const SelArgs &a);
bool selective_scan_bwd_fits(const SelArgs &a);
size_t selective_scan_workspace(const SelArgs &a);
struct SelLayout {
    int states;         // of a lane
    int64_t segments;   // of a sequence
};
SelLayout selective_scan_layout(const SelArgs &a);
SelLayout selective_scan_bwd_layout(const SelArgs &a);
int selective_step_channels(const SelArgs &a);   // of a lane
hipError_t launch_selective_scan(const SelArgs &a, hipStream_t st);
hipError_t launch_selective_step(const SelArgs &a, hipStream_t st);
size_t selective_scan_bwd_workspace(const SelArgs &a);
hipError_t launch_selective_scan_bwd(const SelArgs &a, hipStream_t st);

}  // namespace ssd
