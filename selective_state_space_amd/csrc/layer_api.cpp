// C ABI of the operators around the layer scan: the short causal convolution,
// the per-channel selective scan and the 8-bit state cache.  As for the scan,
// every check runs on the host before the first HIP call, so a rejected call
// launches and writes nothing.

#include <hip/hip_runtime.h>

#include "../../include/ssd.h"
#include "host_check.h"
#include "layer_launch.h"

namespace {

using ssd::fail;
using ssd::hip_result;
using ssd::kMaxDim;
using ssd::misaligned;
using ssd::ok;

ssd_status check_io(int32_t io) {
    if (io != SSD_F32 && io != SSD_BF16)
        return fail(SSD_ERR_UNSUPPORTED, "io_dtype = %d; only SSD_F32 (0) and SSD_BF16 (1)",
                    (int)io);
    return SSD_OK;
}

// element-aligned pointers (x of the convolution: a slice may start anywhere)
bool off_element(const void *p, int32_t io) {
    return reinterpret_cast<uintptr_t>(p) & (io == SSD_BF16 ? 1u : 3u);
}

ssd_status check_conv(const ssd_conv_dims *d, bool need_seq, ssd::ConvArgs *a) {
    if (!d) return fail(SSD_ERR_NULL, "dims is NULL");
    if (d->batch < 0 || d->batch > kMaxDim)
        return fail(SSD_ERR_SHAPE, "batch = %lld out of range [0, 2^30]", (long long)d->batch);
    if (need_seq && (d->seqlen < 0 || d->seqlen > kMaxDim))
        return fail(SSD_ERR_SHAPE, "seqlen = %lld out of range [0, 2^30]", (long long)d->seqlen);
    if (d->width < 2 || d->width > 4)
        return fail(SSD_ERR_UNSUPPORTED, "width = %lld; only 2, 3 and 4 taps are instantiated",
                    (long long)d->width);
    *a = ssd::ConvArgs{};
    for (int i = 0; i < 3; ++i) {
        if (d->channels[i] < (i == 0 ? 1 : 0) || d->channels[i] > (int64_t(1) << 24))
            return fail(SSD_ERR_SHAPE, "channels[%d] = %lld out of range [%d, 2^24]", i,
                        (long long)d->channels[i], i == 0 ? 1 : 0);
        a->ch[i] = d->channels[i];
        a->C += d->channels[i];
    }
    const int64_t most = int64_t(1) << 40;
    if (d->x_batch_stride < 0 || d->x_batch_stride > most || d->x_token_stride < 0 ||
        d->x_token_stride > most)
        return fail(SSD_ERR_SHAPE, "x strides %lld, %lld out of range [0, 2^40]",
                    (long long)d->x_batch_stride, (long long)d->x_token_stride);
    const ssd_status r = check_io(d->io_dtype);
    if (r != SSD_OK) return r;
    a->Bt = d->batch;
    a->T = need_seq ? d->seqlen : 1;
    a->W = (int)d->width;
    a->sxb = d->x_batch_stride;
    a->sxt = d->x_token_stride;
    a->silu = d->silu != 0;
    a->bf16 = d->io_dtype == SSD_BF16;
    if (a->Bt > 0 && !ssd::conv1d_fits(*a))
        return fail(SSD_ERR_SHAPE, "problem too large for one launch (batch %lld, seqlen %lld, "
                    "%lld channels)", (long long)a->Bt, (long long)a->T, (long long)a->C);
    return SSD_OK;
}

// y[3] or dy[3]: one dense 16-byte aligned tensor per channel group that has channels
ssd_status check_parts(const void *const *p, const char *name, const ssd::ConvArgs &a, bool need) {
    if (!p) return fail(SSD_ERR_NULL, "%s is NULL", name);
    for (int i = 0; i < 3; ++i) {
        if (need && a.ch[i] > 0 && !p[i]) return fail(SSD_ERR_NULL, "%s[%d] is NULL", name, i);
        if (misaligned(p[i]))
            return fail(SSD_ERR_ALIGN, "%s[%d] is not 16-byte aligned", name, i);
    }
    return SSD_OK;
}

ssd_status check_slots(const int32_t *slots, int64_t num_slots, int64_t n) {
    if (num_slots < 0 || num_slots > kMaxDim)
        return fail(SSD_ERR_SHAPE, "num_slots = %lld out of range [0, 2^30]",
                    (long long)num_slots);
    if (!slots && num_slots < n)
        return fail(SSD_ERR_SHAPE, "slots is NULL and num_slots = %lld is below %lld sequences",
                    (long long)num_slots, (long long)n);
    OPTIONAL_PTR(slots);
    return SSD_OK;
}

ssd_status check_scan(const ssd_scan_dims *d, bool need_seq, const ssd_layer_opts *o,
                      bool (*fits)(const ssd::SelArgs &), ssd::SelArgs *a) {
    if (!d) return fail(SSD_ERR_NULL, "dims is NULL");
    if (d->batch < 0 || d->batch > kMaxDim)
        return fail(SSD_ERR_SHAPE, "batch = %lld out of range [0, 2^30]", (long long)d->batch);
    if (need_seq && (d->seqlen < 0 || d->seqlen > kMaxDim))
        return fail(SSD_ERR_SHAPE, "seqlen = %lld out of range [0, 2^30]", (long long)d->seqlen);
    if (d->dim < 1 || d->dim > (int64_t(1) << 22))
        return fail(SSD_ERR_SHAPE, "dim = %lld out of range [1, 2^22]", (long long)d->dim);
    if (d->dstate != 8 && d->dstate != 16 && d->dstate != 32 && d->dstate != 64)
        return fail(SSD_ERR_UNSUPPORTED, "dstate = %lld; only 8, 16, 32 and 64 are instantiated",
                    (long long)d->dstate);
    ssd_status r = check_io(d->io_dtype);
    if (r != SSD_OK) return r;
    *a = ssd::SelArgs{};
    a->Bt = d->batch;
    a->T = need_seq ? d->seqlen : 1;
    a->Dm = d->dim;
    a->N = (int)d->dstate;
    a->bf16 = d->io_dtype == SSD_BF16;
    if (o) {
        if (o->y_io_dtype != 0 && o->y_io_dtype != 1)
            return fail(SSD_ERR_UNSUPPORTED, "ssd_layer_opts.y_io_dtype = %d; 0 or 1",
                        (int)o->y_io_dtype);
        if (misaligned(o->dt_bias)) return fail(SSD_ERR_ALIGN, "dt_bias is not 16-byte aligned");
        if (misaligned(o->z)) return fail(SSD_ERR_ALIGN, "z is not 16-byte aligned");
        a->dt_bias = o->dt_bias;
        a->softplus = o->dt_softplus != 0;
        a->ybf = a->bf16 && o->y_io_dtype != 0;
        a->z = o->z;
    }
    if (!fits(*a))
        return fail(SSD_ERR_SHAPE, "problem too large for one launch (batch %lld, seqlen %lld, "
                    "dim %lld)", (long long)a->Bt, (long long)a->T, (long long)a->Dm);
    return SSD_OK;
}

ssd_status check_workspace(void *workspace, size_t bytes, size_t need) {
    if (need && !workspace)
        return fail(SSD_ERR_NULL, "workspace is NULL (%zu bytes needed)", need);
    OPTIONAL_PTR(workspace);
    if (bytes < need)
        return fail(SSD_ERR_WORKSPACE, "workspace_bytes = %zu < %zu required", bytes, need);
    return SSD_OK;
}

// a pointer that is needed where there is something to read or write
#define PTR_IF(cond, p)          \
    do {                         \
        if (cond) REQUIRE_PTR(p); \
        else OPTIONAL_PTR(p);    \
    } while (0)

ssd_status check_cache(int64_t n, int64_t size, const int32_t *slots, int64_t num_slots,
                       int32_t format, ssd::CacheArgs *a) {
    if (n < 0 || n > kMaxDim)
        return fail(SSD_ERR_SHAPE, "n = %lld out of range [0, 2^30]", (long long)n);
    if (size < 8 || size % 8 || size > (int64_t(1) << 34))
        return fail(SSD_ERR_SHAPE, "size = %lld; a multiple of 8 in [8, 2^34]", (long long)size);
    if (format != SSD_CACHE_INT8 && format != SSD_CACHE_FP8)
        return fail(SSD_ERR_UNSUPPORTED,
                    "format = %d; only SSD_CACHE_INT8 (0) and SSD_CACHE_FP8 (1)", (int)format);
    const ssd_status r = check_slots(slots, num_slots, n);
    if (r != SSD_OK) return r;
    a->n = n;
    a->size = size;
    if (!ssd::cache_fits(*a))
        return fail(SSD_ERR_SHAPE, "n * size = %lld * %lld too large for one launch", (long long)n,
                    (long long)size);
    a->slots = slots;
    a->nslots = num_slots;
    a->fp8 = format == SSD_CACHE_FP8;
    return SSD_OK;
}

}  // namespace

extern "C" {

ssd_status ssd_conv1d_fwd(const void *x, const float *weight, const float *bias,
                          const void *init_state, const int32_t *seq_lens, void *const y[3],
                          void *final_state, const ssd_conv_dims *dims, void *stream) {
    ssd::ConvArgs a;
    ssd_status r = check_conv(dims, true, &a);
    if (r != SSD_OK) return r;
    const bool tokens = a.Bt > 0 && a.T > 0;
    if (tokens && !x) return fail(SSD_ERR_NULL, "x is NULL");
    if (off_element(x, dims->io_dtype))
        return fail(SSD_ERR_ALIGN, "x is not aligned to its elements");
    REQUIRE_PTR(weight);
    OPTIONAL_PTR(bias);
    OPTIONAL_PTR(init_state);
    OPTIONAL_PTR(seq_lens);
    OPTIONAL_PTR(final_state);
    if ((r = check_parts(y, "y", a, tokens)) != SSD_OK) return r;
    if (a.Bt == 0 || (a.T == 0 && !final_state)) return ok();
    a.x = x;
    a.weight = weight;
    a.bias = bias;
    a.init = init_state;
    a.lens = seq_lens;
    for (int i = 0; i < 3; ++i) a.y[i] = y[i];
    a.fin = final_state;
    r = hip_result(ssd::launch_conv1d_fwd(a, static_cast<hipStream_t>(stream)), "conv1d_fwd",
                   static_cast<hipStream_t>(stream));
    if (r != SSD_OK) return r;
    return ok();
}

ssd_status ssd_conv1d_step(void *conv_state, int64_t num_slots, const int32_t *slots,
                           const void *x_t, const float *weight, const float *bias,
                           void *const y_t[3], const ssd_conv_dims *dims, void *stream) {
    ssd::ConvArgs a;
    ssd_status r = check_conv(dims, false, &a);
    if (r != SSD_OK) return r;
    if ((r = check_slots(slots, num_slots, a.Bt)) != SSD_OK) return r;
    if (a.Bt > 0) {
        REQUIRE_PTR(conv_state);
        REQUIRE_PTR(weight);
        if (!x_t) return fail(SSD_ERR_NULL, "x_t is NULL");
    }
    if (off_element(x_t, dims->io_dtype))
        return fail(SSD_ERR_ALIGN, "x_t is not aligned to its elements");
    OPTIONAL_PTR(bias);
    if ((r = check_parts(y_t, "y_t", a, a.Bt > 0)) != SSD_OK) return r;
    if (a.Bt == 0) return ok();
    a.x = x_t;
    a.weight = weight;
    a.bias = bias;
    a.state = conv_state;
    a.slots = slots;
    a.nslots = num_slots;
    for (int i = 0; i < 3; ++i) a.y[i] = y_t[i];
    r = hip_result(ssd::launch_conv1d_step(a, static_cast<hipStream_t>(stream)), "conv1d_step",
                   static_cast<hipStream_t>(stream));
    if (r != SSD_OK) return r;
    return ok();
}

size_t ssd_conv1d_bwd_workspace_size(const ssd_conv_dims *dims) {
    ssd::ConvArgs a;
    if (check_conv(dims, true, &a) != SSD_OK) return 0;
    return ssd::conv1d_bwd_workspace(a);
}

ssd_status ssd_conv1d_layout(const ssd_conv_dims *dims, ssd_conv_layout *layout) {
    if (!layout) return fail(SSD_ERR_NULL, "layout is NULL");
    ssd::ConvArgs a;
    const ssd_status r = check_conv(dims, true, &a);
    if (r != SSD_OK) return r;
    const ssd::ConvLayout l = ssd::conv1d_layout(a);
    layout->fwd_run = (int32_t)l.fwd_run;
    layout->bwd_run = (int32_t)l.bwd_run;
    layout->step_rows = l.step_rows;
    return ok();
}

ssd_status ssd_conv1d_bwd(const void *x, const float *weight, const float *bias,
                          const void *init_state, const float *const dy[3], const float *dfinal,
                          float *dx, float *dweight, float *dbias, float *dinit,
                          const ssd_conv_dims *dims, void *workspace, size_t workspace_bytes,
                          void *stream) {
    ssd::ConvArgs a;
    ssd_status r = check_conv(dims, true, &a);
    if (r != SSD_OK) return r;
    const bool tokens = a.Bt > 0 && a.T > 0;
    if (tokens && !x) return fail(SSD_ERR_NULL, "x is NULL");
    PTR_IF(tokens, dx);
    if (off_element(x, dims->io_dtype))
        return fail(SSD_ERR_ALIGN, "x is not aligned to its elements");
    REQUIRE_PTR(weight);
    REQUIRE_PTR(dweight);
    OPTIONAL_PTR(bias);
    OPTIONAL_PTR(init_state);
    OPTIONAL_PTR(dfinal);
    OPTIONAL_PTR(dbias);
    OPTIONAL_PTR(dinit);
    if ((r = check_parts(reinterpret_cast<const void *const *>(dy), "dy", a, tokens)) != SSD_OK)
        return r;
    if ((r = check_workspace(workspace, workspace_bytes, ssd::conv1d_bwd_workspace(a))) != SSD_OK)
        return r;
    a.x = x;
    a.weight = weight;
    a.bias = bias;
    a.init = init_state;
    for (int i = 0; i < 3; ++i) a.dy[i] = dy[i];
    a.dfinal = dfinal;
    a.dx = dx;
    a.dweight = dweight;
    a.dbias = dbias;
    a.dinit = dinit;
    a.part = static_cast<float *>(workspace);
    r = hip_result(ssd::launch_conv1d_bwd(a, static_cast<hipStream_t>(stream)), "conv1d_bwd",
                   static_cast<hipStream_t>(stream));
    if (r != SSD_OK) return r;
    return ok();
}

size_t ssd_selective_scan_workspace_size(const ssd_scan_dims *dims) {
    ssd::SelArgs a;
    if (check_scan(dims, true, nullptr, ssd::selective_scan_fits, &a) != SSD_OK) return 0;
    return ssd::selective_scan_workspace(a);
}

ssd_status ssd_selective_scan_fwd(const void *x, const void *dt, const float *A, const void *B,
                                  const void *C, const float *D, const float *init_state,
                                  const int32_t *seq_lens, void *y, float *final_state,
                                  const ssd_layer_opts *opts, const ssd_scan_dims *dims,
                                  void *workspace, size_t workspace_bytes, void *stream) {
    ssd::SelArgs a;
    ssd_status r = check_scan(dims, true, opts, ssd::selective_scan_fits, &a);
    if (r != SSD_OK) return r;
    const bool tokens = a.Bt > 0 && a.T > 0;
    PTR_IF(tokens, x);
    PTR_IF(tokens, dt);
    PTR_IF(a.Bt > 0, A);
    PTR_IF(tokens, B);
    PTR_IF(tokens, C);
    PTR_IF(a.Bt > 0, D);
    PTR_IF(tokens, y);
    OPTIONAL_PTR(init_state);
    OPTIONAL_PTR(seq_lens);
    OPTIONAL_PTR(final_state);
    if ((r = check_workspace(workspace, workspace_bytes, ssd::selective_scan_workspace(a))) !=
        SSD_OK)
        return r;
    if (a.Bt == 0) return ok();
    a.x = x;
    a.dt = dt;
    a.A = A;
    a.B = B;
    a.C = C;
    a.D = D;
    a.init = init_state;
    a.lens = seq_lens;
    a.y = y;
    a.fin = final_state;
    a.ws = workspace;
    r = hip_result(ssd::launch_selective_scan(a, static_cast<hipStream_t>(stream)),
                   "selective_scan_fwd", static_cast<hipStream_t>(stream));
    if (r != SSD_OK) return r;
    return ok();
}

ssd_status ssd_selective_scan_step(float *state, int64_t num_slots, const int32_t *slots,
                                   const void *x_t, const void *dt_t, const float *A,
                                   const void *B_t, const void *C_t, const float *D, void *y_t,
                                   const ssd_layer_opts *opts, const ssd_scan_dims *dims,
                                   void *stream) {
    ssd::SelArgs a;
    ssd_status r = check_scan(dims, false, opts, ssd::selective_step_fits, &a);
    if (r != SSD_OK) return r;
    if ((r = check_slots(slots, num_slots, a.Bt)) != SSD_OK) return r;
    PTR_IF(a.Bt > 0, state);
    PTR_IF(a.Bt > 0, x_t);
    PTR_IF(a.Bt > 0, dt_t);
    PTR_IF(a.Bt > 0, A);
    PTR_IF(a.Bt > 0, B_t);
    PTR_IF(a.Bt > 0, C_t);
    PTR_IF(a.Bt > 0, D);
    PTR_IF(a.Bt > 0, y_t);
    if (a.Bt == 0) return ok();
    a.state = state;
    a.slots = slots;
    a.nslots = num_slots;
    a.x = x_t;
    a.dt = dt_t;
    a.A = A;
    a.B = B_t;
    a.C = C_t;
    a.D = D;
    a.y = y_t;
    r = hip_result(ssd::launch_selective_step(a, static_cast<hipStream_t>(stream)),
                   "selective_scan_step", static_cast<hipStream_t>(stream));
    if (r != SSD_OK) return r;
    return ok();
}

size_t ssd_selective_scan_bwd_workspace_size(const ssd_scan_dims *dims) {
    ssd::SelArgs a;
    if (check_scan(dims, true, nullptr, ssd::selective_scan_bwd_fits, &a) != SSD_OK) return 0;
    return ssd::selective_scan_bwd_workspace(a);
}

ssd_status ssd_selective_scan_layout(const ssd_scan_dims *dims, ssd_scan_layout *layout) {
    if (!layout) return fail(SSD_ERR_NULL, "layout is NULL");
    ssd::SelArgs a;
    const ssd_status r = check_scan(dims, true, nullptr, ssd::selective_scan_fits, &a);
    if (r != SSD_OK) return r;
    const ssd::SelLayout f = ssd::selective_scan_layout(a), b = ssd::selective_scan_bwd_layout(a);
    layout->fwd_states = f.states;
    layout->fwd_segments = f.segments;
    layout->bwd_states = b.states;
    layout->bwd_segments = b.segments;
    layout->step_channels = ssd::selective_step_channels(a);
    return ok();
}

ssd_status ssd_selective_scan_bwd(const void *x, const void *dt, const float *A, const void *B,
                                  const void *C, const float *D, const float *init_state,
                                  const float *dy, const float *dfinal, float *dx, float *ddt,
                                  float *dA, float *dB, float *dC, float *dD, float *ddt_bias,
                                  float *dz, float *dinit, const ssd_layer_opts *opts,
                                  const ssd_scan_dims *dims, void *workspace,
                                  size_t workspace_bytes, void *stream) {
    ssd::SelArgs a;
    ssd_status r = check_scan(dims, true, opts, ssd::selective_scan_bwd_fits, &a);
    if (r != SSD_OK) return r;
    const bool tokens = a.Bt > 0 && a.T > 0;
    PTR_IF(tokens, x);
    PTR_IF(tokens, dt);
    PTR_IF(a.Bt > 0, A);
    PTR_IF(tokens, B);
    PTR_IF(tokens, C);
    PTR_IF(a.Bt > 0, D);
    PTR_IF(tokens, dy);
    PTR_IF(tokens, dx);
    PTR_IF(tokens, ddt);
    REQUIRE_PTR(dA);
    PTR_IF(tokens, dB);
    PTR_IF(tokens, dC);
    REQUIRE_PTR(dD);
    PTR_IF(tokens && a.z, dz);
    OPTIONAL_PTR(init_state);
    OPTIONAL_PTR(dfinal);
    OPTIONAL_PTR(ddt_bias);
    OPTIONAL_PTR(dinit);
    if ((r = check_workspace(workspace, workspace_bytes, ssd::selective_scan_bwd_workspace(a))) !=
        SSD_OK)
        return r;
    a.x = x;
    a.dt = dt;
    a.A = A;
    a.B = B;
    a.C = C;
    a.D = D;
    a.init = init_state;
    a.dy = dy;
    a.dfinal = dfinal;
    a.dx = dx;
    a.ddt = ddt;
    a.dA = dA;
    a.dB = dB;
    a.dC = dC;
    a.dD = dD;
    a.dbias = ddt_bias;
    a.dz = dz;
    a.dinit = dinit;
    a.ws = workspace;
    r = hip_result(ssd::launch_selective_scan_bwd(a, static_cast<hipStream_t>(stream)),
                   "selective_scan_bwd", static_cast<hipStream_t>(stream));
    if (r != SSD_OK) return r;
    return ok();
}

ssd_status ssd_cache_write(const float *state, int64_t n, int64_t size, const int32_t *slots,
                           int64_t num_slots, void *codes, float *scales, int32_t format,
                           void *stream) {
    ssd::CacheArgs a{};
    ssd_status r = check_cache(n, size, slots, num_slots, format, &a);
    if (r != SSD_OK) return r;
    PTR_IF(n > 0, state);
    PTR_IF(n > 0, codes);
    PTR_IF(n > 0, scales);
    if (n == 0) return ok();
    a.src = state;
    a.codes = codes;
    a.scales = scales;
    r = hip_result(ssd::launch_cache_write(a, static_cast<hipStream_t>(stream)), "cache_write",
                   static_cast<hipStream_t>(stream));
    if (r != SSD_OK) return r;
    return ok();
}

ssd_status ssd_cache_read(const void *codes, const float *scales, int64_t n, int64_t size,
                          const int32_t *slots, int64_t num_slots, float *state, int32_t format,
                          void *stream) {
    ssd::CacheArgs a{};
    ssd_status r = check_cache(n, size, slots, num_slots, format, &a);
    if (r != SSD_OK) return r;
    PTR_IF(n > 0, state);
    PTR_IF(n > 0, codes);
    PTR_IF(n > 0, scales);
    if (n == 0) return ok();
    a.codes = const_cast<void *>(codes);
    a.scales = const_cast<float *>(scales);
    a.dst = state;
    r = hip_result(ssd::launch_cache_read(a, static_cast<hipStream_t>(stream)), "cache_read",
                   static_cast<hipStream_t>(stream));
    if (r != SSD_OK) return r;
    return ok();
}

}  // extern "C"
