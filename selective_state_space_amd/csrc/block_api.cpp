// C ABI of the further operators of a layer: linear attention with a decay for
// each head, the group norm behind a mixer, and projections with 4-bit weights.
// Every check runs on the host before the first HIP call, so a rejected call
// launches and writes nothing.

#include <hip/hip_runtime.h>
#include <math.h>

#include "../../include/ssd.h"
#include "block_launch.h"
#include "host_check.h"
#include "layer_launch.h"

namespace {

using ssd::fail;
using ssd::hip_result;
using ssd::kMaxDim;
using ssd::ok;

constexpr int64_t kMaxStride = int64_t(1) << 40;
constexpr int64_t kMaxTokenStride = int64_t(1) << 24;   // a chunk of tokens spans 32-bit offsets

ssd_status check_io(int32_t io) {
    if (io != SSD_F32 && io != SSD_BF16)
        return fail(SSD_ERR_UNSUPPORTED, "io_dtype = %d; only SSD_F32 (0) and SSD_BF16 (1)",
                    (int)io);
    return SSD_OK;
}

ssd_status check_range(const char *name, int64_t v, int64_t lo, int64_t hi) {
    if (v < lo || v > hi)
        return fail(SSD_ERR_SHAPE, "%s = %lld out of range [%lld, %lld]", name, (long long)v,
                    (long long)lo, (long long)hi);
    return SSD_OK;
}

#define CHECK(call)                          \
    do {                                     \
        const ssd_status r_ = (call);        \
        if (r_ != SSD_OK) return r_;         \
    } while (0)
// a pointer that is needed where there is something to read or write
#define PTR_IF(cond, p)           \
    do {                          \
        if (cond) REQUIRE_PTR(p); \
        else OPTIONAL_PTR(p);     \
    } while (0)

// strides of a tensor that is read 16 bytes at a time
ssd_status check_stride(const char *name, int64_t v, int64_t multiple, int64_t most = kMaxStride) {
    CHECK(check_range(name, v, 0, most));
    if (v % multiple)
        return fail(SSD_ERR_ALIGN, "%s = %lld is not a multiple of %lld elements (16 bytes)", name,
                    (long long)v, (long long)multiple);
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

// States that a launch writes at its workgroups' ends while others may still be to read theirs.
ssd_status check_states_apart(const char *out_name, const float *out, const char *in_name,
                              const float *in, const ssd::AttnArgs &a) {
    const uintptr_t o = reinterpret_cast<uintptr_t>(out), i = reinterpret_cast<uintptr_t>(in);
    const uint64_t bytes = (uint64_t)(a.Bt * a.H) * (uint64_t)(a.K * a.V) * sizeof(float);
    if (out && in && (o < i ? i - o : o - i) < bytes)
        return fail(SSD_ERR_UNSUPPORTED, "%s overlaps %s", out_name, in_name);
    return SSD_OK;
}

ssd_status check_attn(const ssd_attn_dims *d, bool need_seq, ssd::AttnArgs *a) {
    if (!d) return fail(SSD_ERR_NULL, "dims is NULL");
    CHECK(check_range("batch", d->batch, 0, kMaxDim));
    if (need_seq) CHECK(check_range("seqlen", d->seqlen, 0, kMaxDim));
    CHECK(check_range("nheads", d->nheads, 1, 65536));
    CHECK(check_range("ngroups", d->ngroups, 1, d->nheads));
    if (d->nheads % d->ngroups)
        return fail(SSD_ERR_SHAPE, "nheads %% ngroups != 0 (%lld, %lld)", (long long)d->nheads,
                    (long long)d->ngroups);
    for (const int64_t v : {d->dim_k, d->dim_v})
        if (v < 8 || v > 256 || v % 8)
            return fail(SSD_ERR_UNSUPPORTED, "dim_%c = %lld; multiples of 8 in [8, 256]",
                        v == d->dim_k ? 'k' : 'v', (long long)v);
    CHECK(check_io(d->io_dtype));
    if (!isfinite(d->scale)) return fail(SSD_ERR_SHAPE, "scale is not finite");
    const int64_t multiple = d->io_dtype == SSD_BF16 ? 8 : 4;
    CHECK(check_stride("q_batch_stride", d->q_batch_stride, multiple));
    CHECK(check_stride("k_batch_stride", d->k_batch_stride, multiple));
    CHECK(check_stride("v_batch_stride", d->v_batch_stride, multiple));
    if (need_seq) {
        CHECK(check_stride("q_token_stride", d->q_token_stride, multiple, kMaxTokenStride));
        CHECK(check_stride("k_token_stride", d->k_token_stride, multiple, kMaxTokenStride));
        CHECK(check_stride("v_token_stride", d->v_token_stride, multiple, kMaxTokenStride));
    }
    *a = ssd::AttnArgs{};
    a->Bt = d->batch;
    a->T = need_seq ? d->seqlen : 1;
    a->H = d->nheads;
    a->G = d->ngroups;
    a->K = (int)d->dim_k;
    a->V = (int)d->dim_v;
    a->qb = d->q_batch_stride;
    a->qt = d->q_token_stride;
    a->kb = d->k_batch_stride;
    a->kt = d->k_token_stride;
    a->vb = d->v_batch_stride;
    a->vt = d->v_token_stride;
    a->scale = d->scale;
    a->bf16 = d->io_dtype == SSD_BF16;
    if (!ssd::attn_fits(*a))
        return fail(SSD_ERR_SHAPE, "problem too large for one launch (batch %lld, seqlen %lld, "
                    "%lld heads)", (long long)a->Bt, (long long)a->T, (long long)a->H);
    return SSD_OK;
}

ssd_status check_norm(const ssd_norm_dims *d, ssd::NormArgs *a) {
    if (!d) return fail(SSD_ERR_NULL, "dims is NULL");
    CHECK(check_range("batch", d->batch, 0, kMaxDim));
    CHECK(check_range("seqlen", d->seqlen, 0, kMaxDim));
    CHECK(check_range("channels", d->channels, 1, int64_t(1) << 24));
    CHECK(check_range("groups", d->groups, 1, d->channels));
    if (d->channels % d->groups)
        return fail(SSD_ERR_SHAPE, "channels %% groups != 0 (%lld, %lld)", (long long)d->channels,
                    (long long)d->groups);
    if (d->channels / d->groups > 16384)
        return fail(SSD_ERR_UNSUPPORTED, "groups of %lld channels; at most 16384",
                    (long long)(d->channels / d->groups));
    CHECK(check_io(d->io_dtype));
    if (d->form < SSD_NORM_PLAIN || d->form > SSD_NORM_GATED_INPUT)
        return fail(SSD_ERR_UNSUPPORTED, "form = %d; an ssd_norm_form (0 to 3)", (int)d->form);
    if (!(d->eps > 0.f) || !isfinite(d->eps))
        return fail(SSD_ERR_SHAPE, "eps = %g; positive and finite", (double)d->eps);
    CHECK(check_range("x_batch_stride", d->x_batch_stride, 0, kMaxStride));
    CHECK(check_range("x_token_stride", d->x_token_stride, 0, kMaxStride));
    CHECK(check_range("z_batch_stride", d->z_batch_stride, 0, kMaxStride));
    CHECK(check_range("z_token_stride", d->z_token_stride, 0, kMaxStride));
    *a = ssd::NormArgs{};
    a->Bt = d->batch;
    a->T = d->seqlen;
    a->C = d->channels;
    a->groups = d->groups;
    a->xb = d->x_batch_stride;
    a->xt = d->x_token_stride;
    a->zb = d->z_batch_stride;
    a->zt = d->z_token_stride;
    a->eps = d->eps;
    a->form = d->form;
    a->rms = d->rms != 0;
    a->bf16 = d->io_dtype == SSD_BF16;
    if (!ssd::norm_fits(*a))
        return fail(SSD_ERR_SHAPE, "problem too large for one launch (batch %lld, seqlen %lld, "
                    "%lld groups)", (long long)a->Bt, (long long)a->T, (long long)a->groups);
    return SSD_OK;
}

// x and z, which need the alignment of their elements only
ssd_status check_norm_inputs(const void *x, const void *z, const ssd_norm_dims *d, bool tokens) {
    const uintptr_t off = d->io_dtype == SSD_BF16 ? 1u : 3u;
    const bool gated = d->form >= SSD_NORM_GATE;
    if (tokens && !x) return fail(SSD_ERR_NULL, "x is NULL");
    if (tokens && gated && !z) return fail(SSD_ERR_NULL, "z is NULL, and the form is gated");
    if (!gated && z) return fail(SSD_ERR_UNSUPPORTED, "z is given, and the form has no gate");
    if (reinterpret_cast<uintptr_t>(x) & off)
        return fail(SSD_ERR_ALIGN, "x is not aligned to its elements");
    if (reinterpret_cast<uintptr_t>(z) & off)
        return fail(SSD_ERR_ALIGN, "z is not aligned to its elements");
    return SSD_OK;
}

ssd_status check_w4(const ssd_w4_dims *d, bool linear, ssd::W4Args *a) {
    if (!d) return fail(SSD_ERR_NULL, "dims is NULL");
    if (linear) CHECK(check_range("rows", d->rows, 0, kMaxDim));
    if (d->group != 64 && d->group != 128)
        return fail(SSD_ERR_UNSUPPORTED, "group = %lld; only 64 and 128 are instantiated",
                    (long long)d->group);
    CHECK(check_range("inputs", d->inputs, d->group, int64_t(1) << 24));
    if (d->inputs % d->group)
        return fail(SSD_ERR_SHAPE, "inputs = %lld is not a multiple of group = %lld",
                    (long long)d->inputs, (long long)d->group);
    CHECK(check_range("outputs", d->outputs, 1, int64_t(1) << 24));
    CHECK(check_io(d->io_dtype));
    if (linear) CHECK(check_stride("x_row_stride", d->x_row_stride,
                                   d->io_dtype == SSD_BF16 ? 8 : 4, kMaxTokenStride));
    *a = ssd::W4Args{};
    a->rows = linear ? d->rows : 0;
    a->inputs = d->inputs;
    a->outputs = d->outputs;
    a->group = (int)d->group;
    a->xs = d->x_row_stride;
    a->bf16 = d->io_dtype == SSD_BF16;
    if (!ssd::w4_fits(*a))
        return fail(SSD_ERR_SHAPE, "problem too large for one launch (%lld rows, %lld inputs, "
                    "%lld outputs)", (long long)a->rows, (long long)a->inputs,
                    (long long)a->outputs);
    return SSD_OK;
}

}  // namespace

extern "C" {

size_t ssd_linear_attn_workspace_size(const ssd_attn_dims *dims) {
    ssd::AttnArgs a;
    if (check_attn(dims, true, &a) != SSD_OK) return 0;
    return ssd::attn_workspace(a);
}

size_t ssd_linear_attn_bwd_workspace_size(const ssd_attn_dims *dims) {
    ssd::AttnArgs a;
    if (check_attn(dims, true, &a) != SSD_OK) return 0;
    return ssd::attn_bwd_workspace(a);
}

ssd_status ssd_linear_attn_layout(const ssd_attn_dims *dims, ssd_attn_layout *layout) {
    if (!layout) return fail(SSD_ERR_NULL, "layout is NULL");
    ssd::AttnArgs a;
    CHECK(check_attn(dims, true, &a));
    const ssd::AttnLayout f = ssd::attn_layout(a), b = ssd::attn_bwd_layout(a);
    layout->fwd_cols = f.v_cols;
    layout->bwd_cols = b.v_cols;
    layout->fwd_segments = f.segments;
    layout->bwd_segments = b.segments;
    return ok();
}

ssd_status ssd_linear_attn_fwd(const void *q, const void *k, const void *v, const float *log_decay,
                               const float *init_state, const int32_t *seq_lens, void *y,
                               float *final_state, const ssd_attn_dims *dims, void *workspace,
                               size_t workspace_bytes, void *stream) {
    ssd::AttnArgs a;
    CHECK(check_attn(dims, true, &a));
    const bool tokens = a.Bt > 0 && a.T > 0;
    PTR_IF(tokens, q);
    PTR_IF(tokens, k);
    PTR_IF(tokens, v);
    PTR_IF(a.Bt > 0, log_decay);
    PTR_IF(tokens, y);
    OPTIONAL_PTR(init_state);
    OPTIONAL_PTR(seq_lens);
    OPTIONAL_PTR(final_state);
    CHECK(check_workspace(workspace, workspace_bytes, ssd::attn_workspace(a)));
    if (final_state != init_state)
        CHECK(check_states_apart("final_state", final_state, "init_state", init_state, a));
    if (a.Bt == 0 || (a.T == 0 && !final_state)) return ok();
    a.q = q;
    a.k = k;
    a.v = v;
    a.decay = log_decay;
    a.init = init_state;
    a.lens = seq_lens;
    a.y = y;
    a.fin = final_state;
    a.ws = workspace;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    CHECK(hip_result(ssd::launch_attn_fwd(a, st), "linear_attn_fwd", st));
    return ok();
}

ssd_status ssd_linear_attn_step(float *state, int64_t num_slots, const int32_t *slots,
                                const void *q_t, const void *k_t, const void *v_t,
                                const float *log_decay, void *y_t, const ssd_attn_dims *dims,
                                void *stream) {
    ssd::AttnArgs a;
    CHECK(check_attn(dims, false, &a));
    CHECK(check_range("num_slots", num_slots, 0, kMaxDim));
    if (!slots && num_slots < a.Bt)
        return fail(SSD_ERR_SHAPE, "slots is NULL and num_slots = %lld is below %lld sequences",
                    (long long)num_slots, (long long)a.Bt);
    PTR_IF(a.Bt > 0 && num_slots > 0, state);
    OPTIONAL_PTR(slots);
    PTR_IF(a.Bt > 0, q_t);
    PTR_IF(a.Bt > 0, k_t);
    PTR_IF(a.Bt > 0, v_t);
    PTR_IF(a.Bt > 0, log_decay);
    PTR_IF(a.Bt > 0, y_t);
    if (a.Bt == 0) return ok();
    a.state = state;
    a.nslots = num_slots;
    a.slots = slots;
    a.q = q_t;
    a.k = k_t;
    a.v = v_t;
    a.decay = log_decay;
    a.y = y_t;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    CHECK(hip_result(ssd::launch_attn_step(a, st), "linear_attn_step", st));
    return ok();
}

ssd_status ssd_linear_attn_bwd(const void *q, const void *k, const void *v, const float *log_decay,
                               const float *init_state, const int32_t *seq_lens, const void *dy,
                               const float *dfinal, void *dq, void *dk, void *dv, float *dinit,
                               const ssd_attn_dims *dims, void *workspace, size_t workspace_bytes,
                               void *stream) {
    ssd::AttnArgs a;
    CHECK(check_attn(dims, true, &a));
    const bool tokens = a.Bt > 0 && a.T > 0;
    PTR_IF(tokens, q);
    PTR_IF(tokens, k);
    PTR_IF(tokens, v);
    PTR_IF(a.Bt > 0, log_decay);
    PTR_IF(tokens, dy);
    PTR_IF(tokens, dq);
    PTR_IF(tokens, dk);
    PTR_IF(tokens, dv);
    OPTIONAL_PTR(init_state);
    OPTIONAL_PTR(seq_lens);
    OPTIONAL_PTR(dfinal);
    OPTIONAL_PTR(dinit);
    CHECK(check_workspace(workspace, workspace_bytes, ssd::attn_bwd_workspace(a)));
    CHECK(check_states_apart("dinit", dinit, "dfinal", dfinal, a));
    CHECK(check_states_apart("dinit", dinit, "init_state", init_state, a));
    if (a.Bt == 0 || (a.T == 0 && !dinit)) return ok();
    a.q = q;
    a.k = k;
    a.v = v;
    a.decay = log_decay;
    a.init = init_state;
    a.lens = seq_lens;
    a.dy = dy;
    a.dfinal = dfinal;
    a.dq = dq;
    a.dk = dk;
    a.dv = dv;
    a.dinit = dinit;
    a.ws = workspace;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    CHECK(hip_result(ssd::launch_attn_bwd(a, st), "linear_attn_bwd", st));
    return ok();
}

ssd_status ssd_group_norm_fwd(const void *x, const void *z, const float *weight, const float *bias,
                              const int32_t *seq_lens, void *y, const ssd_norm_dims *dims,
                              void *stream) {
    ssd::NormArgs a;
    CHECK(check_norm(dims, &a));
    const bool tokens = a.Bt > 0 && a.T > 0;
    CHECK(check_norm_inputs(x, z, dims, tokens));
    OPTIONAL_PTR(weight);
    OPTIONAL_PTR(bias);
    OPTIONAL_PTR(seq_lens);
    PTR_IF(tokens, y);
    if (!tokens) return ok();
    a.x = x;
    a.z = z;
    a.weight = weight;
    a.bias = bias;
    a.lens = seq_lens;
    a.y = y;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    CHECK(hip_result(ssd::launch_norm_fwd(a, st), "group_norm_fwd", st));
    return ok();
}

size_t ssd_group_norm_bwd_workspace_size(const ssd_norm_dims *dims) {
    ssd::NormArgs a;
    if (check_norm(dims, &a) != SSD_OK) return 0;
    return ssd::norm_bwd_workspace(a);
}

ssd_status ssd_group_norm_bwd(const void *x, const void *z, const float *weight, const float *bias,
                              const int32_t *seq_lens, const void *dy, void *dx, void *dz,
                              float *dweight, float *dbias, const ssd_norm_dims *dims,
                              void *workspace, size_t workspace_bytes, void *stream) {
    ssd::NormArgs a;
    CHECK(check_norm(dims, &a));
    const bool tokens = a.Bt > 0 && a.T > 0;
    CHECK(check_norm_inputs(x, z, dims, tokens));
    OPTIONAL_PTR(weight);
    OPTIONAL_PTR(bias);
    OPTIONAL_PTR(seq_lens);
    PTR_IF(tokens, dy);
    PTR_IF(tokens, dx);
    PTR_IF(tokens && dims->form >= SSD_NORM_GATE, dz);
    OPTIONAL_PTR(dweight);
    OPTIONAL_PTR(dbias);
    const bool sums = dweight || dbias;
    CHECK(check_workspace(workspace, workspace_bytes, sums ? ssd::norm_bwd_workspace(a) : 0));
    if (!tokens && !sums) return ok();
    a.x = x;
    a.z = z;
    a.weight = weight;
    a.bias = bias;
    a.lens = seq_lens;
    a.dy = dy;
    a.dx = dx;
    a.dz = dz;
    a.dweight = dweight;
    a.dbias = dbias;
    a.part = static_cast<float *>(workspace);
    const hipStream_t st = static_cast<hipStream_t>(stream);
    CHECK(hip_result(ssd::launch_norm_bwd(a, st), "group_norm_bwd", st));
    return ok();
}

ssd_status ssd_w4_quantize(const void *weight, void *codes, void *scales, const ssd_w4_dims *dims,
                           void *stream) {
    ssd::W4Args a;
    CHECK(check_w4(dims, false, &a));
    REQUIRE_PTR(weight);
    REQUIRE_PTR(codes);
    REQUIRE_PTR(scales);
    a.weight = weight;
    a.wcodes = static_cast<uint8_t *>(codes);
    a.wscales = static_cast<uint16_t *>(scales);
    const hipStream_t st = static_cast<hipStream_t>(stream);
    CHECK(hip_result(ssd::launch_w4_quantize(a, st), "w4_quantize", st));
    return ok();
}

ssd_status ssd_w4_dequantize(const void *codes, const void *scales, void *weight,
                             const ssd_w4_dims *dims, void *stream) {
    ssd::W4Args a;
    CHECK(check_w4(dims, false, &a));
    REQUIRE_PTR(codes);
    REQUIRE_PTR(scales);
    REQUIRE_PTR(weight);
    a.codes = static_cast<const uint8_t *>(codes);
    a.scales = static_cast<const uint16_t *>(scales);
    a.out = weight;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    CHECK(hip_result(ssd::launch_w4_dequantize(a, st), "w4_dequantize", st));
    return ok();
}

ssd_status ssd_w4_linear(const void *x, const void *codes, const void *scales, const float *bias,
                         void *y, const ssd_w4_dims *dims, void *stream) {
    ssd::W4Args a;
    CHECK(check_w4(dims, true, &a));
    PTR_IF(a.rows > 0, x);
    REQUIRE_PTR(codes);
    REQUIRE_PTR(scales);
    OPTIONAL_PTR(bias);
    PTR_IF(a.rows > 0, y);
    if (a.rows == 0) return ok();
    a.x = x;
    a.codes = static_cast<const uint8_t *>(codes);
    a.scales = static_cast<const uint16_t *>(scales);
    a.bias = bias;
    a.y = y;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    CHECK(hip_result(ssd::launch_w4_linear(a, st), "w4_linear", st));
    return ok();
}

}  // extern "C"
