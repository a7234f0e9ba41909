// C ABI of the operators around the scan: argument validation and dispatch of
// the short causal convolution, the selective scan and the group normalisation.
// The contract of every entry point is in include/ssd.h.
#include "../../include/ssd.h"
#include "ssd_checks.h"
#include "ssd_internal.h"

namespace ssd {

// a tensor argument: its address and the bytes it covers
struct Span {
    const void* p;
    size_t n;
};

// every base 16-byte aligned; no output overlaps an input or another output
template <size_t NI, size_t NO>
static ssd_status_t check_spans(const Span (&in)[NI], const Span (&out)[NO]) {
    for (const Span& r : in)
        if (r.p && !aligned16(r.p)) return SSD_ERR_ALIGNMENT;
    for (const Span& r : out)
        if (r.p && !aligned16(r.p)) return SSD_ERR_ALIGNMENT;
    for (size_t i = 0; i < NO; ++i) {
        for (const Span& r : in)
            if (overlaps(out[i].p, out[i].n, r.p, r.n)) return SSD_ERR_INVALID_ARG;
        for (size_t j = i + 1; j < NO; ++j)
            if (overlaps(out[i].p, out[i].n, out[j].p, out[j].n)) return SSD_ERR_INVALID_ARG;
    }
    return SSD_OK;
}

// the workspace: large enough, 256-byte aligned, apart from every argument
template <size_t NI, size_t NO>
static ssd_status_t check_workspace(const void* ws, size_t bytes, size_t need, const Span (&in)[NI],
                                    const Span (&out)[NO]) {
    if (need && (!ws || bytes < need)) return SSD_ERR_WORKSPACE;
    if ((uintptr_t)ws & 255u) return SSD_ERR_ALIGNMENT;
    for (const Span& r : in)
        if (overlaps(ws, need, r.p, r.n)) return SSD_ERR_INVALID_ARG;
    for (const Span& r : out)
        if (overlaps(ws, need, r.p, r.n)) return SSD_ERR_INVALID_ARG;
    return SSD_OK;
}

// bytes that `rows` strided rows of `width` elements cover
static size_t rows_bytes(int64_t rows, int64_t stride, int64_t width, size_t e) {
    return rows == 0 ? 0 : ((size_t)(rows - 1) * (size_t)stride + (size_t)width) * e;
}

constexpr int64_t kMaxChannels = (int64_t)1 << 20, kMaxStride = (int64_t)1 << 40, kMaxElements = (int64_t)1 << 60;
constexpr int64_t kMaxBatch = (int64_t)1 << 24, kMaxLen = (int64_t)1 << 30, kMaxBlocks = (int64_t)1 << 31;

// strided rows: offsets and byte counts stay within 64 bits
static bool rows_fit(int64_t rows, int64_t stride) {
    return stride <= kMaxStride && (rows == 0 || stride <= kMaxElements / rows);
}

static ssd_status_t check_conv1d_desc(const ssd_conv1d_desc_t* d, bool backward) {
    if (!d) return SSD_ERR_INVALID_ARG;
    if (d->batch < 0 || d->seqlen < 0 || d->channels < 1 || d->split1 < 0 || d->split2 < 0) return SSD_ERR_INVALID_ARG;
    if (!valid_dtype(d->io_dtype) || !valid_dtype(d->y_dtype) || !valid_dtype(d->state_dtype))
        return SSD_ERR_INVALID_ARG;
    if (d->activation != 0 && d->activation != 1) return SSD_ERR_INVALID_ARG;
    if (d->channels > kMaxChannels) return SSD_ERR_UNSUPPORTED;
    if (d->split1 > d->channels || d->split2 > d->channels || d->split1 + d->split2 >= d->channels ||
        (d->split1 == 0 && d->split2 != 0) || d->x_stride < d->channels || (backward && d->dx_stride < d->channels))
        return SSD_ERR_INVALID_ARG;
    if (d->width < 2 || d->width > 4 || d->channels % 8 || d->split1 % 8 || d->split2 % 8 || d->x_stride % 8 ||
        (backward && d->dx_stride % 8))
        return SSD_ERR_UNSUPPORTED;
    if (d->batch > kMaxBatch || d->seqlen > kMaxLen) return SSD_ERR_UNSUPPORTED;
    if (d->batch * (d->seqlen / 16 + 1) >= kMaxBlocks || conv1d_blocks(d->batch, d->seqlen, d->channels) >= kMaxBlocks)
        return SSD_ERR_UNSUPPORTED;
    const int64_t rows = d->batch * d->seqlen;
    if (!rows_fit(rows, d->x_stride) || (backward && !rows_fit(rows, d->dx_stride))) return SSD_ERR_UNSUPPORTED;
    return SSD_OK;
}

static Conv1dArgs conv1d_args(const ssd_conv1d_desc_t* d, const void* x, const float* w, const float* bias) {
    Conv1dArgs a{};
    a.batch = d->batch; a.L = d->seqlen; a.D = d->channels; a.W = d->width; a.xs = d->x_stride; a.dxs = d->dx_stride;
    a.part[0] = d->channels - d->split1 - d->split2; a.part[1] = d->split1; a.part[2] = d->split2;
    a.io_bf16 = d->io_dtype == SSD_BF16; a.y_bf16 = d->y_dtype == SSD_BF16; a.state_bf16 = d->state_dtype == SSD_BF16;
    a.silu = d->activation == 1;
    a.x = x; a.w = w; a.bias = bias;
    return a;
}

static ssd_status_t status_of(cudaError_t e) { return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA; }

static ssd_status_t check_selective_desc(const ssd_selective_desc_t* d, bool gated) {
    if (!d) return SSD_ERR_INVALID_ARG;
    if (d->batch < 0 || d->seqlen < 0 || d->channels < 1 || d->dstate < 1 || d->ngroups < 1 ||
        d->channels % d->ngroups != 0)
        return SSD_ERR_INVALID_ARG;
    if (!valid_dtype(d->io_dtype) || !valid_dtype(d->y_dtype) || !valid_dtype(d->state_dtype))
        return SSD_ERR_INVALID_ARG;
    if (gated && d->z_stride < d->channels) return SSD_ERR_INVALID_ARG;
    if (d->channels > kMaxChannels || (d->channels / d->ngroups) % 8 || d->dstate % 8 || d->dstate > 256)
        return SSD_ERR_UNSUPPORTED;
    if (gated && d->z_stride % 8) return SSD_ERR_UNSUPPORTED;
    if (d->batch > kMaxBatch || d->seqlen > kMaxLen || d->batch * (d->seqlen / 8 + 1) >= kMaxBlocks)
        return SSD_ERR_UNSUPPORTED;
    if (d->batch * (d->seqlen / 8 + 1) * d->ngroups >= kMaxBlocks ||
        selective_blocks(d->batch, d->seqlen, d->channels, d->dstate, d->ngroups) >= kMaxBlocks ||
        selective_bwd_blocks(d->batch, d->seqlen, d->channels, d->dstate, d->ngroups) >= kMaxBlocks)
        return SSD_ERR_UNSUPPORTED;
    if (gated && !rows_fit(d->batch * d->seqlen, d->z_stride)) return SSD_ERR_UNSUPPORTED;
    return SSD_OK;
}

static SelectiveArgs selective_args(const ssd_selective_desc_t* d) {
    SelectiveArgs a{};
    a.batch = d->batch; a.L = d->seqlen; a.D = d->channels; a.N = d->dstate; a.G = d->ngroups; a.zs = d->z_stride;
    a.io_bf16 = d->io_dtype == SSD_BF16; a.y_bf16 = d->y_dtype == SSD_BF16; a.state_bf16 = d->state_dtype == SSD_BF16;
    return a;
}

static ssd_status_t check_norm_desc(const ssd_group_norm_desc_t* d) {
    if (!d) return SSD_ERR_INVALID_ARG;
    if (d->rows < 0 || d->channels < 1 || d->ngroups < 1 || d->channels % d->ngroups != 0) return SSD_ERR_INVALID_ARG;
    if (!valid_dtype(d->x_dtype) || !valid_dtype(d->io_dtype) || !valid_dtype(d->y_dtype)) return SSD_ERR_INVALID_ARG;
    if (d->center != 0 && d->center != 1) return SSD_ERR_INVALID_ARG;
    if (d->activation < SSD_NORM_NONE || d->activation > SSD_NORM_GATE_BEFORE) return SSD_ERR_INVALID_ARG;
    if (!(d->eps > 0.f) || d->eps > 1e30f) return SSD_ERR_INVALID_ARG;
    const bool gated = d->activation >= SSD_NORM_GATE_AFTER;
    if (gated && d->z_stride < d->channels) return SSD_ERR_INVALID_ARG;
    const int64_t gs = d->channels / d->ngroups;
    if (d->channels > kMaxChannels || gs % 8 || gs > 16384) return SSD_ERR_UNSUPPORTED;
    if (gated && d->z_stride % 8) return SSD_ERR_UNSUPPORTED;
    if (d->rows > ((int64_t)1 << 38) || (gated && !rows_fit(d->rows, d->z_stride))) return SSD_ERR_UNSUPPORTED;
    return SSD_OK;
}

static GroupNormArgs norm_args(const ssd_group_norm_desc_t* d, const void* x, const void* z, const float* w,
                               const float* bias) {
    GroupNormArgs a{};
    a.rows = d->rows; a.C = d->channels; a.G = d->ngroups; a.zs = d->z_stride; a.eps = d->eps;
    a.x_bf16 = d->x_dtype == SSD_BF16; a.io_bf16 = d->io_dtype == SSD_BF16; a.y_bf16 = d->y_dtype == SSD_BF16;
    a.center = d->center != 0; a.act = d->activation;
    a.x = x; a.z = z; a.w = w; a.bias = bias;
    return a;
}

}  // namespace ssd

using namespace ssd;

extern "C" {

ssd_status_t ssd_conv1d_fwd(const ssd_conv1d_desc_t* d, const void* x, const float* weight, const float* bias,
                            const void* init_state, const int32_t* pad_left, void* y0, void* y1, void* y2,
                            void* final_state, void* stream) {
    ssd_status_t st = check_conv1d_desc(d, false);
    if (st != SSD_OK) return st;
    const bool empty = d->batch == 0 || d->seqlen == 0;
    if (!weight || (!empty && (!x || !y0))) return SSD_ERR_INVALID_ARG;
    if ((!empty && d->split1 && !y1) || (!d->split1 && y1) || (!empty && d->split2 && !y2) || (!d->split2 && y2))
        return SSD_ERR_INVALID_ARG;
    if ((uintptr_t)pad_left & 3u) return SSD_ERR_ALIGNMENT;
    const int64_t tok = d->batch * d->seqlen;
    const size_t e = dsize(d->y_dtype), keep = (size_t)d->batch * (d->width - 1) * d->channels * dsize(d->state_dtype);
    const Span in[] = {{x, rows_bytes(tok, d->x_stride, d->channels, dsize(d->io_dtype))},
                       {weight, sizeof(float) * d->channels * d->width}, {bias, sizeof(float) * d->channels},
                       {init_state, keep}};
    const Span out[] = {{y0, (size_t)tok * (d->channels - d->split1 - d->split2) * e},
                        {y1, (size_t)tok * d->split1 * e}, {y2, (size_t)tok * d->split2 * e}, {final_state, keep}};
    st = check_spans(in, out);
    if (st != SSD_OK) return st;
    for (const Span& r : out)
        if (overlaps(r.p, r.n, pad_left, sizeof(int32_t) * d->batch)) return SSD_ERR_INVALID_ARG;
    if (d->batch == 0 || (d->seqlen == 0 && !final_state)) return SSD_OK;
    Conv1dArgs a = conv1d_args(d, x, weight, bias);
    a.init = init_state; a.pad_left = pad_left;
    a.y[0] = y0; a.y[1] = y1; a.y[2] = y2; a.final_state = final_state;
    return status_of(launch_conv1d_fwd(a, (cudaStream_t)stream));
}

ssd_status_t ssd_conv1d_update(const ssd_conv1d_desc_t* d, void* state, const void* x, const float* weight,
                               const float* bias, void* y0, void* y1, void* y2, void* stream) {
    ssd_status_t st = check_conv1d_desc(d, false);
    if (st != SSD_OK) return st;
    if (d->seqlen != 1) return SSD_ERR_INVALID_ARG;
    if (!weight || (d->batch && (!state || !x || !y0 || (d->split1 && !y1) || (d->split2 && !y2))))
        return SSD_ERR_INVALID_ARG;
    if ((!d->split1 && y1) || (!d->split2 && y2)) return SSD_ERR_INVALID_ARG;
    const size_t e = dsize(d->y_dtype);
    const Span in[] = {{x, rows_bytes(d->batch, d->x_stride, d->channels, dsize(d->io_dtype))},
                       {weight, sizeof(float) * d->channels * d->width}, {bias, sizeof(float) * d->channels}};
    const Span out[] = {{y0, (size_t)d->batch * (d->channels - d->split1 - d->split2) * e},
                        {y1, (size_t)d->batch * d->split1 * e}, {y2, (size_t)d->batch * d->split2 * e},
                        {state, (size_t)d->batch * (d->width - 1) * d->channels * dsize(d->state_dtype)}};
    st = check_spans(in, out);
    if (st != SSD_OK) return st;
    if (d->batch == 0) return SSD_OK;
    Conv1dArgs a = conv1d_args(d, x, weight, bias);
    a.y[0] = y0; a.y[1] = y1; a.y[2] = y2; a.final_state = state;
    return status_of(launch_conv1d_update(a, (cudaStream_t)stream));
}

ssd_status_t ssd_conv1d_bwd_workspace_size(const ssd_conv1d_desc_t* d, size_t* bytes) {
    if (!bytes) return SSD_ERR_INVALID_ARG;
    const ssd_status_t st = check_conv1d_desc(d, true);
    if (st != SSD_OK) return st;
    *bytes = sizeof(float) * (size_t)conv1d_bwd_segments(d->batch, d->seqlen, d->channels) * d->channels * (d->width + 1);
    return SSD_OK;
}

ssd_status_t ssd_conv1d_bwd(const ssd_conv1d_desc_t* d, const void* x, const float* weight, const float* bias,
                            const void* init_state, const void* dy0, const void* dy1, const void* dy2,
                            const void* dfinal_state, void* dx, float* dweight, float* dbias, void* dinit_state,
                            void* workspace, size_t workspace_bytes, void* stream) {
    size_t need = 0;
    ssd_status_t st = ssd_conv1d_bwd_workspace_size(d, &need);
    if (st != SSD_OK) return st;
    const bool empty = d->batch == 0 || d->seqlen == 0;
    if (!weight || !dweight || (!empty && (!x || !dx || !dy0 || (d->split1 && !dy1) || (d->split2 && !dy2))))
        return SSD_ERR_INVALID_ARG;
    if ((!d->split1 && dy1) || (!d->split2 && dy2)) return SSD_ERR_INVALID_ARG;
    const int64_t tok = d->batch * d->seqlen;
    const size_t e = dsize(d->io_dtype), keep = (size_t)d->batch * (d->width - 1) * d->channels * dsize(d->state_dtype);
    const size_t nw = sizeof(float) * d->channels * d->width, nb = sizeof(float) * d->channels;
    const Span in[] = {{x, rows_bytes(tok, d->x_stride, d->channels, e)}, {weight, nw}, {bias, nb}, {init_state, keep},
                       {dy0, (size_t)tok * (d->channels - d->split1 - d->split2) * e},
                       {dy1, (size_t)tok * d->split1 * e}, {dy2, (size_t)tok * d->split2 * e}, {dfinal_state, keep}};
    const Span out[] = {{dx, rows_bytes(tok, d->dx_stride, d->channels, dsize(d->y_dtype))}, {dweight, nw},
                        {dbias, nb}, {dinit_state, keep}};
    st = check_spans(in, out);
    if (st == SSD_OK) st = check_workspace(workspace, workspace_bytes, need, in, out);
    if (st != SSD_OK) return st;
    Conv1dArgs a = conv1d_args(d, x, weight, bias);
    a.init = init_state; a.dfinal = dfinal_state;
    a.dy[0] = dy0; a.dy[1] = dy1; a.dy[2] = dy2;
    a.dx = dx; a.dw = dweight; a.db = dbias; a.dinit = dinit_state; a.ws = (float*)workspace;
    return status_of(launch_conv1d_bwd(a, (cudaStream_t)stream));
}

ssd_status_t ssd_selective_scan_workspace_size(const ssd_selective_desc_t* d, size_t* bytes) {
    if (!bytes) return SSD_ERR_INVALID_ARG;
    const ssd_status_t st = check_selective_desc(d, false);
    if (st != SSD_OK) return st;
    *bytes = selective_workspace(d->batch, d->seqlen, d->channels, d->dstate, d->ngroups);
    return SSD_OK;
}

ssd_status_t ssd_selective_scan_fwd(const ssd_selective_desc_t* d, const void* x, const void* dt_raw,
                                    const float* dt_bias, const float* A, const void* B, const void* C,
                                    const float* D, const void* z, const void* init_state, const int32_t* pad_left,
                                    void* y, void* final_state, void* workspace, size_t workspace_bytes,
                                    void* stream) {
    ssd_status_t st = check_selective_desc(d, z != nullptr);
    if (st != SSD_OK) return st;
    const bool empty = d->batch == 0 || d->seqlen == 0;
    if (!A || (!empty && (!x || !dt_raw || !B || !C || !y))) return SSD_ERR_INVALID_ARG;
    if ((uintptr_t)pad_left & 3u) return SSD_ERR_ALIGNMENT;
    const int64_t tok = d->batch * d->seqlen;
    const size_t e = dsize(d->io_dtype), nx = (size_t)tok * d->channels * e, nd = sizeof(float) * d->channels;
    const size_t nbc = (size_t)tok * d->ngroups * d->dstate * e;
    const size_t keep = (size_t)d->batch * d->channels * d->dstate * dsize(d->state_dtype);
    const Span in[] = {{x, nx}, {dt_raw, nx}, {dt_bias, nd}, {A, nd * d->dstate}, {B, nbc}, {C, nbc}, {D, nd},
                       {z, z ? rows_bytes(tok, d->z_stride, d->channels, e) : 0}, {init_state, keep}};
    const Span out[] = {{y, (size_t)tok * d->channels * dsize(d->y_dtype)}, {final_state, keep}};
    st = check_spans(in, out);
    const size_t need = selective_workspace(d->batch, d->seqlen, d->channels, d->dstate, d->ngroups);
    if (st == SSD_OK) st = check_workspace(workspace, workspace_bytes, need, in, out);
    if (st != SSD_OK) return st;
    for (const Span& r : out)
        if (overlaps(r.p, r.n, pad_left, sizeof(int32_t) * d->batch)) return SSD_ERR_INVALID_ARG;
    if (overlaps(workspace, need, pad_left, sizeof(int32_t) * d->batch)) return SSD_ERR_INVALID_ARG;
    if (d->batch == 0 || (d->seqlen == 0 && !final_state)) return SSD_OK;
    SelectiveArgs a = selective_args(d);
    a.x = x; a.dt_raw = dt_raw; a.dt_bias = dt_bias; a.A = A; a.B = B; a.C = C; a.Dv = D; a.z = z;
    a.init = init_state; a.pad_left = pad_left; a.y = y; a.final_state = final_state; a.ws = (char*)workspace;
    return status_of(launch_selective_fwd(a, (cudaStream_t)stream));
}

ssd_status_t ssd_selective_state_update(const ssd_selective_desc_t* d, void* state, const void* x,
                                        const void* dt_raw, const float* dt_bias, const float* A, const void* B,
                                        const void* C, const float* D, const void* z, void* y, void* stream) {
    ssd_status_t st = check_selective_desc(d, z != nullptr);
    if (st != SSD_OK) return st;
    if (d->seqlen != 1) return SSD_ERR_INVALID_ARG;
    if (!A || (d->batch && (!state || !x || !dt_raw || !B || !C || !y))) return SSD_ERR_INVALID_ARG;
    const size_t e = dsize(d->io_dtype), nx = (size_t)d->batch * d->channels * e, nd = sizeof(float) * d->channels;
    const size_t nbc = (size_t)d->batch * d->ngroups * d->dstate * e;
    const Span in[] = {{x, nx}, {dt_raw, nx}, {dt_bias, nd}, {A, nd * d->dstate}, {B, nbc}, {C, nbc}, {D, nd},
                       {z, z ? rows_bytes(d->batch, d->z_stride, d->channels, e) : 0}};
    const Span out[] = {{y, (size_t)d->batch * d->channels * dsize(d->y_dtype)},
                        {state, (size_t)d->batch * d->channels * d->dstate * dsize(d->state_dtype)}};
    st = check_spans(in, out);
    if (st != SSD_OK) return st;
    if (d->batch == 0) return SSD_OK;
    SelectiveArgs a = selective_args(d);
    a.x = x; a.dt_raw = dt_raw; a.dt_bias = dt_bias; a.A = A; a.B = B; a.C = C; a.Dv = D; a.z = z;
    a.y = y; a.final_state = state;
    return status_of(launch_selective_update(a, (cudaStream_t)stream));
}

ssd_status_t ssd_selective_scan_bwd_workspace_size(const ssd_selective_desc_t* d, size_t* bytes) {
    if (!bytes) return SSD_ERR_INVALID_ARG;
    const ssd_status_t st = check_selective_desc(d, false);
    if (st != SSD_OK) return st;
    *bytes = selective_bwd_workspace(d->batch, d->seqlen, d->channels, d->dstate, d->ngroups);
    return SSD_OK;
}

ssd_status_t ssd_selective_scan_bwd(const ssd_selective_desc_t* d, const void* x, const void* dt_raw,
                                    const float* dt_bias, const float* A, const void* B, const void* C,
                                    const float* D, const void* z, const void* init_state, const void* dy,
                                    const void* dfinal_state, void* dx, void* ddt_raw, float* ddt_bias, float* dA,
                                    void* dB, void* dC, float* dD, void* dz, void* dinit_state, void* workspace,
                                    size_t workspace_bytes, void* stream) {
    ssd_status_t st = check_selective_desc(d, z != nullptr);
    if (st != SSD_OK) return st;
    const bool empty = d->batch == 0 || d->seqlen == 0;
    if (!A || !dA || (!empty && (!x || !dt_raw || !B || !C || !dy || !dx || !ddt_raw || !dB || !dC || (z && !dz))))
        return SSD_ERR_INVALID_ARG;
    if (!z && dz) return SSD_ERR_INVALID_ARG;
    const int64_t tok = d->batch * d->seqlen;
    const size_t e = dsize(d->io_dtype), eg = dsize(d->y_dtype), nd = sizeof(float) * d->channels;
    const size_t nx = (size_t)tok * d->channels, nbc = (size_t)tok * d->ngroups * d->dstate;
    const size_t keep = (size_t)d->batch * d->channels * d->dstate * dsize(d->state_dtype);
    const Span in[] = {{x, nx * e}, {dt_raw, nx * e}, {dt_bias, nd}, {A, nd * d->dstate}, {B, nbc * e}, {C, nbc * e},
                       {D, nd}, {z, z ? rows_bytes(tok, d->z_stride, d->channels, e) : 0}, {init_state, keep},
                       {dy, nx * e}, {dfinal_state, keep}};
    const Span out[] = {{dx, nx * eg}, {ddt_raw, nx * eg}, {ddt_bias, nd}, {dA, nd * d->dstate}, {dB, nbc * eg},
                        {dC, nbc * eg}, {dD, nd}, {dz, nx * eg}, {dinit_state, keep}};
    st = check_spans(in, out);
    const size_t need = selective_bwd_workspace(d->batch, d->seqlen, d->channels, d->dstate, d->ngroups);
    if (st == SSD_OK) st = check_workspace(workspace, workspace_bytes, need, in, out);
    if (st != SSD_OK) return st;
    SelectiveArgs a = selective_args(d);
    a.x = x; a.dt_raw = dt_raw; a.dt_bias = dt_bias; a.A = A; a.B = B; a.C = C; a.Dv = D; a.z = z;
    a.init = init_state; a.dy = dy; a.dfinal = dfinal_state;
    a.dx = dx; a.ddt = ddt_raw; a.ddt_bias = ddt_bias; a.dA = dA; a.dB = dB; a.dC = dC; a.dD = dD; a.dz = dz;
    a.dinit = dinit_state; a.ws = (char*)workspace;
    return status_of(launch_selective_bwd(a, (cudaStream_t)stream));
}

ssd_status_t ssd_group_norm_fwd(const ssd_group_norm_desc_t* d, const void* x, const void* z, const float* weight,
                                const float* bias, void* y, void* stream) {
    ssd_status_t st = check_norm_desc(d);
    if (st != SSD_OK) return st;
    const bool gated = d->activation >= SSD_NORM_GATE_AFTER;
    if ((d->rows && (!x || !y || (gated && !z))) || (!gated && z)) return SSD_ERR_INVALID_ARG;
    const size_t n = (size_t)d->rows * d->channels, nb = sizeof(float) * d->channels;
    const Span in[] = {{x, n * dsize(d->x_dtype)}, {weight, nb}, {bias, nb},
                       {z, z ? rows_bytes(d->rows, d->z_stride, d->channels, dsize(d->io_dtype)) : 0}};
    const Span out[] = {{y, n * dsize(d->y_dtype)}};
    st = check_spans(in, out);
    if (st != SSD_OK) return st;
    if (d->rows == 0) return SSD_OK;
    GroupNormArgs a = norm_args(d, x, z, weight, bias);
    a.y = y;
    return status_of(launch_group_norm_fwd(a, (cudaStream_t)stream));
}

ssd_status_t ssd_group_norm_bwd_workspace_size(const ssd_group_norm_desc_t* d, size_t* bytes) {
    if (!bytes) return SSD_ERR_INVALID_ARG;
    const ssd_status_t st = check_norm_desc(d);
    if (st != SSD_OK) return st;
    *bytes = group_norm_bwd_workspace(d->rows, d->channels, d->ngroups);
    return SSD_OK;
}

ssd_status_t ssd_group_norm_bwd(const ssd_group_norm_desc_t* d, const void* x, const void* z, const float* weight,
                                const float* bias, const void* dy, void* dx, void* dz, float* dweight, float* dbias,
                                void* workspace, size_t workspace_bytes, void* stream) {
    ssd_status_t st = check_norm_desc(d);
    if (st != SSD_OK) return st;
    const bool gated = d->activation >= SSD_NORM_GATE_AFTER;
    if ((d->rows && (!x || !dy || !dx || (gated && (!z || !dz)))) || (!gated && (z || dz))) return SSD_ERR_INVALID_ARG;
    const size_t n = (size_t)d->rows * d->channels, nb = sizeof(float) * d->channels;
    const Span in[] = {{x, n * dsize(d->x_dtype)}, {weight, nb}, {bias, nb}, {dy, n * dsize(d->io_dtype)},
                       {z, z ? rows_bytes(d->rows, d->z_stride, d->channels, dsize(d->io_dtype)) : 0}};
    const Span out[] = {{dx, n * dsize(d->y_dtype)}, {dz, n * dsize(d->y_dtype)}, {dweight, nb}, {dbias, nb}};
    st = check_spans(in, out);
    const size_t need = group_norm_bwd_workspace(d->rows, d->channels, d->ngroups);
    if (st == SSD_OK) st = check_workspace(workspace, workspace_bytes, need, in, out);
    if (st != SSD_OK) return st;
    GroupNormArgs a = norm_args(d, x, z, weight, bias);
    a.dy = dy; a.dx = dx; a.dz = dz; a.dw = dweight; a.db = dbias; a.ws = (float*)workspace;
    return status_of(launch_group_norm_bwd(a, (cudaStream_t)stream));
}

}  // extern "C"
