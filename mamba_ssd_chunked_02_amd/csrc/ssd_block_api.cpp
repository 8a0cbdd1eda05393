// Host side of the block operators' entry points in include/ssd.h (conv1d
// gradients, gated recurrence, norms): argument validation before any launch,
// then the kernels are queued.  Nothing here allocates, frees or synchronizes.
#include "ssd_checks.h"

using namespace ssd_checks;

namespace {

// ------------------------------------------------------------------ conv1d
ssd_status conv_shape_of(const ssd_conv_shape* sh, ssd::ConvBwdArgs* a) {
    if (!sh) FAIL(SSD_ERR_NULL, "shape is NULL");
    ssd_status st = check_dtypes(sh->dtype, sh->ydtype);
    if (st != SSD_OK) return st;
    if (sh->reserved != 0) FAIL(SSD_ERR_SHAPE, "reserved must be 0");
    if (sh->activation != 0 && sh->activation != 1)
        FAIL(SSD_ERR_VALUE, "activation %d is neither 0 (none) nor 1 (SiLU)", sh->activation);
    if (sh->width < 2 || sh->width > 4) FAIL(SSD_ERR_SHAPE, "width %d must be in [2, 4]", sh->width);
    *a = ssd::ConvBwdArgs{};
    st = check_sequences(sh->batch, sh->seqlen, sh->channels, sh->cu_seqlens, sh->cu_seqlens_host, &a->T);
    if (st != SSD_OK) return st;
    a->cu = sh->cu_seqlens;
    a->nseq = sh->batch;
    a->L = sh->seqlen;
    a->C = sh->channels;
    a->K = sh->width;
    a->dtype = sh->dtype;
    a->y_f32 = sh->ydtype == SSD_F32;
    a->silu = sh->activation;
    ssd::conv_backward_blocks(a->T, a->C, &a->nblocks, &a->block_rows);
    return SSD_OK;
}

size_t conv_workspace(const ssd::ConvBwdArgs& a) { return (size_t)a.nblocks * (a.K + 1) * a.C * 4; }

}  // namespace

SSD_API ssd_status ssd_causal_conv1d_backward_workspace_size(const ssd_conv_shape* shape, size_t* bytes) {
    if (!bytes) FAIL(SSD_ERR_NULL, "bytes is NULL");
    ssd::ConvBwdArgs a;
    const ssd_status st = conv_shape_of(shape, &a);
    if (st != SSD_OK) return st;
    *bytes = conv_workspace(a);
    return ok();
}

SSD_API ssd_status ssd_causal_conv1d_backward(const ssd_conv_outputs* dout, const void* x, const float* weight,
                                              const float* bias, const void* conv_state_in, const void* dstate_out,
                                              void* dx, float* dweight, float* dbias, void* dstate_in,
                                              const ssd_conv_shape* shape, void* workspace, size_t workspace_bytes,
                                              void* stream) {
    ssd::ConvBwdArgs a;
    ssd_status st = conv_shape_of(shape, &a);
    if (st != SSD_OK) return st;
    if (!dout) FAIL(SSD_ERR_NULL, "dout is NULL");
    if (dout->nparts < 1 || dout->nparts > 3) FAIL(SSD_ERR_SHAPE, "nparts %d must be 1, 2 or 3", dout->nparts);
    int64_t sum = 0;
    for (int p = 0; p < 3; ++p) {
        if (p >= dout->nparts) {
            if (dout->channels[p] != 0 || dout->out[p]) FAIL(SSD_ERR_SHAPE, "unused part %d must be 0 / NULL", p);
            continue;
        }
        if (dout->channels[p] < 8 || dout->channels[p] % 8 != 0)
            FAIL(SSD_ERR_SHAPE, "part %d has %d channels (a positive multiple of 8 is needed)", p, dout->channels[p]);
        sum += dout->channels[p];
    }
    if (sum != a.C) FAIL(SSD_ERR_SHAPE, "the parts hold %lld channels, not %d", (long long)sum, a.C);
    const bool any = a.T > 0;
    const Arg args[] = {{dout->out[0], "dout part 0", any, false},
                        {dout->out[1], "dout part 1", any && dout->nparts > 1, false},
                        {dout->out[2], "dout part 2", any && dout->nparts > 2, false},
                        {x, "x", any, false},
                        {weight, "weight", true, false},
                        {bias, "bias", false, false},
                        {conv_state_in, "conv_state_in", false, false},
                        {dstate_out, "dstate_out", false, false},
                        {dx, "dx", any, true},
                        {dweight, "dweight", true, true},
                        {dbias, "dbias", false, true},
                        {dstate_in, "dstate_in", false, true}};
    st = check_args(args, (int)(sizeof(args) / sizeof(args[0])));
    if (st != SSD_OK) return st;
    st = check_workspace(workspace, workspace_bytes, conv_workspace(a));
    if (st != SSD_OK) return st;
    for (int p = 0; p < 3; ++p) {
        a.dy[p] = dout->out[p];
        a.part_ch[p] = dout->channels[p];
    }
    a.nparts = dout->nparts;
    a.x = x;
    a.weight = weight;
    a.bias = bias;
    a.state_in = conv_state_in;
    a.dstate_out = dstate_out;
    a.dx = dx;
    a.dweight = dweight;
    a.dbias = dbias;
    a.dstate_in = dstate_in;
    a.part = (float*)workspace;
    return queued(ssd::launch_conv1d_backward(a, (hipStream_t)stream));
}

// ------------------------------------------------------------------ gated recurrence
namespace {

ssd_status gated_shape_of(const ssd_gated_shape* sh, bool step, ssd::GatedArgs* a) {
    if (!sh) FAIL(SSD_ERR_NULL, "shape is NULL");
    ssd_status st = check_dtypes(sh->dtype, sh->ydtype);
    if (st != SSD_OK) return st;
    if (sh->reserved != 0) FAIL(SSD_ERR_SHAPE, "reserved must be 0");
    if (!(sh->rate > 0.f) || isinf(sh->rate)) FAIL(SSD_ERR_VALUE, "rate %g must be finite and > 0", (double)sh->rate);
    *a = ssd::GatedArgs{};
    st = check_sequences(sh->batch, step ? 1 : sh->seqlen, sh->channels, step ? nullptr : sh->cu_seqlens,
                         step ? nullptr : sh->cu_seqlens_host, &a->T);
    if (st != SSD_OK) return st;
    struct {
        const char* name;
        int64_t given;
        int64_t* to;
    } strides[] = {{"x_stride", sh->x_stride, &a->x_stride},    {"r_stride", sh->r_stride, &a->r_stride},
                   {"i_stride", sh->i_stride, &a->i_stride},    {"dx_stride", sh->dx_stride, &a->dx_stride},
                   {"dr_stride", sh->dr_stride, &a->dr_stride}, {"di_stride", sh->di_stride, &a->di_stride}};
    for (auto& q : strides)
        if ((st = check_stride(q.name, q.given, sh->channels, a->T, q.to)) != SSD_OK) return st;
    a->cu = step ? nullptr : sh->cu_seqlens;
    a->nseq = sh->batch;
    a->L = step ? 1 : sh->seqlen;
    a->C = sh->channels;
    a->dtype = sh->dtype;
    a->y_f32 = sh->ydtype == SSD_F32;
    a->rate = sh->rate;
    // offsets inside a tile of rows are 32 bits; the step has no tiles
    for (auto& q : strides)
        if (!step && *q.to > (1 << 22)) FAIL(SSD_ERR_SHAPE, "%s %lld is over 2^22", q.name, (long long)*q.to);
    // a launch counts its lanes in 32 bits
    if (!step && ssd::gated_layout(a->T, a->C, false, false).blocks > ((int64_t)1 << 22))
        FAIL(SSD_ERR_SHAPE, "tensor too large for one launch");
    return SSD_OK;
}

}  // namespace

SSD_API ssd_status ssd_gated_scan_workspace_size(const ssd_gated_shape* shape, int32_t backward, size_t* bytes) {
    if (!bytes) FAIL(SSD_ERR_NULL, "bytes is NULL");
    if (backward != 0 && backward != 1) FAIL(SSD_ERR_VALUE, "backward must be 0 or 1 (got %d)", backward);
    ssd::GatedArgs a;
    const ssd_status st = gated_shape_of(shape, false, &a);
    if (st != SSD_OK) return st;
    *bytes = ssd::gated_layout(a.T, a.C, a.cu != nullptr, backward).total;
    return ok();
}

SSD_API ssd_status ssd_gated_scan(const void* x, const void* r, const void* i, const float* lam,
                                  const float* init_state, void* y, float* final_state, float* states,
                                  const ssd_gated_shape* shape, void* workspace, size_t workspace_bytes,
                                  void* stream) {
    ssd::GatedArgs a;
    ssd_status st = gated_shape_of(shape, false, &a);
    if (st != SSD_OK) return st;
    const bool any = a.T > 0;
    const Arg args[] = {{x, "x", any, false},
                        {r, "r", any, false},
                        {i, "i", any, false},
                        {lam, "lam", true, false},
                        {init_state, "init_state", false, false},
                        {y, "y", any, true},
                        {final_state, "final_state", false, true},
                        {states, "states", false, true}};
    st = check_args(args, (int)(sizeof(args) / sizeof(args[0])));
    if (st != SSD_OK) return st;
    const ssd::GatedLayout lay = ssd::gated_layout(a.T, a.C, a.cu != nullptr, false);
    st = check_workspace(workspace, workspace_bytes, lay.total);
    if (st != SSD_OK) return st;
    a.x = x;
    a.r = r;
    a.i = i;
    a.lam = lam;
    a.init = init_state;
    a.y = y;
    a.final_state = final_state;
    a.states_out = states;
    return queued(ssd::launch_gated_scan(a, lay, workspace, (hipStream_t)stream));
}

SSD_API ssd_status ssd_gated_scan_backward(const void* dy, const float* dfinal_state, const void* x, const void* r,
                                           const void* i, const float* lam, const float* init_state,
                                           const float* states, void* dx, void* dr, void* di, float* dlam,
                                           float* dinit_state, const ssd_gated_shape* shape, void* workspace,
                                           size_t workspace_bytes, void* stream) {
    ssd::GatedArgs a;
    ssd_status st = gated_shape_of(shape, false, &a);
    if (st != SSD_OK) return st;
    const bool any = a.T > 0;
    const Arg args[] = {{dy, "dy", any, false},
                        {dfinal_state, "dfinal_state", false, false},
                        {x, "x", any, false},
                        {r, "r", any, false},
                        {i, "i", any, false},
                        {lam, "lam", true, false},
                        {init_state, "init_state", false, false},
                        {states, "states", any, false},
                        {dx, "dx", any, true},
                        {dr, "dr", any, true},
                        {di, "di", any, true},
                        {dlam, "dlam", true, true},
                        {dinit_state, "dinit_state", false, true}};
    st = check_args(args, (int)(sizeof(args) / sizeof(args[0])));
    if (st != SSD_OK) return st;
    const ssd::GatedLayout lay = ssd::gated_layout(a.T, a.C, a.cu != nullptr, true);
    st = check_workspace(workspace, workspace_bytes, lay.total);
    if (st != SSD_OK) return st;
    a.x = x;
    a.r = r;
    a.i = i;
    a.lam = lam;
    a.init = init_state;
    a.dy = dy;
    a.states_in = states;
    a.dfinal = dfinal_state;
    a.dx = dx;
    a.dr = dr;
    a.di = di;
    a.dlam = dlam;
    a.dinit = dinit_state;
    return queued(ssd::launch_gated_backward(a, lay, workspace, (hipStream_t)stream));
}

SSD_API ssd_status ssd_gated_scan_step(const float* state, float* state_out, const void* x, const void* r,
                                       const void* i, const float* lam, void* y, const ssd_gated_shape* shape,
                                       void* stream) {
    ssd::GatedArgs a;
    ssd_status st = gated_shape_of(shape, true, &a);
    if (st != SSD_OK) return st;
    const bool any = a.nseq > 0;
    const Arg args[] = {{x, "x", any, false},        {r, "r", any, false},
                        {i, "i", any, false},        {lam, "lam", true, false},
                        {state, "state", any, false}, {y, "y", any, true},
                        {state_out, "state_out", any, true}};
    st = check_args(args, (int)(sizeof(args) / sizeof(args[0])), {6, 1u << 4});
    if (st != SSD_OK) return st;
    a.x = x;
    a.r = r;
    a.i = i;
    a.lam = lam;
    a.y = y;
    return queued(ssd::launch_gated_step(a, state, state_out, (hipStream_t)stream));
}

// ------------------------------------------------------------------ norms
namespace {

ssd_status norm_shape_of(const ssd_norm_shape* sh, bool gated, ssd::NormArgs* a) {
    if (!sh) FAIL(SSD_ERR_NULL, "shape is NULL");
    ssd_status st = check_dtypes(sh->dtype, sh->dtype2);
    if (st != SSD_OK) return st;
    if (sh->reserved != 0) FAIL(SSD_ERR_SHAPE, "reserved must be 0");
    if (!(sh->eps >= 0.f) || isinf(sh->eps)) FAIL(SSD_ERR_VALUE, "eps %g must be finite and >= 0", (double)sh->eps);
    if (sh->norm_before_gate != 0 && (sh->norm_before_gate != 1 || !gated))
        FAIL(SSD_ERR_VALUE, "norm_before_gate %d must be 0%s", sh->norm_before_gate, gated ? " or 1" : "");
    if (sh->groups < 1 || sh->groups > 1024 || (!gated && sh->groups != 1))
        FAIL(SSD_ERR_SHAPE, "groups %d must be %s", sh->groups, gated ? "in [1, 1024]" : "1");
    if (sh->columns < 8 || sh->columns % (8 * sh->groups) != 0)
        FAIL(SSD_ERR_SHAPE, "columns %d must be a positive multiple of 8 * groups", sh->columns);
    if (sh->columns / sh->groups > ssd::kMaxNormColumns)
        FAIL(SSD_ERR_UNSUPPORTED, "%d columns a group (at most %d)", sh->columns / sh->groups, ssd::kMaxNormColumns);
    if (sh->rows < 0 || sh->rows > kMaxRows / sh->groups) FAIL(SSD_ERR_SHAPE, "rows * groups must be in [0, 2^31 - 1]");
    if (sh->rows * sh->columns > kMaxElements) FAIL(SSD_ERR_SHAPE, "tensor too large");
    if (sh->dtype == SSD_F32 && sh->dtype2 != SSD_F32)
        FAIL(SSD_ERR_UNSUPPORTED, "an fp32 stream with a bf16 %s", gated ? "x" : "residual");
    *a = ssd::NormArgs{};
    struct {
        const char* name;
        int64_t given;
        int64_t* to;
    } strides[] = {{"x_stride", sh->x_stride, &a->x_stride},
                   {"z_stride", sh->z_stride, &a->z_stride},
                   {"dx_stride", sh->dx_stride, &a->dx_stride},
                   {"dz_stride", sh->dz_stride, &a->dz_stride}};
    for (auto& q : strides) {
        if (!gated && q.given != 0) FAIL(SSD_ERR_SHAPE, "%s must be 0", q.name);
        if ((st = check_stride(q.name, q.given, sh->columns, sh->rows, q.to)) != SSD_OK) return st;
    }
    a->rows = sh->rows;
    a->D = sh->columns;
    a->G = sh->groups;
    a->eps = sh->eps;
    a->a_f32 = sh->dtype == SSD_F32;
    a->b_f32 = sh->dtype2 == SSD_F32;
    a->norm_first = sh->norm_before_gate;
    a->nparts = ssd::norm_parts(a->rows, a->D, a->G);
    return SSD_OK;
}

// dweight's and dscale's partial sums.
size_t norm_workspace(const ssd::NormArgs& a) { return (size_t)a.nparts * a.D * 8; }

}  // namespace

SSD_API ssd_status ssd_norm_backward_workspace_size(const ssd_norm_shape* shape, size_t* bytes) {
    if (!bytes) FAIL(SSD_ERR_NULL, "bytes is NULL");
    ssd::NormArgs a;
    const ssd_status st = norm_shape_of(shape, true, &a);
    if (st != SSD_OK) return st;
    *bytes = norm_workspace(a);
    return ok();
}

SSD_API ssd_status ssd_add_rms_norm(const void* x, const void* residual, const float* weight, const float* scale,
                                    void* y, void* out, float* rstd, const ssd_norm_shape* shape, void* stream) {
    ssd::NormArgs a;
    ssd_status st = norm_shape_of(shape, false, &a);
    if (st != SSD_OK) return st;
    const bool any = a.rows > 0;
    const Arg args[] = {{x, "x", any, false},         {residual, "residual", any, false},
                        {weight, "weight", true, false}, {scale, "scale", false, false},
                        {y, "y", any, true},          {out, "out", any, true},
                        {rstd, "rstd", false, true}};
    // a lane reads its elements of x and the residual before it writes out; x may be the residual
    const bool in_place = out == residual;
    st = check_args(args, (int)(sizeof(args) / sizeof(args[0])),
                    {in_place ? 5 : -1, 1u << 1 | (a.a_f32 == a.b_f32 ? 1u << 0 : 0)});
    if (st != SSD_OK) return st;
    a.x = x;
    a.z = residual;
    a.weight = weight;
    a.scale = scale;
    a.y = y;
    a.out = out;
    a.rstd = rstd;
    return queued(ssd::launch_residual_norm(a, (hipStream_t)stream));
}

SSD_API ssd_status ssd_add_rms_norm_backward(const void* dy, const void* dout, const void* out, const float* weight,
                                             const float* rstd, const void* x, const float* scale, void* dx,
                                             void* dresidual, float* dweight, float* dscale,
                                             const ssd_norm_shape* shape, void* workspace, size_t workspace_bytes,
                                             void* stream) {
    ssd::NormArgs a;
    ssd_status st = norm_shape_of(shape, false, &a);
    if (st != SSD_OK) return st;
    const bool any = a.rows > 0;
    if (!scale && dscale) FAIL(SSD_ERR_SHAPE, "dscale without scale");
    const Arg args[] = {{dy, "dy", any, false},
                        {dout, "dout", false, false},
                        {out, "out", any, false},
                        {weight, "weight", true, false},
                        {rstd, "rstd", any, false},
                        {x, "x", any && dscale, false},
                        {scale, "scale", false, false},
                        {dx, "dx", any, true},
                        {dresidual, "dresidual", false, true},
                        {dweight, "dweight", true, true},
                        {dscale, "dscale", false, true}};
    // a lane reads its elements of dout, and of dy, out and x where dout is one of them, before it writes the gradient
    const bool one_type = a.a_f32 == a.b_f32;
    const int in_place = !dout ? -1 : dresidual == dout ? 8 : dx == dout && one_type ? 7 : -1;
    st = check_args(args, (int)(sizeof(args) / sizeof(args[0])),
                    {in_place, 1u << 1 | 1u << 2 | (one_type ? 1u << 0 | 1u << 5 : 0)});
    if (st != SSD_OK) return st;
    st = check_workspace(workspace, workspace_bytes, norm_workspace(a));
    if (st != SSD_OK) return st;
    a.dy = dy;
    a.dout = dout;
    a.out = const_cast<void*>(out);  // read only here
    a.weight = weight;
    a.rstd_in = rstd;
    a.x = x;
    a.scale = scale;
    a.dx = dx;
    a.dz = dresidual;
    a.dweight = dweight;
    a.dscale = dscale;
    a.part = (float*)workspace;
    return queued(ssd::launch_residual_norm_backward(a, (hipStream_t)stream));
}

SSD_API ssd_status ssd_gated_rms_norm(const void* x, const void* z, const float* weight, void* y, float* rstd,
                                      const ssd_norm_shape* shape, void* stream) {
    ssd::NormArgs a;
    ssd_status st = norm_shape_of(shape, true, &a);
    if (st != SSD_OK) return st;
    const bool any = a.rows > 0;
    const Arg args[] = {{x, "x", any, false},
                        {z, "z", any, false},
                        {weight, "weight", true, false},
                        {y, "y", any, true},
                        {rstd, "rstd", false, true}};
    st = check_args(args, (int)(sizeof(args) / sizeof(args[0])));
    if (st != SSD_OK) return st;
    a.x = x;
    a.z = z;
    a.weight = weight;
    a.y = y;
    a.rstd = rstd;
    return queued(ssd::launch_gated_norm(a, (hipStream_t)stream));
}

SSD_API ssd_status ssd_gated_rms_norm_backward(const void* dy, const void* x, const void* z, const float* weight,
                                               const float* rstd, void* dx, void* dz, float* dweight,
                                               const ssd_norm_shape* shape, void* workspace, size_t workspace_bytes,
                                               void* stream) {
    ssd::NormArgs a;
    ssd_status st = norm_shape_of(shape, true, &a);
    if (st != SSD_OK) return st;
    const bool any = a.rows > 0;
    const Arg args[] = {{dy, "dy", any, false},
                        {x, "x", any, false},
                        {z, "z", any, false},
                        {weight, "weight", true, false},
                        {rstd, "rstd", any, false},
                        {dx, "dx", any, true},
                        {dz, "dz", any, true},
                        {dweight, "dweight", true, true}};
    st = check_args(args, (int)(sizeof(args) / sizeof(args[0])));
    if (st != SSD_OK) return st;
    st = check_workspace(workspace, workspace_bytes, norm_workspace(a));
    if (st != SSD_OK) return st;
    a.dy = dy;
    a.x = x;
    a.z = z;
    a.weight = weight;
    a.rstd_in = rstd;
    a.dx = dx;
    a.dz = dz;
    a.dweight = dweight;
    a.part = (float*)workspace;
    return queued(ssd::launch_gated_norm_backward(a, (hipStream_t)stream));
}

// ------------------------------------------------------------------ layer norm
namespace {

// dweight's, dbias's and dscale's partial sums, for the kind that has the most workgroups.
size_t layer_norm_workspace(const ssd::NormArgs& a) {
    int32_t parts = 0;
    for (int kind : {ssd::kNormPlain, ssd::kNormResidual, ssd::kNormScaled})
        for (bool f32 : {false, true}) parts = std::max(parts, ssd::layer_norm_parts(a.rows, a.D, kind, f32));
    return (size_t)parts * a.D * 12;
}

}  // namespace

SSD_API ssd_status ssd_layer_norm(const void* x, const void* residual, const float* weight, const float* bias,
                                  const float* scale, void* y, void* out, float* mean, float* rstd,
                                  const ssd_norm_shape* shape, void* stream) {
    ssd::NormArgs a;
    ssd_status st = norm_shape_of(shape, false, &a);
    if (st != SSD_OK) return st;
    const bool any = a.rows > 0;
    if (!residual && (scale || out) && any) FAIL(SSD_ERR_SHAPE, "%s without residual", scale ? "scale" : "out");
    if (!residual && a.a_f32 != a.b_f32 && any) FAIL(SSD_ERR_DTYPE, "a second dtype without residual");
    const Arg args[] = {{x, "x", any, false},           {residual, "residual", false, false},
                        {weight, "weight", true, false}, {bias, "bias", false, false},
                        {scale, "scale", false, false},  {y, "y", any, true},
                        {out, "out", any && residual, true}, {mean, "mean", false, true},
                        {rstd, "rstd", false, true}};
    // a lane reads its elements of x and the residual before it writes out; x may be the residual
    const bool in_place = out && out == residual;
    st = check_args(args, (int)(sizeof(args) / sizeof(args[0])),
                    {in_place ? 6 : -1, 1u << 1 | (a.a_f32 == a.b_f32 ? 1u << 0 : 0)});
    if (st != SSD_OK) return st;
    a.x = x;
    a.z = residual;
    a.weight = weight;
    a.bias = bias;
    a.scale = scale;
    a.y = y;
    a.out = out;
    a.mean = mean;
    a.rstd = rstd;
    return queued(ssd::launch_layer_norm(a, (hipStream_t)stream));
}

SSD_API ssd_status ssd_layer_norm_backward_workspace_size(const ssd_norm_shape* shape, size_t* bytes) {
    if (!bytes) FAIL(SSD_ERR_NULL, "bytes is NULL");
    ssd::NormArgs a;
    const ssd_status st = norm_shape_of(shape, false, &a);
    if (st != SSD_OK) return st;
    *bytes = layer_norm_workspace(a);
    return ok();
}

SSD_API ssd_status ssd_layer_norm_backward(const void* dy, const void* dout, const void* out, const float* weight,
                                           const float* mean, const float* rstd, const void* x, const float* scale,
                                           void* dx, void* dresidual, float* dweight, float* dbias, float* dscale,
                                           const ssd_norm_shape* shape, void* workspace, size_t workspace_bytes,
                                           void* stream) {
    ssd::NormArgs a;
    ssd_status st = norm_shape_of(shape, false, &a);
    if (st != SSD_OK) return st;
    const bool any = a.rows > 0;
    if (!scale && dscale) FAIL(SSD_ERR_SHAPE, "dscale without scale");
    const Arg args[] = {{dy, "dy", any, false},
                        {dout, "dout", false, false},
                        {out, "out", any, false},
                        {weight, "weight", true, false},
                        {mean, "mean", any, false},
                        {rstd, "rstd", any, false},
                        {x, "x", any && dscale, false},
                        {scale, "scale", false, false},
                        {dx, "dx", any, true},
                        {dresidual, "dresidual", false, true},
                        {dweight, "dweight", true, true},
                        {dbias, "dbias", false, true},
                        {dscale, "dscale", false, true}};
    // a lane reads its elements of dout, and of dy, out and x where dout is one of them, before it writes the gradient
    const bool one_type = a.a_f32 == a.b_f32;
    const int in_place = !dout ? -1 : dresidual == dout ? 9 : dx == dout && one_type ? 8 : -1;
    st = check_args(args, (int)(sizeof(args) / sizeof(args[0])),
                    {in_place, 1u << 1 | 1u << 2 | (one_type ? 1u << 0 | 1u << 6 : 0)});
    if (st != SSD_OK) return st;
    st = check_workspace(workspace, workspace_bytes, layer_norm_workspace(a));
    if (st != SSD_OK) return st;
    a.dy = dy;
    a.dout = dout;
    a.out = const_cast<void*>(out);  // read only here
    a.weight = weight;
    a.mean_in = mean;
    a.rstd_in = rstd;
    a.x = x;
    a.scale = scale;
    a.dx = dx;
    a.dz = dresidual;
    a.dweight = dweight;
    a.dbias = dbias;
    a.dscale = dscale;
    a.part = (float*)workspace;
    a.nparts = ssd::layer_norm_parts(a.rows, a.D, ssd::layer_norm_kind(a), a.a_f32);
    return queued(ssd::launch_layer_norm_backward(a, (hipStream_t)stream));
}
