// Host side of the selective scan's entry points in include/ssd.h: argument
// validation before any launch, then the kernels are queued.  Nothing here
// allocates, frees or synchronizes.
#include "ssd_checks.h"

using namespace ssd_checks;

namespace {

constexpr int64_t kMaxStride = 1 << 22;

ssd_status selective_shape_of(const ssd_selective_shape* sh, bool step, ssd::SelArgs* a) {
    if (!sh) FAIL(SSD_ERR_NULL, "shape is NULL");
    ssd_status st = check_dtypes(sh->dtype, sh->ydtype);
    if (st != SSD_OK) return st;
    if (sh->reserved != 0) FAIL(SSD_ERR_SHAPE, "reserved must be 0");
    *a = ssd::SelArgs{};
    st = check_sequences(sh->batch, step ? 1 : sh->seqlen, sh->channels, step ? nullptr : sh->cu_seqlens,
                         step ? nullptr : sh->cu_seqlens_host, &a->T);
    if (st != SSD_OK) return st;
    const int32_t C = sh->channels, N = sh->dstate, G = sh->ngroups;
    if (N < 1 || N > ssd::kMaxSelStates) FAIL(SSD_ERR_SHAPE, "dstate %d must be in [1, %d]", N, ssd::kMaxSelStates);
    if (G < 1 || C % G != 0 || (int64_t)G * N > kMaxStride)
        FAIL(SSD_ERR_SHAPE, "ngroups %d must divide channels %d and be at most 2^22 / dstate", G, C);
    struct {
        const char* name;
        int64_t given;
        int64_t* to;
        bool states;
    } strides[] = {{"x_stride", sh->x_stride, &a->x_stride, false},    {"dt_stride", sh->dt_stride, &a->dt_stride, false},
                   {"z_stride", sh->z_stride, &a->z_stride, false},    {"b_stride", sh->b_stride, &a->b_stride, true},
                   {"c_stride", sh->c_stride, &a->c_stride, true},     {"dx_stride", sh->dx_stride, &a->dx_stride, false},
                   {"ddt_stride", sh->ddt_stride, &a->ddt_stride, false}, {"dz_stride", sh->dz_stride, &a->dz_stride, false},
                   {"db_stride", sh->db_stride, &a->db_stride, true},  {"dc_stride", sh->dc_stride, &a->dc_stride, true}};
    for (auto& q : strides) {
        const int32_t width = q.states ? G * N : C;
        *q.to = q.given ? q.given : width;
        if (q.given < 0 || *q.to < width || (!q.states && *q.to % 8 != 0))
            FAIL(SSD_ERR_SHAPE, "%s %lld must be 0 or %s least %d", q.name, (long long)q.given,
                 q.states ? "at" : "a multiple of 8 of at", width);
        if (!step && *q.to > kMaxStride) FAIL(SSD_ERR_SHAPE, "%s %lld is over 2^22", q.name, (long long)*q.to);
        if (a->T > 0 && *q.to > kMaxElements / a->T) FAIL(SSD_ERR_SHAPE, "%s: tensor too large", q.name);
    }
    a->cu = step ? nullptr : sh->cu_seqlens;
    a->nseq = sh->batch;
    a->L = step ? 1 : sh->seqlen;
    a->C = C;
    a->N = N;
    a->G = G;
    a->dtype = sh->dtype;
    a->y_f32 = sh->ydtype == SSD_F32;
    // states of sequences and of the runs of tokens between two saved ones
    const int64_t most = kMaxElements / ((int64_t)C * N);
    if (a->nseq > most) FAIL(SSD_ERR_SHAPE, "tensor too large");
    if (!step && ssd::sel_saved_states(a->cu != nullptr, a->nseq, a->L, a->T) > most)
        FAIL(SSD_ERR_SHAPE, "tensor too large");
    return SSD_OK;
}

ssd_status activation_of(const ssd_dt_activation* act, ssd::DtAct* out) {
    *out = ssd::DtAct{nullptr, 0.f, 0.f, 0};
    if (!act) return SSD_OK;
    const float lo = act->dt_min, hi = act->dt_max;
    if (!(lo >= 0.f) || isinf(lo)) FAIL(SSD_ERR_VALUE, "dt_min %g must be finite and >= 0", (double)lo);
    if (!(hi >= lo)) FAIL(SSD_ERR_VALUE, "dt_max %g must be >= dt_min %g", (double)hi, (double)lo);
    *out = ssd::DtAct{act->dt_bias, lo, hi, 1};
    return SSD_OK;
}

unsigned element(const ssd::SelArgs& a) { return a.dtype == SSD_BF16 ? 2 : 4; }

}  // namespace

SSD_API ssd_status ssd_selective_scan_workspace_size(const ssd_selective_shape* shape, int32_t backward,
                                                     size_t* bytes) {
    if (!bytes) FAIL(SSD_ERR_NULL, "bytes is NULL");
    if (backward != 0 && backward != 1) FAIL(SSD_ERR_VALUE, "backward must be 0 or 1 (got %d)", backward);
    ssd::SelArgs a;
    const ssd_status st = selective_shape_of(shape, false, &a);
    if (st != SSD_OK) return st;
    *bytes = ssd::sel_layout(a, backward).total;
    return ok();
}

SSD_API ssd_status ssd_selective_scan(const void* x, const void* dt, const float* A, const void* B, const void* C,
                                      const float* D, const void* z, const ssd_dt_activation* act,
                                      const float* init_state, void* y, float* final_state, float* states,
                                      const ssd_selective_shape* shape, void* workspace, size_t workspace_bytes,
                                      void* stream) {
    ssd::SelArgs a;
    ssd_status st = selective_shape_of(shape, false, &a);
    if (st != SSD_OK) return st;
    st = activation_of(act, &a.act);
    if (st != SSD_OK) return st;
    const bool any = a.T > 0;
    const unsigned e = element(a);
    const Arg args[] = {{x, "x", any, false},
                        {dt, "dt", any, false},
                        {A, "A", true, false, 4},
                        {B, "B", any, false, e},
                        {C, "C", any, false, e},
                        {D, "D", false, false, 4},
                        {z, "z", false, false},
                        {a.act.bias, "dt_bias", false, false, 4},
                        {init_state, "init_state", false, false},
                        {y, "y", any, true},
                        {final_state, "final_state", false, true},
                        {states, "states", false, true}};
    st = check_args(args, (int)(sizeof(args) / sizeof(args[0])));
    if (st != SSD_OK) return st;
    const ssd::SelLayout lay = ssd::sel_layout(a, false);
    st = check_workspace(workspace, workspace_bytes, lay.total);
    if (st != SSD_OK) return st;
    a.x = x;
    a.dt = dt;
    a.z = z;
    a.B = B;
    a.Cm = C;
    a.A = A;
    a.D = D;
    a.init = init_state;
    a.y = y;
    a.final_state = final_state;
    a.states_out = states;
    return queued(ssd::launch_selective_scan(a, lay, workspace, (hipStream_t)stream));
}

SSD_API ssd_status ssd_selective_scan_backward(const void* dy, const float* dfinal_state, const void* x,
                                               const void* dt, const float* A, const void* B, const void* C,
                                               const float* D, const void* z, const ssd_dt_activation* act,
                                               const float* init_state, const float* states, void* dx, void* ddt,
                                               float* dA, void* dB, void* dC, float* dD, void* dz, float* ddt_bias,
                                               float* dinit_state, const ssd_selective_shape* shape, void* workspace,
                                               size_t workspace_bytes, void* stream) {
    ssd::SelArgs a;
    ssd_status st = selective_shape_of(shape, false, &a);
    if (st != SSD_OK) return st;
    st = activation_of(act, &a.act);
    if (st != SSD_OK) return st;
    const bool any = a.T > 0;
    const unsigned e = element(a);
    if (!z && dz) FAIL(SSD_ERR_SHAPE, "dz without z");
    if (!D && dD) FAIL(SSD_ERR_SHAPE, "dD without D");
    if (!a.act.bias && ddt_bias) FAIL(SSD_ERR_SHAPE, "ddt_bias without dt_bias");
    const Arg args[] = {{dy, "dy", any, false},
                        {dfinal_state, "dfinal_state", false, false},
                        {x, "x", any, false},
                        {dt, "dt", any, false},
                        {A, "A", true, false, 4},
                        {B, "B", any, false, e},
                        {C, "C", any, false, e},
                        {D, "D", false, false, 4},
                        {z, "z", false, false},
                        {a.act.bias, "dt_bias", false, false, 4},
                        {init_state, "init_state", false, false},
                        {states, "states", any, false},
                        {dx, "dx", any, true},
                        {ddt, "ddt", any, true},
                        {dA, "dA", true, true, 4},
                        {dB, "dB", any, true, e},
                        {dC, "dC", any, true, e},
                        {dD, "dD", false, true, 4},
                        {dz, "dz", any && z, true},
                        {ddt_bias, "ddt_bias", false, true, 4},
                        {dinit_state, "dinit_state", false, true}};
    st = check_args(args, (int)(sizeof(args) / sizeof(args[0])));
    if (st != SSD_OK) return st;
    const ssd::SelLayout lay = ssd::sel_layout(a, true);
    st = check_workspace(workspace, workspace_bytes, lay.total);
    if (st != SSD_OK) return st;
    a.dy = dy;
    a.dfinal = dfinal_state;
    a.x = x;
    a.dt = dt;
    a.z = z;
    a.B = B;
    a.Cm = C;
    a.A = A;
    a.D = D;
    a.states_in = states;
    a.dx = dx;
    a.ddt = ddt;
    a.dA = dA;
    a.dB = dB;
    a.dC = dC;
    a.dD = dD;
    a.dz = dz;
    a.dbias = ddt_bias;
    a.dinit = dinit_state;
    return queued(ssd::launch_selective_backward(a, lay, workspace, (hipStream_t)stream));
}

SSD_API ssd_status ssd_selective_scan_step(const float* state, float* state_out, const void* x, const void* dt,
                                           const float* A, const void* B, const void* C, const float* D,
                                           const void* z, const ssd_dt_activation* act, void* y,
                                           const ssd_selective_shape* shape, void* stream) {
    ssd::SelArgs a;
    ssd_status st = selective_shape_of(shape, true, &a);
    if (st != SSD_OK) return st;
    st = activation_of(act, &a.act);
    if (st != SSD_OK) return st;
    const bool any = a.nseq > 0;
    const unsigned e = element(a);
    const Arg args[] = {{state, "state", any, false},
                        {state_out, "state_out", any, true},
                        {x, "x", any, false},
                        {dt, "dt", any, false},
                        {A, "A", true, false, 4},
                        {B, "B", any, false, e},
                        {C, "C", any, false, e},
                        {D, "D", false, false, 4},
                        {z, "z", false, false},
                        {a.act.bias, "dt_bias", false, false, 4},
                        {y, "y", any, true}};
    // a lane reads its part of a state before it writes it
    st = check_args(args, (int)(sizeof(args) / sizeof(args[0])), {1, 1u << 0});
    if (st != SSD_OK) return st;
    a.x = x;
    a.dt = dt;
    a.z = z;
    a.B = B;
    a.Cm = C;
    a.A = A;
    a.D = D;
    a.y = y;
    return queued(ssd::launch_selective_step(a, state, state_out, (hipStream_t)stream));
}
