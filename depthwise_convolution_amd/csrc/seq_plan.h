// seq_plan.h -- host-side plans and launchers of the sequence operators
// (include/dwconv_seq.h).  Launchers get checked arguments.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/dwconv_seq.h"

struct dwconv_causal_plan {
    int C, K, dtype, act;
};

struct dwconv_delta_plan {
    int Hk, Hv, Dk, Dv, dtype;
    float scale, eps;
    int normalize;
};

struct dwconv_norm_plan {
    int D, dtype, after, before, act;
    float eps;
};

struct dwconv_scan_plan {
    int C, N, G, dtype, softplus, act;
};

struct dwconv_group_plan {
    int C, G, dtype, act;
    float eps;
};

namespace dw {

struct CausalArgs {
    const void *x;
    int64_t ldx;
    const void *w;
    const float *bias;
    const int32_t *offsets;
    int seqs, tokens;
    const void *state_in;
    void *state_out;
    void *y;
    int64_t ldy;
    // step
    void *state;
    const int32_t *slots;
    int n_slots;
    // backward
    const void *dy;
    int64_t lddy;
    const void *dstate_out;
    void *dx;
    int64_t lddx;
    float *dw, *dbias;
    void *dstate_in;
    float *workspace;
};
hipError_t causal_fwd(const dwconv_causal_plan &p, const CausalArgs &a, hipStream_t st);
hipError_t causal_step(const dwconv_causal_plan &p, const CausalArgs &a, hipStream_t st);
hipError_t causal_bwd(const dwconv_causal_plan &p, const CausalArgs &a, hipStream_t st);
size_t causal_bwd_bytes(const dwconv_causal_plan &p, int tokens);

struct DeltaArgs {
    const void *q, *k, *v;
    int64_t ldq, ldk, ldv;
    const float *g, *beta;
    const int32_t *offsets;
    int seqs, tokens;
    const float *state_in;
    float *state_out;
    void *o;
    int64_t ldo;
    // step
    float *state;
    const int32_t *slots;
    int n_slots;
    // backward
    const void *d_o;
    int64_t lddo;
    const float *dstate_out;
    void *dq, *dk, *dv;
    int64_t lddq, lddk, lddv;
    float *dg, *dbeta, *dstate_in;
    void *workspace;
};
hipError_t delta_fwd(const dwconv_delta_plan &p, const DeltaArgs &a, hipStream_t st);
hipError_t delta_step(const dwconv_delta_plan &p, const DeltaArgs &a, hipStream_t st);
hipError_t delta_bwd(const dwconv_delta_plan &p, const DeltaArgs &a, hipStream_t st);
size_t delta_bytes(const dwconv_delta_plan &p, int seqs, int tokens, bool backward);

struct NormArgs {
    int rows;
    const void *o, *residual, *gate;
    int per;  // rows a gate row serves
    const float *scale, *w_after, *b_after, *w_before, *b_before;
    void *h, *y;
    const void *dh, *dy;
    void *d_o, *dresidual, *dgate;
    float *dscale, *dw_after, *db_after, *dw_before, *db_before;
    float *workspace;
};
hipError_t norm_fwd(const dwconv_norm_plan &p, const NormArgs &a, hipStream_t st);
hipError_t norm_bwd(const dwconv_norm_plan &p, const NormArgs &a, hipStream_t st);
size_t norm_bwd_bytes(const dwconv_norm_plan &p, int rows, int per);

struct ScanArgs {
    const void *x, *dt, *b, *c, *gate;
    int64_t ldx, lddt, ldb, ldc, ldgate;
    const float *a, *skip, *bias;
    const int32_t *offsets;
    int seqs, tokens;
    const float *state_in;
    float *state_out;
    void *y;
    int64_t ldy;
    // step
    float *state;
    const int32_t *slots;
    int n_slots;
    // backward
    const void *dy;
    int64_t lddy;
    const float *dstate_out;
    void *dx, *ddt, *db, *dc, *dgate;
    int64_t lddx, ldddt, lddb, lddc, lddgate;
    float *da, *dskip, *dbias, *dstate_in;
    float *workspace;
};
hipError_t scan_fwd(const dwconv_scan_plan &p, const ScanArgs &a, hipStream_t st);
hipError_t scan_step(const dwconv_scan_plan &p, const ScanArgs &a, hipStream_t st);
hipError_t scan_bwd(const dwconv_scan_plan &p, const ScanArgs &a, hipStream_t st);
size_t scan_bytes(const dwconv_scan_plan &p, int seqs, int tokens, bool backward);

struct GroupArgs {
    int images, pixels;
    const void *x;
    int64_t ldx;
    const float *w, *b;
    void *y;
    int64_t ldy;
    const void *dy;
    int64_t lddy;
    void *dx;
    int64_t lddx;
    float *dw, *db;
    float *workspace;
};
hipError_t group_fwd(const dwconv_group_plan &p, const GroupArgs &a, hipStream_t st);
hipError_t group_bwd(const dwconv_group_plan &p, const GroupArgs &a, hipStream_t st);
size_t group_bytes(const dwconv_group_plan &p, int images, int pixels, bool backward);

}  // namespace dw
