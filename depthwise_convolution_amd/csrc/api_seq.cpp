// api_seq.cpp -- the extern "C" entry points declared in include/dwconv_seq.h:
// argument checks in front of the launchers.
#include <initializer_list>
#include <math.h>
#include <new>
#include <stdint.h>

#include "seq_plan.h"

namespace {

bool float_dtype(dwconv_dtype_t t) { return t == DWCONV_F32 || t == DWCONV_F16 || t == DWCONV_BF16; }
int elem(int dtype) { return dtype == DWCONV_F32 ? 4 : 2; }

// aligned to `bytes`; NULL is
bool at(const void *p, uintptr_t bytes) { return ((uintptr_t)p & (bytes - 1)) == 0; }

bool overlap(const void *a, size_t na, const void *b, size_t nb) {
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return a && b && na && nb && x < y + nb && y < x + na;
}

// Counts of tokens and sequences to which a chunk, a run or one may be added.
constexpr int MOST = INT32_MAX - 128;

// Sequences: one without offsets, any number with them.
bool sequences(const int32_t *offsets, int seqs, int tokens) {
    return tokens >= 0 && tokens <= MOST && seqs >= 0 && seqs <= MOST && (offsets || seqs == 1) && at(offsets, 4);
}

// A tensor of `n` tokens with `width` dense channels of `e` bytes.
bool tensor(const void *p, int64_t ld, int64_t width, int n, int e) {
    return n == 0 || (p && at(p, e) && ld >= width && ld <= INT64_MAX / 8 / (n + 1));
}

bool slots_ok(const int32_t *slots, int n_slots, int rows) {
    return rows >= 0 && n_slots >= 0 && at(slots, 4) && (slots || rows <= n_slots);
}

// launchers say hipErrorInvalidConfiguration before a grid that passes its limit
dwconv_status_t status(hipError_t e) {
    return e == hipSuccess ? DWCONV_OK
           : e == hipErrorInvalidConfiguration ? DWCONV_ERR_UNSUPPORTED : DWCONV_ERR_HIP;
}

template <class P>
dwconv_status_t make(P **out, const P &v) {
    P *p = new (std::nothrow) P(v);
    if (!p) return DWCONV_ERR_ALLOC;
    *out = p;
    return DWCONV_OK;
}

}  // namespace

extern "C" {

dwconv_status_t dwconv_causal_create(dwconv_causal_t *out, int C, int K, dwconv_dtype_t dtype,
                                     dwconv_seq_act_t act) {
    if (!out) return DWCONV_ERR_INVALID_ARG;
    *out = nullptr;
    if (C < 1 || K < 2 || K > 8 || !float_dtype(dtype)) return DWCONV_ERR_INVALID_ARG;
    if (act != DWCONV_SEQ_ACT_NONE && act != DWCONV_SEQ_ACT_SILU) return DWCONV_ERR_INVALID_ARG;
    return make(out, dwconv_causal_plan{C, K, (int)dtype, (int)act});
}

dwconv_status_t dwconv_causal_destroy(dwconv_causal_t h) {
    delete h;
    return DWCONV_OK;
}

dwconv_status_t dwconv_causal_fwd(dwconv_causal_t h, const void *x, int64_t ldx, const void *w, const float *bias,
                                  const int32_t *offsets, int seqs, int tokens, const void *state_in, void *state_out,
                                  void *y, int64_t ldy, hipStream_t stream) {
    if (!h || !w) return DWCONV_ERR_INVALID_ARG;
    const int e = elem(h->dtype);
    const size_t st = (size_t)(seqs < 0 ? 0 : seqs) * (h->K - 1) * h->C * e;
    if (!sequences(offsets, seqs, tokens) || !tensor(x, ldx, h->C, tokens, e) || !tensor(y, ldy, h->C, tokens, e) ||
        !at(w, e) || !at(bias, 4) || !at(state_in, e) || !at(state_out, e) || (tokens && x == y) ||
        overlap(state_in, st, state_out, st))
        return DWCONV_ERR_INVALID_ARG;
    dw::CausalArgs a{};
    a.x = x, a.ldx = ldx, a.w = w, a.bias = bias, a.offsets = offsets, a.seqs = seqs, a.tokens = tokens;
    a.state_in = state_in, a.state_out = state_out, a.y = y, a.ldy = ldy;
    return status(dw::causal_fwd(*h, a, stream));
}

dwconv_status_t dwconv_causal_step(dwconv_causal_t h, const void *x, int64_t ldx, const void *w, const float *bias,
                                   void *state, const int32_t *slots, int n_slots, int rows, void *y, int64_t ldy,
                                   hipStream_t stream) {
    if (!h || !w) return DWCONV_ERR_INVALID_ARG;
    const int e = elem(h->dtype);
    if (!slots_ok(slots, n_slots, rows) || !tensor(x, ldx, h->C, rows, e) || !tensor(y, ldy, h->C, rows, e) ||
        !at(w, e) || !at(bias, 4) || !at(state, e) || (rows && (!state || x == y)))
        return DWCONV_ERR_INVALID_ARG;
    dw::CausalArgs a{};
    a.x = x, a.ldx = ldx, a.w = w, a.bias = bias, a.tokens = rows, a.state = state, a.slots = slots;
    a.n_slots = n_slots, a.y = y, a.ldy = ldy;
    return status(dw::causal_step(*h, a, stream));
}

dwconv_status_t dwconv_causal_bwd_workspace(dwconv_causal_t h, int tokens, size_t *bytes) {
    if (!h || !bytes || tokens < 0 || tokens > MOST) return DWCONV_ERR_INVALID_ARG;
    *bytes = dw::causal_bwd_bytes(*h, tokens);
    return DWCONV_OK;
}

dwconv_status_t dwconv_causal_bwd(dwconv_causal_t h, const void *x, int64_t ldx, const void *w, const float *bias,
                                  const int32_t *offsets, int seqs, int tokens, const void *state_in, const void *dy,
                                  int64_t lddy, const void *dstate_out, void *dx, int64_t lddx, float *dw,
                                  float *dbias, void *dstate_in, void *workspace, hipStream_t stream) {
    if (!h || !w || !dw) return DWCONV_ERR_INVALID_ARG;
    const int e = elem(h->dtype);
    const size_t st = (size_t)(seqs < 0 ? 0 : seqs) * (h->K - 1) * h->C * e;
    if (!sequences(offsets, seqs, tokens) || !tensor(x, ldx, h->C, tokens, e) || !tensor(dy, lddy, h->C, tokens, e) ||
        !tensor(dx, lddx, h->C, tokens, e) || !at(w, e) || !at(bias, 4) || !at(state_in, e) || !at(dstate_out, e) ||
        !at(dstate_in, e) || !at(dw, 4) || !at(dbias, 4) || !at(workspace, 4) ||
        (tokens && (!workspace || dx == x || dx == dy)) || overlap(dstate_out, st, dstate_in, st) ||
        overlap(state_in, st, dstate_in, st))
        return DWCONV_ERR_INVALID_ARG;
    dw::CausalArgs a{};
    a.x = x, a.ldx = ldx, a.w = w, a.bias = bias, a.offsets = offsets, a.seqs = seqs, a.tokens = tokens;
    a.state_in = state_in, a.dy = dy, a.lddy = lddy, a.dstate_out = dstate_out, a.dx = dx, a.lddx = lddx;
    a.dw = dw, a.dbias = dbias, a.dstate_in = dstate_in, a.workspace = (float *)workspace;
    return status(dw::causal_bwd(*h, a, stream));
}

dwconv_status_t dwconv_delta_create(dwconv_delta_t *out, int Hk, int Hv, int Dk, int Dv, dwconv_dtype_t dtype,
                                    float scale, int normalize, float eps) {
    if (!out) return DWCONV_ERR_INVALID_ARG;
    *out = nullptr;
    if (Hk < 1 || Hv < 1 || Hv % Hk || Hv > 65536 || Dk < 1 || Dk > 256 || Dv < 1 || Dv > 4096 || !float_dtype(dtype) ||
        !isfinite(scale) || !isfinite(eps) || eps < 0.0f)
        return DWCONV_ERR_INVALID_ARG;
    return make(out, dwconv_delta_plan{Hk, Hv, Dk, Dv, (int)dtype, scale, eps, normalize != 0});
}

dwconv_status_t dwconv_delta_destroy(dwconv_delta_t h) {
    delete h;
    return DWCONV_OK;
}

dwconv_status_t dwconv_delta_workspace(dwconv_delta_t h, int seqs, int tokens, int backward, size_t *bytes) {
    if (!h || !bytes || seqs < 0 || seqs > MOST || tokens < 0 || tokens > MOST) return DWCONV_ERR_INVALID_ARG;
    *bytes = dw::delta_bytes(*h, seqs, tokens, backward != 0);
    return DWCONV_OK;
}

// what the forward and the backward pass check alike
static bool delta_inputs(dwconv_delta_t h, const void *q, int64_t ldq, const void *k, int64_t ldk, const void *v,
                         int64_t ldv, const float *g, const float *beta, int n) {
    const int e = elem(h->dtype);
    const int64_t wk = (int64_t)h->Hk * h->Dk, wv = (int64_t)h->Hv * h->Dv;
    return tensor(q, ldq, wk, n, e) && tensor(k, ldk, wk, n, e) && tensor(v, ldv, wv, n, e) && at(g, 4) &&
           at(beta, 4) && (n == 0 || (g && beta));
}

static dw::DeltaArgs delta_args(const void *q, int64_t ldq, const void *k, int64_t ldk, const void *v, int64_t ldv,
                                const float *g, const float *beta, int n) {
    dw::DeltaArgs a{};
    a.q = q, a.ldq = ldq, a.k = k, a.ldk = ldk, a.v = v, a.ldv = ldv, a.g = g, a.beta = beta, a.tokens = n;
    return a;
}

dwconv_status_t dwconv_delta_fwd(dwconv_delta_t h, const void *q, int64_t ldq, const void *k, int64_t ldk,
                                 const void *v, int64_t ldv, const float *g, const float *beta, const int32_t *offsets,
                                 int seqs, int tokens, const float *state_in, float *state_out, void *o, int64_t ldo,
                                 void *workspace, hipStream_t stream) {
    if (!h || !sequences(offsets, seqs, tokens) || !delta_inputs(h, q, ldq, k, ldk, v, ldv, g, beta, tokens) ||
        !tensor(o, ldo, (int64_t)h->Hv * h->Dv, tokens, elem(h->dtype)) || !at(state_in, 4) || !at(state_out, 4) ||
        !at(workspace, 16) || (tokens && (!workspace || o == q || o == k || o == v)))
        return DWCONV_ERR_INVALID_ARG;
    const size_t st = (size_t)seqs * h->Hv * h->Dk * h->Dv * sizeof(float);
    if (state_in != state_out && overlap(state_in, st, state_out, st)) return DWCONV_ERR_INVALID_ARG;
    dw::DeltaArgs a = delta_args(q, ldq, k, ldk, v, ldv, g, beta, tokens);
    a.offsets = offsets, a.seqs = seqs, a.state_in = state_in, a.state_out = state_out, a.o = o, a.ldo = ldo;
    a.workspace = workspace;
    return status(dw::delta_fwd(*h, a, stream));
}

dwconv_status_t dwconv_delta_step(dwconv_delta_t h, const void *q, int64_t ldq, const void *k, int64_t ldk,
                                  const void *v, int64_t ldv, const float *g, const float *beta, float *state,
                                  const int32_t *slots, int n_slots, int rows, void *o, int64_t ldo,
                                  hipStream_t stream) {
    if (!h || !slots_ok(slots, n_slots, rows) || !delta_inputs(h, q, ldq, k, ldk, v, ldv, g, beta, rows) ||
        !tensor(o, ldo, (int64_t)h->Hv * h->Dv, rows, elem(h->dtype)) || !at(state, 4) ||
        (rows && (!state || o == q || o == k || o == v)))
        return DWCONV_ERR_INVALID_ARG;
    dw::DeltaArgs a = delta_args(q, ldq, k, ldk, v, ldv, g, beta, rows);
    a.state = state, a.slots = slots, a.n_slots = n_slots, a.o = o, a.ldo = ldo;
    return status(dw::delta_step(*h, a, stream));
}

dwconv_status_t dwconv_delta_bwd(dwconv_delta_t h, const void *q, int64_t ldq, const void *k, int64_t ldk,
                                 const void *v, int64_t ldv, const float *g, const float *beta, const int32_t *offsets,
                                 int seqs, int tokens, const float *state_in, const void *d_o, int64_t lddo,
                                 const float *dstate_out, void *dq, int64_t lddq, void *dk, int64_t lddk, void *dv,
                                 int64_t lddv, float *dg, float *dbeta, float *dstate_in, void *workspace,
                                 hipStream_t stream) {
    if (!h || !sequences(offsets, seqs, tokens) || !delta_inputs(h, q, ldq, k, ldk, v, ldv, g, beta, tokens))
        return DWCONV_ERR_INVALID_ARG;
    const int e = elem(h->dtype);
    const int64_t wk = (int64_t)h->Hk * h->Dk, wv = (int64_t)h->Hv * h->Dv;
    if (!tensor(d_o, lddo, wv, tokens, e) || !tensor(dq, lddq, wk, tokens, e) || !tensor(dk, lddk, wk, tokens, e) ||
        !tensor(dv, lddv, wv, tokens, e) || !at(dg, 4) || !at(dbeta, 4) || !at(state_in, 4) || !at(dstate_out, 4) ||
        !at(dstate_in, 4) || !at(workspace, 16) || (tokens && (!dg || !dbeta || !workspace)))
        return DWCONV_ERR_INVALID_ARG;
    // q, k, v and d_o are read until the last kernel
    const void *in[] = {q, k, v, d_o, g, beta}, *out[] = {dq, dk, dv, dg, dbeta};
    if (tokens)
        for (const void *i : in)
            for (const void *o : out)
                if (i == o) return DWCONV_ERR_INVALID_ARG;
    const size_t st = (size_t)seqs * h->Hv * h->Dk * h->Dv * sizeof(float);
    if (overlap(state_in, st, dstate_in, st) || (dstate_in != dstate_out && overlap(dstate_out, st, dstate_in, st)))
        return DWCONV_ERR_INVALID_ARG;
    dw::DeltaArgs a = delta_args(q, ldq, k, ldk, v, ldv, g, beta, tokens);
    a.offsets = offsets, a.seqs = seqs, a.state_in = state_in, a.d_o = d_o, a.lddo = lddo, a.dstate_out = dstate_out;
    a.dq = dq, a.lddq = lddq, a.dk = dk, a.lddk = lddk, a.dv = dv, a.lddv = lddv, a.dg = dg, a.dbeta = dbeta;
    a.dstate_in = dstate_in, a.workspace = workspace;
    return status(dw::delta_bwd(*h, a, stream));
}

dwconv_status_t dwconv_norm_create(dwconv_norm_t *out, int D, dwconv_dtype_t dtype, dwconv_norm_kind_t after,
                                   dwconv_norm_kind_t before, dwconv_seq_act_t gate_act, float eps) {
    if (!out) return DWCONV_ERR_INVALID_ARG;
    *out = nullptr;
    if (D < 1 || D > 16384 || !float_dtype(dtype) || (int)after < 0 || after > DWCONV_NORM_LAYER || (int)before < 0 ||
        before > DWCONV_NORM_LAYER || (int)gate_act < 0 || gate_act > DWCONV_SEQ_ACT_SIGMOID || !isfinite(eps) ||
        eps < 0.0f)
        return DWCONV_ERR_INVALID_ARG;
    return make(out, dwconv_norm_plan{D, (int)dtype, (int)after, (int)before, (int)gate_act, eps});
}

dwconv_status_t dwconv_norm_destroy(dwconv_norm_t p) {
    delete p;
    return DWCONV_OK;
}

// fills `a` with the forward inputs; false where they are not usable
static bool norm_inputs(dw::NormArgs &a, dwconv_norm_t p, int rows, const void *o, const void *residual,
                        const void *gate, int rows_per_gate, const float *scale, const float *w_after,
                        const float *b_after, const float *w_before, const float *b_before) {
    if (!p || rows < 0 || rows_per_gate < 1 || (rows && !o)) return false;
    const int e = elem(p->dtype);
    if (!at(o, e) || !at(residual, e) || !at(gate, e) || !at(scale, 4) || !at(w_after, 4) || !at(b_after, 4) ||
        !at(w_before, 4) || !at(b_before, 4))
        return false;
    if ((p->after != DWCONV_NORM_NONE && !w_after) || (p->before != DWCONV_NORM_NONE && !w_before)) return false;
    a.rows = rows, a.o = o, a.residual = residual, a.gate = gate, a.per = rows_per_gate, a.scale = scale;
    a.w_after = p->after != DWCONV_NORM_NONE ? w_after : nullptr;
    a.b_after = p->after == DWCONV_NORM_LAYER ? b_after : nullptr;
    a.w_before = p->before != DWCONV_NORM_NONE ? w_before : nullptr;
    a.b_before = p->before == DWCONV_NORM_LAYER ? b_before : nullptr;
    return true;
}

dwconv_status_t dwconv_norm_fwd(dwconv_norm_t p, int rows, const void *o, const void *residual, const void *gate,
                                int rows_per_gate, const float *scale, const float *w_after, const float *b_after,
                                const float *w_before, const float *b_before, void *h, void *y, hipStream_t stream) {
    dw::NormArgs a{};
    if (!norm_inputs(a, p, rows, o, residual, gate, rows_per_gate, scale, w_after, b_after, w_before, b_before))
        return DWCONV_ERR_INVALID_ARG;
    const int e = elem(p->dtype);
    if (p->before == DWCONV_NORM_NONE) y = nullptr;
    if (!at(h, e) || !at(y, e) || (rows && (p->before == DWCONV_NORM_NONE ? !h : !y))) return DWCONV_ERR_INVALID_ARG;
    const size_t n = (size_t)rows * p->D * e;
    if ((h != o && overlap(h, n, o, n)) || (h != residual && overlap(h, n, residual, n)) || (y != o && overlap(y, n, o, n)) ||
        overlap(y, n, residual, n) || overlap(h, n, y, n))
        return DWCONV_ERR_INVALID_ARG;
    a.h = h, a.y = y;
    return status(dw::norm_fwd(*p, a, stream));
}

dwconv_status_t dwconv_norm_bwd_workspace(dwconv_norm_t p, int rows, int rows_per_gate, size_t *bytes) {
    if (!p || !bytes || rows < 0 || rows_per_gate < 1) return DWCONV_ERR_INVALID_ARG;
    *bytes = dw::norm_bwd_bytes(*p, rows, rows_per_gate);
    return DWCONV_OK;
}

dwconv_status_t dwconv_norm_bwd(dwconv_norm_t p, int rows, const void *o, const void *residual, const void *gate,
                                int rows_per_gate, const float *scale, const float *w_after, const float *b_after,
                                const float *w_before, const float *b_before, const void *dh, const void *dy,
                                void *d_o, void *dresidual, void *dgate, float *dscale, float *dw_after,
                                float *db_after, float *dw_before, float *db_before, void *workspace,
                                hipStream_t stream) {
    dw::NormArgs a{};
    if (!norm_inputs(a, p, rows, o, residual, gate, rows_per_gate, scale, w_after, b_after, w_before, b_before))
        return DWCONV_ERR_INVALID_ARG;
    const int e = elem(p->dtype);
    const bool second = p->before != DWCONV_NORM_NONE;
    if (!at(dh, e) || !at(dy, e) || !at(d_o, e) || !at(dresidual, e) || !at(dgate, e) || !at(dscale, 4) ||
        !at(dw_after, 4) || !at(db_after, 4) || !at(dw_before, 4) || !at(db_before, 4) || !at(workspace, 4) ||
        (rows && (!workspace || (second && !dy))))
        return DWCONV_ERR_INVALID_ARG;
    const size_t n = (size_t)rows * p->D * e;
    const size_t ng = (size_t)((rows + (int64_t)rows_per_gate - 1) / rows_per_gate) * p->D * e;
    const void *in[] = {o, residual, dh, dy};
    void *out[] = {d_o, dresidual};
    for (const void *i : in) {
        for (void *q : out)
            if (overlap(i, n, q, n)) return DWCONV_ERR_INVALID_ARG;
        if (overlap(i, n, dgate, ng)) return DWCONV_ERR_INVALID_ARG;
    }
    if (overlap(gate, ng, d_o, n) || overlap(gate, ng, dresidual, n) || overlap(gate, ng, dgate, ng) ||
        overlap(d_o, n, dresidual, n))
        return DWCONV_ERR_INVALID_ARG;
    a.dh = dh, a.dy = second ? dy : nullptr, a.d_o = d_o, a.dresidual = residual ? dresidual : nullptr;
    a.dgate = gate ? dgate : nullptr, a.dscale = scale ? dscale : nullptr;
    a.dw_after = a.w_after ? dw_after : nullptr, a.db_after = a.b_after ? db_after : nullptr;
    a.dw_before = second ? dw_before : nullptr, a.db_before = a.b_before ? db_before : nullptr;
    a.workspace = (float *)workspace;
    return status(dw::norm_bwd(*p, a, stream));
}

dwconv_status_t dwconv_scan_create(dwconv_scan_t *out, int C, int N, int G, dwconv_dtype_t dtype, int softplus,
                                   dwconv_seq_act_t gate_act) {
    if (!out) return DWCONV_ERR_INVALID_ARG;
    *out = nullptr;
    if (C < 1 || C > 1 << 24 || N < 1 || N > 128 || G < 1 || C % G || !float_dtype(dtype) ||
        (int)gate_act < 0 || gate_act > DWCONV_SEQ_ACT_SIGMOID)
        return DWCONV_ERR_INVALID_ARG;
    return make(out, dwconv_scan_plan{C, N, G, (int)dtype, softplus != 0, (int)gate_act});
}

dwconv_status_t dwconv_scan_destroy(dwconv_scan_t h) {
    delete h;
    return DWCONV_OK;
}

dwconv_status_t dwconv_scan_workspace(dwconv_scan_t h, int seqs, int tokens, int backward, size_t *bytes) {
    if (!h || !bytes || seqs < 0 || seqs > MOST || tokens < 0 || tokens > MOST) return DWCONV_ERR_INVALID_ARG;
    *bytes = dw::scan_bytes(*h, seqs, tokens, backward != 0);
    return DWCONV_OK;
}

// fills `s` with what the three passes read; false where it is not usable
static bool scan_inputs(dw::ScanArgs &s, dwconv_scan_t h, const void *x, int64_t ldx, const void *dt, int64_t lddt,
                        const float *a, const void *b, int64_t ldb, const void *c, int64_t ldc, const float *skip,
                        const float *dt_bias, const void *gate, int64_t ldgate, int n) {
    if (!h || !a) return false;
    const int e = elem(h->dtype);
    const int64_t states = (int64_t)h->G * h->N;
    if (!tensor(x, ldx, h->C, n, e) || !tensor(dt, lddt, h->C, n, e) || !tensor(b, ldb, states, n, e) ||
        !tensor(c, ldc, states, n, e) || (gate && !tensor(gate, ldgate, h->C, n, e)) || !at(a, 4) || !at(skip, 4) ||
        !at(dt_bias, 4))
        return false;
    s.x = x, s.ldx = ldx, s.dt = dt, s.lddt = lddt, s.a = a, s.b = b, s.ldb = ldb, s.c = c, s.ldc = ldc, s.skip = skip;
    s.bias = dt_bias, s.gate = gate, s.ldgate = ldgate, s.tokens = n;
    return true;
}

// Kernels keep a lane's place in 16 tokens in 32 bits.
static bool scan_strides(std::initializer_list<int64_t> lds) {
    for (int64_t ld : lds)
        if (ld > 1 << 26) return false;
    return true;
}

dwconv_status_t dwconv_scan_fwd(dwconv_scan_t h, const void *x, int64_t ldx, const void *dt, int64_t lddt, const float *a,
                                const void *b, int64_t ldb, const void *c, int64_t ldc, const float *skip,
                                const float *dt_bias, const void *gate, int64_t ldgate, const int32_t *offsets, int seqs,
                                int tokens, const float *state_in, float *state_out, void *y, int64_t ldy, void *workspace,
                                hipStream_t stream) {
    dw::ScanArgs s{};
    if (!sequences(offsets, seqs, tokens) ||
        !scan_inputs(s, h, x, ldx, dt, lddt, a, b, ldb, c, ldc, skip, dt_bias, gate, ldgate, tokens) ||
        !tensor(y, ldy, h->C, tokens, elem(h->dtype)) || !at(state_in, 4) || !at(state_out, 4) || !at(workspace, 16) ||
        (tokens && (y == x || y == dt || y == b || y == c || y == gate)) ||
        (!workspace && dw::scan_bytes(*h, seqs, tokens, false)))
        return DWCONV_ERR_INVALID_ARG;
    const size_t st = (size_t)seqs * h->C * h->N * sizeof(float);
    if (state_in != state_out && overlap(state_in, st, state_out, st)) return DWCONV_ERR_INVALID_ARG;
    if (!scan_strides({ldx, lddt, ldb, ldc, gate ? ldgate : 0, ldy})) return DWCONV_ERR_UNSUPPORTED;
    s.offsets = offsets, s.seqs = seqs, s.state_in = state_in, s.state_out = state_out, s.y = y, s.ldy = ldy;
    s.workspace = (float *)workspace;
    return status(dw::scan_fwd(*h, s, stream));
}

dwconv_status_t dwconv_scan_step(dwconv_scan_t h, const void *x, int64_t ldx, const void *dt, int64_t lddt, const float *a,
                                 const void *b, int64_t ldb, const void *c, int64_t ldc, const float *skip,
                                 const float *dt_bias, const void *gate, int64_t ldgate, float *state,
                                 const int32_t *slots, int n_slots, int rows, void *y, int64_t ldy, hipStream_t stream) {
    dw::ScanArgs s{};
    if (!slots_ok(slots, n_slots, rows) ||
        !scan_inputs(s, h, x, ldx, dt, lddt, a, b, ldb, c, ldc, skip, dt_bias, gate, ldgate, rows) ||
        !tensor(y, ldy, h->C, rows, elem(h->dtype)) || !at(state, 4) ||
        (rows && (!state || y == x || y == dt || y == b || y == c || y == gate)))
        return DWCONV_ERR_INVALID_ARG;
    s.state = state, s.slots = slots, s.n_slots = n_slots, s.y = y, s.ldy = ldy;
    return status(dw::scan_step(*h, s, stream));
}

dwconv_status_t dwconv_scan_bwd(dwconv_scan_t h, const void *x, int64_t ldx, const void *dt, int64_t lddt, const float *a,
                                const void *b, int64_t ldb, const void *c, int64_t ldc, const float *skip,
                                const float *dt_bias, const void *gate, int64_t ldgate, const int32_t *offsets, int seqs,
                                int tokens, const float *state_in, const void *dy, int64_t lddy, const float *dstate_out,
                                void *dx, int64_t lddx, void *ddt, int64_t ldddt, float *da, void *db, int64_t lddb,
                                void *dc, int64_t lddc, float *dskip, float *ddt_bias, void *dgate, int64_t lddgate,
                                float *dstate_in, void *workspace, hipStream_t stream) {
    dw::ScanArgs s{};
    if (!sequences(offsets, seqs, tokens) ||
        !scan_inputs(s, h, x, ldx, dt, lddt, a, b, ldb, c, ldc, skip, dt_bias, gate, ldgate, tokens) || !da)
        return DWCONV_ERR_INVALID_ARG;
    if (!gate) dgate = nullptr;
    if (!skip) dskip = nullptr;
    if (!dt_bias) ddt_bias = nullptr;
    const int e = elem(h->dtype);
    const int64_t states = (int64_t)h->G * h->N;
    if (!tensor(dy, lddy, h->C, tokens, e) || !tensor(dx, lddx, h->C, tokens, e) || !tensor(ddt, ldddt, h->C, tokens, e) ||
        !tensor(db, lddb, states, tokens, e) || !tensor(dc, lddc, states, tokens, e) ||
        (dgate && !tensor(dgate, lddgate, h->C, tokens, e)) || !at(da, 4) || !at(dskip, 4) || !at(ddt_bias, 4) ||
        !at(state_in, 4) || !at(dstate_out, 4) || !at(dstate_in, 4) || !at(workspace, 16) ||
        (!workspace && dw::scan_bytes(*h, seqs, tokens, true)))
        return DWCONV_ERR_INVALID_ARG;
    const void *in[] = {x, dt, b, c, gate, dy, a}, *out[] = {dx, ddt, db, dc, dgate, da};
    if (tokens)
        for (const void *i : in)
            for (const void *o : out)
                if (i && i == o) return DWCONV_ERR_INVALID_ARG;
    const size_t st = (size_t)seqs * h->C * h->N * sizeof(float);
    if (overlap(state_in, st, dstate_in, st) || (dstate_in != dstate_out && overlap(dstate_out, st, dstate_in, st)))
        return DWCONV_ERR_INVALID_ARG;
    if (!scan_strides({ldx, lddt, ldb, ldc, gate ? ldgate : 0, lddy, lddx, ldddt, lddb, lddc, dgate ? lddgate : 0}))
        return DWCONV_ERR_UNSUPPORTED;
    s.offsets = offsets, s.seqs = seqs, s.state_in = state_in, s.dy = dy, s.lddy = lddy, s.dstate_out = dstate_out;
    s.dx = dx, s.lddx = lddx, s.ddt = ddt, s.ldddt = ldddt, s.da = da, s.db = db, s.lddb = lddb, s.dc = dc, s.lddc = lddc;
    s.dskip = dskip, s.dbias = ddt_bias, s.dgate = dgate, s.lddgate = lddgate, s.dstate_in = dstate_in;
    s.workspace = (float *)workspace;
    return status(dw::scan_bwd(*h, s, stream));
}

dwconv_status_t dwconv_group_create(dwconv_group_t *out, int C, int G, dwconv_dtype_t dtype, dwconv_group_act_t act,
                                    float eps) {
    if (!out) return DWCONV_ERR_INVALID_ARG;
    *out = nullptr;
    if (C < 1 || C > 65536 || G < 1 || C % G || !float_dtype(dtype) || (int)act < 0 || act > DWCONV_GROUP_ACT_RELU ||
        !isfinite(eps) || eps < 0.0f)
        return DWCONV_ERR_INVALID_ARG;
    return make(out, dwconv_group_plan{C, G, (int)dtype, (int)act, eps});
}

dwconv_status_t dwconv_group_destroy(dwconv_group_t h) {
    delete h;
    return DWCONV_OK;
}

// images x pixels rows that an int counts, with the few thousand that a kernel's loops look ahead
static bool group_rows(int images, int pixels) {
    return images >= 0 && pixels >= 0 && (int64_t)images * pixels <= INT32_MAX - 65536;
}

dwconv_status_t dwconv_group_workspace(dwconv_group_t h, int images, int pixels, int backward, size_t *bytes) {
    if (!h || !bytes || !group_rows(images, pixels)) return DWCONV_ERR_INVALID_ARG;
    *bytes = dw::group_bytes(*h, images, pixels, backward != 0);
    return DWCONV_OK;
}

dwconv_status_t dwconv_group_fwd(dwconv_group_t h, int images, int pixels, const void *x, int64_t ldx, const float *w,
                                 const float *b, void *y, int64_t ldy, void *workspace, hipStream_t stream) {
    if (!h || !group_rows(images, pixels)) return DWCONV_ERR_INVALID_ARG;
    const int e = elem(h->dtype), n = images * pixels;
    if (!tensor(x, ldx, h->C, n, e) || !tensor(y, ldy, h->C, n, e) || !at(w, 4) || !at(b, 4) || !at(workspace, 16) ||
        (n && x == y && ldx != ldy) || (!workspace && dw::group_bytes(*h, images, pixels, false)))
        return DWCONV_ERR_INVALID_ARG;
    dw::GroupArgs a{};
    a.images = images, a.pixels = pixels, a.x = x, a.ldx = ldx, a.w = w, a.b = b, a.y = y, a.ldy = ldy;
    a.workspace = (float *)workspace;
    return status(dw::group_fwd(*h, a, stream));
}

dwconv_status_t dwconv_group_bwd(dwconv_group_t h, int images, int pixels, const void *x, int64_t ldx, const float *w,
                                 const float *b, const void *dy, int64_t lddy, void *dx, int64_t lddx, float *dw,
                                 float *db, void *workspace, hipStream_t stream) {
    if (!h || !group_rows(images, pixels)) return DWCONV_ERR_INVALID_ARG;
    const int e = elem(h->dtype), n = images * pixels;
    if (!tensor(x, ldx, h->C, n, e) || !tensor(dy, lddy, h->C, n, e) || !tensor(dx, lddx, h->C, n, e) || !at(w, 4) ||
        !at(b, 4) || !at(dw, 4) || !at(db, 4) || !at(workspace, 16) || (n && (dx == x || (dx == dy && lddx != lddy))) ||
        (!workspace && dw::group_bytes(*h, images, pixels, true)))
        return DWCONV_ERR_INVALID_ARG;
    dw::GroupArgs a{};
    a.images = images, a.pixels = pixels, a.x = x, a.ldx = ldx, a.w = w, a.b = b, a.dy = dy, a.lddy = lddy;
    a.dx = dx, a.lddx = lddx, a.dw = dw, a.db = db, a.workspace = (float *)workspace;
    return status(dw::group_bwd(*h, a, stream));
}

}  // extern "C"
