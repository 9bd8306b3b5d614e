// k_scan_step.hip -- selective scan, one token for each cached sequence
// (include/dwconv_seq.h).
//
// Bound by HBM for many rows: a state is read and written once, eight bytes against
// seven operations; by latency for few.  A lane owns four states of a channel, LPC
// lanes a channel, so that a wavefront's states are one run of memory.
#include "scan_common.h"

namespace dw {
namespace {

template <class DT, int LPC>
__global__ void __launch_bounds__(256)
    k_step(ScanGeo G, ScanIn in, float *state, const int32_t *slots, int n_slots, int rows, typename DT::X *y,
           int64_t ldy) {
    using X = typename DT::X;
    const int row = (int)(blockIdx.x / G.nblk);
    const ScanLane<LPC> w(G, blockIdx.x % G.nblk);
    const SlotRows sr = slot_rows(slots, n_slots, rows, row);
    if (sr.slot < 0 || !w.live) return;
    float a2[4], h[4];
    float *st = state + ((int64_t)sr.slot * G.C + w.c) * G.N;
    load_states(h, st, 4 * w.j, G.N, true);
    load_rates(a2, in.a, G, w.c, 4 * w.j, true);
    const float bias = in.bias ? in.bias[w.c] : 0.0f, skip = in.skip ? in.skip[w.c] : 0.0f;
    for (int i = row; i < rows; ++i) {
        if (i != row && slots[i] != sr.slot) continue;
        const float xv = DT::widen(((const X *)in.x)[(int64_t)i * in.ldx + w.c]);
        const float dv = DT::widen(((const X *)in.dt)[(int64_t)i * in.lddt + w.c]);
        const float zv = in.gate ? DT::widen(((const X *)in.gate)[(int64_t)i * in.ldgate + w.c]) : 0.0f;
        const X *b = (const X *)in.b + (int64_t)i * in.ldb + (int64_t)w.g * G.N + 4 * w.j;
        const X *c = (const X *)in.c + (int64_t)i * in.ldc + (int64_t)w.g * G.N + 4 * w.j;
        float bv[4], cv[4], slope;
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const bool in_row = 4 * w.j + n < G.N;
            bv[n] = in_row ? DT::widen(b[n]) : 0.0f;
            cv[n] = in_row ? DT::widen(c[n]) : 0.0f;
        }
        const float d = step_width<DT>(dv + bias, G.soft, slope), u = d * xv;
        float v = 0.0f;
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            h[n] = __builtin_fmaf(__builtin_amdgcn_exp2f(d * a2[n]), h[n], u * bv[n]);
            v = __builtin_fmaf(h[n], cv[n], v);
        }
        v = __builtin_fmaf(skip, xv, sum_states<LPC>(v));
        if (in.gate) v *= gate_value<DT>(zv, G.act);
        if (w.j == 0) y[(int64_t)i * ldy + w.c] = rounded<DT>(v);
        if (!sr.shared) break;
    }
    store_states(st, h, 4 * w.j, G.N, true);
}

template <class DT, int LPC>
hipError_t step(const dwconv_scan_plan &p, const ScanArgs &a, hipStream_t st) {
    const ScanGeo G = scan_blocks(p, LPC);
    const uint64_t blocks = (uint64_t)G.nblk * (uint32_t)a.tokens;
    if (too_many(blocks)) return hipErrorInvalidConfiguration;
    if (blocks)
        k_step<DT, LPC><<<(uint32_t)blocks, 256, 0, st>>>(G, scan_inputs(a), a.state, a.slots, a.n_slots, a.tokens,
                                                          (typename DT::X *)a.y, a.ldy);
    return hipGetLastError();
}

template <class DT>
hipError_t pick_lanes(const dwconv_scan_plan &p, const ScanArgs &a, hipStream_t st) {
    switch (scan_lanes(p.N)) {
        case 4: return step<DT, 4>(p, a, st);
        case 8: return step<DT, 8>(p, a, st);
        case 16: return step<DT, 16>(p, a, st);
        default: return step<DT, 32>(p, a, st);
    }
}

}  // namespace

hipError_t scan_step(const dwconv_scan_plan &p, const ScanArgs &a, hipStream_t st) {
    switch (p.dtype) {
        case DWCONV_F32: return pick_lanes<F32>(p, a, st);
        case DWCONV_F16: return pick_lanes<F16>(p, a, st);
        default: return pick_lanes<BF16>(p, a, st);
    }
}

}  // namespace dw
