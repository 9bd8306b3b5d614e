// k_scan_step.hip -- selective scan, one token for each cached sequence
// (include/dwconv_seq.h).
//
// Bound by HBM for many rows: a state is read and written once, eight bytes against
// seven operations; by latency for few.  A lane owns four states of a channel, LPC
// lanes a channel, so that a wavefront's states are one run of memory; it walks every
// `walkers`-th row and has the next one's loads on their way while it computes.
//
// 8192 channels of 16 states, bf16, caches that change from call to call so that none is in the
// last-level cache: one row 4.1 us, 8 rows 5.7, 32 rows 11.4, 96 rows 29 (107 MB, 3.7 TB/s; a
// large copy's rate would be 20), 192 rows 57.5; 96 rows of one or two caches (51 MB each) 24.
// A workgroup for every row, which has nothing on its way while it computes: 13.2, 40 and 78
// for 32, 96 and 192.
#include "scan_common.h"

namespace dw {
namespace {

// What a row's lane reads.
template <class DT>
struct Row {
    using X = typename DT::X;
    struct __attribute__((packed, aligned(sizeof(X)))) Four {
        X v[4];
    };
    int slot;  // -1: outside the cache
    X x, dt, z, b[4], c[4];
    float h[4];
    // four elements at index n0 of a row of N, zeros past it
    static __device__ __forceinline__ void four(X (&v)[4], const X *row, int n0, int N) {
        if (n0 + 4 <= N) {
            const Four a = *(const Four *)(row + n0);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = a.v[i];
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = n0 + i < N ? row[n0 + i] : (X)0;
        }
    }
    template <int LPC>
    __device__ __forceinline__ void token(const ScanGeo &G, const ScanIn &in, const ScanLane<LPC> &w, int i) {
        x = ((const X *)in.x)[(int64_t)i * in.ldx + w.c];
        dt = ((const X *)in.dt)[(int64_t)i * in.lddt + w.c];
        if (in.gate) z = ((const X *)in.gate)[(int64_t)i * in.ldgate + w.c];
        four(b, (const X *)in.b + (int64_t)i * in.ldb + (int64_t)w.g * G.N, 4 * w.j, G.N);
        four(c, (const X *)in.c + (int64_t)i * in.ldc + (int64_t)w.g * G.N, 4 * w.j, G.N);
    }
    template <int LPC>
    __device__ __forceinline__ void fetch(const ScanGeo &G, const ScanIn &in, const ScanLane<LPC> &w, const float *state,
                                          const int32_t *slots, int n_slots, int i) {
        slot = slots ? uniform(slots[i]) : i;
        if (slot < 0 || slot >= n_slots) slot = -1;
        if (!w.live) return;
        if (slot >= 0) load_states(h, state + ((int64_t)slot * G.C + w.c) * G.N, 4 * w.j, G.N, true);
        token(G, in, w, i);
    }
};

template <class DT, int LPC>
__global__ void __launch_bounds__(256, 8)
    k_step(ScanGeo G, ScanIn in, float *state, const int32_t *slots, int n_slots, int rows, typename DT::X *y, int64_t ldy) {
    const ScanLane<LPC> w(G, blockIdx.x % G.nblk);
    const int step = (int)G.walkers, lane = (int)threadIdx.x & 63;
    // the first 128 rows' slots
    const int s0 = slots && lane < rows ? slots[lane] : -1, s1 = slots && lane + 64 < rows ? slots[lane + 64] : -1;
    float a2[4];
    load_rates(a2, in.a, G, w.c, 4 * w.j, w.live);
    const float bias = in.bias && w.live ? in.bias[w.c] : 0.0f, skip = in.skip && w.live ? in.skip[w.c] : 0.0f;
    // Rows with the same slot are consecutive tokens of one sequence: the first one's
    // workgroup takes them all in order, the others' leave them (what they have read of the
    // entry by then is not used).
    auto compute = [&](Row<DT> &q, int row) {
        bool before = false, after = false;
        if (slots) {
            before = (s0 == q.slot && lane < row) || (s1 == q.slot && lane + 64 < row);
            after = (s0 == q.slot && lane > row) || (s1 == q.slot && lane + 64 > row);
            for (int j = lane + 128; j < rows; j += 64) {
                const bool same = slots[j] == q.slot;
                before |= same && j < row;
                after |= same && j > row;
            }
        }
        const bool shared = __any(after);
        if (q.slot < 0 || __any(before) || !w.live) return;
        for (int i = row; i < rows; ++i) {
            if (i != row) {
                if (slots[i] != q.slot) continue;
                q.token(G, in, w, i);
            }
            float slope, v = 0.0f;
            const float xv = DT::widen(q.x), d = step_width<DT>(DT::widen(q.dt) + bias, G.soft, slope), u = d * xv;
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                q.h[n] = __builtin_fmaf(__builtin_amdgcn_exp2f(d * a2[n]), q.h[n], u * DT::widen(q.b[n]));
                v = __builtin_fmaf(q.h[n], DT::widen(q.c[n]), v);
            }
            v = __builtin_fmaf(skip, xv, sum_states<LPC>(v));
            if (in.gate) v *= gate_value<DT>(DT::widen(q.z), G.act);
            if (w.j == 0) y[(int64_t)i * ldy + w.c] = rounded<DT>(v);
            if (!shared) break;
        }
        store_states(state + ((int64_t)q.slot * G.C + w.c) * G.N, q.h, 4 * w.j, G.N, true);
    };
    Row<DT> q0, q1;
    int row = (int)(blockIdx.x / G.nblk);
    q0.fetch(G, in, w, state, slots, n_slots, row);
    for (;;) {
        if (rows - row > step) q1.fetch(G, in, w, state, slots, n_slots, row + step);
        compute(q0, row);
        if (rows - row <= step) return;
        row += step;
        if (rows - row > step) q0.fetch(G, in, w, state, slots, n_slots, row + step);
        compute(q1, row);
        if (rows - row <= step) return;
        row += step;
    }
}

// As many workgroups as the card holds at once, eight a CU: 96 and 192 rows of 8192
// channels take 29 and 57.5 us, with half of them 35.7 and 79, with twice 30.5 and 58.4.
constexpr uint32_t WGS = 2048;

template <class DT, int LPC>
hipError_t step(const dwconv_scan_plan &p, const ScanArgs &a, hipStream_t st) {
    ScanGeo G = scan_blocks(p, LPC);
    if (too_many((uint64_t)G.nblk * (uint32_t)a.tokens)) return hipErrorInvalidConfiguration;
    if (a.tokens == 0) return hipSuccess;
    const uint32_t most = (WGS + G.nblk - 1) / G.nblk;
    G.walkers = (uint32_t)a.tokens < most ? (uint32_t)a.tokens : most;
    k_step<DT, LPC><<<G.nblk * G.walkers, 256, 0, st>>>(G, scan_inputs(a), a.state, a.slots, a.n_slots, a.tokens,
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
