// k_norm.hip -- the norm after a block, its gate, residual scale and residual,
// and the norm before the next block (include/dwconv_seq.h), in one pass over
// the rows, and their gradients.
//
// Bound by HBM: each tensor is read or written once.  A row lives in the
// registers of TPR lanes (part of a wavefront, or a workgroup where rows are
// long), E channels a lane, so that the second norm and the backward pass's
// row sums need no second read; the backward pass forms the forward pass's
// values again from its inputs instead of reading stored statistics.
// Sums over rows (gradients of scales, weights and shared gates) stay in
// registers while a workgroup walks its rows and are joined in a fixed order.
#include "seq_common.h"
#include "seq_plan.h"

namespace dw {
namespace {

struct Opt {
    int D, rows, per;
    int after, before, act;
    float eps, inv_d;
};

// sum over the TPR lanes of a row; every lane gets it
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float *sh) {
#pragma unroll
    for (int m = 1; m < (TPR < 64 ? TPR : 64); m <<= 1) v += __shfl_xor(v, m, 64);
    if (TPR > 64) {
        constexpr int W = TPR / 64;
        __syncthreads();  // the previous sum has been read
        if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
        __syncthreads();
        v = 0.0f;
#pragma unroll
        for (int i = 0; i < W; ++i) v += sh[i];
    }
    return v;
}

__device__ __forceinline__ float gate_value(float g, int act) {
    if (act == DWCONV_SEQ_ACT_NONE) return g;
    const float p = sigmoid_f32(g);
    return act == DWCONV_SEQ_ACT_SILU ? g * p : p;
}
__device__ __forceinline__ float gate_slope(float g, int act) {
    if (act == DWCONV_SEQ_ACT_NONE) return 1.0f;
    const float p = sigmoid_f32(g);
    return act == DWCONV_SEQ_ACT_SILU ? p * (1.0f + g * (1.0f - p)) : p * (1.0f - p);
}

// A lane's E channels: NV vectors of VEC, TPR vectors apart.
template <class DT, int VEC, int TPR, int E>
struct Lane {
    static constexpr int NV = E / VEC;
    int D, lane;
    __device__ __forceinline__ int channel(int n) const { return (n * TPR + lane) * VEC; }
    __device__ __forceinline__ void load(float (&v)[E], const typename DT::X *p) const {
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            float part[VEC];
            if (channel(n) < D) {
                load_f32<DT, VEC>(part, p + channel(n));
            } else {
#pragma unroll
                for (int i = 0; i < VEC; ++i) part[i] = 0.0f;
            }
#pragma unroll
            for (int i = 0; i < VEC; ++i) v[n * VEC + i] = part[i];
        }
    }
    __device__ __forceinline__ void store(typename DT::X *p, const float (&v)[E]) const {
#pragma unroll
        for (int n = 0; n < NV; ++n)
            if (channel(n) < D) {
                float part[VEC];
#pragma unroll
                for (int i = 0; i < VEC; ++i) part[i] = v[n * VEC + i];
                store_f32<DT, VEC>(p + channel(n), part);
            }
    }
    __device__ __forceinline__ bool inside(int e) const { return channel(e / VEC) < D; }
};

// Statistics of a norm: v becomes (v - mean) r (the unit row), r is returned.
// Channels past D stay zero.
template <class L, int TPR, int E>
__device__ __forceinline__ float unit_row(float (&v)[E], const L &ln, const Opt &o, int kind, float *sh) {
    if (kind == DWCONV_NORM_NONE) return 1.0f;
    if (kind == DWCONV_NORM_LAYER) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < E; ++i) s += v[i];
        const float mean = row_sum<TPR>(s, sh) * o.inv_d;
#pragma unroll
        for (int i = 0; i < E; ++i) v[i] = ln.inside(i) ? v[i] - mean : 0.0f;
    }
    float q = 0.0f;
#pragma unroll
    for (int i = 0; i < E; ++i) q = __builtin_fmaf(v[i], v[i], q);
    const float r = 1.0f / sqrtf(row_sum<TPR>(q, sh) * o.inv_d + o.eps);
#pragma unroll
    for (int i = 0; i < E; ++i) v[i] *= r;
    return r;
}

// d becomes the gradient of the norm's input: d holds the gradient of the unit
// row (already times w), u the unit row.
template <int TPR, int E>
__device__ __forceinline__ void norm_back(float (&d)[E], const float (&u)[E], float r, const Opt &o, int kind, float *sh) {
    if (kind == DWCONV_NORM_NONE) return;
    float a = 0.0f, m = 0.0f;
#pragma unroll
    for (int i = 0; i < E; ++i) a = __builtin_fmaf(d[i], u[i], a);
    a = row_sum<TPR>(a, sh) * o.inv_d;
    if (kind == DWCONV_NORM_LAYER) {
#pragma unroll
        for (int i = 0; i < E; ++i) m += d[i];
        m = row_sum<TPR>(m, sh) * o.inv_d;
    }
#pragma unroll
    for (int i = 0; i < E; ++i) d[i] = r * (d[i] - m - u[i] * a);
}

template <class DT, int VEC, int TPR, int E>
__global__ void __launch_bounds__(TPR > 256 ? TPR : 256)
    k_fwd(Opt o, const typename DT::X *po, const typename DT::X *pres, const typename DT::X *pgate, const float *scale,
          const float *wa, const float *ba, const float *wb, const float *bb, typename DT::X *ph, typename DT::X *py) {
    __shared__ float sh[16];
    constexpr int RPB = TPR > 256 ? 1 : 256 / TPR;
    using L = Lane<DT, VEC, TPR, E>;
    using LF = Lane<F32, VEC, TPR, E>;
    const L ln{o.D, (int)threadIdx.x % TPR};
    const LF lf{o.D, (int)threadIdx.x % TPR};
    const int64_t row0 = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
    const bool live = row0 < o.rows;
    const int64_t at = (live ? row0 : o.rows - 1) * o.D;  // idle lanes follow the last row
    float v[E], t[E];
    ln.load(v, po + at);
    unit_row<L, TPR, E>(v, ln, o, o.after, sh);
    if (o.after != DWCONV_NORM_NONE) {
        lf.load(t, wa);
#pragma unroll
        for (int i = 0; i < E; ++i) v[i] *= t[i];
        if (ba && o.after == DWCONV_NORM_LAYER) {
            lf.load(t, ba);
#pragma unroll
            for (int i = 0; i < E; ++i) v[i] += t[i];
        }
    }
    if (pgate) {
        ln.load(t, pgate + (live ? row0 : o.rows - 1) / o.per * o.D);
#pragma unroll
        for (int i = 0; i < E; ++i) v[i] *= gate_value(t[i], o.act);
    }
    if (scale) {
        lf.load(t, scale);
#pragma unroll
        for (int i = 0; i < E; ++i) v[i] *= t[i];
    }
    if (pres) {
        ln.load(t, pres + at);
#pragma unroll
        for (int i = 0; i < E; ++i) v[i] += t[i];
    }
    if (ph && live) ln.store(ph + at, v);
    if (o.before == DWCONV_NORM_NONE) return;
    unit_row<L, TPR, E>(v, ln, o, o.before, sh);
    lf.load(t, wb);
#pragma unroll
    for (int i = 0; i < E; ++i) v[i] *= t[i];
    if (bb && o.before == DWCONV_NORM_LAYER) {
        lf.load(t, bb);
#pragma unroll
        for (int i = 0; i < E; ++i) v[i] += t[i];
    }
    if (live) ln.store(py + at, v);
}

// How the backward pass's rows are dealt to workgroups: groups of rows_in rows
// (those of one shared gate row, else all rows), each cut into `segs` pieces of
// seg_rows rows, or `chunk` whole groups to a workgroup (segs == 1).
struct Deal {
    int64_t groups;
    int rows_in, segs, seg_rows, chunk;
    uint32_t blocks;
};

struct Grad {
    const void *dh, *dy;
    void *d_o, *dres, *dgate;
    float *part;       // blocks x 5 x D: dscale, dw_after, db_after, dw_before, db_before
    float *gate_part;  // groups x segs x D, where segs > 1
};

template <class DT, int VEC, int TPR, int E>
__global__ void __launch_bounds__(TPR > 256 ? TPR : 256)
    k_bwd(Opt o, Deal deal, const typename DT::X *po, const typename DT::X *pres, const typename DT::X *pgate,
          const float *scale, const float *wa, const float *ba, const float *wb, Grad gr) {
    using X = typename DT::X;
    constexpr int RPB = TPR > 256 ? 1 : 256 / TPR;
    using L = Lane<DT, VEC, TPR, E>;
    using LF = Lane<F32, VEC, TPR, E>;
    __shared__ float sh[16];
    __shared__ float join[RPB > 1 ? 256 * E : 1];
    const L ln{o.D, (int)threadIdx.x % TPR};
    const LF lf{o.D, (int)threadIdx.x % TPR};
    const int sub = threadIdx.x / TPR;
    const bool shared_gate = pgate && o.per > 1;
    const bool affine = o.after == DWCONV_NORM_LAYER && ba;
    float sum[5][E], gsum[E];
#pragma unroll
    for (int j = 0; j < 5; ++j)
#pragma unroll
        for (int i = 0; i < E; ++i) sum[j][i] = 0.0f;
    // the sum over the workgroup's row lanes, in lane order; lanes of the first
    // row have it
    auto joined = [&](float (&v)[E]) {
        if (RPB == 1) return;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < E; ++i) join[threadIdx.x * E + i] = v[i];
        __syncthreads();
        if (sub == 0) {
            for (int r = 1; r < RPB; ++r)
#pragma unroll
                for (int i = 0; i < E; ++i) v[i] += join[(r * TPR + threadIdx.x) * E + i];
        }
    };
    const int64_t first = deal.segs > 1 ? blockIdx.x / deal.segs : (int64_t)blockIdx.x * deal.chunk;
    const int seg = deal.segs > 1 ? blockIdx.x % deal.segs : 0;
    const int64_t last = first + deal.chunk < deal.groups ? first + deal.chunk : deal.groups;
    for (int64_t grp = first; grp < last; ++grp) {
        const int64_t g0 = grp * deal.rows_in;
        const int64_t g1 = g0 + deal.rows_in < o.rows ? g0 + deal.rows_in : o.rows;
        const int64_t r0 = g0 + (int64_t)seg * deal.seg_rows;
        const int64_t r1 = r0 + deal.seg_rows < g1 ? r0 + deal.seg_rows : g1;
#pragma unroll
        for (int i = 0; i < E; ++i) gsum[i] = 0.0f;
        for (int64_t base = r0; base < r1; base += RPB) {
            const bool live = base + sub < r1;
            const int64_t row = live ? base + sub : r1 - 1;
            const int64_t at = row * o.D;
            float ua[E], n[E], a[E], t[E], h[E], d[E], w[E];
            // forward values
            ln.load(ua, po + at);
            const float ra = unit_row<L, TPR, E>(ua, ln, o, o.after, sh);
#pragma unroll
            for (int i = 0; i < E; ++i) n[i] = ua[i];
            if (o.after != DWCONV_NORM_NONE) {
                lf.load(w, wa);
#pragma unroll
                for (int i = 0; i < E; ++i) n[i] *= w[i];
                if (affine) {
                    lf.load(w, ba);
#pragma unroll
                    for (int i = 0; i < E; ++i) n[i] += w[i];
                }
            }
            if (pgate) {
                ln.load(a, pgate + row / o.per * o.D);
            }
#pragma unroll
            for (int i = 0; i < E; ++i) t[i] = pgate ? n[i] * gate_value(a[i], o.act) : n[i];
            // gradient of h
            if (gr.dh) {
                ln.load(d, (const X *)gr.dh + at);
            } else {
#pragma unroll
                for (int i = 0; i < E; ++i) d[i] = 0.0f;
            }
            if (o.before != DWCONV_NORM_NONE) {
                float dy[E];
#pragma unroll
                for (int i = 0; i < E; ++i) h[i] = t[i];
                if (scale) {
                    lf.load(w, scale);
#pragma unroll
                    for (int i = 0; i < E; ++i) h[i] *= w[i];
                }
                if (pres) {
                    ln.load(w, pres + at);
#pragma unroll
                    for (int i = 0; i < E; ++i) h[i] += w[i];
                }
                const float rb = unit_row<L, TPR, E>(h, ln, o, o.before, sh);
                ln.load(dy, (const X *)gr.dy + at);
                if (live) {
#pragma unroll
                    for (int i = 0; i < E; ++i) {
                        sum[3][i] = __builtin_fmaf(dy[i], h[i], sum[3][i]);
                        sum[4][i] += dy[i];
                    }
                }
                lf.load(w, wb);
#pragma unroll
                for (int i = 0; i < E; ++i) dy[i] *= w[i];
                norm_back<TPR, E>(dy, h, rb, o, o.before, sh);
#pragma unroll
                for (int i = 0; i < E; ++i) d[i] += dy[i];
            }
            if (gr.dres && live) ln.store((X *)gr.dres + at, d);
            // through scale and gate
            if (scale) {
                lf.load(w, scale);
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    if (live) sum[0][i] = __builtin_fmaf(d[i], t[i], sum[0][i]);
                    d[i] *= w[i];
                }
            }
            if (pgate) {
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    w[i] = d[i] * n[i] * gate_slope(a[i], o.act);
                    d[i] *= gate_value(a[i], o.act);
                    if (live) gsum[i] += w[i];
                }
                if (!shared_gate && gr.dgate && live) ln.store((X *)gr.dgate + at, w);
            }
            // through the norm after the block
            if (o.after != DWCONV_NORM_NONE) {
                if (live) {
#pragma unroll
                    for (int i = 0; i < E; ++i) {
                        sum[1][i] = __builtin_fmaf(d[i], ua[i], sum[1][i]);
                        sum[2][i] += d[i];
                    }
                }
                lf.load(w, wa);
#pragma unroll
                for (int i = 0; i < E; ++i) d[i] *= w[i];
                norm_back<TPR, E>(d, ua, ra, o, o.after, sh);
            }
            if (gr.d_o && live) ln.store((X *)gr.d_o + at, d);
        }
        if (shared_gate && gr.dgate) {
            joined(gsum);
            if (sub == 0) {
                if (deal.segs > 1)
                    lf.store(gr.gate_part + (grp * deal.segs + seg) * o.D, gsum);
                else
                    ln.store((X *)gr.dgate + grp * o.D, gsum);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < 5; ++j) {
        joined(sum[j]);
        if (sub == 0) lf.store(gr.part + ((int64_t)blockIdx.x * 5 + j) * o.D, sum[j]);
    }
}

struct Params {
    float *out[5];
};

// Column sums of the workgroups' partial sums: 64 columns a workgroup, wave w
// takes every 16th row from w on, the 16 sums are added in order.
__global__ void __launch_bounds__(1024) k_sum(const float *part, int64_t blocks, int D, Params p) {
    __shared__ float sh[16][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t col = (int64_t)blockIdx.x * 64 + lane, n = 5 * (int64_t)D;
    float s = 0.0f;
    if (col < n && p.out[col / D])
        for (int64_t b = wave; b < blocks; b += 16) s += part[b * n + col];
    sh[wave][lane] = s;
    __syncthreads();
    if (wave || col >= n || !p.out[col / D]) return;
    float r = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) r += sh[i][lane];
    p.out[col / D][col % D] = r;
}

template <class DT>
__global__ void __launch_bounds__(256) k_gate_sum(const float *part, int64_t groups, int segs, int D, typename DT::X *out) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= groups * D) return;
    const float *p = part + i / D * segs * D + i % D;
    float s = 0.0f;
    for (int k = 0; k < segs; ++k) s += p[(int64_t)k * D];
    out[i] = rounded<DT>(s);
}

// Lanes a row and channels a lane.  Short rows share a wavefront; a lane has 8
// channels (five arrays and five sums of them stay in registers), 16 only for
// the longest rows.
int lanes_of(int D) { return D <= 128 ? 16 : D <= 512 ? 64 : D <= 2048 ? 256 : 1024; }

// About 2048 workgroups of 256 lanes fill the chip twice over; each has at
// least 4 rows a lane group to walk, so that its sums are worth writing.
Deal deal_of(int D, int rows, int per) {
    const int tpr = lanes_of(D), rpb = tpr >= 256 ? 1 : 256 / tpr, target = tpr > 256 ? 512 : 2048;
    Deal d{};
    d.rows_in = per > 1 ? per : (rows > 0 ? rows : 1);
    d.groups = ((int64_t)rows + d.rows_in - 1) / d.rows_in;
    d.chunk = 1;
    d.segs = 1;
    if (d.groups >= target) {
        d.chunk = (int)((d.groups + target - 1) / target);
    } else if (d.groups > 0) {
        const int64_t want = (target + d.groups - 1) / d.groups, most = ((int64_t)d.rows_in + 4 * rpb - 1) / (4 * rpb);
        d.segs = (int)(want < most ? want : most);
    }
    d.seg_rows = (d.rows_in + d.segs - 1) / d.segs;
    d.segs = (d.rows_in + d.seg_rows - 1) / d.seg_rows;
    d.blocks = (uint32_t)(d.segs > 1 ? d.groups * d.segs : (d.groups + d.chunk - 1) / d.chunk);
    return d;
}

template <class DT, int VEC, int TPR, int E>
hipError_t launch(bool back, const dwconv_norm_plan &p, const NormArgs &a, hipStream_t st) {
    using X = typename DT::X;
    const Opt o{p.D, a.rows, a.per, p.after, p.before, p.act, p.eps, 1.0f / (float)p.D};
    constexpr int RPB = TPR > 256 ? 1 : 256 / TPR, BLOCK = TPR > 256 ? TPR : 256;
    if (!back) {
        const uint32_t blocks = (uint32_t)(((int64_t)a.rows + RPB - 1) / RPB);
        if ((uint64_t)blocks * BLOCK >= (1ull << 32)) return hipErrorInvalidConfiguration;
        if (blocks)
            k_fwd<DT, VEC, TPR, E><<<blocks, BLOCK, 0, st>>>(o, (const X *)a.o, (const X *)a.residual, (const X *)a.gate,
                                                             a.scale, a.w_after, a.b_after, a.w_before, a.b_before,
                                                             (X *)a.h, (X *)a.y);
        return hipGetLastError();
    }
    const Deal d = deal_of(p.D, a.rows, a.per);
    const Grad gr{a.dh, a.dy, a.d_o, a.dresidual, a.dgate, a.workspace, a.workspace + (int64_t)d.blocks * 5 * p.D};
    if (d.blocks)
        k_bwd<DT, VEC, TPR, E><<<d.blocks, BLOCK, 0, st>>>(o, d, (const X *)a.o, (const X *)a.residual,
                                                           (const X *)a.gate, a.scale, a.w_after, a.b_after,
                                                           a.w_before, gr);
    if (a.gate && a.dgate && a.per > 1 && d.segs > 1)
        k_gate_sum<DT><<<(uint32_t)((d.groups * p.D + 255) / 256), 256, 0, st>>>(gr.gate_part, d.groups, d.segs, p.D,
                                                                                 (X *)a.dgate);
    const Params out{{a.dscale, a.dw_after, a.db_after, a.dw_before, a.db_before}};
    if (a.dscale || a.dw_after || a.db_after || a.dw_before || a.db_before)
        k_sum<<<(uint32_t)((5 * (int64_t)p.D + 63) / 64), 1024, 0, st>>>(gr.part, d.blocks, p.D, out);
    return hipGetLastError();
}

template <class DT, int VEC>
hipError_t pick_row(bool back, const dwconv_norm_plan &p, const NormArgs &a, hipStream_t st) {
    switch (lanes_of(p.D)) {
        case 16: return launch<DT, VEC, 16, 8>(back, p, a, st);
        case 64: return launch<DT, VEC, 64, 8>(back, p, a, st);
        case 256: return launch<DT, VEC, 256, 8>(back, p, a, st);
        default:
            return p.D <= 8192 ? launch<DT, VEC, 1024, 8>(back, p, a, st) : launch<DT, VEC, 1024, 16>(back, p, a, st);
    }
}

template <class DT>
hipError_t pick_vec(bool back, const dwconv_norm_plan &p, const NormArgs &a, hipStream_t st) {
    constexpr int V = 16 / (int)sizeof(typename DT::X);
    const void *ptrs[] = {a.o, a.residual, a.gate, a.scale, a.w_after, a.b_after, a.w_before, a.b_before, a.h, a.y,
                          a.dh, a.dy, a.d_o, a.dresidual, a.dgate, a.workspace};
    uintptr_t bits = 0;
    for (const void *q : ptrs) bits |= (uintptr_t)q;
    return (bits & 15) == 0 && p.D % V == 0 ? pick_row<DT, V>(back, p, a, st) : pick_row<DT, 1>(back, p, a, st);
}

hipError_t pick(bool back, const dwconv_norm_plan &p, const NormArgs &a, hipStream_t st) {
    switch (p.dtype) {
        case DWCONV_F32: return pick_vec<F32>(back, p, a, st);
        case DWCONV_F16: return pick_vec<F16>(back, p, a, st);
        default: return pick_vec<BF16>(back, p, a, st);
    }
}

}  // namespace

hipError_t norm_fwd(const dwconv_norm_plan &p, const NormArgs &a, hipStream_t st) { return pick(false, p, a, st); }
hipError_t norm_bwd(const dwconv_norm_plan &p, const NormArgs &a, hipStream_t st) { return pick(true, p, a, st); }

size_t norm_bwd_bytes(const dwconv_norm_plan &p, int rows, int per) {
    const Deal d = deal_of(p.D, rows, per);
    return ((size_t)d.blocks * 5 + (d.segs > 1 ? (size_t)d.groups * d.segs : 0)) * p.D * sizeof(float);
}

}  // namespace dw
