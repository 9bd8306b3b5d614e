// k_norm.hip -- the norm after a block, its gate, residual scale and residual,
// and the norm before the next block (include/dwconv_seq.h), in one pass over
// the rows, and their gradients.
//
// Bound by HBM up to 4096 channels: each tensor is read or written once.  A row lives in the
// registers of TPR lanes (part of a wavefront, or a workgroup where rows are
// long), E channels a lane, so that the second norm and the backward pass's
// row sums need no second read; the backward pass forms the forward pass's
// values again from its inputs instead of reading stored statistics.
// Sums over rows (gradients of scales, weights and shared gates) stay in
// registers while a workgroup walks its rows and are joined in a fixed order.
// Measured, inputs from HBM: gated norm of 262144 bf16 rows of 128 38 us
// (5.3 TB/s; a large copy 5.15), residual block norm of 8192 rows of 4096 55 us
// (4.9 TB/s); gradients of 200704 fp16 rows of 96 with a gate an image 96 us
// (2.4 TB/s): there vector operations bound, some 60 a channel and eight sums a
// row, with 12 of a row's 16 lanes at work; of 8192 bf16 rows of 4096, residual and
// two norms, 143 us (2.8 TB/s).  Gradients of longer rows run 1024 lanes, which have
// 128 registers each and spill 180 to 1208 of them to memory, again for every row:
// 4096 bf16 rows of 5120 432 us and of 8192 466, where their bytes take 49 and 78.
#include "seq_common.h"
#include "seq_plan.h"

namespace dw {
namespace {

struct Opt {
    int D, rows, per;
    int after, before, act;
    float eps, inv_d;
};

// Sums over the TPR lanes of a row; every lane gets them.  Rows of more than a
// wavefront exchange through LDS, in two places by turns: by the time a place
// is written again all lanes have passed the barrier behind the other one's
// write, and so have read it.
template <int TPR>
struct RowSum {
    float *sh;  // 2 x 2 x 16
    int turn = 0;
    __device__ __forceinline__ RowSum(float *sh) : sh(sh) {}
    __device__ __forceinline__ void two(float &a, float &b) {
        if (TPR == 16) {
            a = sum_row16(a);
            b = sum_row16(b);
            return;
        }
        a = sum_wave(a);
        b = sum_wave(b);
        if (TPR > 64) {
            constexpr int W = TPR / 64;
            float *p = sh + turn * 32;
            turn ^= 1;
            if ((threadIdx.x & 63) == 0) {
                p[threadIdx.x >> 6] = a;
                p[16 + (threadIdx.x >> 6)] = b;
            }
            __syncthreads();
            a = b = 0.0f;
#pragma unroll
            for (int i = 0; i < W; ++i) {
                a += p[i];
                b += p[16 + i];
            }
        }
    }
    __device__ __forceinline__ float one(float a) {
        float b = 0.0f;
        two(a, b);
        return a;
    }
};

// A lane's E channels: NV vectors of VEC, TPR vectors apart.  Vectors past D
// are read as the row's first one (no branch around a load) and count as zeros.
template <class DT, int VEC, int TPR, int E>
struct Lane {
    using X = typename DT::X;
    static constexpr int NV = E / VEC;
    struct Raw {
        Vec<X, VEC> v[NV];
    };
    int D, lane;
    __device__ __forceinline__ int channel(int n) const { return (n * TPR + lane) * VEC; }
    __device__ __forceinline__ bool inside(int e) const { return channel(e / VEC) < D; }
    __device__ __forceinline__ void fetch(Raw &r, const X *p) const {
#pragma unroll
        for (int n = 0; n < NV; ++n) r.v[n] = *(const Vec<X, VEC> *)(p + (channel(n) < D ? channel(n) : 0));
    }
    __device__ __forceinline__ void widen(float (&v)[E], const Raw &r) const {
#pragma unroll
        for (int i = 0; i < E; ++i) v[i] = inside(i) ? DT::widen(r.v[i / VEC].v[i % VEC]) : 0.0f;
    }
    __device__ __forceinline__ void load(float (&v)[E], const X *p) const {
        Raw r;
        fetch(r, p);
        widen(v, r);
    }
    __device__ __forceinline__ void store(X *p, const float (&v)[E]) const {
#pragma unroll
        for (int n = 0; n < NV; ++n)
            if (channel(n) < D) {
                float part[VEC];
#pragma unroll
                for (int i = 0; i < VEC; ++i) part[i] = v[n * VEC + i];
                store_f32<DT, VEC>(p + channel(n), part);
            }
    }
};

// Statistics of a norm: v becomes (v - mean) r (the unit row), r is returned.
// Channels past D stay zero.
template <int TPR, class L, int E>
__device__ __forceinline__ float unit_row(float (&v)[E], const L &ln, const Opt &o, int kind, RowSum<TPR> &sum) {
    if (kind == DWCONV_NORM_NONE) return 1.0f;
    if (kind == DWCONV_NORM_LAYER) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < E; ++i) s += v[i];
        const float mean = sum.one(s) * o.inv_d;
#pragma unroll
        for (int i = 0; i < E; ++i) v[i] = ln.inside(i) ? v[i] - mean : 0.0f;
    }
    float q = 0.0f;
#pragma unroll
    for (int i = 0; i < E; ++i) q = __builtin_fmaf(v[i], v[i], q);
    const float r = 1.0f / sqrtf(sum.one(q) * o.inv_d + o.eps);
#pragma unroll
    for (int i = 0; i < E; ++i) v[i] *= r;
    return r;
}

// d becomes the gradient of the norm's input: d holds the gradient of the unit
// row (already times w), u the unit row.
template <int TPR, int E>
__device__ __forceinline__ void norm_back(float (&d)[E], const float (&u)[E], float r, const Opt &o, int kind, RowSum<TPR> &sum) {
    if (kind == DWCONV_NORM_NONE) return;
    float a = 0.0f, m = 0.0f;
#pragma unroll
    for (int i = 0; i < E; ++i) {
        a = __builtin_fmaf(d[i], u[i], a);
        m += d[i];
    }
    sum.two(a, m);
    a *= o.inv_d;
    m = kind == DWCONV_NORM_LAYER ? m * o.inv_d : 0.0f;
#pragma unroll
    for (int i = 0; i < E; ++i) d[i] = r * (d[i] - m - u[i] * a);
}

template <class DT, int VEC, int TPR, int E>
__global__ void __launch_bounds__(TPR > 256 ? TPR : 256)
    k_fwd(Opt o, const typename DT::X *po, const typename DT::X *pres, const typename DT::X *pgate, const float *scale,
          const float *wa, const float *ba, const float *wb, const float *bb, typename DT::X *ph, typename DT::X *py) {
    __shared__ float sh[64];
    RowSum<TPR> sum(sh);
    constexpr int RPB = TPR > 256 ? 1 : 256 / TPR;
    using L = Lane<DT, VEC, TPR, E>;
    using LF = Lane<F32, VEC, TPR, E>;
    const L ln{o.D, (int)threadIdx.x % TPR};
    const LF lf{o.D, (int)threadIdx.x % TPR};
    const int64_t row0 = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
    const bool live = row0 < o.rows;
    const int64_t at = (live ? row0 : o.rows - 1) * o.D;  // idle lanes follow the last row
    // the row's tensors at once, then the parameters
    typename L::Raw ro, rg, rr;
    ln.fetch(ro, po + at);
    if (pgate) ln.fetch(rg, pgate + (live ? row0 : o.rows - 1) / o.per * o.D);
    if (pres) ln.fetch(rr, pres + at);
    float v[E], t[E];
    ln.widen(v, ro);
    unit_row(v, ln, o, o.after, sum);
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
        ln.widen(t, rg);
#pragma unroll
        for (int i = 0; i < E; ++i) v[i] *= gate_value<DT>(t[i], o.act);
    }
    if (scale) {
        lf.load(t, scale);
#pragma unroll
        for (int i = 0; i < E; ++i) v[i] *= t[i];
    }
    if (pres) {
        ln.widen(t, rr);
#pragma unroll
        for (int i = 0; i < E; ++i) v[i] += t[i];
    }
    if (ph && live) ln.store(ph + at, v);
    if (o.before == DWCONV_NORM_NONE) return;
    unit_row(v, ln, o, o.before, sum);
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
    // workgroups of 1024 lanes have 128 registers a lane: they read parameters
    // again for each row and take its tensors when it is its turn
    constexpr bool AHEAD = TPR <= 512;
    using L = Lane<DT, VEC, TPR, E>;
    using LF = Lane<F32, VEC, TPR, E>;
    __shared__ float sh[64];
    __shared__ float join[RPB > 1 ? 256 * E : 1];
    RowSum<TPR> rs(sh);
    const L ln{o.D, (int)threadIdx.x % TPR};
    const LF lf{o.D, (int)threadIdx.x % TPR};
    const int sub = threadIdx.x / TPR;
    const bool shared_gate = pgate && o.per > 1;
    if (o.after != DWCONV_NORM_LAYER) ba = nullptr;
    if (o.after == DWCONV_NORM_NONE) wa = nullptr;
    if (o.before == DWCONV_NORM_NONE) wb = nullptr;
    float sum[5][E], gsum[E];
#pragma unroll
    for (int j = 0; j < 5; ++j)
#pragma unroll
        for (int i = 0; i < E; ++i) sum[j][i] = 0.0f;
    // parameters (scale, w_after, b_after, w_before), where they are given
    float par[AHEAD ? 4 : 1][E];
    auto param = [&](int k) { return k == 0 ? scale : k == 1 ? wa : k == 2 ? ba : wb; };
    if (AHEAD) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (param(k)) lf.load(par[AHEAD ? k : 0], param(k));
    }
    auto get = [&](int k) -> const float(&)[E] {
        if (!AHEAD) lf.load(par[0], param(k));
        return par[AHEAD ? k : 0];
    };
    // the sum over the workgroup's row lanes, in lane order; lanes of the first
    // row have it
    auto joined = [&](float (&v)[E]) {
        if (RPB == 1) return;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < E; ++i) join[i * 256 + threadIdx.x] = v[i];
        __syncthreads();
        if (sub == 0) {
#pragma unroll
            for (int i = 0; i < E; ++i)
                for (int r = 1; r < RPB; ++r) v[i] += join[i * 256 + r * TPR + threadIdx.x];
        }
    };
    typename L::Raw ro, rr, rh, ry, rg;
    auto take = [&](int64_t row) {
        const int64_t at = row * o.D;
        ln.fetch(ro, po + at);
        if (pres && wb) ln.fetch(rr, pres + at);
        if (gr.dh) ln.fetch(rh, (const X *)gr.dh + at);
        if (wb) ln.fetch(ry, (const X *)gr.dy + at);
        if (pgate && !shared_gate) ln.fetch(rg, pgate + row / o.per * o.D);
    };
    // act(gate) and its slope, of a row or of all rows of a shared gate
    float a[E], slope[E];
    auto gates = [&] {
        ln.widen(a, rg);
#pragma unroll
        for (int i = 0; i < E; ++i) a[i] = gate_value<DT>(a[i], o.act, slope[i]);
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
        if (r0 < r1) {
            if (AHEAD) take(r0 + sub < r1 ? r0 + sub : r1 - 1);
            if (shared_gate) {
                ln.fetch(rg, pgate + grp * o.D);
                gates();
            }
        }
        for (int64_t base = r0; base < r1; base += RPB) {
            const bool live = base + sub < r1;
            const int64_t row = live ? base + sub : r1 - 1;
            const int64_t at = row * o.D;
            float ua[E], t[E], h[E], d[E], dy[E];
            if (!AHEAD) take(row);
            ln.widen(ua, ro);
            if (pgate && !shared_gate) gates();
#pragma unroll
            for (int i = 0; i < E; ++i) d[i] = dy[i] = h[i] = 0.0f;
            if (gr.dh) ln.widen(d, rh);
            if (wb) {
                ln.widen(dy, ry);
                if (pres) ln.widen(h, rr);
            }
            if (AHEAD && base + RPB < r1) take(base + RPB + sub < r1 ? base + RPB + sub : r1 - 1);
            // forward values: t = N_after(o) act(gate)
            const float ra = unit_row(ua, ln, o, o.after, rs);
#pragma unroll
            for (int i = 0; i < E; ++i) t[i] = ua[i];
            if (wa) {
                const float(&w)[E] = get(1);
#pragma unroll
                for (int i = 0; i < E; ++i) t[i] *= w[i];
            }
            if (ba) {
                const float(&w)[E] = get(2);
#pragma unroll
                for (int i = 0; i < E; ++i) t[i] += w[i];
            }
            float dgate[E];
            if (pgate) {
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    dgate[i] = t[i] * slope[i];
                    t[i] *= a[i];
                }
            }
            // gradient of h
            if (wb) {
                if (scale) {
                    const float(&w)[E] = get(0);
#pragma unroll
                    for (int i = 0; i < E; ++i) h[i] = __builtin_fmaf(t[i], w[i], h[i]);
                } else {
#pragma unroll
                    for (int i = 0; i < E; ++i) h[i] += t[i];
                }
                const float rb = unit_row(h, ln, o, o.before, rs);
                if (live) {
#pragma unroll
                    for (int i = 0; i < E; ++i) {
                        sum[3][i] = __builtin_fmaf(dy[i], h[i], sum[3][i]);
                        sum[4][i] += dy[i];
                    }
                }
                const float(&w)[E] = get(3);
#pragma unroll
                for (int i = 0; i < E; ++i) dy[i] *= w[i];
                norm_back(dy, h, rb, o, o.before, rs);
#pragma unroll
                for (int i = 0; i < E; ++i) d[i] += dy[i];
            }
            if (gr.dres && live) ln.store((X *)gr.dres + at, d);
            // through scale and gate
            if (scale) {
                const float(&w)[E] = get(0);
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    if (live) sum[0][i] = __builtin_fmaf(d[i], t[i], sum[0][i]);
                    d[i] *= w[i];
                }
            }
            if (pgate) {
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    dgate[i] *= d[i];
                    d[i] *= a[i];
                    if (live) gsum[i] += dgate[i];
                }
                if (!shared_gate && gr.dgate && live) ln.store((X *)gr.dgate + at, dgate);
            }
            // through the norm after the block
            if (wa) {
                if (live) {
#pragma unroll
                    for (int i = 0; i < E; ++i) {
                        sum[1][i] = __builtin_fmaf(d[i], ua[i], sum[1][i]);
                        sum[2][i] += d[i];
                    }
                }
                const float(&w)[E] = get(1);
#pragma unroll
                for (int i = 0; i < E; ++i) d[i] *= w[i];
                norm_back(d, ua, ra, o, o.after, rs);
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
// takes every 16th row from w on (four rows at a time), the 16 sums are added in
// order.  Workgroups behind `param_blocks` sum the pieces of shared gates.
template <class DT>
__global__ void __launch_bounds__(1024) k_sum(const float *part, int64_t blocks, int D, Params p, uint32_t param_blocks,
                                              const float *gates, int64_t groups, int segs, typename DT::X *dgate) {
    if (blockIdx.x >= param_blocks) {
        const int64_t i = (int64_t)(blockIdx.x - param_blocks) * 1024 + threadIdx.x;
        if (i >= groups * D) return;
        const float *q = gates + i / D * segs * D + i % D;
        float s = 0.0f;
        int k = 0;
        for (; k + 4 <= segs; k += 4) {
            const float a = q[(int64_t)k * D], b = q[(int64_t)(k + 1) * D], c = q[(int64_t)(k + 2) * D],
                        d = q[(int64_t)(k + 3) * D];
            s += (a + b) + (c + d);
        }
        for (; k < segs; ++k) s += q[(int64_t)k * D];
        dgate[i] = rounded<DT>(s);
        return;
    }
    __shared__ float sh[16][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t col = (int64_t)blockIdx.x * 64 + lane, n = 5 * (int64_t)D;
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (col < n && p.out[col / D]) {
        const float *q = part + col;
        int64_t b = wave;
        for (; b + 48 < blocks; b += 64) {
#pragma unroll
            for (int i = 0; i < 4; ++i) s[i] += q[(b + 16 * i) * n];
        }
        for (; b < blocks; b += 16) s[0] += q[b * n];
    }
    sh[wave][lane] = (s[0] + s[1]) + (s[2] + s[3]);
    __syncthreads();
    if (wave || col >= n || !p.out[col / D]) return;
    float r = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) r += sh[i][lane];
    p.out[col / D][col % D] = r;
}

// Lanes a row of the backward pass, 8 channels each (their arrays and sums stay
// in registers up to 512 lanes; 16 only for rows of more than 8192); the forward
// pass takes 16 channels a lane where that saves lanes (8192 bf16 rows from HBM, 16
// channels against 8: 16 and 23 us at D = 1024, 38 and 43 at 2560, 53 and 52 at 4096).
int lanes_of(int D) { return D <= 128 ? 16 : D <= 512 ? 64 : D <= 2048 ? 256 : D <= 4096 ? 512 : 1024; }

// Two workgroups a CU (one of more than 256 lanes), each with rows enough for
// its sums to be worth writing: more write more sums and read parameters more
// often, fewer leave loads without company.  Inputs from HBM, with the join, one, two,
// three and four a CU: 200704 fp16 rows of 96 146, 97, 124 and 109 us, 262144 bf16
// rows of 128 157, 101, 129 and 106; 8192 bf16 rows of 4096, one, three and four:
// 143, 157 and 164 us, 4096 of 8192 466, 558 and 565.
Deal deal_of(int D, int rows, int per) {
    const int tpr = lanes_of(D), rpb = tpr >= 256 ? 1 : 256 / tpr, target = tpr > 256 ? 256 : 512;
    Deal d{};
    d.rows_in = per > 1 && per < rows ? per : (rows > 0 ? rows : 1);
    d.groups = ((int64_t)rows + d.rows_in - 1) / d.rows_in;
    d.chunk = 1;
    d.segs = 1;
    if (d.groups >= target) {
        d.chunk = (int)((d.groups + target - 1) / target);
    } else if (d.groups > 0) {
        const int64_t want = (target + d.groups - 1) / d.groups, most = ((int64_t)d.rows_in + 4 * rpb - 1) / (4 * rpb);
        d.segs = (int)(want < most ? want : most);
    }
    d.seg_rows = (int)(((int64_t)d.rows_in + d.segs - 1) / d.segs);
    d.segs = (int)(((int64_t)d.rows_in + d.seg_rows - 1) / d.seg_rows);
    d.blocks = (uint32_t)(d.segs > 1 ? d.groups * d.segs : (d.groups + d.chunk - 1) / d.chunk);
    return d;
}

template <bool BACK, class DT, int VEC, int TPR, int E>
hipError_t launch(const dwconv_norm_plan &p, const NormArgs &a, hipStream_t st) {
    using X = typename DT::X;
    const Opt o{p.D, a.rows, a.per, p.after, p.before, p.act, p.eps, 1.0f / (float)p.D};
    constexpr int RPB = TPR > 256 ? 1 : 256 / TPR, BLOCK = TPR > 256 ? TPR : 256;
    if constexpr (!BACK) {
        const uint32_t blocks = (uint32_t)(((int64_t)a.rows + RPB - 1) / RPB);
        if ((uint64_t)blocks * BLOCK >= (1ull << 32)) return hipErrorInvalidConfiguration;
        if (blocks)
            k_fwd<DT, VEC, TPR, E><<<blocks, BLOCK, 0, st>>>(o, (const X *)a.o, (const X *)a.residual, (const X *)a.gate,
                                                             a.scale, a.w_after, a.b_after, a.w_before, a.b_before,
                                                             (X *)a.h, (X *)a.y);
        return hipGetLastError();
    } else {
        const Deal d = deal_of(p.D, a.rows, a.per);
        const Grad gr{a.dh, a.dy, a.d_o, a.dresidual, a.dgate, a.workspace, a.workspace + (int64_t)d.blocks * 5 * p.D};
        if (d.blocks)
            k_bwd<DT, VEC, TPR, E><<<d.blocks, BLOCK, 0, st>>>(o, d, (const X *)a.o, (const X *)a.residual,
                                                               (const X *)a.gate, a.scale, a.w_after, a.b_after,
                                                               a.w_before, gr);
        const Params out{{a.dscale, a.dw_after, a.db_after, a.dw_before, a.db_before}};
        const bool any = a.dscale || a.dw_after || a.db_after || a.dw_before || a.db_before;
        const uint32_t pb = any ? (uint32_t)((5 * (int64_t)p.D + 63) / 64) : 0;
        const uint32_t gb = a.gate && a.dgate && a.per > 1 && d.segs > 1 ? (uint32_t)((d.groups * p.D + 1023) / 1024) : 0;
        if (pb + gb)
            k_sum<DT><<<pb + gb, 1024, 0, st>>>(gr.part, d.blocks, p.D, out, pb, gr.gate_part, d.groups, d.segs,
                                                (X *)a.dgate);
        return hipGetLastError();
    }
}

template <bool BACK, class DT, int VEC>
hipError_t pick_row(const dwconv_norm_plan &p, const NormArgs &a, hipStream_t st) {
    const int D = p.D;
    if (D <= 128) return launch<BACK, DT, VEC, 16, 8>(p, a, st);
    if (D <= 512) return launch<BACK, DT, VEC, 64, 8>(p, a, st);
    if constexpr (BACK) {
        if (D <= 2048) return launch<true, DT, VEC, 256, 8>(p, a, st);
        if (D <= 4096) return launch<true, DT, VEC, 512, 8>(p, a, st);
    } else {
        if (D <= 1024) return launch<false, DT, VEC, 64, 16>(p, a, st);
        if (D <= 2048) return launch<false, DT, VEC, 256, 8>(p, a, st);
        if (D <= 4096) return launch<false, DT, VEC, 256, 16>(p, a, st);
    }
    return D <= 8192 ? launch<BACK, DT, VEC, 1024, 8>(p, a, st) : launch<BACK, DT, VEC, 1024, 16>(p, a, st);
}

template <bool BACK, class DT>
hipError_t pick_vec(const dwconv_norm_plan &p, const NormArgs &a, hipStream_t st) {
    constexpr int V = 16 / (int)sizeof(typename DT::X);
    const void *ptrs[] = {a.o, a.residual, a.gate, a.scale, a.w_after, a.b_after, a.w_before, a.b_before, a.h, a.y,
                          a.dh, a.dy, a.d_o, a.dresidual, a.dgate, a.workspace};
    uintptr_t bits = 0;
    for (const void *q : ptrs) bits |= (uintptr_t)q;
    return (bits & 15) == 0 && p.D % V == 0 ? pick_row<BACK, DT, V>(p, a, st) : pick_row<BACK, DT, 1>(p, a, st);
}

template <bool BACK>
hipError_t pick(const dwconv_norm_plan &p, const NormArgs &a, hipStream_t st) {
    switch (p.dtype) {
        case DWCONV_F32: return pick_vec<BACK, F32>(p, a, st);
        case DWCONV_F16: return pick_vec<BACK, F16>(p, a, st);
        default: return pick_vec<BACK, BF16>(p, a, st);
    }
}

}  // namespace

hipError_t norm_fwd(const dwconv_norm_plan &p, const NormArgs &a, hipStream_t st) { return pick<false>(p, a, st); }
hipError_t norm_bwd(const dwconv_norm_plan &p, const NormArgs &a, hipStream_t st) { return pick<true>(p, a, st); }

size_t norm_bwd_bytes(const dwconv_norm_plan &p, int rows, int per) {
    const Deal d = deal_of(p.D, rows, per);
    return ((size_t)d.blocks * 5 + (per > 1 && d.segs > 1 ? (size_t)d.groups * d.segs : 0)) * p.D * sizeof(float);
}

}  // namespace dw
