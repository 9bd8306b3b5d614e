// k_delta_step.hip -- one token of the gated delta rule for each of many
// cached sequences (include/dwconv_seq.h).
//
// Bound by HBM: a head's state is read and written once (8 bytes an element
// against 6 operations).  A workgroup holds columns of one head's state in
// registers, lanes side by side along a row of it.  With a = e^g and the sums
// x = S^T k and y = S^T q over the state as it was,
//   u = beta (v - a x),   o = a y + (k . q) u,   S <- a S + k u^T
// so both sums come from one pass and one exchange through LDS.
// Measured, bf16, 32 heads of 128 x 128, states from HBM: 96 sequences 86 us
// (4.7 TB/s; a large copy 5.15), one sequence 5.5 us.
#include "seq_common.h"
#include "seq_plan.h"

namespace dw {
namespace {

struct Ctx {
    int Hk, Hv, Dk, Dv, rows, n_slots, nb;  // nb: workgroups a head
    float scale, eps;
    int normalize;
    const void *q, *k, *v;
    int64_t ldq, ldk, ldv, ldo;
    const float *g, *beta;
    float *state;
    const int32_t *slots;
    void *o;
};

// LC lanes side by side, VEC columns each; 256 / LC row groups; a lane has
// rows group, group + 256 / LC, ... of the state, NR of them.
template <class DT, int VEC, int LC, int NR>
__global__ void __launch_bounds__(256) k_step(Ctx c) {
    using X = typename DT::X;
    constexpr int RG = 256 / LC, COLS = LC * VEC;
    __shared__ float sk[256], sq[256], red[2][4][COLS];
    const int blk = blockIdx.x % c.nb, h = blockIdx.x / c.nb % c.Hv, row0 = blockIdx.x / c.nb / c.Hv;
    const SlotRows sr = slot_rows(c.slots, c.n_slots, c.rows, row0);
    if (sr.slot < 0) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int lc = tid % LC, rg = tid / LC, col = blk * COLS + lc * VEC;
    const bool in = col < c.Dv;
    float *st = c.state + ((int64_t)sr.slot * c.Hv + h) * c.Dk * c.Dv + col;
    float S[NR][VEC];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        const int x = rg + i * RG;
        if (in && x < c.Dk) {
            load_f32<F32, VEC>(S[i], st + (int64_t)x * c.Dv);
        } else {
#pragma unroll
            for (int j = 0; j < VEC; ++j) S[i][j] = 0.0f;
        }
    }
    const int hk = h / (c.Hv / c.Hk);
    for (int row = row0; row < c.rows; ++row) {
        if (row != row0 && c.slots[row] != sr.slot) continue;
        const float kx = tid < c.Dk ? DT::widen(((const X *)c.k)[row * c.ldk + (int64_t)hk * c.Dk + tid]) : 0.0f;
        const float qx = tid < c.Dk ? DT::widen(((const X *)c.q)[row * c.ldq + (int64_t)hk * c.Dk + tid]) : 0.0f;
        const float gx = c.g[(int64_t)row * c.Hv + h], be = c.beta[(int64_t)row * c.Hv + h];
        float v[VEC];
        if (in) {
            load_f32<DT, VEC>(v, (const X *)c.v + row * c.ldv + (int64_t)h * c.Dv + col);
        } else {
#pragma unroll
            for (int j = 0; j < VEC; ++j) v[j] = 0.0f;
        }
        sk[tid] = kx;
        sq[tid] = qx;
        __syncthreads();
        // |k|, |q| and k . q: every wavefront for itself
        float kk = 0.0f, qq = 0.0f, kq = 0.0f;
#pragma unroll
        for (int i = 0; i < 256; i += 64) {
            const float a = sk[i + lane], b = sq[i + lane];
            kk = __builtin_fmaf(a, a, kk);
            qq = __builtin_fmaf(b, b, qq);
            kq = __builtin_fmaf(a, b, kq);
        }
        float xs[VEC], ys[VEC], kr[NR];
#pragma unroll
        for (int j = 0; j < VEC; ++j) xs[j] = ys[j] = 0.0f;
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            const int x = rg + i * RG;  // < 256
            kr[i] = sk[x];
            const float b = sq[x];
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                xs[j] = __builtin_fmaf(S[i][j], kr[i], xs[j]);
                ys[j] = __builtin_fmaf(S[i][j], b, ys[j]);
            }
        }
#pragma unroll
        for (int m = 1; m < 64; m <<= 1) {
            kk += __shfl_xor(kk, m, 64);
            qq += __shfl_xor(qq, m, 64);
            kq += __shfl_xor(kq, m, 64);
        }
#pragma unroll
        for (int m = LC; m < 64; m <<= 1)
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                xs[j] += __shfl_xor(xs[j], m, 64);
                ys[j] += __shfl_xor(ys[j], m, 64);
            }
        if (lane < LC)
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                red[0][wave][lc * VEC + j] = xs[j];
                red[1][wave][lc * VEC + j] = ys[j];
            }
        __syncthreads();
        const float rk = c.normalize ? 1.0f / sqrtf(kk + c.eps) : 1.0f;
        const float rq = c.scale * (c.normalize ? 1.0f / sqrtf(qq + c.eps) : 1.0f);
        const float a = expf(gx);
        float u[VEC], o[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            const int x = lc * VEC + j;
            const float sx = (red[0][0][x] + red[0][1][x]) + (red[0][2][x] + red[0][3][x]);
            const float sy = (red[1][0][x] + red[1][1][x]) + (red[1][2][x] + red[1][3][x]);
            u[j] = be * (v[j] - a * (rk * sx));
            o[j] = a * (rq * sy) + kq * rk * rq * u[j];
        }
        if (in && rg == 0) store_f32<DT, VEC>((X *)c.o + row * c.ldo + (int64_t)h * c.Dv + col, o);
#pragma unroll
        for (int i = 0; i < NR; ++i)
#pragma unroll
            for (int j = 0; j < VEC; ++j) S[i][j] = __builtin_fmaf(kr[i] * rk, u[j], a * S[i][j]);
        if (!sr.shared) break;
        __syncthreads();  // the next row's values overwrite LDS
    }
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        const int x = rg + i * RG;
        if (in && x < c.Dk) store_f32<F32, VEC>(st + (int64_t)x * c.Dv, S[i]);
    }
}

template <class DT, int VEC, int LC, int NR>
hipError_t launch(Ctx c, hipStream_t st) {
    c.nb = (c.Dv + LC * VEC - 1) / (LC * VEC);
    const uint64_t blocks = (uint64_t)c.rows * c.Hv * c.nb;
    if (blocks >= (1u << 24)) return hipErrorInvalidConfiguration;
    if (blocks) k_step<DT, VEC, LC, NR><<<(uint32_t)blocks, 256, 0, st>>>(c);
    return hipGetLastError();
}

template <class DT>
hipError_t pick(const Ctx &c, hipStream_t st) {
    using X = typename DT::X;
    const bool vec = c.Dv % 4 == 0 && c.ldv % 4 == 0 && c.ldo % 4 == 0 && ((uintptr_t)c.state & 15) == 0 &&
                     (((uintptr_t)c.v | (uintptr_t)c.o) & (4 * sizeof(X) - 1)) == 0;
    const int pad = (c.Dk + 63) / 64;
    if (!vec) return pad <= 2 ? launch<DT, 1, 32, 16>(c, st) : launch<DT, 1, 32, 32>(c, st);
    // 32 columns a workgroup, whose lanes have few rows each; 128, which read whole
    // 512-byte rows, where the heads make two to four workgroups a CU.  States from
    // HBM, bf16, 32 heads of 128 x 128, 32 and 128 columns: 1 sequence 5.5 and 7.8 us,
    // 4: 7.8 and 9.6, 8: 13.0 and 12.8, 16: 21.4 and 19.4, 32: 34.9 and 36.0, 64: 59.6
    // and 64.7, 96: 86 and 90, 192: 167 and 165; 16 and 48 sequences with keys of 256:
    // 34.1 and 33.5, 84.8 and 93.2; 24 and (16 heads of 64 x 64) 192 sequences with keys
    // of 64: 20.4 and 15.7, 63.5 and 65.9.  (Where the finer grid passes its limit too.)
    const int64_t heads = (int64_t)c.rows * c.Hv;
    if (heads < 512 || (heads >= 1024 && heads * ((c.Dv + 31) / 32) < (1 << 24)))
        return pad <= 2 ? launch<DT, 4, 8, 4>(c, st) : launch<DT, 4, 8, 8>(c, st);
    return pad <= 2 ? launch<DT, 4, 32, 16>(c, st) : launch<DT, 4, 32, 32>(c, st);
}

}  // namespace

hipError_t delta_step(const dwconv_delta_plan &p, const DeltaArgs &a, hipStream_t st) {
    const Ctx c{p.Hk, p.Hv, p.Dk, p.Dv, a.tokens, a.n_slots, 0, p.scale, p.eps, p.normalize, a.q, a.k, a.v,
                a.ldq, a.ldk, a.ldv, a.ldo, a.g, a.beta, a.state, a.slots, a.o};
    switch (p.dtype) {
        case DWCONV_F32: return pick<F32>(c, st);
        case DWCONV_F16: return pick<F16>(c, st);
        default: return pick<BF16>(c, st);
    }
}

}  // namespace dw
