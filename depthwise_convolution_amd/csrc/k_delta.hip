// k_delta.hip -- the gated delta rule over packed sequences, forward and
// backward (include/dwconv_seq.h), 64 tokens (a chunk) at a time.
//
// With b the running sum of g within a chunk, S0 the state before it and
// D_ij = e^{b_i - b_j} for i >= j (rows are tokens; q and k stand for the unit
// vectors, c for the scale):
//
//   A = strictly lower part of beta_i D_ij (k_i . k_j),  T = (1 + A)^-1
//   R = beta (V - e^b (K S0)),   U = T R
//   O = c e^b (Q S0) + P U,      P = c D (Q K^T), lower part
//   S1 = e^{b_last} S0 + K^T (e^{b_last - b} U)
//
// T and P need no state: k_prepare makes them for all chunks at once.  The
// scan then walks a sequence's chunks; its columns of S are independent, so a
// wavefront owns 16 columns, holds its part of S in registers for the whole
// sequence and never waits for another wavefront's result.  The result layout
// of a 16x16 matrix product (lane: column l % 16, rows 4 (l / 16) + i) is the
// layout of its right operand if the sum runs over 4 (l / 16) + i, so
// products chain from register to register and only left operands come from
// LDS.
//
// Backward, with dS the gradient of S1 and dO of O:
//
//   dU = P^T dO + e^{b_last - b} (K dS),  dR = T^T dU,  dV = beta dR
//   dS0 = e^{b_last} dS + Q^T (c e^b dO) - K^T (e^b beta dR)
//
// walks the chunks backwards in the same way (k_rscan) after a forward walk
// that keeps every chunk's S0 and U.  The rest needs no order and sums over
// the columns of S (k_grad):
//
//   dP = dO U^T, dA = -dR U^T, E = c dP D, M = beta dA D
//   dQ = c e^b (dO S0^T) + E K
//   dK = E^T Q + (M + M^T) K + e^{b_last - b} (U dS^T) - e^b beta (dR S0^T)
//   db: each exponent's derivative; dg_i = sum of db_j, j >= i
//   dbeta = dR . (V - e^b K S0) + row sums of dA D (K K^T)
//
// b is summed in 64 bits (a difference of two far sums would lose the small
// exponents next to a reset); decays below e^-1000 are zero either way, so g
// is cut there and -infinity needs no case of its own.
//
// The kernels of this file do all products on the fp32 matrix cores and serve
// fp32 data; bf16 and fp16 data take the same steps in k_delta_split.hip and
// k_delta_grad.hip.
//
// Bound by fp32 matrix products (the walks: one wavefront's chain of them).
// Measured, fp32, heads of 128 x 128: 8192 tokens, 16 key and 32 value heads,
// five sequences: k_prepare 176 us, k_scan 646; gradients of 4096 tokens, 8 and
// 16 heads, four sequences: k_prepare 61, k_scan 230, k_rscan 302, k_grad 422 (with
// 62 spilled registers a lane; 319 and 393 at keys of 192 and 256).  The forward walk's
// products would take 197 us at the rate of a large fp32 product; here one wavefront
// has the whole chain for 16 columns.
#include <type_traits>

#include "delta_common.h"

namespace dw {
namespace {

using namespace delta;

template <class DT, int DK>
__global__ void __launch_bounds__(256) k_prepare(Ctx c) {
    using X = typename DT::X;
    extern __shared__ float lds[];
    float (*K)[DK + 4] = (float (*)[DK + 4])lds;
    float (*Q)[DK + 4] = K + CH;
    float *At = (float *)(Q + CH);  // A, lower tiles
    float *Td = At + TRI;           // inverses of A's diagonal tiles
    __shared__ double b[CH];
    __shared__ float beta[CH];
    const int slot = blockIdx.x / c.Hk, hk = blockIdx.x % c.Hk;
    const Chunk ch = chunk_of(c.seq, slot);
    if (ch.n == 0) return;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r = lane & 15, g4 = (lane >> 4) * 4;
    stage_unit<DT, DK>(K, (const X *)c.k + ch.tok * c.ldk + (int64_t)hk * c.Dk, c.ldk, ch.n, c, nullptr);
    stage_unit<DT, DK>(Q, (const X *)c.q + ch.tok * c.ldq + (int64_t)hk * c.Dk, c.ldq, ch.n, c, nullptr);
    __syncthreads();
    // wave w: tiles (w, j), j <= w, of K K^T and Q K^T
    f32x4 kk[4], qk[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        kk[j] = qk[j] = splat(0.0f);
        if (j > wave) continue;
        for (int t = 0; t < DK; t += 16) {
            const f32x4 x = *(const f32x4 *)&K[16 * j + r][t + g4];
            kk[j] = mfma16(*(const f32x4 *)&K[16 * wave + r][t + g4], x, kk[j]);
            qk[j] = mfma16(*(const f32x4 *)&Q[16 * wave + r][t + g4], x, qk[j]);
        }
    }
    const int group = c.Hv / c.Hk;
    for (int h = hk * group; h < (hk + 1) * group; ++h) {
        const int64_t at = (int64_t)slot * c.Hv + h;
        __syncthreads();  // the previous head's values have been read
        if (wave == 0) {
            const double x = running_sum(c.g + (int64_t)ch.tok * c.Hv + h, c.Hv, ch.n, lane);
            const double last = __shfl(x, 63, 64);
            const float be = lane < ch.n ? c.beta[((int64_t)ch.tok + lane) * c.Hv + h] : 0.0f;
            b[lane] = x;
            beta[lane] = be;
            float *v = c.vecs + at * NV;
            v[lane] = expf((float)x);
            v[CH + lane] = expf((float)(last - x));
            v[2 * CH + lane] = be;
        }
        __syncthreads();
        float z = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (j > wave) continue;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = 16 * wave + g4 + i, col = 16 * j + r;
                const float d = row >= col ? expf((float)(b[row] - b[col])) : 0.0f;
                c.P[at * TRI + tri(wave, j) + (g4 + i) * 16 + r] = row >= col ? c.scale * d * qk[j][i] : 0.0f;
                const float a = row > col ? beta[row] * d * kk[j][i] : 0.0f;
                At[tri(wave, j) + (g4 + i) * 16 + r] = a;
                z = __builtin_fmaf(a, 0.0f, z);
            }
        }
        take_out_rows(z, At, c.vecs + at * NV + 2 * CH, wave, r, g4);
        __syncthreads();
        f32x4 Tc[4];
        invert(At, Td, wave, r, g4, Tc);
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            if (wave + n >= 4) break;
#pragma unroll
            for (int i = 0; i < 4; ++i) c.T[at * TRI + tri(wave + n, wave) + (g4 + i) * 16 + r] = Tc[n][i];
        }
    }
}

// One chunk's left operands in LDS.
template <int DK>
struct Stage {
    float K[CH][DK + 4];
    float Q[CH][DK + 4];
    float T[TRI], P[TRI];
    float eb[CH], er[CH], beta[CH];
};

template <class DT, int DK>
__device__ __forceinline__ void stage_chunk(Stage<DK> &L, const Ctx &c, const Chunk &ch, int slot, int h) {
    using X = typename DT::X;
    const int hk = h / (c.Hv / c.Hk);
    const int64_t at = (int64_t)slot * c.Hv + h;
    stage_unit<DT, DK>(L.K, (const X *)c.k + ch.tok * c.ldk + (int64_t)hk * c.Dk, c.ldk, ch.n, c, nullptr);
    stage_unit<DT, DK>(L.Q, (const X *)c.q + ch.tok * c.ldq + (int64_t)hk * c.Dk, c.ldq, ch.n, c, nullptr);
    for (int i = threadIdx.x; i < TRI / 4; i += 256) {
        ((f32x4 *)L.T)[i] = ((const f32x4 *)(c.T + at * TRI))[i];
        ((f32x4 *)L.P)[i] = ((const f32x4 *)(c.P + at * TRI))[i];
    }
    if (threadIdx.x < NV) L.eb[threadIdx.x] = c.vecs[at * NV + threadIdx.x];
}

// Forward walk.  SAVE: keeps each chunk's state and U for the backward pass
// instead of making outputs.
template <class DT, int DK, bool SAVE>
__global__ void __launch_bounds__(256) k_scan(Ctx c, const float *state_in, float *state_out, typename DT::X *o,
                                              int64_t ldo, float *S0s, float *Us) {
    using X = typename DT::X;
    extern __shared__ float lds[];
    Stage<DK> &L = *(Stage<DK> *)lds;
    const int nb = (c.Dv + 63) / 64;
    const int vb = blockIdx.x % nb, h = blockIdx.x / nb % c.Hv, s = blockIdx.x / nb / c.Hv;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r = lane & 15, g4 = (lane >> 4) * 4;
    const int dv = vb * 64 + wave * 16 + r;
    const bool in = dv < c.Dv;
    const int a = c.seq.begin(s), b = c.seq.end(s);
    const int64_t st = ((int64_t)s * c.Hv + h) * c.Dk * c.Dv + dv;
    f32x4 S[DK / 16];
#pragma unroll
    for (int t = 0; t < DK / 16; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = 16 * t + g4 + i;
            S[t][i] = state_in && in && row < c.Dk ? state_in[st + (int64_t)row * c.Dv] : 0.0f;
        }
    int slot = first_slot(c.seq, s);
    for (int tok = a; tok < b; tok += CH, ++slot) {
        const Chunk ch{s, tok, b - tok < CH ? b - tok : CH};
        __syncthreads();
        stage_chunk<DT, DK>(L, c, ch, slot, h);
        f32x4 V[4];
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = 16 * m + g4 + i;
                V[m][i] = in && t < ch.n ? DT::widen(((const X *)c.v)[(ch.tok + t) * c.ldv + (int64_t)h * c.Dv + dv]) : 0.0f;
            }
        if (SAVE && dv < c.DvP) {
            float *d = S0s + ((int64_t)slot * c.Hv + h) * DK * c.DvP + dv;
#pragma unroll
            for (int t = 0; t < DK / 16; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) d[(int64_t)(16 * t + g4 + i) * c.DvP] = S[t][i];
        }
        __syncthreads();
        f32x4 R[4], Uc[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            f32x4 x = splat(0.0f);
#pragma unroll
            for (int t = 0; t < DK / 16; ++t) x = mfma16(*(const f32x4 *)&L.K[16 * m + r][16 * t + g4], S[t], x);
            R[m] = *(const f32x4 *)&L.beta[16 * m + g4] * (V[m] - *(const f32x4 *)&L.eb[16 * m + g4] * x);
        }
        // the column's first token that is no number
        const bool mend = !SAVE && any_no_number(R);
        const int first = mend ? take_out(R, g4) : CH;
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            f32x4 x = splat(0.0f);
#pragma unroll
            for (int j = 0; j <= m; ++j) x = mfma16(*(const f32x4 *)&L.T[tri(m, j) + r * 16 + g4], R[j], x);
            if (mend) put_from(x, 16 * m + g4, first, 0.0f);
            Uc[m] = x;
        }
        if (SAVE) {
            if (dv < c.DvP) {
                float *d = Us + ((int64_t)slot * c.Hv + h) * CH * c.DvP + dv;
#pragma unroll
                for (int m = 0; m < 4; ++m)
#pragma unroll
                    for (int i = 0; i < 4; ++i) d[(int64_t)(16 * m + g4 + i) * c.DvP] = Uc[m][i];
            }
        } else {
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                f32x4 x = splat(0.0f);
#pragma unroll
                for (int t = 0; t < DK / 16; ++t) x = mfma16(*(const f32x4 *)&L.Q[16 * m + r][16 * t + g4], S[t], x);
                x = x * *(const f32x4 *)&L.eb[16 * m + g4] * c.scale;
#pragma unroll
                for (int j = 0; j <= m; ++j) x = mfma16(*(const f32x4 *)&L.P[tri(m, j) + r * 16 + g4], Uc[j], x);
                if (mend) put_from(x, 16 * m + g4, first, __builtin_nanf(""));
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int t = 16 * m + g4 + i;
                    if (in && t < ch.n) o[(ch.tok + t) * ldo + (int64_t)h * c.Dv + dv] = rounded<DT>(x[i]);
                }
            }
        }
        const float el = L.eb[CH - 1];
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            Uc[m] *= *(const f32x4 *)&L.er[16 * m + g4];
            if (mend) put_from(Uc[m], 16 * m + g4, first, __builtin_nanf(""));
        }
#pragma unroll
        for (int t = 0; t < DK / 16; ++t) {
            f32x4 x = S[t] * el;
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                f32x4 k;
#pragma unroll
                for (int i = 0; i < 4; ++i) k[i] = L.K[16 * m + g4 + i][16 * t + r];
                x = mfma16(k, Uc[m], x);
            }
            S[t] = x;
        }
    }
    if (state_out && in) {
#pragma unroll
        for (int t = 0; t < DK / 16; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = 16 * t + g4 + i;
                if (row < c.Dk) state_out[st + (int64_t)row * c.Dv] = S[t][i];
            }
    }
}

// Backward walk: dV, every chunk's dR and dS (the gradient of the state behind
// it), and the gradient of the state in front of the sequence.
template <class DT, int DK>
__global__ void __launch_bounds__(256) k_rscan(Ctx c, const typename DT::X *d_o, int64_t lddo, const float *dstate_out,
                                               float *dstate_in, typename DT::X *dvo, int64_t lddv, float *dSs,
                                               float *dRs) {
    extern __shared__ float lds[];
    Stage<DK> &L = *(Stage<DK> *)lds;
    const int nb = (c.Dv + 63) / 64;
    const int vb = blockIdx.x % nb, h = blockIdx.x / nb % c.Hv, s = blockIdx.x / nb / c.Hv;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r = lane & 15, g4 = (lane >> 4) * 4;
    const int dv = vb * 64 + wave * 16 + r;
    const bool in = dv < c.Dv;
    const int a = c.seq.begin(s), b = c.seq.end(s);
    const int64_t st = ((int64_t)s * c.Hv + h) * c.Dk * c.Dv + dv;
    f32x4 S[DK / 16];
#pragma unroll
    for (int t = 0; t < DK / 16; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = 16 * t + g4 + i;
            S[t][i] = dstate_out && in && row < c.Dk ? dstate_out[st + (int64_t)row * c.Dv] : 0.0f;
        }
    const int nc = (b - a + CH - 1) / CH;
    for (int k = nc - 1; k >= 0; --k) {
        const int tok = a + k * CH, slot = first_slot(c.seq, s) + k;
        const Chunk ch{s, tok, b - tok < CH ? b - tok : CH};
        __syncthreads();
        stage_chunk<DT, DK>(L, c, ch, slot, h);
        f32x4 dO[4];
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = 16 * m + g4 + i;
                dO[m][i] = in && t < ch.n ? DT::widen(d_o[(ch.tok + t) * lddo + (int64_t)h * c.Dv + dv]) : 0.0f;
            }
        if (dv < c.DvP) {
            float *d = dSs + ((int64_t)slot * c.Hv + h) * DK * c.DvP + dv;
#pragma unroll
            for (int t = 0; t < DK / 16; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) d[(int64_t)(16 * t + g4 + i) * c.DvP] = S[t][i];
        }
        __syncthreads();
        f32x4 dU[4], dR[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            f32x4 x = splat(0.0f);
#pragma unroll
            for (int t = 0; t < DK / 16; ++t) x = mfma16(*(const f32x4 *)&L.K[16 * m + r][16 * t + g4], S[t], x);
            x *= *(const f32x4 *)&L.er[16 * m + g4];
#pragma unroll
            for (int j = m; j < 4; ++j) {
                f32x4 p;
#pragma unroll
                for (int i = 0; i < 4; ++i) p[i] = L.P[tri(j, m) + (g4 + i) * 16 + r];
                x = mfma16(p, dO[j], x);
            }
            dU[m] = x;
        }
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            f32x4 x = splat(0.0f);
#pragma unroll
            for (int j = m; j < 4; ++j) {
                f32x4 p;
#pragma unroll
                for (int i = 0; i < 4; ++i) p[i] = L.T[tri(j, m) + (g4 + i) * 16 + r];
                x = mfma16(p, dU[j], x);
            }
            dR[m] = x;
            const f32x4 y = x * *(const f32x4 *)&L.beta[16 * m + g4];
            float *d = dRs + ((int64_t)slot * c.Hv + h) * CH * c.DvP + dv;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = 16 * m + g4 + i;
                if (dv < c.DvP) d[(int64_t)t * c.DvP] = x[i];
                if (in && t < ch.n) dvo[(ch.tok + t) * lddv + (int64_t)h * c.Dv + dv] = rounded<DT>(y[i]);
            }
        }
        const float el = L.eb[CH - 1];
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const f32x4 e = *(const f32x4 *)&L.eb[16 * m + g4];
            dO[m] *= e * c.scale;
            dR[m] *= -e * *(const f32x4 *)&L.beta[16 * m + g4];
        }
#pragma unroll
        for (int t = 0; t < DK / 16; ++t) {
            f32x4 x = S[t] * el;
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                f32x4 q, k2;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    q[i] = L.Q[16 * m + g4 + i][16 * t + r];
                    k2[i] = L.K[16 * m + g4 + i][16 * t + r];
                }
                x = mfma16(q, dO[m], x);
                x = mfma16(k2, dR[m], x);
            }
            S[t] = x;
        }
    }
    if (dstate_in && in) {
#pragma unroll
        for (int t = 0; t < DK / 16; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = 16 * t + g4 + i;
                if (row < c.Dk) dstate_in[st + (int64_t)row * c.Dv] = S[t][i];
            }
    }
}

// A workgroup: one chunk and one key head, its value heads one after the other
// (their shares of dQ and dK add up in registers).  Wave w has tokens 16 w ..
// 16 w + 15.
template <class DT, int DK>
__global__ void __launch_bounds__(256) k_grad(Ctx c, GradArgs ga) {
    using X = typename DT::X;
    extern __shared__ float lds[];
    // while sums over S's columns run
    float (*Sb)[36] = (float (*)[36])lds;  // 32 columns of S0
    float (*Db)[36] = Sb + DK;             // ... of dS
    float (*Ub)[36] = Db + DK;             // ... of U
    // afterwards
    float (*K)[DK + 4] = (float (*)[DK + 4])lds;
    float (*Q)[DK + 4] = K + CH;
    float *Et = (float *)(Q + CH), *Mt = Et + TRI;
    __shared__ double b[CH];
    __shared__ float eb[NV], rk[CH], rq[CH], db[CH], dbe[CH], a2[CH], colP[4][CH], colA[4][CH], dots[4];
    float *er = eb + CH, *beta = eb + 2 * CH;
    const int slot = blockIdx.x / c.Hk, hk = blockIdx.x % c.Hk;
    const Chunk ch = chunk_of(c.seq, slot);
    if (ch.n == 0) return;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r = lane & 15, g4 = (lane >> 4) * 4;
    const int group = c.Hv / c.Hk;
    f32x4 dQ[DK / 16], dK[DK / 16];
#pragma unroll
    for (int t = 0; t < DK / 16; ++t) dQ[t] = dK[t] = splat(0.0f);
    for (int h = hk * group; h < (hk + 1) * group; ++h) {
        const int64_t at = (int64_t)slot * c.Hv + h;
        f32x4 X1[DK / 16], X2[DK / 16], X3[DK / 16], dP[4], dA[4];
#pragma unroll
        for (int t = 0; t < DK / 16; ++t) X1[t] = X2[t] = X3[t] = splat(0.0f);
#pragma unroll
        for (int j = 0; j < 4; ++j) dP[j] = dA[j] = splat(0.0f);
        float rv = 0.0f, sd = 0.0f;  // dR . V of row 16 w + r; <S0, dS>
        const int row = 16 * wave + r;
        for (int col = 0; col < c.DvP; col += 32) {
            __syncthreads();
            for (int i = threadIdx.x; i < DK * 8; i += 256) {
                const int x = i >> 3, y = (i & 7) * 4;
                const int64_t src = (at * DK + x) * c.DvP + col + y;
                const f32x4 s0 = *(const f32x4 *)(ga.S0s + src), ds = *(const f32x4 *)(ga.dSs + src);
                *(f32x4 *)&Sb[x][y] = s0;
                *(f32x4 *)&Db[x][y] = ds;
#pragma unroll
                for (int j = 0; j < 4; ++j) sd = __builtin_fmaf(s0[j], ds[j], sd);
            }
            for (int i = threadIdx.x; i < CH * 8; i += 256) {
                const int x = i >> 3, y = (i & 7) * 4;
                *(f32x4 *)&Ub[x][y] = *(const f32x4 *)(ga.Us + (at * CH + x) * c.DvP + col + y);
            }
            __syncthreads();
#pragma unroll
            for (int t = 0; t < 32; t += 16) {
                const int x = col + t + g4;
                const f32x4 u = *(const f32x4 *)&Ub[row][t + g4];
                const f32x4 dr = *(const f32x4 *)(ga.dRs + (at * CH + row) * c.DvP + x);
                f32x4 od = splat(0.0f);
                if (row < ch.n) {
                    od = load4<DT>((const X *)ga.d_o + (ch.tok + row) * ga.lddo + (int64_t)h * c.Dv + x, c.Dv - x, ga.vec_o);
                    const f32x4 vv = load4<DT>((const X *)c.v + (ch.tok + row) * c.ldv + (int64_t)h * c.Dv + x, c.Dv - x, ga.vec_v);
#pragma unroll
                    for (int j = 0; j < 4; ++j) rv = __builtin_fmaf(dr[j], vv[j], rv);
                }
#pragma unroll
                for (int n = 0; n < DK / 16; ++n) {
                    const f32x4 s0 = *(const f32x4 *)&Sb[16 * n + r][t + g4];
                    X1[n] = mfma16(od, s0, X1[n]);
                    X3[n] = mfma16(dr, s0, X3[n]);
                    X2[n] = mfma16(u, *(const f32x4 *)&Db[16 * n + r][t + g4], X2[n]);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (j > wave) continue;
                    const f32x4 uj = *(const f32x4 *)&Ub[16 * j + r][t + g4];
                    dP[j] = mfma16(od, uj, dP[j]);
                    dA[j] = mfma16(-dr, uj, dA[j]);
                }
            }
        }
        __syncthreads();
        stage_unit<DT, DK>(K, (const X *)c.k + ch.tok * c.ldk + (int64_t)hk * c.Dk, c.ldk, ch.n, c, rk);
        stage_unit<DT, DK>(Q, (const X *)c.q + ch.tok * c.ldq + (int64_t)hk * c.Dk, c.ldq, ch.n, c, rq);
        if (threadIdx.x < NV) eb[threadIdx.x] = c.vecs[at * NV + threadIdx.x];
        if (wave == 0) b[lane] = running_sum(c.g + (int64_t)ch.tok * c.Hv + h, c.Hv, ch.n, lane);
#pragma unroll
        for (int m = 1; m < 64; m <<= 1) sd += __shfl_xor(sd, m, 64);
        if (lane == 0) dots[wave] = sd;
        rv += __shfl_xor(rv, 16, 64);
        rv += __shfl_xor(rv, 32, 64);
        if (lane < 16) dbe[row] = rv;
        __syncthreads();
        // row sums: tokens 16 w + g4 + i
        const f32x4 ebr = *(const f32x4 *)&eb[16 * wave + g4], err = *(const f32x4 *)&er[16 * wave + g4];
        const f32x4 ber = *(const f32x4 *)&beta[16 * wave + g4];
        f32x4 s1 = splat(0.0f), s2 = splat(0.0f), s3 = splat(0.0f);
#pragma unroll
        for (int t = 0; t < DK / 16; ++t) {
            f32x4 kr, qr;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                kr[i] = K[16 * wave + g4 + i][16 * t + r];
                qr[i] = Q[16 * wave + g4 + i][16 * t + r];
            }
            s1 += qr * X1[t];
            s2 += kr * X2[t];
            s3 += kr * X3[t];
            dQ[t] += c.scale * ebr * X1[t];
            dK[t] += err * X2[t] - ebr * ber * X3[t];
        }
        s1 = sum16(s1) * ebr * c.scale;
        s2 = sum16(s2) * err;
        s3 = sum16(s3) * ebr;
        f32x4 rowP = splat(0.0f), rowA = splat(0.0f), rowB = splat(0.0f);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float cp = 0.0f, ca = 0.0f;
            if (j <= wave) {
                f32x4 kk = splat(0.0f);
                for (int t = 0; t < DK; t += 16)
                    kk = mfma16(*(const f32x4 *)&K[16 * wave + r][t + g4], *(const f32x4 *)&K[16 * j + r][t + g4], kk);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int x = 16 * wave + g4 + i, y = 16 * j + r;
                    const float d = x >= y ? expf((float)(b[x] - b[y])) : 0.0f;
                    const float p = x >= y ? dP[j][i] * c.P[at * TRI + tri(wave, j) + (g4 + i) * 16 + r] : 0.0f;
                    const float m = x > y ? dA[j][i] * d : 0.0f;
                    const float mk = x > y ? m * kk[i] : 0.0f;
                    Et[tri(wave, j) + (g4 + i) * 16 + r] = x >= y ? c.scale * dP[j][i] * d : 0.0f;
                    Mt[tri(wave, j) + (g4 + i) * 16 + r] = ber[i] * m;
                    rowP[i] += p;
                    rowB[i] += mk;
                    rowA[i] += ber[i] * mk;
                    cp += p;
                    ca += ber[i] * mk;
                }
            }
            cp += __shfl_xor(cp, 16, 64);
            cp += __shfl_xor(cp, 32, 64);
            ca += __shfl_xor(ca, 16, 64);
            ca += __shfl_xor(ca, 32, 64);
            if (lane < 16) {
                colP[wave][16 * j + r] = cp;
                colA[wave][16 * j + r] = ca;
            }
        }
        rowP = sum16(rowP);
        rowA = sum16(rowA);
        rowB = sum16(rowB);
        if (r == 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int x = 16 * wave + g4 + i;
                db[x] = s1[i] + rowP[i] + rowA[i] - ber[i] * s3[i] - s2[i];
                a2[x] = s2[i];
                dbe[x] += rowB[i] - s3[i];
            }
        }
        __syncthreads();
        if (wave == 0) {
            float x = db[lane];
#pragma unroll
            for (int w = 0; w < 4; ++w) x -= colP[w][lane] + colA[w][lane];
            double all = a2[lane];
#pragma unroll
            for (int m = 1; m < 64; m <<= 1) all += __shfl_xor(all, m, 64);
            double y = x;
            if (lane == 63) y += all + (double)eb[CH - 1] * ((dots[0] + dots[1]) + (dots[2] + dots[3]));
#pragma unroll
            for (int m = 1; m < 64; m <<= 1) {
                const double z = __shfl_down(y, m, 64);
                if (lane + m < 64) y += z;
            }
            if (lane < ch.n) {
                ga.dg[((int64_t)ch.tok + lane) * c.Hv + h] = (float)y;
                ga.dbeta[((int64_t)ch.tok + lane) * c.Hv + h] = dbe[lane];
            }
        }
        // E K, E^T Q, (M + M^T) K
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f32x4 e, m, et, mt;
            if (j <= wave) {
                e = *(const f32x4 *)&Et[tri(wave, j) + r * 16 + g4];
                m = *(const f32x4 *)&Mt[tri(wave, j) + r * 16 + g4];
            }
            if (j >= wave) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    et[i] = Et[tri(j, wave) + (g4 + i) * 16 + r];
                    mt[i] = Mt[tri(j, wave) + (g4 + i) * 16 + r];
                }
            }
            for (int t = 0; t < DK / 16; ++t) {
                f32x4 kr, qr;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    kr[i] = K[16 * j + g4 + i][16 * t + r];
                    qr[i] = Q[16 * j + g4 + i][16 * t + r];
                }
                f32x4 xq = dQ[t], xk = dK[t];
                if (j <= wave) {
                    xq = mfma16(e, kr, xq);
                    xk = mfma16(m, kr, xk);
                }
                if (j >= wave) {
                    xk = mfma16(et, qr, xk);
                    xk = mfma16(mt, kr, xk);
                }
                dQ[t] = xq;
                dK[t] = xk;
            }
        }
    }
    // from the unit vectors to q and k: d - u (u . d), over the length
    f32x4 uq = splat(0.0f), uk = splat(0.0f);
    if (c.normalize) {
#pragma unroll
        for (int t = 0; t < DK / 16; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uq[i] = __builtin_fmaf(dQ[t][i], Q[16 * wave + g4 + i][16 * t + r], uq[i]);
                uk[i] = __builtin_fmaf(dK[t][i], K[16 * wave + g4 + i][16 * t + r], uk[i]);
            }
        uq = sum16(uq);
        uk = sum16(uk);
    }
#pragma unroll
    for (int t = 0; t < DK / 16; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int x = 16 * wave + g4 + i, y = 16 * t + r;
            if (x >= ch.n || y >= c.Dk) continue;
            const float q = rq[x] * (dQ[t][i] - Q[x][y] * uq[i]), k = rk[x] * (dK[t][i] - K[x][y] * uk[i]);
            ((X *)ga.dq)[(ch.tok + x) * ga.lddq + (int64_t)hk * c.Dk + y] = rounded<DT>(q);
            ((X *)ga.dk)[(ch.tok + x) * ga.lddk + (int64_t)hk * c.Dk + y] = rounded<DT>(k);
        }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
int padded_keys(int Dk) { return (Dk + 63) / 64 * 64; }

struct Layout {
    size_t T, P, vecs, keys, heads, sums, S0s, Us, dSs, dRs, end;  // offsets in floats
    size_t key_bytes, head_bytes;
};
Layout layout(const dwconv_delta_plan &p, int seqs, int tokens, bool backward) {
    const size_t slots = (size_t)tokens / CH + seqs, n = slots * p.Hv;
    const size_t DvP = (p.Dv + 31) / 32 * 32, DK = padded_keys(p.Dk);
    const bool split = split_runs(p.dtype);
    Layout l{};
    size_t at = 0;
    auto take = [&](size_t f) {
        const size_t here = at;
        at += (f + 255) / 256 * 256;
        return here;
    };
    if (split) {
        l.key_bytes = (size_t)key_frags((int)DK, key_terms(p.dtype)) * (backward ? 4 : 3) * FRAG;
        l.head_bytes = (size_t)(backward ? HEAD_BWD : HEAD_FWD) * FRAG;
        l.keys = take(slots * p.Hk * l.key_bytes / 4);
        l.heads = take(n * l.head_bytes / 4);
    } else {
        l.T = take(n * TRI);
    }
    if (!split) {
        l.P = take(n * TRI);
        l.vecs = take(n * NV);
    }
    if (split && backward) l.sums = take(n * CH * 2);
    if (backward) {
        l.S0s = take(n * DK * DvP);
        l.Us = take(n * CH * DvP);
        l.dSs = take(n * DK * DvP);
        l.dRs = take(n * CH * DvP);
    }
    l.end = at;
    return l;
}

template <class X>
bool rows_of(int n, const void *p, int64_t ld, int d) {
    return ((uintptr_t)p & (n * sizeof(X) - 1)) == 0 && ld % n == 0 && d % n == 0;
}

template <class DT, int DK>
hipError_t run(const dwconv_delta_plan &p, const DeltaArgs &a, bool backward, hipStream_t st) {
    using X = typename DT::X;
    if (a.seqs == 0) return hipSuccess;
    const Layout l = layout(p, a.seqs, a.tokens, backward);
    float *ws = (float *)a.workspace;
    Ctx c{};
    c.seq = {a.offsets, a.seqs, a.tokens};
    c.Hk = p.Hk, c.Hv = p.Hv, c.Dk = p.Dk, c.Dv = p.Dv, c.DvP = (p.Dv + 31) / 32 * 32;
    c.scale = p.scale, c.eps = p.eps, c.normalize = p.normalize;
    c.vec4 = rows_of<X>(4, a.q, a.ldq, p.Dk) && rows_of<X>(4, a.k, a.ldk, p.Dk);
    c.vec8 = rows_of<X>(8, a.q, a.ldq, p.Dk) && rows_of<X>(8, a.k, a.ldk, p.Dk);
    c.q = a.q, c.k = a.k, c.v = a.v, c.ldq = a.ldq, c.ldk = a.ldk, c.ldv = a.ldv;
    c.g = a.g, c.beta = a.beta;
    c.T = ws + l.T, c.P = ws + l.P, c.vecs = ws + l.vecs;
    c.keys = (char *)(ws + l.keys), c.heads = (char *)(ws + l.heads), c.sums = (double *)(ws + l.sums);
    c.key_bytes = (int64_t)l.key_bytes, c.head_bytes = (int64_t)l.head_bytes;
    const uint64_t chunks = ((uint64_t)(a.tokens / CH) + a.seqs) * p.Hk, walks = (uint64_t)a.seqs * p.Hv * ((p.Dv + 63) / 64);
    // a grid holds fewer than 2^32 lanes; the 16-bit walks' grid is rounded up (eight
    // times at most), so it is looked at as it will be, before anything is launched
    if (chunks >= (1u << 23) || walks >= (1u << 21)) return hipErrorInvalidConfiguration;
    c.slots = a.tokens / CH + a.seqs;
    if (split_runs(p.dtype) && split_blocks(c, backward) >= (1u << 24)) return hipErrorInvalidConfiguration;
    const int vec = std::is_same<DT, F32>::value ? 4 : 8;
    const GradArgs ga{ws + l.S0s, ws + l.Us, ws + l.dSs, ws + l.dRs, a.d_o, a.lddo, a.dq, a.dk, a.lddq, a.lddk, a.dg,
                      a.dbeta, rows_of<X>(vec, a.d_o, a.lddo, p.Dv), rows_of<X>(vec, a.v, a.ldv, p.Dv)};
    hipError_t e = hipSuccess;
    auto ok = [&](hipError_t x) { return (e = x) == hipSuccess; };
    if constexpr (!std::is_same<DT, F32>::value) {
        if (a.tokens > 0 && !ok(split_prepare(p.dtype, DK, c, backward, st))) return e;
        if (!backward) return split_scan(p.dtype, DK, c, a.state_in, a.state_out, a.o, a.ldo, nullptr, nullptr, st);
        if (a.tokens > 0 &&
            !ok(split_scan(p.dtype, DK, c, a.state_in, nullptr, nullptr, 0, ws + l.S0s, ws + l.Us, st)))
            return e;
        if (!ok(split_rscan(p.dtype, DK, c, a.d_o, a.lddo, a.dstate_out, a.dstate_in, a.dv, a.lddv, ws + l.dSs,
                            ws + l.dRs, st)))
            return e;
        return a.tokens > 0 ? split_grad(p.dtype, DK, c, ga, st) : hipSuccess;
    } else {
        const size_t keys = 2 * sizeof(float) * CH * (DK + 4);
        auto lds = [&](const void *f, size_t bytes) {
            return ok(hipFuncSetAttribute(f, hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes));
        };
        if (a.tokens > 0) {
            const size_t n = keys + (TRI + 4 * 256) * sizeof(float);
            if (!lds((const void *)k_prepare<DT, DK>, n)) return e;
            k_prepare<DT, DK><<<(uint32_t)chunks, 256, n, st>>>(c);
        }
        if (!backward) {
            if (!lds((const void *)k_scan<DT, DK, false>, sizeof(Stage<DK>))) return e;
            k_scan<DT, DK, false><<<(uint32_t)walks, 256, sizeof(Stage<DK>), st>>>(c, a.state_in, a.state_out,
                                                                                   (X *)a.o, a.ldo, nullptr, nullptr);
            return hipGetLastError();
        }
        if (a.tokens > 0) {
            if (!lds((const void *)k_scan<DT, DK, true>, sizeof(Stage<DK>))) return e;
            k_scan<DT, DK, true><<<(uint32_t)walks, 256, sizeof(Stage<DK>), st>>>(
                c, a.state_in, nullptr, (X *)nullptr, 0, ws + l.S0s, ws + l.Us);
        }
        if (!lds((const void *)k_rscan<DT, DK>, sizeof(Stage<DK>))) return e;
        k_rscan<DT, DK><<<(uint32_t)walks, 256, sizeof(Stage<DK>), st>>>(c, (const X *)a.d_o, a.lddo, a.dstate_out,
                                                                         a.dstate_in, (X *)a.dv, a.lddv, ws + l.dSs,
                                                                         ws + l.dRs);
        if (a.tokens > 0) {
            const size_t blocks = sizeof(float) * 36 * (2 * DK + CH), tiles = keys + 2 * TRI * sizeof(float);
            const size_t n = blocks > tiles ? blocks : tiles;
            if (!lds((const void *)k_grad<DT, DK>, n)) return e;
            k_grad<DT, DK><<<(uint32_t)chunks, 256, n, st>>>(c, ga);
        }
        return hipGetLastError();
    }
}

template <class DT>
hipError_t pick_keys(const dwconv_delta_plan &p, const DeltaArgs &a, bool backward, hipStream_t st) {
    switch (padded_keys(p.Dk)) {
        case 64: return run<DT, 64>(p, a, backward, st);
        case 128: return run<DT, 128>(p, a, backward, st);
        case 192: return run<DT, 192>(p, a, backward, st);
        default: return run<DT, 256>(p, a, backward, st);
    }
}

hipError_t pick(const dwconv_delta_plan &p, const DeltaArgs &a, bool backward, hipStream_t st) {
    switch (p.dtype) {
        case DWCONV_F32: return pick_keys<F32>(p, a, backward, st);
        case DWCONV_F16: return pick_keys<F16>(p, a, backward, st);
        default: return pick_keys<BF16>(p, a, backward, st);
    }
}

}  // namespace

hipError_t delta_fwd(const dwconv_delta_plan &p, const DeltaArgs &a, hipStream_t st) { return pick(p, a, false, st); }
hipError_t delta_bwd(const dwconv_delta_plan &p, const DeltaArgs &a, hipStream_t st) { return pick(p, a, true, st); }

size_t delta_bytes(const dwconv_delta_plan &p, int seqs, int tokens, bool backward) {
    return layout(p, seqs, tokens, backward).end * sizeof(float);
}

}  // namespace dw
