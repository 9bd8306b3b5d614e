// delta_common.h -- chunks, arguments and small device functions shared by the
// gated delta rule's kernels.
#pragma once

#include "seq_common.h"
#include "seq_plan.h"

namespace dw {
namespace delta {

constexpr int CH = 64;             // tokens a chunk
constexpr int TRI = 10 * 256;      // floats of a lower triangle of 4x4 tiles of 16x16
constexpr int NV = 3 * CH;         // per-chunk vectors: e^b, e^{b_last - b}, beta

using f32x4 = __attribute__((ext_vector_type(4))) float;

__device__ __forceinline__ f32x4 mfma4(float a, float b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}
// c += A B over 16 terms: a[i] is the left operand's term 4 (l / 16) + i of row
// l % 16, b[i] the right operand's term 4 (l / 16) + i of column l % 16
__device__ __forceinline__ f32x4 mfma16(f32x4 a, f32x4 b, f32x4 c) {
#pragma unroll
    for (int i = 0; i < 4; ++i) c = mfma4(a[i], b[i], c);
    return c;
}
__device__ __forceinline__ f32x4 splat(float v) { return f32x4{v, v, v, v}; }
__host__ __device__ constexpr int tri(int i, int j) { return (i * (i + 1) / 2 + j) * 256; }

// Sizes and inputs; T, P, vectors and norms of every chunk in the workspace.
struct Ctx {
    Packed seq;
    int Hk, Hv, Dk, Dv, DvP;  // DvP: Dv rounded up to 32
    int slots;
    float scale, eps;
    int normalize, vec4;      // vec4: rows of q and k load 4 elements at once
    const void *q, *k, *v;
    int64_t ldq, ldk, ldv;
    const float *g, *beta;
    float *T, *P;             // slots x Hv x TRI
    float *vecs;              // slots x Hv x NV
    // operands of the 16-bit products, in fragments: a slot's key head (Q, K,
    // K^T and, backward, Q^T) and value head
    char *keys, *heads;
    double *sums;             // slots x Hv x CH: b, backward
    int64_t key_bytes, head_bytes;
    int vec8;                 // rows of q and k load 8 elements at once
};

// A chunk's place.  Sequence s begins at slot begin / 64 + s: a sequence of L
// tokens needs ceil(L / 64) slots, and no two chunks share one.
struct Chunk {
    int s, tok, n;  // sequence, first token, tokens (0: an unused slot)
};
__device__ __forceinline__ int first_slot(const Packed &p, int s) { return p.begin(s) / CH + s; }
__device__ __forceinline__ Chunk chunk_of(const Packed &p, int slot) {
    int lo = 0, hi = p.seqs;  // first_slot(lo) <= slot
    while (hi - lo > 1) {
        const int m = lo + ((hi - lo) >> 1);
        if (first_slot(p, m) <= slot) lo = m; else hi = m;
    }
    const int c = slot - first_slot(p, lo), a = p.begin(lo), b = p.end(lo);
    if (c < 0 || (int64_t)a + (int64_t)c * CH >= b) return {lo, 0, 0};
    const int tok = a + c * CH;
    return {lo, tok, b - tok < CH ? b - tok : CH};
}

template <class DT>
__device__ __forceinline__ f32x4 load4(const typename DT::X *p, int valid, bool vec4) {
    f32x4 r = splat(0.0f);
    if (valid >= 4 && vec4) {
        float t[4];
        load_f32<DT, 4>(t, p);
        r = f32x4{t[0], t[1], t[2], t[3]};
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < valid) r[i] = DT::widen(p[i]);
    }
    return r;
}

// Rows [tok, tok + n) of q or k into LDS as unit vectors (zeros behind), four
// threads a row; rnorm, where given, gets 1 / |row|.
template <class DT, int DK>
__device__ __forceinline__ void stage_unit(float (*dst)[DK + 4], const typename DT::X *src, int64_t ld, int n,
                                           const Ctx &c, float *rnorm) {
    const int row = threadIdx.x >> 2, part = threadIdx.x & 3;
    f32x4 v[DK / 16];
    float sq = 0.0f;
#pragma unroll
    for (int i = 0; i < DK / 16; ++i) {
        const int col = i * 16 + part * 4;
        v[i] = row < n ? load4<DT>(src + (int64_t)row * ld + col, c.Dk - col, c.vec4) : splat(0.0f);
#pragma unroll
        for (int j = 0; j < 4; ++j) sq = __builtin_fmaf(v[i][j], v[i][j], sq);
    }
    sq += __shfl_xor(sq, 1, 64);
    sq += __shfl_xor(sq, 2, 64);
    const float r = c.normalize && row < n ? 1.0f / sqrtf(sq + c.eps) : 1.0f;
    if (rnorm && part == 0) rnorm[row] = r;
#pragma unroll
    for (int i = 0; i < DK / 16; ++i) *(f32x4 *)&dst[row][i * 16 + part * 4] = v[i] * r;
}

// The running sum of g over the chunk's tokens, lane i: token i (one wavefront).
__device__ __forceinline__ double running_sum(const float *g, int Hv, int n, int lane) {
    float x = lane < n ? g[(int64_t)lane * Hv] : 0.0f;
    if (x < -1000.0f) x = -1000.0f;
    double b = x;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
        const double o = __shfl_up(b, m, 64);
        if (lane >= m) b += o;
    }
    return b;
}

// NaN or infinite: x * 0 is not 0.
__device__ __forceinline__ bool no_number(float x) { return !(x * 0.0f == 0.0f); }

// Rows of A and R that hold NaN or infinity.  A matrix product multiplies them
// with the zeros above the diagonal of T and P as well, which would carry them to
// the tokens before; the definition is causal.  So the forward walks take such
// values out of the operands and make the results of their own and all later
// tokens of the column NaN instead (the state behind the chunk becomes NaN by its
// own product).  Looking for them takes 2 to 5 % of a walk (8192 tokens of 32
// heads, bf16, five sequences: 206 and 197 us).
//
// take_out_rows: z has 0 times the sum of this lane's elements of A, rows 16 w +
// g4 + i, which the lane has written to At.  Rows that hold NaN or infinity
// become zeros, and beta of their tokens NaN, which makes R NaN in all columns.
__device__ __forceinline__ void take_out_rows(float z, float *At, float *beta, int wave, int r, int g4) {
    if (!__any(z != 0.0f)) return;
#pragma unroll 1
    for (int i = 0; i < 4; ++i) {
        float s = 0.0f;
        for (int j = 0; j <= wave; ++j) s = __builtin_fmaf(At[tri(wave, j) + (g4 + i) * 16 + r], 0.0f, s);
        if (sum_row16(s) == 0.0f) continue;
        for (int j = 0; j <= wave; ++j) At[tri(wave, j) + (g4 + i) * 16 + r] = 0.0f;
        if (r == 0) beta[16 * wave + g4 + i] = __builtin_nanf("");
    }
}
// First token of each column among N tiles of a wavefront's R (tile n: tokens
// row + 16 n ..), CH: none; the values are replaced by zeros.
template <int N>
__device__ __forceinline__ int take_out(f32x4 (&x)[N], int row) {
    int f = CH;
#pragma unroll
    for (int n = N - 1; n >= 0; --n)
#pragma unroll
        for (int i = 3; i >= 0; --i)
            if (no_number(x[n][i])) f = row + 16 * n + i, x[n][i] = 0.0f;
    f = min(f, __shfl_xor(f, 16, 64));
    return min(f, __shfl_xor(f, 32, 64));
}
template <int N>
__device__ __forceinline__ bool any_no_number(const f32x4 (&x)[N]) {
    float z = 0.0f;
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) z = __builtin_fmaf(x[n][i], 0.0f, z);
    return __any(z != 0.0f);
}
// tokens row + i from `first` on
__device__ __forceinline__ void put_from(f32x4 &x, int row, int first, float value) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (row + i >= first) x[i] = value;
}

// Column `wave` of T = (1 + A)^-1, tiles wave .. 3, from A's lower tiles in LDS
// (four wavefronts; Td: room for the diagonal tiles' inverses).
__device__ __forceinline__ void invert(const float *At, float *Td, int wave, int r, int g4, f32x4 (&Tc)[4]) {
    // wave w inverts diagonal tile w: a lane solves one column downwards, two
    // rows of the tile read at a time (and no more: registers)
    const float *a = At + tri(wave, wave);
    float x[16];
    x[0] = r == 0 ? 1.0f : 0.0f;
    x[1] = __builtin_fmaf(-a[16], x[0], r == 1 ? 1.0f : 0.0f);
#pragma unroll
    for (int b = 2; b < 16; b += 2) {
        f32x4 v[2][4];
        asm volatile("" ::: "memory");
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j <= b / 4; ++j) v[i][j] = *(const f32x4 *)(a + (b + i) * 16 + 4 * j);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float s = b + i == r ? 1.0f : 0.0f;
#pragma unroll
            for (int j = 0; j < b + i; ++j) s = __builtin_fmaf(-v[i][j / 4][j % 4], x[j], s);
            x[b + i] = s;
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        Tc[0][i] = g4 == 0 ? x[i] : g4 == 4 ? x[4 + i] : g4 == 8 ? x[8 + i] : x[12 + i];
        Td[wave * 256 + (g4 + i) * 16 + r] = Tc[0][i];
    }
    __syncthreads();
    // tiles below it: T_ij = -T_ii sum_m A_im T_mj; n counts tiles below the diagonal
#pragma unroll
    for (int n = 1; n < 4; ++n) {
        const int i = wave + n;
        if (i >= 4) break;
        f32x4 s = splat(0.0f);
#pragma unroll
        for (int m = 0; m < n; ++m) s = mfma16(*(const f32x4 *)&At[tri(i, wave + m) + r * 16 + g4], Tc[m], s);
        Tc[n] = mfma16(-*(const f32x4 *)&Td[i * 256 + r * 16 + g4], s, splat(0.0f));
    }
}

// ---------------------------------------------------------------------------
// Operands of the 16-bit matrix products (k_delta_split.hip).  A fragment is a
// left operand of v_mfma_f32_16x16x32: lane l has row l % 16 and eight terms,
// 16 bytes, a fragment 1 KB.  Its terms run in the order in which two result
// tiles one above the other are right operand: slot j of lane group g = l / 16
// is term 4 g + j (j < 4) or 16 + 4 g + j - 4.
// ---------------------------------------------------------------------------
constexpr int FRAG = 1024;
constexpr int NBLK = 6;         // blocks of 16 x 32 that a 64 x 64 triangle touches
constexpr int TRI_TERMS = 3;    // of T and P
constexpr int AT_P = 0, AT_T = AT_P + NBLK * TRI_TERMS, AT_VEC = AT_T + NBLK * TRI_TERMS, VEC_FRAGS = 2,
              HEAD_FWD = AT_VEC + VEC_FRAGS, AT_TT = HEAD_FWD, AT_PT = AT_TT + NBLK * TRI_TERMS,
              HEAD_BWD = AT_PT + NBLK * TRI_TERMS;
// vectors of a chunk, 64 floats each: e^b / |k|, e^{b_last - b} / |k|, beta,
// scale e^b / |q|, e^b and, backward, e^{b_last - b}, 1 / |k|, 1 / |q|
enum { V_EK, V_RK, V_BETA, V_EQ, V_EB, V_ER, V_NK, V_NQ };

__host__ __device__ constexpr int key_frags(int DK, int terms) { return DK / 8 * terms; }  // one matrix
// bf16 values are one term, fp16 values two bf16 terms
__host__ __device__ constexpr int key_terms(int dtype) { return dtype == DWCONV_BF16 ? 1 : 2; }

inline bool split_runs(int dtype) { return dtype != DWCONV_F32; }

// What the gradients of q, k, g and beta need: each chunk's states and U, dS, dR.
struct GradArgs {
    const float *S0s, *Us, *dSs, *dRs;
    const void *d_o;
    int64_t lddo;
    void *dq, *dk;
    int64_t lddq, lddk;
    float *dg, *dbeta;
    int vec_o, vec_v;  // rows of d_o and v load 4 (fp32) or 8 elements at once
};

// sum over the 16 lanes that share rows
__device__ __forceinline__ f32x4 sum16(f32x4 v) {
    return f32x4{sum_row16(v[0]), sum_row16(v[1]), sum_row16(v[2]), sum_row16(v[3])};
}

// launchers (k_delta_split.hip, k_delta_grad.hip)
hipError_t split_grad(int dtype, int DK, const Ctx &c, const GradArgs &ga, hipStream_t st);
uint64_t split_blocks(const Ctx &c, bool backward);  // workgroups of the walks
hipError_t split_prepare(int dtype, int DK, const Ctx &c, bool backward, hipStream_t st);
hipError_t split_scan(int dtype, int DK, const Ctx &c, const float *state_in, float *state_out, void *o, int64_t ldo,
                      float *S0s, float *Us, hipStream_t st);
hipError_t split_rscan(int dtype, int DK, const Ctx &c, const void *d_o, int64_t lddo, const float *dstate_out,
                       float *dstate_in, void *dv, int64_t lddv, float *dSs, float *dRs, hipStream_t st);

}  // namespace delta
}  // namespace dw
