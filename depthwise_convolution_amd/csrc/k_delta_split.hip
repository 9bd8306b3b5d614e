// k_delta_split.hip -- the gated delta rule's walks on the 16-bit matrix cores,
// for bf16 and fp16 data (the algebra is in k_delta.hip).
//
// A 16-bit product of 32 terms takes half the time of an fp32 product of 4,
// sixteen times the rate, but state and intermediates are fp32 values.  They
// are split into bf16 terms that add up to them (x = x0 + x1 + x2, each the
// rounding of what the ones before leave: 24 bits), q and k stay as they came:
// bf16 is one term, fp16 exactly two.  Lengths and decays are factored out of
// q and k as vectors over tokens.  Products of terms below 2^-24 of the whole
// are left out: three products for a bf16 operand times a state (one term
// times three), six for two fp32 ones.  What only makes o (its own rounding is
// 2^-9 or 2^-12) takes two terms: 2^-18.
//
// k_prepare lays all left operands out as fragments (delta_common.h) in the
// workspace, once for all wavefronts that use them, so that a walk copies them
// to LDS in a line, through registers that are loaded a chunk ahead, and reads
// them without bank conflicts.
#include <type_traits>

#include "delta_common.h"

namespace dw {
namespace {

using namespace delta;

using bf16x8 = __attribute__((ext_vector_type(8))) __bf16;
using bf16x4 = __attribute__((ext_vector_type(4))) __bf16;
using f16x8 = __attribute__((ext_vector_type(8))) _Float16;
using f32x8 = __attribute__((ext_vector_type(8))) float;
using u32x4 = __attribute__((ext_vector_type(4))) uint32_t;

__device__ __forceinline__ f32x4 mfma32(bf16x8 a, bf16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// x = t[0] + t[1] + ... : each the nearest bf16 of what is left
template <int N>
__device__ __forceinline__ void split(f32x4 a, f32x4 b, bf16x8 (&t)[N]) {
    f32x8 x = __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
#pragma unroll
    for (int n = 0; n < N; ++n) {
        t[n] = __builtin_convertvector(x, bf16x8);
        if (n + 1 < N) x -= __builtin_convertvector(t[n], f32x8);
    }
}

template <class DT>
struct Raw;
template <>
struct Raw<BF16> {
    static constexpr int TERMS = 1;
    using V8 = bf16x8;
    static __device__ __forceinline__ f32x4 mfma(V8 a, V8 b, f32x4 c) { return mfma32(a, b, c); }
    static __device__ __forceinline__ void terms(V8 x, bf16x8 (&t)[1]) { t[0] = x; }
};
template <>
struct Raw<F16> {
    static constexpr int TERMS = 2;
    using V8 = f16x8;
    static __device__ __forceinline__ f32x4 mfma(V8 a, V8 b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    }
    // 11 bits: the nearest bf16 leaves at most 3, exactly
    static __device__ __forceinline__ void terms(V8 x, bf16x8 (&t)[2]) {
        const f32x8 f = __builtin_convertvector(x, f32x8);
        t[0] = __builtin_convertvector(f, bf16x8);
        t[1] = __builtin_convertvector(f - __builtin_convertvector(t[0], f32x8), bf16x8);
    }
};

// Products of NA terms times NB terms down to order `last` (term i times term j
// has order i + j)
template <int NA, int NB>
__device__ __forceinline__ f32x4 mac(const bf16x8 (&a)[NA], const bf16x8 (&b)[NB], int last, f32x4 c) {
#pragma unroll
    for (int o = 0; o < NA + NB - 1; ++o) {
        if (o > last) break;
#pragma unroll
        for (int i = 0; i < NA; ++i)
            if (o - i >= 0 && o - i < NB) c = mfma32(a[i], b[o - i], c);
    }
    return c;
}

// place of block (m, kb) of a lower triangle's six (kb <= m / 2), and of an
// upper one's (kb >= m / 2)
__host__ __device__ constexpr int lower_block(int m, int kb) { return m < 2 ? m : 2 * (m - 1) + kb; }
__host__ __device__ constexpr int upper_block(int m, int kb) { return m < 2 ? 2 * m + kb : 2 + m; }

// One chunk and key head: lengths, the triangles of its value heads, and all
// left operands as fragments.
template <class DT, int DK, bool BACK>
__global__ void __launch_bounds__(256) k_prepare(Ctx c) {
    using X = typename DT::X;
    using R = Raw<DT>;
    using V8 = typename R::V8;
    constexpr int NA = R::TERMS, PITCH = DK + 8;
    extern __shared__ char lds_raw[];
    X(*K)[PITCH] = (X(*)[PITCH])lds_raw;
    X(*Q)[PITCH] = K + CH;
    float *At = (float *)(Q + CH), *Pl = At + TRI, *Tl = Pl + TRI, *Td = Tl + TRI;
    __shared__ double b[CH];
    __shared__ float beta[CH], rk[CH], rq[CH];
    const int slot = blockIdx.x / c.Hk, hk = blockIdx.x % c.Hk;
    const Chunk ch = chunk_of(c.seq, slot);
    if (ch.n == 0) return;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r = lane & 15, g4 = (lane >> 4) * 4;
    {  // rows of q and k, four threads a row; zeros behind
        const int row = threadIdx.x >> 2, part = threadIdx.x & 3;
        const X *pk = (const X *)c.k + (ch.tok + row) * c.ldk + (int64_t)hk * c.Dk;
        const X *pq = (const X *)c.q + (ch.tok + row) * c.ldq + (int64_t)hk * c.Dk;
        const bool live = row < ch.n;
#pragma unroll
        for (int i = 0; i < DK / 32; ++i) {
            const int col = i * 32 + part * 8;
            Vec<X, 8> a, d;
            if (live && c.vec8 && col < c.Dk) {
                a = *(const Vec<X, 8> *)(pk + col);
                d = *(const Vec<X, 8> *)(pq + col);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const bool in = live && col + j < c.Dk;
                    a.v[j] = in ? pk[col + j] : (X)0;
                    d.v[j] = in ? pq[col + j] : (X)0;
                }
            }
            *(Vec<X, 8> *)&K[row][col] = a;
            *(Vec<X, 8> *)&Q[row][col] = d;
        }
    }
    __syncthreads();
    // wave w: tiles (w, j), j <= w, of K K^T and Q K^T, and the squares
    f32x4 kk[4], qk[4], qq = splat(0.0f);
#pragma unroll
    for (int j = 0; j < 4; ++j) kk[j] = qk[j] = splat(0.0f);
#pragma unroll
    for (int t = 0; t < DK; t += 32) {
        const V8 kw = *(const V8 *)&K[16 * wave + r][t + 2 * g4], qw = *(const V8 *)&Q[16 * wave + r][t + 2 * g4];
        qq = R::mfma(qw, qw, qq);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (j > wave) continue;
            const V8 x = *(const V8 *)&K[16 * j + r][t + 2 * g4];
            kk[j] = R::mfma(kw, x, kk[j]);
            qk[j] = R::mfma(qw, x, qk[j]);
        }
    }
    if (r >= g4 && r < g4 + 4) {  // the diagonal: row g4 + i is column r
        float sk = 0.0f, sq = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (j == wave && g4 + i == r) sk = kk[j][i], sq = qq[i];
        const int row = 16 * wave + r;
        const bool norm = c.normalize && row < ch.n;
        rk[row] = norm ? 1.0f / sqrtf(sk + c.eps) : 1.0f;
        rq[row] = norm ? 1.0f / sqrtf(sq + c.eps) : 1.0f;
    }
    // fragments of Q, K, K^T and Q^T
    {
        constexpr int NF = DK / 8;
        char *base = c.keys + ((int64_t)slot * c.Hk + hk) * c.key_bytes;
        for (int f = wave; f < (BACK ? 4 : 3) * NF; f += 4) {
            const int mat = f / NF, i = f % NF;
            V8 x;
            if (mat < 2) {  // rows 16 m, terms 32 kb
                const X(*S)[PITCH] = mat == 0 ? Q : K;
                const int m = i / (DK / 32), kb = i % (DK / 32);
                const X *p = &S[16 * m + r][32 * kb + g4];
                Vec<X, 8> v;
                *(Vec<X, 4> *)&v.v[0] = *(const Vec<X, 4> *)p;
                *(Vec<X, 4> *)&v.v[4] = *(const Vec<X, 4> *)(p + 16);
                x = __builtin_bit_cast(V8, v);
            } else {  // channel rows 16 t, tokens 32 kb
                const X(*S)[PITCH] = mat == 2 ? K : Q;
                const int t = i / 2, kb = i % 2;
                Vec<X, 8> v;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    v.v[j] = S[32 * kb + g4 + j][16 * t + r];
                    v.v[4 + j] = S[32 * kb + 16 + g4 + j][16 * t + r];
                }
                x = __builtin_bit_cast(V8, v);
            }
            bf16x8 terms[NA];
            R::terms(x, terms);
#pragma unroll
            for (int n = 0; n < NA; ++n) *(bf16x8 *)(base + (int64_t)(f * NA + n) * FRAG + lane * 16) = terms[n];
        }
    }
    const int group = c.Hv / c.Hk;
    for (int h = hk * group; h < (hk + 1) * group; ++h) {
        const int64_t at = (int64_t)slot * c.Hv + h;
        char *base = c.heads + at * c.head_bytes;
        __syncthreads();  // the previous head's values have been read
        if (wave == 0) {
            const double x = running_sum(c.g + (int64_t)ch.tok * c.Hv + h, c.Hv, ch.n, lane);
            const double last = __shfl(x, 63, 64);
            const float be = lane < ch.n ? c.beta[((int64_t)ch.tok + lane) * c.Hv + h] : 0.0f;
            const float eb = expf((float)x), er = expf((float)(last - x));
            b[lane] = x;
            beta[lane] = be;
            float *v = (float *)(base + AT_VEC * FRAG);
            v[V_EK * CH + lane] = eb * rk[lane];
            v[V_RK * CH + lane] = er * rk[lane];
            v[V_BETA * CH + lane] = be;
            v[V_EQ * CH + lane] = c.scale * eb * rq[lane];
            v[V_EB * CH + lane] = eb;
            if (BACK) {
                float *u = c.vecs + at * NV;
                u[lane] = eb;
                u[CH + lane] = er;
                u[2 * CH + lane] = be;
            }
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (j > wave) continue;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = 16 * wave + g4 + i, col = 16 * j + r;
                const float d = row >= col ? expf((float)(b[row] - b[col])) : 0.0f;
                const float p = row >= col ? c.scale * d * (rq[row] * rk[col] * qk[j][i]) : 0.0f;
                const int e = tri(wave, j) + (g4 + i) * 16 + r;
                At[e] = row > col ? beta[row] * d * (rk[row] * rk[col] * kk[j][i]) : 0.0f;
                Pl[e] = p;
                if (BACK) c.P[at * TRI + e] = p;
            }
        }
        __syncthreads();
        f32x4 Tc[4];
        invert(At, Td, wave, r, g4, Tc);
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            if (wave + n >= 4) break;
#pragma unroll
            for (int i = 0; i < 4; ++i) Tl[tri(wave + n, wave) + (g4 + i) * 16 + r] = Tc[n][i];
        }
        __syncthreads();
        for (int f = wave; f < (BACK ? 4 : 2) * NBLK; f += 4) {
            const int what = f / NBLK, blk = f % NBLK;  // P, T, T^T, P^T
            const float *S = what == 0 || what == 3 ? Pl : Tl;
            f32x4 x[2];
            if (what < 2) {
                const int m = blk < 2 ? blk : blk / 2 + 1, kb = blk < 2 ? 0 : blk % 2;
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    x[j] = 2 * kb + j <= m ? *(const f32x4 *)&S[tri(m, 2 * kb + j) + r * 16 + g4] : splat(0.0f);
            } else {
                const int m = blk < 4 ? blk / 2 : blk - 2, kb = blk < 4 ? blk % 2 : 1;
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        x[j][i] = 2 * kb + j >= m ? S[tri(2 * kb + j, m) + (g4 + i) * 16 + r] : 0.0f;
            }
            bf16x8 t[T_TERMS];
            split(x[0], x[1], t);
            const int first = what == 0 ? AT_P : what == 1 ? AT_T : what == 2 ? AT_TT : AT_PT;
            const int terms = what == 0 ? P_TERMS : T_TERMS;
#pragma unroll
            for (int n = 0; n < T_TERMS; ++n)
                if (n < terms) *(bf16x8 *)(base + (int64_t)(first + blk * terms + n) * FRAG + lane * 16) = t[n];
        }
    }
}

// A walk's operands on their way from the workspace to LDS: the first N1
// fragments from the key head's part, the rest from the value head's; every
// wavefront moves every fourth.
template <int N1, int N2>
struct Feed {
    static constexpr int N = N1 + N2, PER = (N + 3) / 4;
    u32x4 v[PER];
    __device__ __forceinline__ void load(const char *a, const char *b, int wave, int lane) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int f = i * 4 + wave;
            if (f >= N) break;
            v[i] = *(const u32x4 *)((f < N1 ? a + f * FRAG : b + (f - N1) * FRAG) + lane * 16);
        }
    }
    __device__ __forceinline__ void store(char *lds, int wave, int lane) const {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int f = i * 4 + wave;
            if (f >= N) break;
            *(u32x4 *)(lds + f * FRAG + lane * 16) = v[i];
        }
    }
};

template <int N>
__device__ __forceinline__ void frag(bf16x8 (&t)[N], const char *lds, int first, int lane) {
#pragma unroll
    for (int n = 0; n < N; ++n) t[n] = *(const bf16x8 *)(lds + (first + n) * FRAG + lane * 16);
}

// Forward walk (as k_scan in k_delta.hip).
template <class DT, int DK, bool SAVE>
__global__ void __launch_bounds__(256) k_scan(Ctx c, const float *state_in, float *state_out, typename DT::X *o,
                                              int64_t ldo, float *S0s, float *Us) {
    using X = typename DT::X;
    constexpr int NA = Raw<DT>::TERMS, NK = DK / 32, NF = DK / 8 * NA;
    // LDS: [Q] K K^T | [P] T vectors
    constexpr int ATK = SAVE ? 0 : NF, ATKT = ATK + NF, N1 = ATKT + NF;
    constexpr int ATP = N1, ATT = SAVE ? N1 : N1 + NBLK * P_TERMS, ATV = ATT + NBLK * T_TERMS, N2 = ATV + VEC_FRAGS - N1;
    extern __shared__ char L[];
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
    const int slot0 = first_slot(c.seq, s), nc = (b - a + CH - 1) / CH, hk = h / (c.Hv / c.Hk);
    const char *keys = c.keys + ((int64_t)slot0 * c.Hk + hk) * c.key_bytes + (SAVE ? NF * FRAG : 0);
    const char *heads = c.heads + ((int64_t)slot0 * c.Hv + h) * c.head_bytes + (SAVE ? AT_T * FRAG : 0);
    const X *pv = (const X *)c.v + (int64_t)a * c.ldv + (int64_t)h * c.Dv + dv;
    Feed<N1, N2> feed;
    X vn[16];
    auto ahead = [&](int k) {
        feed.load(keys + (int64_t)k * c.Hk * c.key_bytes, heads + (int64_t)k * c.Hv * c.head_bytes, wave, lane);
        const int n = b - a - k * CH;
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = 16 * m + g4 + i;
                vn[4 * m + i] = in && t < n ? pv[((int64_t)k * CH + t) * c.ldv] : (X)0;
            }
    };
    if (nc > 0) ahead(0);
    for (int k = 0; k < nc; ++k) {
        const int n = b - a - k * CH;  // tokens left
        __syncthreads();
        feed.store(L, wave, lane);
        f32x4 x[4];
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) x[m][i] = DT::widen(vn[4 * m + i]);
        if (k + 1 < nc) ahead(k + 1);
        const int64_t at = (int64_t)(slot0 + k) * c.Hv + h;
        if (SAVE && dv < c.DvP) {
            float *d = S0s + at * DK * c.DvP + dv;
#pragma unroll
            for (int t = 0; t < DK / 16; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) d[(int64_t)(16 * t + g4 + i) * c.DvP] = S[t][i];
        }
        __syncthreads();
        const float *vec = (const float *)(L + ATV * FRAG);
        auto v4 = [&](int which, int m) { return *(const f32x4 *)&vec[which * CH + 16 * m + g4]; };
        f32x4 ks[4], os[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) ks[m] = os[m] = splat(0.0f);
#pragma unroll
        for (int kb = 0; kb < NK; ++kb) {
            bf16x8 t[3], w[NA];
            split(S[2 * kb], S[2 * kb + 1], t);
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                frag(w, L, ATK + (m * NK + kb) * NA, lane);
                ks[m] = mac(w, t, 2, ks[m]);
                if (!SAVE) {
                    frag(w, L, (m * NK + kb) * NA, lane);
                    os[m] = mac(w, t, 1, os[m]);
                }
            }
        }
        // R = beta (V - e^b K S), then U = T R
        bf16x8 rt[2][3];
#pragma unroll
        for (int m = 0; m < 4; ++m) x[m] = v4(V_BETA, m) * (x[m] - v4(V_EK, m) * ks[m]);
#pragma unroll
        for (int q = 0; q < 2; ++q) split(x[2 * q], x[2 * q + 1], rt[q]);
        f32x4 u[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            u[m] = splat(0.0f);
#pragma unroll
            for (int kb = 0; kb <= m / 2; ++kb) {
                bf16x8 w[T_TERMS];
                frag(w, L, ATT + lower_block(m, kb) * T_TERMS, lane);
                u[m] = mac(w, rt[kb], 2, u[m]);
            }
        }
        if (SAVE) {
            if (dv < c.DvP) {
                float *d = Us + at * CH * c.DvP + dv;
#pragma unroll
                for (int m = 0; m < 4; ++m)
#pragma unroll
                    for (int i = 0; i < 4; ++i) d[(int64_t)(16 * m + g4 + i) * c.DvP] = u[m][i];
            }
        } else {
            bf16x8 ut[2][2];
#pragma unroll
            for (int q = 0; q < 2; ++q) split(u[2 * q], u[2 * q + 1], ut[q]);
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                f32x4 y = v4(V_EQ, m) * os[m];
#pragma unroll
                for (int kb = 0; kb <= m / 2; ++kb) {
                    bf16x8 w[P_TERMS];
                    frag(w, L, ATP + lower_block(m, kb) * P_TERMS, lane);
                    y = mac(w, ut[kb], 1, y);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int t = 16 * m + g4 + i;
                    if (in && t < n) o[(a + k * CH + t) * ldo + (int64_t)h * c.Dv + dv] = DT::narrow(y[i]);
                }
            }
        }
        // S = e^{b_last} S + K^T (e^{b_last - b} U)
        const float el = vec[V_EB * CH + CH - 1];
#pragma unroll
        for (int m = 0; m < 4; ++m) u[m] *= v4(V_RK, m);
#pragma unroll
        for (int q = 0; q < 2; ++q) split(u[2 * q], u[2 * q + 1], rt[q]);
#pragma unroll
        for (int t = 0; t < DK / 16; ++t) {
            f32x4 y = S[t] * el;
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) {
                bf16x8 w[NA];
                frag(w, L, ATKT + (2 * t + kb) * NA, lane);
                y = mac(w, rt[kb], 2, y);
            }
            S[t] = y;
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

// Backward walk (as k_rscan in k_delta.hip).
template <class DT, int DK>
__global__ void __launch_bounds__(256) k_rscan(Ctx c, const typename DT::X *d_o, int64_t lddo, const float *dstate_out,
                                               float *dstate_in, typename DT::X *dvo, int64_t lddv, float *dSs,
                                               float *dRs) {
    using X = typename DT::X;
    constexpr int NA = Raw<DT>::TERMS, NK = DK / 32, NF = DK / 8 * NA;
    // LDS: K K^T Q^T | vectors T^T P^T
    constexpr int ATKT = NF, ATQT = 2 * NF, N1 = 3 * NF, ATV = N1, ATTT = ATV + VEC_FRAGS,
                  ATPT = ATTT + NBLK * T_TERMS, N2 = ATPT + NBLK * T_TERMS - N1;
    extern __shared__ char L[];
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
    const int slot0 = first_slot(c.seq, s), nc = (b - a + CH - 1) / CH, hk = h / (c.Hv / c.Hk);
    const char *keys = c.keys + ((int64_t)slot0 * c.Hk + hk) * c.key_bytes + NF * FRAG;
    const char *heads = c.heads + ((int64_t)slot0 * c.Hv + h) * c.head_bytes + AT_VEC * FRAG;
    const X *pd = d_o + (int64_t)a * lddo + (int64_t)h * c.Dv + dv;
    Feed<N1, N2> feed;
    X dn[16];
    auto ahead = [&](int k) {
        feed.load(keys + (int64_t)k * c.Hk * c.key_bytes, heads + (int64_t)k * c.Hv * c.head_bytes, wave, lane);
        const int n = b - a - k * CH;
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = 16 * m + g4 + i;
                dn[4 * m + i] = in && t < n ? pd[((int64_t)k * CH + t) * lddo] : (X)0;
            }
    };
    if (nc > 0) ahead(nc - 1);
    for (int k = nc - 1; k >= 0; --k) {
        const int n = b - a - k * CH;
        __syncthreads();
        feed.store(L, wave, lane);
        f32x4 dO[4];
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) dO[m][i] = DT::widen(dn[4 * m + i]);
        if (k > 0) ahead(k - 1);
        const int64_t at = (int64_t)(slot0 + k) * c.Hv + h;
        if (dv < c.DvP) {
            float *d = dSs + at * DK * c.DvP + dv;
#pragma unroll
            for (int t = 0; t < DK / 16; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) d[(int64_t)(16 * t + g4 + i) * c.DvP] = S[t][i];
        }
        __syncthreads();
        const float *vec = (const float *)(L + ATV * FRAG);
        auto v4 = [&](int which, int m) { return *(const f32x4 *)&vec[which * CH + 16 * m + g4]; };
        // dU = e^{b_last - b} (K dS) + P^T dO; dO's terms are exact
        f32x4 x[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) x[m] = splat(0.0f);
#pragma unroll
        for (int kb = 0; kb < NK; ++kb) {
            bf16x8 t[3], w[NA];
            split(S[2 * kb], S[2 * kb + 1], t);
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                frag(w, L, (m * NK + kb) * NA, lane);
                x[m] = mac(w, t, 2, x[m]);
            }
        }
        bf16x8 ot[2][NA], rt[2][3];
#pragma unroll
        for (int q = 0; q < 2; ++q) split(dO[2 * q], dO[2 * q + 1], ot[q]);
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            x[m] *= v4(V_RK, m);
#pragma unroll
            for (int kb = m / 2; kb < 2; ++kb) {
                bf16x8 w[T_TERMS];
                frag(w, L, ATPT + upper_block(m, kb) * T_TERMS, lane);
                x[m] = mac(w, ot[kb], 2, x[m]);
            }
        }
#pragma unroll
        for (int q = 0; q < 2; ++q) split(x[2 * q], x[2 * q + 1], rt[q]);
        f32x4 dR[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            dR[m] = splat(0.0f);
#pragma unroll
            for (int kb = m / 2; kb < 2; ++kb) {
                bf16x8 w[T_TERMS];
                frag(w, L, ATTT + upper_block(m, kb) * T_TERMS, lane);
                dR[m] = mac(w, rt[kb], 2, dR[m]);
            }
            const f32x4 y = dR[m] * v4(V_BETA, m);
            float *d = dRs + at * CH * c.DvP + dv;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = 16 * m + g4 + i;
                if (dv < c.DvP) d[(int64_t)t * c.DvP] = dR[m][i];
                if (in && t < n) dvo[(a + k * CH + t) * lddv + (int64_t)h * c.Dv + dv] = DT::narrow(y[i]);
            }
        }
        // dS = e^{b_last} dS + Q^T (scale e^b dO) - K^T (e^b beta dR)
        const float el = vec[V_EB * CH + CH - 1];
        bf16x8 qt[2][3];
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            dO[m] *= v4(V_EQ, m);
            dR[m] *= -v4(V_EK, m) * v4(V_BETA, m);
        }
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            split(dO[2 * q], dO[2 * q + 1], qt[q]);
            split(dR[2 * q], dR[2 * q + 1], rt[q]);
        }
#pragma unroll
        for (int t = 0; t < DK / 16; ++t) {
            f32x4 y = S[t] * el;
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) {
                bf16x8 w[NA];
                frag(w, L, ATQT + (2 * t + kb) * NA, lane);
                y = mac(w, qt[kb], 2, y);
                frag(w, L, ATKT + (2 * t + kb) * NA, lane);
                y = mac(w, rt[kb], 2, y);
            }
            S[t] = y;
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

hipError_t lds_room(const void *f, size_t bytes) {
    return hipFuncSetAttribute(f, hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

// Calls f with the type and the padded key size; sizes that split_runs leaves
// out never come here.
template <class F>
hipError_t pick(int dtype, int DK, F f) {
    if (dtype == DWCONV_BF16) {
        switch (DK) {
            case 64: return f(BF16{}, std::integral_constant<int, 64>{});
            case 128: return f(BF16{}, std::integral_constant<int, 128>{});
            case 192: return f(BF16{}, std::integral_constant<int, 192>{});
            default: return f(BF16{}, std::integral_constant<int, 256>{});
        }
    }
    return DK == 64 ? f(F16{}, std::integral_constant<int, 64>{}) : f(F16{}, std::integral_constant<int, 128>{});
}

}  // namespace

namespace delta {

hipError_t split_prepare(int dtype, int DK_, const Ctx &c, bool backward, hipStream_t st) {
    return pick(dtype, DK_, [&](auto dt, auto dk) {
        using DT = decltype(dt);
        constexpr int DK = decltype(dk)::value;
        const size_t n = 2 * CH * (DK + 8) * 2 + (3 * TRI + 4 * 256) * sizeof(float);
        const uint32_t blocks = (uint32_t)((int64_t)c.slots * c.Hk);
        auto f = backward ? k_prepare<DT, DK, true> : k_prepare<DT, DK, false>;
        hipError_t e = lds_room((const void *)f, n);
        if (e != hipSuccess) return e;
        f<<<blocks, 256, n, st>>>(c);
        return hipGetLastError();
    });
}

hipError_t split_scan(int dtype, int DK_, const Ctx &c, const float *state_in, float *state_out, void *o, int64_t ldo,
                      float *S0s, float *Us, hipStream_t st) {
    return pick(dtype, DK_, [&](auto dt, auto dk) {
        using DT = decltype(dt);
        using X = typename DT::X;
        constexpr int DK = decltype(dk)::value;
        const uint32_t blocks = (uint32_t)((int64_t)c.seq.seqs * c.Hv * ((c.Dv + 63) / 64));
        const size_t n = lds_fwd(DK, Raw<DT>::TERMS);
        auto f = S0s ? k_scan<DT, DK, true> : k_scan<DT, DK, false>;
        hipError_t e = lds_room((const void *)f, n);
        if (e != hipSuccess) return e;
        f<<<blocks, 256, n, st>>>(c, state_in, state_out, (X *)o, ldo, S0s, Us);
        return hipGetLastError();
    });
}

hipError_t split_rscan(int dtype, int DK_, const Ctx &c, const void *d_o, int64_t lddo, const float *dstate_out,
                       float *dstate_in, void *dv, int64_t lddv, float *dSs, float *dRs, hipStream_t st) {
    return pick(dtype, DK_, [&](auto dt, auto dk) {
        using DT = decltype(dt);
        using X = typename DT::X;
        constexpr int DK = decltype(dk)::value;
        const uint32_t blocks = (uint32_t)((int64_t)c.seq.seqs * c.Hv * ((c.Dv + 63) / 64));
        const size_t n = lds_bwd(DK, Raw<DT>::TERMS);
        hipError_t e = lds_room((const void *)k_rscan<DT, DK>, n);
        if (e != hipSuccess) return e;
        k_rscan<DT, DK><<<blocks, 256, n, st>>>(c, (const X *)d_o, lddo, dstate_out, dstate_in, (X *)dv, lddv, dSs, dRs);
        return hipGetLastError();
    });
}

}  // namespace delta
}  // namespace dw
