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
// times three), six for two fp32 ones.  What makes o is no exception: Q S0 and
// P U can cancel, and their errors stay.
//
// A workgroup walks one sequence's chunks for one head and 16 NT columns of the
// state.  Wavefront w has tokens 16 w .. 16 w + 15 of every chunk and a quarter
// of the state's rows, so that a chunk's chain of products (K S, T R, K^T U) is
// a quarter as long as in one wavefront; right operands are split by the
// wavefront that made them and pass through LDS, three barriers a chunk.  Left
// operands each serve one wavefront: they go from the workspace, where
// k_prepare lays them out as fragments (delta_common.h), straight to registers,
// and a register is loaded for the next chunk as soon as it has been used.
//
// Bound by each chunk's chain of dependent products, splits and barriers, not
// by a rate: measured, bf16, heads of 128 x 128, 8192 tokens of 32 value heads
// in five sequences, k_scan 188 to 197 us (108 matrix instructions of 16 cycles a
// wavefront and chunk in some nine thousand cycles), 640 workgroups on 512 places;
// gradients of 4096 tokens, 16 heads, four sequences: k_scan 60, k_rscan 94.  One
// fp16 sequence of 5003 tokens, 6 heads of 96 x 104: 154 us, 1.9 us a chunk.  Few
// registers spill: 6 a lane in k_rscan of bf16 with 32 columns at keys of 128 and
// with 16 at keys of 256, 11 in k_scan of bf16 with 16 columns at keys of 256.
#include "delta_split.h"

namespace dw {
namespace {

using namespace delta;

// One chunk and key head: lengths, the triangles of its value heads, and all
// left operands as fragments.  8192 tokens, 16 key and 32 value heads of 128,
// bf16: 90 us, bound by the latency of the triangle's inverse (16 dependent
// steps a tile, then the tiles below it), three workgroups a CU, for which four
// registers a lane spill at keys of up to 128 channels.  It writes 38 KB a value head
// and chunk and 48 KB a key head, 260 MB here, which the walks read back once for
// each group of columns.
// (LDS: the rows of q and k, later the triangles.)
template <int DK>
constexpr size_t lds_prepare() {
    constexpr size_t rows = 2 * CH * (DK + 8) * 2, triangles = (2 * TRI + 4 * 256) * sizeof(float);
    return rows > triangles ? rows : triangles;
}
template <class DT, int DK, bool BACK>
__global__ void __launch_bounds__(256, (DK <= 128 ? 3 : 2)) k_prepare(Ctx c) {
    using X = typename DT::X;
    using R = Raw<DT>;
    using V8 = typename R::V8;
    constexpr int NA = R::TERMS, PITCH = DK + 8;
    extern __shared__ char lds_raw[];
    X(*K)[PITCH] = (X(*)[PITCH])lds_raw;
    X(*Q)[PITCH] = K + CH;
    float *At = (float *)lds_raw, *Pl = At + TRI, *Tl = At, *Td = Pl + TRI;  // T takes A's place
    __shared__ double b[4][CH];
    __shared__ float beta[4][CH], rk[CH], rq[CH];
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
#pragma unroll
        for (int f4 = 0; f4 < (BACK ? 4 : 3) * NF; f4 += 4) {
            const int f = f4 + wave, mat = f4 / NF, i = f % NF;
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
    const int group = c.Hv / c.Hk, h0 = hk * group;
    for (int n = 0; n < group; ++n) {
        // made anew for each head: kept over the loop, the addresses and
        // comparisons that follow from these would take the registers
        int lane = threadIdx.x & 63;
        asm volatile("" : "+v"(lane));
        const int r = lane & 15, g4 = (lane >> 4) * 4;
        const int h = h0 + n;
        const int64_t at = (int64_t)slot * c.Hv + h;
        char *base = c.heads + at * c.head_bytes;
        const int w = n & 3;
        __syncthreads();  // rows, or the previous head's values, have been read
        if (w == 0) {     // the vectors of four heads, one a wavefront
            const int hw = h + wave;
            if (n + wave < group) {
                const float be = lane < ch.n ? c.beta[((int64_t)ch.tok + lane) * c.Hv + hw] : 0.0f;
                const double x = running_sum(c.g + (int64_t)ch.tok * c.Hv + hw, c.Hv, ch.n, lane);
                const double last = __shfl(x, 63, 64);
                const float eb = expf((float)x), er = expf((float)(last - x));
                b[wave][lane] = x;
                beta[wave][lane] = be;
                float *v = (float *)(base + wave * c.head_bytes + AT_VEC * FRAG);
                v[V_EK * CH + lane] = eb * rk[lane];
                v[V_RK * CH + lane] = er * rk[lane];
                v[V_BETA * CH + lane] = be;
                v[V_EQ * CH + lane] = c.scale * eb * rq[lane];
                v[V_EB * CH + lane] = eb;
                if (BACK) {
                    v[V_ER * CH + lane] = er;
                    v[V_NK * CH + lane] = rk[lane];
                    v[V_NQ * CH + lane] = rq[lane];
                    c.sums[(at + wave) * CH + lane] = x;
                }
            }
            __syncthreads();
        }
        float z = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (j > wave) continue;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = 16 * wave + g4 + i, col = 16 * j + r;
                const float d = row >= col ? expf((float)(b[w][row] - b[w][col])) : 0.0f;
                const float p = row >= col ? c.scale * d * (rq[row] * rk[col] * qk[j][i]) : 0.0f;
                const int e = tri(wave, j) + (g4 + i) * 16 + r;
                const float a = row > col ? beta[w][row] * d * (rk[row] * rk[col] * kk[j][i]) : 0.0f;
                At[e] = a;
                z = __builtin_fmaf(a, 0.0f, z);
                Pl[e] = p;
            }
        }
        take_out_rows(z, At, (float *)(base + AT_VEC * FRAG) + V_BETA * CH, wave, r, g4);
        __syncthreads();
        f32x4 Tc[4];
        invert(At, Td, wave, r, g4, Tc);
        __syncthreads();
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            if (wave + n >= 4) break;
#pragma unroll
            for (int i = 0; i < 4; ++i) Tl[tri(wave + n, wave) + (g4 + i) * 16 + r] = Tc[n][i];
        }
        __syncthreads();
#pragma unroll
        for (int f4 = 0; f4 < (BACK ? 4 : 2) * NBLK; f4 += 4) {
            const int f = f4 + wave, what = f / NBLK, blk = f % NBLK;  // P, T, T^T, P^T
            const float *S = what == 0 || what == 3 ? Pl : Tl;
            f32x4 x[2];
            if (what < 2) {
                const int m = lower_m(blk), kb = lower_kb(blk);
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    x[j] = 2 * kb + j <= m ? *(const f32x4 *)&S[tri(m, 2 * kb + j) + r * 16 + g4] : splat(0.0f);
            } else {
                const int m = upper_m(blk), kb = upper_kb(blk);
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        x[j][i] = 2 * kb + j >= m ? S[tri(2 * kb + j, m) + (g4 + i) * 16 + r] : 0.0f;
            }
            bf16x8 t[TRI_TERMS];
            split(x[0], x[1], t);
            const int first = what == 0 ? AT_P : what == 1 ? AT_T : what == 2 ? AT_TT : AT_PT;
#pragma unroll
            for (int n = 0; n < TRI_TERMS; ++n)
                *(bf16x8 *)(base + (int64_t)(first + blk * TRI_TERMS + n) * FRAG + lane * 16) = t[n];
        }
    }
}

// The columns of a walk: NT tiles of 16 from `first` on; a lane's column of
// tile t is first + 16 t + lane % 16.
template <int NT>
struct Columns {
    int dv[NT], at[NT];  // the column, and the column itself or the last one
    bool in[NT];
    __device__ __forceinline__ Columns(int first, int r, int Dv) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            dv[t] = first + 16 * t + r;
            in[t] = dv[t] < Dv;
            at[t] = in[t] ? dv[t] : Dv - 1;
        }
    }
};

// Four tokens (row .. row + 3, row = row0 + g4 of a chunk at p) x NT columns of
// v or dO.  Loads are clamped to the n tokens that are left and not looked at
// (that would wait for them); `widened` puts zeros in place of what is not
// there.  Whole chunks take addresses of a uniform part and a 32-bit one.
struct Rows {
    int64_t ld;
    uint32_t lane;  // elements from the wavefront's first row to the lane's
    bool narrow;    // lane parts fit 32 bits
    __device__ __forceinline__ Rows(int64_t ld, int g4) : ld(ld), lane((uint32_t)ld * g4), narrow(ld < (1 << 26)) {}
};
template <class X, int NT>
__device__ __forceinline__ void fetch_tokens(X (&v)[NT][4], const X *p, const Rows &R, int n, int row0, int g4,
                                             const Columns<NT> &cl) {
    if (n >= CH && R.narrow) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const X *q = p + (row0 + i) * R.ld;
#pragma unroll
            for (int t = 0; t < NT; ++t) v[t][i] = q[R.lane + (uint32_t)cl.at[t]];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const X *q = p + min(row0 + g4 + i, n - 1) * R.ld;
#pragma unroll
            for (int t = 0; t < NT; ++t) v[t][i] = q[cl.at[t]];
        }
    }
}
template <class DT, int NT>
__device__ __forceinline__ f32x4 widened(const typename DT::X (&v)[NT][4], int t, int n, int row, const Columns<NT> &cl) {
    f32x4 x;
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = cl.in[t] && row + i < n ? DT::widen(v[t][i]) : 0.0f;
    return x;
}
template <class DT, int NT>
__device__ __forceinline__ void store_tokens(typename DT::X *p, const Rows &R, const f32x4 (&x)[NT], int n, int row0,
                                             int g4, const Columns<NT> &cl) {
    if (n >= CH && R.narrow) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
            if (cl.in[t]) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    (p + (row0 + i) * R.ld)[R.lane + (uint32_t)cl.dv[t]] = rounded<DT>(x[t][i]);
            }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (row0 + g4 + i < n) {
                typename DT::X *q = p + (row0 + g4 + i) * R.ld;
#pragma unroll
                for (int t = 0; t < NT; ++t)
                    if (cl.in[t]) q[cl.dv[t]] = rounded<DT>(x[t][i]);
            }
    }
}

// A wavefront's rows of the state: tiles w T .. w T + T - 1, T = DK / 64.
template <int DK, int NT>
struct State {
    static constexpr int T = DK / 64;
    f32x4 S[T][NT];
    __device__ __forceinline__ void load(const float *p, const Ctx &c, int wave, int g4, const Columns<NT> &cl) {
#pragma unroll
        for (int x = 0; x < T; ++x)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int row = 16 * (wave * T + x) + g4 + i;
                    S[x][t][i] = p && cl.in[t] && row < c.Dk ? p[(int64_t)row * c.Dv + cl.dv[t]] : 0.0f;
                }
    }
    __device__ __forceinline__ void store(float *p, const Ctx &c, int wave, int g4, const Columns<NT> &cl) const {
#pragma unroll
        for (int x = 0; x < T; ++x)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int row = 16 * (wave * T + x) + g4 + i;
                    if (cl.in[t] && row < c.Dk) p[(int64_t)row * c.Dv + cl.dv[t]] = S[x][t][i];
                }
    }
    // all DK rows of all DvP columns, for the backward pass
    __device__ __forceinline__ void keep(float *p, const Ctx &c, int wave, int g4, const Columns<NT> &cl) const {
        const uint32_t lane = g4 * c.DvP;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int x = 0; x < T; ++x)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    (p + (16 * (wave * T + x) + i) * c.DvP)[lane + (uint32_t)cl.dv[t]] = S[x][t][i];
    }
    __device__ __forceinline__ void put(const Right<NT, 3> &r, int wave, int lane) const {
#pragma unroll
        for (int x = 0; x < T; ++x)
#pragma unroll
            for (int t = 0; t < NT; ++t) r.put(wave * T + x, t, S[x][t], lane);
    }
};
template <int NT>
__device__ __forceinline__ void keep_tokens(float *p, const Ctx &c, const f32x4 (&x)[NT], int row0, int g4,
                                            const Columns<NT> &cl) {
    const uint32_t lane = g4 * c.DvP;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) (p + (row0 + i) * c.DvP)[lane + (uint32_t)cl.dv[t]] = x[t][i];
}

// Which walk a workgroup has.  The column groups of the value heads of one key
// head and sequence (a unit) share operands: they go to one XCD, one behind the
// other; units go round the XCDs, so that each gets its share of every
// sequence.  Fewer than eight units leave XCDs without work: 8192 bf16 tokens in
// one sequence, 16 value heads of 128 x 128, k_scan with 16 key heads 224 us, with
// one 577.  `width`: columns walked (the backward pass also fills the padded ones).
// A grid that the XCDs do not divide has workgroups without a walk.
struct Walk {
    int first, h, s;
    __device__ __forceinline__ Walk(const Ctx &c, int cols, int width) {
        const uint32_t nb = (width + cols - 1) / cols, group = c.Hv / c.Hk, per = nb * group;
        const uint32_t j = blockIdx.x / 8, unit = j / per * 8 + blockIdx.x % 8, i = j % per;
        first = (int)(i % nb) * cols;
        h = (int)(unit % c.Hk * group + i / nb);
        s = (int)(unit / c.Hk);
    }
    static uint64_t blocks(const Ctx &c, int cols, int width) {
        const uint64_t units = (uint64_t)c.seq.seqs * c.Hk, per = (uint64_t)((width + cols - 1) / cols) * (c.Hv / c.Hk);
        return (units + 7) / 8 * 8 * per;
    }
};

// Two workgroups a CU where their registers allow it (a wavefront that may have
// more than 256 also keeps results in accumulation registers and moves them).
template <class DT, int DK, int NT>
constexpr int walks_a_cu() { return DK * Raw<DT>::TERMS * NT <= 256 ? 2 : 1; }

// Forward walk.  SAVE: keeps each chunk's state and U for the backward pass
// instead of making outputs.
template <class DT, int DK, int NT, bool SAVE>
__global__ void __launch_bounds__(256, (walks_a_cu<DT, DK, NT>())) k_scan(Ctx c, const float *state_in, float *state_out, typename DT::X *o,
                                              int64_t ldo, float *S0s, float *Us) {
    using X = typename DT::X;
    constexpr int NA = Raw<DT>::TERMS, NK = DK / 32, NF = DK / 8 * NA, T = DK / 64;
    extern __shared__ char L[];
    const Right<NT, 3> SB{L}, RB{SB.p + SB.bytes(NK)}, EB{RB.p + RB.bytes(2)}, UB{EB.p + EB.bytes(2)};
    const Walk wk(c, 16 * NT, SAVE ? c.DvP : c.Dv);
    if (wk.s >= c.seq.seqs) return;
    // each column's first token that is no number, CH: none.  A column stays spoiled:
    // its state is NaN behind the chunk, so all of R in the next one
    __shared__ int spoiled[16 * NT];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r = lane & 15,
              g4 = (lane >> 4) * 4;
    const int h = wk.h, row = 16 * wave + g4;  // this lane's tokens: row .. row + 3
    if (!SAVE && threadIdx.x < 16 * NT) spoiled[threadIdx.x] = CH;
    const Columns<NT> cl(wk.first, r, c.Dv);
    const Rows rv(c.ldv, g4), ro(ldo, g4);
    const int a = uniform(c.seq.begin(wk.s)), b = uniform(c.seq.end(wk.s));
    const int64_t st = ((int64_t)wk.s * c.Hv + h) * c.Dk * c.Dv;
    State<DK, NT> S;
    S.load(state_in ? state_in + st : nullptr, c, wave, g4, cl);
    const int slot0 = a / CH + wk.s, nc = (b - a + CH - 1) / CH, hk = h / (c.Hv / c.Hk);
    const X *pv = (const X *)c.v + (int64_t)a * c.ldv + (int64_t)h * c.Dv;
    X *po = SAVE ? nullptr : o + (int64_t)a * ldo + (int64_t)h * c.Dv;
    // operands of the chunk at hand
    bf16x8 wK[NK][NA], wQ[SAVE ? 1 : NK][NA], wT[2][TRI_TERMS], wP[2][TRI_TERMS], wKT[T][2][NA];
    f32x4 ek, rk, beta, eq;
    float el;
    X vn[NT][4];
    auto keys_of = [&](int k) { return c.keys + ((int64_t)(slot0 + k) * c.Hk + hk) * c.key_bytes; };
    auto head_of = [&](int k) { return c.heads + ((int64_t)(slot0 + k) * c.Hv + h) * c.head_bytes; };
    // (fetches stand between the products, a few at a time: a wavefront that
    // issues many at once waits for the load path, which its neighbours share)
    auto fetch_row = [&](int k, int kb) {  // what the first products need
        const char *p = keys_of(k);
        fetch(wK[kb], p + (NF + (wave * NK + kb) * NA) * FRAG, lane);
        if (!SAVE) fetch(wQ[kb], p + (wave * NK + kb) * NA * FRAG, lane);
    };
    auto fetch_V = [&](int k) {
        fetch_tokens<X, NT>(vn, pv + (int64_t)k * CH * c.ldv, rv, b - a - k * CH, 16 * wave, g4, cl);
        const float *v = (const float *)(head_of(k) + AT_VEC * FRAG);
        ek = *(const f32x4 *)(v + V_EK * CH + row);
        beta = *(const f32x4 *)(v + V_BETA * CH + row);
        if (!SAVE) eq = *(const f32x4 *)(v + V_EQ * CH + row);
    };
    auto fetch_T = [&](int k) {
        const char *p = head_of(k);
        fetch(wT[0], p + (AT_T + lower_block(wave, 0) * TRI_TERMS) * FRAG, lane);
        if (wave >= 2) fetch(wT[1], p + (AT_T + lower_block(wave, 1) * TRI_TERMS) * FRAG, lane);
        rk = *(const f32x4 *)((const float *)(p + AT_VEC * FRAG) + V_RK * CH + row);
    };
    auto fetch_KT = [&](int k, int kb) {
        const char *p = keys_of(k) + 2 * NF * FRAG;
#pragma unroll
        for (int x = 0; x < T; ++x) fetch(wKT[x][kb], p + (2 * (wave * T + x) + kb) * NA * FRAG, lane);
        if (kb) el = ((const float *)(head_of(k) + AT_VEC * FRAG))[V_EB * CH + CH - 1];
    };
    // (P is fetched in its own chunk, behind the first products: three terms of it kept
    // from the chunk before spill; 8192 tokens, 32 heads of 128, bf16: 252 and 284 us a call)
    auto fetch_P = [&](int k) {
        const char *p = head_of(k);
        fetch(wP[0], p + (AT_P + lower_block(wave, 0) * TRI_TERMS) * FRAG, lane);
        if (wave >= 2) fetch(wP[1], p + (AT_P + lower_block(wave, 1) * TRI_TERMS) * FRAG, lane);
    };
    if (nc > 0) {
#pragma unroll
        for (int kb = 0; kb < NK; ++kb) fetch_row(0, kb);
        fetch_V(0);
        fetch_T(0);
        fetch_KT(0, 0);
        fetch_KT(0, 1);
        S.put(SB, wave, lane);
    }
    for (int k = 0; k < nc; ++k) {
        const int n = b - a - k * CH, next = k + 1 < nc ? k + 1 : k;  // tokens left; the last chunk is fetched again
        const int64_t at = (int64_t)(slot0 + k) * c.Hv + h;
        __syncthreads();
        if (SAVE) S.keep(S0s + at * DK * c.DvP, c, wave, g4, cl);
        // R = beta (V - e^b K S)
        f32x4 ks[NT], y[NT], u[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) ks[t] = y[t] = u[t] = splat(0.0f);
        bf16x8 s[2][NT][3];
        SB.get(0, s[0], lane);
#pragma unroll
        for (int kb = 0; kb < NK; ++kb) {
            if (kb + 1 < NK) SB.get(kb + 1, s[(kb + 1) & 1], lane);
            fence();
            mac(wK[kb], s[kb & 1], 2, ks);
            if (!SAVE) mac(wQ[kb], s[kb & 1], 2, y);
            fetch_row(next, kb);
            fence();
        }
        f32x4 R[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            R[t] = beta * (widened<DT, NT>(vn, t, n, row, cl) - ek * ks[t]);
            if (!SAVE) y[t] *= eq;
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) RB.put(wave, t, R[t], lane);
        fetch_V(next);
        // (the paths that hardly any chunk takes stand apart, at the barriers: the
        // compiler keeps them out of the way of the others' registers)
        if (!SAVE && __builtin_expect(any_no_number(R), 0)) {
#pragma unroll
            for (int t = 0; t < NT; ++t) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (no_number(R[t][i])) atomicMin(&spoiled[16 * t + r], row + i), R[t][i] = 0.0f;
                RB.put(wave, t, R[t], lane);
            }
        }
        __syncthreads();
        // U = T R
        RB.get(0, s[0], lane);
        RB.get(1, s[1], lane);
        int from[NT];
        bool some = false;
#pragma unroll
        for (int t = 0; t < NT; ++t) from[t] = SAVE ? CH : spoiled[16 * t + r];
        fence();
        mac(wT[0], s[0], 2, u);
        if (wave >= 2) mac(wT[1], s[1], 2, u);
        const f32x4 rk_now = rk;
        fetch_T(next);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            EB.put(wave, t, u[t] * rk_now, lane);
            if (!SAVE) UB.put(wave, t, u[t], lane);
        }
        if (!SAVE) fetch_P(k);
        if (!SAVE) {
#pragma unroll
            for (int t = 0; t < NT; ++t) some |= from[t] < CH;
            if (__builtin_expect(__any(some), 0)) {
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    if (row + 3 < from[t]) continue;
                    put_from(u[t], row, from[t], 0.0f);
                    put_from(y[t], row, from[t], __builtin_nanf(""));
                    UB.put(wave, t, u[t], lane);
                    EB.put(wave, t, splat(__builtin_nanf("")), lane);
                }
            }
        }
        if (SAVE) keep_tokens<NT>(Us + at * CH * c.DvP, c, u, 16 * wave, g4, cl);
        __syncthreads();
        // S = e^{b_last} S + K^T (e^{b_last - b} U)
        EB.get(0, s[0], lane);
        EB.get(1, s[1], lane);
        fence();
#pragma unroll
        for (int x = 0; x < T; ++x)
#pragma unroll
            for (int t = 0; t < NT; ++t) S.S[x][t] *= el;
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
#pragma unroll
            for (int x = 0; x < T; ++x) mac(wKT[x][kb], s[kb], 2, S.S[x]);
            fetch_KT(next, kb);
        }
        S.put(SB, wave, lane);
        // O = scale e^b (Q S0) + P U
        if (!SAVE) {
            UB.get(0, s[0], lane);
            UB.get(1, s[1], lane);
            mac(wP[0], s[0], 2, y);
            if (wave >= 2) mac(wP[1], s[1], 2, y);
            store_tokens<DT, NT>(po + (int64_t)k * CH * ldo, ro, y, n, 16 * wave, g4, cl);
        }
    }
    if (state_out) S.store(state_out + st, c, wave, g4, cl);
}

// Backward walk.
template <class DT, int DK, int NT>
__global__ void __launch_bounds__(256, (walks_a_cu<DT, DK, NT>())) k_rscan(Ctx c, const typename DT::X *d_o, int64_t lddo, const float *dstate_out,
                                               float *dstate_in, typename DT::X *dvo, int64_t lddv, float *dSs,
                                               float *dRs) {
    using X = typename DT::X;
    constexpr int NA = Raw<DT>::TERMS, NK = DK / 32, NF = DK / 8 * NA, T = DK / 64;
    extern __shared__ char L[];
    const Right<NT, 3> SB{L}, XB{SB.p + SB.bytes(NK)}, QB{XB.p + XB.bytes(2)}, ZB{QB.p + QB.bytes(2)};
    const Right<NT, NA> OB{ZB.p + ZB.bytes(2)};
    const Walk wk(c, 16 * NT, c.DvP);
    if (wk.s >= c.seq.seqs) return;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r = lane & 15,
              g4 = (lane >> 4) * 4;
    const int h = wk.h, row = 16 * wave + g4;
    const Columns<NT> cl(wk.first, r, c.Dv);
    const Rows rd(lddo, g4), rv(lddv, g4);
    const int a = uniform(c.seq.begin(wk.s)), b = uniform(c.seq.end(wk.s));
    const int64_t st = ((int64_t)wk.s * c.Hv + h) * c.Dk * c.Dv;
    State<DK, NT> S;
    S.load(dstate_out ? dstate_out + st : nullptr, c, wave, g4, cl);
    const int slot0 = a / CH + wk.s, nc = (b - a + CH - 1) / CH, hk = h / (c.Hv / c.Hk);
    const X *pd = d_o + (int64_t)a * lddo + (int64_t)h * c.Dv;
    X *pv = dvo + (int64_t)a * lddv + (int64_t)h * c.Dv;
    bf16x8 wK[NK][NA], wPT[2][TRI_TERMS], wTT[2][TRI_TERMS], wKT[T][2][NA], wQT[T][2][NA];
    f32x4 ek, rk, beta, eq;
    float el;
    X dn[NT][4];
    auto keys_of = [&](int k) { return c.keys + ((int64_t)(slot0 + k) * c.Hk + hk) * c.key_bytes; };
    auto head_of = [&](int k) { return c.heads + ((int64_t)(slot0 + k) * c.Hv + h) * c.head_bytes; };
    auto fetch_tokens_of = [&](int k) {
        fetch_tokens<X, NT>(dn, pd + (int64_t)k * CH * lddo, rd, b - a - k * CH, 16 * wave, g4, cl);
        eq = *(const f32x4 *)((const float *)(head_of(k) + AT_VEC * FRAG) + V_EQ * CH + row);
    };
    auto fetch_row = [&](int k, int kb) { fetch(wK[kb], keys_of(k) + (NF + (wave * NK + kb) * NA) * FRAG, lane); };
    auto fetch_P = [&](int k) {
        const char *q = head_of(k);
        fetch(wPT[1], q + (AT_PT + upper_block(wave, 1) * TRI_TERMS) * FRAG, lane);
        if (wave < 2) fetch(wPT[0], q + (AT_PT + upper_block(wave, 0) * TRI_TERMS) * FRAG, lane);
        rk = *(const f32x4 *)((const float *)(q + AT_VEC * FRAG) + V_RK * CH + row);
    };
    auto fetch_T = [&](int k) {
        const char *q = head_of(k);
        const float *v = (const float *)(q + AT_VEC * FRAG);
        fetch(wTT[1], q + (AT_TT + upper_block(wave, 1) * TRI_TERMS) * FRAG, lane);
        if (wave < 2) fetch(wTT[0], q + (AT_TT + upper_block(wave, 0) * TRI_TERMS) * FRAG, lane);
        beta = *(const f32x4 *)(v + V_BETA * CH + row);
        ek = *(const f32x4 *)(v + V_EK * CH + row);
    };
    auto fetch_columns = [&](int k, int kb, bool q) {
        const char *p = keys_of(k) + (q ? 3 : 2) * NF * FRAG;
#pragma unroll
        for (int x = 0; x < T; ++x) fetch(q ? wQT[x][kb] : wKT[x][kb], p + (2 * (wave * T + x) + kb) * NA * FRAG, lane);
        if (q && kb) el = ((const float *)(head_of(k) + AT_VEC * FRAG))[V_EB * CH + CH - 1];
    };
    // dO's terms (exact) and those of scale e^b dO, for all wavefronts
    auto put_tokens = [&](int k) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const f32x4 x = widened<DT, NT>(dn, t, b - a - k * CH, row, cl);
            OB.put(wave, t, x, lane);
            QB.put(wave, t, x * eq, lane);
        }
    };
    if (nc > 0) {
        fetch_tokens_of(nc - 1);
#pragma unroll
        for (int kb = 0; kb < NK; ++kb) fetch_row(nc - 1, kb);
        fetch_P(nc - 1);
        fetch_T(nc - 1);
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            fetch_columns(nc - 1, kb, true);
            fetch_columns(nc - 1, kb, false);
        }
        put_tokens(nc - 1);
        fetch_tokens_of(nc > 1 ? nc - 2 : 0);
        S.put(SB, wave, lane);
    }
    for (int k = nc - 1; k >= 0; --k) {
        const int n = b - a - k * CH, next = k > 0 ? k - 1 : 0;
        const int64_t at = (int64_t)(slot0 + k) * c.Hv + h;
        __syncthreads();
        S.keep(dSs + at * DK * c.DvP, c, wave, g4, cl);
        // dU = e^{b_last - b} (K dS) + P^T dO
        f32x4 x[NT], y[NT], dR[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) x[t] = dR[t] = splat(0.0f);
        bf16x8 s[2][NT][3], ot[2][NT][NA];
        SB.get(0, s[0], lane);
#pragma unroll
        for (int kb = 0; kb < NK; ++kb) {
            if (kb + 1 < NK) {
                SB.get(kb + 1, s[(kb + 1) & 1], lane);
            } else {
                OB.get(0, ot[0], lane);
                OB.get(1, ot[1], lane);
            }
            fence();
            mac(wK[kb], s[kb & 1], 2, x);
            fetch_row(next, kb);
            fence();
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) x[t] *= rk;
        mac(wPT[1], ot[1], 2, x);
        if (wave < 2) mac(wPT[0], ot[0], 2, x);
        fetch_P(next);
#pragma unroll
        for (int t = 0; t < NT; ++t) XB.put(wave, t, x[t], lane);
        __syncthreads();
        // dR = T^T dU, dV = beta dR; the part of dS that needs no dR
        XB.get(0, s[0], lane);
        XB.get(1, s[1], lane);
        fence();
        mac(wTT[1], s[1], 2, dR);
        if (wave < 2) mac(wTT[0], s[0], 2, dR);
        const f32x4 beta_now = beta, ek_now = ek;
        fetch_T(next);
        QB.get(0, s[0], lane);
        QB.get(1, s[1], lane);
        fence();
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            y[t] = beta_now * dR[t];
            ZB.put(wave, t, -ek_now * y[t], lane);
        }
#pragma unroll
        for (int z = 0; z < T; ++z)
#pragma unroll
            for (int t = 0; t < NT; ++t) S.S[z][t] *= el;
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
#pragma unroll
            for (int z = 0; z < T; ++z) mac(wQT[z][kb], s[kb], 2, S.S[z]);
            fetch_columns(next, kb, true);
        }
        keep_tokens<NT>(dRs + at * CH * c.DvP, c, dR, 16 * wave, g4, cl);
        store_tokens<DT, NT>(pv + (int64_t)k * CH * lddv, rv, y, n, 16 * wave, g4, cl);
        __syncthreads();
        // dS = e^{b_last} dS + Q^T (scale e^b dO) - K^T (e^b beta dR)
        ZB.get(0, s[0], lane);
        ZB.get(1, s[1], lane);
        fence();
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
#pragma unroll
            for (int z = 0; z < T; ++z) mac(wKT[z][kb], s[kb], 2, S.S[z]);
            fetch_columns(next, kb, false);
        }
        S.put(SB, wave, lane);
        put_tokens(next);
        fetch_tokens_of(next > 0 ? next - 1 : 0);
    }
    if (dstate_in) S.store(dstate_in + st, c, wave, g4, cl);
}

// Columns of the state a workgroup walks: 32, or 16 where a CU would have no
// second walk to fill its waits, were the walks spread over all CUs (Walk says when
// they are not).  8192 bf16 tokens, 16 key and 32 value heads of 128 x 128, k_scan
// with 16 columns against 32: one sequence (128 walks of 32 columns) 294 and
// 355 us, two 230 and 232, three 245 and 202, five 258 and 189; one fp16 sequence of
// 5003 tokens, 6 heads of 96 x 104: 154 and 261.
int walk_tiles(const Ctx &c) { return (int64_t)c.seq.seqs * c.Hv * ((c.Dv + 31) / 32) <= 256 ? 1 : 2; }

template <int NT>
size_t lds_scan(int DK) { return (size_t)(DK / 32 + 6) * NT * 3 * FRAG; }
template <int NT>
size_t lds_rscan(int DK, int terms) { return (size_t)(DK / 32 + 6) * NT * 3 * FRAG + (size_t)2 * NT * terms * FRAG; }

}  // namespace

namespace delta {

uint64_t split_blocks(const Ctx &c, bool backward) {
    return Walk::blocks(c, 16 * walk_tiles(c), backward ? c.DvP : c.Dv);
}

hipError_t split_prepare(int dtype, int DK_, const Ctx &c, bool backward, hipStream_t st) {
    return pick(dtype, DK_, [&](auto dt, auto dk) {
        using DT = decltype(dt);
        constexpr int DK = decltype(dk)::value;
        const size_t n = lds_prepare<DK>();
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
        const int nt = walk_tiles(c);
        const uint32_t blocks = (uint32_t)Walk::blocks(c, 16 * nt, S0s ? c.DvP : c.Dv);
        const size_t n = nt == 1 ? lds_scan<1>(DK) : lds_scan<2>(DK);
        auto f = nt == 1 ? (S0s ? k_scan<DT, DK, 1, true> : k_scan<DT, DK, 1, false>)
                         : (S0s ? k_scan<DT, DK, 2, true> : k_scan<DT, DK, 2, false>);
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
        const int nt = walk_tiles(c);
        const uint32_t blocks = (uint32_t)Walk::blocks(c, 16 * nt, c.DvP);
        const size_t n = nt == 1 ? lds_rscan<1>(DK, Raw<DT>::TERMS) : lds_rscan<2>(DK, Raw<DT>::TERMS);
        auto f = nt == 1 ? k_rscan<DT, DK, 1> : k_rscan<DT, DK, 2>;
        hipError_t e = lds_room((const void *)f, n);
        if (e != hipSuccess) return e;
        f<<<blocks, 256, n, st>>>(c, (const X *)d_o, lddo, dstate_out, dstate_in, (X *)dv, lddv, dSs, dRs);
        return hipGetLastError();
    });
}

}  // namespace delta
}  // namespace dw
