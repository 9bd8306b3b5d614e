// k_causal.hip -- causal depthwise 1-D convolution of packed sequences
// (include/dwconv_seq.h): forward, one cached token, gradients.
//
// Bound by HBM: 2K operations an element against 4 to 8 bytes moved.  A lane
// owns one 16-byte vector of channels and walks a run of TT tokens with the K
// rows of the window in registers, so that every row is loaded once a run
// (plus K-1 rows before it, and behind it in the backward pass, which the
// neighbouring run has just read).  The next U tokens' rows are in flight
// while the present ones are computed.  Sequence borders are met on the way:
// at a border the window is filled from the state instead.
// Measured, K = 4, bf16, inputs from HBM: forward 16384 tokens x 8192 channels
// 124 us (4.3 TB/s; a large copy 5.15), gradients of 8192 x 8192 95 us
// (4.2 TB/s), one token of 8192 channels 3.1 us.  Rows that are not 16-byte aligned
// run single elements here, which is this kernel's choice (the loads themselves need
// only the element's alignment): fp32 gradients of 8191 x 2049, K = 3, 68 us (3.0 TB/s).
#include "seq_common.h"
#include "seq_plan.h"

namespace dw {
namespace {

// Tokens in flight: single elements (rows that are not aligned) need more to
// keep as many bytes on their way (fp32 gradients of 8191 x 2049: 70 us with
// four, 68 with eight).
__host__ __device__ constexpr int in_flight(int vec) { return vec == 1 ? 8 : 4; }

struct Geo {
    Packed seq;
    int C, TT;
    uint32_t ncv;  // channel vectors
    uint32_t main_blocks;
};

template <class DT, int VEC>
__device__ __forceinline__ void zero(float (&a)[VEC]) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) a[i] = 0.0f;
}

// The K-1 rows of ext in front of token t of the sequence that begins at a:
// win[j] = ext row (t - a) + j, from x where the sequence has begun by then.
template <class DT, int VEC, int K>
__device__ __forceinline__ void fill_window(float (&win)[K][VEC], const typename DT::X *x, int64_t ldx,
                                            const typename DT::X *state, int C, int a, int t) {
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
        const int e = t - a + j;  // row of ext
        if (e >= K - 1)
            load_f32<DT, VEC>(win[j], x + (int64_t)(a + e - (K - 1)) * ldx);
        else if (state)
            load_f32<DT, VEC>(win[j], state + (int64_t)e * C);
        else
            zero<DT, VEC>(win[j]);
    }
}

template <class DT, int VEC, int K>
__global__ void __launch_bounds__(256) k_fwd(Geo G, const typename DT::X *x, int64_t ldx, const typename DT::X *w,
                                             const float *bias, const typename DT::X *state_in,
                                             typename DT::X *state_out, typename DT::X *y, int64_t ldy, int silu) {
    using X = typename DT::X;
    constexpr int U = in_flight(VEC);
    const Packed &P = G.seq;
    if (blockIdx.x >= G.main_blocks) {  // the last K-1 rows of every sequence
        const uint64_t i = (uint64_t)(blockIdx.x - G.main_blocks) * 256 + threadIdx.x;
        const uint64_t row = i / G.ncv;
        if (row >= (uint64_t)P.seqs * (K - 1)) return;
        const int s = (int)(row / (K - 1)), r = (int)(row % (K - 1)), c = (int)(i % G.ncv) * VEC;
        const int a = P.begin(s), e = P.end(s) - a + r;
        Vec<X, VEC> v;
        if (e >= K - 1) {
            v = *(const Vec<X, VEC> *)(x + (int64_t)(a + e - (K - 1)) * ldx + c);
        } else if (state_in) {
            v = *(const Vec<X, VEC> *)(state_in + ((int64_t)s * (K - 1) + e) * G.C + c);
        } else {
#pragma unroll
            for (int j = 0; j < VEC; ++j) v.v[j] = (X)0;
        }
        *(Vec<X, VEC> *)(state_out + (int64_t)row * G.C + c) = v;
        return;
    }
    const uint64_t idx = (uint64_t)xcd_remap(blockIdx.x, G.main_blocks) * 256 + threadIdx.x;
    const uint64_t tile = idx / G.ncv;
    const int c = (int)(idx % G.ncv) * VEC;
    if (tile * G.TT >= (uint64_t)P.tokens) return;
    int t = (int)(tile * G.TT);
    int s = P.find(t);
    if (s < 0) return;
    int a = P.begin(s), b = P.end(s);
    const int stop = P.tokens - t < G.TT ? P.tokens : t + G.TT;
    x += c;
    float wt[K][VEC], bi[VEC], win[K][VEC];
#pragma unroll
    for (int k = 0; k < K; ++k) load_f32<DT, VEC>(wt[k], w + (int64_t)k * G.C + c);
    if (bias) load_f32<F32, VEC>(bi, bias + c); else zero<DT, VEC>(bi);
    const X *st = state_in ? state_in + (int64_t)s * (K - 1) * G.C + c : nullptr;
    fill_window<DT, VEC, K>(win, x, ldx, st, G.C, a, t);
    Vec<X, VEC> now[U], next[U];
#pragma unroll
    for (int u = 0; u < U; ++u) now[u] = *(const Vec<X, VEC> *)(x + (int64_t)min(t + u, stop - 1) * ldx);
    for (; t < stop; t += U) {
#pragma unroll
        for (int u = 0; u < U; ++u) next[u] = *(const Vec<X, VEC> *)(x + (int64_t)min(t + U + u, stop - 1) * ldx);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int tt = t + u;
            if (tt >= stop) break;
            if (tt >= b) {  // the next sequence that holds a token
                P.advance(tt, s, a, b);
                if (tt < a || tt >= b) return;  // behind the last sequence
                const X *sn = state_in ? state_in + (int64_t)s * (K - 1) * G.C + c : nullptr;
                fill_window<DT, VEC, K>(win, x, ldx, sn, G.C, a, tt);
            }
            float z[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                win[K - 1][i] = DT::widen(now[u].v[i]);
                z[i] = bi[i];
#pragma unroll
                for (int k = 0; k < K; ++k) z[i] = __builtin_fmaf(wt[k][i], win[k][i], z[i]);
                if (silu) z[i] *= sigmoid_f32<DT>(z[i]);
#pragma unroll
                for (int k = 0; k + 1 < K; ++k) win[k][i] = win[k + 1][i];
            }
            store_f32<DT, VEC>(y + (int64_t)tt * ldy + c, z);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) now[u] = next[u];
    }
}

template <class DT, int VEC, int K>
__global__ void __launch_bounds__(256) k_step(int C, uint32_t ncv, uint32_t cblocks, const typename DT::X *x,
                                              int64_t ldx, const typename DT::X *w, const float *bias,
                                              typename DT::X *state, const int32_t *slots, int n_slots, int rows,
                                              typename DT::X *y, int64_t ldy, int silu) {
    using X = typename DT::X;
    const int row = blockIdx.x / cblocks;
    const uint32_t cv = (blockIdx.x % cblocks) * 256 + threadIdx.x;
    const SlotRows sr = slot_rows(slots, n_slots, rows, row);
    if (sr.slot < 0 || cv >= ncv) return;
    const int c = (int)cv * VEC;
    float wt[K][VEC], bi[VEC], win[K][VEC];
    X *st = state + (int64_t)sr.slot * (K - 1) * C + c;
#pragma unroll
    for (int j = 0; j + 1 < K; ++j) load_f32<DT, VEC>(win[j], st + (int64_t)j * C);
#pragma unroll
    for (int k = 0; k < K; ++k) load_f32<DT, VEC>(wt[k], w + (int64_t)k * C + c);
    if (bias) load_f32<F32, VEC>(bi, bias + c); else zero<DT, VEC>(bi);
    for (int i = row; i < rows; ++i) {
        if (i != row && slots[i] != sr.slot) continue;
        load_f32<DT, VEC>(win[K - 1], x + (int64_t)i * ldx + c);
        float z[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            z[e] = bi[e];
#pragma unroll
            for (int k = 0; k < K; ++k) z[e] = __builtin_fmaf(wt[k][e], win[k][e], z[e]);
            if (silu) z[e] *= sigmoid_f32<DT>(z[e]);
#pragma unroll
            for (int k = 0; k + 1 < K; ++k) win[k][e] = win[k + 1][e];
        }
        store_f32<DT, VEC>(y + (int64_t)i * ldy + c, z);
        if (!sr.shared) break;
    }
    // element values pass through unchanged: widening and narrowing are exact
#pragma unroll
    for (int j = 0; j + 1 < K; ++j) store_f32<DT, VEC>(st + (int64_t)j * C, win[j]);
}

template <class DT>
__device__ __forceinline__ float silu_slope(float z) {
    float q;
    const float p = sigmoid_f32<DT>(z, q);
    return p * (1.0f + z * q);
}

// dstate_in: ext row e < K-1 gets shares from tokens 0 .. e, and is row e - L
// of the state behind a sequence of L <= e tokens.
template <class DT, int VEC, int K>
__device__ __forceinline__ void state_gradient(const Geo &G, uint64_t i, const typename DT::X *x, int64_t ldx,
                                               const typename DT::X *w, const float *bias,
                                               const typename DT::X *state_in, const typename DT::X *dy, int64_t lddy,
                                               const typename DT::X *dstate_out, typename DT::X *dstate_in, int silu) {
    const Packed &P = G.seq;
    const uint64_t row = i / G.ncv;
    if (row >= (uint64_t)P.seqs * (K - 1)) return;
    const int s = (int)(row / (K - 1)), e = (int)(row % (K - 1)), c = (int)(i % G.ncv) * VEC;
    const int a = P.begin(s), L = P.end(s) - a;
    const typename DT::X *st = state_in ? state_in + (int64_t)s * (K - 1) * G.C + c : nullptr;
    float sum[VEC];
    if (dstate_out && e >= L)
        load_f32<DT, VEC>(sum, dstate_out + ((int64_t)s * (K - 1) + (e - L)) * G.C + c);
    else
        zero<DT, VEC>(sum);
    for (int t = 0; t <= e && t < L; ++t) {
        float win[K][VEC], z[VEC], d[VEC], wt[VEC];
        fill_window<DT, VEC, K>(win, x + c, ldx, st, G.C, a, a + t);
        load_f32<DT, VEC>(win[K - 1], x + c + (int64_t)(a + t) * ldx);
        load_f32<DT, VEC>(d, dy + c + (int64_t)(a + t) * lddy);
        if (silu) {
            if (bias) load_f32<F32, VEC>(z, bias + c); else zero<DT, VEC>(z);
#pragma unroll
            for (int k = 0; k < K; ++k) {
                load_f32<DT, VEC>(wt, w + (int64_t)k * G.C + c);
#pragma unroll
                for (int j = 0; j < VEC; ++j) z[j] = __builtin_fmaf(wt[j], win[k][j], z[j]);
            }
#pragma unroll
            for (int j = 0; j < VEC; ++j) d[j] *= silu_slope<DT>(z[j]);
        }
        load_f32<DT, VEC>(wt, w + (int64_t)(e - t) * G.C + c);
#pragma unroll
        for (int j = 0; j < VEC; ++j) sum[j] = __builtin_fmaf(wt[j], d[j], sum[j]);
    }
    store_f32<DT, VEC>(dstate_in + (int64_t)row * G.C + c, sum);
}

// dx, and this run's sums for dw and dbias.  Token t's dz = dy act'(z) goes to
// the K rows of ext that z read; acc[k] holds the row K-1-k tokens back, which
// is complete once token t has given its share.  The run continues K-1 tokens
// past its end (or to the end of the sequence) for the rows it still owes.
template <class DT, int VEC, int K>
__global__ void __launch_bounds__(256) k_bwd(Geo G, const typename DT::X *x, int64_t ldx, const typename DT::X *w,
                                             const float *bias, const typename DT::X *state_in,
                                             const typename DT::X *dy, int64_t lddy,
                                             const typename DT::X *dstate_out, typename DT::X *dx, int64_t lddx,
                                             typename DT::X *dstate_in, float *part, int silu) {
    using X = typename DT::X;
    constexpr int U = in_flight(VEC);
    const Packed &P = G.seq;
    if (blockIdx.x >= G.main_blocks) {
        state_gradient<DT, VEC, K>(G, (uint64_t)(blockIdx.x - G.main_blocks) * 256 + threadIdx.x, x, ldx, w, bias,
                                   state_in, dy, lddy, dstate_out, dstate_in, silu);
        return;
    }
    const uint64_t idx = (uint64_t)xcd_remap(blockIdx.x, G.main_blocks) * 256 + threadIdx.x;
    const uint64_t tile = idx / G.ncv;
    const int c = (int)(idx % G.ncv) * VEC;
    if (tile * G.TT >= (uint64_t)P.tokens) return;
    const int t0 = (int)(tile * G.TT);
    const int t1 = P.tokens - t0 < G.TT ? P.tokens : t0 + G.TT;  // end of the run
    const int t2 = P.tokens - t1 < K - 1 ? P.tokens : t1 + K - 1;
    float gw[K][VEC], gb[VEC];
    zero<DT, VEC>(gb);
#pragma unroll
    for (int k = 0; k < K; ++k) zero<DT, VEC>(gw[k]);
    int s = P.find(t0);
    int a = 0, b = 0;
    if (s >= 0) a = P.begin(s), b = P.end(s);
    if (s >= 0 && t0 < b) {
        x += c;
        dy += c;
        dx += c;
        float wt[K][VEC], bi[VEC], win[K][VEC], acc[K][VEC];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            load_f32<DT, VEC>(wt[k], w + (int64_t)k * G.C + c);
            zero<DT, VEC>(acc[k]);
        }
        if (bias) load_f32<F32, VEC>(bi, bias + c); else zero<DT, VEC>(bi);
        fill_window<DT, VEC, K>(win, x, ldx, state_in ? state_in + (int64_t)s * (K - 1) * G.C + c : nullptr, G.C, a, t0);
        // the rows of the last K-1 tokens before `end` get no more shares,
        // except from the gradient of the state that they are
        auto flush = [&](int end) {
#pragma unroll
            for (int j = 1; j < K; ++j) {  // after the shift acc[j-1] holds token end-K+j
                const int tok = end - K + j;
                if (tok >= t0 && tok < t1 && tok >= a) {
                    float v[VEC];
#pragma unroll
                    for (int i = 0; i < VEC; ++i) v[i] = acc[j - 1][i];
                    if (dstate_out) {
                        float d[VEC];
                        // ext row tok - a + K-1 is row tok + K-1 - end of the state
                        load_f32<DT, VEC>(d, dstate_out + ((int64_t)s * (K - 1) + (tok + K - 1 - end)) * G.C + c);
#pragma unroll
                        for (int i = 0; i < VEC; ++i) v[i] += d[i];
                    }
                    store_f32<DT, VEC>(dx + (int64_t)tok * lddx, v);
                }
            }
#pragma unroll
            for (int k = 0; k < K; ++k) zero<DT, VEC>(acc[k]);
        };
        Vec<X, VEC> xn[U], dn[U], x1[U], d1[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            xn[u] = *(const Vec<X, VEC> *)(x + (int64_t)min(t0 + u, t2 - 1) * ldx);
            dn[u] = *(const Vec<X, VEC> *)(dy + (int64_t)min(t0 + u, t2 - 1) * lddy);
        }
        bool live = true;
        int t = t0;
        while (live && t < t2) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                x1[u] = *(const Vec<X, VEC> *)(x + (int64_t)min(t + U + u, t2 - 1) * ldx);
                d1[u] = *(const Vec<X, VEC> *)(dy + (int64_t)min(t + U + u, t2 - 1) * lddy);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int tt = t + u;
                if (!live || tt >= t2) break;
                if (tt >= b) {
                    flush(b);
                    live = tt < t1;
                    if (!live) break;
                    P.advance(tt, s, a, b);
                    live = tt >= a && tt < b;
                    if (!live) break;
                    fill_window<DT, VEC, K>(win, x, ldx, state_in ? state_in + (int64_t)s * (K - 1) * G.C + c : nullptr,
                                            G.C, a, tt);
                }
                const bool own = tt < t1;
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    win[K - 1][i] = DT::widen(xn[u].v[i]);
                    float d = DT::widen(dn[u].v[i]);
                    if (silu) {
                        float z = bi[i];
#pragma unroll
                        for (int k = 0; k < K; ++k) z = __builtin_fmaf(wt[k][i], win[k][i], z);
                        d *= silu_slope<DT>(z);
                    }
#pragma unroll
                    for (int k = 0; k < K; ++k) acc[k][i] = __builtin_fmaf(wt[k][i], d, acc[k][i]);
                    if (own) {
                        gb[i] += d;
#pragma unroll
                        for (int k = 0; k < K; ++k) gw[k][i] = __builtin_fmaf(d, win[k][i], gw[k][i]);
                    }
#pragma unroll
                    for (int k = 0; k + 1 < K; ++k) win[k][i] = win[k + 1][i];
                }
                const int tok = tt - (K - 1);
                if (tok >= t0 && tok >= a) store_f32<DT, VEC>(dx + (int64_t)tok * lddx, acc[0]);
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
#pragma unroll
                    for (int k = 0; k + 1 < K; ++k) acc[k][i] = acc[k + 1][i];
                    acc[K - 1][i] = 0.0f;
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) xn[u] = x1[u], dn[u] = d1[u];
            t += U;
        }
        if (live && t2 >= b) flush(b);
    }
    float *o = part + (int64_t)tile * (K + 1) * G.C + c;
#pragma unroll
    for (int k = 0; k < K; ++k) store_f32<F32, VEC>(o + (int64_t)k * G.C, gw[k]);
    store_f32<F32, VEC>(o + (int64_t)K * G.C, gb);
}

// Sum of the runs' rows: 64 columns a workgroup, four waves take every fourth
// run and their sums are added in wave order.
__global__ void __launch_bounds__(256) k_sum(const float *part, int64_t runs, int C, int K, float *dw, float *dbias) {
    __shared__ float sh[4][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t col = (int64_t)blockIdx.x * 64 + lane, n = (int64_t)(K + 1) * C;
    float s0 = 0.0f, s1 = 0.0f, s2 = 0.0f, s3 = 0.0f;
    if (col < n) {
        int64_t r = wave;
        for (; r + 12 < runs; r += 16) {
            s0 += part[r * n + col];
            s1 += part[(r + 4) * n + col];
            s2 += part[(r + 8) * n + col];
            s3 += part[(r + 12) * n + col];
        }
        for (; r < runs; r += 4) s0 += part[r * n + col];
    }
    sh[wave][lane] = (s0 + s1) + (s2 + s3);
    __syncthreads();
    if (wave || col >= n) return;
    const float s = (sh[0][lane] + sh[1][lane]) + (sh[2][lane] + sh[3][lane]);
    if (col < (int64_t)K * C) dw[col] = s;
    else if (dbias) dbias[col - (int64_t)K * C] = s;
}

// Tokens a lane walks: long runs spend less on the rows around them (and on
// the run's sums in the backward pass); short ones give the chip enough waves.
// bf16, K = 4, inputs from HBM, runs of 8 and of 64 tokens: forward 136 and 125 us
// at 16384 tokens x 8192 channels, 15 and 36 us at 4096 x 2048; backward with its
// sums 195 and 100 us at 8192 x 8192, 35 and 63 us at 4096 x 2048.  The backward
// pass, which writes sums for every run, stops at half the lanes (4096 x 2048,
// runs of 8 and 16 tokens: 35 and 32 us; forward 15 and 17 us).
int run_tokens(int tokens, int C, int vec, bool back) {
    int tt = 64;
    const int64_t ncv = (C + vec - 1) / vec, lanes = back ? 65536 : 131072;
    while (tt > 8 && (int64_t)((tokens + tt - 1) / tt) * ncv < lanes) tt /= 2;
    return tt;
}

// Elements a lane moves at once: 16 bytes, 8 bytes for filters of more than
// four taps (registers), one element where rows or pointers are not aligned.
int vec_of(const dwconv_causal_plan &p) {
    const int e = p.dtype == DWCONV_F32 ? 4 : 2;
    return (p.K <= 4 ? 16 : 8) / e;
}

struct Align {
    uintptr_t bits = 0;
    void add(const void *p) { bits |= (uintptr_t)p; }
    void stride(int64_t ld, int e) { bits |= (uintptr_t)(ld * e); }
    bool ok(int bytes) const { return (bits & (uintptr_t)(bytes - 1)) == 0; }
};

uint64_t blocks_of(uint64_t n) { return (n + 255) / 256; }
// a grid holds fewer than 2^32 lanes
bool too_many(uint64_t blocks) { return blocks >= (1u << 24); }

template <class DT, int VEC, int K>
hipError_t fwd(const dwconv_causal_plan &p, const CausalArgs &a, hipStream_t st) {
    using X = typename DT::X;
    Geo G{{a.offsets, a.seqs, a.tokens}, p.C, run_tokens(a.tokens, p.C, VEC, false), (uint32_t)(p.C / VEC), 0};
    const uint64_t tiles = ((uint64_t)a.tokens + G.TT - 1) / G.TT;
    const uint64_t blocks = blocks_of(tiles * G.ncv);
    const uint64_t extra = a.state_out ? blocks_of((uint64_t)a.seqs * (K - 1) * G.ncv) : 0;
    if (blocks + extra == 0) return hipSuccess;
    if (too_many(blocks + extra)) return hipErrorInvalidConfiguration;
    G.main_blocks = (uint32_t)blocks;
    k_fwd<DT, VEC, K><<<(uint32_t)(blocks + extra), 256, 0, st>>>(G, (const X *)a.x, a.ldx, (const X *)a.w, a.bias,
                                                             (const X *)a.state_in, (X *)a.state_out, (X *)a.y,
                                                             a.ldy, p.act == DWCONV_SEQ_ACT_SILU);
    return hipGetLastError();
}

template <class DT, int VEC, int K>
hipError_t step(const dwconv_causal_plan &p, const CausalArgs &a, hipStream_t st) {
    using X = typename DT::X;
    const uint32_t ncv = p.C / VEC, cb = (uint32_t)blocks_of(ncv);
    if (a.tokens == 0) return hipSuccess;
    if (too_many((uint64_t)cb * (uint32_t)a.tokens)) return hipErrorInvalidConfiguration;
    k_step<DT, VEC, K><<<cb * (uint32_t)a.tokens, 256, 0, st>>>(p.C, ncv, cb, (const X *)a.x, a.ldx, (const X *)a.w,
                                                                a.bias, (X *)a.state, a.slots, a.n_slots, a.tokens,
                                                                (X *)a.y, a.ldy, p.act == DWCONV_SEQ_ACT_SILU);
    return hipGetLastError();
}

template <class DT, int VEC, int K>
hipError_t bwd(const dwconv_causal_plan &p, const CausalArgs &a, hipStream_t st) {
    using X = typename DT::X;
    const int silu = p.act == DWCONV_SEQ_ACT_SILU;
    // the run length of the widest vectors, whatever width runs: the
    // workspace's size does not depend on alignment
    Geo G{{a.offsets, a.seqs, a.tokens}, p.C, run_tokens(a.tokens, p.C, vec_of(p), true), (uint32_t)(p.C / VEC), 0};
    const uint64_t tiles = ((uint64_t)a.tokens + G.TT - 1) / G.TT;
    const uint64_t blocks = blocks_of(tiles * G.ncv);
    const uint64_t sb = a.dstate_in ? blocks_of((uint64_t)a.seqs * (K - 1) * G.ncv) : 0;
    const uint64_t cols = ((uint64_t)(K + 1) * p.C + 63) / 64;
    if (too_many(blocks + sb) || too_many(cols)) return hipErrorInvalidConfiguration;
    G.main_blocks = (uint32_t)blocks;
    if (blocks + sb)
        k_bwd<DT, VEC, K><<<(uint32_t)(blocks + sb), 256, 0, st>>>(
            G, (const X *)a.x, a.ldx, (const X *)a.w, a.bias, (const X *)a.state_in, (const X *)a.dy, a.lddy,
            (const X *)a.dstate_out, (X *)a.dx, a.lddx, (X *)a.dstate_in, a.workspace, silu);
    k_sum<<<(uint32_t)cols, 256, 0, st>>>(a.workspace, (int64_t)tiles, p.C, K, a.dw, a.dbias);
    return hipGetLastError();
}

enum Pass { FWD, STEP, BWD };

template <class DT, int VEC, int K>
hipError_t go(Pass pass, const dwconv_causal_plan &p, const CausalArgs &a, hipStream_t st) {
    return pass == FWD ? fwd<DT, VEC, K>(p, a, st) : pass == STEP ? step<DT, VEC, K>(p, a, st) : bwd<DT, VEC, K>(p, a, st);
}

template <class DT, int K>
hipError_t pick_vec(Pass pass, const dwconv_causal_plan &p, const CausalArgs &a, hipStream_t st) {
    constexpr int E = (int)sizeof(typename DT::X), V = (K <= 4 ? 16 : 8) / E;
    Align al, al32;
    const void *ptrs[] = {a.x, a.w, a.y, a.state_in, a.state_out, a.state, a.dy, a.dstate_out, a.dx, a.dstate_in};
    for (const void *q : ptrs) al.add(q);
    const int64_t lds[] = {a.ldx, a.ldy, a.lddy, a.lddx, (int64_t)p.C};
    for (int64_t l : lds) al.stride(l, E);
    al32.add(a.bias);
    al32.add(a.workspace);
    if (al.ok(V * E) && al32.ok(V == 2 ? 8 : 16)) return go<DT, V, K>(pass, p, a, st);
    return go<DT, 1, K>(pass, p, a, st);
}

template <class DT>
hipError_t pick_k(Pass pass, const dwconv_causal_plan &p, const CausalArgs &a, hipStream_t st) {
    switch (p.K) {
        case 2: return pick_vec<DT, 2>(pass, p, a, st);
        case 3: return pick_vec<DT, 3>(pass, p, a, st);
        case 4: return pick_vec<DT, 4>(pass, p, a, st);
        case 5: return pick_vec<DT, 5>(pass, p, a, st);
        case 6: return pick_vec<DT, 6>(pass, p, a, st);
        case 7: return pick_vec<DT, 7>(pass, p, a, st);
        default: return pick_vec<DT, 8>(pass, p, a, st);
    }
}

hipError_t pick(Pass pass, const dwconv_causal_plan &p, const CausalArgs &a, hipStream_t st) {
    switch (p.dtype) {
        case DWCONV_F32: return pick_k<F32>(pass, p, a, st);
        case DWCONV_F16: return pick_k<F16>(pass, p, a, st);
        default: return pick_k<BF16>(pass, p, a, st);
    }
}

}  // namespace

hipError_t causal_fwd(const dwconv_causal_plan &p, const CausalArgs &a, hipStream_t st) { return pick(FWD, p, a, st); }
hipError_t causal_step(const dwconv_causal_plan &p, const CausalArgs &a, hipStream_t st) { return pick(STEP, p, a, st); }
hipError_t causal_bwd(const dwconv_causal_plan &p, const CausalArgs &a, hipStream_t st) { return pick(BWD, p, a, st); }

size_t causal_bwd_bytes(const dwconv_causal_plan &p, int tokens) {
    const int tt = run_tokens(tokens, p.C, vec_of(p), true);
    return ((size_t)tokens + tt - 1) / tt * (size_t)(p.K + 1) * p.C * sizeof(float);
}

}  // namespace dw
