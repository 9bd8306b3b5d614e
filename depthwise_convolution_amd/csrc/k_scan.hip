// k_scan.hip -- selective scan of packed sequences (include/dwconv_seq.h):
// forward and gradients.
//
//   d = softplus(dt + bias)    h = e^(d a) h + d x b    y = (sum_n h c + skip x) act(gate)
//
// A workgroup walks the tokens of one piece of a sequence for 256 / LPC channels; a
// channel's states lie in LPC lanes, four each, so that what four tokens need once a
// channel (step width, gate, the sum's last digits) is done by the four lanes of a
// quad, a token each, and handed round by lane permutations inside the arithmetic.
// Tiles of 16 tokens pass through LDS: rows of channels come in and go out as whole
// vectors, b and c of all states once a workgroup.
//
// Pieces: whole sequences where those fill the chip, else runs of CH tokens, which
// takes a pass before (k_ends: what a run makes of a zero state, and how far its
// tokens fade) and a walk over the runs (k_join) that gives every run its first state.
//
// Gradients, with G the gradient of the state after a token:
//   G += c dy     dc = sum_channels dy h     db = sum_channels d x G
//   du = sum_n G b     G *= e^(d a)     dd = sum_n G h_before a + x du     da += d G h_before
// walk back over blocks of 16 tokens whose first states a walk forward has left in the
// workspace; a block's states and decays are formed again and stay in registers.
#include "seq_common.h"
#include "seq_plan.h"
#include "scan_common.h"

namespace dw {
namespace {

constexpr int TT = 16;         // tokens a tile, and between two kept states
constexpr int THREADS = 256;
// ---------------------------------------------------------------------------
// lanes
// ---------------------------------------------------------------------------
// Sums over the channels of a wavefront of V = 16 values (LPC 4) or 8 a lane: halves
// the values as it doubles the lanes summed, so that each lane ends with R of them.
// Which ones: value index i = first half or second half by lane bit, highest first.
template <int LPC>
struct Across {
    static constexpr int V = LPC == 4 ? 16 : 8;        // values that go in: tokens x (b, c) x 4 states
    static constexpr int TOK = V / 8;                  // of so many tokens
    static constexpr int R = V * LPC / 64;             // values a lane keeps
    static __device__ __forceinline__ void sum(float (&v)[V], int lane) {
        int n = V;
        if (LPC <= 8) {  // lane bit 3
            const bool hi = lane & 8;
            n /= 2;
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                const float m = hi ? v[i + V / 2] : v[i], o = hi ? v[i] : v[i + V / 2];
                v[i] = m + dpp<0x128>(o);  // lane ^ 8
            }
        }
        if (LPC <= 4) {  // lane bit 2
            const bool hi = lane & 4;
#pragma unroll
            for (int i = 0; i < V / 4; ++i) {
                float m = hi ? v[i + V / 4] : v[i];
                m += dpp_banks<0x104, 0x5>(v[i]);           // from four lanes on, in quads 0 and 2
                v[i] = m + dpp_banks<0x114, 0xa>(v[i + V / 4]);  // from four lanes back, in quads 1 and 3
            }
            n /= 2;
        }
        if (LPC <= 16) {  // lane bit 4
            n /= 2;
#pragma unroll
            for (int i = 0; i < V / 2; ++i)
                if (i < n) {
                    swap16(v[i], v[i + n]);
                    v[i] += v[i + n];
                }
        }
        n /= 2;  // lane bit 5
#pragma unroll
        for (int i = 0; i < V / 2; ++i)
            if (i < n) {
                swap32(v[i], v[i + n]);
                v[i] += v[i + n];
            }
    }
    // index of the value that ends in v[0] of this lane; v[r] is r after it
    static __device__ __forceinline__ int first(int lane) {
        int at = 0, n = V;
        if (LPC <= 8) n /= 2, at += lane & 8 ? n : 0;
        if (LPC <= 4) n /= 2, at += lane & 4 ? n : 0;
        if (LPC <= 16) n /= 2, at += lane & 16 ? n : 0;
        n /= 2;
        return at + (lane & 32 ? n : 0);
    }
};

// ---------------------------------------------------------------------------
// geometry
// ---------------------------------------------------------------------------
// A run of piece `slot`: [t0, t1) of sequence s.  The pieces of sequence s have the
// slots begin / CH + s and up: no table, and no two alike.
struct Piece {
    int s, t0, t1;
    bool last;
};
__device__ __forceinline__ int64_t slot_base(const ScanGeo &G, int s) { return G.CH ? (int64_t)(G.seq.begin(s) / G.CH) + s : s; }
__device__ __forceinline__ Piece piece(const ScanGeo &G, int64_t slot) {
    if (!G.CH) {
        const int s = (int)slot;
        return {s, G.seq.begin(s), G.seq.end(s), true};
    }
    int lo = 0, hi = G.seq.seqs;
    while (hi - lo > 1) {
        const int m = lo + ((hi - lo) >> 1);
        if (slot_base(G, m) <= slot) lo = m; else hi = m;
    }
    const int b = G.seq.begin(lo), e = G.seq.end(lo);
    const int64_t t = b + (slot - slot_base(G, lo)) * G.CH;
    if (t < b || t >= e) return {lo, e, e, false};
    return {lo, (int)t, e - t > G.CH ? (int)t + G.CH : e, e - t <= G.CH};
}

// ---------------------------------------------------------------------------
// tiles
// ---------------------------------------------------------------------------
// 16 tokens of the workgroup's channels, a vector of four a lane.  The vectors need
// no more than the element's alignment: the loads take any.
template <class DT, int LPC>
struct Rows {
    using X = typename DT::X;
    struct __attribute__((packed, aligned(sizeof(X)))) Any {
        X v[4];
    };
    static constexpr int CPW = THREADS / LPC, VPR = CPW / 4, LD = CPW + 16;
    static constexpr int SIZE = TT * LD;
    Vec<X, 4> v;
    static __device__ __forceinline__ int row() { return (int)threadIdx.x / VPR; }
    static __device__ __forceinline__ int col() { return (int)threadIdx.x % VPR * 4; }
    __device__ __forceinline__ void fetch(const X *p, int64_t ld, int t, int cnt, int c0, int cend) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v.v[i] = (X)0;
        const int c = c0 + col();
        if (row() >= cnt || c >= cend) return;
        const X *at = p + (int64_t)(t + row()) * ld + c;
        if (c + 4 <= cend) {
            const Any a = *(const Any *)at;
#pragma unroll
            for (int i = 0; i < 4; ++i) v.v[i] = a.v[i];
        } else {
#pragma unroll
            for (int i = 0; i < 3; ++i)
                if (c + i < cend) v.v[i] = at[i];
        }
    }
    __device__ __forceinline__ void put(X *lds) const {
        if (row() < TT) *(Vec<X, 4> *)(lds + row() * LD + col()) = v;
    }
    static __device__ __forceinline__ void flush(const X *lds, X *p, int64_t ld, int t, int cnt, int c0, int cend) {
        const int c = c0 + col();
        if (row() >= cnt || c >= cend) return;
        const Vec<X, 4> w = *(const Vec<X, 4> *)(lds + row() * LD + col());
        X *at = p + (int64_t)(t + row()) * ld + c;
        if (c + 4 <= cend) {
            Any a;
#pragma unroll
            for (int i = 0; i < 4; ++i) a.v[i] = w.v[i];
            *(Any *)at = a;
        } else {
#pragma unroll
            for (int i = 0; i < 3; ++i)
                if (c + i < cend) at[i] = w.v[i];
        }
    }
    static __device__ __forceinline__ float get(const X *lds, int tok, int ch) { return DT::widen(lds[tok * LD + ch]); }
    static __device__ __forceinline__ void set(X *lds, int tok, int ch, float v) { lds[tok * LD + ch] = rounded<DT>(v); }
};

// b or c of 16 tokens, fp32, states past N zero
template <class DT, int LPC>
struct Shared {
    using X = typename DT::X;
    static constexpr int NP = 4 * LPC, PT = TT * NP / THREADS, SIZE = TT * NP;
    X v[PT];
    __device__ __forceinline__ void fetch(const X *p, int64_t ld, int t, int cnt, int n0, int N) {
#pragma unroll
        for (int k = 0; k < PT; ++k) {
            const int i = (int)threadIdx.x + k * THREADS, n = i % NP, r = i / NP;
            v[k] = r < cnt && n < N ? p[(int64_t)(t + r) * ld + n0 + n] : (X)0;
        }
    }
    __device__ __forceinline__ void put(float *lds) const {
#pragma unroll
        for (int k = 0; k < PT; ++k) lds[threadIdx.x + k * THREADS] = DT::widen(v[k]);
    }
    static __device__ __forceinline__ void get(float (&o)[4], const float *lds, int tok, int j) {
        load_f32<F32, 4>(o, lds + tok * NP + 4 * j);
    }
};

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------
template <class DT, int LPC>
__global__ void __launch_bounds__(THREADS)
    k_out(ScanGeo G, ScanIn in, const float *state_in, const float *starts, float *state_out, typename DT::X *y, int64_t ldy) {
    using X = typename DT::X;
    using R = Rows<DT, LPC>;
    using S = Shared<DT, LPC>;
    __shared__ __align__(16) X sx[2][R::SIZE], sd[2][R::SIZE], sz[2][R::SIZE], sy[2][R::SIZE];
    __shared__ __align__(16) float sb[2][S::SIZE], sc[2][S::SIZE];
    const uint32_t id = xcd_remap(blockIdx.x, gridDim.x);
    const ScanLane<LPC> w(G, id % G.nblk);
    const uint32_t slot = id / G.nblk;
    const Piece p = piece(G, slot);
    if (G.CH && p.t0 >= p.t1) return;
    float a2[4], h[4];
    load_rates(a2, in.a, G, w.c, 4 * w.j, w.live);
    const int64_t srow = ((int64_t)p.s * G.C + (w.live ? w.c : 0)) * G.N;
    if (starts) load_f32<F32, 4>(h, starts + ((int64_t)id * THREADS + threadIdx.x) * 4);
    else load_states(h, state_in ? state_in + srow : nullptr, 4 * w.j, G.N, w.live && state_in);
    const float bias = in.bias && w.live ? in.bias[w.c] : 0.0f, skip = in.skip && w.live ? in.skip[w.c] : 0.0f;
    R rx, rd, rz;
    S rb, rc;
    auto fetch = [&](int t) {
        const int cnt = min(TT, p.t1 - t);
        rx.fetch((const X *)in.x, in.ldx, t, cnt, w.c0, w.cend);
        rd.fetch((const X *)in.dt, in.lddt, t, cnt, w.c0, w.cend);
        if (in.gate) rz.fetch((const X *)in.gate, in.ldgate, t, cnt, w.c0, w.cend);
        rb.fetch((const X *)in.b, in.ldb, t, cnt, w.g * G.N, G.N);
        rc.fetch((const X *)in.c, in.ldc, t, cnt, w.g * G.N, G.N);
    };
    int k = 0;
    if (p.t0 < p.t1) fetch(p.t0);
    for (int t = p.t0; t < p.t1; t += TT, k ^= 1) {
        rx.put(sx[k]);
        rd.put(sd[k]);
        if (in.gate) rz.put(sz[k]);
        rb.put(sb[k]);
        rc.put(sc[k]);
        __syncthreads();  // the one barrier a tile: what a tile writes is read in its own turn or the next
        if (t > p.t0) R::flush(sy[k ^ 1], y, ldy, t - TT, TT, w.c0, w.cend);
        if (p.t1 - t > TT) fetch(t + TT);
        const int cnt = min(TT, p.t1 - t);
        for (int u = 0; u < cnt; u += 4) {
            const int own = u + w.q;
            const float xv = R::get(sx[k], own, w.ch);
            float slope;
            float d = step_width<DT>(R::get(sd[k], own, w.ch) + bias, G.soft, slope);
            d = own < cnt ? d : 0.0f;
            const float dx = d * xv;
            float yy = 0.0f;
            auto token = [&](int s, float ds, float us) {
                float bv[4], cv[4], v = 0.0f;
                S::get(bv, sb[k], u + s, w.j);
                S::get(cv, sc[k], u + s, w.j);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    h[i] = __builtin_fmaf(__builtin_amdgcn_exp2f(ds * a2[i]), h[i], us * bv[i]);
                    v = __builtin_fmaf(h[i], cv[i], v);
                }
                v = sum_states<LPC>(v);
                yy = w.q == s ? v : yy;
            };
            token(0, quad<0>(d), quad<0>(dx));
            token(1, quad<1>(d), quad<1>(dx));
            token(2, quad<2>(d), quad<2>(dx));
            token(3, quad<3>(d), quad<3>(dx));
            yy = __builtin_fmaf(skip, xv, yy);
            if (in.gate) yy *= gate_value<DT>(R::get(sz[k], own, w.ch), G.act);
            if (w.j < 4) R::set(sy[k], own, w.ch, yy);
        }
    }
    if (p.t0 < p.t1) {
        __syncthreads();
        const int t = p.t0 + (p.t1 - p.t0 - 1) / TT * TT;
        R::flush(sy[k ^ 1], y, ldy, t, p.t1 - t, w.c0, w.cend);
    }
    if (state_out && !starts) store_states(state_out + srow, h, 4 * w.j, G.N, w.live);
}

// What a run leaves of a zero state (ends), the sum of its step widths (width), and
// with BACK the gradient that its outputs leave at the state before it (back): there
// token t counts c dy times the decays of all tokens from the run's first to it.
template <class DT, int LPC, bool BACK>
__global__ void __launch_bounds__(THREADS) k_ends(ScanGeo G, ScanIn in, float *ends, float *width, float *back) {
    using X = typename DT::X;
    using R = Rows<DT, LPC>;
    using S = Shared<DT, LPC>;
    constexpr int B = BACK ? 1 : 0;
    __shared__ __align__(16) X sx[2][R::SIZE], sd[2][R::SIZE], sy[B + 1][B ? R::SIZE : 8], sz[B + 1][B ? R::SIZE : 8];
    __shared__ __align__(16) float sb[2][S::SIZE], sc[B + 1][B ? S::SIZE : 4];
    const uint32_t id = xcd_remap(blockIdx.x, gridDim.x);
    const ScanLane<LPC> w(G, id % G.nblk);
    const Piece p = piece(G, id / G.nblk);
    if (p.t0 >= p.t1) return;
    float a2[4], h[4], fade[4], g[4], sum = 0.0f;
    load_rates(a2, in.a, G, w.c, 4 * w.j, w.live);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = g[i] = 0.0f, fade[i] = 1.0f;
    const float bias = in.bias && w.live ? in.bias[w.c] : 0.0f;
    R rx, rd, ry, rz;
    S rb, rc;
    auto fetch = [&](int t) {
        const int cnt = min(TT, p.t1 - t);
        rx.fetch((const X *)in.x, in.ldx, t, cnt, w.c0, w.cend);
        rd.fetch((const X *)in.dt, in.lddt, t, cnt, w.c0, w.cend);
        rb.fetch((const X *)in.b, in.ldb, t, cnt, w.g * G.N, G.N);
        if (BACK) {
            ry.fetch((const X *)in.dy, in.lddy, t, cnt, w.c0, w.cend);
            if (in.gate) rz.fetch((const X *)in.gate, in.ldgate, t, cnt, w.c0, w.cend);
            rc.fetch((const X *)in.c, in.ldc, t, cnt, w.g * G.N, G.N);
        }
    };
    int k = 0;
    fetch(p.t0);
    for (int t = p.t0; t < p.t1; t += TT, k ^= 1) {
        rx.put(sx[k]);
        rd.put(sd[k]);
        rb.put(sb[k]);
        if (BACK) {
            ry.put(sy[k & B]);
            if (in.gate) rz.put(sz[k & B]);
            rc.put(sc[k & B]);
        }
        __syncthreads();
        if (p.t1 - t > TT) fetch(t + TT);
        const int cnt = min(TT, p.t1 - t);
        for (int u = 0; u < cnt; u += 4) {
            const int own = u + w.q;
            float slope, dy = 0.0f;
            float d = step_width<DT>(R::get(sd[k], own, w.ch) + bias, G.soft, slope);
            d = own < cnt ? d : 0.0f;
            sum += d;
            const float dx = d * R::get(sx[k], own, w.ch);
            if (BACK) {
                dy = R::get(sy[k & B], own, w.ch);
                if (in.gate) dy *= gate_value<DT>(R::get(sz[k & B], own, w.ch), G.act);
            }
            auto token = [&](int s, float ds, float us, float ys) {
                float bv[4], cv[4];
                S::get(bv, sb[k], u + s, w.j);
                if (BACK) S::get(cv, sc[k & B], u + s, w.j);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float e = __builtin_amdgcn_exp2f(ds * a2[i]);
                    h[i] = __builtin_fmaf(e, h[i], us * bv[i]);
                    if (BACK) {
                        fade[i] *= e;
                        g[i] = __builtin_fmaf(fade[i], cv[i] * ys, g[i]);
                    }
                }
            };
            token(0, quad<0>(d), quad<0>(dx), quad<0>(dy));
            token(1, quad<1>(d), quad<1>(dx), quad<1>(dy));
            token(2, quad<2>(d), quad<2>(dx), quad<2>(dy));
            token(3, quad<3>(d), quad<3>(dx), quad<3>(dy));
        }
    }
    const int64_t at = ((int64_t)id * THREADS + threadIdx.x) * 4;
    store_f32<F32, 4>(ends + at, h);
    if (BACK) store_f32<F32, 4>(back + at, g);
    sum += dpp<0xB1>(sum);
    sum += dpp<0x4E>(sum);
    if (w.j == 0) width[(int64_t)id * ScanLane<LPC>::CPW + w.ch] = sum;
}

// Walks the runs of a sequence: `ends` becomes the state before each run, `back` the
// gradient of the state after it.  Four runs are on their way at a time.
template <int LPC, bool BACK>
__global__ void __launch_bounds__(THREADS)
    k_join(ScanGeo G, const float *a, const float *state_in, float *state_out, const float *dstate_out, float *dstate_in,
           float *ends, const float *width, float *back) {
    constexpr int U = 4, CPW = ScanLane<LPC>::CPW;
    const uint32_t cb = blockIdx.x % G.nblk;
    const int s = (int)(blockIdx.x / G.nblk);
    const ScanLane<LPC> w(G, cb);
    float a2[4], v[4];
    load_rates(a2, a, G, w.c, 4 * w.j, w.live);
    const int64_t srow = ((int64_t)s * G.C + (w.live ? w.c : 0)) * G.N;
    const int64_t base = slot_base(G, s), runs = ((int64_t)G.seq.end(s) - G.seq.begin(s) + G.CH - 1) / G.CH;
    auto at = [&](int64_t r) { return ((base + r) * G.nblk + cb) * THREADS + threadIdx.x; };
    auto wide = [&](int64_t r) { return width[((base + r) * G.nblk + cb) * CPW + w.ch]; };
    auto walk = [&](float *p, bool down) {
        for (int64_t r = 0; r < runs; r += U) {
            float e[U][4], d[U];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int64_t n = r + i < runs ? r + i : runs - 1, m = down ? runs - 1 - n : n;
                load_f32<F32, 4>(e[i], p + at(m) * 4);
                d[i] = wide(m);
            }
#pragma unroll
            for (int i = 0; i < U; ++i) {
                if (r + i >= runs) break;
                store_f32<F32, 4>(p + at(down ? runs - 1 - (r + i) : r + i) * 4, v);
#pragma unroll
                for (int n = 0; n < 4; ++n) v[n] = __builtin_fmaf(__builtin_amdgcn_exp2f(d[i] * a2[n]), v[n], e[i][n]);
            }
        }
    };
    load_states(v, state_in ? state_in + srow : nullptr, 4 * w.j, G.N, w.live && state_in);
    walk(ends, false);
    if (state_out) store_states(state_out + srow, v, 4 * w.j, G.N, w.live);
    if (BACK) {
        load_states(v, dstate_out ? dstate_out + srow : nullptr, 4 * w.j, G.N, w.live && dstate_out);
        walk(back, true);
        if (dstate_in) store_states(dstate_in + srow, v, 4 * w.j, G.N, w.live);
    }
}

// ---------------------------------------------------------------------------
// gradients
// ---------------------------------------------------------------------------
struct Out {
    void *dx, *ddt, *dgate;
    int64_t lddx, ldddt, lddgate;
    float *kept;            // states before each block of 16 tokens
    float *part;            // channel blocks x tokens x 2 x NP: db, dc
    float *pa, *ps;         // walkers x channel blocks x (256 x 4: da; 2 x CPW: dskip, dbias)
};

template <class DT, int LPC>
__global__ void __launch_bounds__(THREADS, 2)
    k_grad(ScanGeo G, ScanIn in, Out o, const float *state_in, const float *dstate_out, float *dstate_in, const float *starts,
           const float *afters) {
    using X = typename DT::X;
    using R = Rows<DT, LPC>;
    using S = Shared<DT, LPC>;
    using A = Across<LPC>;
    constexpr int NP = 4 * LPC, CPW = THREADS / LPC;
    constexpr int ROUND = LPC <= 8 ? 16 : LPC == 16 ? 8 : 4;  // tokens whose sums over channels LDS holds (16 KB)
    __shared__ __align__(16) X sx[R::SIZE], sd[R::SIZE], sy[R::SIZE], sz[R::SIZE];
    __shared__ __align__(16) float sb[S::SIZE], sc[S::SIZE];
    __shared__ float red[4][ROUND * 2 * NP];
    const uint32_t id = xcd_remap(blockIdx.x, gridDim.x), cb = id % G.nblk, walker = id / G.nblk;
    const ScanLane<LPC> w(G, cb);
    const int lane = (int)threadIdx.x & 63, wave = (int)threadIdx.x >> 6;
    float a2[4], da[4] = {0.0f, 0.0f, 0.0f, 0.0f}, dskip = 0.0f, dbias = 0.0f;
    load_rates(a2, in.a, G, w.c, 4 * w.j, w.live);
    const float bias = in.bias && w.live ? in.bias[w.c] : 0.0f, skip = in.skip && w.live ? in.skip[w.c] : 0.0f;
    for (uint32_t slot = walker; slot < G.slots; slot += G.walkers) {
        const Piece p = piece(G, slot);
        if (G.CH && p.t0 >= p.t1) continue;
        const int64_t srow = ((int64_t)p.s * G.C + (w.live ? w.c : 0)) * G.N;
        const int64_t mine = ((int64_t)slot * G.nblk + cb) * THREADS + threadIdx.x;
        const int begin = G.seq.begin(p.s);
        // the kept state of the block that begins at token t
        auto kept = [&](int t) {
            const int64_t block = (int64_t)(begin / TT) + p.s + (t - begin) / TT;
            return o.kept + ((block * G.nblk + cb) * THREADS + threadIdx.x) * 4;
        };
        float h[4], g[4];
        if (starts) load_f32<F32, 4>(h, starts + mine * 4);
        else load_states(h, state_in ? state_in + srow : nullptr, 4 * w.j, G.N, w.live && state_in);
        if (afters) load_f32<F32, 4>(g, afters + mine * 4);
        else load_states(g, dstate_out ? dstate_out + srow : nullptr, 4 * w.j, G.N, w.live && dstate_out);
        const int tl = p.t1 > p.t0 ? p.t0 + (p.t1 - p.t0 - 1) / TT * TT : p.t0;  // the last block
        R rx, rd, ry, rz;
        S rb, rc;
        // forward to the last block, keeping the states before each
        auto fetch_in = [&](int t) {
            rx.fetch((const X *)in.x, in.ldx, t, TT, w.c0, w.cend);
            rd.fetch((const X *)in.dt, in.lddt, t, TT, w.c0, w.cend);
            rb.fetch((const X *)in.b, in.ldb, t, TT, w.g * G.N, G.N);
        };
        if (p.t0 < tl) fetch_in(p.t0);
        for (int t = p.t0; t < tl; t += TT) {
            __syncthreads();
            rx.put(sx);
            rd.put(sd);
            rb.put(sb);
            __syncthreads();
            if (t + TT < tl) fetch_in(t + TT);
            store_f32<F32, 4>(kept(t), h);
            for (int u = 0; u < TT; u += 4) {
                const int own = u + w.q;
                float slope;
                const float d = step_width<DT>(R::get(sd, own, w.ch) + bias, G.soft, slope);
                const float dx = d * R::get(sx, own, w.ch);
                auto token = [&](int s, float ds, float us) {
                    float bv[4];
                    S::get(bv, sb, u + s, w.j);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        h[i] = __builtin_fmaf(__builtin_amdgcn_exp2f(ds * a2[i]), h[i], us * bv[i]);
                };
                token(0, quad<0>(d), quad<0>(dx));
                token(1, quad<1>(d), quad<1>(dx));
                token(2, quad<2>(d), quad<2>(dx));
                token(3, quad<3>(d), quad<3>(dx));
            }
        }
        // back over the blocks
        auto fetch = [&](int t) {
            const int cnt = min(TT, p.t1 - t);
            rx.fetch((const X *)in.x, in.ldx, t, cnt, w.c0, w.cend);
            rd.fetch((const X *)in.dt, in.lddt, t, cnt, w.c0, w.cend);
            ry.fetch((const X *)in.dy, in.lddy, t, cnt, w.c0, w.cend);
            if (in.gate) rz.fetch((const X *)in.gate, in.ldgate, t, cnt, w.c0, w.cend);
            rb.fetch((const X *)in.b, in.ldb, t, cnt, w.g * G.N, G.N);
            rc.fetch((const X *)in.c, in.ldc, t, cnt, w.g * G.N, G.N);
        };
        if (p.t0 < p.t1) fetch(tl);
        for (int t = tl; t >= p.t0 && p.t0 < p.t1; t -= TT) {
            const int cnt = min(TT, p.t1 - t);
            __syncthreads();  // the tile before has been written out
            rx.put(sx);
            rd.put(sd);
            ry.put(sy);
            if (in.gate) rz.put(sz);
            rb.put(sb);
            rc.put(sc);
            __syncthreads();
            float h0[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) h0[i] = h[i];
            if (t > p.t0) {
                fetch(t - TT);
                load_f32<F32, 4>(h, kept(t - TT));  // for the next block
            }
            // the block's states and decays, and what its tokens need once a channel
            float hs[TT][4], es[TT][4], d[4], slope[4], dy[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int own = 4 * k + w.q;
                d[k] = step_width<DT>(R::get(sd, own, w.ch) + bias, G.soft, slope[k]);
                d[k] = own < cnt ? d[k] : 0.0f;
                const float xv = R::get(sx, own, w.ch), dx = d[k] * xv;
                dy[k] = R::get(sy, own, w.ch);
                float yy = 0.0f;
                auto token = [&](int s, float ds, float us) {
                    float bv[4], cv[4], v = 0.0f;
                    S::get(bv, sb, 4 * k + s, w.j);
                    if (in.gate) S::get(cv, sc, 4 * k + s, w.j);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float e = __builtin_amdgcn_exp2f(ds * a2[i]);
                        const float before = k + s ? hs[k + s ? 4 * k + s - 1 : 0][i] : h0[i];
                        es[4 * k + s][i] = e;
                        hs[4 * k + s][i] = __builtin_fmaf(e, before, us * bv[i]);
                        if (in.gate) v = __builtin_fmaf(hs[4 * k + s][i], cv[i], v);
                    }
                    if (in.gate) {
                        v = sum_states<LPC>(v);
                        yy = w.q == s ? v : yy;
                    }
                };
                token(0, quad<0>(d[k]), quad<0>(dx));
                token(1, quad<1>(d[k]), quad<1>(dx));
                token(2, quad<2>(d[k]), quad<2>(dx));
                token(3, quad<3>(d[k]), quad<3>(dx));
                if (in.gate) {
                    float gs;
                    const float gv = gate_value<DT>(R::get(sz, own, w.ch), G.act, gs);
                    yy = __builtin_fmaf(skip, xv, yy);
                    if (w.j < 4) R::set(sz, own, w.ch, dy[k] * yy * gs);
                    dy[k] *= gv;
                }
            }
            // back over its tokens
            float v[A::V];
            const int first = A::first(lane);
#pragma unroll
            for (int k = 3; k >= 0; --k) {
                const int own = 4 * k + w.q;
                const float xv = R::get(sx, own, w.ch), dx = d[k] * xv;
                float du = 0.0f, dd = 0.0f;
                auto token = [&](int s, float ds, float us, float ys) {
                    float bv[4], cv[4], vu = 0.0f, vd = 0.0f;
                    S::get(bv, sb, 4 * k + s, w.j);
                    S::get(cv, sc, 4 * k + s, w.j);
                    const int to = (4 * k + s) % A::TOK * 8;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        g[i] = __builtin_fmaf(cv[i], ys, g[i]);
                        v[to + i] = g[i] * us;
                        v[to + 4 + i] = hs[4 * k + s][i] * ys;
                        vu = __builtin_fmaf(g[i], bv[i], vu);
                        g[i] *= es[4 * k + s][i];
                        const float gh = g[i] * (k + s ? hs[k + s ? 4 * k + s - 1 : 0][i] : h0[i]);
                        vd = __builtin_fmaf(gh, a2[i], vd);
                        da[i] = __builtin_fmaf(gh, ds, da[i]);
                    }
                    vu = sum_states<LPC>(vu);
                    vd = sum_states<LPC>(vd);
                    du = w.q == s ? vu : du;
                    dd = w.q == s ? vd : dd;
                    if ((4 * k + s) % A::TOK == 0) {
                        A::sum(v, lane);
#pragma unroll
                        for (int r = 0; r < A::R; ++r) {
                            const int i = first + r, tok = (4 * k + s) % ROUND + i / 8;
                            red[wave][(tok * 2 + i / 4 % 2) * NP + 4 * w.j + i % 4] = v[r];
                        }
                    }
                };
                token(3, quad<3>(d[k]), quad<3>(dx), quad<3>(dy[k]));
                token(2, quad<2>(d[k]), quad<2>(dx), quad<2>(dy[k]));
                token(1, quad<1>(d[k]), quad<1>(dx), quad<1>(dy[k]));
                token(0, quad<0>(d[k]), quad<0>(dx), quad<0>(dy[k]));
                // own tokens past the end have d = dy = 0: they add nothing
                const float dw = __builtin_fmaf(du, xv, dd * LN2) * slope[k];
                const float add = own < cnt ? dw : 0.0f;
                dbias += add;
                dskip = __builtin_fmaf(dy[k], xv, dskip);
                if (w.j < 4) {
                    R::set(sx, own, w.ch, __builtin_fmaf(du, d[k], skip * dy[k]));
                    R::set(sd, own, w.ch, dw);
                }
                if (4 * k % ROUND == 0) {
                    __syncthreads();
                    for (int i = threadIdx.x; i < ROUND * 2 * NP; i += THREADS) {
                        const int tok = t + 4 * k + i / (2 * NP);
                        const float sum = (red[0][i] + red[1][i]) + (red[2][i] + red[3][i]);
                        if (tok < p.t1) o.part[((int64_t)cb * G.seq.tokens + tok) * (2 * NP) + i % (2 * NP)] = sum;
                    }
                    if (k) __syncthreads();
                }
            }
            R::flush(sx, (X *)o.dx, o.lddx, t, cnt, w.c0, w.cend);
            R::flush(sd, (X *)o.ddt, o.ldddt, t, cnt, w.c0, w.cend);
            if (in.gate && o.dgate) R::flush(sz, (X *)o.dgate, o.lddgate, t, cnt, w.c0, w.cend);
        }
        if (dstate_in && !afters) store_states(dstate_in + srow, g, 4 * w.j, G.N, w.live);
    }
    const int64_t at = (int64_t)walker * G.nblk + cb;
    store_f32<F32, 4>(o.pa + (at * THREADS + threadIdx.x) * 4, da);
    dskip += dpp<0xB1>(dskip);
    dskip += dpp<0x4E>(dskip);
    dbias += dpp<0xB1>(dbias);
    dbias += dpp<0x4E>(dbias);
    if (w.j == 0) {
        o.ps[at * 2 * CPW + w.ch] = dskip;
        o.ps[at * 2 * CPW + CPW + w.ch] = dbias;
    }
}

struct Total {
    void *db, *dc;
    int64_t lddb, lddc;
    float *da, *dskip, *dbias;
    uint32_t blocks_bc, blocks_a;   // workgroups of db and dc, of da; the others dskip and dbias
};

// n values `step` apart, four at a time
__device__ __forceinline__ float column(const float *p, int64_t step, int64_t n) {
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    int64_t i = 0;
    for (; i + 8 <= n; i += 8) {
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = p[(i + k) * step];
#pragma unroll
        for (int k = 0; k < 8; ++k) s[k & 3] += v[k];
    }
    for (; i < n; ++i) s[i & 3] += p[i * step];
    return (s[0] + s[1]) + (s[2] + s[3]);
}

// The sums of the workgroups' sums, each by one lane in order.
template <class DT, int LPC>
__global__ void __launch_bounds__(THREADS) k_total(ScanGeo G, Out o, Total z) {
    using X = typename DT::X;
    constexpr int NP = 4 * LPC, CPW = THREADS / LPC;
    const int cg = G.C / G.G;
    auto channel = [&](uint32_t cb, int ch) {  // -1: none
        const int c = (int)(cb % G.per_group) * CPW + ch;
        return c < cg ? (int)(cb / G.per_group) * cg + c : -1;
    };
    if (blockIdx.x < z.blocks_bc) {
        const int64_t i = (int64_t)blockIdx.x * THREADS + threadIdx.x, row = (int64_t)G.seq.tokens * 2 * NP;
        const int64_t grp = i / row, at = i % row;
        const int n = (int)(at % NP), second = (int)(at / NP % 2), t = (int)(at / (2 * NP));
        if (grp >= G.G || n >= G.N || G.seq.seqs == 0 || t >= G.seq.end(G.seq.seqs - 1)) return;
        const float s = column(o.part + grp * G.per_group * row + at, row, G.per_group);
        X *p = second ? (X *)z.dc + (int64_t)t * z.lddc : (X *)z.db + (int64_t)t * z.lddb;
        p[grp * G.N + n] = rounded<DT>(s);
        return;
    }
    if (blockIdx.x < z.blocks_bc + z.blocks_a) {
        const int64_t i = (int64_t)(blockIdx.x - z.blocks_bc) * THREADS + threadIdx.x, row = (int64_t)G.nblk * THREADS * 4;
        if (i >= row) return;
        const int at = (int)(i % (THREADS * 4)), n = at % NP, c = channel((uint32_t)(i / (THREADS * 4)), at / NP);
        if (c >= 0 && n < G.N) z.da[(int64_t)c * G.N + n] = column(o.pa + i, row, G.walkers);
        return;
    }
    const int64_t i = (int64_t)(blockIdx.x - z.blocks_bc - z.blocks_a) * THREADS + threadIdx.x, row = (int64_t)G.nblk * 2 * CPW;
    if (i >= row) return;
    const int at = (int)(i % (2 * CPW)), c = channel((uint32_t)(i / (2 * CPW)), at % CPW);
    float *out = at < CPW ? z.dskip : z.dbias;
    if (c >= 0 && out) out[c] = column(o.ps + i, row, G.walkers);
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
ScanGeo geometry(const dwconv_scan_plan &p, const int32_t *offsets, int seqs, int tokens, bool back) {
    ScanGeo G = scan_blocks(p, scan_lanes(p.N));
    G.seq = {offsets, seqs, tokens};
    const int64_t enough = back ? 512 : 768, want = back ? 1024 : 1536;
    if ((int64_t)seqs * G.nblk < enough && seqs > 0) {
        int ch = 1024;
        while (ch > 64 && ((int64_t)tokens / ch + seqs) * G.nblk < want) ch /= 2;
        if (tokens / seqs > ch) G.CH = ch;
    }
    const int64_t slots = G.CH ? (int64_t)tokens / G.CH + seqs : seqs;
    G.slots = (uint32_t)slots;
    const int64_t most = (2048 + G.nblk - 1) / G.nblk;
    G.walkers = (uint32_t)(slots < most ? slots : most);
    return G;
}

struct Sizes {
    size_t ends, width, back, kept, part, pa, ps, all;  // floats
};
Sizes sizes(const ScanGeo &G, int lpc, bool back) {
    const size_t block = (size_t)G.nblk * THREADS * 4, cpw = THREADS / lpc;
    Sizes z{};
    if (G.CH) {
        z.ends = G.slots * block;
        z.width = (size_t)G.slots * G.nblk * cpw;
        z.back = back ? z.ends : 0;
    }
    if (back) {
        z.kept = ((size_t)G.seq.tokens / TT + G.seq.seqs) * block;
        z.part = (size_t)G.nblk * G.seq.tokens * 8 * lpc;
        z.pa = G.walkers * block;
        z.ps = (size_t)G.walkers * G.nblk * 2 * cpw;
    }
    z.all = z.ends + z.width + z.back + z.kept + z.part + z.pa + z.ps;
    return z;
}

template <class DT, int LPC>
hipError_t fwd(const dwconv_scan_plan &p, const ScanArgs &a, hipStream_t st) {
    const ScanGeo G = geometry(p, a.offsets, a.seqs, a.tokens, false);
    const ScanIn in = scan_inputs(a);
    const uint64_t blocks = (uint64_t)G.slots * G.nblk, joins = (uint64_t)a.seqs * G.nblk;
    if (too_many(blocks)) return hipErrorInvalidConfiguration;
    if (!blocks) return hipSuccess;
    float *starts = nullptr;
    if (G.CH) {
        starts = a.workspace;
        float *width = starts + sizes(G, LPC, false).ends;
        k_ends<DT, LPC, false><<<(uint32_t)blocks, THREADS, 0, st>>>(G, in, starts, width, nullptr);
        k_join<LPC, false><<<(uint32_t)joins, THREADS, 0, st>>>(G, a.a, a.state_in, a.state_out, nullptr, nullptr, starts,
                                                                width, nullptr);
    }
    k_out<DT, LPC><<<(uint32_t)blocks, THREADS, 0, st>>>(G, in, a.state_in, starts, a.state_out, (typename DT::X *)a.y, a.ldy);
    return hipGetLastError();
}

template <class DT, int LPC>
hipError_t bwd(const dwconv_scan_plan &p, const ScanArgs &a, hipStream_t st) {
    const ScanGeo G = geometry(p, a.offsets, a.seqs, a.tokens, true);
    const Sizes z = sizes(G, LPC, true);
    const ScanIn in = scan_inputs(a);
    float *f = a.workspace;
    Out o{a.dx, a.ddt, a.dgate, a.lddx, a.ldddt, a.lddgate, nullptr, nullptr, nullptr, nullptr};
    float *ends = f, *back = ends + z.ends, *width;
    o.kept = back + z.back;
    o.part = o.kept + z.kept;
    o.pa = o.part + z.part;
    o.ps = o.pa + z.pa;
    width = o.ps + z.ps;
    const uint64_t pieces = (uint64_t)G.slots * G.nblk, joins = (uint64_t)a.seqs * G.nblk;
    const uint64_t walks = (uint64_t)G.walkers * G.nblk;
    const uint64_t bc = ((uint64_t)G.G * a.tokens * 8 * LPC + THREADS - 1) / THREADS, ab = (uint64_t)G.nblk * 4;
    const uint64_t sb = ((uint64_t)G.nblk * 2 * (THREADS / LPC) + THREADS - 1) / THREADS;
    if (too_many(pieces) || too_many(walks) || too_many(bc + ab + sb) || (uint64_t)a.tokens * G.nblk >= (1ull << 44))
        return hipErrorInvalidConfiguration;
    if (G.CH) {
        k_ends<DT, LPC, true><<<(uint32_t)pieces, THREADS, 0, st>>>(G, in, ends, width, back);
        k_join<LPC, true><<<(uint32_t)joins, THREADS, 0, st>>>(G, a.a, a.state_in, nullptr, a.dstate_out, a.dstate_in, ends,
                                                               width, back);
    }
    if (walks)
        k_grad<DT, LPC><<<(uint32_t)walks, THREADS, 0, st>>>(G, in, o, a.state_in, a.dstate_out, a.dstate_in,
                                                             G.CH ? ends : nullptr, G.CH ? back : nullptr);
    const Total tot{a.db, a.dc, a.lddb, a.lddc, a.da, a.dskip, a.dbias, (uint32_t)bc, (uint32_t)ab};
    k_total<DT, LPC><<<(uint32_t)(bc + ab + sb), THREADS, 0, st>>>(G, o, tot);
    return hipGetLastError();
}

template <bool BACK, class DT>
hipError_t pick_lanes(const dwconv_scan_plan &p, const ScanArgs &a, hipStream_t st) {
    auto go = [&](auto lanes) {
        constexpr int L = decltype(lanes)::value;
        if constexpr (BACK) return bwd<DT, L>(p, a, st);
        else return fwd<DT, L>(p, a, st);
    };
    switch (scan_lanes(p.N)) {
        case 4: return go(std::integral_constant<int, 4>());
        case 8: return go(std::integral_constant<int, 8>());
        case 16: return go(std::integral_constant<int, 16>());
        default: return go(std::integral_constant<int, 32>());
    }
}

template <bool BACK>
hipError_t pick(const dwconv_scan_plan &p, const ScanArgs &a, hipStream_t st) {
    switch (p.dtype) {
        case DWCONV_F32: return pick_lanes<BACK, F32>(p, a, st);
        case DWCONV_F16: return pick_lanes<BACK, F16>(p, a, st);
        default: return pick_lanes<BACK, BF16>(p, a, st);
    }
}

}  // namespace

hipError_t scan_fwd(const dwconv_scan_plan &p, const ScanArgs &a, hipStream_t st) { return pick<false>(p, a, st); }
hipError_t scan_bwd(const dwconv_scan_plan &p, const ScanArgs &a, hipStream_t st) { return pick<true>(p, a, st); }

size_t scan_bytes(const dwconv_scan_plan &p, int seqs, int tokens, bool back) {
    const ScanGeo G = geometry(p, nullptr, seqs, tokens, back);
    // as many pieces as no grid holds: more than there is (their bytes may pass 2^64)
    if (too_many((uint64_t)G.slots * G.nblk) || (uint64_t)tokens * G.nblk >= (1ull << 44)) return SIZE_MAX;
    return sizes(G, scan_lanes(p.N), back).all * sizeof(float);
}

}  // namespace dw
