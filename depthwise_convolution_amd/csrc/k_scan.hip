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
// walk back over blocks of 8 tokens whose first states a walk forward has left in the
// workspace; a block's states and decays are formed again and stay in registers.
//
// Vector instructions bound all of it, an exponential (8 cycles) and four operations (4 each)
// a state and token forward, in the gradients about 76 cycles: 16384 tokens x 8192 channels x
// 16 states, bf16, 1.39 million cycles, of which vector units are busy 84 % (97 % where sequences
// are equally long), 574 us at 2.41 GHz and 645 to 700 at 2.16 to 1.97, as under a profiler
// (0.79 million for those instructions alone; 204 us for the bytes at a copy's rate); fp32 687.
// Gradients of 4096 x 8192 1.40 million, 595 us (0.62; bytes 90, with the states and sums that
// they keep and read again 217).  One sequence of 5003 x 2048 in runs of 64: k_ends 36, k_join
// 11, k_out 49 us; gradients of 2048 x 2048 33, 11 and 76.  Sums over channels on the matrix
// units, with a left operand of zeros and ones, take longer (gradients 870): an fp32 product's
// 32 cycles add to the vector unit's time.
#include <type_traits>

#include "scan_common.h"

namespace dw {
namespace {

constexpr int TT = 16;         // tokens a tile
constexpr int HT = 8;          // tokens between two kept states
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
        if constexpr (LPC == 4) {
            // Lane bits 3 and 2: lanes whose bit is 0 keep the value v[i] and add their partner's,
            // the others v[i + n / 2].  Two instructions a value, since a bank mask leaves the other
            // lanes of the destination as they are; the compiler takes a select and two (gradients of
            // 4096 x 8192 690 -> 643 us).  It knows neither that these are lane moves, which read a
            // register two wait states after its writing at the earliest, nor that the next may be.
            asm("s_nop 1\n\t"
                "v_add_f32_dpp %0, %0, %0 row_shl:8 row_mask:0xf bank_mask:0x3\n\t"
                "v_add_f32_dpp %0, %8, %8 row_shr:8 row_mask:0xf bank_mask:0xc\n\t"
                "v_add_f32_dpp %1, %1, %1 row_shl:8 row_mask:0xf bank_mask:0x3\n\t"
                "v_add_f32_dpp %1, %9, %9 row_shr:8 row_mask:0xf bank_mask:0xc\n\t"
                "v_add_f32_dpp %2, %2, %2 row_shl:8 row_mask:0xf bank_mask:0x3\n\t"
                "v_add_f32_dpp %2, %10, %10 row_shr:8 row_mask:0xf bank_mask:0xc\n\t"
                "v_add_f32_dpp %3, %3, %3 row_shl:8 row_mask:0xf bank_mask:0x3\n\t"
                "v_add_f32_dpp %3, %11, %11 row_shr:8 row_mask:0xf bank_mask:0xc\n\t"
                "v_add_f32_dpp %4, %4, %4 row_shl:8 row_mask:0xf bank_mask:0x3\n\t"
                "v_add_f32_dpp %4, %12, %12 row_shr:8 row_mask:0xf bank_mask:0xc\n\t"
                "v_add_f32_dpp %5, %5, %5 row_shl:8 row_mask:0xf bank_mask:0x3\n\t"
                "v_add_f32_dpp %5, %13, %13 row_shr:8 row_mask:0xf bank_mask:0xc\n\t"
                "v_add_f32_dpp %6, %6, %6 row_shl:8 row_mask:0xf bank_mask:0x3\n\t"
                "v_add_f32_dpp %6, %14, %14 row_shr:8 row_mask:0xf bank_mask:0xc\n\t"
                "v_add_f32_dpp %7, %7, %7 row_shl:8 row_mask:0xf bank_mask:0x3\n\t"
                "v_add_f32_dpp %7, %15, %15 row_shr:8 row_mask:0xf bank_mask:0xc\n\t"
                "v_add_f32_dpp %0, %0, %0 row_shl:4 row_mask:0xf bank_mask:0x5\n\t"
                "v_add_f32_dpp %0, %4, %4 row_shr:4 row_mask:0xf bank_mask:0xa\n\t"
                "v_add_f32_dpp %1, %1, %1 row_shl:4 row_mask:0xf bank_mask:0x5\n\t"
                "v_add_f32_dpp %1, %5, %5 row_shr:4 row_mask:0xf bank_mask:0xa\n\t"
                "v_add_f32_dpp %2, %2, %2 row_shl:4 row_mask:0xf bank_mask:0x5\n\t"
                "v_add_f32_dpp %2, %6, %6 row_shr:4 row_mask:0xf bank_mask:0xa\n\t"
                "v_add_f32_dpp %3, %3, %3 row_shl:4 row_mask:0xf bank_mask:0x5\n\t"
                "v_add_f32_dpp %3, %7, %7 row_shr:4 row_mask:0xf bank_mask:0xa\n\t"
                "s_nop 1"
                : "+&v"(v[0]), "+&v"(v[1]), "+&v"(v[2]), "+&v"(v[3]),
                  "+&v"(v[4]), "+&v"(v[5]), "+&v"(v[6]), "+&v"(v[7])
                : "v"(v[8]), "v"(v[9]), "v"(v[10]), "v"(v[11]),
                  "v"(v[12]), "v"(v[13]), "v"(v[14]), "v"(v[15]));
            n = 4;
        }
        if (LPC == 8) {  // lane bit 3
            const bool hi = lane & 8;
            n /= 2;
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                const float m = hi ? v[i + V / 2] : v[i], o = hi ? v[i] : v[i + V / 2];
                v[i] = m + dpp<0x128>(o);  // lane ^ 8
            }
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
};
__device__ __forceinline__ int64_t slot_base(const ScanGeo &G, int s) { return G.CH ? (int64_t)(G.seq.begin(s) / G.CH) + s : s; }
__device__ __forceinline__ Piece piece(const ScanGeo &G, int64_t slot) {
    int s = (int)slot, t0, t1;
    if (G.CH) {
        int lo = 0, hi = G.seq.seqs;
        while (hi - lo > 1) {
            const int m = lo + ((hi - lo) >> 1);
            if (slot_base(G, m) <= slot) lo = m; else hi = m;
        }
        const int b = G.seq.begin(lo), e = G.seq.end(lo);
        const int64_t t = b + (slot - slot_base(G, lo)) * G.CH;
        const bool in = t >= b && t < e;
        s = lo;
        t0 = in ? (int)t : 0;
        t1 = !in ? 0 : e - t > G.CH ? (int)t + G.CH : e;
    } else {
        t0 = G.seq.begin(s);
        t1 = G.seq.end(s);
    }
    return {uniform(s), uniform(t0), uniform(t1)};  // the same for all lanes, which loads from memory do not tell
}

// Whole sequences, longest first.  Workgroups of a launch that fits the chip go to its CUs
// in rounds of 256, every second one backwards here, so that the CU with the longest
// sequence of one round has the shortest of the next; later ones go where a place is free.
// For up to 64 sequences, whose lengths a wavefront sorts; of more, every CU has some of each.
// 7 sequences of 1553 to 3465 tokens, 8192 channels: 630 us, in their order 692; gradients of
// 4 of 593 to 1266 tokens 640 and 708.
__device__ __forceinline__ void longest_first(const ScanGeo &G, uint32_t &id, uint32_t all) {
    if (G.CH || !G.seq.offsets || G.seq.seqs > 64 || G.slots != (uint32_t)G.seq.seqs || G.seq.seqs < 2) return;
    const uint32_t round = id / 256;
    if (round & 1) id = round * 256 + min(255u, all - 1 - round * 256) - id % 256;
    const int j = (int)threadIdx.x & 63, len = j < G.seq.seqs ? G.seq.end(j) - G.seq.begin(j) : -1;
    int rank = 0;
    for (int k = 0; k < G.seq.seqs; ++k) {
        const int other = __builtin_amdgcn_readlane(len, k);
        rank += other > len || (other == len && k < j);
    }
    const uint64_t mine = __ballot(j < G.seq.seqs && rank == (int)(id / G.nblk));
    id = (uint32_t)__builtin_ctzll(mine) * G.nblk + id % G.nblk;
}

// Workgroups are handed to the 8 XCDs round-robin, and so to their CUs: the pieces of a
// long sequence, which lie one beside the other, on all of them.  Only the workgroups
// that share 128-byte lines of a row (LPC / 4 of 16-bit data) keep to one XCD, whose L2
// they share.
template <int LPC>
__device__ __forceinline__ uint32_t spread(uint32_t b, uint32_t all) {
    constexpr uint32_t U = LPC / 4;
    if (U == 1 || b >= all / (8 * U) * (8 * U)) return b;
    const uint32_t k = b / 8;
    return (k / U * 8 + b % 8) * U + k % U;
}

// ---------------------------------------------------------------------------
// tiles
// ---------------------------------------------------------------------------
// A tensor as a workgroup walks it: the address of its first token (a scalar) and the
// lane's offset in a tile, 32 bits (strides are at most 2^26 elements): whole tiles of
// whole vectors cost a load each and no other vector instruction.
template <class X>
struct Walk {
    const X *p;
    int64_t ld;
    uint32_t off;  // bytes
    __device__ __forceinline__ Walk(const void *base, int64_t ld, int row, int col) : p((const X *)base), ld(ld) {
        off = ((uint32_t)row * (uint32_t)ld + (uint32_t)col) * (uint32_t)sizeof(X);
    }
    __device__ __forceinline__ X *at(int t) const { return (X *)((char *)(p + (int64_t)t * ld) + off); }
};

// 16 tokens of the workgroup's channels, a vector of four a lane.  The vectors need
// no more than the element's alignment: the loads take any.
template <class DT, int LPC>
struct Rows {
    using X = typename DT::X;
    // four elements as words: what is on its way stays as it comes (elements taken apart
    // would wait for the load)
    static constexpr int W = (int)sizeof(X);
    using Words = Vec<uint32_t, W>;
    struct __attribute__((packed, aligned(sizeof(X)))) Any {
        uint32_t w[W];
    };
    static constexpr int CPW = THREADS / LPC, VPR = CPW / 4, LD = CPW + 16;
    static constexpr int SIZE = TT * LD;
    Any v;
    static __device__ __forceinline__ int row() { return (int)threadIdx.x / VPR; }
    static __device__ __forceinline__ int col() { return (int)threadIdx.x % VPR * 4; }
    // the tensor from channel c0 on; lanes past a tile follow its first row
    static __device__ __forceinline__ Walk<X> walk(const void *p, int64_t ld, int c0) {
        return {p ? (const X *)p + c0 : nullptr, ld, row() < TT ? row() : 0, col()};
    }
    // `width`: channels of the workgroup
    __device__ __forceinline__ void fetch(const Walk<X> &w, int t, int cnt, int width) {
        const X *at = w.at(t);
        if (cnt == TT && width >= CPW) {
            v = *(const Any *)at;
            return;
        }
        X e[4] = {(X)0, (X)0, (X)0, (X)0};
        if (row() < cnt) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (col() + i < width) e[i] = at[i];
        }
        __builtin_memcpy(&v, e, sizeof(v));
    }
    __device__ __forceinline__ void put(X *lds) const {
        if (row() < TT) *(Words *)(lds + row() * LD + col()) = __builtin_bit_cast(Words, v);
    }
    static __device__ __forceinline__ void flush(const X *lds, const Walk<X> &w, int t, int cnt, int width) {
        if (row() >= cnt) return;
        const Words u = *(const Words *)(lds + row() * LD + col());
        X *at = w.at(t);
        if (width >= CPW) {
            *(Any *)at = __builtin_bit_cast(Any, u);
        } else {
            X e[4];
            __builtin_memcpy(e, &u, sizeof(e));
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (col() + i < width) at[i] = e[i];
        }
    }
    static __device__ __forceinline__ float get(const X *lds, int tok, int ch) { return DT::widen(lds[tok * LD + ch]); }
    static __device__ __forceinline__ void set(X *lds, int tok, int ch, float v) { lds[tok * LD + ch] = rounded<DT>(v); }
};

// b or c of 16 tokens, fp32, states past N zero
template <class DT, int LPC>
struct Shared {
    using X = typename DT::X;
    static constexpr int NP = 4 * LPC, PT = TT * NP / THREADS, SIZE = TT * NP, ROWS = THREADS / NP > 0 ? THREADS / NP : 1;
    X v[PT];
    static __device__ __forceinline__ int state() { return (int)threadIdx.x % NP; }
    // the tensor from state n0 on; a lane has one state of every ROWS-th token
    static __device__ __forceinline__ Walk<X> walk(const void *p, int64_t ld, int n0, int N) {
        return {(const X *)p + n0, ld, (int)threadIdx.x / NP, state() < N ? state() : 0};
    }
    __device__ __forceinline__ void fetch(const Walk<X> &w, int t, int cnt) {
#pragma unroll
        for (int k = 0; k < PT; ++k) {
            const int r = (int)threadIdx.x / NP + k * ROWS;
            v[k] = (X)0;
            if (cnt == TT || r < cnt) v[k] = *w.at(t + k * ROWS);
        }
    }
    __device__ __forceinline__ void put(float *lds, int N) const {
#pragma unroll
        for (int k = 0; k < PT; ++k) lds[threadIdx.x + k * THREADS] = state() < N ? DT::widen(v[k]) : 0.0f;
    }
    static __device__ __forceinline__ void get(float (&o)[4], const float *lds, int tok, int j) {
        load_f32<F32, 4>(o, lds + tok * NP + 4 * j);
    }
};

// What a tile's tokens need once a channel; lane q of a quad has tokens q, 4 + q ...
// Tokens past the end have width zero: they change no state.
template <class DT, int LPC>
struct Own {
    float x[4], d[4], u[4], slope[4];  // u = d x
    __device__ __forceinline__ Own(const typename DT::X *sx, const typename DT::X *sd, const ScanLane<LPC> &w, float bias,
                                   int soft, int cnt) {
        using R = Rows<DT, LPC>;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int own = 4 * k + w.q;
            x[k] = R::get(sx, own, w.ch);
            d[k] = R::get(sd, own, w.ch) + bias;
            slope[k] = 1.0f;
        }
        if (soft) {
#pragma unroll
            for (int k = 0; k < 4; ++k) d[k] = softplus<DT>(d[k], slope[k]);
        }
        if (cnt < TT) {
#pragma unroll
            for (int k = 0; k < 4; ++k) d[k] = 4 * k + w.q < cnt ? d[k] : 0.0f;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) u[k] = d[k] * x[k];
    }
};
// The value of lane S of each quad, for a token's number in the tile
__device__ __forceinline__ float of_token(const float (&v)[4], int t) {
    const float w = v[t / 4];
    return t % 4 == 0 ? quad<0>(w) : t % 4 == 1 ? quad<1>(w) : t % 4 == 2 ? quad<2>(w) : quad<3>(w);
}
// f(k) for the four quads of tokens that a tile of cnt has; all of them at once where it
// is full, so that one quad's sums run beside the next one's products
template <class F>
__device__ __forceinline__ void quads(int cnt, F f) {
    if (cnt == TT) {
#pragma unroll
        for (int k = 0; k < 4; ++k) f(k);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (4 * k < cnt) f(k);
    }
}

// 2^p, for p past 127 2^127 (NaN stays): one of two factors.  The product of both at 2^127
// takes any normal number out of fp32's range, as whatever is larger would.
__device__ __forceinline__ float grown(float p) { return __builtin_amdgcn_exp2f(p > 127.0f ? 127.0f : p); }

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------
template <class DT, int LPC, bool GATE>
__global__ void __launch_bounds__(THREADS, sizeof(typename DT::X) == 2 && LPC <= 8 ? 5 : 3)
    k_out(ScanGeo G, ScanIn in, const float *state_in, const float *starts, float *state_out, typename DT::X *y, int64_t ldy) {
    using X = typename DT::X;
    using R = Rows<DT, LPC>;
    using S = Shared<DT, LPC>;
    __shared__ __align__(16) X sx[2][R::SIZE], sd[2][R::SIZE], sz[2][GATE ? R::SIZE : 8], sy[2][R::SIZE];
    __shared__ __align__(16) float sb[2][S::SIZE], sc[2][S::SIZE];
    uint32_t id = spread<LPC>(blockIdx.x, gridDim.x);
    longest_first(G, id, gridDim.x);
    id = (uint32_t)uniform((int)id);
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
    const Walk<X> wx = R::walk(in.x, in.ldx, w.c0), wd = R::walk(in.dt, in.lddt, w.c0), wz = R::walk(in.gate, in.ldgate, w.c0),
                  wy = R::walk(y, ldy, w.c0), wb = S::walk(in.b, in.ldb, w.g * G.N, G.N), wc = S::walk(in.c, in.ldc, w.g * G.N, G.N);
    const int width = w.cend - w.c0;
    R rx, rd, rz;
    S rb, rc;
    auto fetch = [&](int t) {
        const int cnt = min(TT, p.t1 - t);
        rx.fetch(wx, t, cnt, width);
        rd.fetch(wd, t, cnt, width);
        if (GATE) rz.fetch(wz, t, cnt, width);
        rb.fetch(wb, t, cnt);
        rc.fetch(wc, t, cnt);
    };
    int k = 0;
    if (p.t0 < p.t1) fetch(p.t0);
    for (int t = p.t0; t < p.t1; t += TT, k ^= 1) {
        rx.put(sx[k]);
        rd.put(sd[k]);
        if (GATE) rz.put(sz[k]);
        rb.put(sb[k], G.N);
        rc.put(sc[k], G.N);
        __syncthreads();  // the one barrier a tile: what a tile writes is read in its own turn or the next
        if (t > p.t0) R::flush(sy[k ^ 1], wy, t - TT, TT, width);
        if (p.t1 - t > TT) fetch(t + TT);
        const int cnt = min(TT, p.t1 - t);
        const Own<DT, LPC> own(sx[k], sd[k], w, bias, G.soft, cnt);
        quads(cnt, [&](int n) {
            float v[4];
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const float ds = of_token(own.d, 4 * n + s), us = of_token(own.u, 4 * n + s);
                float bv[4], cv[4];
                S::get(bv, sb[k], 4 * n + s, w.j);
                S::get(cv, sc[k], 4 * n + s, w.j);
                v[s] = 0.0f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    h[i] = __builtin_fmaf(__builtin_amdgcn_exp2f(ds * a2[i]), h[i], us * bv[i]);
                    v[s] = __builtin_fmaf(h[i], cv[i], v[s]);
                }
            }
            float yy = __builtin_fmaf(skip, own.x[n], sum_states4<LPC>(v, w.q));
            if (GATE) yy *= gate_value<DT>(R::get(sz[k], 4 * n + w.q, w.ch), G.act);
            if (w.j < 4) R::set(sy[k], 4 * n + w.q, w.ch, yy);
        });
    }
    if (p.t0 < p.t1) {
        __syncthreads();
        const int t = p.t0 + (p.t1 - p.t0 - 1) / TT * TT;
        R::flush(sy[k ^ 1], wy, t, p.t1 - t, width);
    }
    if (state_out && p.t1 == G.seq.end(p.s)) store_states(state_out + srow, h, 4 * w.j, G.N, w.live);
}

// What a run leaves of a zero state (ends; in the forward pass of all but a sequence's last
// run, which no other begins with: 4096 x 1024 x 64 147 -> 143 us), the sum of its step
// widths (width), and with BACK the gradient that its outputs leave at the state before it (back): there
// token t counts c dy times the decays of all tokens from the run's first to it.  Four tokens'
// c dy are led back to the first of them as k_grad does it, and from there to the run's first
// by e^(D a), D the widths before them, as the square of its root: where states grow it may
// pass fp32's range while what it meets is zero or small.
template <class DT, int LPC, bool BACK>
__global__ void __launch_bounds__(THREADS) k_ends(ScanGeo G, ScanIn in, float *ends, float *width, float *back) {
    using X = typename DT::X;
    using R = Rows<DT, LPC>;
    using S = Shared<DT, LPC>;
    constexpr int B = BACK ? 1 : 0;
    __shared__ __align__(16) X sx[2][R::SIZE], sd[2][R::SIZE], sy[B + 1][B ? R::SIZE : 8], sz[B + 1][B ? R::SIZE : 8];
    __shared__ __align__(16) float sb[2][S::SIZE], sc[B + 1][B ? S::SIZE : 4];
    const uint32_t id = spread<LPC>(blockIdx.x, gridDim.x);
    const ScanLane<LPC> w(G, id % G.nblk);
    const Piece p = piece(G, id / G.nblk);
    if (p.t0 >= p.t1 || (!BACK && p.t1 == G.seq.end(p.s))) return;
    float a2[4], h[4], g[4], sum = 0.0f, half = 0.0f;  // half of D
    load_rates(a2, in.a, G, w.c, 4 * w.j, w.live);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = g[i] = 0.0f;
    const float bias = in.bias && w.live ? in.bias[w.c] : 0.0f;
    const Walk<X> wx = R::walk(in.x, in.ldx, w.c0), wd = R::walk(in.dt, in.lddt, w.c0), wz = R::walk(in.gate, in.ldgate, w.c0),
                  wy = R::walk(in.dy, in.lddy, w.c0), wb = S::walk(in.b, in.ldb, w.g * G.N, G.N),
                  wc = S::walk(in.c, in.ldc, w.g * G.N, G.N);
    const int chans = w.cend - w.c0;
    R rx, rd, ry, rz;
    S rb, rc;
    auto fetch = [&](int t) {
        const int cnt = min(TT, p.t1 - t);
        rx.fetch(wx, t, cnt, chans);
        rd.fetch(wd, t, cnt, chans);
        rb.fetch(wb, t, cnt);
        if (BACK) {
            ry.fetch(wy, t, cnt, chans);
            if (in.gate) rz.fetch(wz, t, cnt, chans);
            rc.fetch(wc, t, cnt);
        }
    };
    int k = 0;
    fetch(p.t0);
    for (int t = p.t0; t < p.t1; t += TT, k ^= 1) {
        rx.put(sx[k]);
        rd.put(sd[k]);
        rb.put(sb[k], G.N);
        if (BACK) {
            ry.put(sy[k & B]);
            if (in.gate) rz.put(sz[k & B]);
            rc.put(sc[k & B], G.N);
        }
        __syncthreads();
        if (p.t1 - t > TT) fetch(t + TT);
        const int cnt = min(TT, p.t1 - t);
        const Own<DT, LPC> own(sx[k], sd[k], w, bias, G.soft, cnt);
        quads(cnt, [&](int n) {
            sum += own.d[n];
            float dy[4], es[4][4];
            if (BACK) {
                dy[n] = R::get(sy[k & B], 4 * n + w.q, w.ch);
                if (in.gate) dy[n] *= gate_value<DT>(R::get(sz[k & B], 4 * n + w.q, w.ch), G.act);
            }
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const float ds = of_token(own.d, 4 * n + s), us = of_token(own.u, 4 * n + s);
                float bv[4];
                S::get(bv, sb[k], 4 * n + s, w.j);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    es[s][i] = __builtin_amdgcn_exp2f(ds * a2[i]);
                    h[i] = __builtin_fmaf(es[s][i], h[i], us * bv[i]);
                }
            }
            if (BACK) {
                float back4[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int s = 3; s >= 0; --s) {
                    const float ys = of_token(dy, 4 * n + s);
                    float cv[4];
                    S::get(cv, sc[k & B], 4 * n + s, w.j);
#pragma unroll
                    for (int i = 0; i < 4; ++i) back4[i] = es[s][i] * __builtin_fmaf(cv[i], ys, back4[i]);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    // at most 2^127 as in grown(); a width or rate that is NaN has made g NaN by now
                    const float root = __builtin_amdgcn_exp2f(fminf(half * a2[i], 127.0f));
                    g[i] = __builtin_fmaf(back4[i] * root, root, g[i]);
                }
                const float two = own.d[n] + dpp<0xB1>(own.d[n]);
                half = __builtin_fmaf(two + dpp<0x4E>(two), 0.5f, half);
            }
        });
    }
    const int64_t at = ((int64_t)id * THREADS + threadIdx.x) * 4;
    store_f32<F32, 4>(ends + at, h);
    if (BACK) store_f32<F32, 4>(back + at, g);
    sum += dpp<0xB1>(sum);
    sum += dpp<0x4E>(sum);
    if (w.j == 0) width[(int64_t)id * ScanLane<LPC>::CPW + w.ch] = sum;
}

// Walks the runs of a sequence: `ends` becomes the state before each run, `back` the
// gradient of the state after it.  Sixteen runs are on their way at a time (79 runs of 2048
// channels 11.4 us; with sixteen more on their way 12.6, a wavefront a workgroup 10.9).
// Forward, what stands for the last run is read and not used: its end is k_out's.
// A run in which states grow may have a factor beyond fp32's range.  Sixteen runs with such a
// one are walked again with factors in two parts: a state of zero stays zero, and a small one
// is where it should be.  (Always in two parts 16.2 us.)
template <int LPC, bool BACK>
__global__ void __launch_bounds__(THREADS)
    k_join(ScanGeo G, const float *a, const float *state_in, float *state_out, const float *dstate_out, float *dstate_in,
           float *ends, const float *width, float *back) {
    constexpr int U = 16, CPW = ScanLane<LPC>::CPW;
    const uint32_t cb = blockIdx.x % G.nblk;
    const int s = (int)(blockIdx.x / G.nblk);
    const ScanLane<LPC> w(G, cb);
    float a2[4], v[4];
    load_rates(a2, a, G, w.c, 4 * w.j, w.live);
    const int64_t srow = ((int64_t)s * G.C + (w.live ? w.c : 0)) * G.N;
    const int64_t base = slot_base(G, s), runs = ((int64_t)G.seq.end(s) - G.seq.begin(s) + G.CH - 1) / G.CH;
    const int64_t row = (int64_t)G.nblk * THREADS * 4;  // floats between two runs
    auto walk = [&](float *p, bool down) {
        const int64_t first = base + (down && runs ? runs - 1 : 0), by = down ? -1 : 1;
        float *out = p + (first * G.nblk + cb) * THREADS * 4 + threadIdx.x * 4;
        const float *in = out, *wd = width + (first * G.nblk + cb) * CPW + w.ch;
        for (int64_t r = 0; r < runs; r += U) {
            float e[U][4], d[U];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                load_f32<F32, 4>(e[i], in);
                d[i] = *wd;
                if (r + i + 1 < runs) in += by * row, wd += by * G.nblk * CPW;
            }
            // f: v over a run of width d, for state n
            auto over = [&](auto f) {
#pragma unroll
                for (int i = 0; i < U; ++i) {
                    if (r + i >= runs) break;
                    store_f32<F32, 4>(out + i * by * row, v);
#pragma unroll
                    for (int n = 0; n < 4; ++n) v[n] = f(d[i] * a2[n], v[n], e[i][n]);
                }
            };
            float first[4], top = 0.0f;
#pragma unroll
            for (int n = 0; n < 4; ++n) first[n] = v[n];
            over([&](float p, float s, float end) {
                const float decay = __builtin_amdgcn_exp2f(p);
                top = fmaxf(top, decay);
                return __builtin_fmaf(decay, s, end);
            });
            if (__any(top == __builtin_inff())) {
#pragma unroll
                for (int n = 0; n < 4; ++n) v[n] = first[n];
                over([&](float p, float s, float end) {
                    return __builtin_fmaf(grown(p), s * grown(p > 127.0f ? p - 127.0f : 0.0f), end);
                });
            }
            out += U * by * row;
        }
    };
    load_states(v, state_in ? state_in + srow : nullptr, 4 * w.j, G.N, w.live && state_in);
    walk(ends, false);
    if (state_out && !runs) store_states(state_out + srow, v, 4 * w.j, G.N, w.live);
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
    float *kept;            // states before each block of HT tokens
    float *part;            // channel blocks x tokens x 2 x NP: db, dc
    float *pa, *ps;         // walkers x channel blocks x (256 x 4: da; 2 x CPW: dskip, dbias)
};

template <class DT, int LPC, bool GATE>
__global__ void __launch_bounds__(THREADS, 2)
    k_grad(ScanGeo G, ScanIn in, Out o, const float *state_in, const float *dstate_out, float *dstate_in, const float *starts,
           const float *afters) {
    using X = typename DT::X;
    using R = Rows<DT, LPC>;
    using S = Shared<DT, LPC>;
    using A = Across<LPC>;
    constexpr int NP = 4 * LPC, CPW = THREADS / LPC;
    constexpr int ROUND = LPC <= 8 ? 16 : LPC == 16 ? 8 : 4;  // tokens whose sums over channels LDS holds (16 KB)
    __shared__ __align__(16) X sx[2][R::SIZE], sd[2][R::SIZE], sy[2][R::SIZE], sz[2][GATE ? R::SIZE : 8];
    __shared__ __align__(16) float sb[2][S::SIZE], sc[2][S::SIZE];
    __shared__ float red[4][ROUND * 2 * NP];
    uint32_t id = spread<LPC>(blockIdx.x, gridDim.x);
    if (G.walkers == G.slots) longest_first(G, id, gridDim.x);
    const uint32_t cb = id % G.nblk, walker = id / G.nblk;
    const ScanLane<LPC> w(G, cb);
    const int lane = (int)threadIdx.x & 63, wave = (int)threadIdx.x >> 6;
    float a2[4], da[4] = {0.0f, 0.0f, 0.0f, 0.0f}, dskip = 0.0f, dbias = 0.0f;
    load_rates(a2, in.a, G, w.c, 4 * w.j, w.live);
    const float bias = in.bias && w.live ? in.bias[w.c] : 0.0f, skip = in.skip && w.live ? in.skip[w.c] : 0.0f;
    int m = 0;  // the half of LDS that the tile has
    for (uint32_t slot = walker; slot < G.slots; slot += G.walkers) {
        const Piece p = piece(G, slot);
        if (G.CH && p.t0 >= p.t1) continue;
        const int64_t srow = ((int64_t)p.s * G.C + (w.live ? w.c : 0)) * G.N;
        const int64_t mine = ((int64_t)slot * G.nblk + cb) * THREADS + threadIdx.x;
        const int begin = uniform(G.seq.begin(p.s));
        // the kept state of the block of HT tokens that begins at token t
        auto kept = [&](int t) {
            const int64_t block = (int64_t)(begin / HT) + p.s + (t - begin) / HT;
            return o.kept + ((block * G.nblk + cb) * THREADS + threadIdx.x) * 4;
        };
        float h[4], g[4];
        if (starts) load_f32<F32, 4>(h, starts + mine * 4);
        else load_states(h, state_in ? state_in + srow : nullptr, 4 * w.j, G.N, w.live && state_in);
        if (afters) load_f32<F32, 4>(g, afters + mine * 4);
        else load_states(g, dstate_out ? dstate_out + srow : nullptr, 4 * w.j, G.N, w.live && dstate_out);
        const Walk<X> wx = R::walk(in.x, in.ldx, w.c0), wd = R::walk(in.dt, in.lddt, w.c0),
                      wz = R::walk(in.gate, in.ldgate, w.c0), wy = R::walk(in.dy, in.lddy, w.c0),
                      wb = S::walk(in.b, in.ldb, w.g * G.N, G.N), wc = S::walk(in.c, in.ldc, w.g * G.N, G.N);
        const int width = w.cend - w.c0;
        R rx, rd, ry, rz;
        S rb, rc;
        // forward to the last block, keeping the states before each
        auto fetch_in = [&](int t) {
            const int cnt = min(TT, p.t1 - t);
            rx.fetch(wx, t, cnt, width);
            rd.fetch(wd, t, cnt, width);
            rb.fetch(wb, t, cnt);
        };
        if (p.t0 + HT < p.t1) fetch_in(p.t0);
        for (int t = p.t0; t + HT < p.t1; t += TT, m ^= 1) {
            rx.put(sx[m]);
            rd.put(sd[m]);
            rb.put(sb[m], G.N);
            __syncthreads();
            if (t + TT + HT < p.t1) fetch_in(t + TT);
            const Own<DT, LPC> own(sx[m], sd[m], w, bias, G.soft, min(TT, p.t1 - t));
#pragma unroll
            for (int s = 0; s < TT; ++s) {
                if (s % HT == 0) {
                    if (t + s + HT >= p.t1) break;
                    store_f32<F32, 4>(kept(t + s), h);
                }
                const float ds = of_token(own.d, s), us = of_token(own.u, s);
                float bv[4];
                S::get(bv, sb[m], s, w.j);
#pragma unroll
                for (int i = 0; i < 4; ++i) h[i] = __builtin_fmaf(__builtin_amdgcn_exp2f(ds * a2[i]), h[i], us * bv[i]);
            }
        }
        // back over the blocks
        auto fetch = [&](int t) {
            const int cnt = min(TT, p.t1 - t);
            rx.fetch(wx, t, cnt, width);
            rd.fetch(wd, t, cnt, width);
            ry.fetch(wy, t, cnt, width);
            if (GATE) rz.fetch(wz, t, cnt, width);
            rb.fetch(wb, t, cnt);
            rc.fetch(wc, t, cnt);
        };
        const int tl = p.t1 > p.t0 ? p.t0 + (p.t1 - p.t0 - 1) / TT * TT : p.t0;  // the last tile
        if (p.t0 < p.t1) fetch(tl);
        for (int t = tl; t >= p.t0 && p.t0 < p.t1; t -= TT, m ^= 1) {
            const int cnt = min(TT, p.t1 - t);
            rx.put(sx[m]);
            rd.put(sd[m]);
            ry.put(sy[m]);
            if (GATE) rz.put(sz[m]);
            rb.put(sb[m], G.N);
            rc.put(sc[m], G.N);
            __syncthreads();
            if (t > p.t0) fetch(t - TT);
            const Own<DT, LPC> own(sx[m], sd[m], w, bias, G.soft, cnt);
            float v[A::V];
            const int first = A::first(lane);
            // the tokens of quads K and K + 1, the last first
            auto block = [&](auto quad_of) {
                constexpr int K = decltype(quad_of)::value;
                // the block's states and decays
                float h0[4], hs[HT][4], es[HT][4], dy[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) h0[i] = h[i];
                if (t + 4 * K > p.t0) load_f32<F32, 4>(h, kept(t + 4 * K - HT));  // for the next block
#pragma unroll
                for (int k = K; k < K + 2; ++k) {
                    dy[k] = R::get(sy[m], 4 * k + w.q, w.ch);
                    float y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int s = 0; s < 4; ++s) {
                        const int n = 4 * k + s, l = n - 4 * K;
                        const float ds = of_token(own.d, n), us = of_token(own.u, n);
                        float bv[4], cv[4];
                        S::get(bv, sb[m], n, w.j);
                        if (GATE) S::get(cv, sc[m], n, w.j);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            es[l][i] = __builtin_amdgcn_exp2f(ds * a2[i]);
                            hs[l][i] = __builtin_fmaf(es[l][i], l ? hs[l ? l - 1 : 0][i] : h0[i], us * bv[i]);
                            if (GATE) y[s] = __builtin_fmaf(hs[l][i], cv[i], y[s]);
                        }
                    }
                    if (GATE) {
                        float gs;
                        const float gv = gate_value<DT>(R::get(sz[m], 4 * k + w.q, w.ch), G.act, gs);
                        const float yy = __builtin_fmaf(skip, own.x[k], sum_states4<LPC>(y, w.q));
                        if (w.j < 4) R::set(sz[m], 4 * k + w.q, w.ch, dy[k] * yy * gs);
                        dy[k] *= gv;
                    }
                }
                // back over its tokens
#pragma unroll
                for (int k = K + 1; k >= K; --k) {
                    float vu[4] = {0.0f, 0.0f, 0.0f, 0.0f}, vd[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int s = 3; s >= 0; --s) {
                        const int n = 4 * k + s, l = n - 4 * K, to = n % A::TOK * 8;
                        const float ds = of_token(own.d, n), us = of_token(own.u, n), ys = of_token(dy, n);
                        float bv[4], cv[4];
                        S::get(bv, sb[m], n, w.j);
                        S::get(cv, sc[m], n, w.j);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            g[i] = __builtin_fmaf(cv[i], ys, g[i]);
                            v[to + i] = g[i] * us;
                            v[to + 4 + i] = hs[l][i] * ys;
                            vu[s] = __builtin_fmaf(g[i], bv[i], vu[s]);
                            g[i] *= es[l][i];
                            const float gh = g[i] * (l ? hs[l ? l - 1 : 0][i] : h0[i]);
                            vd[s] = __builtin_fmaf(gh, a2[i], vd[s]);
                            da[i] = __builtin_fmaf(gh, ds, da[i]);
                        }
                        if (n % A::TOK == 0) {
                            A::sum(v, lane);
#pragma unroll
                            for (int r = 0; r < A::R; ++r) {
                                const int i = first + r, tok = n % ROUND + i / 8;
                                red[wave][(tok * 2 + i / 4 % 2) * NP + 4 * w.j + i % 4] = v[r];
                            }
                        }
                    }
                    const float du = sum_states4<LPC>(vu, w.q), dd = sum_states4<LPC>(vd, w.q);
                    // tokens past the end have d = dy = 0: they add nothing
                    const float dw = __builtin_fmaf(du, own.x[k], dd * LN2) * own.slope[k];
                    dbias += 4 * k + w.q < cnt ? dw : 0.0f;
                    dskip = __builtin_fmaf(dy[k], own.x[k], dskip);
                    if (w.j < 4) {
                        R::set(sx[m], 4 * k + w.q, w.ch, __builtin_fmaf(du, own.d[k], skip * dy[k]));
                        R::set(sd[m], 4 * k + w.q, w.ch, dw);
                    }
                    if (4 * k % ROUND == 0) {
                        __syncthreads();
                        for (int i = threadIdx.x; i < ROUND * 2 * NP; i += THREADS) {
                            const int tok = t + 4 * k + i / (2 * NP);
                            const float sum = (red[0][i] + red[1][i]) + (red[2][i] + red[3][i]);
                            if (tok < p.t1) o.part[((int64_t)cb * G.seq.tokens + tok) * (2 * NP) + i % (2 * NP)] = sum;
                        }
                        if (k) __syncthreads();  // the next tile's first barrier stands behind the last round
                    }
                }
            };
            if (cnt > HT) block(std::integral_constant<int, 2>());
            block(std::integral_constant<int, 0>());
            R::flush(sx[m], R::walk(o.dx, o.lddx, w.c0), t, cnt, width);
            R::flush(sd[m], R::walk(o.ddt, o.ldddt, w.c0), t, cnt, width);
            if (GATE && o.dgate) R::flush(sz[m], R::walk(o.dgate, o.lddgate, w.c0), t, cnt, width);
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
    auto channel = [&](uint32_t cb, int ch) {  // -1: none
        const int c = (int)(cb % G.per_group) * CPW + ch;
        return c < G.cg ? (int)(cb / G.per_group) * G.cg + c : -1;
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
    // Whole sequences where they give each CU a workgroup, and in the forward pass two
    // where there are several long ones, whose lengths may differ.  Else runs of as many
    // tokens as give a CU six (four in the gradients).  N = 16, whole sequences and runs:
    // 16384 and 32768 channels x 2048 tokens 220 and 312 us, 246 and 479; two sequences of
    // 150 tokens, 8192 channels 29 and 38; four of 593 to 1266, 1024 channels, N = 64, 160
    // and 142; gradients of four of 297 to 633 tokens, 4096 channels, 229 and 253.  The host
    // knows no lengths but the average: one sequence of 16000 tokens, 2048 channels, takes 248
    // us in runs and 1690 beside fifteen of 32 tokens, whole (gradients 770, and 5470 from
    // seven of them on).
    const int64_t blocks = (int64_t)seqs * G.nblk, want = back ? 1024 : 1536;
    const bool ragged = !back && seqs > 1 && tokens / seqs >= 512;
    if (seqs > 0 && blocks < (ragged ? 512 : 256)) {
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
        z.kept = ((size_t)G.seq.tokens / HT + G.seq.seqs) * block;
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
    (a.gate ? k_out<DT, LPC, true> : k_out<DT, LPC, false>)<<<(uint32_t)blocks, THREADS, 0, st>>>(
        G, in, a.state_in, starts, a.state_out, (typename DT::X *)a.y, a.ldy);
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
        (a.gate ? k_grad<DT, LPC, true> : k_grad<DT, LPC, false>)<<<(uint32_t)walks, THREADS, 0, st>>>(
            G, in, o, a.state_in, a.dstate_out, a.dstate_in, G.CH ? ends : nullptr, G.CH ? back : nullptr);
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
