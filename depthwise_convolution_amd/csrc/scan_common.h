// scan_common.h -- what the selective scan's kernels share: lanes and their states,
// the step width, geometry.
#pragma once

#include "seq_common.h"
#include "seq_plan.h"

namespace dw {

constexpr float LOG2E = 1.44269504f, LN2 = 0.693147182f;

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}
// zero outside the banks (quads of a row) of the mask
template <int CTRL, int BANKS>
__device__ __forceinline__ float dpp_banks(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, BANKS, false));
}
// the value of lane S of each quad
template <int S>
__device__ __forceinline__ float quad(float v) { return dpp<S * 0x55>(v); }

// v, w -> (rows 0 and 2 of both, rows 1 and 3 of both) and (lower halves, upper halves)
__device__ __forceinline__ void swap16(float &v, float &w) {
    const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, w), false, false);
    v = __builtin_bit_cast(float, (uint32_t)r[0]);
    w = __builtin_bit_cast(float, (uint32_t)r[1]);
}
__device__ __forceinline__ void swap32(float &v, float &w) {
    const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, w), false, false);
    v = __builtin_bit_cast(float, (uint32_t)r[0]);
    w = __builtin_bit_cast(float, (uint32_t)r[1]);
}

// Sum over the LPC lanes of a channel, in all of them.
template <int LPC>
__device__ __forceinline__ float sum_states(float v) {
    v += dpp<0xB1>(v);                    // lane ^ 1
    v += dpp<0x4E>(v);                    // lane ^ 2
    if (LPC >= 8) v += dpp<0x141>(v);     // the other quad of eight (all of a quad are equal)
    if (LPC >= 16) v += dpp<0x140>(v);    // the other half of the row
    if (LPC >= 32) {
        float w = v;
        swap16(v, w);
        v += w;
    }
    return v;
}

// Of four tokens' values at once: lane q of each quad gets the sum over the channel's
// lanes of token q's value.
template <int LPC>
__device__ __forceinline__ float sum_states4(const float (&v)[4], int q) {
    const bool odd = q & 1, hi = q & 2;
    const float a = (odd ? v[1] : v[0]) + dpp<0xB1>(odd ? v[0] : v[1]);
    const float b = (odd ? v[3] : v[2]) + dpp<0xB1>(odd ? v[2] : v[3]);
    float s = (hi ? b : a) + dpp<0x4E>(hi ? a : b);
    if (LPC == 8) s += dpp_banks<0x104, 0x5>(s) + dpp_banks<0x114, 0xa>(s);  // lane ^ 4
    if (LPC >= 16) {
        s += dpp<0x128>(s);  // eight lanes round
        s += dpp<0x124>(s);  // four
    }
    if (LPC >= 32) {
        float w = s;
        swap16(s, w);
        s += w;
    }
    return s;
}

// softplus(v) = max(v, 0) + ln(1 + t), t = e^-|v| <= 1, and its slope 1 / (1 + e^-v).
// ln(1 + t) is ln w of the rounded w = 1 + t plus what the rounding left, t - (w - 1)
// (over w, but that factor only counts where t is next to 1 and so the rest next to
// nothing): 4 units of 2^-24 of itself where t is, at any t.  t is 2^-h of a rounded
// h = |v| / ln 2, so off by |v| units more, which fp32 data puts right.
template <class DT>
__device__ __forceinline__ float softplus(float v, float &slope) {
    float t = __builtin_amdgcn_exp2f(__builtin_fabsf(v) * -LOG2E);
    if (sizeof(typename DT::X) == 4) {
        const float m = __builtin_fabsf(v), lim = m > 200.0f ? 200.0f : m, h = lim * LOG2E;
        const float r = __builtin_fmaf(h, 1.90465421e-9f, __builtin_fmaf(h, -LN2, lim));
        t = __builtin_amdgcn_exp2f(-h);
        t = __builtin_fmaf(t, -r, t);
    }
    const float w = 1.0f + t, s = __builtin_amdgcn_rcpf(w);
    slope = v < 0.0f ? t * s : s;
    return (v > 0.0f ? v : 0.0f) + __builtin_fmaf(__builtin_amdgcn_logf(w), LN2, t - (w - 1.0f));
}
template <class DT>
__device__ __forceinline__ float step_width(float v, int soft, float &slope) {
    slope = 1.0f;
    return soft ? softplus<DT>(v, slope) : v;
}

struct ScanGeo {
    Packed seq;
    int C, N, G, cg, CH;           // cg channels a group; CH 0: a piece is a whole sequence
    uint32_t per_group, nblk;      // workgroups' channels: so many a group, so many in all
    uint32_t slots, walkers;       // pieces; workgroups that share them
    int soft, act;
};

struct ScanIn {
    const void *x, *dt, *b, *c, *gate, *dy;
    int64_t ldx, lddt, ldb, ldc, ldgate, lddy;
    const float *a, *skip, *bias;
};

// The channels and states of a lane.
template <int LPC>
struct ScanLane {
    static constexpr int CPW = 256 / LPC, NP = 4 * LPC;
    int g, c0, cend, ch, j, q, c;
    bool live;
    __device__ __forceinline__ ScanLane(const ScanGeo &G, uint32_t cb) {
        g = G.G > 1 ? (int)(cb / G.per_group) : 0;
        c0 = g * G.cg + (int)(cb - g * G.per_group) * CPW;
        cend = (g + 1) * G.cg;
        ch = (int)threadIdx.x / LPC;
        j = (int)threadIdx.x % LPC;
        q = (int)threadIdx.x & 3;
        c = c0 + ch;
        live = c < cend;
    }
};

// Four states at state index 4 j of a row of N; past N and for idle lanes zeros.
__device__ __forceinline__ void load_states(float (&v)[4], const float *row, int n0, int N, bool live) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = 0.0f;
    if (!live || n0 >= N) return;
    if ((N & 3) == 0 && ((uintptr_t)row & 15) == 0) {
        load_f32<F32, 4>(v, row + n0);
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (n0 + i < N) v[i] = row[n0 + i];
}
__device__ __forceinline__ void store_states(float *row, const float (&v)[4], int n0, int N, bool live) {
    if (!live || n0 >= N) return;
    if ((N & 3) == 0 && ((uintptr_t)row & 15) == 0) {
        store_f32<F32, 4>(row + n0, v);
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (n0 + i < N) row[n0 + i] = v[i];
}

// a log2 e, finite: a token of width zero (there are such behind the end of a tile)
// has a decay of one whatever the rate
__device__ __forceinline__ void load_rates(float (&v)[4], const float *a, const ScanGeo &G, int c, int n0, bool live) {
    load_states(v, a + (int64_t)(live ? c : 0) * G.N, n0, G.N, live);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float r = v[i] * LOG2E;
        v[i] = r < -3e38f ? -3e38f : r > 3e38f ? 3e38f : r;  // NaN stays
    }
}

// Lanes a channel: four states each, and at least a quad.
inline int scan_lanes(int N) { return N <= 16 ? 4 : N <= 32 ? 8 : N <= 64 ? 16 : 32; }

inline bool too_many(uint64_t blocks) { return blocks >= (1u << 24); }

inline ScanIn scan_inputs(const ScanArgs &a) {
    return {a.x, a.dt, a.b, a.c, a.gate, a.dy, a.ldx, a.lddt, a.ldb, a.ldc, a.ldgate, a.lddy, a.a, a.skip, a.bias};
}


// Blocks of channels: 256 / lpc of one group each, also where a group has fewer (2048 tokens of
// 1024 channels, N = 16: 1 group 33 us, 64 groups 94, 1024 groups of one channel 621).
inline ScanGeo scan_blocks(const dwconv_scan_plan &p, int lpc) {
    ScanGeo G{{nullptr, 0, 0}, p.C, p.N, p.G, p.C / p.G, 0, 0, 0, 0, 0, p.softplus, p.act};
    const int cpw = 256 / lpc;
    G.per_group = (uint32_t)((G.cg + cpw - 1) / cpw);
    G.nblk = G.per_group * (uint32_t)p.G;
    return G;
}

}  // namespace dw
