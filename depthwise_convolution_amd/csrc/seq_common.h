// seq_common.h -- what the sequence operators' kernels share: arguments,
// vectors of elements, packed sequences and activations.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/dwconv_seq.h"
#include "dw_common.h"

namespace dw {

// N consecutive elements moved by one load or store (two of 16 bytes for 32).
template <class X, int N>
struct alignas(sizeof(X) * N > 16 ? 16 : sizeof(X) * N) Vec {
    X v[N];
};

template <class DT, int N>
__device__ __forceinline__ void load_f32(float (&out)[N], const typename DT::X *p) {
    const Vec<typename DT::X, N> a = *(const Vec<typename DT::X, N> *)p;
#pragma unroll
    for (int i = 0; i < N; ++i) out[i] = DT::widen(a.v[i]);
}

// fp32 to the storage type, to nearest even.  bf16 by the conversion instruction
// (NaN stays NaN); the other types as everywhere.
template <class DT>
__device__ __forceinline__ typename DT::X rounded(float v) {
    return DT::narrow(v);
}
template <>
__device__ __forceinline__ uint16_t rounded<BF16>(float v) {
    return __builtin_bit_cast(uint16_t, (__bf16)v);
}

// a value that is the same in all lanes, in a scalar register
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

template <class DT, int N>
__device__ __forceinline__ void store_f32(typename DT::X *p, const float (&in)[N]) {
    Vec<typename DT::X, N> a;
#pragma unroll
    for (int i = 0; i < N; ++i) a.v[i] = rounded<DT>(in[i]);
    *(Vec<typename DT::X, N> *)p = a;
}

// sigmoid(z), and 1 - sigmoid(z) in `rest`.
// 16-bit data: the reciprocal (one unit of 2^-23) and exp2 of a rounded product (|z|
// units of 2^-24, so at most 2^-17 of itself, of which half a step is 2^-9 or 2^-12).
template <class DT>
__device__ __forceinline__ float sigmoid_f32(float z, float &rest) {
    const float p = __builtin_amdgcn_rcpf(1.0f + __expf(-z));
    rest = 1.0f - p;
    return p;
}
// fp32 data: both off by at most 8 units of 2^-24 of themselves wherever they are
// normal numbers.  They come from t = e^-|z| <= 1: no overflow, no difference of near
// values.  t is 2^-h for the rounded h = |z| / ln 2, times 1 - r for what the rounding
// left, r = |z| - h ln 2.  Beyond 200 t is 0 (an infinite |z| would make r NaN).
// For 16-bit data as well it would cost (bf16, before and after) causal gradients of
// 8192 x 8192 93.7 and 100.5 us, gated norms of 262144 x 128 35.5 and 38.0 us.
template <>
__device__ __forceinline__ float sigmoid_f32<F32>(float z, float &rest) {
    const float m = __builtin_fabsf(z), a = m > 200.0f ? 200.0f : m, h = a * 1.44269504f;
    const float r = __builtin_fmaf(h, 1.90465421e-9f, __builtin_fmaf(h, -0.693147182f, a));
    float t = __builtin_amdgcn_exp2f(-h);
    t = __builtin_fmaf(t, -r, t);
    const float s = __builtin_amdgcn_rcpf(1.0f + t);
    rest = z < 0.0f ? s : t * s;
    return z < 0.0f ? t * s : s;
}
template <class DT>
__device__ __forceinline__ float sigmoid_f32(float z) {
    float rest;
    return sigmoid_f32<DT>(z, rest);
}

// act(g), and act'(g) in `slope`
template <class DT>
__device__ __forceinline__ float gate_value(float g, int act, float &slope) {
    float rest;
    const float p = sigmoid_f32<DT>(g, rest), q = p * rest;
    slope = act == DWCONV_SEQ_ACT_NONE ? 1.0f : act == DWCONV_SEQ_ACT_SILU ? __builtin_fmaf(g, q, p) : q;
    return act == DWCONV_SEQ_ACT_NONE ? g : act == DWCONV_SEQ_ACT_SILU ? g * p : p;
}
template <class DT>
__device__ __forceinline__ float gate_value(float g, int act) {
    float slope;
    return gate_value<DT>(g, act, slope);
}

// v plus the value n lanes round in each row of 16 (one instruction).
template <int N>
__device__ __forceinline__ float add_ror(float v) {
    return v + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x120 + N, 0xf, 0xf, true));
}
// sum over each row of 16 lanes, in all of them
__device__ __forceinline__ float sum_row16(float v) { return add_ror<1>(add_ror<2>(add_ror<4>(add_ror<8>(v)))); }
// sum over the wavefront, in all lanes
__device__ __forceinline__ float sum_wave(float v) {
    const int x = __builtin_bit_cast(int, sum_row16(v));
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < 64; i += 16) s += __builtin_bit_cast(float, __builtin_amdgcn_readlane(x, i));
    return s;
}

// Packed sequences.  Wrong offsets are clamped, so that begin <= end lie in
// [0, tokens] whatever the device array holds.
struct Packed {
    const int32_t *offsets;  // seqs + 1, or nullptr: one sequence of all tokens
    int seqs, tokens;
    __device__ __forceinline__ int begin(int s) const {
        if (!offsets) return 0;
        const int a = offsets[s];
        return a < 0 ? 0 : (a > tokens ? tokens : a);
    }
    __device__ __forceinline__ int end(int s) const {
        if (!offsets) return tokens;
        const int a = begin(s), b = offsets[s + 1];
        return b < a ? a : (b > tokens ? tokens : b);
    }
    // The last sequence s with offsets[s] <= t, -1 if there is none.  Of
    // several that begin at t it is the last, so the one that may hold t.
    __device__ __forceinline__ int find(int t) const {
        if (!offsets) return 0;
        int lo = -1, hi = seqs;  // offsets[lo] <= t < offsets[hi], hi past the end
        while (hi - lo > 1) {
            const int m = lo + ((hi - lo) >> 1);  // (lo + hi may pass 2^31)
            if (offsets[m] <= t) lo = m; else hi = m;
        }
        return lo;
    }
    // From sequence s, which ends at or before t, to the one that may hold t: the next
    // one as a rule, else by the search (any number of empty ones may lie between).
    __device__ __forceinline__ void advance(int t, int &s, int &a, int &b) const {
        if (s + 1 < seqs && end(s + 1) > t) ++s;
        else s = find(t);
        if (s < 0) {
            a = b = 0;
            return;
        }
        a = begin(s);
        b = end(s);
    }
};

// Which rows of a step share this row's cache entry.  Rows with the same slot
// are consecutive tokens of one sequence: the first one's workgroup takes them
// all in order, the others' workgroups leave.
struct SlotRows {
    int slot;     // -1: nothing to do
    bool shared;  // later rows have it too
};
__device__ __forceinline__ SlotRows slot_rows(const int32_t *slots, int n_slots, int rows, int row) {
    if (!slots) return {row, false};
    const int s = slots[row];
    if (s < 0 || s >= n_slots) return {-1, false};
    bool before = false, after = false;
    for (int j = threadIdx.x & 63; j < rows; j += 64) {
        const bool same = slots[j] == s;
        before |= same && j < row;
        after |= same && j > row;
    }
    if (__any(before)) return {-1, false};
    return {s, (bool)__any(after)};
}

}  // namespace dw
