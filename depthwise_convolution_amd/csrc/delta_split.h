// delta_split.h -- fp32 values as bf16 terms on the 16-bit matrix cores: what
// the gated delta rule's kernels for bf16 and fp16 data share.
#pragma once

#include <type_traits>

#include "delta_common.h"

namespace dw {
namespace delta {
namespace {

using bf16x8 = __attribute__((ext_vector_type(8))) __bf16;
using f16x8 = __attribute__((ext_vector_type(8))) _Float16;
using f32x8 = __attribute__((ext_vector_type(8))) float;
using u32x4 = __attribute__((ext_vector_type(4))) uint32_t;
using u32x2 = __attribute__((ext_vector_type(2))) uint32_t;

__device__ __forceinline__ f32x4 mfma32(bf16x8 a, bf16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

using bf16x2 = __attribute__((ext_vector_type(2))) __bf16;
using f32x2 = __attribute__((ext_vector_type(2))) float;

// a and b split into N bf16 terms, each the nearest of what is left, in pairs.
// (On the words: conversions of single values would be made a second time.)
template <int N>
__device__ __forceinline__ void split(float a, float b, uint32_t (&t)[N]) {
// a product is rounded before it is split, so that the same value has the same terms everywhere
#pragma clang fp contract(off)
#pragma unroll
    for (int n = 0; n < N; ++n) {
        t[n] = __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a, b}), bf16x2));
        if (n + 1 < N) {
            a -= __uint_as_float(t[n] << 16);
            b -= __uint_as_float(t[n] & 0xffff0000u);
        }
    }
}
template <int N>
__device__ __forceinline__ void split(f32x4 x, u32x2 (&t)[N]) {
    uint32_t lo[N], hi[N];
    split(x[0], x[1], lo);
    split(x[2], x[3], hi);
#pragma unroll
    for (int n = 0; n < N; ++n) t[n] = u32x2{lo[n], hi[n]};
}
template <int N>
__device__ __forceinline__ void split(f32x4 a, f32x4 b, bf16x8 (&t)[N]) {
    u32x2 lo[N], hi[N];
    split(a, lo);
    split(b, hi);
#pragma unroll
    for (int n = 0; n < N; ++n) t[n] = __builtin_bit_cast(bf16x8, (u32x4{lo[n][0], lo[n][1], hi[n][0], hi[n][1]}));
}

// Keeps loads in front of the products that hide them.
__device__ __forceinline__ void fence() { __builtin_amdgcn_sched_barrier(0); }

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

// c += products of NA terms times NB terms down to order `last` (term i times
// term j has order i + j), for NT neighbouring column tiles
template <int NA, int NB, int NT>
__device__ __forceinline__ void mac(const bf16x8 (&a)[NA], const bf16x8 (&b)[NT][NB], int last, f32x4 (&c)[NT]) {
#pragma unroll
    for (int o = 0; o < NA + NB - 1; ++o) {
        if (o > last) break;
#pragma unroll
        for (int i = 0; i < NA; ++i)
            if (o - i >= 0 && o - i < NB) {
#pragma unroll
                for (int t = 0; t < NT; ++t) c[t] = mfma32(a[i], b[t][o - i], c[t]);
            }
    }
}

// the place of block (m, kb) among a triangle's six
__device__ __forceinline__ int lower_block(int m, int kb) { return m < 2 ? m : 2 * (m - 1) + kb; }
__device__ __forceinline__ int upper_block(int m, int kb) { return m < 2 ? 2 * m + kb : 2 + m; }
// the row tile and term block of a lower triangle's six blocks (kb <= m / 2),
// and of an upper one's (kb >= m / 2)
__host__ __device__ constexpr int lower_m(int blk) { return blk < 2 ? blk : blk / 2 + 1; }
__host__ __device__ constexpr int lower_kb(int blk) { return blk < 2 ? 0 : blk % 2; }
__host__ __device__ constexpr int upper_m(int blk) { return blk < 4 ? blk / 2 : blk - 2; }
__host__ __device__ constexpr int upper_kb(int blk) { return blk < 4 ? blk % 2 : 1; }

// A wavefront's left operands from the workspace: N fragments' terms.
template <int N>
__device__ __forceinline__ void fetch(bf16x8 (&w)[N], const char *p, int lane) {
    const uint32_t off = (uint32_t)lane * 16;
#pragma unroll
    for (int n = 0; n < N; ++n) w[n] = *(const bf16x8 *)(p + n * FRAG + off);
}

// Right operands in LDS: [block of 32 terms][column tile][term], a fragment
// each.  A wavefront writes a tile's terms (half of a block: `half`) and reads
// whole blocks.
template <int NT, int TERMS>
struct Right {
    char *p;
    static constexpr int bytes(int blocks) { return blocks * NT * TERMS * FRAG; }
    __device__ __forceinline__ void put(int tile, int t, f32x4 x, int lane) const {
        u32x2 v[TERMS];
        split(x, v);
#pragma unroll
        for (int n = 0; n < TERMS; ++n)
            *(u32x2 *)(p + ((tile / 2 * NT + t) * TERMS + n) * FRAG + lane * 16 + tile % 2 * 8) = v[n];
    }
    template <int N>
    __device__ __forceinline__ void get(int blk, bf16x8 (&v)[NT][N], int lane) const {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int n = 0; n < N; ++n) v[t][n] = *(const bf16x8 *)(p + ((blk * NT + t) * TERMS + n) * FRAG + lane * 16);
    }
};

hipError_t lds_room(const void *f, size_t bytes) {
    return hipFuncSetAttribute(f, hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

// Calls f with the type and the padded key size.
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
    switch (DK) {
        case 64: return f(F16{}, std::integral_constant<int, 64>{});
        case 128: return f(F16{}, std::integral_constant<int, 128>{});
        case 192: return f(F16{}, std::integral_constant<int, 192>{});
        default: return f(F16{}, std::integral_constant<int, 256>{});
    }
}

}  // namespace
}  // namespace delta
}  // namespace dw
