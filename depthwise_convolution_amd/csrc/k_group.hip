// k_group.hip -- norm over groups of channels of an image, with an activation
// (include/dwconv_seq.h): forward and gradients.
//
//   u = (x - mean) r,  r = 1 / sqrt(var + eps)      y = act(z), z = u w + b
//   dz = dy act'(z)    dw = sum dz u    db = sum dz
//   dx = r (dz w - mean(dz w) - u mean(dz w u))     means over the group
//
// A workgroup takes whole groups of channels (a slice) of a run of pixels; a lane one
// vector of 16 bytes of channels, the same for all its pixels, so that sums over pixels
// stay in registers until the lanes' sums meet in LDS.  Mean and squares around it are
// two sums over values in registers: no difference of large sums.  Two ways to run it:
//   resident   an image's slice fits the registers of a workgroup: one launch, every
//              element read and written once
//   in passes  runs of pixels give their mean and squares around it, which k_join puts
//              together; further launches read the image again
//
// Resident: 64 images of 56x56x128 bf16 with silu 25 to 28 us (103 MB, 3.7 to 4.1 TB/s; 19 at
// a copy's rate; loads, sums and stores follow each other in the one workgroup of a CU),
// gradients of 64x56x56x96 fp16 46 and 4 for dw and db (116 MB; vector instructions: with no
// activation 39).  In passes: 2 fp32 images of 256x256x256 84 to 91 us: moments 35 to 39, joins
// 4, outputs 45 (a copy of 134 MB takes 50, a plain reading of them 21 to 29, so that the
// moments are not at the memory's rate); gradients 157: 35, 4, sums 42, joins 4, dx 70.
// Gradients of 16x112x112x61 bf16 without activation 40 to 43: sums 17, joins 9, dx 17.
#include <type_traits>

#include "seq_common.h"
#include "seq_plan.h"

namespace dw {
namespace {

// How an image's channels and pixels are dealt to workgroups.
struct Geo {
    int images, S, C, G, cg;      // S pixels, cg channels a group
    int slices;                   // parts <= 1: slice i has the groups i G / slices up to (i + 1) G / slices
    int parts, part;              // parts > 1: slice i is channels part (i % parts) up of group i / parts
    int vpr, rpp;                 // vectors of a slice's row; rows a workgroup has in hand
    int runs, rows;               // runs of so many pixels an image
    int act;
    float eps;
};

struct Slice {
    int g0, ng, c0, w;  // its first group, groups (1 where it is part of one), channels
};
__device__ __forceinline__ Slice slice_of(const Geo &g, int i) {
    if (g.parts > 1) {
        const int grp = i / g.parts, at = i % g.parts * g.part;
        return {grp, 1, grp * g.cg + at, min(g.part, g.cg - at)};
    }
    const int a = (int)((int64_t)i * g.G / g.slices), b = (int)((int64_t)(i + 1) * g.G / g.slices);
    return {a, b - a, a * g.cg, (b - a) * g.cg};
}

// V elements at any element's alignment, as they come: words that are taken apart where
// they are used (elements would take a register each, and wait for their load).
template <class DT, int V>
struct __attribute__((packed, aligned(sizeof(typename DT::X)))) Any {
    using X = typename DT::X;
    using W = std::conditional_t<V * sizeof(X) % 4 == 0, uint32_t, X>;
    static constexpr int N = V * (int)sizeof(X) / (int)sizeof(W);
    W w[N];
    __device__ __forceinline__ float operator[](int i) const {
        if constexpr (sizeof(W) == sizeof(X)) {
            return DT::widen(__builtin_bit_cast(X, w[i]));
        } else if constexpr (std::is_same_v<DT, BF16>) {
            return __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
        } else {
            return DT::widen(__builtin_bit_cast(X, (uint16_t)(i & 1 ? w[i / 2] >> 16 : w[i / 2])));
        }
    }
};

// A lane's vector of channels.  The last vector of a row ends with the row; what it
// has in common with the one before (`skip` elements) counts there.
template <class DT, int V>
struct Lane {
    using X = typename DT::X;
    int row, c, skip;
    bool live;  // lanes without a vector follow the first one of the first row, and count and write nothing
    __device__ __forceinline__ Lane(const Geo &g, const Slice &s) {
        const int col = (int)threadIdx.x % g.vpr;
        row = (int)threadIdx.x / g.vpr;
        const int at = min(col * V, s.w - V);
        c = s.c0 + at;
        skip = col * V - at;
        live = row < g.rpp && skip < V;
        if (!live) row = 0, skip = V, c = s.c0;
    }
    __device__ __forceinline__ bool counts(int i) const { return i >= skip; }
    static __device__ __forceinline__ Any<DT, V> load(const X *p) { return *(const Any<DT, V> *)p; }
    // `whole`: elements of the vector before may be written too (with the same values)
    __device__ __forceinline__ void store(X *p, const float (&v)[V], bool whole) const {
        if (whole || skip == 0) {
            struct __attribute__((packed, aligned(sizeof(X)))) {
                X v[V];
            } a;
#pragma unroll
            for (int i = 0; i < V; ++i) a.v[i] = rounded<DT>(v[i]);
            *(decltype(a) *)p = a;
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (counts(i)) p[i] = rounded<DT>(v[i]);
        }
    }
};

// z becomes act(z)
template <class DT, int ACT, int V>
__device__ __forceinline__ void activate(float (&z)[V]) {
    if (ACT == DWCONV_GROUP_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < V; ++i) z[i] *= sigmoid_f32<DT>(z[i]);
    } else if (ACT == DWCONV_GROUP_ACT_RELU) {
#pragma unroll
        for (int i = 0; i < V; ++i) z[i] = z[i] < 0.0f ? 0.0f : z[i];  // NaN stays
    }
}
// d times the slope of act at z
template <class DT, int ACT, int V>
__device__ __forceinline__ void back_through(float (&d)[V], const float (&z)[V]) {
    if (ACT == DWCONV_GROUP_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float q;
            const float p = sigmoid_f32<DT>(z[i], q);
            d[i] *= p * __builtin_fmaf(z[i], q, 1.0f);
        }
    } else if (ACT == DWCONV_GROUP_ACT_RELU) {
#pragma unroll
        for (int i = 0; i < V; ++i) d[i] *= z[i] > 0.0f ? 1.0f : z[i] <= 0.0f ? 0.0f : z[i];  // NaN stays
    }
}

// The same words, of which the compiler does not know that it has taken them apart before:
// else it keeps the fp32 values from one use to the next, in twice the registers.
template <class DT, int V, int K>
__device__ __forceinline__ void fresh(Any<DT, V> (&x)[K]) {
    if constexpr (sizeof(typename DT::X) == 2 && V > 1) {
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < Any<DT, V>::N; ++i) {
                uint32_t w = x[k].w[i];
                asm("" : "+v"(w));
                x[k].w[i] = w;
            }
    }
}

// Sums over a workgroup's lanes.  `cols` becomes the sums over rows of each column of the
// slice's vectors, `of_groups` those over the groups' channels.  Every lane calls them; a
// barrier stands at the end of each.
template <int TH, int V>
struct Sums {
    float *lanes, *cols;  // rpp rows of `ld`, a row
    int wide, ld;
    __device__ __forceinline__ Sums(float *sh, const Geo &g) : lanes(sh), wide(g.vpr * V), ld(g.vpr * V + 4) {
        cols = sh + g.rpp * ld;
    }
    template <class L>
    __device__ __forceinline__ void rows(const float (&v)[V], const L &ln, const Geo &g) {
        if ((int)threadIdx.x < g.rpp * g.vpr) {
            float *at = lanes + (int)threadIdx.x / g.vpr * ld + (int)threadIdx.x % g.vpr * V;
#pragma unroll
            for (int i = 0; i < V; ++i) at[i] = ln.live && ln.counts(i) ? v[i] : 0.0f;
        }
        __syncthreads();
        if (g.rpp >= 16) {  // 16 lanes a column, every 16th row each (rows are 4 banks apart)
            const int part = (int)threadIdx.x & 15;
            for (int k = (int)threadIdx.x >> 4; k < (wide + TH / 16 - 1) / (TH / 16) * (TH / 16); k += TH / 16) {
                float s = 0.0f;
                if (k < wide)
                    for (int r = part; r < g.rpp; r += 16) s += lanes[r * ld + k];
                s = sum_row16(s);
                if (part == 0 && k < wide) cols[k] = s;
            }
        } else {
            for (int k = threadIdx.x; k < wide; k += TH) {
                float s = 0.0f;
                for (int r = 0; r < g.rpp; ++r) s += lanes[r * ld + k];
                cols[k] = s;
            }
        }
        __syncthreads();
    }
    // Sum of channel i of the slice: the last vector is moved back by what it shares.
    __device__ __forceinline__ float channel(const Slice &s, int i) const {
        const int last = (s.w + V - 1) / V - 1;
        return cols[i >= last * V ? i + (last + 1) * V - s.w : i];
    }
    // done(j, sum of f(channel) over group j's channels): 16 lanes a group, or a wavefront
    template <class F, class D>
    __device__ __forceinline__ void of_groups(const Slice &s, int cg, F f, D done) {
        const int n = s.ng > 1 ? cg : s.w;
        if (n == 1) {
            for (int j = threadIdx.x; j < s.ng; j += TH) done(j, f(j, channel(s, j)));
        } else if (n <= 16) {
            const int i = (int)threadIdx.x & 15;
            for (int j = (int)threadIdx.x >> 4; j < (s.ng + TH / 16 - 1) / (TH / 16) * (TH / 16); j += TH / 16) {
                const float t = sum_row16(i < n && j < s.ng ? f(j * n + i, channel(s, j * n + i)) : 0.0f);
                if (i == 0 && j < s.ng) done(j, t);
            }
        } else {
            for (int j = (int)threadIdx.x >> 6; j < s.ng; j += TH / 64) {
                float t = 0.0f;
                for (int i = (int)threadIdx.x & 63; i < n; i += 64) t += f(j * n + i, channel(s, j * n + i));
                t = sum_wave(t);
                if (((int)threadIdx.x & 63) == 0) done(j, t);
            }
        }
        __syncthreads();
    }
};

__device__ __forceinline__ float inverse_root(float var, float eps) { return 1.0f / sqrtf(var + eps); }

// A group's mean and r, where a lane's channel i of the slice belongs to it
template <int V>
struct Group {
    int of[V];  // group of the slice, for each of the lane's channels
    template <class L>
    __device__ __forceinline__ Group(const Geo &g, const Slice &s, const L &ln) {
        int at = s.ng > 1 ? ln.c / g.cg - s.g0 : 0, in = s.ng > 1 ? ln.c % g.cg : 0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            of[i] = at;
            if (s.ng > 1 && ++in == g.cg) in = 0, ++at;
        }
    }
};

// A lane's V parameters from channel c on, all at once; `other` where there are none.
template <int V>
__device__ __forceinline__ void params(float (&v)[V], const float *p, int c, float other) {
    if (p) {
        const Any<F32, V> a = *(const Any<F32, V> *)(p + c);
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = a[i];
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = other;
    }
}

// A lane's pixels row, row + rpp ... of a run of n: `whole` of them every lane has, the
// next one the first `rest` rows.  f(k) for each; the test costs no vector instruction
// but for that one.
struct Have {
    int whole;
    bool more;
    template <class L>
    __device__ __forceinline__ Have(const Geo &g, const L &ln, int n) : whole(n / g.rpp), more(ln.row < n % g.rpp) {}
    __device__ __forceinline__ bool has(int k) const { return k < whole || (k == whole && more); }
    template <int K, class F>
    __device__ __forceinline__ void each(F f) const {
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (has(k)) f(k);
    }
    // the same for any number of them, U at a time: fetch(u, k), then use(u, k)
    template <int U, class F, class G>
    __device__ __forceinline__ void stream(F fetch, G use) const {
        int k = 0;
        for (; k + U <= whole; k += U) {
#pragma unroll
            for (int u = 0; u < U; ++u) fetch(u, k + u);
#pragma unroll
            for (int u = 0; u < U; ++u) use(u, k + u);
        }
        for (; k <= whole; ++k)
            if (has(k)) {
                fetch(0, k);
                use(0, k);
            }
    }
};

// The run's or image's mean of each group (in stat) and squares around it (in sq); one lane a
// group calls seen(mean, squares), before a barrier.
template <class DT, int V, int TH, int K, class L, class F>
__device__ __forceinline__ void moments(const Geo &g, const Slice &s, const L &ln, const Group<V> &gr,
                                        Any<DT, V> (&x)[K], int n, const Have &have, Sums<TH, V> &sum, float *stat, float *sq,
                                        float (&mean)[V], F seen) {
    const float count = (float)n * (float)(s.ng > 1 ? g.cg : s.w);
    float v[V];
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = 0.0f;
    have.each<K>([&](int k) {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] += x[k][i];
    });
    sum.rows(v, ln, g);
    sum.of_groups(s, g.cg, [](int, float t) { return t; }, [&](int j, float t) { stat[j] = t / count; });
#pragma unroll
    for (int i = 0; i < V; ++i) mean[i] = stat[gr.of[i]], v[i] = 0.0f;
    fresh(x);
    have.each<K>([&](int k) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float d = x[k][i] - mean[i];
            v[i] = __builtin_fmaf(d, d, v[i]);
        }
    });
    sum.rows(v, ln, g);
    sum.of_groups(s, g.cg, [](int, float t) { return t; }, [&](int j, float t) { sq[j] = t, seen(stat[j], t); });
    fresh(x);
}

// K vectors of a lane
template <class DT, int V, int K>
__device__ __forceinline__ void take(Any<DT, V> (&x)[K], const typename DT::X *p, int64_t step, const Have &have) {
    have.each<K>([&](int k) { x[k] = Lane<DT, V>::load(p + k * step); });
}

// A run's moments of a slice's groups in stats[image][group][run x parts]
__device__ __forceinline__ void leave(const Geo &g, const Slice &s, float2 *stats, int img, int run, int sl, const float *stat,
                                      const float *sq) {
    const int parts = max(g.parts, 1), at = run * parts + (g.parts > 1 ? sl % g.parts : 0);
    for (int j = threadIdx.x; j < s.ng; j += blockDim.x)
        stats[((int64_t)img * g.G + s.g0 + j) * (g.runs * parts) + at] = make_float2(stat[j], sq[j]);
}

// The lanes' two sums of each channel, C apart
template <int TH, int V, class L>
__device__ __forceinline__ void channel_sums(const Geo &g, const Slice &s, const L &ln, Sums<TH, V> &sum, const float (&s1)[V],
                                             const float (&s2)[V], float *out) {
    sum.rows(s1, ln, g);
    for (int i = threadIdx.x; i < s.w; i += TH) out[i] = sum.channel(s, i);
    __syncthreads();
    sum.rows(s2, ln, g);
    for (int i = threadIdx.x; i < s.w; i += TH) out[g.C + i] = sum.channel(s, i);
}

// Forward: resident (RUNS false), or the moments of a run of pixels (RUNS true), left
// as mean and squares in stats[image][group][run x parts].
template <class DT, int V, int TH, int K, bool RUNS, int ACT>
__global__ void __launch_bounds__(TH) k_fwd(Geo g, const typename DT::X *x, int64_t ldx, const float *w, const float *b,
                                            typename DT::X *y, int64_t ldy, float2 *stats, int max_groups) {
    extern __shared__ __align__(16) float sh[];
    Sums<TH, V> sum(sh, g);
    float *stat = sum.cols + sum.wide, *sq = stat + max_groups;
    const uint32_t id = xcd_remap(blockIdx.x, gridDim.x);
    const int sl = (int)(id % g.slices), run = (int)(id / g.slices % g.runs), img = (int)(id / g.slices / g.runs);
    const Slice s = slice_of(g, sl);
    const Lane<DT, V> ln(g, s);
    const Group<V> gr(g, s, ln);
    const int p0 = run * g.rows, n = min(g.rows, g.S - p0);
    const Have have(g, ln, n);
    Any<DT, V> v[K];
    take(v, x + ((int64_t)img * g.S + p0 + ln.row) * ldx + ln.c, g.rpp * ldx, have);
    float mean[V], scale[V], shift[V];
    if (!RUNS) {
        params(scale, w, ln.c, 1.0f);
        params(shift, b, ln.c, 0.0f);
    }
    const float inv = 1.0f / ((float)n * (float)g.cg);
    constexpr bool NEAR = !RUNS && sizeof(typename DT::X) == 2 && ACT != DWCONV_GROUP_ACT_RELU;
    __shared__ int far;  // a mean of 16 deviations or more
    if (NEAR && threadIdx.x == 0) far = 0;
    moments<DT, V, TH, K>(g, s, ln, gr, v, n, have, sum, stat, sq, mean, [&](float m, float q) {
        if (NEAR && !(m * m < 256.0f * __builtin_fmaf(q, inv, g.eps))) far = 1;
    });
    if (RUNS) {
        leave(g, s, stats, img, run, sl, stat, sq);
        return;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) scale[i] *= inverse_root(sq[gr.of[i]] * inv, g.eps);
    y += ((int64_t)img * g.S + p0 + ln.row) * ldy + ln.c;
    const int64_t step = g.rpp * ldy;
    auto outputs = [&](auto z) {
        if (!ln.live) return;
        have.each<K>([&](int k) {
            float o[V];
#pragma unroll
            for (int i = 0; i < V; ++i) o[i] = z(v[k][i], i);
            activate<DT, ACT>(o);
            ln.store(y + k * step, o, true);  // all loads of the slice are behind a barrier
        });
    };
    // 16-bit data whose means are all less than 16 deviations: (x - mean) scale in one operation,
    // off by 16 units of 2^-24 of a deviation (64 images of 56x56x128 bf16 28.2 us, with the
    // difference taken first 30.2).  The same for the workgroup, of which two lanes may write
    // one element; not with a rectifier, whose corner the gradients find by the difference.
    if (NEAR && !uniform(far)) {
#pragma unroll
        for (int i = 0; i < V; ++i) shift[i] = __builtin_fmaf(-mean[i], scale[i], shift[i]);
        outputs([&](float x, int i) { return __builtin_fmaf(x, scale[i], shift[i]); });
    } else {
        outputs([&](float x, int i) { return __builtin_fmaf(x - mean[i], scale[i], shift[i]); });
    }
}

// Two sums over the W wavefronts that share a group, in all of their lanes.
template <int W>
__device__ __forceinline__ void sum_group(float &a, float &b, float *sh) {
    a = sum_wave(a);
    b = sum_wave(b);
    if (W == 1) return;
    const int wave = (int)threadIdx.x >> 6;
    __syncthreads();
    if (((int)threadIdx.x & 63) == 0) sh[wave] = a, sh[16 + wave] = b;
    __syncthreads();
    a = b = 0.0f;
#pragma unroll
    for (int i = 0; i < W; ++i) a += sh[i], b += sh[16 + i];
}

// Puts the moments of a group's runs together: W wavefronts a group.  With counts n_i,
// means m_i and squares q_i: m = m_0 + sum n_i (m_i - m_0) / n, which is m_0 where all are
// equal, and q = sum (q_i + n_i (m_i - m)^2).
// out: mean and r.  part: the sums that k_both has left, or nullptr.
template <int W>
__global__ void __launch_bounds__(W > 4 ? W * 64 : 256) k_join(Geo g, const float2 *stats, float2 *out, float *part) {
    constexpr int TH = W > 4 ? W * 64 : 256;
    __shared__ float sh[32];
    const int64_t id = (int64_t)blockIdx.x * (TH / 64 / W) + (W == 1 ? threadIdx.x >> 6 : 0);
    if (id >= (int64_t)g.images * g.G) return;
    const int lane = (int)threadIdx.x % (64 * W), parts = max(g.parts, 1), per = g.runs * parts;
    const float2 *p = stats + id * per;
    auto count = [&](int i) {
        const int run = i / parts, part = i % parts;
        return (float)min(g.rows, g.S - run * g.rows) * (float)(parts > 1 ? min(g.part, g.cg - part * g.part) : g.cg);
    };
    const float inv = 1.0f / ((float)g.S * (float)g.cg);
    const float m0 = p[0].x;
    float m = 0.0f, q = 0.0f, none = 0.0f;
    for (int i = lane; i < per; i += 64 * W) m = __builtin_fmaf(count(i) * inv, p[i].x - m0, m);
    sum_group<W>(m, none, sh);
    m += m0;
    for (int i = lane; i < per; i += 64 * W) {
        const float d = p[i].x - m;
        q += __builtin_fmaf(count(i) * d, d, p[i].y);
    }
    sum_group<W>(q, none, sh);
    const float r = inverse_root(q * inv, g.eps);
    if (lane == 0) out[id] = make_float2(m, r);
    if (!part) return;
    part += id / g.G * g.runs * 2 * g.C + id % g.G * g.cg;
    for (int run = lane / g.cg, c = lane % g.cg; run < g.runs;) {
        float *at = part + (int64_t)run * 2 * g.C + c;
        at[g.C] = r * __builtin_fmaf(p[run * parts + (parts > 1 ? c / g.part : 0)].x - m, at[0], at[g.C]);
        run += 64 * W / g.cg;
        c += 64 * W % g.cg;
        if (c >= g.cg) c -= g.cg, ++run;
    }
}

// A lane's channels: with d = x - mean, u = d r and z = d scale + shift, scale = r w.  The
// mean is taken from x before any product: x r - mean r would leave a rounding of mean r
// where the deviations are nothing beside the mean (groups of one value, blank images).
template <int V>
struct Known {
    float r[V], mean[V], scale[V], shift[V];
    Known() = default;
    // from mean and r
    __device__ __forceinline__ void ready(const float *w, const float *b, int c) {
        params(scale, w, c, 1.0f);
        params(shift, b, c, 0.0f);
#pragma unroll
        for (int i = 0; i < V; ++i) scale[i] *= r[i];
    }
    template <class L>
    __device__ __forceinline__ Known(const Geo &g, const Slice &s, const L &ln, const float2 *joined, int img, const float *w,
                                     const float *b) {
        const Group<V> gr(g, s, ln);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float2 m = joined[(int64_t)img * g.G + s.g0 + gr.of[i]];
            mean[i] = m.x;
            r[i] = m.y;
        }
        ready(w, b, ln.c);
    }
};

template <class DT, int V, int TH, int U, int ACT>
__global__ void __launch_bounds__(TH) k_apply(Geo g, const typename DT::X *x, int64_t ldx, const float2 *joined,
                                              const float *w, const float *b, typename DT::X *y, int64_t ldy) {
    const uint32_t id = xcd_remap(blockIdx.x, gridDim.x);
    const int sl = (int)(id % g.slices), run = (int)(id / g.slices % g.runs), img = (int)(id / g.slices / g.runs);
    const Slice s = slice_of(g, sl);
    const Lane<DT, V> ln(g, s);
    if (!ln.live) return;
    const int p0 = run * g.rows, n = min(g.rows, g.S - p0);
    const bool apart = (const void *)x != (const void *)y;
    x += ((int64_t)img * g.S + p0 + ln.row) * ldx + ln.c;
    y += ((int64_t)img * g.S + p0 + ln.row) * ldy + ln.c;
    const int64_t sx = g.rpp * ldx, sy = g.rpp * ldy;
    const Known<V> kn(g, s, ln, joined, img, w, b);
    Any<DT, V> v[U];
    Have(g, ln, n).stream<U>([&](int u, int k) { v[u] = Lane<DT, V>::load(x + k * sx); },
                             [&](int u, int k) {
                                 float o[V];
#pragma unroll
                                 for (int i = 0; i < V; ++i) o[i] = __builtin_fmaf(v[u][i] - kn.mean[i], kn.scale[i], kn.shift[i]);
                                 activate<DT, ACT>(o);
                                 ln.store(y + k * sy, o, apart);
                             });
}

// x - mean: of fp16 data in one operation with the conversion, as a product with a one that the
// compiler does not know
template <class DT>
struct Minus {
    float one = 1.0f;
    __device__ __forceinline__ Minus() {
        if constexpr (std::is_same_v<DT, F16>) asm("" : "+s"(one));
    }
    __device__ __forceinline__ float operator()(float x, float mean) const {
        if constexpr (std::is_same_v<DT, F16>) return __builtin_fmaf(x, one, -mean);
        return x - mean;
    }
};

// d and dz of one vector
template <int ACT, class DT, int V>
__device__ __forceinline__ void make_dz(float (&dz)[V], float (&d)[V], const Any<DT, V> &x, const Any<DT, V> &dy,
                                        const Known<V> &kn) {
    float z[V];
    const Minus<DT> minus;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        d[i] = minus(x[i], kn.mean[i]);
        z[i] = __builtin_fmaf(d[i], kn.scale[i], kn.shift[i]);
        dz[i] = dy[i];
    }
    back_through<DT, ACT>(dz, z);
}

// A lane's share of the sums dz and dz d of one vector
template <int ACT, class DT, int V>
__device__ __forceinline__ void add_sums(float (&s1)[V], float (&s2)[V], const Any<DT, V> &x, const Any<DT, V> &dy,
                                         const Known<V> &kn) {
    float dz[V], d[V];
    make_dz<ACT>(dz, d, x, dy, kn);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        s1[i] += dz[i];
        s2[i] = __builtin_fmaf(dz[i], d[i], s2[i]);
    }
}
// sums of dz d to those of dz u; where the squares have left fp32, r and u are 0
template <int V>
__device__ __forceinline__ void of_units(float (&s2)[V], const Known<V> &kn) {
#pragma unroll
    for (int i = 0; i < V; ++i) s2[i] = kn.r[i] == 0.0f ? 0.0f : s2[i] * kn.r[i];
}

// r (dz w - m1 - u m2) as dz scale + d slope + rest
template <int V>
struct Grad {
    float scale[V], slope[V], rest[V];
    __device__ __forceinline__ Grad(const Geo &g, const Known<V> &kn, const float (&m1)[V], const float (&m2)[V]) {
        const bool one = g.cg == 1 && g.S == 1;  // nothing depends on the one value of a group
#pragma unroll
        for (int i = 0; i < V; ++i) {
            scale[i] = one ? 0.0f : kn.scale[i];
            slope[i] = one ? 0.0f : -kn.r[i] * (kn.r[i] * m2[i]);
            rest[i] = one ? 0.0f : -kn.r[i] * m1[i];
        }
    }
    template <int ACT, class DT>
    __device__ __forceinline__ void of(float (&o)[V], const Any<DT, V> &x, const Any<DT, V> &dy, const Known<V> &kn) const {
        float dz[V], d[V];
        make_dz<ACT>(dz, d, x, dy, kn);
#pragma unroll
        for (int i = 0; i < V; ++i) o[i] = __builtin_fmaf(dz[i], scale[i], __builtin_fmaf(d[i], slope[i], rest[i]));
    }
};

// Gradients with x and dy of an image's slice in registers.  sums: [image][2][C], dz and
// dz u over the pixels.
template <class DT, int V, int TH, int K, int ACT>
__global__ void __launch_bounds__(TH) k_resident(Geo g, const typename DT::X *x, int64_t ldx, const typename DT::X *dy,
                                                 int64_t lddy, const float *w, const float *b, typename DT::X *dx,
                                                 int64_t lddx, float *sums, int max_groups) {
    extern __shared__ __align__(16) float sh[];
    Sums<TH, V> sum(sh, g);
    float *stat = sum.cols + sum.wide, *sq = stat + max_groups;
    const uint32_t id = xcd_remap(blockIdx.x, gridDim.x);
    const int sl = (int)(id % g.slices), img = (int)(id / g.slices);
    const Slice s = slice_of(g, sl);
    const Lane<DT, V> ln(g, s);
    const Group<V> gr(g, s, ln);
    const int n = g.S;
    dx += ((int64_t)img * n + ln.row) * lddx + ln.c;
    const int64_t sx = g.rpp * lddx;
    const Have have(g, ln, n);
    Any<DT, V> v[K], d[K];  // dy is on its way while the moments of x are formed
    take(v, x + ((int64_t)img * n + ln.row) * ldx + ln.c, g.rpp * ldx, have);
    take(d, dy + ((int64_t)img * n + ln.row) * lddy + ln.c, g.rpp * lddy, have);
    Known<V> kn;
    moments<DT, V, TH, K>(g, s, ln, gr, v, n, have, sum, stat, sq, kn.mean, [](float, float) {});
    const float inv = 1.0f / ((float)n * (float)g.cg);
    float s1[V], s2[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        kn.r[i] = inverse_root(sq[gr.of[i]] * inv, g.eps);
        s1[i] = s2[i] = 0.0f;
    }
    kn.ready(w, b, ln.c);
    have.each<K>([&](int k) { add_sums<ACT>(s1, s2, v[k], d[k], kn); });
    of_units(s2, kn);
    float *o = sums + (int64_t)img * 2 * g.C + s.c0;
    float m1[V], m2[V];
    __syncthreads();  // stat and sq have been read
    auto both = [&](float *out, const float (&part)[V], float *mean) {
        sum.rows(part, ln, g);
        sum.of_groups(s, g.cg, [&](int i, float c) {
            out[i] = c;  // each channel once
            return w ? c * w[s.c0 + i] : c;
        }, [&](int j, float a) { mean[j] = a * inv; });
    };
    both(o, s1, stat);
    both(o + g.C, s2, sq);
#pragma unroll
    for (int i = 0; i < V; ++i) m1[i] = stat[gr.of[i]], m2[i] = sq[gr.of[i]];
    if (!ln.live) return;  // all loads of the slice are behind a barrier
    fresh(v);
    fresh(d);
    const Grad<V> grad(g, kn, m1, m2);
    have.each<K>([&](int k) {
        float r[V];
        grad.template of<ACT>(r, v[k], d[k], kn);
        ln.store(dx + k * sx, r, true);
    });
}

// Sums of dz and dz u over a run's pixels, for each channel: part[image][run][2][C].
template <class DT, int V, int TH, int U, int ACT>
__global__ void __launch_bounds__(TH) k_sums(Geo g, const typename DT::X *x, int64_t ldx, const typename DT::X *dy,
                                             int64_t lddy, const float2 *joined, const float *w, const float *b, float *part) {
    extern __shared__ __align__(16) float sh[];
    Sums<TH, V> sum(sh, g);
    const uint32_t id = xcd_remap(blockIdx.x, gridDim.x);
    const int sl = (int)(id % g.slices), run = (int)(id / g.slices % g.runs), img = (int)(id / g.slices / g.runs);
    const Slice s = slice_of(g, sl);
    const Lane<DT, V> ln(g, s);
    const int p0 = run * g.rows, n = min(g.rows, g.S - p0);
    x += ((int64_t)img * g.S + p0 + ln.row) * ldx + ln.c;
    dy += ((int64_t)img * g.S + p0 + ln.row) * lddy + ln.c;
    const int64_t sx = g.rpp * ldx, sy = g.rpp * lddy;
    const Known<V> kn(g, s, ln, joined, img, w, b);
    float s1[V], s2[V];
#pragma unroll
    for (int i = 0; i < V; ++i) s1[i] = s2[i] = 0.0f;
    Any<DT, V> vx[U], vd[U];
    Have(g, ln, n).stream<U>([&](int u, int k) { vx[u] = Lane<DT, V>::load(x + k * sx), vd[u] = Lane<DT, V>::load(dy + k * sy); },
                             [&](int u, int) { add_sums<ACT>(s1, s2, vx[u], vd[u], kn); });
    of_units(s2, kn);
    channel_sums<TH>(g, s, ln, sum, s1, s2, part + ((int64_t)img * g.runs + run) * 2 * g.C + s.c0);
}

// Gradients without an activation, where dz = dy does not wait for the statistics: a run's
// moments as k_fwd leaves them and, in one reading, the sums of dy and dy (x - m) with the
// run's own mean m: part[image][run][2][C].  k_join makes of them the run's sum of dy u,
// r (sum dy (x - m) + (m - mean) sum dy): no difference of large sums.
template <class DT, int V, int TH, int K>
__global__ void __launch_bounds__(TH) k_both(Geo g, const typename DT::X *x, int64_t ldx, const typename DT::X *dy,
                                             int64_t lddy, float2 *stats, float *part, int max_groups) {
    extern __shared__ __align__(16) float sh[];
    Sums<TH, V> sum(sh, g);
    float *stat = sum.cols + sum.wide, *sq = stat + max_groups;
    const uint32_t id = xcd_remap(blockIdx.x, gridDim.x);
    const int sl = (int)(id % g.slices), run = (int)(id / g.slices % g.runs), img = (int)(id / g.slices / g.runs);
    const Slice s = slice_of(g, sl);
    const Lane<DT, V> ln(g, s);
    const Group<V> gr(g, s, ln);
    const int p0 = run * g.rows, n = min(g.rows, g.S - p0);
    const Have have(g, ln, n);
    Any<DT, V> v[K], d[K];
    take(v, x + ((int64_t)img * g.S + p0 + ln.row) * ldx + ln.c, g.rpp * ldx, have);
    take(d, dy + ((int64_t)img * g.S + p0 + ln.row) * lddy + ln.c, g.rpp * lddy, have);
    float mean[V], s1[V], s2[V];
    moments<DT, V, TH, K>(g, s, ln, gr, v, n, have, sum, stat, sq, mean, [](float, float) {});
    leave(g, s, stats, img, run, sl, stat, sq);
#pragma unroll
    for (int i = 0; i < V; ++i) s1[i] = s2[i] = 0.0f;
    have.each<K>([&](int k) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            s1[i] += d[k][i];
            s2[i] = __builtin_fmaf(d[k][i], v[k][i] - mean[i], s2[i]);
        }
    });
    channel_sums<TH>(g, s, ln, sum, s1, s2, part + ((int64_t)img * g.runs + run) * 2 * g.C + s.c0);
}

// From the runs' sums of each channel ([image][run][2][C]: dz, dz u): the first `param`
// workgroups db and dw over images and runs, 16 columns each, of which every 64th row is
// one lane's and the 64 sums are added in order; the others the means of dz w and of
// dz w u of each group, W wavefronts a group.
template <int W>
__global__ void __launch_bounds__(1024) k_means(Geo g, const float *sums, int64_t rows, const float *w, float *dw, float *db,
                                                uint32_t param, float2 *means) {
    __shared__ float sh[64][17];
    if (blockIdx.x < param) {
        const int c = (int)threadIdx.x & 15, first = (int)threadIdx.x >> 4;
        const int64_t cols = 2 * (int64_t)g.C, col = (int64_t)blockIdx.x * 16 + c;
        float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (col < cols) {
            int64_t r = first;
            for (; r + 192 < rows; r += 256) {
#pragma unroll
                for (int k = 0; k < 4; ++k) s[k] += sums[(r + 64 * k) * cols + col];
            }
            for (; r < rows; r += 64) s[0] += sums[r * cols + col];
        }
        sh[first][c] = (s[0] + s[1]) + (s[2] + s[3]);
        __syncthreads();
        if (threadIdx.x >= 16 || col >= cols) return;
        float t = 0.0f;
        for (int k = 0; k < 64; ++k) t += sh[k][c];
        if (col < g.C) {
            if (db) db[col] = t;
        } else if (dw) {
            dw[col - g.C] = t;
        }
        return;
    }
    const int64_t id = (int64_t)(blockIdx.x - param) * (16 / W) + (W == 1 ? threadIdx.x >> 6 : 0);
    if (id >= (int64_t)g.images * g.G) return;
    const int64_t img = id / g.G;
    const int c0 = (int)(id % g.G) * g.cg, lane = (int)threadIdx.x % (64 * W);
    const float *p = sums + img * g.runs * 2 * g.C + c0;
    const float inv = 1.0f / ((float)g.S * (float)g.cg);
    float a = 0.0f, b = 0.0f;
    const int64_t all = (int64_t)g.runs * g.cg;
    for (int64_t i = lane; i < all; i += 64 * W) {
        const int64_t run = i / g.cg, c = i % g.cg;
        const float v = w ? w[c0 + c] : 1.0f, *q = p + run * 2 * g.C + c;
        a = __builtin_fmaf(v, q[0], a);
        b = __builtin_fmaf(v, q[g.C], b);
    }
    sum_group<W>(a, b, &sh[0][0]);
    if (lane == 0) means[id] = make_float2(a * inv, b * inv);
}

template <class DT, int V, int TH, int U, int ACT>
__global__ void __launch_bounds__(TH) k_dx(Geo g, const typename DT::X *x, int64_t ldx, const typename DT::X *dy, int64_t lddy,
                                           const float2 *joined, const float2 *means, const float *w, const float *b,
                                           typename DT::X *dx, int64_t lddx) {
    const uint32_t id = xcd_remap(blockIdx.x, gridDim.x);
    const int sl = (int)(id % g.slices), run = (int)(id / g.slices % g.runs), img = (int)(id / g.slices / g.runs);
    const Slice s = slice_of(g, sl);
    const Lane<DT, V> ln(g, s);
    if (!ln.live) return;
    const int p0 = run * g.rows, n = min(g.rows, g.S - p0);
    const bool apart = (const void *)dx != (const void *)dy;
    x += ((int64_t)img * g.S + p0 + ln.row) * ldx + ln.c;
    dy += ((int64_t)img * g.S + p0 + ln.row) * lddy + ln.c;
    dx += ((int64_t)img * g.S + p0 + ln.row) * lddx + ln.c;
    const int64_t sx = g.rpp * ldx, sy = g.rpp * lddy, so = g.rpp * lddx;
    const Known<V> kn(g, s, ln, joined, img, w, b);
    const Group<V> gr(g, s, ln);
    float m1[V], m2[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const float2 m = means[(int64_t)img * g.G + s.g0 + gr.of[i]];
        m1[i] = m.x;
        m2[i] = m.y;
    }
    const Grad<V> grad(g, kn, m1, m2);
    Any<DT, V> vx[U], vd[U];
    Have(g, ln, n).stream<U>([&](int u, int k) { vx[u] = Lane<DT, V>::load(x + k * sx), vd[u] = Lane<DT, V>::load(dy + k * sy); },
                             [&](int u, int k) {
                                 float o[V];
                                 grad.template of<ACT>(o, vx[u], vd[u], kn);
                                 ln.store(dx + k * so, o, apart);
                             });
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
constexpr int PASS_TH = 256, PASS_K = 16;

Geo base(const dwconv_group_plan &p, int images, int pixels) {
    return {images, pixels, p.C, p.G, p.C / p.G, 1, 1, 0, 1, 1, 1, pixels, p.act, p.eps};
}

// Runs of 4 to `most` rows a lane, as many as make `want` workgroups of all images.
Geo in_runs(Geo g, int want, int most) {
    const int64_t all = (int64_t)g.images * g.slices * (((int64_t)g.S + g.rpp - 1) / g.rpp), each = (all + want - 1) / want;
    const int64_t rows = (each < 4 ? 4 : each > most ? most : each) * g.rpp;
    g.rows = (int)(rows < g.S ? rows : g.S > 0 ? g.S : 1);
    g.runs = (int)(((int64_t)g.S + g.rows - 1) / g.rows);
    return g;
}

// Gradients whose channels' sums k_both forms beside the moments
bool with_sums(const dwconv_group_plan &p, bool back) { return back && p.act == DWCONV_GROUP_ACT_NONE; }

// In passes: slices of at most 256 vectors, whole groups or parts of one.
Geo passes(const dwconv_group_plan &p, int images, int pixels, int V) {
    Geo g = base(p, images, pixels);
    const int most = PASS_TH * V;
    if (g.cg > most) {
        g.parts = (g.cg + most - 1) / most;
        g.part = ((g.cg + g.parts - 1) / g.parts + V - 1) / V * V;
        g.parts = (g.cg + g.part - 1) / g.part;
        g.slices = g.G * g.parts;
        g.vpr = g.part / V;
    } else {
        g.slices = (p.C + most - 1) / most;
        while ((g.G + g.slices - 1) / g.slices * g.cg > most) ++g.slices;
        g.vpr = ((g.G + g.slices - 1) / g.slices * g.cg + V - 1) / V;
    }
    g.rpp = PASS_TH / g.vpr;
    return in_runs(g, 1024, PASS_K);
}
// The same for passes that know the statistics, whose workgroups read parameters first: two a
// CU.  16 images of 112x112x61, no activation: sums (as a pass of their own) 13.3 and gradients
// 16.5 us; with 1024 15.0 and 18.6.
Geo streams(const Geo &g) { return in_runs(g, 512, g.S); }

// Resident: slices of whole groups, `least` bytes of a row or more, that TH lanes hold in K
// vectors each.  The width is a multiple of the vector where groups allow it.  false: none.
bool resident(const dwconv_group_plan &p, int images, int pixels, int V, int TH, int K, int least, Geo &g) {
    g = base(p, images, pixels);
    if (V == 1 || pixels < 1 || images < 1) return false;
    int unit = 1;  // groups that make whole vectors
    while (unit < V && unit * g.cg % V) ++unit;
    if (unit > p.G || p.G % unit) unit = 1;
    int k = unit;
    while (k < p.G && (k * g.cg * (16 / V) < least || p.G % k)) k += unit;
    if (k > p.G) k = p.G;
    if (k * g.cg < V) return false;
    g.slices = p.G / k;
    g.vpr = (k * g.cg + V - 1) / V;
    if (g.vpr > TH) return false;
    g.rpp = TH / g.vpr;
    // rows of 64 bytes only where they leave half the CUs a slice: 8 images of 56x56x128 take
    // 23 us in 32 slices of 64 bytes, 18 in 64 of 32; 64 images 32 and 34
    return ((int64_t)pixels + g.rpp - 1) / g.rpp <= K && (least < 64 || k == p.G || (int64_t)images * g.slices >= 128);
}

// more lanes than a grid counts
bool too_many(int64_t blocks, int lanes) { return blocks >= (int64_t)1 << 32 || blocks * lanes >= (int64_t)1 << 32; }

struct Sizes {
    size_t stats, joined, part, means, all;  // floats
};
Sizes sizes(const dwconv_group_plan &p, const Geo &g, bool back) {
    Sizes z{};
    const int runs = with_sums(p, back) ? g.runs : streams(g).runs;
    const size_t groups = (size_t)g.images * g.G;
    z.stats = groups * g.runs * (g.parts > 1 ? g.parts : 1) * 2;
    z.joined = groups * 2;
    if (back) {
        z.part = (size_t)g.images * runs * 2 * g.C;
        z.means = groups * 2;
    }
    z.all = z.stats + z.joined + z.part + z.means;
    return z;
}

// LDS of a workgroup: lanes' values, columns, two values a group.  At most 131080 bytes, for a
// slice of 8191 groups of one channel, of the 160 KB that a CU has; the passes take 32 KB.
size_t lds_bytes(const Geo &g, int V, int groups) {
    const size_t wide = (size_t)g.vpr * V;
    return (g.rpp * (wide + 4) + wide + 2 * (size_t)groups) * sizeof(float);
}

// groups a slice has at most
int most_groups(const Geo &g) { return (g.G + g.slices - 1) / g.slices; }

// as many values a group as are worth a workgroup
bool many(int64_t values) { return values > 512; }

void join(const Geo &g, const float2 *stats, float2 *joined, float *part, hipStream_t st) {
    const int64_t groups = (int64_t)g.images * g.G;
    if (many((int64_t)g.runs * (part ? g.cg : g.parts))) k_join<16><<<(uint32_t)groups, 1024, 0, st>>>(g, stats, joined, part);
    else k_join<1><<<(uint32_t)((groups + 3) / 4), 256, 0, st>>>(g, stats, joined, part);
}

template <class DT, int V, int TH, int K, int ACT>
hipError_t fwd_resident(const Geo &g, const GroupArgs &a, hipStream_t st) {
    using X = typename DT::X;
    const int64_t blocks = (int64_t)g.images * g.slices;
    if (too_many(blocks, TH)) return hipErrorInvalidConfiguration;
    const int mg = most_groups(g);
    k_fwd<DT, V, TH, K, false, ACT><<<(uint32_t)blocks, TH, lds_bytes(g, V, mg), st>>>(
        g, (const X *)a.x, a.ldx, a.w, a.b, (X *)a.y, a.ldy, nullptr, mg);
    return hipGetLastError();
}

template <class DT, int V, int ACT>
hipError_t fwd(const dwconv_group_plan &p, const GroupArgs &a, hipStream_t st) {
    using X = typename DT::X;
    if constexpr (V > 1) {
        Geo g;
        for (int least : {64, 32}) {
            if (resident(p, a.images, a.pixels, V, 256, 4, least, g)) return fwd_resident<DT, V, 256, 4, ACT>(g, a, st);
            if (resident(p, a.images, a.pixels, V, 256, 16, least, g)) return fwd_resident<DT, V, 256, 16, ACT>(g, a, st);
            if (resident(p, a.images, a.pixels, V, 512, 16, least, g)) return fwd_resident<DT, V, 512, 16, ACT>(g, a, st);
            if (resident(p, a.images, a.pixels, V, 1024, 16, least, g)) return fwd_resident<DT, V, 1024, 16, ACT>(g, a, st);
        }
    }
    const Geo g = passes(p, a.images, a.pixels, V), f = streams(g);
    const Sizes z = sizes(p, g, false);
    const int64_t blocks = (int64_t)g.images * g.slices * g.runs, groups = (int64_t)g.images * g.G;
    if (too_many(blocks, PASS_TH) || groups >= 1 << 22) return hipErrorInvalidConfiguration;
    if (!blocks) return hipSuccess;
    float2 *stats = (float2 *)a.workspace, *joined = (float2 *)(a.workspace + z.stats);
    const int mg = most_groups(g);
    const size_t lds = lds_bytes(g, V, mg);
    k_fwd<DT, V, PASS_TH, PASS_K, true, 0><<<(uint32_t)blocks, PASS_TH, lds, st>>>(g, (const X *)a.x, a.ldx, a.w, a.b, nullptr, 0,
                                                                               stats, mg);
    join(g, stats, joined, nullptr, st);
    k_apply<DT, V, PASS_TH, 4, ACT><<<(uint32_t)((int64_t)f.images * f.slices * f.runs), PASS_TH, 0, st>>>(
        f, (const X *)a.x, a.ldx, joined, a.w, a.b, (X *)a.y, a.ldy);
    return hipGetLastError();
}

template <class DT, int V, int TH, int K, int ACT>
hipError_t bwd_resident(const Geo &g, const GroupArgs &a, hipStream_t st) {
    using X = typename DT::X;
    const int64_t blocks = (int64_t)g.images * g.slices;
    if (too_many(blocks, TH)) return hipErrorInvalidConfiguration;
    const int mg = most_groups(g);
    k_resident<DT, V, TH, K, ACT><<<(uint32_t)blocks, TH, lds_bytes(g, V, mg), st>>>(
        g, (const X *)a.x, a.ldx, (const X *)a.dy, a.lddy, a.w, a.b, (X *)a.dx, a.lddx, a.workspace, mg);
    const uint32_t param = a.dw || a.db ? (uint32_t)((2 * (int64_t)g.C + 15) / 16) : 0;
    if (param)
        k_means<1><<<param, 1024, 0, st>>>(g, a.workspace, g.images, a.w, a.dw, a.db, param, nullptr);
    return hipGetLastError();
}

template <class DT, int V, int ACT>
hipError_t bwd(const dwconv_group_plan &p, const GroupArgs &a, hipStream_t st) {
    using X = typename DT::X;
    if constexpr (V > 1) {
        Geo g;
        // 20 vectors of x and of dy are what 512 lanes have registers for: 64 fp16 images of
        // 56x56x96 take 51 us; of 64x64x96, in passes, 73, a tenth more for an element.
        for (int least : {64, 32}) {
            if (resident(p, a.images, a.pixels, V, 256, 8, least, g)) return bwd_resident<DT, V, 256, 8, ACT>(g, a, st);
            if (resident(p, a.images, a.pixels, V, 512, 20, least, g)) return bwd_resident<DT, V, 512, 20, ACT>(g, a, st);
        }
    }
    constexpr bool BOTH = ACT == DWCONV_GROUP_ACT_NONE;
    const Geo g = passes(p, a.images, a.pixels, V), f = streams(g), &sums = BOTH ? g : f;
    const Sizes z = sizes(p, g, true);
    const int64_t blocks = (int64_t)g.images * g.slices * g.runs, groups = (int64_t)g.images * g.G;
    const uint32_t param = a.dw || a.db ? (uint32_t)((2 * (int64_t)g.C + 15) / 16) : 0;
    if (too_many(blocks, PASS_TH) || groups + param >= 1 << 22) return hipErrorInvalidConfiguration;
    float2 *stats = (float2 *)a.workspace, *joined = (float2 *)(a.workspace + z.stats);
    float *part = (float *)joined + z.joined;
    float2 *means = (float2 *)(part + z.part);
    const int mg = most_groups(g);
    const size_t lds = lds_bytes(g, V, mg);
    const uint32_t streaming = (uint32_t)((int64_t)f.images * f.slices * f.runs);
    if (blocks) {
        const X *x = (const X *)a.x, *dy = (const X *)a.dy;
        if constexpr (BOTH)
            // 16 images of 112x112x61 have 7 rows a lane: 18.4 us, with room for 16 21.7; 2 fp32
            // images of 256x256x256 16: 67 us, 69 in runs of 8 and then 11 more in the joins
            (g.rows <= 8 * g.rpp ? k_both<DT, V, PASS_TH, 8> : k_both<DT, V, PASS_TH, PASS_K>)<<<(uint32_t)blocks, PASS_TH, lds,
                                                                                               st>>>(
                g, x, a.ldx, dy, a.lddy, stats, part, mg);
        else
            k_fwd<DT, V, PASS_TH, PASS_K, true, 0><<<(uint32_t)blocks, PASS_TH, lds, st>>>(g, x, a.ldx, a.w, a.b, nullptr, 0,
                                                                                       stats, mg);
        join(g, stats, joined, BOTH ? part : nullptr, st);
        if constexpr (!BOTH)
            k_sums<DT, V, PASS_TH, 4, ACT><<<streaming, PASS_TH, lds_bytes(f, V, 0), st>>>(f, x, a.ldx, dy, a.lddy, joined, a.w,
                                                                                       a.b, part);
    }
    const bool wide = many((int64_t)sums.runs * sums.cg);
    const uint32_t wg = !blocks ? 0 : (uint32_t)(wide ? groups : (groups + 15) / 16);
    if (param + wg)
        (wide ? k_means<16> : k_means<1>)<<<param + wg, 1024, 0, st>>>(
            sums, part, blocks ? (int64_t)sums.images * sums.runs : 0, a.w, a.dw, a.db, param, means);
    if (blocks)
        k_dx<DT, V, PASS_TH, 4, ACT><<<streaming, PASS_TH, 0, st>>>(f, (const X *)a.x, a.ldx, (const X *)a.dy, a.lddy, joined, means,
                                                              a.w, a.b, (X *)a.dx, a.lddx);
    return hipGetLastError();
}

// Vectors of 16 bytes where a slice has as many channels, else single elements.
int vec_of(const dwconv_group_plan &p) {
    const int v = p.dtype == DWCONV_F32 ? 4 : 8;
    return p.C >= v ? v : 1;
}

template <bool BACK, class DT, int V>
hipError_t pick_act(const dwconv_group_plan &p, const GroupArgs &a, hipStream_t st) {
    auto go = [&](auto act) {
        if constexpr (BACK) return bwd<DT, V, decltype(act)::value>(p, a, st);
        else return fwd<DT, V, decltype(act)::value>(p, a, st);
    };
    switch (p.act) {
        case DWCONV_GROUP_ACT_SILU: return go(std::integral_constant<int, DWCONV_GROUP_ACT_SILU>());
        case DWCONV_GROUP_ACT_RELU: return go(std::integral_constant<int, DWCONV_GROUP_ACT_RELU>());
        default: return go(std::integral_constant<int, DWCONV_GROUP_ACT_NONE>());
    }
}

template <bool BACK, class DT>
hipError_t pick_vec(const dwconv_group_plan &p, const GroupArgs &a, hipStream_t st) {
    constexpr int V = 16 / (int)sizeof(typename DT::X);
    return vec_of(p) == V ? pick_act<BACK, DT, V>(p, a, st) : pick_act<BACK, DT, 1>(p, a, st);
}

template <bool BACK>
hipError_t pick(const dwconv_group_plan &p, const GroupArgs &a, hipStream_t st) {
    switch (p.dtype) {
        case DWCONV_F32: return pick_vec<BACK, F32>(p, a, st);
        case DWCONV_F16: return pick_vec<BACK, F16>(p, a, st);
        default: return pick_vec<BACK, BF16>(p, a, st);
    }
}

}  // namespace

hipError_t group_fwd(const dwconv_group_plan &p, const GroupArgs &a, hipStream_t st) { return pick<false>(p, a, st); }
hipError_t group_bwd(const dwconv_group_plan &p, const GroupArgs &a, hipStream_t st) { return pick<true>(p, a, st); }

// The gradients always have one: small images too keep their channels' sums.
size_t group_bytes(const dwconv_group_plan &p, int images, int pixels, bool back) {
    const int V = vec_of(p);
    Geo g;
    for (int least : {64, 32}) {
        if (!back && resident(p, images, pixels, V, 1024, 16, least, g)) return 0;
        if (back && resident(p, images, pixels, V, 512, 20, least, g)) return (size_t)images * 2 * p.C * sizeof(float);
    }
    return sizes(p, passes(p, images, pixels, V), back).all * sizeof(float);
}

}  // namespace dw
