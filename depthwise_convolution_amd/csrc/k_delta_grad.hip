// k_delta_grad.hip -- the gated delta rule's gradients of q, k, g and beta for
// bf16 and fp16 data, on the 16-bit matrix cores (the algebra is in
// k_delta.hip, the terms in delta_split.h).
//
// A workgroup has one chunk and one key head; its value heads come one after
// the other and their shares of dQ and dK add up in registers.  Wavefronts w
// and w + 4 have tokens 16 w .. 16 w + 15, the first half of the channels of q
// and k and the second (one wavefront's sums for all channels need more
// registers than two wavefronts on a SIMD have).  Per value head, first the
// sums over the state's columns, 32 at a time: the rows of S0 and dS, split into
// terms by one wavefront each, and U pass through LDS; dO, dR and U rows are
// left operands that a lane loads as they lie.  Then the sums over tokens: E and
// M = beta dA D go through LDS once as left operands by rows and once, in terms,
// by columns; their right operands are the fragments of K^T and Q^T in the
// workspace, which also hold a lane's own elements of k and q in the result
// layout.
//
// 2900 products of 16x16x32 a head and chunk at Dk = Dv = 128 (11.6 thousand
// cycles of a CU) against 128 KB of states read.  Measured, bf16, 4096 tokens in
// four sequences, 8 key and 16 value heads: 165 us, some 65 thousand cycles a head
// and chunk: bound by waits for loads and barriers with two wavefronts a SIMD,
// and by whole rounds of workgroups, one a CU (here 528: one sequence's 512 take
// 112 us, 520 take 151, 768 take 168).
#include "delta_split.h"

namespace dw {
namespace {

using namespace delta;

template <int NA, int NB>
__device__ __forceinline__ void mac1(const bf16x8 (&a)[NA], const bf16x8 (&b)[NB], int last, f32x4 &c) {
#pragma unroll
    for (int o = 0; o < NA + NB - 1; ++o) {
        if (o > last) break;
#pragma unroll
        for (int i = 0; i < NA; ++i)
            if (o - i >= 0 && o - i < NB) c = mfma32(a[i], b[o - i], c);
    }
}

template <int N>
__device__ __forceinline__ void put_frag(char *p, const bf16x8 (&t)[N], int lane) {
#pragma unroll
    for (int n = 0; n < N; ++n) *(bf16x8 *)(p + n * FRAG + lane * 16) = t[n];
}
template <int N>
__device__ __forceinline__ void get_frag(bf16x8 (&t)[N], const char *p, int lane) {
#pragma unroll
    for (int n = 0; n < N; ++n) t[n] = *(const bf16x8 *)(p + n * FRAG + lane * 16);
}

// Eight 16-bit elements of a row of v or dO, zeros past `valid`.
__device__ __forceinline__ u32x4 load8(const void *p, int valid, bool vec) {
    u32x4 r = {0, 0, 0, 0};
    if (valid >= 8 && vec) {
        r = *(const u32x4 *)p;
    } else {
        const uint16_t *q = (const uint16_t *)p;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < valid) r[i / 2] |= (uint32_t)q[i] << (i % 2 * 16);
    }
    return r;
}

// A lane's four elements k[token 16 w + g4 + i][channel 16 t + lane % 16], half
// of a fragment of K^T (Q^T).
template <int NA>
__device__ __forceinline__ f32x4 own_elements(const char *kt, int t, int wave, int lane) {
    f32x4 x = splat(0.0f);
#pragma unroll
    for (int n = 0; n < NA; ++n) {
        const u32x2 v = *(const u32x2 *)(kt + ((2 * t + wave / 2) * NA + n) * FRAG + (uint32_t)lane * 16 + wave % 2 * 8);
        x += f32x4{__uint_as_float(v[0] << 16), __uint_as_float(v[0] & 0xffff0000u), __uint_as_float(v[1] << 16),
                   __uint_as_float(v[1] & 0xffff0000u)};
    }
    return x;
}

constexpr int PITCH = 20;  // of a 16x16 tile that is written by columns and read by rows
constexpr int WAVE_TILES = 2 * 4 * 16 * PITCH * 4;  // bytes of a wavefront's tiles of E and M
__host__ __device__ constexpr int lds_blocks(int DK) { return (2 * DK / 16 + 8) * 3 * FRAG; }
constexpr int LDS_TILES = 4 * WAVE_TILES + 2 * Right<4, 3>::bytes(2);
// columns' blocks, later tiles; the tiles of Q K^T and K K^T lie behind
__host__ __device__ constexpr int lds_work(int DK) { return lds_blocks(DK) > LDS_TILES ? lds_blocks(DK) : LDS_TILES; }
constexpr int LDS_KQ = 8 * 4 * FRAG;

template <class DT, int DK>
__global__ void __launch_bounds__(512) k_grad(Ctx c, GradArgs ga) {
    using X = typename DT::X;
    using R = Raw<DT>;
    constexpr int NA = R::TERMS, NT = DK / 16, NH = NT / 2, T = (NT + 7) / 8, NF = DK / 8 * NA, NK = DK / 32;
    extern __shared__ char L[];
    char *SF = L, *DF = SF + NT * 3 * FRAG, *UF = DF + NT * 3 * FRAG, *RF = UF + 4 * 3 * FRAG;
    // by halves: rows of db, dbeta and of the S1 term, column sums, q and k dots
    __shared__ __align__(16) float db[2][CH], dbe[2][CH], a2[2][CH], cols[2][4][CH], rvs[CH], uqs[2][CH], uks[2][CH], dots[8];
    const int slot = blockIdx.x / c.Hk, hk = blockIdx.x % c.Hk;
    const Chunk found = chunk_of(c.seq, slot);
    const int n = uniform(found.n), tok = uniform(found.tok);
    if (n == 0) return;
    const int lane = threadIdx.x & 63, wave8 = uniform(threadIdx.x >> 6), wave = wave8 & 3, half = wave8 >> 2, t0 = half * NH, r = lane & 15, g4 = (lane >> 4) * 4;
    const int row = 16 * wave + g4;  // result layout: tokens row .. row + 3
    float *ET = (float *)(L + wave * WAVE_TILES), *MT = ET + 4 * 16 * PITCH;
    const Right<4, 3> ER{L + 4 * WAVE_TILES}, MR{ER.p + ER.bytes(2)};
    const char *keys = c.keys + ((int64_t)slot * c.Hk + hk) * c.key_bytes;
    const char *rows_k = keys + NF * FRAG, *kt = keys + 2 * NF * FRAG, *qt = keys + 3 * NF * FRAG;
    const int group = c.Hv / c.Hk;
    f32x4 dQ[NH], dK[NH];
#pragma unroll
    for (int t = 0; t < NH; ++t) dQ[t] = dK[t] = splat(0.0f);
    // the wavefront's tiles of Q K^T (first half) or K K^T, of the unit vectors,
    // kept in LDS for all value heads
    f32x4 *const KQ = (f32x4 *)(L + lds_work(DK)) + wave8 * 4 * 64 + lane;
    {
        const float *vec = (const float *)(c.heads + ((int64_t)slot * c.Hv + hk * group) * c.head_bytes + AT_VEC * FRAG);
        const f32x4 nr = *(const f32x4 *)(vec + (half ? V_NK : V_NQ) * CH + row);
        f32x4 kq[4];
        float nky[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            kq[j] = splat(0.0f);
            nky[j] = vec[V_NK * CH + 16 * j + r];
        }
#pragma unroll
        for (int kb = 0; kb < NK; ++kb) {
            bf16x8 z[NA], x[4][NA];
            fetch(z, (half ? rows_k : keys) + (wave * NK + kb) * NA * FRAG, lane);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j <= wave) fetch(x[j], rows_k + (j * NK + kb) * NA * FRAG, lane);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j <= wave) mac1(z, x[j], 2, kq[j]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) KQ[j * 64] = kq[j] * nr * nky[j];
    }
    // Operands of a head's next 32 columns.  The next head's first ones are on their
    // way while the sums over tokens run (167 -> 164 us at the sizes above), where there
    // are registers for it: keys of more than 128 channels would spill (those of 256 do as
    // it is, 65 and 75 registers a lane for bf16 and fp16).
    constexpr bool AHEAD = T == 1;
    f32x4 s0[T][2], ds[T][2], ud[2];  // ud: U (first half) or dR
    u32x4 od, vv;
    auto ahead = [&](int h, int col) {
        const int64_t at = (int64_t)slot * c.Hv + h;
        int lane = threadIdx.x & 63;
        asm volatile("" : "+v"(lane));
        const int r = lane & 15, g8 = (lane >> 4) * 8, mine = 16 * wave + r;
        const uint32_t off = r * c.DvP + g8;
#pragma unroll
        for (int x = 0; x < T; ++x) {
            const int y = min(wave8 + 8 * x, NT - 1);  // (4 and 12 tiles leave wavefronts without one)
            const int64_t p = (at * DK + 16 * y) * c.DvP + col;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                s0[x][j] = *(const f32x4 *)(ga.S0s + p + off + 4 * j);
                ds[x][j] = *(const f32x4 *)(ga.dSs + p + off + 4 * j);
            }
        }
        const int64_t p = (at * CH + 16 * wave) * c.DvP + col;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            ud[j] = *(const f32x4 *)((half ? ga.dRs : ga.Us) + p + off + 4 * j);
        }
        const int x = col + g8, token = tok + min(mine, n - 1), valid = mine < n ? c.Dv - x : 0;
        od = load8((const X *)ga.d_o + token * ga.lddo + (int64_t)h * c.Dv + x, valid, ga.vec_o);
        vv = load8((const X *)c.v + token * c.ldv + (int64_t)h * c.Dv + x, valid, ga.vec_v);
    };
    if (AHEAD) ahead(hk * group, 0);
    for (int h = hk * group; h < (hk + 1) * group; ++h) {
        // made anew for each head: kept over the loop, the addresses that follow
        // from these would take a third of the registers
        int lane = threadIdx.x & 63;
        asm volatile("" : "+v"(lane));
        const int r = lane & 15, g4 = (lane >> 4) * 4, row = 16 * wave + g4;
        const int mine = 16 * wave + r;  // left operands: the lane's token
        const int64_t at = (int64_t)slot * c.Hv + h;
        f32x4 X1[NH], X2[NH], X3[NH], dD[4];  // dD: tiles of dP (first half) or -dA
#pragma unroll
        for (int t = 0; t < NH; ++t) X1[t] = X2[t] = X3[t] = splat(0.0f);
#pragma unroll
        for (int j = 0; j < 4; ++j) dD[j] = splat(0.0f);
        float rv = 0.0f, sd = 0.0f;  // dR . V of token `mine`; <S0, dS>
        // ---- sums over the state's columns
        if (!AHEAD) ahead(h, 0);
        for (int col = 0; col < c.DvP; col += 32) {
            __syncthreads();
            bf16x8 ot[NA], ut[3], rt[3];
            R::terms(__builtin_bit_cast(typename R::V8, od), ot);
            split(ud[0], ud[1], ut);
            put_frag((half ? RF : UF) + wave * 3 * FRAG, ut, lane);
            if (half)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    rv = __builtin_fmaf(ud[j / 4][j % 4], DT::widen(__builtin_bit_cast(X, (uint16_t)(vv[j / 2] >> (j % 2 * 16)))), rv);
#pragma unroll
            for (int x = 0; x < T; ++x) {
                const int y = wave8 + 8 * x;
                if (y >= NT) break;
                bf16x8 t[3];
                split(s0[x][0], s0[x][1], t);
                put_frag(SF + y * 3 * FRAG, t, lane);
                split(ds[x][0], ds[x][1], t);
                put_frag(DF + y * 3 * FRAG, t, lane);
#pragma unroll
                for (int j = 0; j < 8; ++j) sd = __builtin_fmaf(s0[x][j / 4][j % 4], ds[x][j / 4][j % 4], sd);
            }
            if (col + 32 < c.DvP) ahead(h, col + 32);
            __syncthreads();
            get_frag(ut, UF + wave * 3 * FRAG, lane);
            get_frag(rt, RF + wave * 3 * FRAG, lane);
#pragma unroll
            for (int t = 0; t < NH; ++t) {
                bf16x8 st[3], dt[3];
                get_frag(st, SF + (t0 + t) * 3 * FRAG, lane);
                get_frag(dt, DF + (t0 + t) * 3 * FRAG, lane);
                mac1(rt, st, 2, X3[t]);
                mac1(ot, st, 2, X1[t]);
                mac1(ut, dt, 2, X2[t]);
                fence();
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (j > wave) continue;
                bf16x8 u[3];
                get_frag(u, UF + j * 3 * FRAG, lane);
                if (half) mac1(rt, u, 2, dD[j]);
                else mac1(ot, u, 2, dD[j]);
            }
        }
        // ---- sums over tokens
        const float *vec = (const float *)(c.heads + at * c.head_bytes + AT_VEC * FRAG);
        auto rows4 = [&](int which) { return *(const f32x4 *)(vec + which * CH + row); };
        const f32x4 eb = rows4(V_EB), er = rows4(V_ER), be = rows4(V_BETA), nk = rows4(V_NK), nq = rows4(V_NQ);
        const double *bs = c.sums + at * CH;
        double br[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) br[i] = bs[row + i];
        double by[4];
        float nky[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            by[j] = bs[16 * j + r];
            nky[j] = vec[V_NK * CH + 16 * j + r];
        }
        f32x4 s1 = splat(0.0f), s2 = splat(0.0f), s3 = splat(0.0f);
#pragma unroll
        for (int t = 0; t < NH; ++t) {
            const f32x4 kr = own_elements<NA>(kt, t0 + t, wave, lane), qr = own_elements<NA>(qt, t0 + t, wave, lane);
            s1 += qr * X1[t];
            s2 += kr * X2[t];
            s3 += kr * X3[t];
            dQ[t] += c.scale * eb * X1[t];
            dK[t] += er * X2[t] - eb * be * X3[t];
        }
        s1 = sum16(s1) * eb * nq * c.scale;
        s2 = sum16(s2) * er * nk;
        s3 = sum16(s3) * eb * nk;
#pragma unroll
        for (int m = 1; m < 64; m <<= 1) sd += __shfl_xor(sd, m, 64);
        rv += __shfl_xor(rv, 16, 64);
        rv += __shfl_xor(rv, 32, 64);
        if (AHEAD && h + 1 < (hk + 1) * group) ahead(h + 1, 0);
        __syncthreads();  // the blocks have been read: tiles take their place
        if (lane == 0) dots[wave8] = sd;
        if (half && lane < 16) rvs[mine] = rv;
        // the first half makes E from dP, the second M from dA
        f32x4 rowD = splat(0.0f), rowB = splat(0.0f);
        float *tile = half ? MT : ET;
        const f32x4 left = half ? nk : nq;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float cd = 0.0f;
            f32x4 e = splat(0.0f);
            if (j <= wave) {
                const int y = 16 * j + r;
                const f32x4 kq = KQ[j * 64];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float d = expf((float)(br[i] - by[j]));  // as k_prepare made it
                    const float x = half ? -dD[j][i] * d : c.scale * dD[j][i] * d;
                    const bool in = half ? row + i > y : row + i >= y;
                    const float z = in ? x : 0.0f, zk = in ? x * kq[i] : 0.0f;
                    e[i] = half ? be[i] * z : z;
                    rowB[i] += zk;
                    rowD[i] += half ? be[i] * zk : zk;
                    cd += half ? be[i] * zk : zk;
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) tile[(j * 16 + g4 + i) * PITCH + r] = e[i] * nky[j];
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) tile[(j * 16 + g4 + i) * PITCH + r] = 0.0f;
            }
            (half ? MR : ER).put(wave, j, e * left, lane);
            cd += __shfl_xor(cd, 16, 64);
            cd += __shfl_xor(cd, 32, 64);
            if (lane < 16) cols[half][wave][16 * j + r] = cd;
        }
        rowD = sum16(rowD);
        rowB = sum16(rowB);
        if (r == 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                db[half][row + i] = s1[i] + rowD[i] - be[i] * s3[i] - s2[i];
                a2[half][row + i] = s2[i];
                dbe[half][row + i] = (half ? rowB[i] : 0.0f) - s3[i];
            }
        }
        __syncthreads();
        if (wave8 == 0) {
            float x = db[0][lane] + db[1][lane];
#pragma unroll
            for (int w = 0; w < 4; ++w) x -= cols[0][w][lane] + cols[1][w][lane];
            double all = a2[0][lane] + a2[1][lane];
#pragma unroll
            for (int m = 1; m < 64; m <<= 1) all += __shfl_xor(all, m, 64);
            double y = x;
            if (lane == 63) {
                float sum = 0.0f;
#pragma unroll
                for (int w = 0; w < 8; ++w) sum += dots[w];
                y += all + (double)vec[V_EB * CH + CH - 1] * sum;
            }
#pragma unroll
            for (int m = 1; m < 64; m <<= 1) {
                const double z = __shfl_down(y, m, 64);
                if (lane + m < 64) y += z;
            }
            if (lane < n) {
                ga.dg[((int64_t)tok + lane) * c.Hv + h] = (float)y;
                ga.dbeta[((int64_t)tok + lane) * c.Hv + h] = dbe[0][lane] + dbe[1][lane] + rvs[lane];
            }
        }
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            bf16x8 er3[3], mr3[3], et3[3], mt3[3];
            const bool low = kb <= wave / 2, high = kb >= wave / 2;  // E K and M K; E^T Q and M^T K
            {
                const float *pe = ET + (2 * kb * 16 + r) * PITCH + g4, *pm = MT + (2 * kb * 16 + r) * PITCH + g4;
                split(*(const f32x4 *)pe, *(const f32x4 *)(pe + 16 * PITCH), er3);
                split(*(const f32x4 *)pm, *(const f32x4 *)(pm + 16 * PITCH), mr3);
            }
            get_frag(et3, ER.p + (kb * 4 + wave) * 3 * FRAG, lane);
            get_frag(mt3, MR.p + (kb * 4 + wave) * 3 * FRAG, lane);
            bf16x8 fk[NH][NA], fq[NH][NA];
#pragma unroll
            for (int t = 0; t < NH; ++t) {
                fetch(fk[t], kt + (2 * (t0 + t) + kb) * NA * FRAG, lane);
                fetch(fq[t], qt + (2 * (t0 + t) + kb) * NA * FRAG, lane);
            }
            if (low) {
#pragma unroll
                for (int t = 0; t < NH; ++t) {
                    mac1(er3, fk[t], 2, dQ[t]);
                    mac1(mr3, fk[t], 2, dK[t]);
                }
            }
            if (high) {
#pragma unroll
                for (int t = 0; t < NH; ++t) {
                    mac1(et3, fq[t], 2, dK[t]);
                    mac1(mt3, fk[t], 2, dK[t]);
                }
            }
        }
    }
    // from the unit vectors to q and k: d - u (u . d), over the length
    const float *vec = (const float *)(c.heads + ((int64_t)slot * c.Hv + hk * group) * c.head_bytes + AT_VEC * FRAG);
    const f32x4 nk = *(const f32x4 *)(vec + V_NK * CH + row), nq = *(const f32x4 *)(vec + V_NQ * CH + row);
    f32x4 uq = splat(0.0f), uk = splat(0.0f);
    if (c.normalize) {
#pragma unroll
        for (int t = 0; t < NH; ++t) {
            uq += dQ[t] * own_elements<NA>(qt, t0 + t, wave, lane);
            uk += dK[t] * own_elements<NA>(kt, t0 + t, wave, lane);
        }
        uq = sum16(uq) * nq * nq;
        uk = sum16(uk) * nk * nk;
        if (r == 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uqs[half][row + i] = uq[i];
                uks[half][row + i] = uk[i];
            }
        }
        __syncthreads();
        uq = *(const f32x4 *)&uqs[0][row] + *(const f32x4 *)&uqs[1][row];
        uk = *(const f32x4 *)&uks[0][row] + *(const f32x4 *)&uks[1][row];
    }
#pragma unroll
    for (int t = 0; t < NH; ++t) {
        const f32x4 q = nq * (dQ[t] - uq * own_elements<NA>(qt, t0 + t, wave, lane));
        const f32x4 k = nk * (dK[t] - uk * own_elements<NA>(kt, t0 + t, wave, lane));
        const int y = 16 * (t0 + t) + r;
        if (y < c.Dk) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (row + i < n) {
                    ((X *)ga.dq)[(tok + row + i) * ga.lddq + (int64_t)hk * c.Dk + y] = rounded<DT>(q[i]);
                    ((X *)ga.dk)[(tok + row + i) * ga.lddk + (int64_t)hk * c.Dk + y] = rounded<DT>(k[i]);
                }
        }
    }
}

}  // namespace

namespace delta {

hipError_t split_grad(int dtype, int DK_, const Ctx &c, const GradArgs &ga, hipStream_t st) {
    return pick(dtype, DK_, [&](auto dt, auto dk) {
        using DT = decltype(dt);
        constexpr int DK = decltype(dk)::value;
        const size_t n = lds_work(DK) + LDS_KQ;
        hipError_t e = lds_room((const void *)k_grad<DT, DK>, n);
        if (e != hipSuccess) return e;
        k_grad<DT, DK><<<(uint32_t)((int64_t)c.slots * c.Hk), 512, n, st>>>(c, ga);
        return hipGetLastError();
    });
}

}  // namespace delta
}  // namespace dw
