// Gated feed-forward on packed weights for decode-sized M (1..16 tokens): both projections, the
// activation and the product in one launch,
//     h = act(g) * u,  (g | u) = (x / s) dequant(W)^T,  W [2F, in]: gate rows, then up rows.
//
// Bound: reading the packed weights once from HBM.  One CTA per SM over a contiguous range of
// tiles; a tile is 16 columns f of h: the gate rows f and the up rows f, eight of each as rows 0-7
// and 8-15 of the A operand of mma.sync.m16n8k16, so the lane that ends up with g also holds the u
// it multiplies and the epilogue needs no exchange.  Tokens are the MMA's 8 columns (two column
// tiles for 9..16).
//
// Split: a CTA's tiles x 128-column chunks are one sequence of steps, cut into equal contiguous
// ranges for its 16 warps (the last step of a range and the first of the next share a tile), so
// all warps finish together whatever the layer's shape; the fp32 partial sums of a tile's segments
// meet in shared memory and are added in the order of the warps.
//
// Each lane loads the packed words of its four rows straight into registers, GD_PF steps ahead (2
// KB a warp and step), while the bulk of the CTA's weights is on its way to L2 by a prefetch hint,
// so HBM streams from the start, through the staging of the activations.
// Unpacking: one shift and four LOP3 turn a packed word into fp16 pairs 1024 + c or 1024 + 16 c
// (exact; the activations of the latter pairs are staged divided by 16), and per (row, group)
//     sum_i (c_i - z) Delta x_i / s_i = Delta 2^k ((D - 1024 T1) - z T2),
// T1 the sum of the staged values and T2 that of the activations they stand for: xs = fp16((x / s)
// 2^-k), one power of two per (token, group), so staging needs no pass over the whole row first.
//
// Measured: 22016 x 4096, group 128, one token 15.5 us a call back to back (46.8 MB, 3.0 TB/s, 46% of HBM); 27648 x
// 5120 with zero points, 8 tokens 31.9 us.  What holds it: the packed loop is about 17500 of the
// kernel's cycles, of which the MMAs (16 cycles of a sub-core each) need 10200 and the unpacking the integer pipe, 52%
// busy over the whole kernel; the staging of activations and scales in front of it is latency.  Sums of the
// activations by an extra MMA instead of in the staging make 16 tokens faster (32.2 -> 27.2 us) and one token
// slower (15.5 -> 16.8); not kept.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "awq_internal.h"
#include "awq_ptx.cuh"
#include "w4a16_act.cuh"
#include "w4a16_frag.cuh"

namespace awq {

namespace {

constexpr int GD_WARPS = 16;
constexpr int GD_THREADS = GD_WARPS * 32;
constexpr int GD_PF = 1;                              // steps of weights in flight per warp (two: registers spill, 4% slower)
constexpr int GD_TILE = 16;                           // columns of h per tile
constexpr int GD_MAX_TILES = 32;                      // tiles of one pass of a CTA
constexpr uint32_t GD_EARLY = 65536;                  // bytes of gate and of up rows asked for first

struct GdArgs {
    const uint16_t *x;
    const uint32_t *q;
    const uint16_t *scales;
    const uint32_t *zeros;
    const uint16_t *s16;
    uint16_t *h;
    int64_t F;
    int M, I, act;
    int tiles;                                        // ceil(F / GD_TILE)
    int pass_tiles;                                   // tiles per pass of a CTA (shared memory)
};

// Shared-memory plan (bytes), for M tokens.
struct GdPlan {
    int chunks, groups;                               // 128-column chunks, groups (both over the padded width)
    int rs;                                           // (Delta, z) entries of a row: odd, so rows fall into other banks
    int x, sums, sc, slots, total;
};
__host__ __device__ inline GdPlan gd_plan(int M, int I, int gs, int nt, int pass_tiles) {
    GdPlan p;
    p.chunks = (I + 127) / 128;
    p.groups = p.chunks * (128 / gs);
    p.rs = p.groups | 1;
    p.x = (p.chunks * 16 * M + 1) * 16;               // [chunk][word slot][token][lane t] 16-byte entries, one of zeros
    p.sums = p.groups * nt * 8 * 16;                  // [group][token] (1024 T1, T2, 2^k)
    p.sc = (pass_tiles * 2 * GD_TILE * p.rs * 8 + 15) / 16 * 16;   // [tile][row][group] (Delta, z)
    p.slots = (pass_tiles + GD_WARPS) * 32 * nt * 32; // partial sums [tile + warp][lane]
    p.total = p.x + p.sums + p.sc + p.slots + (GD_WARPS + 1) * 4;
    return p;
}

// Where word r (0..15) of a 128-column chunk sits: lane t (of the 4 sharing a row) and slot j.  The
// four words that meet in one MMA lie in one group, and a lane's words are as contiguous as that allows.
template <int GS>
__device__ __forceinline__ void word_place(int r, int &t, int &j) {
    if (GS == 128) {
        t = r >> 2;
        j = r & 3;
    } else if (GS == 64) {
        t = (r & 7) >> 1;
        j = (r >> 3) * 2 + (r & 1);
    } else {
        t = r & 3;
        j = r >> 2;
    }
}

// This lane's four packed words of one row in a chunk, `row` at the chunk's first word; words from
// `left` on are zero (the last chunk of a width that is an odd multiple of 64).
template <int GS>
__device__ __forceinline__ void load_words(const uint32_t *row, int t, int left, uint32_t (&v)[4]) {
    if (GS == 128) {
        const uint4 q = __ldcs(reinterpret_cast<const uint4 *>(row + 4 * t));
        v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
    } else if (GS == 64) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const uint2 q = 8 * k < left ? __ldcs(reinterpret_cast<const uint2 *>(row + 8 * k + 2 * t)) : make_uint2(0u, 0u);
            v[2 * k] = q.x;
            v[2 * k + 1] = q.y;
        }
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = 4 * k < left ? __ldcs(row + 4 * k + t) : 0u;
    }
}

// Power of two above a group's largest magnitude: k with mx * 2^-k in [2^14, 2^15), from its
// exponent field (0 and subnormals: the smallest; inf and NaN: 0, so that they stay what they are).
__device__ __forceinline__ int pow2_above(float mx) {
    const int b = __float_as_int(mx) >> 23;           // mx >= 0
    const int k = b - 127 - 14;
    return b == 255 ? 0 : (k < -125 ? -125 : k);
}

__device__ __forceinline__ float rcp_approx(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// 1 / s of the 8 columns of word w: products with it are within 2 ulp of fp32 of x / s, far below
// the fp16 rounding that follows.
__device__ __forceinline__ void inverse_s(const uint16_t *s16, int w, float (&r)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) r[e] = 1.0f;
    if (s16) {
        const uint4 sv = __ldg(reinterpret_cast<const uint4 *>(s16) + w);
        const uint32_t sw[4] = {sv.x, sv.y, sv.z, sv.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const __half2 h = *reinterpret_cast<const __half2 *>(&sw[e]);
            r[2 * e] = rcp_approx(__low2float(h));
            r[2 * e + 1] = rcp_approx(__high2float(h));
        }
    }
}

// A fresh product: d = A B.
__device__ __forceinline__ void mma_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}

template <int GS, int NT>
__global__ void __launch_bounds__(GD_THREADS, 1) gated_dec_kernel(const GdArgs a) {
    extern __shared__ __align__(16) uint8_t smem[];
    constexpr int GPC = 128 / GS;                     // groups per chunk
    constexpr int JPG = 4 / GPC;                      // word slots per group
    const GdPlan p = gd_plan(a.M, a.I, GS, NT, a.pass_tiles);
    uint4 *xsm = reinterpret_cast<uint4 *>(smem);
    float4 *sums = reinterpret_cast<float4 *>(smem + p.x);
    float2 *scm = reinterpret_cast<float2 *>(smem + p.x + p.sums);
    float4 *slots = reinterpret_cast<float4 *>(smem + p.x + p.sums + p.sc);
    int *first = reinterpret_cast<int *>(smem + p.x + p.sums + p.sc + p.slots);   // [GD_WARPS + 1] range starts

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int wpr = a.I / 8, nG = a.I / GS, nzw = (nG + 7) / 8, nC = p.chunks;
    const int t0 = static_cast<int>(static_cast<int64_t>(a.tiles) * blockIdx.x / gridDim.x);
    const int t1 = static_cast<int>(static_cast<int64_t>(a.tiles) * (blockIdx.x + 1) / gridDim.x);

    // The preceding kernel of the stream may still run: until it is done, only ask L2 for the first
    // of the weights (all of them would hold up the activations and scales behind them).
    const int64_t row0 = static_cast<int64_t>(t0) * GD_TILE;
    const int64_t row1 = static_cast<int64_t>(t1) * GD_TILE < a.F ? static_cast<int64_t>(t1) * GD_TILE : a.F;
    const uint64_t part = static_cast<uint64_t>(row1 - row0) * wpr * 4;     // bytes of the gate rows; the up rows' alike
    const uint8_t *mine = reinterpret_cast<const uint8_t *>(a.q + ((threadIdx.x & 1) * a.F + row0) * wpr);
    if (threadIdx.x < 2) l2_prefetch_range(mine, part < GD_EARLY ? part : GD_EARLY);
    griddep_launch_dependents();
    griddep_wait();

    for (int p0 = t0; p0 < t1; p0 += a.pass_tiles) {
        const int nt = t1 - p0 < a.pass_tiles ? t1 - p0 : a.pass_tiles;   // tiles of this pass
        const int steps = nt * nC;
        const int s0 = static_cast<int>(static_cast<int64_t>(steps) * warp / GD_WARPS);
        const int s1 = static_cast<int>(static_cast<int64_t>(steps) * (warp + 1) / GD_WARPS);
        if (threadIdx.x <= GD_WARPS)
            first[threadIdx.x] = static_cast<int>(static_cast<int64_t>(steps) * threadIdx.x / GD_WARPS);

        // ---- weights in flight: the row pointers run ahead of the arithmetic by GD_PF steps
        uint32_t wa[GD_PF][2][4], wb[GD_PF][2][4];    // gate and up words of rows f0 + g, f0 + 8 + g
        const int tile0 = s0 / nC, c0 = s0 - tile0 * nC;
        int lc = c0, left = s1 - s0;                  // chunk of the next load, loads to issue
        int64_t lf = static_cast<int64_t>(p0 + tile0) * GD_TILE + g;
        // rows past the last (of the last tile alone): any row, its results are dropped
        const uint32_t *ra[2], *rb[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            ra[e] = a.q + (lf + 8 * e < a.F ? lf + 8 * e : a.F - 1) * wpr + c0 * 16;
            rb[e] = ra[e] + a.F * wpr;
        }
        auto fetch = [&](uint32_t (&va)[2][4], uint32_t (&vb)[2][4]) {
            if (left > 0) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    load_words<GS>(ra[e], t, wpr - lc * 16, va[e]);
                    load_words<GS>(rb[e], t, wpr - lc * 16, vb[e]);
                    ra[e] += 16;
                    rb[e] += 16;
                }
                --left;
                if (++lc == nC) {                     // the same rows of the next tile
                    lc = 0;
                    lf += GD_TILE;
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int64_t adv = (lf + 8 * e < a.F ? static_cast<int64_t>(GD_TILE) * wpr : 0) - nC * 16;
                        ra[e] += adv;
                        rb[e] += adv;
                    }
                }
            }
        };
#pragma unroll
        for (int u = 0; u < GD_PF; ++u) fetch(wa[u], wb[u]);
        // ---- scales and zero points of the pass's rows, a warp per row and a lane per group: asked for
        // here, put in place after the activations, so that the two latencies overlap
        constexpr int SR = 10;                        // rows of a warp in flight
        uint16_t sraw[SR];
        uint32_t zraw[SR];
        const int srows = nt * 2 * GD_TILE;
        auto scale_row = [&](int r) -> int64_t {      // row r of the pass: tile r / 32, then 8 gate rows, their 8 up rows, the next 8 of each
            const int64_t f = static_cast<int64_t>(p0) * GD_TILE + ((r >> 4) << 3) + (r & 7);
            return f < a.F ? (r & 8 ? a.F : 0) + f : -1;
        };
        auto ask = [&](int r0, int j) {
#pragma unroll
            for (int i = 0; i < SR; ++i) {
                const int r = r0 + i * GD_WARPS;
                sraw[i] = 0;
                zraw[i] = 0x88888888u;
                if (r < srows && j < nG) {
                    const int64_t o = scale_row(r);
                    if (o >= 0) {
                        sraw[i] = __ldg(a.scales + o * nG + j);
                        if (a.zeros) zraw[i] = __ldg(a.zeros + o * nzw + (j >> 3));
                    }
                }
            }
        };
        auto put = [&](int r0, int j) {
#pragma unroll
            for (int i = 0; i < SR; ++i) {
                const int r = r0 + i * GD_WARPS;
                if (r < srows && j < p.groups)
                    scm[r * p.rs + j] = make_float2(__half2float(__ushort_as_half(sraw[i])),
                                                    static_cast<float>((zraw[i] >> (4 * (j & 7))) & 15u));
            }
        };
        ask(warp, lane);

        // ---- activations, once: a lane per packed word, the warps over (block of words, tokens)
        if (p0 == t0) {
            const int words = nC * 16;                // padded width, a multiple of 16
            if (threadIdx.x == 0) xsm[nC * 16 * a.M] = make_uint4(0u, 0u, 0u, 0u);
            for (int i = threadIdx.x; i < p.groups * NT * 8; i += GD_THREADS)   // the columns of no token
                if (i % (NT * 8) >= a.M) sums[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            // one token: 32 words a warp; more: 16 words of two tokens, whose 1 / s a lane forms once
            const int bw = a.M == 1 ? 32 : 16, tpw = a.M == 1 ? 1 : 2;
            for (int w0 = warp * bw; w0 < words; w0 += GD_WARPS * bw) {
                const int w = w0 + (lane & (bw - 1));
                const bool inside = w < wpr;
                float rs[8];
                inverse_s(a.s16, inside ? w : 0, rs);
                int tt, jj;
                word_place<GS>(w & 15, tt, jj);
                uint4 *xd = xsm + (((w >> 4) * 4 + jj) * a.M) * 4 + tt;
#pragma unroll 4
                for (int mb = 0; mb < a.M; mb += tpw) {
                    const int m = mb + (tpw == 2 ? lane >> 4 : 0);
                    const bool real = inside && m < a.M;
                    const uint4 xv = real ? __ldcg(reinterpret_cast<const uint4 *>(a.x + static_cast<int64_t>(m) * a.I) + w)
                                          : make_uint4(0u, 0u, 0u, 0u);
                    const uint32_t xw[4] = {xv.x, xv.y, xv.z, xv.w};
                    float v[8];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        v[2 * e] = __uint_as_float(xw[e] << 16) * rs[2 * e];
                        v[2 * e + 1] = __uint_as_float(xw[e] & 0xFFFF0000u) * rs[2 * e + 1];
                    }
                    float mx = fmaxf(fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3]))),
                                     fmaxf(fmaxf(fabsf(v[4]), fabsf(v[5])), fmaxf(fabsf(v[6]), fabsf(v[7]))));
#pragma unroll
                    for (int off = GS / 16; off > 0; off >>= 1)   // a group's words are GS / 8 neighbouring lanes
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
                    const int k = pow2_above(mx);
                    const float sc = __int_as_float((127 - k) << 23);
                    uint32_t h[4];
                    float even = 0.0f, odd = 0.0f;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        __half2 hv = __floats2half2_rn(v[e] * sc, v[e + 4] * sc);
                        if (e & 1) hv = __hmul2(hv, __floats2half2_rn(0.0625f, 0.0625f));
                        h[e] = *reinterpret_cast<const uint32_t *>(&hv);
                        const float2 f = __half22float2(hv);
                        (e & 1 ? odd : even) += f.x + f.y;
                    }
                    float t1s = even + odd, t2s = fmaf(16.0f, odd, even);
#pragma unroll
                    for (int off = GS / 16; off > 0; off >>= 1) {
                        t1s += __shfl_xor_sync(0xffffffffu, t1s, off);
                        t2s += __shfl_xor_sync(0xffffffffu, t2s, off);
                    }
                    if (w < words && m < a.M) {
                        xd[m * 4] = make_uint4(h[0], h[1], h[2], h[3]);
                        if ((w & (GS / 8 - 1)) == 0)
                            sums[(w / (GS / 8)) * (NT * 8) + m] =
                                make_float4(1024.0f * t1s, t2s, __int_as_float((127 + k) << 23), 0.0f);
                    }
                }
            }
            if (threadIdx.x < 2 && part > GD_EARLY) l2_prefetch_range(mine + GD_EARLY, part - GD_EARLY);
        }
        put(warp, lane);
        for (int j = lane; j < p.groups; j += 32)     // what one round did not cover
            for (int r = warp + (j == lane ? SR * GD_WARPS : 0); r < srows; r += SR * GD_WARPS) {
                ask(r, j);
                put(r, j);
            }
        __syncthreads();

        // ---- this warp's steps
        int tile = tile0, c = c0;
        // lanes of no token read the entry of zeros, with strides of zero
        const bool has = g < a.M, has2 = NT > 1 && 8 + g < a.M;
        const int js = has ? a.M * 4 : 0, js2 = has2 ? a.M * 4 : 0;     // entries of one word slot
        const uint4 *const x0 = xsm + (has ? lane : nC * 16 * a.M), *const x02 = xsm + (has2 ? lane + 32 : nC * 16 * a.M);
        const uint4 *xp = x0 + c * 4 * js, *xp2 = x02 + c * 4 * js2;
        const float4 *tp = sums + c * GPC * (NT * 8) + 2 * t;
        const float2 *sp = scm + (tile * 2 * GD_TILE + g) * p.rs + c * GPC;
        const int r8 = 8 * p.rs;
        float tot[2][NT][4];
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int k = 0; k < 4; ++k) tot[e][n][k] = 0.0f;
        for (int todo = s1 - s0; todo > 0; todo -= GD_PF) {
#pragma unroll
            for (int u = 0; u < GD_PF; ++u) {
                if (u < todo) {
                    float acc[2][NT][4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t P = 0x64006400u;
                        uint4 b[NT];
                        b[0] = xp[j * js];
                        if (NT > 1) b[NT - 1] = xp2[j * js2];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const uint32_t va = wa[u][e][j], vb = wb[u][e][j], va8 = va >> 8, vb8 = vb >> 8;
                            const uint32_t A0[4] = {(va & 0x000F000Fu) | P, (vb & 0x000F000Fu) | P,
                                                    (va & 0x00F000F0u) | P, (vb & 0x00F000F0u) | P};
                            const uint32_t A1[4] = {(va8 & 0x000F000Fu) | P, (vb8 & 0x000F000Fu) | P,
                                                    (va8 & 0x00F000F0u) | P, (vb8 & 0x00F000F0u) | P};
#pragma unroll
                            for (int n = 0; n < NT; ++n) {
                                if (j % JPG == 0)
                                    mma_first(acc[e][n], A0, b[n].x, b[n].y);
                                else
                                    frag_mma16816(acc[e][n], A0, b[n].x, b[n].y);
                                frag_mma16816(acc[e][n], A1, b[n].z, b[n].w);
                            }
                        }
                        if (j % JPG == JPG - 1) {     // the group's sums to the rows'
#pragma unroll
                            for (int n = 0; n < NT; ++n) {
                                const float4 T0 = tp[j / JPG * (NT * 8) + n * 8], T1 = tp[j / JPG * (NT * 8) + n * 8 + 1];
#pragma unroll
                                for (int e = 0; e < 2; ++e) {
                                    const float2 sa = sp[2 * e * r8 + j / JPG], sb = sp[(2 * e + 1) * r8 + j / JPG];
                                    float (&o)[4] = tot[e][n];
                                    const float (&d)[4] = acc[e][n];
                                    o[0] = fmaf(sa.x * T0.z, fmaf(-sa.y, T0.y, d[0] - T0.x), o[0]);
                                    o[1] = fmaf(sa.x * T1.z, fmaf(-sa.y, T1.y, d[1] - T1.x), o[1]);
                                    o[2] = fmaf(sb.x * T0.z, fmaf(-sb.y, T0.y, d[2] - T0.x), o[2]);
                                    o[3] = fmaf(sb.x * T1.z, fmaf(-sb.y, T1.y, d[3] - T1.x), o[3]);
                                }
                            }
                        }
                    }
                    fetch(wa[u], wb[u]);
                    xp += 4 * js;
                    xp2 += 4 * js2;
                    tp += GPC * (NT * 8);
                    sp += GPC;
                    if (++c == nC || u + 1 == todo) { // the tile's or the range's end: hand over
#pragma unroll
                        for (int e = 0; e < 2; ++e)
#pragma unroll
                            for (int n = 0; n < NT; ++n) {
                                float (&o)[4] = tot[e][n];
                                slots[((tile + warp) * 2 * NT + e * NT + n) * 32 + lane] = make_float4(o[0], o[1], o[2], o[3]);
                                o[0] = o[1] = o[2] = o[3] = 0.0f;
                            }
                        c = 0;
                        ++tile;
                        xp = x0;
                        xp2 = x02;
                        tp = sums + 2 * t;
                        sp = scm + (tile * 2 * GD_TILE + g) * p.rs;
                    }
                }
            }
        }
        __syncthreads();

        // ---- a warp per half tile: its segments in the order of the warps, then h
        for (int i2 = warp; i2 < 2 * nt; i2 += GD_WARPS) {
            const int i = i2 >> 1, e = i2 & 1;
            const int b0 = i * nC, b1 = b0 + nC;      // the tile's steps
            float4 s[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) s[n] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
            for (int w = 0; w < GD_WARPS; ++w) {
                const int w0 = first[w], w1 = first[w + 1];
                if (w0 < b1 && w1 > b0 && w1 > w0) {
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const float4 v = slots[((i + w) * 2 * NT + e * NT + n) * 32 + lane];
                        s[n].x += v.x;
                        s[n].y += v.y;
                        s[n].z += v.z;
                        s[n].w += v.w;
                    }
                }
            }
            const int64_t f = static_cast<int64_t>(p0 + i) * GD_TILE + e * 8 + g;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const int m = n * 8 + 2 * t;
                if (f < a.F && m < a.M)
                    a.h[m * a.F + f] = __bfloat16_as_ushort(__float2bfloat16_rn(act_value(s[n].x, a.act) * s[n].z));
                if (f < a.F && m + 1 < a.M)
                    a.h[(m + 1) * a.F + f] = __bfloat16_as_ushort(__float2bfloat16_rn(act_value(s[n].y, a.act) * s[n].w));
            }
        }
        __syncthreads();                              // the next pass reuses the slots and the scales
    }
}

constexpr int GD_SMEM = 224 * 1024;

// Tiles per pass that fit beside the activations; 0: not even one.
int gd_pass_tiles(int M, int I, int gs, int nt, int most) {
    for (int n = most < GD_MAX_TILES ? most : GD_MAX_TILES; n >= 1; --n)
        if (gd_plan(M, I, gs, nt, n).total <= GD_SMEM) return n;
    return 0;
}

template <int GS, int NT>
cudaError_t launch_gd(const GdArgs &a, int grid, cudaStream_t st) {
    const int smem = gd_plan(a.M, a.I, GS, NT, a.pass_tiles).total;
    static bool attr_set[64] = {};                    // per device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64 || !attr_set[dev]) {
        e = cudaFuncSetAttribute(gated_dec_kernel<GS, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, GD_SMEM);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) attr_set[dev] = true;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(GD_THREADS);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, gated_dec_kernel<GS, NT>, a);
}

}  // namespace

bool gated_dec_supported(int64_t M, int64_t I, int64_t F, int gs, int num_sms) {
    if (M > GATED_DEC_MAX_M) return false;
    const int64_t tiles = (F + GD_TILE - 1) / GD_TILE, grid = tiles < num_sms ? tiles : num_sms;
    const int64_t own = (tiles + grid - 1) / grid;    // tiles of a CTA
    const int want = own < 4 ? static_cast<int>(own) : 4;
    const int fit = gd_pass_tiles(static_cast<int>(M), static_cast<int>(I), gs, M <= 8 ? 1 : 2, want);
    return fit >= want || (fit >= 2 && !skinny_supported(M, GATED_DEC_MAX_M, 2 * F, I));
}

cudaError_t launch_gated_dec(const uint16_t *x, int64_t M, int64_t I, int64_t F, const uint32_t *q,
                             const uint16_t *scales, const uint32_t *zeros, const uint16_t *s16, int gs, int act,
                             uint16_t *h, int num_sms, cudaStream_t st) {
    GdArgs a;
    a.x = x;
    a.q = q;
    a.scales = scales;
    a.zeros = zeros;
    a.s16 = s16;
    a.h = h;
    a.F = F;
    a.M = static_cast<int>(M);
    a.I = static_cast<int>(I);
    a.act = act;
    a.tiles = static_cast<int>((F + GD_TILE - 1) / GD_TILE);
    const int grid = a.tiles < num_sms ? a.tiles : num_sms, nt = M <= 8 ? 1 : 2;
    a.pass_tiles = gd_pass_tiles(a.M, a.I, gs, nt, (a.tiles + grid - 1) / grid);
    if (a.pass_tiles < 1) return cudaErrorInvalidConfiguration;
    if (nt == 1)
        return gs == 128 ? launch_gd<128, 1>(a, grid, st) : gs == 64 ? launch_gd<64, 1>(a, grid, st) : launch_gd<32, 1>(a, grid, st);
    return gs == 128 ? launch_gd<128, 2>(a, grid, st) : gs == 64 ? launch_gd<64, 2>(a, grid, st) : launch_gd<32, 2>(a, grid, st);
}

}  // namespace awq
