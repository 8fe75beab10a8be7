// Dense 16-bit products on the tensor cores, D[m, n] = sum_k A[m, k] B[n, k] with fp32
// accumulation, and the epilogues of the operators that train through packed weights and
// score a vocabulary:
//
//   EPI_GATED      A = x / s (fp16), B = dequantised gate rows | up rows:
//                  h = act(g) * u, both projections, the activation and the product in one pass;
//   EPI_GATED_BWD  the same product, then dg = dh * u * act'(g) and du = dh * act(g) as fp16,
//                  each token scaled by a power of two (the operand of the product with W);
//   EPI_OUT        D * row scale / s[n], optionally added to an fp32 buffer: the input gradients
//                  (B read along its rows: K is W's row) and the head's weight gradient;
//   EPI_CE         logits = x W^T of one vocabulary tile: each row's maximum and sum of
//                  exponentials over the tile, and the label's logit; the logits stay on chip;
//   EPI_CE_T, EPI_CE_BWD_T   the same and the next for few tokens, the vocabulary on D's rows;
//   EPI_CE_BWD     exp(logit - lse) * dloss as bf16, one piece of the vocabulary, the label's entry apart.
//
// CTA pairs (clusters of two, one CTA per SM, persistent over output tiles): a tile is 256 rows
// x bn columns (bn <= 256, a multiple of 32) on tcgen05.mma.cta_group::2, M = 256, N = bn,
// K = 16.  Each CTA stages its own 128 rows of A and half of B's columns, 64 deep, by TMA into a
// 192 KB ring (six stages at bn = 256); the accumulator has two 256-column halves of TMEM, so the epilogue of a
// tile overlaps the main loop of the next.  Warps: 0 TMA, 1 MMA, from 4 on the epilogue (lane =
// row, two or four warps taking a row's 16-column chunks in turn).
// A K-major operand lies as [rows][64 k] in 128-byte swizzled rows; an operand read along its
// rows (MN-major) as blocks of [64 k][64 n], 8 KB each, in the same swizzle.
//
// Tiles are walked in bands of eight row tiles, the row tile fastest, so the pairs that run at
// one time share a few column tiles of B and one band of A in L2.
//
// The TMA and MMA warps run their loops warp-wide, one elected lane issuing, so that ring counters
// and descriptors live in uniform registers.  With one lane running the loop alone, a slab took
// at least 570 cycles whatever its width, and a 2048 x 32000 x 4096 product 359 us; so it is 326 us
// (1645 TFLOP/s, 99% of the measured 1652), 341 us with the K chunks of EPI_CE.
//
// Bound: the tensor pipe (active 94% of the cycles of a 2048 x 22016 x 4096 gated product, 245 us, and of EPI_CE's;
// in a loop the power limit sets its clock) wherever the tokens fill tiles of 256 rows; for few tokens the reading
// of the operand from HBM (EPI_CE_T, 13 tokens, 32000 x 4096: 45 us of 49 a call, 5.8 TB/s).
//
// Every wait is bounded, as in the other kernels: a CTA that gives up raises its abort flag, writes NaN for
// its remaining tiles (results, partial sums and gradients alike, so that no later step of the call adds
// what was in the workspace before), and leaves once the MMAs and the copies of both CTAs of the pair
// that are in flight have finished (bounded, too).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "awq_internal.h"
#include "awq_ptx.cuh"
#include "w4a16_act.cuh"

namespace awq {

namespace {

constexpr int GM_MAX_STAGES = 12;
constexpr int GM_A_BYTES = 128 * SLAB_K * 2;          // 16 KB: this CTA's rows of A
constexpr int GM_RING = 192 * 1024;                   // operand ring
constexpr int GM_EPI_WARP0 = 4;                       // the epilogue's warps: a row's 16-column chunks dealt to those of its quadrant
// Warps per TMEM lane quadrant; EPI_CE keeps 256 columns of a row in its threads' registers.
template <int EPI>
constexpr int GM_EPI_Q = EPI == EPI_CE ? 4 : 2;
template <int EPI>
constexpr int GM_THREADS = (GM_EPI_WARP0 + 4 * GM_EPI_Q<EPI>) * 32;
// The cross entropy's logits are accumulated GM_KCHUNK slabs (1024 columns) at a time on the tensor cores
// and added up in registers: the tensor cores truncate each 16-column step towards zero, and over
// a whole row the losses came out 1e-6 of themselves too low.  The gradients take K in one go: the same 1e-6 to
// 2.5e-6 of a logit (4096 columns; in proportion to the columns, 3e-5 at the most that are allowed) is a relative
// error of exp(logit - lse) of 5e-5 at a logit of 20, 6e-4 at the most columns, below the 2^-8 of the
// rounding to bf16 that follows.  It is not below it in the label's entry, a difference of nearly equal
// numbers: that one is formed from an fp32 logit (ce_labels).
template <int EPI>
constexpr int GM_KCHUNK = EPI == EPI_CE || EPI == EPI_CE_T ? 16 : 1 << 30;
constexpr int GM_BAND = 8;                            // row tiles walked together
constexpr uint32_t GM_TMEM = 512;
constexpr int GM_BARS = 2 * GM_MAX_STAGES + 4 + 2;
constexpr int GM_SMEM = 1024 + GM_RING + GM_BARS * 8 + 16;   // ... and four words behind the barriers
static_assert(GM_SMEM <= 232448, "shared memory plan");

// Shared-memory descriptor of an MN-major operand in the 128-byte swizzle: blocks of 64
// elements along MN (8192 bytes apart: 64 k rows of 128 bytes), 8 k rows per 1024-byte atom.
__device__ __forceinline__ uint64_t sdesc_mnmajor_sw128(uint32_t saddr) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>(8192 >> 4) << 16;              // leading byte offset: next 64 along MN
    d |= static_cast<uint64_t>(1024 >> 4) << 32;              // stride byte offset: next 8 along K
    d |= static_cast<uint64_t>(1) << 46;
    d |= static_cast<uint64_t>(2) << 61;
    return d;
}

struct Tile {
    int m, n;
};
__device__ __forceinline__ Tile decode_tile(int t, int mt, int nt) {
    const int band = t / (GM_BAND * nt);
    const int r = t - band * (GM_BAND * nt);
    const int h = mt - band * GM_BAND < GM_BAND ? mt - band * GM_BAND : GM_BAND;
    Tile o;
    o.n = r / h;
    o.m = band * GM_BAND + (r - o.n * h);
    return o;
}

// First slab of K split i.
__device__ __forceinline__ int split_at(int i, int nk, int splits) {
    return static_cast<int>(static_cast<int64_t>(nk) * i / splits);
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ float bf16f(uint16_t b) { return __uint_as_float(static_cast<uint32_t>(b) << 16); }

// 16 consecutive values to bf16 at p[0..16): 16-byte stores when the row allows (`vec`),
// else one by one below `n` values.
__device__ __forceinline__ void store_bf16_16(uint16_t *p, const float (&v)[16], bool vec, int64_t n) {
    if (vec && n >= 16) {
        uint4 *q = reinterpret_cast<uint4 *>(p);
        q[0] = make_uint4(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]), bf16x2(v[4], v[5]), bf16x2(v[6], v[7]));
        q[1] = make_uint4(bf16x2(v[8], v[9]), bf16x2(v[10], v[11]), bf16x2(v[12], v[13]), bf16x2(v[14], v[15]));
        return;
    }
#pragma unroll
    for (int k = 0; k < 16; ++k)
        if (k < n) p[k] = __bfloat16_as_ushort(__float2bfloat16_rn(v[k]));
}

// ---- epilogues of one thread's row (its TMEM lane at `acc`), tile columns [0, bn).  The TMEM
// loads are warp-wide: rows beyond M skip only the work between them, and every loop ends in a
// warp barrier.  `done` is false where the accumulator was never completed (a wait ran out): a scale
// of NaN then makes every result NaN.
constexpr float GM_NAN = __builtin_nanf("");

__device__ __forceinline__ void epi_gated(const GemmArgs &a, uint32_t acc, int64_t row, int64_t f0, int par, bool done) {
    const int half = a.bn / 2;
    const float sc = !done ? GM_NAN : row < a.M ? __ldcg(a.sx + row) : 0.0f;
    const float sw = dq_scale(a.dmax);
    const bool vec = a.F % 8 == 0;
#pragma unroll 1
    for (int c = 16 * par; c < half; c += 32) {
        uint32_t g[16], u[16];
        tmem_ld16_wait(acc + c, g);
        tmem_ld16_wait(acc + half + c, u);
        float h[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            // the two power-of-two factors one after the other, each a normal float, the layer's first: it is
            // between 2^-34 and 2^5 and takes no sum out of fp32's range, the token's may
            const float gv = (__uint_as_float(g[k]) * sw) * sc, uv = (__uint_as_float(u[k]) * sw) * sc;
            h[k] = act_value(gv, a.act) * uv;
        }
        if (row < a.M && f0 + c < a.F) store_bf16_16(a.out + row * a.F + f0 + c, h, vec, a.F - f0 - c);
        __syncwarp();
    }
}

__device__ __forceinline__ void epi_gated_bwd(const GemmArgs &a, uint32_t acc, int64_t row, int64_t f0, int par,
                                              bool done) {
    const int half = a.bn / 2;
    const bool ok = row < a.M;
    const float sc = !done ? GM_NAN : ok ? __ldcg(a.sx + row) : 0.0f;
    const int kw = dq_exp(a.dmax);
    const float sw = ldexpf(1.0f, kw);
    // 2^-e of this token's gradients
    const float sd = ok ? ldexpf(1.0f, -dgu_exp(__ldcg(a.grow + row), a.inner, kw)) : 0.0f;
    const uint16_t *dh = a.dh + (ok ? row : 0) * a.F;
    const bool vec = a.F % 8 == 0;
#pragma unroll 1
    for (int c = 16 * par; c < half; c += 32) {
        uint32_t g[16], u[16];
        tmem_ld16_wait(acc + c, g);
        tmem_ld16_wait(acc + half + c, u);
        if (ok && f0 + c < a.Fp) {
        uint32_t pg[8], pu[8];
        float dv[16];
        if (vec && f0 + c + 16 <= a.F) {
            const uint4 *p = reinterpret_cast<const uint4 *>(dh + f0 + c);
            const uint4 p0 = __ldcg(p), p1 = __ldcg(p + 1);
            const uint32_t w[8] = {p0.x, p0.y, p0.z, p0.w, p1.x, p1.y, p1.z, p1.w};
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                dv[2 * k] = __uint_as_float(w[k] << 16);
                dv[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
            }
        } else {
#pragma unroll
            for (int k = 0; k < 16; ++k) dv[k] = f0 + c + k < a.F ? bf16f(__ldcg(dh + f0 + c + k)) : 0.0f;
        }
#pragma unroll
        for (int k = 0; k < 16; k += 2) {
            float dg[2], du[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int64_t f = f0 + c + k + j;
                const float gv = (__uint_as_float(g[k + j]) * sw) * sc, uv = (__uint_as_float(u[k + j]) * sw) * sc;
                float da;
                const float av = act_both(gv, a.act, da);
                const float d = dv[k + j] * sd;
                // columns of the padding are exact zeros whatever the tile holds there
                dg[j] = f < a.F ? (d * uv) * da : 0.0f;
                du[j] = f < a.F ? d * av : 0.0f;
            }
            const __half2 hg = __floats2half2_rn(dg[0], dg[1]), hu = __floats2half2_rn(du[0], du[1]);
            pg[k / 2] = *reinterpret_cast<const uint32_t *>(&hg);
            pu[k / 2] = *reinterpret_cast<const uint32_t *>(&hu);
        }
        uint4 *qg = reinterpret_cast<uint4 *>(a.d16 + row * a.ldd + f0 + c);
        uint4 *qu = reinterpret_cast<uint4 *>(a.d16 + row * a.ldd + a.Fp + f0 + c);
        qg[0] = make_uint4(pg[0], pg[1], pg[2], pg[3]);
        qg[1] = make_uint4(pg[4], pg[5], pg[6], pg[7]);
        qu[0] = make_uint4(pu[0], pu[1], pu[2], pu[3]);
        qu[1] = make_uint4(pu[4], pu[5], pu[6], pu[7]);
        }
        __syncwarp();
    }
}

// A K split's partial sums: this unit's slot [bn / 4][256 rows] of four columns.
__device__ __forceinline__ void epi_part(const GemmArgs &a, uint32_t acc, int unit, int r, int par, bool done) {
    float4 *p = a.part4 + static_cast<int64_t>(unit) * (a.bn / 4) * 256;
#pragma unroll 1
    for (int c = 16 * par; c < a.bn; c += 32) {
        uint32_t v[16];
        tmem_ld16_wait(acc + c, v);
        if (!done)
#pragma unroll
            for (int k = 0; k < 16; ++k) v[k] = __float_as_uint(GM_NAN);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            p[(c / 4 + k) * 256 + r] = make_float4(__uint_as_float(v[4 * k]), __uint_as_float(v[4 * k + 1]),
                                                   __uint_as_float(v[4 * k + 2]), __uint_as_float(v[4 * k + 3]));
        __syncwarp();
    }
}

// A row's scale, as two factors that are normal floats each; sw, the layer's, is applied first (epi_gated).  (Warp-wide: the layer's exponent.)
__device__ __forceinline__ void out_scales(const GemmArgs &a, bool ok, int64_t row, float &sc, float &sw) {
    sc = sw = 1.0f;
    if (a.grow) {                                     // gated gradient: 2^e of the token
        const int kw = dq_exp(a.dmax);
        sc = ok ? ldexpf(1.0f, dgu_exp(__ldcg(a.grow + row), a.inner, kw)) : 0.0f;
        sw = ldexpf(1.0f, kw);
    } else if (a.sx) {
        sc = ok ? __ldcg(a.sx + row) : 0.0f;
        sw = dq_scale(a.dmax);
    }
}

// The gradient of a token's label, which is in fp32 and no part of the 16-bit ones: it adds its multiple of the
// label's row of the head to dx.
struct LabelTerm {
    const uint16_t *w;                                // null: none
    float r;
};
// (The head's gradient, a.owner: a row is an entry of the vocabulary, and what rounding took off the gradient of the
// first token that it labels adds its multiple of the token's row of x.)
__device__ __forceinline__ LabelTerm label_term(const GemmArgs &a, bool ok, int64_t row) {
    LabelTerm t = {nullptr, 0.0f};
    if (a.owner) {
        const int m = ok ? __ldcg(a.owner + row) : CE_NO_TOKEN;
        if (m != CE_NO_TOKEN) {
            t.w = a.x + m * a.N;
            t.r = bf16_rest(__ldcg(a.res + m));
        }
    } else if (a.res && a.last && ok) {
        const int64_t lab = __ldcg(a.labels + row);
        if (lab >= 0 && lab < a.V) {
            t.w = a.w + lab * a.N;
            t.r = __ldcg(a.res + row);
        }
    }
    return t;
}

// C columns n .. of the row that a label term adds.
template <int C>
__device__ __forceinline__ void label_columns(const LabelTerm &t, int64_t n, uint2 (&w)[C / 4]) {
    const bool any = t.w && t.r != 0.0f;
#pragma unroll
    for (int k = 0; k < C / 4; ++k)
        w[k] = any ? __ldcg(reinterpret_cast<const uint2 *>(t.w + n) + k) : make_uint2(0u, 0u);
}

// C consecutive scaled columns n .. of a row: divided by s, added to the pieces before, with the label's term, stored.
template <int C>
__device__ __forceinline__ void out_columns(const GemmArgs &a, int64_t row, int64_t n, const LabelTerm &t,
                                            const uint2 (&lw)[C / 4], float (&v)[C]) {
    if (a.s16) {
#pragma unroll
        for (int k = 0; k < C; k += 4) {
            const uint2 sv = __ldcg(reinterpret_cast<const uint2 *>(a.s16 + n + k));
            const __half2 s0 = *reinterpret_cast<const __half2 *>(&sv.x), s1 = *reinterpret_cast<const __half2 *>(&sv.y);
            v[k] = __fdividef(v[k], __low2float(s0));
            v[k + 1] = __fdividef(v[k + 1], __high2float(s0));
            v[k + 2] = __fdividef(v[k + 2], __low2float(s1));
            v[k + 3] = __fdividef(v[k + 3], __high2float(s1));
        }
    }
    if (a.acc) {
        float4 *q = reinterpret_cast<float4 *>(a.acc + row * a.N + n);
        if (!a.first) {
#pragma unroll
            for (int k = 0; k < C / 4; ++k) {
                const float4 p = q[k];
                v[4 * k] += p.x; v[4 * k + 1] += p.y; v[4 * k + 2] += p.z; v[4 * k + 3] += p.w;
            }
        }
        if (!a.last) {
#pragma unroll
            for (int k = 0; k < C / 4; ++k) q[k] = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
            return;
        }
    }
    if (t.w && t.r != 0.0f) {
#pragma unroll
        for (int k = 0; k < C; k += 4) {
            const uint2 w = lw[k / 4];
            v[k] = fmaf(t.r, __uint_as_float(w.x << 16), v[k]);
            v[k + 1] = fmaf(t.r, __uint_as_float(w.x & 0xFFFF0000u), v[k + 1]);
            v[k + 2] = fmaf(t.r, __uint_as_float(w.y << 16), v[k + 2]);
            v[k + 3] = fmaf(t.r, __uint_as_float(w.y & 0xFFFF0000u), v[k + 3]);
        }
    }
    uint2 *o = reinterpret_cast<uint2 *>(a.out + row * a.N + n);
    if constexpr (C % 8 == 0) {
#pragma unroll
        for (int k = 0; k < C / 8; ++k)
            reinterpret_cast<uint4 *>(o)[k] =
                make_uint4(bf16x2(v[8 * k], v[8 * k + 1]), bf16x2(v[8 * k + 2], v[8 * k + 3]),
                           bf16x2(v[8 * k + 4], v[8 * k + 5]), bf16x2(v[8 * k + 6], v[8 * k + 7]));
    } else {
        o[0] = make_uint2(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]));
    }
}

// (sc, sw, t: the row's, read before the accumulator is waited for)
__device__ __forceinline__ void epi_out(const GemmArgs &a, uint32_t acc, int64_t row, int64_t n0, int par, float sc,
                                        float sw, const LabelTerm &t) {
    const bool ok = row < a.M;
#pragma unroll 1
    for (int c = 16 * par; c < a.bn; c += 32) {
        const bool in = ok && n0 + c < a.N;           // N is a multiple of 64: a 16-column chunk is in or out
        uint2 lw[4];
        label_columns<16>(in ? t : LabelTerm{nullptr, 0.0f}, n0 + c, lw);
        uint32_t r[16];
        tmem_ld16_wait(acc + c, r);
        if (in) {
            float v[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) v[k] = (__uint_as_float(r[k]) * sw) * sc;
            out_columns<16>(a, row, n0 + c, t, lw, v);
        }
        __syncwarp();
    }
}

// Split tiles: block (tile, four columns), thread = row; the splits in order.
__global__ void __launch_bounds__(256) gemm_finish_kernel(const __grid_constant__ GemmArgs a) {
    griddep_launch_dependents();
    griddep_wait();
    const Tile tl = decode_tile(static_cast<int>(blockIdx.x), a.mt, a.nt);
    const int64_t row = static_cast<int64_t>(tl.m) * 256 + threadIdx.x;
    const int64_t n = static_cast<int64_t>(tl.n) * a.bn + blockIdx.y * 4;
    const bool ok = row < a.M && n < a.N;
    const float4 *p = a.part4 + (static_cast<int64_t>(blockIdx.x) * a.splits * (a.bn / 4) + blockIdx.y) * 256 + threadIdx.x;
    // the first partial sums are asked for before the scales: the kernel is as long as its chain of reads
    constexpr int AHEAD = 8;
    float4 w[AHEAD];
    auto slot = [&](int i) { return __ldcg(p + static_cast<int64_t>(i) * (a.bn / 4) * 256); };
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) w[i] = ok && i < a.splits ? slot(i) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float sc, sw;
    out_scales(a, row < a.M, row, sc, sw);
    if (!ok) return;
    const LabelTerm t = label_term(a, true, row);
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int i0 = 0; i0 < a.splits; i0 += AHEAD) {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            v[0] += w[i].x;
            v[1] += w[i].y;
            v[2] += w[i].z;
            v[3] += w[i].w;
        }
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
            w[i] = i0 + AHEAD + i < a.splits ? slot(i0 + AHEAD + i) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = (v[k] * sw) * sc;
    uint2 lw[1];
    label_columns<4>(t, n, lw);
    out_columns<4>(a, row, n, t, lw, v);
}

constexpr float LOG2E = 1.4426950408889634f;

// The logits of a row's chunks in registers, chunk i = columns 16 (sub + W i) .. + 15.
constexpr int CE_CHUNKS = 4;

// Add this K chunk's accumulator to them.
template <int W>
__device__ __forceinline__ void ce_gather(uint32_t acc, int bn, int sub, float (&v)[CE_CHUNKS][16]) {
#pragma unroll
    for (int i = 0; i < CE_CHUNKS; ++i) {
        const int c = 16 * (sub + W * i);
        if (c < bn) {
            uint32_t r[16];
            tmem_ld16_wait(acc + c, r);
#pragma unroll
            for (int k = 0; k < 16; ++k) v[i][k] += __uint_as_float(r[k]);
        }
    }
}

__device__ __forceinline__ void epi_ce(const GemmArgs &a, float (&v)[CE_CHUNKS][16], int64_t row, int64_t n0, int slot,
                                       int sub) {
    if (row >= a.M) return;
    const int64_t lab = __ldcg(a.labels + row);
    float mx = -INFINITY, sum = 0.0f;
#pragma unroll
    for (int i = 0; i < CE_CHUNKS; ++i) {
        const int c = 16 * (sub + 4 * i);
        const int64_t left = c < a.bn ? a.N - n0 - c : 0, j = lab - n0 - c;
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            // the label's own term joins in the last step (ce_final_kernel)
            if (k >= left || j == k) v[i][k] = -INFINITY;
            mx = fmaxf(mx, v[i][k]);
        }
    }
    // a tile of nothing but -inf (or NaN) keeps a finite reference
    const float ref = mx == -INFINITY ? 0.0f : mx;
#pragma unroll
    for (int i = 0; i < CE_CHUNKS; ++i)
#pragma unroll
        for (int k = 0; k < 16; ++k) sum += exp2f((v[i][k] - ref) * LOG2E);
    a.part[static_cast<int64_t>(slot) * a.M + row] = make_float2(mx, sum);
}

// The same for few tokens, the vocabulary on the rows (D's row = entry, column = token): a warp
// reduces its 32 entries of 16 tokens at a time.  Halving exchange: at each step a lane gives away half of
// its tokens and takes the partner's part of the other half, 8 + 4 + 2 + 1 shuffles and one more
// for 16 tokens; lane l then holds token l / 2.
template <bool SUM>
__device__ __forceinline__ float warp_reduce16(const float (&v)[16]) {
    const int lane = threadIdx.x & 31;
    auto op = [](float x, float y) { return SUM ? x + y : fmaxf(x, y); };
    float a8[8], a4[4], a2[2];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const float keep = lane & 16 ? v[8 + k] : v[k], give = lane & 16 ? v[k] : v[8 + k];
        a8[k] = op(keep, __shfl_xor_sync(0xffffffffu, give, 16));
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float keep = lane & 8 ? a8[4 + k] : a8[k], give = lane & 8 ? a8[k] : a8[4 + k];
        a4[k] = op(keep, __shfl_xor_sync(0xffffffffu, give, 8));
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const float keep = lane & 4 ? a4[2 + k] : a4[k], give = lane & 4 ? a4[k] : a4[2 + k];
        a2[k] = op(keep, __shfl_xor_sync(0xffffffffu, give, 4));
    }
    const float keep = lane & 2 ? a2[1] : a2[0], give = lane & 2 ? a2[0] : a2[1];
    const float r = op(keep, __shfl_xor_sync(0xffffffffu, give, 2));
    return op(r, __shfl_xor_sync(0xffffffffu, r, 1));
}

__device__ __forceinline__ void epi_ce_t(const GemmArgs &a, float (&v)[CE_CHUNKS][16], int64_t row, int slot, int sub) {
    const int lane = threadIdx.x & 31;
    const bool ok = row < a.M;
#pragma unroll
    for (int i = 0; i < CE_CHUNKS; ++i) {
        const int c = 16 * (sub + 2 * i);
        if (c < a.bn) {
            const int64_t m = c + (lane >> 1);        // the token this lane ends up with
            const int64_t mine = m < a.N ? __ldcg(a.labels + m) : -1;
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                const int64_t lab = __shfl_sync(0xffffffffu, mine, 2 * k);
                if (!ok || lab == row) v[i][k] = -INFINITY;
            }
            const float mx = warp_reduce16<false>(v[i]);
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                const float t = __shfl_sync(0xffffffffu, mx, 2 * k);
                v[i][k] = exp2f((v[i][k] - (t == -INFINITY ? 0.0f : t)) * LOG2E);
            }
            const float sum = warp_reduce16<true>(v[i]);
            if (m < a.N && (lane & 1) == 0) a.part[m * (8 * a.mt) + slot] = make_float2(mx, sum);
        }
    }
}

// The labels' logits in fp32 by the two warps that have no other work, a warp per token: products of
// bf16 values are exact, so this is the fp32 rounding of a few additions per lane.  The tensor
// cores' truncation shows most where the label dominates its row (2.5e-6 of the loss at 4096
// columns without this); the other terms of the sum average it out.  GRAD: the gradients of the labels' logits,
// (exp(t - lse) - 1) * dloss, of the labels in this piece of n entries: for a confident token t is nearly lse, and
// with a logit from the tensor cores 1 - p = 1e-4 came out 30% off.
template <bool GRAD>
__device__ __forceinline__ void ce_labels(const GemmArgs &a, int64_t tokens, int64_t n, int first, int step) {
    const int lane = threadIdx.x & 31;
    for (int64_t m = first; m < tokens; m += step) {
        const int64_t lab = __ldcg(a.labels + m);
        if (GRAD ? lab < a.v0 || lab >= a.v0 + n : lab < 0 || lab >= a.V) continue;
        const uint4 *x = reinterpret_cast<const uint4 *>(a.x + m * a.inner);
        const uint4 *w = reinterpret_cast<const uint4 *>(a.w + lab * a.inner);
        float s0 = 0.0f, s1 = 0.0f;
#pragma unroll 4
        for (int i = lane; i < a.inner / 8; i += 32) {
            const uint4 p = __ldcg(x + i), q = __ldcg(w + i);
            const uint32_t pv[4] = {p.x, p.y, p.z, p.w}, qv[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                s0 = fmaf(__uint_as_float(pv[k] << 16), __uint_as_float(qv[k] << 16), s0);
                s1 = fmaf(__uint_as_float(pv[k] & 0xFFFF0000u), __uint_as_float(qv[k] & 0xFFFF0000u), s1);
            }
        }
        float s = s0 + s1;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
        if (lane == 0) {
            if (GRAD)
                a.res[m] = expm1f(s - __ldcg(a.lse + m)) * __ldcg(a.dloss + m);
            else
                a.tgt[m] = s;
        }
    }
}

__device__ __forceinline__ void epi_ce_bwd(const GemmArgs &a, uint32_t acc, int64_t row, int64_t n0, int par, bool done) {
    const bool ok = row < a.M;
    const int64_t lab = ok ? __ldcg(a.labels + row) : -1;
    const bool scored = lab >= 0 && lab < a.V;
    const float lse = !done ? GM_NAN : ok ? __ldcg(a.lse + row) : 0.0f;
    const float w = ok ? __ldcg(a.dloss + row) : 0.0f;
#pragma unroll 1
    for (int c = 16 * par; c < a.bn; c += 32) {
        uint32_t r[16];
        tmem_ld16_wait(acc + c, r);
        if (ok && n0 + c < a.N) {
        float v[16];
        const int64_t j = lab - a.v0 - n0 - c;
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            const float p = exp2f((__uint_as_float(r[k]) - lse) * LOG2E);
            v[k] = scored && j != k ? p * w : 0.0f;
        }
        // the row stride is a multiple of 64: the store may run into the row's own padding
        store_bf16_16(a.d16 + row * a.ldd + n0 + c, v, true, 16);
        if (a.lo) {
#pragma unroll
            for (int k = 0; k < 16; ++k) v[k] = bf16_rest(v[k]);
            store_bf16_16(a.d16 + (a.lo + row) * a.ldd + n0 + c, v, true, 16);
        }
        }
        __syncwarp();
    }
}

// The gradients of few tokens, the vocabulary on the rows: the lanes of a warp are 32 neighbouring
// entries of a token's row.
__device__ __forceinline__ void epi_ce_bwd_t(const GemmArgs &a, uint32_t acc, int64_t row, int par, bool done) {
    const int lane = threadIdx.x & 31;
#pragma unroll 1
    for (int c = 16 * par; c < a.bn; c += 32) {
        uint32_t r[16];
        tmem_ld16_wait(acc + c, r);
        // lane k holds token c + k's label, log-sum and weight
        const int64_t m = c + (lane & 15);
        const bool in = m < a.N;
        const int64_t lab = in ? __ldcg(a.labels + m) : -1;
        const float lse = !done ? GM_NAN : in ? __ldcg(a.lse + m) : 0.0f, w = in ? __ldcg(a.dloss + m) : 0.0f;
        const int rel = lab >= 0 && lab < a.V ? static_cast<int>(lab) : -1;   // V <= 2^24
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            const int lk = __shfl_sync(0xffffffffu, rel, k);
            const float sk = __shfl_sync(0xffffffffu, lse, k), wk = __shfl_sync(0xffffffffu, w, k);
            const float p = exp2f((__uint_as_float(r[k]) - sk) * LOG2E);
            if (row < a.M && c + k < a.N) {
                const float d = lk >= 0 && lk != a.v0 + row ? p * wk : 0.0f;
                a.d16[(c + k) * a.ldd + row] = __bfloat16_as_ushort(__float2bfloat16_rn(d));
                if (a.lo) a.d16[(a.lo + c + k) * a.ldd + row] = __bfloat16_as_ushort(__float2bfloat16_rn(bf16_rest(d)));
            }
        }
    }
}

template <int EPI, bool BF16, bool A_MN, bool B_MN>
__global__ void __launch_bounds__(GM_THREADS<EPI>, 1)
    gemm16_kernel(const __grid_constant__ GemmMaps maps, const __grid_constant__ GemmArgs a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *ring = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint64_t *full = reinterpret_cast<uint64_t *>(ring + GM_RING);
    uint64_t *empty = full + GM_MAX_STAGES;
    uint64_t *acc_full = empty + GM_MAX_STAGES;            // [2]: accumulator halves
    uint64_t *acc_empty = acc_full + 2;                // [2]
    uint64_t *drain = acc_empty + 2;
    uint64_t *stopped = drain + 1;                     // the leader's: neither CTA issues any more copies
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(stopped + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    volatile uint32_t *issued = reinterpret_cast<volatile uint32_t *>(tmem_slot + 2);   // [2] the leader's: their numbers

    griddep_launch_dependents();
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    const int tiles = a.mt * a.nt * a.splits;          // units: the K splits of a tile are neighbours
    const int nk = a.nk[0] + a.nk[1];                  // 64-deep slabs of both K segments
    const int bh = a.bn / 2;                           // B columns of this CTA
    const int nb = (bh + 63) / 64;                     // blocks of 64 columns when B is MN-major
    const uint32_t stage = GM_A_BYTES + (B_MN ? nb * 8192 : (bh * 128 + 1023) / 1024 * 1024);
    const int fit = static_cast<int>(GM_RING / stage), stages = fit < GM_MAX_STAGES ? fit : GM_MAX_STAGES;

    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) {
            mbar_init(&full[s], 1);                    // the leader's expect_tx; bytes of both CTAs
            mbar_init(&empty[s], 1);                   // the leader's multicast commit
        }
        for (int h = 0; h < 2; ++h) {
            mbar_init(&acc_full[h], 1);
            mbar_init(&acc_empty[h], 2 * 4 * GM_EPI_Q<EPI>);   // epilogue warps of both CTAs
        }
        mbar_init(drain, 1);
        mbar_init(stopped, 2);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc_pair(tmem_slot, GM_TMEM);
        tmem_relinquish_pair();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&maps.a);
        tma_prefetch_desc(&maps.b);
    }
    tc_fence_before();
    cluster_sync_all();
    tc_fence_after();
    griddep_wait();                                   // the operands, scales and buffers of the kernels before
    // All 512 columns: the allocation starts at column 0, and a constant base keeps the MMAs' operands
    // in uniform registers.
    constexpr uint32_t tmem_base = 0;

    if (warp == 0) {
        uint32_t st = 0, ph = 1, n_issued = 0;
        bool ok = true;
        const uint32_t bytes = GM_A_BYTES + (B_MN ? nb * 8192 : bh * 128);
        for (int t = pair; t < tiles && ok; t += pairs) {
            const Tile tl = decode_tile(t / a.splits, a.mt, a.nt);
            const int m0 = tl.m * 256 + static_cast<int>(rank) * 128;
            const int n0 = EPI == EPI_GATED || EPI == EPI_GATED_BWD
                               ? tl.n * bh + static_cast<int>(rank) * static_cast<int>(a.F)   // gate | up rows
                               : tl.n * a.bn + static_cast<int>(rank) * bh;
            const int k0 = split_at(t % a.splits, nk, a.splits), k1 = split_at(t % a.splits + 1, nk, a.splits);
            for (int kb = k0; kb < k1; ++kb) {
                ok = mbar_wait_warp(&empty[st], ph, abort_flag);
                if (!ok) break;
                const uint32_t bar = cluster_addr(&full[st], 0);
                uint8_t *sa = ring + st * stage, *sb = sa + GM_A_BYTES;
                const bool seg = kb >= a.nk[0];
                const int ks = (seg ? kb - a.nk[0] : kb) * SLAB_K;
                const int ka = ks + (seg ? a.a_seg : 0), kk = ks + (seg ? a.b_seg : 0);
                if (elect_one()) {
                    if (rank == 0) mbar_arrive_expect_tx(&full[st], 2 * bytes);
                    if constexpr (A_MN) {
                        tma_load_2d_pair(sa, &maps.a, bar, m0, ka);
                        tma_load_2d_pair(sa + 8192, &maps.a, bar, m0 + 64, ka);
                    } else {
                        tma_load_2d_pair(sa, &maps.a, bar, ka, m0);
                    }
                    if constexpr (B_MN) {
                        tma_load_2d_pair(sb, &maps.b, bar, n0, kk);
                        if (nb > 1) tma_load_2d_pair(sb + 8192, &maps.b, bar, n0 + 64, kk);
                    } else {
                        tma_load_2d_pair(sb, &maps.b, bar, kk, n0);
                    }
                }
                __syncwarp();
                ++n_issued;
                if (++st == static_cast<uint32_t>(stages)) {
                    st = 0;
                    ph ^= 1u;
                }
            }
        }
        // Where this CTA's copies ended, for the leader (below).
        if (lane == 0) {
            st_cluster_u32(cluster_addr(const_cast<uint32_t *>(issued) + rank, 0), n_issued);
            mbar_arrive_release_cluster(cluster_addr(stopped, 0));
        }
        __syncwarp();
    } else if (warp == 1) {
        if (rank == 0) {
            const uint32_t idesc = idesc_f16_f32(256, a.bn, BF16) | (A_MN ? 1u << 15 : 0u) | (B_MN ? 1u << 16 : 0u);
            const uint32_t ring0 = smem_u32(ring), lead = elect_one() ? 1u : 0u;
            const uint64_t da0 = A_MN ? sdesc_mnmajor_sw128(ring0) : sdesc_kmajor_sw128(ring0);
            const uint64_t db0 = B_MN ? sdesc_mnmajor_sw128(ring0 + GM_A_BYTES) : sdesc_kmajor_sw128(ring0 + GM_A_BYTES);
            uint32_t st = 0, ph = 0, ti = 0;
            bool ok = true;
            for (int t = pair; t < tiles && ok; t += pairs) {
                const int k0 = split_at(t % a.splits, nk, a.splits), k1 = split_at(t % a.splits + 1, nk, a.splits);
                for (int kc = k0; kc < k1 && ok; kc += GM_KCHUNK<EPI>, ++ti) {
                    const uint32_t h = ti & 1u;
                    const int ke = k1 - kc < GM_KCHUNK<EPI> ? k1 : kc + GM_KCHUNK<EPI>;
                    ok = mbar_wait_warp(&acc_empty[h], ((ti >> 1) & 1u) ^ 1u, abort_flag);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t d = tmem_base + h * 256;
                    for (int kb = kc; kb < ke; ++kb) {
                        ok = mbar_wait_warp(&full[st], ph, abort_flag);
                        if (!ok) break;
                        tc_fence_after();
                        const uint64_t da = sdesc_at(da0, st * stage), db = sdesc_at(db0, st * stage);
#pragma unroll
                        for (int k = 0; k < SLAB_K / 16; ++k)
                            umma_f16_pair_lead(lead, d, sdesc_at(da, A_MN ? k * 2048 : k * 32),
                                               sdesc_at(db, B_MN ? k * 2048 : k * 32), idesc, (kb > kc || k > 0) ? 1u : 0u);
                        umma_commit_pair_lead(lead, &empty[st], 0x3);
                        if (kb == ke - 1) umma_commit_pair_lead(lead, &acc_full[h], 0x3);
                        if (++st == static_cast<uint32_t>(stages)) {
                            st = 0;
                            ph ^= 1u;
                        }
                    }
                }
            }
            if (elect_one()) umma_commit_pair(drain, 0x3);
            __syncwarp();
            // Every slab multiplied: every copy has landed.  Else a wait ran out, and copies may be in flight,
            // counted on this CTA's barriers: wait (bounded) for the last of every stage before either
            // CTA leaves.  A stage that only one of the CTAs asked for gets the other's part of its barrier here,
            // when no MMA waits for it any more.  (The copying warps may only now begin to wait for their last stage.)
            if (!ok && lane == 0 && mbar_wait_drain(drain, 0, 2 * AWQ_WAIT_CYCLES) &&
                mbar_wait_drain(stopped, 0, 2 * AWQ_WAIT_CYCLES)) {
                fence_cluster();
                const uint32_t i0 = issued[0], i1 = issued[1], most = i0 > i1 ? i0 : i1, n_st = static_cast<uint32_t>(stages);
                const uint32_t bytes = GM_A_BYTES + (B_MN ? nb * 8192 : bh * 128);
                for (uint32_t n = most > n_st ? most - n_st : 0; n < most; ++n) {
                    if (n >= i1) mbar_complete_tx(&full[n % n_st], bytes);
                    if (n >= i0) mbar_arrive_expect_tx(&full[n % n_st], bytes);
                    mbar_wait_drain(&full[n % n_st], (n / n_st) & 1u);
                }
            }
            __syncwarp();
        }
    } else if (warp < GM_EPI_WARP0) {
        if constexpr (EPI == EPI_CE || EPI == EPI_CE_T)
            ce_labels<false>(a, EPI == EPI_CE ? a.M : a.N, 0, static_cast<int>(blockIdx.x) * 2 + warp - 2, static_cast<int>(gridDim.x) * 2);
        if (EPI == EPI_CE_BWD && a.owner)
            for (int64_t v = (static_cast<int64_t>(blockIdx.x) * 2 + warp - 2) * 32 + lane; v < a.N; v += static_cast<int64_t>(gridDim.x) * 64)
                a.owner[v] = CE_NO_TOKEN;
        if constexpr (EPI == EPI_CE_BWD || EPI == EPI_CE_BWD_T)
            ce_labels<true>(a, EPI == EPI_CE_BWD ? a.M : a.N, EPI == EPI_CE_BWD ? a.N : a.M,
                            static_cast<int>(blockIdx.x) * 2 + warp - 2, static_cast<int>(gridDim.x) * 2);
    } else {
        const int quad = warp & 3, par = (warp - GM_EPI_WARP0) >> 2;
        const uint32_t acc0 = tmem_base + (static_cast<uint32_t>(quad * 32) << 16);
        uint32_t ti = 0;
        bool ok = true;
        auto await = [&]() {                          // the next accumulator half (none after one that did not come)
            if (ok) ok = __all_sync(0xffffffffu, mbar_wait_sleep(&acc_full[ti & 1u], (ti >> 1) & 1u, abort_flag));
            tc_fence_after();
            return ok;
        };
        auto release = [&]() {                        // ... may be overwritten
            tc_fence_before();
            __syncwarp();
            if (ok && lane == 0) mbar_arrive_cluster(cluster_addr(&acc_empty[ti & 1u], 0));
            ++ti;
        };
        for (int t = pair; t < tiles; t += pairs) {
            const Tile tl = decode_tile(t / a.splits, a.mt, a.nt);
            const int64_t row = static_cast<int64_t>(tl.m) * 256 + rank * 128 + quad * 32 + lane;
            if constexpr (EPI == EPI_CE || EPI == EPI_CE_T) {
                float v[CE_CHUNKS][16];
#pragma unroll
                for (int i = 0; i < CE_CHUNKS; ++i)
#pragma unroll
                    for (int k = 0; k < 16; ++k) v[i][k] = 0.0f;
                for (int kc = 0; kc < nk && await(); kc += GM_KCHUNK<EPI>) {
                    ce_gather<GM_EPI_Q<EPI>>(acc0 + (ti & 1u) * 256, a.bn, par, v);
                    release();
                }
                if (!ok)
#pragma unroll
                    for (int i = 0; i < CE_CHUNKS; ++i)
#pragma unroll
                        for (int k = 0; k < 16; ++k) v[i][k] = GM_NAN;
                if constexpr (EPI == EPI_CE)
                    epi_ce(a, v, row, static_cast<int64_t>(tl.n) * a.bn, 4 * tl.n + par, par);
                else
                    epi_ce_t(a, v, row, tl.m * 8 + static_cast<int>(rank) * 4 + quad, par);
                __syncwarp();
                continue;
            }
            float sc = 1.0f, sw = 1.0f;
            LabelTerm lt = {nullptr, 0.0f};
            if constexpr (EPI == EPI_OUT)
                if (a.splits == 1) {
                    out_scales(a, row < a.M, row, sc, sw);
                    lt = label_term(a, row < a.M, row);
                }
            if (!await()) sc = GM_NAN;
            const uint32_t acc = acc0 + (ti & 1u) * 256;
            if constexpr (EPI == EPI_GATED) epi_gated(a, acc, row, static_cast<int64_t>(tl.n) * bh, par, ok);
            if constexpr (EPI == EPI_GATED_BWD) epi_gated_bwd(a, acc, row, static_cast<int64_t>(tl.n) * bh, par, ok);
            if constexpr (EPI == EPI_OUT) {
                if (a.splits > 1)
                    epi_part(a, acc, t, static_cast<int>(rank) * 128 + quad * 32 + lane, par, ok);
                else
                    epi_out(a, acc, row, static_cast<int64_t>(tl.n) * a.bn, par, sc, sw, lt);
            }
            if constexpr (EPI == EPI_CE_BWD_T) epi_ce_bwd_t(a, acc, row, par, ok);
            if constexpr (EPI == EPI_CE_BWD) epi_ce_bwd(a, acc, row, static_cast<int64_t>(tl.n) * a.bn, par, ok);
            release();
        }
    }

    tc_fence_before();
    __syncthreads();
    // Every pair MMA has finished (the leader's last commit reaches both CTAs) before TMEM is
    // freed, and neither CTA leaves while the other may still signal its barriers or read its
    // shared memory.
    if (warp == 1 && lane == 0) mbar_wait_drain(drain, 0);
    __syncwarp();
    cluster_sync_all();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(*tmem_slot, GM_TMEM);
    }
}

template <int EPI, bool BF16, bool A_MN, bool B_MN>
cudaError_t launch_t(const GemmMaps &maps, const GemmArgs &a, int num_sms, cudaStream_t st) {
    auto *kernel = gemm16_kernel<EPI, BF16, A_MN, B_MN>;
    cudaError_t e;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(GM_THREADS<EPI>);
    cfg.dynamicSmemBytes = GM_SMEM;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    // Persistent: as many pairs as can be resident at once (one CTA per SM).
    static int max_pairs[64] = {};
    int dev = 0;
    e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    int pairs = dev >= 0 && dev < 64 ? max_pairs[dev] : 0;
    if (pairs == 0) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, GM_SMEM);
        if (e != cudaSuccess) return e;
        cfg.gridDim = dim3(static_cast<unsigned>(2 * (num_sms / 2)));
        e = cudaOccupancyMaxActiveClusters(&pairs, kernel, &cfg);
        if (e != cudaSuccess) return e;
        if (pairs < 1) return cudaErrorInvalidConfiguration;
        if (dev >= 0 && dev < 64) max_pairs[dev] = pairs;
    }
    const int tiles = a.mt * a.nt * a.splits;
    cfg.gridDim = dim3(static_cast<unsigned>(2 * (tiles < pairs ? tiles : pairs)));
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, maps, a);
}

}  // namespace

// Measured cycles (at 1.9 GHz) of a 64-deep slab of a tile bn columns wide, K-major and MN-major B alike: 64
// columns 410-450, 128 460-490, 192 530-560, 224 610, 256 690-720: a handshake and the A tile cost
// about 350 beside one a column, until the MMAs themselves take over at 224.
static int slab_cycles(int bn) { return bn <= 192 ? 350 + bn : 272 * bn / 100; }

// Tile columns: of the multiples of 32 up to 256 the one with the least waves x time of a slab.
int gemm_tile_cols(int64_t M, int64_t N, int num_sms) {
    const int64_t mt = (M + 255) / 256, pairs = num_sms / 2;
    int best = 256;
    int64_t cost = INT64_MAX;
    for (int bn = 256; bn >= 64; bn -= 32) {
        const int64_t tiles = mt * ((N + bn - 1) / bn);
        const int64_t c = (tiles + pairs - 1) / pairs * slab_cycles(bn);
        if (c < cost) {
            cost = c;
            best = bn;
        }
    }
    return best;
}

GemmPlan gemm_plan(int64_t M, int64_t N, int64_t k, int num_sms) {
    const int64_t mt = (M + 255) / 256, pairs = num_sms / 2, nk = (k + 63) / 64;
    GemmPlan p{256, 1, 0};
    int64_t cost = INT64_MAX;
    for (int bn = 256; bn >= 64; bn -= 32) {
        const int64_t tiles = mt * ((N + bn - 1) / bn);
        // Tiles that leave pairs idle: K is split among them, at least 8 slabs to a split; the second
        // kernel costs about 3 us.
        int64_t s = pairs / tiles;
        s = s < nk / 8 ? s : nk / 8;
        if (s < 2) s = 1;
        const int64_t c = (tiles * s + pairs - 1) / pairs * ((nk + s - 1) / s) * slab_cycles(bn) + (s > 1 ? 6000 : 0);
        if (c < cost) {
            cost = c;
            p.bn = bn;
            p.splits = static_cast<int>(s);
            p.part_vecs = s > 1 ? tiles * s * (bn / 4) * 256 : 0;
        }
    }
    return p;
}

cudaError_t launch_gemm16(int epi, bool bf16, bool a_mn, const GemmMaps &maps, const GemmArgs &a, int num_sms,
                          cudaStream_t st) {
    if (a.splits > 1) {
        const cudaError_t e = a_mn ? launch_t<EPI_OUT, true, true, true>(maps, a, num_sms, st)
                              : bf16 ? launch_t<EPI_OUT, true, false, true>(maps, a, num_sms, st)
                                     : launch_t<EPI_OUT, false, false, true>(maps, a, num_sms, st);
        if (e != cudaSuccess) return e;
        return launch_after(gemm_finish_kernel, dim3(static_cast<unsigned>(a.mt * a.nt), static_cast<unsigned>(a.bn / 4)), 256, st, a);
    }
    switch (epi) {
        case EPI_GATED: return launch_t<EPI_GATED, false, false, false>(maps, a, num_sms, st);
        case EPI_GATED_BWD: return launch_t<EPI_GATED_BWD, false, false, false>(maps, a, num_sms, st);
        case EPI_CE: return launch_t<EPI_CE, true, false, false>(maps, a, num_sms, st);
        case EPI_CE_T: return launch_t<EPI_CE_T, true, false, false>(maps, a, num_sms, st);
        case EPI_CE_BWD_T: return launch_t<EPI_CE_BWD_T, true, false, false>(maps, a, num_sms, st);
        case EPI_CE_BWD: return launch_t<EPI_CE_BWD, true, false, false>(maps, a, num_sms, st);
        default:
            if (a_mn) return launch_t<EPI_OUT, true, true, true>(maps, a, num_sms, st);
            return bf16 ? launch_t<EPI_OUT, true, false, true>(maps, a, num_sms, st)
                        : launch_t<EPI_OUT, false, false, true>(maps, a, num_sms, st);
    }
}

// ------------------------------------------------------------------ cross entropy, last step
namespace {

__device__ __forceinline__ void join(float &mx, float &sum, float om, float os) {
    const float nm = fmaxf(mx, om), ref = nm == -INFINITY ? 0.0f : nm;
    sum = sum * exp2f((mx - ref) * LOG2E) + os * exp2f((om - ref) * LOG2E);
    mx = nm;
}

// The partial (maximum, sum) pairs of each token to the log of its sum of exponentials.  ROWS: one
// token per block, pairs [token][n] (few tokens, many pairs); else eight tokens per block, pairs
// [n][token], 64 contiguous bytes a pair.  Each thread takes its pairs in order, the threads meet in a
// fixed tree.
template <bool ROWS>
__global__ void __launch_bounds__(256) ce_final_kernel(const float2 *__restrict__ part, int n, int64_t M,
                                                       const int64_t *__restrict__ labels, int64_t V,
                                                       const float *__restrict__ tgt, float *__restrict__ loss,
                                                       float *__restrict__ lse) {
    griddep_wait();
    __shared__ float2 sm[8][8];
    constexpr int T = ROWS ? 1 : 8;                   // tokens of the block
    const int tok = threadIdx.x % T, at = threadIdx.x / T;
    const int64_t m = static_cast<int64_t>(blockIdx.x) * T + tok;
    float mx = -INFINITY, sum = 0.0f;
    if (m < M) {
#pragma unroll 4
        for (int t = at; t < n; t += 256 / T) {
            const float2 p = __ldcg(ROWS ? part + m * n + t : part + static_cast<int64_t>(t) * M + m);
            join(mx, sum, p.x, p.y);
        }
    }
#pragma unroll
    for (int off = 16; off >= T; off >>= 1) {
        const float om = __shfl_xor_sync(0xffffffffu, mx, off), os = __shfl_xor_sync(0xffffffffu, sum, off);
        join(mx, sum, om, os);
    }
    if ((threadIdx.x & 31) < T) sm[threadIdx.x >> 5][tok] = make_float2(mx, sum);
    __syncthreads();
    if (threadIdx.x >= T || m >= M) return;
    mx = sm[0][tok].x;
    sum = sm[0][tok].y;
#pragma unroll
    for (int w = 1; w < 8; ++w) join(mx, sum, sm[w][tok].x, sm[w][tok].y);
    const int64_t lab = __ldcg(labels + m);
    if (lab < 0 || lab >= V) {
        lse[m] = mx + logf(sum);
        loss[m] = 0.0f;
        return;
    }
    // with the label's term t, which `part` leaves out: loss = log(1 + sum e^(mx - t)), written so
    // that neither a label far above the others nor one far below loses digits
    const float t = __ldcg(tgt + m), d = mx - t;
    const float l = d > 0.0f ? d + logf(sum + expf(-d)) : log1pf(sum * expf(d));
    loss[m] = l;
    lse[m] = t + l;
}

}  // namespace

cudaError_t launch_ce_final(const float2 *part, int n, bool rows, int64_t M, const int64_t *labels, int64_t V,
                            const float *tgt, float *loss, float *lse, cudaStream_t st) {
    return rows ? launch_after(ce_final_kernel<true>, dim3(static_cast<unsigned>(M)), 256, st, part, n, M, labels, V, tgt, loss, lse)
                : launch_after(ce_final_kernel<false>, dim3(static_cast<unsigned>((M + 7) / 8)), 256, st, part, n, M, labels, V,
                               tgt, loss, lse);
}

}  // namespace awq
