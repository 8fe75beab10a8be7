// Products with a packed weight matrix for up to a few hundred tokens, the weights dequantised on
// the way into the tensor cores (tcgen05), in both directions:
//
//   forward   D[o, m] = sum_i W[o, i] xs[m, i]     (the gated projections; A = W, K = in)
//   gradient  D[i, m] = sum_o W[o, i] dy[m, o]     (A = W^T, K = out)
//
// with the tokens on the MMA's N side (N = tokens rounded to 16, at most 144), so that few tokens
// cost few cycles, and 128 rows or columns of W on its M side.  Both directions share one stage:
// 128 rows x 128 columns of W as fp16, two blocks of [128 rows][64 columns] in 128-byte swizzled
// rows.  Read K-major, they are 128 rows of A and two 64-deep slabs of K; read MN-major, 128 columns
// of A^T and eight 16-deep steps of K.  Nothing but the descriptors differs.
//
// Bound: the dequantising warps' stages, 13 instructions a packed word and about 1300 cycles for 128 x 128.  No pipe
// is saturated (issue 54%, integer pipe 51%, shared-memory pipe 47%, tensor pipe 23% at 77 tokens): the warps wait for
// their codes, first of all, and for one another.  The packed weights need a third of that time from HBM.
// Measured: 22016 x 4096, 77 tokens 41 us a call (33 this kernel, 4 the second one, 3 the tokens' rows); 11008 <- 4096
// gradient, 19 tokens 25 us, of which 19 stages a CTA are 13.
//
// Roles: 24 warps dequantise, in three groups that take the stages in turn, so that one group computes
// while another stores (a thread: 32 columns of two rows, two 16-byte loads of codes fetched SK_PF
// of its stages ahead into registers; shift, LOP3, exact HSUB2 or HFMA2 to code - z, HMUL2 by
// Delta 2^-kW, eight 16-byte stores); one warp fetches the token tiles by TMA, one
// issues the MMAs, four write the results from TMEM, whose two accumulators let a tile's
// epilogue run beside the next tile's products.  Where every CTA has whole tiles (small layers), its last
// tile's results, which nothing runs beside, are shared out among these four and the dequantising warps.
//
// Split: the (tile, 128-deep stage) sequence is cut into equal contiguous ranges, one per CTA,
// one CTA per SM.  A tile that several CTAs share leaves fp32 partial sums in the workspace, and a
// second, small kernel adds them in the order of the CTAs and finishes the tile (four tokens a block:
// the last CTA of a tile doing it alone took 10 to 20 us more).  Nobody waits for another CTA.
//
// The nibble pairs (e, e + 4) of a word become neighbouring fp16 values, so the 8 columns of a word
// lie in the order (0,4,1,5,2,6,3,7).  Forward, the tokens' columns are stored in the same order;
// in the gradient it is the order of the accumulator's lanes, and the epilogue writes lane p to
// column frag_perm8(p) of its word.
//
// Every wait is bounded: a CTA that gives up raises its abort flag, writes NaN for its remaining tiles
// (partial sums and gradients, too: the steps that follow would add what was in the workspace before), waits
// (bounded) for its copies and MMAs in flight, frees its TMEM and leaves.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "awq_internal.h"
#include "awq_ptx.cuh"
#include "w4a16_act.cuh"
#include "w4a16_frag.cuh"

namespace awq {

namespace {

constexpr float SK_NAN = __builtin_nanf("");
constexpr int SK_GROUPS = 3;                           // groups of eight dequantising warps
constexpr int SK_DQ_WARPS = 8 * SK_GROUPS;
constexpr int SK_WARP_EPI = SK_DQ_WARPS, SK_WARP_TMA = SK_DQ_WARPS + 4, SK_WARP_MMA = SK_DQ_WARPS + 5;   // four epilogue warps: TMEM lane quadrants 0-3
constexpr int SK_THREADS = (SK_DQ_WARPS + 6) * 32;
constexpr int SK_PF = 1;                              // units of packed codes in flight per thread (SK_GROUPS times that per CTA)
constexpr int SK_A_BYTES = 32768;                     // 128 x 128 fp16
constexpr int SK_MAX_STAGES = 5;
constexpr int SK_MAX_N = 144;                         // tokens per tile: the most with three stages
static_assert(3 * (SK_A_BYTES + SK_MAX_N * 256) + 1024 + 2 * 16 * 128 * 4 + 2 * 256 * 4 + 512 <= 232448 && SK_GROUPS <= 3,
              "a ring stage for each group");
constexpr int SK_XBUF = 2 * 16 * 128 * 4;             // the epilogue's exchange of gate and up values
constexpr int SK_SETS = 1 + SK_DQ_WARPS / 4;          // sets of four warps, one per TMEM lane quadrant
constexpr int SK_SET_BYTES = SK_XBUF + 2 * 256 * 4;   // a set's exchange and token scales
static_assert((SK_SETS - 1) * SK_SET_BYTES <= 3 * (SK_A_BYTES + 16 * 256), "the dequantising sets' lie in the ring");
constexpr int SK_TAIL = SK_SET_BYTES + (4 * SK_MAX_STAGES + 5) * 8 + 32;

__device__ __forceinline__ uint64_t sk_desc_mn(uint32_t saddr) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>(16384 >> 4) << 16;             // the next 64 columns
    d |= static_cast<uint64_t>(1024 >> 4) << 32;              // the next 8 rows of K
    d |= static_cast<uint64_t>(1) << 46;
    d |= static_cast<uint64_t>(2) << 61;
    return d;
}

__device__ __forceinline__ uint32_t sk_sub(uint32_t a, uint32_t b) {
    const __half2 r = __hsub2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ uint32_t sk_fma(uint32_t a, uint32_t b, uint32_t c) {
    const __half2 r = __hfma2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b),
                              *reinterpret_cast<const __half2 *>(&c));
    return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ uint32_t sk_mul(uint32_t a, uint32_t b) {
    const __half2 r = __hmul2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&r);
}

__device__ __forceinline__ float sk_bf16(uint16_t b) { return __uint_as_float(static_cast<uint32_t>(b) << 16); }

// First unit of CTA c's range, and the CTA whose range holds unit u: the largest c with
// units c < (u + 1) grid.  (units (grid + 1) < 2^31, checked at the launch: a 64-bit division takes
// several times as long, and the finishing kernel waits for it.)
__device__ __forceinline__ int sk_first(const SkinnyArgs &a, int c) {
    return static_cast<int>(static_cast<uint32_t>(a.units) * static_cast<uint32_t>(c) / static_cast<uint32_t>(a.grid));
}
__device__ __forceinline__ int sk_owner(const SkinnyArgs &a, int u) {
    return static_cast<int>((static_cast<uint32_t>(u + 1) * static_cast<uint32_t>(a.grid) - 1u) / static_cast<uint32_t>(a.units));
}

// What thread e reads of the caller's tensors for K tokens' results: its column's s, or its tokens' dh.
template <int EPI, int K>
struct SkPre {
    uint16_t s, dh[K / 2];
};
template <int EPI, int K>
__device__ __forceinline__ SkPre<EPI, K> sk_pre(const SkinnyArgs &a, int t, int m0, int mcount, int c, int e) {
    SkPre<EPI, K> p;
    if (EPI == EPI_OUT) {
        const int64_t col = static_cast<int64_t>(t) * 128 + (e & ~7) + frag_perm8(e & 7);
        p.s = a.s16 && col < a.I ? __ldg(a.s16 + col) : 0x3C00;     // 1.0
    }
    if (EPI == EPI_GATED_BWD) {
        const int64_t f = static_cast<int64_t>(t) * 64 + (e & 63);
#pragma unroll
        for (int k2 = 0; k2 < K / 2; ++k2) {
            const int m = c + (e >> 6) * (K / 2) + k2;
            p.dh[k2] = f < a.F && m < mcount ? __ldcg(a.dh + (m0 + m) * a.F + f) : 0;
        }
    }
    return p;
}

// The results of K tokens (the tile's tokens c .. c + K - 1) from the accumulator's 128 lanes, thread e
// holding lane e's values.  sw: the layer's scale, NaN where the accumulator was never completed (a wait ran out), which
// makes every result NaN.  tsc, tsd: the tile's token scales.  bar: hardware barrier of the 128 threads.
// x: [K][128] floats of shared memory (gated products: lanes 64-127 hold the up values of lanes 0-63).
template <int EPI, int K>
__device__ __forceinline__ void sk_finish(const SkinnyArgs &a, int t, int m0, int mcount, int c, const float (&v)[K],
                                          const SkPre<EPI, K> &pre, int e, float sw, const float *tsc, const float *tsd, float *x, int bar) {
    if (EPI == EPI_OUT) {
        const int64_t col = static_cast<int64_t>(t) * 128 + (e & ~7) + frag_perm8(e & 7);
        if (col < a.I) {
            const float s = __half2float(__ushort_as_half(pre.s));
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (c + k < mcount)
                    a.out[(m0 + c + k) * a.I + col] =
                        __bfloat16_as_ushort(__float2bfloat16_rn(__fdividef((v[k] * sw) * tsc[c + k], s)));
        }
        return;
    }
#pragma unroll
    for (int k = 0; k < K; ++k) x[k * 128 + e] = v[k];
    named_bar_sync(bar, 128);
    const int64_t f = static_cast<int64_t>(t) * 64 + (e & 63);
    if (f < a.F) {
#pragma unroll
        for (int k2 = 0; k2 < K / 2; ++k2) {
            const int k = (e >> 6) * (K / 2) + k2, m = c + k;
            if (m < mcount) {
                // (the layer's factor first: it takes no sum out of fp32's range, the token's may)
                const float gv = (x[k * 128 + (e & 63)] * sw) * tsc[m];
                const float uv = (x[k * 128 + 64 + (e & 63)] * sw) * tsc[m];
                if (EPI == EPI_GATED) {
                    a.out[(m0 + m) * a.F + f] = __bfloat16_as_ushort(__float2bfloat16_rn(act_value(gv, a.act) * uv));
                } else {
                    float da;
                    const float av = act_both(gv, a.act, da);
                    const float dv = sk_bf16(pre.dh[k2]) * tsd[m];
                    uint16_t *dst = a.d16 + (m0 + m) * a.ldd + f;
                    dst[0] = __half_as_ushort(__float2half_rn((dv * uv) * da));
                    dst[a.F] = __half_as_ushort(__float2half_rn(dv * av));
                }
            }
        }
    }
}

// A token's scales: forward, its own; gradient of the gated product, 2^e; tsd: 2^-e of the gradients
// that EPI_GATED_BWD writes.
template <bool GRAD, int EPI>
__device__ __forceinline__ void sk_token_scale(const SkinnyArgs &a, int m, int kw, float &sc, float &sd) {
    const int ex = a.grow ? dgu_exp(__ldcg(a.grow + m), a.inner, kw) : 0;
    sc = GRAD && a.grow ? ldexpf(1.0f, ex) : __ldcg(a.sx + m);
    sd = EPI == EPI_GATED_BWD ? ldexpf(1.0f, -ex) : 0.0f;
}

// Tiles that several CTAs share: block (tile, four tokens), 128 threads.
template <bool GRAD, int EPI>
__global__ void __launch_bounds__(128) skinny_finish_kernel(const __grid_constant__ SkinnyArgs a) {
    __shared__ float x[4 * 128], tsc[4], tsd[4];
    griddep_launch_dependents();
    griddep_wait();
    const int T = blockIdx.x, b0 = T * a.ks, b1 = b0 + a.ks;
    // the CTAs that share the tile, [c0, c1]: ranges cover the units in order
    const int c0 = sk_owner(a, b0), c1 = sk_owner(a, b1 - 1);
    if (c0 == c1) return;                             // one CTA's own: done
    const int e = threadIdx.x, c = blockIdx.y * 4;
    const int tt = T / a.tiles, t = T - tt * a.tiles, m0 = tt * a.n;
    const int mcount = static_cast<int>(a.M - m0 < a.n ? a.M - m0 : a.n);
    if (c >= mcount) return;
    // Everything is asked for before anything is used: the kernel is as long as its chain of reads.
    const SkPre<EPI, 4> pre = sk_pre<EPI, 4>(a, t, m0, mcount, c, e);
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    // their slots: the first CTA's range began with or before the tile, the others' inside it
    const float4 *p = a.part + (static_cast<int64_t>(2 * c0 + 1) * (a.n / 4) + blockIdx.y) * 128 + e;
    constexpr int AHEAD = 4;
    float4 w[AHEAD];
    const int n = c1 - c0 + 1;
    auto slot = [&](int i) { return __ldcg(p + static_cast<int64_t>(2 * i - (i > 0 ? 1 : 0)) * (a.n / 4) * 128); };
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) w[i] = i < n ? slot(i) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const int kw = dq_exp(a.dmax);
    if (e < 4) {
        float sc = 0.0f, sd = 0.0f;
        if (c + e < mcount) sk_token_scale<GRAD, EPI>(a, m0 + c + e, kw, sc, sd);
        tsc[e] = sc;
        tsd[e] = sd;
    }
    for (int i0 = 0; i0 < n; i0 += AHEAD) {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            v[0] += w[i].x;
            v[1] += w[i].y;
            v[2] += w[i].z;
            v[3] += w[i].w;
        }
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
            w[i] = i0 + AHEAD + i < n ? slot(i0 + AHEAD + i) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
    __syncthreads();
    sk_finish<EPI, 4>(a, t, m0, mcount, c, v, pre, e, ldexpf(1.0f, kw), tsc - c, tsd - c, x, 0);
}

// WHOLE: no tile is shared, and the last tile's results are shared out among the sets of warps.
template <bool GRAD, int EPI, bool WHOLE>
__global__ void __launch_bounds__(SK_THREADS, 1)
    skinny_kernel(const __grid_constant__ CUtensorMap bmap, const __grid_constant__ SkinnyArgs a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *ring = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const int b_bytes = a.n * 256;                    // a token tile: two slabs of [n][64]
    const int stage = SK_A_BYTES + b_bytes, stages = a.stages;
    float *xbuf = reinterpret_cast<float *>(ring + stages * stage);     // [2][16 tokens][128 lanes]
    float *tsc = xbuf + 2 * 16 * 128, *tsd = tsc + 256;                 // per token: result scale, gradient scale
    uint64_t *a_full = reinterpret_cast<uint64_t *>(tsd + 256);
    uint64_t *b_full = a_full + SK_MAX_STAGES, *empty = b_full + SK_MAX_STAGES;
    uint64_t *acc_full = empty + SK_MAX_STAGES, *acc_empty = acc_full + 2, *drain = acc_empty + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

    griddep_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int u0 = sk_first(a, blockIdx.x), u1 = sk_first(a, blockIdx.x + 1);

    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) {
            mbar_init(&a_full[s], 8);                // the warps of one group
            mbar_init(&b_full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int h = 0; h < 2; ++h) {
            mbar_init(&acc_full[h], 1);
            mbar_init(&acc_empty[h], 4);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == SK_WARP_MMA) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    if (warp == SK_WARP_TMA && lane == 0) tma_prefetch_desc(&bmap);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // All 512 columns: the allocation starts at column 0, and a constant base keeps the MMAs'
    // operands in uniform registers.
    constexpr uint32_t tmem_base = 0;

    if (warp < SK_DQ_WARPS) {
        // ---- dequantise: group `grp` of eight warps takes every SK_GROUPS-th unit; thread = 32 columns
        // 32 q4 .. + 31 of rows r and r + 64 of the stage.  The four lanes of a row read its 64 bytes of
        // codes in one instruction: with a lane per half row and block instead, twice as many cache
        // lines an instruction made the L1 pipe the limit (77% busy).
        const int grp = warp >> 3, r = (threadIdx.x & 255) >> 2, q4 = threadIdx.x & 3;
        const int wpr = static_cast<int>(a.I / 8), nG = static_cast<int>(a.I >> a.lg), nzw = (nG + 7) / 8;
        // Raw loads of the units to come: nothing touches a value before its unit, so nothing waits
        // for it earlier.  Addresses are 32-bit offsets from the three base pointers (the packed
        // matrix is below 4 GB); a row or column past the end reads the first word instead and gets
        // a scale of zero.
        struct Raw {
            uint4 q[2];                               // codes of the two rows
            uint16_t s[2];
            uint32_t z[2];
            int g;                                    // the columns' group; bits 29, 30: row r, r + 64 is real
        } raw[SK_PF];
        int pt = (u0 + grp) / a.ks % a.tiles, pk = (u0 + grp) % a.ks;   // tile and K stage of the next load
        uint32_t qo = 0, so = 0, zo = 0;              // of row r; codes: words; scales: elements; zero words
        int g = 0, rem0 = 0, rem1 = 0;                // group; K positions left from row r's, row r + 64's first (<= 0: none)
        constexpr uint32_t GK = 128 * SK_GROUPS;      // K positions from a group's unit to its next
        const uint32_t qstep = GRAD ? GK * static_cast<uint32_t>(wpr) : GK / 8;
        const uint32_t sstep = GRAD ? GK * static_cast<uint32_t>(nG) : GK >> a.lg;
        const uint32_t zstep = GRAD ? GK * static_cast<uint32_t>(nzw) : 0u;
        const int gstep = GRAD ? 0 : static_cast<int>(GK >> a.lg);
        // from row r to row r + 64 of the stage: gate row to up row, or 64 rows of K
        const uint32_t drow = GRAD ? 64u : static_cast<uint32_t>(a.F);
        const uint32_t dq = drow * static_cast<uint32_t>(wpr), ds = drow * static_cast<uint32_t>(nG),
                       dz = drow * static_cast<uint32_t>(nzw);
        auto place = [&]() {
            int o, col;
            if (GRAD) {
                o = pk * 128 + r;
                col = pt * 128 + q4 * 32;
                rem0 = col < static_cast<int>(a.I) ? static_cast<int>(a.O) - o : -(1 << 30);
                rem1 = rem0 - 64;
            } else {                                  // 64 gate rows, then their up rows
                o = pt * 64 + r;
                col = pk * 128 + q4 * 32;
                rem0 = rem1 = o < static_cast<int>(a.F) ? static_cast<int>(a.I) - col : -(1 << 30);
            }
            g = col >> a.lg;
            qo = static_cast<uint32_t>(o) * static_cast<uint32_t>(wpr) + (static_cast<uint32_t>(col) >> 3);
            so = static_cast<uint32_t>(o) * static_cast<uint32_t>(nG) + static_cast<uint32_t>(g);
            zo = static_cast<uint32_t>(o) * static_cast<uint32_t>(nzw);
        };
        auto fetch = [&](Raw &w) {
            const bool r0 = rem0 > 0, r1 = rem1 > 0;
            w.g = g | (r0 ? 1 << 29 : 0) | (r1 ? 1 << 30 : 0);
            w.q[0] = __ldcs(reinterpret_cast<const uint4 *>(a.q + (r0 ? qo : 0u)));
            w.q[1] = __ldcs(reinterpret_cast<const uint4 *>(a.q + (r1 ? qo + dq : 0u)));
            w.s[0] = __ldg(a.scales + (r0 ? so : 0u));
            w.s[1] = __ldg(a.scales + (r1 ? so + ds : 0u));
            if (a.zeros) {
                const uint32_t zw = zo + (static_cast<uint32_t>(g) >> 3);
                w.z[0] = __ldg(a.zeros + (r0 ? zw : 0u));
                w.z[1] = __ldg(a.zeros + (r1 ? zw + dz : 0u));
            }
            pk += SK_GROUPS;
            if (pk < a.ks) {
                qo += qstep;
                so += sstep;
                zo += zstep;
                g += gstep;
                rem0 -= static_cast<int>(GK);
                rem1 -= static_cast<int>(GK);
            } else {
                while (pk >= a.ks) {                  // (K may be a single stage)
                    pk -= a.ks;
                    if (++pt == a.tiles) pt = 0;      // the next token tile
                }
                place();
            }
        };
        place();
#pragma unroll
        for (int u = 0; u < SK_PF; ++u) fetch(raw[u]);
        // The packed weights are the caller's, complete before the kernel in front of this one let it
        // start (rows16_kernel waits first); the exponent comes from that kernel.
        griddep_wait();
        const float dscale = ldexpf(1.0f, -dq_exp(a.dmax));
        const uint32_t P = 0x64006400u;
        // block of columns, row, and the first of this quarter's four 16-byte columns, swizzled.  The upper
        // block's lanes store their words in the order 2, 3, 0, 1, so that the eight lanes of a store
        // phase (two rows, four quarters) fall into eight 16-byte columns.
        const bool rot = q4 >= 2;
        const uint32_t row_off = static_cast<uint32_t>((q4 >> 1) * 16384 + r * 128);
        const uint32_t sx0 = static_cast<uint32_t>(((q4 & 1) * 4) ^ (r & 7) ^ (rot ? 2 : 0));
        // Unit n of the CTA sits in ring stage n % stages, in the phase of its n / stages-th use.  A
        // parity tells neighbouring phases apart only: unit n waits for unit n - stages, and unit n - 2
        // stages must be done by then, which the group's last unit, n - SK_GROUPS, has waited for
        // (units are consumed in order) if stages >= SK_GROUPS.
        uint32_t st = static_cast<uint32_t>(grp), ph = 1;
        bool ok = true;
        for (int ub = u0 + grp; ub < u1 && ok; ub += SK_GROUPS * SK_PF) {
#pragma unroll
            for (int u = 0; u < SK_PF; ++u) {
                if (ub + SK_GROUPS * u >= u1) break;
                uint4 v[4];
                auto dequant = [&](int b) {
                    uint32_t z = 8u;
                    if (a.zeros) z = (raw[u].z[b] >> (4 * (raw[u].g & 7))) & 15u;
                    const float df = raw[u].g & (1 << (29 + b)) ? __half2float(__ushort_as_half(raw[u].s[b])) * dscale : 0.0f;
                    const __half2 dh2 = __floats2half2_rn(df, df);
                    const uint32_t d = *reinterpret_cast<const uint32_t *>(&dh2);
                    const uint32_t z0 = (0x6400u | z) * 0x00010001u;             // 1024 + z
                    const uint32_t z1 = sk_sub(0x63806380u, z0);                 // 960 - (1024 + z) = -(64 + z)
                    const uint4 qv = raw[u].q[b];
                    const uint32_t w[4] = {rot ? qv.z : qv.x, rot ? qv.w : qv.y, rot ? qv.x : qv.z, rot ? qv.y : qv.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t w8 = w[j] >> 8;
                        // 1024 + c minus (1024 + z); (1024 + 16 c) / 16 minus (64 + z): both exact
                        v[j].x = sk_mul(sk_sub((w[j] & 0x000F000Fu) | P, z0), d);
                        v[j].y = sk_mul(sk_fma((w[j] & 0x00F000F0u) | P, 0x2C002C00u, z1), d);
                        v[j].z = sk_mul(sk_sub((w8 & 0x000F000Fu) | P, z0), d);
                        v[j].w = sk_mul(sk_fma((w8 & 0x00F000F0u) | P, 0x2C002C00u, z1), d);
                    }
                };
                dequant(0);
                ok = mbar_wait_warp(&empty[st], ph, abort_flag);
                if (!ok) break;
                uint8_t *dst = ring + st * stage + row_off;
#pragma unroll
                for (int j = 0; j < 4; ++j) *reinterpret_cast<uint4 *>(dst + ((sx0 ^ j) << 4)) = v[j];
                dequant(1);
#pragma unroll
                for (int j = 0; j < 4; ++j) *reinterpret_cast<uint4 *>(dst + 64 * 128 + ((sx0 ^ j) << 4)) = v[j];
                fetch(raw[u]);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&a_full[st]);
                st += SK_GROUPS;
                if (st >= static_cast<uint32_t>(stages)) {
                    st -= static_cast<uint32_t>(stages);
                    ph ^= 1u;
                }
            }
        }
        if (WHOLE) {
            // The last tile's results: this set's chunks of 16 tokens.  Its buffers lie in the ring, which the
            // MMAs have read by then.  (The barrier that every MMA is done has a single phase, unlike
            // acc_full, whose phases these warps have not followed.)
            const int e = threadIdx.x & 127, set = 1 + static_cast<int>(threadIdx.x >> 7), kw = dq_exp(a.dmax);
            const int T = (u1 - 1) / a.ks, tt = T / a.tiles, t = T - tt * a.tiles;
            const int m0 = tt * a.n, mcount = static_cast<int>(a.M - m0 < a.n ? a.M - m0 : a.n);
            float sc[2] = {0.0f, 0.0f}, sd[2] = {0.0f, 0.0f};
            for (int i = 0; i < 2; ++i)
                if (e + 128 * i < mcount) sk_token_scale<GRAD, EPI>(a, m0 + e + 128 * i, kw, sc[i], sd[i]);
            if (ok) ok = mbar_wait_warp(drain, 0, abort_flag);
            // (after a wait that ran out, NaN: whatever still lands in the ring, or is left in the accumulator)
            const float sw = named_bar_and(1 + set, 128, ok && !*abort_flag) ? ldexpf(1.0f, kw) : SK_NAN;
            tc_fence_after();
            float *xs = reinterpret_cast<float *>(ring + (set - 1) * SK_SET_BYTES), *ss = xs + 2 * 16 * 128;
            for (int i = 0; i < 2; ++i) {
                ss[e + 128 * i] = sc[i];
                ss[256 + e + 128 * i] = sd[i];
            }
            named_bar_sync(1 + set, 128);
            const uint32_t acc = tmem_base + (static_cast<uint32_t>(e & 96) << 16) +
                                 (static_cast<uint32_t>(T - u0 / a.ks) & 1u) * a.acc_cols;
            uint32_t flip = 0;
            for (int c = 16 * set; c < a.n; c += 16 * SK_SETS, flip ^= 1u) {
                const SkPre<EPI, 16> pre = sk_pre<EPI, 16>(a, t, m0, mcount, c, e);
                uint32_t rv[16];
                tmem_ld16_wait(acc + c, rv);
                float v[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) v[k] = __uint_as_float(rv[k]);
                sk_finish<EPI, 16>(a, t, m0, mcount, c, v, pre, e, sw, ss, ss + 256, xs + flip * (16 * 128), 1 + set);
                __syncwarp();
            }
        }
    } else if (warp == SK_WARP_TMA) {
        // ---- token tiles
        griddep_wait();
        uint32_t st = 0, ph = 1;
        int issued = 0;
        int tt = u0 / a.ks / a.tiles, t = u0 / a.ks - tt * a.tiles, k = u0 % a.ks;
        for (int u = u0; u < u1; ++u, ++issued) {
            if (!mbar_wait_warp(&empty[st], ph, abort_flag)) break;
            if (elect_one()) {
                uint8_t *dst = ring + st * stage + SK_A_BYTES;
                mbar_arrive_expect_tx(&b_full[st], static_cast<uint32_t>(b_bytes));
                tma_load_2d(dst, &bmap, &b_full[st], k * 128, tt * a.n);
                tma_load_2d(dst + a.n * 128, &bmap, &b_full[st], k * 128 + 64, tt * a.n);
            }
            __syncwarp();
            if (++st == static_cast<uint32_t>(stages)) {
                st = 0;
                ph ^= 1u;
            }
            if (++k == a.ks) {
                k = 0;
                if (++t == a.tiles) {
                    t = 0;
                    ++tt;
                }
            }
        }
        if (lane == 0)                                // wait (bounded) for the copies in flight
            for (int s = 0; s < stages; ++s)
                if (issued > s)
                    mbar_wait_drain(&b_full[(issued - 1 - s) % stages],
                                    static_cast<uint32_t>(((issued - 1 - s) / stages) & 1));
        __syncwarp();
    } else if (warp == SK_WARP_MMA) {
        const uint32_t idesc = idesc_f16_f32(128, a.n, false) | (GRAD ? 1u << 15 : 0u);
        const uint32_t ring0 = smem_u32(ring), lead = elect_one() ? 1u : 0u;
        const uint64_t da0 = GRAD ? sk_desc_mn(ring0) : sdesc_kmajor_sw128(ring0), db0 = sdesc_kmajor_sw128(ring0 + SK_A_BYTES);
        uint32_t st = 0, ph = 0, seg = 0;
        bool ok = true;
        int k = u0 % a.ks;
        bool fresh = true;                            // the first stage of a segment
        for (int u = u0; u < u1; ++u) {
            const uint32_t h = seg & 1u;
            if (fresh) {
                ok = mbar_wait_warp(&acc_empty[h], ((seg >> 1) & 1u) ^ 1u, abort_flag);
                if (!ok) break;
            }
            ok = mbar_wait_warp(&b_full[st], ph, abort_flag) && mbar_wait_warp(&a_full[st], ph, abort_flag);
            if (!ok) break;
            tc_fence_after();
            const uint32_t d = tmem_base + h * a.acc_cols;
            const uint64_t da = sdesc_at(da0, st * stage), db = sdesc_at(db0, st * stage), db2 = sdesc_at(db, a.n * 128);
            const bool end = k + 1 == a.ks || u + 1 == u1;
#pragma unroll
            for (int s = 0; s < 8; ++s)
                umma_f16_lead(lead, d, sdesc_at(da, GRAD ? s * 2048 : (s >> 2) * 16384 + (s & 3) * 32),
                              sdesc_at(s < 4 ? db : db2, (s & 3) * 32), idesc, s > 0 ? 1u : (fresh ? 0u : 1u));
            umma_commit_lead(lead, &empty[st]);
            if (end) umma_commit_lead(lead, &acc_full[h]);
            fresh = end;
            if (end) ++seg;
            if (++k == a.ks) k = 0;
            if (++st == static_cast<uint32_t>(stages)) {
                st = 0;
                ph ^= 1u;
            }
        }
        if (elect_one()) umma_commit(drain);
        __syncwarp();
        if (lane == 0) mbar_wait_drain(drain, 0);
        __syncwarp();
    } else {
        // ---- results
        griddep_wait();
        const int e = threadIdx.x - SK_WARP_EPI * 32; // lane of the accumulator
        const uint32_t quad = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const int kw = dq_exp(a.dmax);
        float sw = ldexpf(1.0f, kw);
        uint32_t seg = 0, flip = 0;
        int have = -1;                                // token tile whose scales are in tsc
        bool ok = true;
        for (int u = u0; u < u1; ++seg) {
            const int T = u / a.ks, tt = T / a.tiles, t = T - tt * a.tiles;
            const int b0 = T * a.ks, b1 = b0 + a.ks, end = b1 < u1 ? b1 : u1;
            const bool whole = WHOLE || (u == b0 && end == b1);
            const int m0 = tt * a.n, mcount = static_cast<int>(a.M - m0 < a.n ? a.M - m0 : a.n);
            const uint32_t h = seg & 1u, acc = tmem_base + quad + h * a.acc_cols;
            if (whole && tt != have) {
                named_bar_sync(1, 128);
                for (int m = e; m < mcount; m += 128) sk_token_scale<GRAD, EPI>(a, m0 + m, kw, tsc[m], tsd[m]);
                named_bar_sync(1, 128);
                have = tt;
            }
            // (one outcome for the four warps: they meet at barriers below; no wait after one that ran out)
            if (ok) ok = named_bar_and(1, 128, mbar_wait_sleep(&acc_full[h], (seg >> 1) & 1u, abort_flag));
            if (!ok) sw = SK_NAN;
            tc_fence_after();
            // a shared tile's partial sums: this CTA's slot [n / 4][128] of four tokens
            float4 *mine = a.part + static_cast<int64_t>(2 * blockIdx.x + (u0 > b0 ? 0 : 1)) * a.n * 32;
            for (int c = 0; c < a.n; c += WHOLE && end == u1 ? 16 * SK_SETS : 16) {
                uint32_t rv[16];
                tmem_ld16_wait(acc + c, rv);
                float v[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) v[k] = __uint_as_float(rv[k]);
                if (whole) {
                    sk_finish<EPI, 16>(a, t, m0, mcount, c, v, sk_pre<EPI, 16>(a, t, m0, mcount, c, e), e, sw, tsc, tsd, xbuf + flip * (16 * 128), 1);
                    flip ^= 1u;
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mine[(c / 4 + k) * 128 + e] = ok ? make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3])
                                                         : make_float4(SK_NAN, SK_NAN, SK_NAN, SK_NAN);
                }
                __syncwarp();
            }
            tc_fence_before();
            __syncwarp();
            if (ok && lane == 0) mbar_arrive(&acc_empty[h]);
            u = end;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == SK_WARP_MMA) {
        tc_fence_after();
        tmem_dealloc(*tmem_slot, 512);
    }
}

template <bool GRAD, int EPI>
cudaError_t launch_sk(const CUtensorMap &bmap, const SkinnyArgs &a, bool split, cudaStream_t st) {
    static bool attr_set[64][2] = {};                 // per device
    auto *kernel = split ? skinny_kernel<GRAD, EPI, false> : skinny_kernel<GRAD, EPI, true>;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64 || !attr_set[dev][split]) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 232448);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) attr_set[dev][split] = true;
    }
    const size_t smem = 1024 + static_cast<size_t>(a.stages) * (SK_A_BYTES + a.n * 256) + SK_TAIL;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.grid));
    cfg.blockDim = dim3(SK_THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kernel, bmap, a);
    if (e != cudaSuccess || !split) return e;
    return launch_after(skinny_finish_kernel<GRAD, EPI>,
                        dim3(static_cast<unsigned>(a.units / a.ks), static_cast<unsigned>(a.n / 4)), 128, st, a);
}

}  // namespace

SkinnyPlan skinny_plan(int64_t M, int64_t tiles, int64_t k, int num_sms) {
    SkinnyPlan p;
    const int64_t tt = (M + SK_MAX_N - 1) / SK_MAX_N; // token tiles, of equal width
    p.n = static_cast<int>(((M + tt - 1) / tt + 15) / 16 * 16);
    p.token_tiles = static_cast<int>((M + p.n - 1) / p.n);
    p.tiles = static_cast<int>(tiles);
    p.ks = static_cast<int>((k + 127) / 128);
    // CTAs.  Either as many to a tile as pay, c of them, all ranges inside one tile where c divides its
    // stages; or one on every SM, whose ranges begin and end anywhere in a tile.  A stage costs its CTA about 600
    // ns, the second kernel that shared tiles need 1 us (it starts while the first ends) and 60 ns per CTA of a
    // tile, ranges that cross tiles 600 ns to 3 us.  Measured (us on the device, without the aligned choice /
    // with it): 5632 x 1024 17 tokens 12.2 / 9.6, its gradient 25.8 / 20.2, 2816 x 1024 gradient 12.6 / 8.7; 11008 x
    // 2048, where every SM has work either way, 16.8 / 16.8.
    const int64_t T = tiles * p.token_tiles, units = T * p.ks;
    p.grid = num_sms;
    int64_t best = (units + num_sms - 1) / num_sms * 600 + 3000 + (num_sms + T - 1) / T * 60;
    for (int64_t c = 1; c <= p.ks && c <= 64 && T * c <= num_sms; ++c) {
        const int64_t cost = (p.ks + c - 1) / c * 600 + (c > 1 ? c * 60 + 1000 : 0) + (p.ks % c ? 600 : 0);
        if (cost < best) {
            best = cost;
            p.grid = static_cast<int>(T * c);
        }
    }
    if (p.grid > units) p.grid = static_cast<int>(units);
    p.part_vecs = static_cast<int64_t>(2) * p.grid * p.n * 32;
    return p;
}

cudaError_t launch_skinny(bool grad, int epi, const CUtensorMap &bmap, SkinnyArgs a, const SkinnyPlan &p, cudaStream_t st) {
    a.n = p.n;
    a.tiles = p.tiles;
    a.ks = p.ks;
    a.units = static_cast<int>(static_cast<int64_t>(p.tiles) * p.ks * p.token_tiles);
    a.grid = p.grid;
    // whether some CTA's range ends inside a tile
    bool split = false;
    for (int c = 1; c < p.grid && !split; ++c) split = static_cast<int64_t>(a.units) * c / p.grid % p.ks != 0;
    a.acc_cols = p.n <= 32 ? 32 : p.n <= 64 ? 64 : p.n <= 128 ? 128 : 256;
    const int fit = (232448 - 1024 - SK_TAIL) / (SK_A_BYTES + p.n * 256);
    a.stages = fit < SK_MAX_STAGES ? fit : SK_MAX_STAGES;
    if (a.stages < SK_GROUPS || static_cast<int64_t>(a.units) * (p.grid + 1) > INT32_MAX) return cudaErrorInvalidConfiguration;
    if (grad) return launch_sk<true, EPI_OUT>(bmap, a, split, st);
    return epi == EPI_GATED ? launch_sk<false, EPI_GATED>(bmap, a, split, st)
                            : launch_sk<false, EPI_GATED_BWD>(bmap, a, split, st);
}

}  // namespace awq
