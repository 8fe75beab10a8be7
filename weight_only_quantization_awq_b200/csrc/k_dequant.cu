// Operand preparation of the dense products (k_dense.cu): packed 4-bit weights to fp16, and token
// rows to fp16 with a power-of-two scale of their own.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "awq_internal.h"
#include "awq_ptx.cuh"
#include "w4a16_act.cuh"

namespace awq {

namespace {

// Largest |Delta| of one of DMAX_PARTS parts of the layer's scales, as fp16 bits, into dmax[part]
// (a block of 128 or 256 threads).
__device__ __forceinline__ void scales_max(const uint16_t *__restrict__ scales, int64_t n, int part, unsigned *dmax) {
    __shared__ unsigned wm[8];
    const int T = static_cast<int>(blockDim.x);
    const int64_t first = static_cast<int64_t>(part) * T + threadIdx.x, step = static_cast<int64_t>(DMAX_PARTS) * T;
    // 16 bytes at a time from the first 16-byte boundary on; the ragged ends one by one
    unsigned mb = 0u;
    const int64_t head = ((16 - (reinterpret_cast<uintptr_t>(scales) & 15)) & 15) / 2;
    const int64_t h = head < n ? head : n, vecs = (n - h) / 8;
    const uint4 *v = reinterpret_cast<const uint4 *>(scales + h);
    for (int64_t i = first; i < vecs; i += step) {
        const uint4 q = __ldg(v + i);
        // two 15-bit magnitudes to a word: the maximum of each half on its own
        const unsigned m = __vmaxu2(__vmaxu2(q.x & 0x7FFF7FFFu, q.y & 0x7FFF7FFFu),
                                    __vmaxu2(q.z & 0x7FFF7FFFu, q.w & 0x7FFF7FFFu));
        mb = max(mb, max(m >> 16, m & 0xFFFFu));
    }
    const int64_t rest = h + n - (h + vecs * 8);
    for (int64_t i = first; i < rest; i += step)
        mb = max(mb, static_cast<unsigned>(__ldg(scales + (i < h ? i : vecs * 8 + i))) & 0x7FFFu);
    mb = __reduce_max_sync(0xffffffffu, mb);
    if ((threadIdx.x & 31) == 0) wm[threadIdx.x >> 5] = mb;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int k = 1; k < T / 32; ++k) mb = max(mb, wm[k]);
        dmax[part] = mb;
    }
}

// Row elements [c, c + 8) as bf16 bits, zeros past the end.
__device__ __forceinline__ uint4 row_chunk(const uint16_t *__restrict__ r, int64_t c, int64_t cols, bool vec) {
    if (c >= cols) return make_uint4(0u, 0u, 0u, 0u);
    if (vec) return __ldcg(reinterpret_cast<const uint4 *>(r + c));
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint32_t lo = c + 2 * e < cols ? __ldcg(r + c + 2 * e) : 0u;
        const uint32_t hi = c + 2 * e + 1 < cols ? __ldcg(r + c + 2 * e + 1) : 0u;
        w[e] = lo | hi << 16;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// 1 / y of an fp16 value y, to 1 ulp: inside its range the plain instruction needs no scaling around it.
__device__ __forceinline__ float rcp16(float y) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(y));
    return r;
}

// v[0..8) = the chunk's values, divided by s where given (2 ulp: far below the fp16 rounding that follows).
__device__ __forceinline__ void row_values(const uint4 &x, const uint16_t *__restrict__ s16, int64_t c, float (&v)[8]) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        v[2 * e] = __uint_as_float(w[e] << 16);
        v[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
    }
    if (s16) {                                        // cols is a multiple of 64 here
        const uint4 sv = __ldg(reinterpret_cast<const uint4 *>(s16 + c));
        const uint32_t sw[4] = {sv.x, sv.y, sv.z, sv.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const __half2 h = *reinterpret_cast<const __half2 *>(&sw[e]);
            v[2 * e] *= rcp16(__low2float(h));
            v[2 * e + 1] *= rcp16(__high2float(h));
        }
    }
}

__device__ __forceinline__ float block_max(float v, float *sm) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
    if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
    __syncthreads();
    v = sm[0];
    for (int k = 1; k < static_cast<int>(blockDim.x >> 5); ++k) v = fmaxf(v, sm[k]);
    __syncthreads();
    return v;
}

__device__ __forceinline__ float block_sum(float v, float *sm) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
    __syncthreads();
    v = sm[0];
    for (int k = 1; k < static_cast<int>(blockDim.x >> 5); ++k) v += sm[k];
    __syncthreads();
    return v;
}

// Blocks from DMAX_PARTS on: one token each.  out[m] = fp16((row / s) * 2^-k), k from the row's largest
// magnitude so that it lands in [2^14, 2^15); sx[m] = 2^k.  With dh: grow[m], an exponent
// that bounds max |dh[m]| * ||row / s||.  The first blocks: the parts' largest |Delta|.
// Bound: latency for few tokens (3 us), the reads and writes of the rows and each warp's share of scalar work for
// many (2048 rows of 4096: 12.6 us; the row stays packed in registers between the two passes).
template <bool GROW>
__global__ void __launch_bounds__(256) rows16_kernel(const uint16_t *__restrict__ x, const uint16_t *__restrict__ s16,
                                                     int64_t M, int64_t cols, int64_t ld,
                                                     const uint16_t *__restrict__ dh, int64_t F,
                                                     const uint16_t *__restrict__ scales, int64_t n_scales,
                                                     bool permute, uint16_t *__restrict__ out, float *__restrict__ sx,
                                                     int *__restrict__ grow, unsigned *__restrict__ dmax) {
    griddep_wait();
    // The products that follow wait for this kernel themselves, but read their weights before: by now the
    // kernel before this one, which may have written them, is done.
    griddep_launch_dependents();
    if (blockIdx.x < DMAX_PARTS) {
        scales_max(scales, n_scales, static_cast<int>(blockIdx.x), dmax);
        return;
    }
    __shared__ float sm[8];
    const int64_t m = blockIdx.x - DMAX_PARTS;
    const uint16_t *r = x + m * cols;
    const bool vec = cols % 8 == 0;
    const int T = static_cast<int>(blockDim.x);
    constexpr int KEEP = 4;                           // chunks of a thread that stay in registers between the passes
    uint4 kept[KEEP];
    float mx = 0.0f, v[8];
#pragma unroll
    for (int i = 0; i < KEEP; ++i) kept[i] = row_chunk(r, (i * T + threadIdx.x) * 8, cols, vec);
    float md = 0.0f;
    if (GROW) {                                       // the token's largest |dh|
        const uint16_t *dr = dh + m * F;
        if (F % 8 == 0) {
            unsigned mb = 0u;                         // magnitudes of bf16 order as their bits
#pragma unroll 4
            for (int64_t f = threadIdx.x; f < F / 8; f += T) {
                const uint4 q = __ldcg(reinterpret_cast<const uint4 *>(dr) + f);
                mb = __vmaxu2(mb, __vmaxu2(__vmaxu2(q.x & 0x7FFF7FFFu, q.y & 0x7FFF7FFFu),
                                           __vmaxu2(q.z & 0x7FFF7FFFu, q.w & 0x7FFF7FFFu)));
            }
            md = __uint_as_float(max(mb >> 16, mb & 0xFFFFu) << 16);
        } else {
            for (int64_t f = threadIdx.x; f < F; f += T)
                md = fmaxf(md, fabsf(__uint_as_float(static_cast<uint32_t>(__ldcg(dr + f)) << 16)));
        }
    }
    auto largest = [&](int64_t c, const uint4 &x8) {
        row_values(x8, s16, c, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) mx = fmaxf(mx, fabsf(v[e]));
    };
#pragma unroll
    for (int i = 0; i < KEEP; ++i) {
        const int64_t c = (i * T + threadIdx.x) * 8;
        if (c < cols) largest(c, kept[i]);
    }
    for (int64_t c = (KEEP * T + threadIdx.x) * 8; c < cols; c += T * 8) largest(c, row_chunk(r, c, cols, vec));
    mx = block_max(mx, sm);
    const int k = scale_exp(mx, 15);
    const float sc = ldexpf(1.0f, -k);
    float sq = 0.0f;                                  // of the scaled values: no overflow
    auto put = [&](int64_t c, const uint4 &x8) {
        row_values(x8, s16, c, v);
        uint32_t h[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float lo = (permute ? v[e] : v[2 * e]) * sc, hi = (permute ? v[e + 4] : v[2 * e + 1]) * sc;
            if (GROW) sq = fmaf(lo, lo, fmaf(hi, hi, sq));
            const __half2 hv = __floats2half2_rn(lo, hi);
            h[e] = *reinterpret_cast<const uint32_t *>(&hv);
        }
        // ld is a multiple of 8: a last partial chunk stays inside its own row
        *reinterpret_cast<uint4 *>(out + m * ld + c) = make_uint4(h[0], h[1], h[2], h[3]);
    };
#pragma unroll
    for (int i = 0; i < KEEP; ++i) {
        const int64_t c = (i * T + threadIdx.x) * 8;
        if (c < cols) put(c, kept[i]);
    }
    for (int64_t c = (KEEP * T + threadIdx.x) * 8; c < cols; c += T * 8) put(c, row_chunk(r, c, cols, vec));
    if (threadIdx.x == 0) sx[m] = ldexpf(1.0f, k);
    if (GROW) {
        sq = block_sum(sq, sm);
        md = block_max(md, sm);
        if (threadIdx.x == 0) {
            const float nx = sqrtf(sq);               // ||x / s|| = nx * 2^k
            int ed = 0, ex = 0;
            frexpf(md, &ed);
            frexpf(nx, &ex);
            grow[m] = md > 0.0f && nx > 0.0f && !isinf(md) && !isinf(nx) ? ed + ex + k : DGU_NONE;
        }
    }
}

__device__ __forceinline__ __half2 dq_h2(uint32_t v) { return *reinterpret_cast<const __half2 *>(&v); }
__device__ __forceinline__ uint32_t dq_u32(__half2 v) { return *reinterpret_cast<const uint32_t *>(&v); }

// W16[o][i] = fp16((code - z) * Delta * 2^-kW): the difference is exact, the product rounded once (and
// Delta 2^-kW itself only below 2^-14, that is below 2^-24 of the largest).  A
// block takes DQ_ROWS rows, a thread the same packed word (8 columns, one 16-byte store) of each: their
// loads are in flight together, and a warp's loads and stores are contiguous.
// Bound: HBM, half a byte read and two written per weight: 22016 x 4096 in 41 us, 5.5 TB/s (four rows a block 43,
// eight 49; tiles of the matrix taken as one long row of words, by 8 resident blocks an SM, 46 to 49).
constexpr int DQ_ROWS = 2;
__global__ void __launch_bounds__(256) dequant_kernel(const uint32_t *__restrict__ q,
                                                      const uint16_t *__restrict__ scales,
                                                      const uint32_t *__restrict__ zeros, int64_t O, int wpr, int lg,
                                                      int nG, const unsigned *dmax,
                                                      uint16_t *__restrict__ out) {
    griddep_launch_dependents();
    griddep_wait();
    const float sw = ldexpf(1.0f, -dq_exp(dmax));
    const int nzw = (nG + 7) / 8;
    const int64_t o0 = static_cast<int64_t>(blockIdx.x) * DQ_ROWS;
    const int rows = static_cast<int>(O - o0 < DQ_ROWS ? O - o0 : DQ_ROWS);
    q += o0 * wpr;
    scales += o0 * nG;
    if (zeros) zeros += o0 * nzw;
    uint4 *dst = reinterpret_cast<uint4 *>(out) + o0 * wpr;
    for (int w = threadIdx.x; w < wpr; w += blockDim.x) {
        const int g = w >> (lg - 3), zsh = 4 * (g & 7);
        uint32_t v[DQ_ROWS], zw[DQ_ROWS];
        uint16_t sv[DQ_ROWS];
#pragma unroll
        for (int u = 0; u < DQ_ROWS; ++u) {
            const int r = u < rows ? u : 0;           // (wpr <= 2^28: DQ_ROWS rows of words fit 32 bits)
            v[u] = __ldcs(q + static_cast<uint32_t>(r * wpr + w));    // read once
            sv[u] = __ldg(scales + static_cast<uint32_t>(r * nG + g));
            zw[u] = zeros ? __ldg(zeros + static_cast<uint32_t>(r * nzw + (g >> 3))) : 0x88888888u;
        }
#pragma unroll
        for (int u = 0; u < DQ_ROWS; ++u) {
            if (u >= rows) break;
            const float df = __half2float(__ushort_as_half(sv[u])) * sw;
            const __half2 d = __floats2half2_rn(df, df);
            // 1024 + code as fp16 bits minus (1024 + z); (1024 + 16 code) / 16 minus (64 + z): both exact
            const __half2 z0 = dq_h2((0x6400u | ((zw[u] >> zsh) & 15u)) * 0x00010001u);
            const __half2 z1 = __hsub2(dq_h2(0x63806380u), z0);
            const __half2 r16 = dq_h2(0x2C002C00u);   // 1 / 16
            const uint32_t v8 = v[u] >> 8, P = 0x64006400u;
            const uint32_t e04 = dq_u32(__hmul2(__hsub2(dq_h2((v[u] & 0x000F000Fu) | P), z0), d));
            const uint32_t e15 = dq_u32(__hmul2(__hfma2(dq_h2((v[u] & 0x00F000F0u) | P), r16, z1), d));
            const uint32_t e26 = dq_u32(__hmul2(__hsub2(dq_h2((v8 & 0x000F000Fu) | P), z0), d));
            const uint32_t e37 = dq_u32(__hmul2(__hfma2(dq_h2((v8 & 0x00F000F0u) | P), r16, z1), d));
            dst[static_cast<uint32_t>(u * wpr + w)] =
                make_uint4(__byte_perm(e04, e15, 0x5410), __byte_perm(e26, e37, 0x5410), __byte_perm(e04, e15, 0x7632),
                           __byte_perm(e26, e37, 0x7632));
        }
    }
}

// The operands of the head's gradient that the products before it do not need: out[m] = x[m] where the label is scored,
// zeros elsewhere, `copies` times over (an unscored row adds nothing to the gradient, whatever (NaN, inf) its
// activations hold); and the labels' own gradients res[m] as bf16 in their places in d, [token][ldd] of the
// vocabulary's entries [v0, v0 + nv), with what the rounding takes off in row lo + m (lo: 0, none), and with the first
// token of each label in owner (null: not), all CE_NO_TOKEN before.
__global__ void __launch_bounds__(256) scored_rows_kernel(const uint4 *__restrict__ x,
                                                          const int64_t *__restrict__ labels, int64_t V, int64_t n,
                                                          int cpr, int copies, uint4 *__restrict__ out, int64_t M,
                                                          const float *res, uint16_t *d, int64_t ldd, int64_t v0,
                                                          int64_t nv, int64_t lo, int *owner) {
    griddep_wait();
    griddep_launch_dependents();
    const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.x, i0 = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    for (int64_t m = i0; m < M; m += step) {
        const int64_t lab = __ldcg(labels + m);
        if (lab < v0 || lab >= v0 + nv) continue;
        const float g = __ldcg(res + m);
        d[m * ldd + lab - v0] = __bfloat16_as_ushort(__float2bfloat16_rn(g));
        if (owner) atomicMin(owner + lab - v0, static_cast<int>(m));     // (the same whatever the order)
        if (lo) d[(lo + m) * ldd + lab - v0] = __bfloat16_as_ushort(__float2bfloat16_rn(bf16_rest(g)));
    }
    if (copies == 0) return;
    for (int64_t i = i0; i < n; i += step) {
        const int64_t lab = __ldcg(labels + i / cpr);
        const uint4 v = lab >= 0 && lab < V ? __ldcg(x + i) : make_uint4(0u, 0u, 0u, 0u);
        for (int k = 0; k < copies; ++k) out[k * n + i] = v;
    }
}

}  // namespace

cudaError_t launch_scored_rows(const uint16_t *x, const int64_t *labels, int64_t V, int64_t M, int64_t I,
                               int copies, uint16_t *out, const float *res, uint16_t *d, int64_t ldd, int64_t v0,
                               int64_t nv, int64_t lo, int *owner, int num_sms, cudaStream_t st) {
    const int64_t n = M * (I / 8), blocks = ((copies ? n : M) + 255) / 256, most = static_cast<int64_t>(num_sms) * 8;
    return launch_after(scored_rows_kernel, dim3(static_cast<unsigned>(blocks < most ? blocks : most)), 256, st,
                        reinterpret_cast<const uint4 *>(x), labels, V, n, static_cast<int>(I / 8), copies,
                        reinterpret_cast<uint4 *>(out), M, res, d, ldd, v0, nv, lo, owner);
}

cudaError_t launch_rows16(const uint16_t *x, const uint16_t *s16, int64_t M, int64_t cols, int64_t ld,
                          const uint16_t *dh, int64_t F, const uint16_t *scales, int64_t n_scales, bool permute,
                          uint16_t *out, float *sx, int *grow, unsigned *dmax, cudaStream_t st) {
    // Threads per row: few tokens are a matter of latency (77 rows of 4096: 3.1 us with 256 threads, 3.4 with
    // 128), many of the instructions that each warp spends whatever its share (2048 rows of 4096: 14.9
    // with 256, 12.6 with 128; of 13824: 25.5 with 256, 27.4 with 512).
    const int threads = M > 512 && cols <= 4096 ? 128 : 256;
    return launch_after(grow ? rows16_kernel<true> : rows16_kernel<false>, dim3(static_cast<unsigned>(M + DMAX_PARTS)), threads,
                        st, x, s16, M, cols, ld, dh, F, scales, n_scales, permute, out, sx, grow, dmax);
}

cudaError_t launch_dequant(const uint32_t *q, const uint16_t *scales, const uint32_t *zeros, int64_t O, int64_t I,
                           int gs, const unsigned *dmax, uint16_t *out, cudaStream_t st) {
    const int wpr = static_cast<int>(I / 8), threads = wpr < 256 ? (wpr + 31) / 32 * 32 : 256;
    return launch_after(dequant_kernel, dim3(static_cast<unsigned>((O + DQ_ROWS - 1) / DQ_ROWS)), threads, st, q, scales, zeros, O,
                        wpr, gs == 32 ? 5 : (gs == 64 ? 6 : 7), static_cast<int>(I / gs), dmax, out);
}

}  // namespace awq
