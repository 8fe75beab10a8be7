// Operand preparation of the dense products (k_dense.cu): packed 4-bit weights to fp16, and token
// rows to fp16 with a power-of-two scale of their own.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "awq_internal.h"
#include "w4a16_act.cuh"

namespace awq {

namespace {

// Largest |Delta| of the layer, as fp16 bits, into *dmax (zeroed by the caller).  A maximum does
// not depend on the order of its terms.
__device__ __forceinline__ void scales_max(const uint16_t *__restrict__ scales, int64_t n, int64_t first,
                                           int64_t step, unsigned *dmax) {
    unsigned mb = 0u;
    for (int64_t i = first; i < n; i += step) {
        const unsigned b = __ldg(scales + i) & 0x7FFFu;
        mb = b > mb ? b : mb;
    }
    mb = __reduce_max_sync(0xffffffffu, mb);
    if ((threadIdx.x & 31) == 0) atomicMax(dmax, mb);
}

// v[0..8) = source row elements [c, c + 8), divided by s where given.
__device__ __forceinline__ void row_chunk(const uint16_t *__restrict__ r, const uint16_t *__restrict__ s16, int64_t c,
                                          int64_t cols, bool vec, float (&v)[8]) {
    if (vec) {
        const uint4 xv = __ldg(reinterpret_cast<const uint4 *>(r + c));
        const uint32_t w[4] = {xv.x, xv.y, xv.z, xv.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[2 * e] = __uint_as_float(w[e] << 16);
            v[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = c + e < cols ? __uint_as_float(static_cast<uint32_t>(__ldg(r + c + e)) << 16) : 0.0f;
    }
    if (s16) {                                        // cols is a multiple of 64 here
        const uint4 sv = __ldg(reinterpret_cast<const uint4 *>(s16 + c));
        const uint32_t w[4] = {sv.x, sv.y, sv.z, sv.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const __half2 h = *reinterpret_cast<const __half2 *>(&w[e]);
            v[2 * e] = v[2 * e] / __low2float(h);
            v[2 * e + 1] = v[2 * e + 1] / __high2float(h);
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

// Blocks [0, M): one token each.  out[m] = fp16((row / s) * 2^-k), k from the row's largest
// magnitude so that it lands in [2^14, 2^15); sx[m] = 2^k.  With dh: grow[m], an exponent
// that bounds max |dh[m]| * ||row / s||.  Further blocks: the layer's largest |Delta|.
__global__ void __launch_bounds__(256) rows16_kernel(const uint16_t *__restrict__ x, const uint16_t *__restrict__ s16,
                                                     int64_t M, int64_t cols, int64_t ld,
                                                     const uint16_t *__restrict__ dh, int64_t F,
                                                     const uint16_t *__restrict__ scales, int64_t n_scales,
                                                     uint16_t *__restrict__ out, float *__restrict__ sx,
                                                     int *__restrict__ grow, unsigned *__restrict__ dmax) {
    if (blockIdx.x >= M) {
        const int64_t nb = gridDim.x - M;
        scales_max(scales, n_scales, (blockIdx.x - M) * blockDim.x + threadIdx.x, nb * blockDim.x, dmax);
        return;
    }
    __shared__ float sm[8];
    const int64_t m = blockIdx.x;
    const uint16_t *r = x + m * cols;
    const bool vec = cols % 8 == 0;
    float mx = 0.0f;
    for (int64_t c = threadIdx.x * 8; c < cols; c += blockDim.x * 8) {
        float v[8];
        row_chunk(r, s16, c, cols, vec, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) mx = fmaxf(mx, fabsf(v[e]));
    }
    mx = block_max(mx, sm);
    const int k = scale_exp(mx, 15);
    const float sc = ldexpf(1.0f, -k);
    float sq = 0.0f;                                  // of the scaled values: no overflow
    for (int64_t c = threadIdx.x * 8; c < cols; c += blockDim.x * 8) {
        float v[8];
        row_chunk(r, s16, c, cols, vec, v);
        uint32_t h[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[2 * e] *= sc;
            v[2 * e + 1] *= sc;
            sq = fmaf(v[2 * e], v[2 * e], fmaf(v[2 * e + 1], v[2 * e + 1], sq));
            const __half2 hv = __floats2half2_rn(v[2 * e], v[2 * e + 1]);
            h[e] = *reinterpret_cast<const uint32_t *>(&hv);
        }
        // ld is a multiple of 8: a last partial chunk stays inside its own row
        *reinterpret_cast<uint4 *>(out + m * ld + c) = make_uint4(h[0], h[1], h[2], h[3]);
    }
    if (threadIdx.x == 0) sx[m] = ldexpf(1.0f, k);
    if (grow) {
        sq = block_sum(sq, sm);
        const uint16_t *dr = dh + m * F;
        float md = 0.0f;
        for (int64_t f = threadIdx.x; f < F; f += blockDim.x)
            md = fmaxf(md, fabsf(__uint_as_float(static_cast<uint32_t>(__ldg(dr + f)) << 16)));
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

// W16[o][i] = fp16((code - z) * Delta * 2^-kW): one rounding, the difference and the power of two
// are exact.  One packed word (8 columns, one 16-byte store) per thread and step.
__global__ void __launch_bounds__(256) dequant_kernel(const uint32_t *__restrict__ q,
                                                      const uint16_t *__restrict__ scales,
                                                      const uint32_t *__restrict__ zeros, int64_t words, int wpr,
                                                      int lg, int nG, const unsigned *__restrict__ dmax,
                                                      uint16_t *__restrict__ out) {
    const float sw = ldexpf(1.0f, -dq_exp(dmax));
    const int nzw = (nG + 7) / 8;
    const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.x;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < words; i += step) {
        const int64_t o = i / wpr;
        const int w = static_cast<int>(i - o * wpr);
        const int g = w >> (lg - 3);
        const uint32_t v = __ldg(q + i);
        const float d = __half2float(__ushort_as_half(__ldg(scales + o * nG + g))) * sw;
        const int z = zeros ? (__ldg(zeros + o * nzw + (g >> 3)) >> (4 * (g & 7))) & 15 : 8;
        uint32_t h[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float a = static_cast<float>(static_cast<int>((v >> (8 * e)) & 15u) - z) * d;
            const float b = static_cast<float>(static_cast<int>((v >> (8 * e + 4)) & 15u) - z) * d;
            const __half2 hv = __floats2half2_rn(a, b);
            h[e] = *reinterpret_cast<const uint32_t *>(&hv);
        }
        *reinterpret_cast<uint4 *>(out + i * 8) = make_uint4(h[0], h[1], h[2], h[3]);
    }
}

// out[m] = x[m] where the label is scored, zeros elsewhere: an unscored row adds nothing to the
// head's gradient, whatever (NaN, inf) its activations hold.
__global__ void __launch_bounds__(256) scored_rows_kernel(const uint4 *__restrict__ x,
                                                          const int64_t *__restrict__ labels, int64_t V, int64_t n,
                                                          int cpr, uint4 *__restrict__ out) {
    const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.x;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < n; i += step) {
        const int64_t lab = __ldg(labels + i / cpr);
        out[i] = lab >= 0 && lab < V ? __ldg(x + i) : make_uint4(0u, 0u, 0u, 0u);
    }
}

}  // namespace

cudaError_t launch_scored_rows(const uint16_t *x, const int64_t *labels, int64_t V, int64_t M, int64_t I,
                               uint16_t *out, int num_sms, cudaStream_t st) {
    const int64_t n = M * (I / 8), blocks = (n + 255) / 256, most = static_cast<int64_t>(num_sms) * 8;
    scored_rows_kernel<<<static_cast<unsigned>(blocks < most ? blocks : most), 256, 0, st>>>(
        reinterpret_cast<const uint4 *>(x), labels, V, n, static_cast<int>(I / 8), reinterpret_cast<uint4 *>(out));
    return cudaGetLastError();
}

cudaError_t launch_rows16(const uint16_t *x, const uint16_t *s16, int64_t M, int64_t cols, int64_t ld,
                          const uint16_t *dh, int64_t F, const uint16_t *scales, int64_t n_scales, uint16_t *out,
                          float *sx, int *grow, unsigned *dmax, cudaStream_t st) {
    cudaError_t e = cudaMemsetAsync(dmax, 0, sizeof(unsigned), st);
    if (e != cudaSuccess) return e;
    const int64_t extra = (n_scales + 2047) / 2048 < 148 ? (n_scales + 2047) / 2048 : 148;
    rows16_kernel<<<static_cast<unsigned>(M + extra), 256, 0, st>>>(x, s16, M, cols, ld, dh, F, scales, n_scales, out,
                                                                     sx, grow, dmax);
    return cudaGetLastError();
}

cudaError_t launch_dequant(const uint32_t *q, const uint16_t *scales, const uint32_t *zeros, int64_t O, int64_t I,
                           int gs, const unsigned *dmax, uint16_t *out, int num_sms, cudaStream_t st) {
    const int64_t words = O * (I / 8);
    const int64_t blocks = (words + 255) / 256, most = static_cast<int64_t>(num_sms) * 8;
    dequant_kernel<<<static_cast<unsigned>(blocks < most ? blocks : most), 256, 0, st>>>(
        q, scales, zeros, words, static_cast<int>(I / 8), gs == 32 ? 5 : (gs == 64 ? 6 : 7), static_cast<int>(I / gs),
        dmax, out);
    return cudaGetLastError();
}

}  // namespace awq
