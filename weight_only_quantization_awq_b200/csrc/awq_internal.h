// Internal launch interface between the C-ABI layer (awq_api.cu) and the
// kernels.  Every launcher enqueues on `st` and returns the launch status.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>
#include <stdint.h>

namespace awq {

// An NVTX range around one C-ABI call, so that each call shows on a profiler's
// timeline with its kernels under it.  Without a profiler's NVTX injection library
// the push and pop return at once.
struct NvtxRange {
    explicit NvtxRange(const char *name) { nvtxRangePushA(name); }
    ~NvtxRange() { nvtxRangePop(); }
    NvtxRange(const NvtxRange &) = delete;
    NvtxRange &operator=(const NvtxRange &) = delete;
};

// Record the calling host thread's last-error text (read back by awq_last_error()).
void set_last_error(const char *msg);

constexpr int STATS_CHUNK = 128;   // tokens per fp64 partial sum of mean|X|
constexpr int64_t STATS_MAX_GRID_Y = 65535;   // chunks beyond this are strided over the grid

// Optional CUDA-event timing of an entry point's main kernels (awq_set_kernel_timing):
// kt_reset clears the record of `kind`, kt_begin / kt_end bracket launches on `st`.
void kt_reset(int kind);
void kt_begin(int kind, cudaStream_t st);
void kt_end(int kind, cudaStream_t st);
constexpr int MAX_GRID = 64;       // grid points per search phase

// Default bound of an in-kernel mbarrier wait: ~2 s of SM clock at 2 GHz, far
// above any legitimate wait in these kernels.
constexpr long long AWQ_DEFAULT_WAIT_CYCLES = 4000000000LL;

// Search tile shape: 128 output rows per CTA (256 per CTA pair) x 512 tokens per
// work unit (two MMA halves of 256), K slabs of 64.
constexpr int TILE_O = 128;
constexpr int TILE_N = 512;
constexpr int SUB_N = 256;
constexpr int SLAB_K = 64;

struct GridParams {
    double value[MAX_GRID];   // alpha per grid point (phase 1) or clip ratio (phase 2)
};

// ---- statistics
cudaError_t launch_stats_partial(const void *X, bool x_bf16, int64_t N, int64_t I, double *part,
                                 cudaStream_t st);
cudaError_t launch_stats_final(const double *part, int64_t N, int64_t I, float clamp_min,
                               float *sX, cudaStream_t st);
// fp16 copy of X scaled by 2^-k (k written to *k_out on the device); *max_bits zeroed by the caller.
cudaError_t launch_x_to_f16(const void *X, bool x_bf16, int64_t n, unsigned *max_bits, int *k_out,
                            uint16_t *dst, cudaStream_t st);

// ---- scale table sn[G][2][I]: row 2g holds s_g, row 2g+1 holds -1/s_g.
// alpha.value[g] is grid point g's alpha; if best_idx != nullptr every row uses
// alpha.value[*best_idx] instead (the second, clip phase).
// scratch: scale_scratch_bytes(G, I) bytes of device workspace.
int64_t scale_scratch_bytes(int G, int64_t I);
cudaError_t launch_scale_table(const float *sX, int64_t I, const GridParams &alpha, int G,
                               const int *best_idx, float *sn, void *scratch, cudaStream_t st);

// ---- per-(grid point, group, row) quantiser parameters {Delta, 1/Delta, -qhi, -qlo},
// layout qparam[g][group][row] (rows fastest).  Also picks each grid point's
// power-of-two range scale 2^k of dW (dw_exp[g] = k, device), multiplying the
// -1/s rows of sn by it; dw_bits: G words of device scratch.
cudaError_t launch_group_params(const void *W, bool w_bf16, int64_t O, int64_t I, int gs,
                                bool asym, int wbit, float *sn, const GridParams &clip,
                                int G, float4 *qparam, unsigned *dw_bits, int *dw_exp,
                                cudaStream_t st);

// ---- fused search
// Tensor maps of the kernel's four inputs:
//   x  : fp16 copy of X [N, I], box 64 x 128 (one CTA's half of a 256-token tile), 128B swizzle
//   w  : W [O, I] (bf16: box 64 x 128; fp32: box 32 x 128), 128B swizzle
//   sn : scale table [2G, I] fp32, box 64 x 2
//   qp : group parameters [G * I/gs][O][4] fp32 (3-D), box 4 x 128 rows x groups per slab
struct SearchMaps {
    CUtensorMap x, w, sn, qp;
};
struct SearchArgs {
    int64_t O, I, N;
    int gs;
    int G;
    bool w_bf16;
    bool clamp;                 // asymmetric or clipped: clamp codes to [qlo, qhi]
    float *part;                // [G][TB][O]
    int *err;
    long long wait;             // bound of every mbarrier wait, in SM clock cycles
};
cudaError_t launch_search(const SearchArgs &a, const SearchMaps &maps, int num_sms,
                          cudaStream_t st);

// ---- loss reduction and selection
// blocksum: scratch of reduce_scratch_doubles(G, O) doubles.
int64_t reduce_scratch_doubles(int G, int64_t O);
// Row sums of grid point g are multiplied by 2^(-2 * (*x_exp + dw_exp[g])) (the exact
// undo of the power-of-two scales of X and dW in the contraction).
cudaError_t launch_reduce_loss(const float *part, int G, int64_t TB, int64_t O, int64_t N,
                               const int *x_exp, const int *dw_exp, double *loss, float *loss_row,
                               double *blocksum, cudaStream_t st);
cudaError_t launch_argmin(const double *loss, int G, int *best, cudaStream_t st);

// ---- packing
// clip_idx (optional, [O][I/gs] device): each group's index into clip_grid, used
// instead of the layer ratio `clip`.
cudaError_t launch_pack(const void *W, bool w_bf16, int64_t O, int64_t I, int gs, bool asym,
                        int wbit, double clip, const uint8_t *clip_idx, const GridParams &clip_grid,
                        const float *s, uint32_t *qweight, uint16_t *scales, uint32_t *zeros,
                        uint16_t *s16, float *scales_f32, cudaStream_t st);

// ---- W4A16 apply on the tensor cores (M >= 17)
struct TcMaps {
    CUtensorMap q;    // qweight [O][I/8] u32, box 32 words (4 slabs) x 128 rows, 128B swizzle
    CUtensorMap xs;   // permuted, power-of-two scaled fp16 x/s [M][I], box 64 x n_tile, 128B swizzle
};
struct TcPlan {
    int n_tile;            // tokens per tile (multiple of 16, <= 256)
    int splits;            // K splits
    int slabs_per_split;
    int64_t xs_bytes, part_bytes, counter_bytes, scale_bytes;   // workspace pieces (256-byte rounded)
};
TcPlan w4a16_tc_plan(int64_t M, int64_t I, int64_t O, int num_sms);
// workspace: xs (plan.xs_bytes), the fp32 split-K accumulator (plan.part_bytes), the
// tile counters (plan.counter_bytes), then the token scales sx [M] fp32 and the row exponents
// kd [O] int32 (plan.scale_bytes).
cudaError_t launch_w4a16_tc(const uint16_t *x, int64_t M, int64_t I, int64_t O,
                            const uint16_t *scales, const uint32_t *zeros, const uint16_t *s16,
                            int gs, uint16_t *y, const TcPlan &plan, char *workspace,
                            const TcMaps &maps, cudaStream_t st);

// ---- W4A16 decode (M <= 8) over up to DEC_MAX_LINEARS independent linears in one
// persistent launch, one CTA per SM.  Each CTA works on one linear: linear l owns
// the CTAs [cta0[l], cta0[l + 1]) (their number in proportion to its bytes), and
// its tiles of rows[l] output rows (a multiple of 8; all input columns) are split
// into equal contiguous ranges among them.  A CTA's ring holds stages[l] slots of
// slot_bytes[l]; activations take xbuf_bytes[l].  All sizes come from
// w4a16_dec_config.
constexpr int DEC_MAX_LINEARS = 8;
constexpr int64_t DEC_MAX_M = 8;
constexpr int64_t DEC_MAX_SMEM = 227 * 1024;
struct DecLinear {
    const uint16_t *x;
    const uint32_t *qweight;
    const uint16_t *scales;
    const uint32_t *zeros;
    const uint16_t *s16;
    uint16_t *y;
    int64_t I, O;
};
struct DecBatch {
    DecLinear lin[DEC_MAX_LINEARS];
    int cta0[DEC_MAX_LINEARS + 1];
    int rows[DEC_MAX_LINEARS];
    int stages[DEC_MAX_LINEARS];
    int slot_bytes[DEC_MAX_LINEARS];
    int xbuf_bytes[DEC_MAX_LINEARS];
    int n, ctas;
    int64_t smem;                 // dynamic shared memory of the launch
};
// Fills the CTA split and the buffer plan of `b` (lin[] and n set by the caller);
// false when M or a linear does not fit the kernel's shared memory, or the
// linears outnumber the SMs.
bool w4a16_dec_config(DecBatch &b, int64_t M, int gs, bool zeros, int num_sms);
cudaError_t launch_w4a16_dec(const DecBatch &b, int M, int gs, bool zeros, cudaStream_t st);

// ---- W4A16 apply for decode-sized M (1..16): xs preparation + warp-level MMA kernel
constexpr int64_t W4A16_MMA_MAX_M = 16;
int64_t w4a16_mma_workspace_bytes(int64_t M, int64_t I, int gs);
cudaError_t launch_w4a16_mma(const uint16_t *x, int64_t M, int64_t I, int64_t O,
                             const uint32_t *qweight, const uint16_t *scales, const uint32_t *zeros,
                             const uint16_t *s16, int gs, uint16_t *y, char *workspace,
                             cudaStream_t st);

// ---- W4A16 apply
// Streaming GEMV for 1 <= M <= 4 (activations staged per CTA; see k_w4a16_stream.cu).
bool w4a16_stream_supported(int64_t M, int64_t I);
cudaError_t launch_w4a16_stream(const uint16_t *x, int64_t M, int64_t I, int64_t O,
                                const uint32_t *qweight, const uint16_t *scales, const uint32_t *zeros,
                                const uint16_t *s16, int gs, uint16_t *y, int num_sms, cudaStream_t st);
cudaError_t launch_w4a16(const uint16_t *x, int64_t M, int64_t I, int64_t O,
                         const uint32_t *qweight, const uint16_t *scales, const uint32_t *zeros,
                         const uint16_t *s16, int gs, uint16_t *y, cudaStream_t st);

// ---- per-group clip choice: Gram matrices of X per group (H: gclip_scratch_doubles
// device doubles), then for every (row, group) the first ratio of `grid` that
// minimises the group's output error; best [O][I/gs] u8, err (optional) [O][I/gs][n_clip].
int64_t gclip_scratch_doubles(int64_t I, int gs);
cudaError_t launch_group_clip(const void *W, bool w_bf16, int64_t O, int64_t I, const void *X,
                              bool x_bf16, int64_t N, const float *s, int gs, bool asym, int wbit,
                              const GridParams &grid, int n_clip, double *H, uint8_t *best,
                              float *err, cudaStream_t st);

// ---- bounded-wait self-test: one CTA waits on an mbarrier (arrived on only if
// `arrive`) with a limit of `limit` cycles; a wait that gives up writes the
// timeout code to *err.
cudaError_t launch_wait_selftest(long long limit, bool arrive, int *err, cudaStream_t st);

// ---- dense 16-bit products on the tensor cores and the epilogues of the operators that train
// through packed weights and score a vocabulary (k_dense.cu), with their operand preparation
// (k_dequant.cu)
enum { ACT_SILU = 0, ACT_GELU = 1, ACT_GELU_TANH = 2 };
enum { EPI_GATED = 0, EPI_GATED_BWD = 1, EPI_OUT = 2, EPI_CE = 3, EPI_CE_BWD = 4, EPI_CE_T = 5, EPI_CE_BWD_T = 6 };
// Tokens up to which the vocabulary goes on the rows (32000 x 4096: 13 tokens 45 against 64 us, 128 tokens
// 50 against 53: the products cost the columns, and 256 rows of tokens are mostly padding).
constexpr int64_t CE_T_MAX_M = 128;
// The same for the gradients of the logits (40062 x 1024, one token: 23 against 31 us; 1007 x 384, 111 tokens 11.5
// against 6.5: a token's row is written 64 bytes at a time).
constexpr int64_t CE_BWD_T_MAX_M = 64;
// Tokens up to which the head's gradient takes the remainders of the rounded gradients, too (twice the K, which the
// writing of dW hides).  A label's rounding error, up to 2^-8 of its gradient, is common to all elements of that token's
// part of a head row.  Above, where twice the K would cost twice the time, the remainder of the first token of each label
// is added in fp32 (GemmArgs::owner): of 2048 tokens and 32000 entries most rows with a label have one, and without
// it dW was off by 2.35e-3 in the norm instead of 1.7e-3.  A row of many tokens keeps the roundings of the others.
constexpr int64_t CE_LO_MAX_M = 128;
constexpr int CE_NO_TOKEN = 0x7FFFFFFF;
static_assert(CE_LO_MAX_M >= CE_BWD_T_MAX_M, "owners go with EPI_CE_BWD");
struct GemmMaps {
    CUtensorMap a, b;           // K-major: box 64 k x 128 rows (b: bn / 2 rows); MN-major: box 64 x 64
};
struct GemmArgs {
    int64_t M, N;               // rows and columns of D (EPI_GATED*: N unused)
    int mt, nt;                 // tiles of 256 rows and of bn columns (EPI_GATED*: of bn / 2 gate columns)
    int bn;                     // tile columns of the pair
    int nk[2];                  // 64-deep K slabs of the two K segments
    int splits;                 // K splits of each tile (EPI_OUT; 1 otherwise)
    float4 *part4;              // their partial sums [tiles * splits][bn / 4][256]
    int a_seg, b_seg;           // first K coordinate of the second segment in A and in B
    // scales
    const float *sx;            // [M]: A's row m carries 1 / sx[m] (a power of two)
    const unsigned *dmax;       // [DMAX_PARTS] largest |Delta| (the weights carry 2^-kW)
    const int *grow;            // [M]: exponent bound of the token's gradients (DGU_NONE: none)
    const uint16_t *s16;        // [N] fp16: divides column n (EPI_OUT)
    int inner;                  // in, of the gated product
    int act;
    int64_t F, Fp;              // gate columns; rounded up to 64
    const uint16_t *dh;         // [M][F] bf16
    // cross entropy
    const int64_t *labels;      // [M]
    int64_t V, v0;              // vocabulary; first entry of this piece
    const float *lse, *dloss;   // [M]
    float *tgt;                 // [M] the label's logit
    float2 *part;               // [4 nt][M] (EPI_CE_T: [N][8 mt]) (maximum, sum of exponentials) without the label's
    const uint16_t *x, *w;      // the operands themselves, rows of `inner` columns (the labels' logits); EPI_OUT: w, rows of N
    float *res;                 // [M] the gradient of the label's logit, whose place in d16 EPI_CE_BWD* leave zero: they
                                // write it, EPI_OUT adds res[m] w[labels[m]] to row m (null: does not)
    int *owner;                 // [N of the piece] the first token of each label, CE_NO_TOKEN: none.  EPI_CE_BWD clears it;
                                // EPI_OUT adds the remainder of res[owner[n]] times that token's row of x to row n
    int64_t lo;                 // EPI_CE_BWD*: rows of d16 from a token's to its row of rounding remainders (0: none)
    // outputs
    uint16_t *out;              // bf16
    uint16_t *d16;              // [M][ldd] 16-bit gradients
    int64_t ldd;
    float *acc;                 // [M][N] fp32, pieces meet here (EPI_OUT), or null
    bool first, last;           // first: acc is not read; last: the result goes to out
};
int gemm_tile_cols(int64_t M, int64_t N, int num_sms);
// Tile columns and K splits of an EPI_OUT product, and the float4 of workspace for its partial sums.
struct GemmPlan {
    int bn, splits;
    int64_t part_vecs;
};
GemmPlan gemm_plan(int64_t M, int64_t N, int64_t k, int num_sms);
cudaError_t launch_gemm16(int epi, bool bf16, bool a_mn, const GemmMaps &maps, const GemmArgs &a, int num_sms,
                          cudaStream_t st);
cudaError_t launch_ce_final(const float2 *part, int n, bool rows, int64_t M, const int64_t *labels, int64_t V,
                            const float *tgt, float *loss, float *lse, cudaStream_t st);
// Token rows to fp16 with a power-of-two scale each (out [M][ld], sx [M]); dh [M][F] with grow [M]
// optional; dmax [DMAX_PARTS] = the largest |Delta| of the parts of the layer's scales, as fp16 bits.
// permute: the columns of each 8 in the order (0,4,1,5,2,6,3,7).
constexpr int DMAX_PARTS = 128;
cudaError_t launch_rows16(const uint16_t *x, const uint16_t *s16, int64_t M, int64_t cols, int64_t ld,
                          const uint16_t *dh, int64_t F, const uint16_t *scales, int64_t n_scales, bool permute,
                          uint16_t *out, float *sx, int *grow, unsigned *dmax, cudaStream_t st);
cudaError_t launch_dequant(const uint32_t *q, const uint16_t *scales, const uint32_t *zeros, int64_t O, int64_t I,
                           int gs, const unsigned *dmax, uint16_t *out, cudaStream_t st);
cudaError_t launch_scored_rows(const uint16_t *x, const int64_t *labels, int64_t V, int64_t M, int64_t I,
                               int copies, uint16_t *out, const float *res, uint16_t *d, int64_t ldd, int64_t v0,
                               int64_t nv, int64_t lo, int *owner, int num_sms, cudaStream_t st);

// ---- products with a packed matrix for up to a few hundred tokens, dequantised on the way into
// the tensor cores (k_skinny.cu): forward EPI_GATED / EPI_GATED_BWD (64 gate and 64 up rows per tile, K
// = in), gradient EPI_OUT (128 columns per tile, K = out)
struct SkinnyPlan {
    int n, token_tiles;         // tokens per tile (a multiple of 16, <= 144), tiles of tokens
    int tiles, ks, grid;        // tiles of W, 128-deep stages of K, CTAs
    int64_t part_vecs;          // workspace: fp32 partial sums, by four
};
// Up to how many tokens, and below 4 GB of codes; above, the weights are dequantised once for dense
// products: two tiles of 144 tokens, one for the gradient of the gated product, whose two dense products share the
// dequantised weights.  Measured (us a call, this way / dense): 22016 x 4096 gated 144 tokens 54 / 89, 288
// 90 / 114, 304 127 / 125; its gradient 144 tokens 106 / 136, 208 158 / 142; 4096 x 11008 gradient 144 tokens 36 /
// 52, 208 56 / 54, 288 65 / 75, 304 91 / 79; 5504 x 2048 gradient 250 tokens 22 / 28.
constexpr int64_t SKINNY_MAX_M = 288, SKINNY_MAX_M_GATED_GRAD = 144;
inline bool skinny_supported(int64_t M, int64_t most, int64_t O, int64_t I) { return M <= most && O * I <= int64_t(1) << 32; }
// The gated product: of more than one token tile only if the dequantised matrix does not stay in L2 from the pass
// that writes it to the product, or is so small that the pass and its launch are what counts (us a call, this way /
// dense: 11008 x 2048 150 tokens 30 / 29, 250 37 / 29; 13824 x 2560 200 tokens 42 / 39, 250 45 / 39; 22016 x 4096
// 250 tokens 85 / 93; 8192 x 1536 150 tokens 17 / 22, 250 19 / 22; 5632 x 1024 250 tokens 15 / 17).
inline bool skinny_gated(int64_t M, int64_t O, int64_t I) {
    const bool in_l2 = O * I >= (int64_t(16) << 20) && O * I <= (int64_t(50) << 20);
    return skinny_supported(M, M > 144 && in_l2 ? 144 : SKINNY_MAX_M, O, I);
}
SkinnyPlan skinny_plan(int64_t M, int64_t tiles, int64_t k, int num_sms);
struct SkinnyArgs {
    const uint32_t *q;
    const uint16_t *scales;
    const uint32_t *zeros;
    int64_t O, I, F, M;
    int lg;                     // log2 of the group size
    const float *sx;            // [M]: the token tile's row m carries 1 / sx[m]
    const unsigned *dmax;       // [DMAX_PARTS] largest |Delta| (the weights carry 2^-kW)
    const int *grow;            // [M] exponent bound of the token's gradients, or null
    const uint16_t *s16;        // [I]: divides column i (EPI_OUT)
    int inner, act;
    const uint16_t *dh;         // [M][F] bf16
    uint16_t *out;              // bf16 result
    uint16_t *d16;              // [M][ldd]: gate gradients, then up gradients, fp16
    int64_t ldd;
    float4 *part;
    // set by launch_skinny
    int n, tiles, ks, units, acc_cols, stages, grid;
};
// bmap: the tokens' fp16 rows [M][K] (forward: columns of each 8 in the order (0,4,1,5,2,6,3,7)), box 64 x n.
cudaError_t launch_skinny(bool grad, int epi, const CUtensorMap &bmap, SkinnyArgs a, const SkinnyPlan &p,
                          cudaStream_t st);

// ---- gated feed-forward for decode-sized M (k_gated_dec.cu); supported: the staged activations and the
// scales of all of a CTA's tiles, or of four at a time, fit one SM's shared memory.  With fewer the
// passes cost more than dequantising on the way into the tensor cores (22016 x 4096: group 32, 8 tokens, three
// of five tiles a pass 39 / 36 us, 9 tokens, two 56 / 36; group 64, 12 tokens, four 36 / 35, 16 tokens, two 43 / 35).
constexpr int64_t GATED_DEC_MAX_M = 16;
bool gated_dec_supported(int64_t M, int64_t I, int64_t F, int gs, int num_sms);
cudaError_t launch_gated_dec(const uint16_t *x, int64_t M, int64_t I, int64_t F, const uint32_t *q,
                             const uint16_t *scales, const uint32_t *zeros, const uint16_t *s16, int gs, int act,
                             uint16_t *h, int num_sms, cudaStream_t st);

// ---- fold of 1/s into the previous operator: out[r][c] = P[r][c] / s16[r]
// (one IEEE fp32 division, then bf16 rounding when bf16).
cudaError_t launch_fold_scale(const void *P, bool bf16, int64_t R, int64_t C, const uint16_t *s16,
                              void *out, cudaStream_t st);

}  // namespace awq
