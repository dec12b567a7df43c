// Internal launch interface between the C ABI (api.cu) and the kernels.
#pragma once

#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "common.cuh"

namespace llmint8 {

// Adds n to the process-wide count of kernels launched by the library.
void note_launches(int n);

// Row-split plan of the outlier scan: the columns are covered by `col_blocks` CTAs of
// 256 threads x 8 columns, the rows by `splits` ranges of `rows_per_split` rows.
struct ScanPlan {
    int64_t col_blocks = 0, splits = 0, rows_per_split = 0, nwords = 0;
};
ScanPlan scan_plan(int64_t M, int64_t K);

cudaError_t launch_outlier_detect(const __half *X, int64_t M, int64_t K, float threshold,
                                  const ScanPlan &plan, uint32_t *partial, uint32_t *bitmap,
                                  int32_t *idx, int64_t cap, int32_t *count, StatusRef status,
                                  cudaStream_t s);
// The outlier set as the OR of n_bitmaps caller-supplied column bitmaps [n][ceil(K/32)]
// (bits at columns >= K ignored): merged bitmap, ascending list (first cap), count, status.
cudaError_t launch_outlier_merge(const uint32_t *bitmaps, int64_t n_bitmaps, int64_t K,
                                 uint32_t *bitmap, int32_t *idx, int64_t cap, int32_t *count,
                                 StatusRef status, cudaStream_t s);
// Row quantization of X (and, with Wo non-null, the gather of the outlier weights Wo
// [N, xo_pitch] from CB/SCB or W16, in the same launch).  The scan, compaction and this
// kernel are programmatic dependents of whatever precedes them in the stream.
cudaError_t launch_quantize_rows(const __half *X, int64_t M, int64_t K, const uint32_t *bitmap,
                                 const int32_t *idx, const int32_t *count, int64_t cap,
                                 int64_t xo_pitch, int8_t *Xq, float *SCA, __half *Xo,
                                 const int8_t *CB, const float *SCB, const __half *W16, int64_t N,
                                 __half *Wo, cudaStream_t s);
cudaError_t launch_quantize_weight(const __half *W, int64_t N, int64_t K, int8_t *CB, float *SCB,
                                   cudaStream_t s);
cudaError_t launch_dequant(const int8_t *CB, const float *SCB, int64_t N, int64_t K,
                           __half *W_out, cudaStream_t s);

// The tcgen05 GEMM with the fused fp16 outlier product and dequantizing epilogue.
struct GemmLaunch {
    const int8_t *Xq;        // [M, K]
    const int8_t *CB;        // [N, K]
    const __half *Xo;        // [M, pitch]   (may be null when cap == 0)
    const __half *Wo;        // [N, pitch]
    int64_t pitch;           // columns of Xo / Wo (multiple of 64)
    const int32_t *count;    // device outlier count
    int64_t cap;             // capacity (columns usable in Xo / Wo)
    const float *SCA;        // [M]
    const float *SCB;        // [N]
    const __half *bias;      // [N] or null
    __half *Y;               // [M, N]
    int32_t *C_debug;        // [M, N] or null
    uint32_t *ybits;         // [ceil(M/32)][ceil(N/32)] outlier bitmaps of Y for the next
                             // layer (|Y| >= ythreshold per column and 32-row block), or null
    float ythreshold;
    StatusRef status;
    int64_t M, N, K;
    uint64_t timeout_ns;
};
cudaError_t launch_gemm(const GemmLaunch &g, cudaStream_t s);

}  // namespace llmint8

namespace llmint8 {

// Decode path (M <= kDecodeMaxM, K <= kDecodeMaxK, at most kDecodeMaxOutliers outlier
// columns): one weight-streaming tcgen05 kernel per call.  Its first CTAs quantize X (each a
// slice of the columns; they exchange their partial row maxima and outlier counts) and publish
// the outlier columns, row scales and the int8 operand image through a DecodeTable and the
// image in the workspace; every other CTA streams a band of weight rows.
constexpr int kDecodeMaxM = 16;
constexpr int kDecodeMaxK = 16384;
constexpr int kDecodeMaxOutliers = 256;

// What the quantizer CTAs publish (workspace, 256-byte aligned).
//   part[q][m]  (call << 32) | fp32 bits of quantizer q's row-m maximum of |x| over the regular
//               columns of its slice (m < kDecodeMaxM), then (call << 32) | the number of
//               outlier columns in its slice: one 64-bit store each, so a word that carries
//               the call's number carries its value;
//   done[q]     the call's number, stored with release semantics once quantizer q's k-blocks of
//               the operand image and its entries of idx are written (quantizer 0: also sca,
//               total and n_out);
//   readers     the streamers' threads that have seen every done word; after the last of them
//               quantizer 0 clears part and done, so that a call replayed from a graph, under the
//               number it was captured with, does not take the last replay's words for its own.
constexpr int kDecodeMaxQuantizers = 8;
struct DecodeTable {
    unsigned long long done[kDecodeMaxQuantizers];
    unsigned long long part[kDecodeMaxQuantizers][kDecodeMaxM + 1];
    int32_t total;                            // outlier columns found
    int32_t n_out;                            // ... of them listed (<= capacity)
    float sca[kDecodeMaxM];                   // row absmax over the regular columns
    int32_t idx[kDecodeMaxOutliers];          // outlier columns, ascending
    unsigned long long readers;
};

// Bytes of the int8 operand image the quantizer writes: one block of 16 rows (8 when M <= 8)
// x 128 bytes per 128-column k-block.
__host__ __device__ constexpr int64_t decode_image_bytes(int64_t M, int64_t K) {
    return (K + 127) / 128 * (M <= 8 ? 8 : kDecodeMaxM) * 128;
}

// Launch geometry of the decode kernel for one shape.
struct DecodePlan {
    int Rt = 0;              // weight rows (output channels) per tile
    int tiles = 0, grid = 0, kblocks = 0;
    int rows = 0;            // rows of an operand-image block (8 or 16)
    int stages = 0, smem = 0;
    int inflight = 0;        // weight stages a streamer keeps on their way at most
    int nq = 0;              // quantizer CTAs (the first nq of the grid)
    int bpq = 0;             // k-blocks per quantizer
    int nst = 0;             // weight stages per tile (2 k-blocks each)
    int nistage = 0;         // operand-image stages of a streamer
    bool resident = false;   // ... holding every k-block (filled once)
    uint32_t tail_off = 0, xo_off = 0, ring_off = 0;
};
DecodePlan decode_plan(int64_t M, int64_t N, int64_t K, int64_t cap, int sms);

struct DecodeLaunch {
    const __half *X;         // [M, K]
    const int8_t *CB;        // [N, K]
    const float *SCB;        // [N]
    const __half *W16;       // [N, K] or null
    const __half *bias;      // [N] or null
    __half *Y;               // [M, N]
    int32_t *C_debug;        // [M, N] or null
    __half *Wo;              // [N, wo_pitch] or null: receives the outlier weights used
    int64_t wo_pitch;
    const uint32_t *bitmaps; // [n_bitmaps][ceil(K/32)]: the outlier set given, or null
    int64_t n_bitmaps;
    uint32_t *ybits;         // [ceil(N/32)]: outlier bitmap of Y for the next layer, or null
    float ythreshold;
    int32_t *count;          // device outlier count (workspace header)
    DecodeTable *table;      // workspace
    uint8_t *image;          // workspace: decode_image_bytes(M, K), 1024-byte aligned
    StatusRef status;
    int64_t M, N, K, cap;
    float threshold;
    uint64_t timeout_ns;
};
cudaError_t launch_decode(const DecodeLaunch &d, cudaStream_t s);

// MXFP4 (mxfp4.cu): codes uint8 [R, K/2], scales uint8 [ceil(R/128)][ceil(K/256)][1024].  dtype is
// a llmint8_dtype.  pad: the scales of every row up to a multiple of 128 are written (zero past R);
// without it some stay as they are.
cudaError_t launch_mxfp4_quantize(const void *X, int dtype, int64_t ldx, int64_t R, bool pad,
                                  int64_t K, uint8_t *codes, uint8_t *scales, cudaStream_t s);
cudaError_t launch_mxfp4_dequant(const uint8_t *codes, const uint8_t *scales, int64_t R,
                                 int64_t K, void *out, int dtype, cudaStream_t s);

// The MXFP4 product (gemm_mxfp4.cu).
constexpr int kMxfp4FusedRows = 8;       // rows of X that the product quantises itself at most
struct Mxfp4Gemm {
    const void *X;           // [M, K] of dtype, rows ldx apart, to be quantised in the kernel
    int64_t ldx;             // (M <= kMxfp4FusedRows); or null, and
    const uint8_t *Xc, *Xs;  // X [M, K] as MXFP4
    const uint8_t *Wc, *Ws;  // W [N, K]
    const void *bias;        // [N] or null
    void *Y;                 // [M, N]
    int dtype;               // of bias and Y
    StatusRef status;
    int64_t M, N, K;
    uint64_t timeout_ns;
};
cudaError_t launch_mxfp4_gemm(const Mxfp4Gemm &g, cudaStream_t s);

// The residual norm (norm.cu).
constexpr int64_t kNormMaxK = 32768;
struct NormArgs {
    const void *X, *residual;            // [M, K]; residual may be null
    const void *post_weight, *post_bias; // [K] or null
    const void *gate;                    // [M / gate_group, K] or null
    const void *weight, *bias;           // [K] or null
    void *H, *Y;                         // [M, K] or null
    uint8_t *codes, *scales;             // y as MXFP4, or null
    uint32_t x_pitch, r_pitch, pitch;    // bytes from row to row: X, residual, dense rows (2 K)
    uint32_t M;
    uint32_t gate_group;                 // rows that share a row of the gate
    uint32_t rows_out, tiles_k;          // of the scales
    int norm, post_norm;                 // llmint8_norm
    float scale, eps, inv_k;             // inv_k = 1 / K
};
cudaError_t launch_residual_norm(const NormArgs &a, int dtype, cudaStream_t s);

}  // namespace llmint8
