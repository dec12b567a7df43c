// MXFP4 quantisation of the rows of a matrix, and the way back.  Both are bound by HBM: they
// read and write each value once (17/32 byte an element in MXFP4 form) and compute little.
//
// A warp takes one row of a scale tile (256 columns, 8 elements a lane), so a block's maximum is
// two shuffles among four lanes, its codes one 32-bit store a lane and the row's eight scales two
// 32-bit stores.  A warp keeps U such pieces in flight (U = 4 once the grid fills the machine
// several times over; 1 below that, where more warps hide more latency than deeper ones).
#include "kernels.h"
#include "launch.cuh"
#include "mxfp4.cuh"

namespace llmint8 {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// The pieces of a warp: row `row`, scale-tile columns kt0 + i * step (i < U).
struct Place {
    int64_t row;
    int64_t kt0;
    int step;
};
template <int U>
__device__ __forceinline__ Place place_of_warp(int wpr_log2) {
    const int w = threadIdx.x >> 5;
    Place p;
    p.step = 1 << wpr_log2;
    p.row = (int64_t)blockIdx.x * (kWarps >> wpr_log2) + (w >> wpr_log2);
    p.kt0 = (int64_t)blockIdx.y * (U << wpr_log2) + (w & (p.step - 1));
    return p;
}

// rows_out >= R: rows [R, rows_out) get zero scales (they pad the last row of scale tiles).
template <int DT, int U>
__global__ void __launch_bounds__(kThreads)
mxfp4_quantize_kernel(const uint8_t *__restrict__ X, int64_t row_bytes, int64_t R,
                      int64_t rows_out, int64_t chunks, int64_t tiles_k, int wpr_log2,
                      uint32_t *__restrict__ codes, uint8_t *__restrict__ scales) {
    pdl_wait_then_release();
    const int lane = threadIdx.x & 31;
    const Place p = place_of_warp<U>(wpr_log2);
    if (p.row >= rows_out) return;
    Chunk<DT> c[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {        // issue every load before using any
        const int64_t ch = (p.kt0 + i * p.step) * 32 + lane;
        c[i] = p.row < R && ch < chunks ? load_chunk<DT>(X + p.row * row_bytes, ch)
                                        : zero_chunk<DT>();
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const int64_t kt = p.kt0 + i * p.step;
        if (kt < tiles_k)
            quantize_tile_row<DT>(c[i], p.row < R && kt * 32 + lane < chunks, p.row, kt, chunks,
                                  tiles_k, codes, scales, lane);
    }
}

template <int DT, int U>
__global__ void __launch_bounds__(kThreads)
mxfp4_dequant_kernel(const uint32_t *__restrict__ codes, const uint8_t *__restrict__ scales,
                     int64_t R, int64_t chunks, int64_t tiles_k, int wpr_log2,
                     uint8_t *__restrict__ out) {
    pdl_wait_then_release();
    const int lane = threadIdx.x & 31;
    const Place p = place_of_warp<U>(wpr_log2);
    if (p.row >= R) return;
    uint32_t q[U], s[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {        // issue every load before using any
        const int64_t kt = p.kt0 + i * p.step;
        q[i] = 0u;
        s[i] = 0u;
        if (kt * 32 + lane < chunks) {
            q[i] = codes[p.row * chunks + kt * 32 + lane];
            s[i] = scales[scale_word_offset(p.row, kt, tiles_k, lane >> 4) + ((lane >> 2) & 3)];
        }
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const int64_t ch = (p.kt0 + i * p.step) * 32 + lane;
        if (ch >= chunks) continue;
        uint32_t h[4];
        asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
            "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
            "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
            "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
            "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
            "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
            : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
            : "r"(q[i]));
        // 2^(s - 127): an exponent field, or the subnormal 2^-127; 255 stands for NaN
        const float scale = __uint_as_float(s[i] == 0u     ? 0x00400000u
                                            : s[i] == 255u ? 0x7fc00000u
                                                           : s[i] << 23);
        float f[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 t = __half22float2(*reinterpret_cast<const __half2 *>(&h[e]));
            f[2 * e] = t.x * scale;      // exact but beyond fp32's range
            f[2 * e + 1] = t.y * scale;
        }
        store_chunk<DT>(out + p.row * chunks * (DT == kF32 ? 32 : 16), ch, pack_chunk<DT>(f));
    }
}

// Warps to a row (1, 2, 4 or 8 of a CTA's 8), and the CTAs, for pieces of U scale tiles.
struct Shape {
    int wpr_log2;
    dim3 grid;
};
Shape shape_for(int64_t rows, int64_t tiles_k, int U) {
    Shape s;
    s.wpr_log2 = 0;
    while (s.wpr_log2 < 3 && ((int64_t)U << s.wpr_log2) < tiles_k) ++s.wpr_log2;
    s.grid = dim3((unsigned)ceil_div(rows, kWarps >> s.wpr_log2),
                  (unsigned)ceil_div(tiles_k, (int64_t)U << s.wpr_log2));
    return s;
}
// Four pieces a warp once that still leaves every SM (148, up to 64 warps each) full twice over.
bool deep(int64_t rows, int64_t tiles_k) { return rows * tiles_k >= 4 * 2 * 148 * 64; }

template <int DT, int U>
cudaError_t quantize_launch(const void *X, int64_t row_bytes, int64_t R, int64_t rows_out,
                            int64_t K, uint8_t *codes, uint8_t *scales, cudaStream_t s) {
    const int64_t tiles_k = ceil_div(K, kMxCols);
    const Shape sh = shape_for(rows_out, tiles_k, U);
    return launch_pdl(mxfp4_quantize_kernel<DT, U>, sh.grid, dim3(kThreads), s,
                      static_cast<const uint8_t *>(X), row_bytes, R, rows_out, K / 8, tiles_k,
                      sh.wpr_log2, reinterpret_cast<uint32_t *>(codes), scales);
}

template <int DT, int U>
cudaError_t dequant_launch(const uint8_t *codes, const uint8_t *scales, int64_t R, int64_t K,
                           void *out, cudaStream_t s) {
    const int64_t tiles_k = ceil_div(K, kMxCols);
    const Shape sh = shape_for(R, tiles_k, U);
    return launch_pdl(mxfp4_dequant_kernel<DT, U>, sh.grid, dim3(kThreads), s,
                      reinterpret_cast<const uint32_t *>(codes), scales, R, K / 8, tiles_k,
                      sh.wpr_log2, static_cast<uint8_t *>(out));
}

}  // namespace

cudaError_t launch_mxfp4_quantize(const void *X, int dtype, int64_t ldx, int64_t R,
                                  int64_t rows_out, int64_t K, uint8_t *codes, uint8_t *scales,
                                  cudaStream_t s) {
    const int64_t rb = ldx * (dtype == kF32 ? 4 : 2);
    const bool d = deep(rows_out, ceil_div(K, kMxCols));
    cudaError_t e;
    if (dtype == kF16)
        e = d ? quantize_launch<kF16, 4>(X, rb, R, rows_out, K, codes, scales, s)
              : quantize_launch<kF16, 1>(X, rb, R, rows_out, K, codes, scales, s);
    else if (dtype == kBF16)
        e = d ? quantize_launch<kBF16, 4>(X, rb, R, rows_out, K, codes, scales, s)
              : quantize_launch<kBF16, 1>(X, rb, R, rows_out, K, codes, scales, s);
    else
        e = d ? quantize_launch<kF32, 4>(X, rb, R, rows_out, K, codes, scales, s)
              : quantize_launch<kF32, 1>(X, rb, R, rows_out, K, codes, scales, s);
    note_launches(1);
    return e;
}

cudaError_t launch_mxfp4_dequant(const uint8_t *codes, const uint8_t *scales, int64_t R,
                                 int64_t K, void *out, int dtype, cudaStream_t s) {
    const bool d = deep(R, ceil_div(K, kMxCols));
    cudaError_t e;
    if (dtype == kF16)
        e = d ? dequant_launch<kF16, 4>(codes, scales, R, K, out, s)
              : dequant_launch<kF16, 1>(codes, scales, R, K, out, s);
    else if (dtype == kBF16)
        e = d ? dequant_launch<kBF16, 4>(codes, scales, R, K, out, s)
              : dequant_launch<kBF16, 1>(codes, scales, R, K, out, s);
    else
        e = d ? dequant_launch<kF32, 4>(codes, scales, R, K, out, s)
              : dequant_launch<kF32, 1>(codes, scales, R, K, out, s);
    note_launches(1);
    return e;
}

}  // namespace llmint8
