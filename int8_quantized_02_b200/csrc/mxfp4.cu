// MXFP4 quantisation of the rows of a matrix, and the way back.  Both are bound by HBM: they
// read and write each value once (17/32 byte an element in MXFP4 form) and compute little.
//
// A warp takes 256 columns (a scale tile's width, 8 elements a lane) of the four rows r, r + 32,
// r + 64 and r + 96 of a scale tile, all of whose loads are in flight at once.  A block's maximum
// is two shuffles among four lanes, its codes one 32-bit store a lane; and the scales of those
// four rows are neighbours in the tile, so that half a warp's four blocks of each row make one
// 16-byte store.  16384 x 4096 fp16: 30 us, 5.7 TB/s (with one row to a warp and 4-byte stores 38 us).
#include "kernels.h"
#include "launch.cuh"
#include "mxfp4.cuh"

namespace llmint8 {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

constexpr int kRows = 4;                 // rows of a warp, 32 apart

// A warp's tile column and first row, and where the scales of its half warp's blocks lie: four
// words in a row, one for each of its rows.
struct Place {
    uint32_t row, kt;
    __device__ __forceinline__ explicit Place(int wpr_log2) {
        const uint32_t w = threadIdx.x >> 5;
        const uint32_t g = blockIdx.x * (kWarps >> wpr_log2) + (w >> wpr_log2);
        row = (g >> 5) * kMxRows + (g & 31);
        kt = (blockIdx.y << wpr_log2) + (w & ((1u << wpr_log2) - 1));
    }
    __device__ __forceinline__ uint64_t scales(uint32_t tiles_k, int lane) const {
        return (uint64_t)((row / kMxRows) * tiles_k + kt) * kMxTile + (lane >> 4) * 512 +
               (row & 31) * 16;
    }
};

// Rows R to the next multiple of 128 get zero scales; with `pad` false that is left out for those
// that no row below R shares a store with.
template <int DT>
__global__ void __launch_bounds__(kThreads)
mxfp4_quantize_kernel(const uint8_t *__restrict__ X, uint32_t row_bytes, uint32_t R, bool pad,
                      uint32_t chunks, uint32_t tiles_k, int wpr_log2,
                      uint32_t *__restrict__ codes, uint8_t *__restrict__ scales) {
    // a product that follows sets up, and asks L2 for its weight, while this waits and works
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31;
    const Place p(wpr_log2);
    if (p.kt >= tiles_k || (!pad && p.row >= R)) return;
    const uint32_t ch = p.kt * 32 + lane;
    const bool in = ch < chunks;
    const uint8_t *x = X + (uint64_t)p.row * row_bytes + ch * (DT == kF32 ? 32 : 16);
    Chunk<DT> c[kRows];
#pragma unroll
    for (int j = 0; j < kRows; ++j)      // issue every load before using any
        c[j] = in && p.row + 32 * j < R ? load_chunk<DT>(x + (uint64_t)(32 * j) * row_bytes, 0)
                                        : zero_chunk<DT>();
    uint32_t *q = codes + (uint64_t)p.row * chunks + ch;
    uint32_t word[kRows];
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
        const uint32_t v = quantize_chunk<DT>(c[j], word[j], lane);
        if (in && p.row + 32 * j < R) q[(uint64_t)(32 * j) * chunks] = v;
    }
    if ((lane & 15) == 0)
        *reinterpret_cast<uint4 *>(scales + p.scales(tiles_k, lane)) =
            make_uint4(word[0], word[1], word[2], word[3]);
}

template <int DT>
__global__ void __launch_bounds__(kThreads)
mxfp4_dequant_kernel(const uint32_t *__restrict__ codes, const uint8_t *__restrict__ scales,
                     uint32_t R, uint32_t chunks, uint32_t tiles_k, int wpr_log2,
                     uint8_t *__restrict__ out) {
    pdl_wait_then_release();
    const int lane = threadIdx.x & 31;
    const Place p(wpr_log2);
    const uint32_t ch = p.kt * 32 + lane;
    if (ch >= chunks || p.row >= R) return;
    const uint32_t here = min(chunks - p.kt * 32, 32u);       // lanes that go on, from 0
    uint32_t q[kRows];
    const uint32_t *at = codes + (uint64_t)p.row * chunks + ch;
#pragma unroll
    for (int j = 0; j < kRows; ++j)      // issue every load before using any
        q[j] = p.row + 32 * j < R ? at[(uint64_t)(32 * j) * chunks] : 0u;
    const uint4 words = *reinterpret_cast<const uint4 *>(scales + p.scales(tiles_k, lane));
    const uint32_t word[kRows] = {words.x, words.y, words.z, words.w};
    constexpr int kBytes = DT == kF32 ? 32 : 16;
    const uint32_t pitch = chunks * kBytes;
    uint8_t *o = out + (uint64_t)p.row * pitch + ch * kBytes;
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
        if (p.row + 32 * j >= R) break;
        uint32_t h[4];
        asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
            "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
            "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
            "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
            "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
            "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
            : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
            : "r"(q[j]));
        // 2^(s - 127): an exponent field, or the subnormal 2^-127; 255 stands for NaN
        const uint32_t s = (word[j] >> (8 * ((lane >> 2) & 3))) & 0xffu;
        const float scale = __uint_as_float(s == 0u     ? 0x00400000u
                                            : s == 255u ? 0x7fc00000u
                                                        : s << 23);
        float f[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 t = __half22float2(*reinterpret_cast<const __half2 *>(&h[e]));
            f[2 * e] = t.x * scale;      // exact but beyond fp32's range
            f[2 * e + 1] = t.y * scale;
        }
        if constexpr (DT == kF32) {
            // two neighbours trade halves, so that each store of the warp is one run of bytes
            // (chunks come in fours, so both are there)
            const bool odd = lane & 1;
            float g[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                g[e] = __shfl_xor_sync(0xffffffffu >> (32 - here), odd ? f[e] : f[4 + e], 1);
            float4 *pair = reinterpret_cast<float4 *>(o + (uint64_t)(32 * j) * pitch) - (odd ? 1 : 0);
            pair[0] = odd ? make_float4(g[0], g[1], g[2], g[3]) : make_float4(f[0], f[1], f[2], f[3]);
            pair[2] = odd ? make_float4(f[4], f[5], f[6], f[7]) : make_float4(g[0], g[1], g[2], g[3]);
        } else {
            store_chunk<DT>(o + (uint64_t)(32 * j) * pitch, 0, pack_chunk<DT>(f));
        }
    }
}

// Warps to a row (1, 2, 4 or 8 of a CTA's 8), and the CTAs.
struct Shape {
    int wpr_log2;
    dim3 grid;
};
Shape shape_for(int64_t R, int64_t tiles_k) {
    Shape s;
    s.wpr_log2 = 0;
    while (s.wpr_log2 < 3 && (1 << s.wpr_log2) < tiles_k) ++s.wpr_log2;
    const int64_t groups = ceil_div(R, kMxRows) * 32;
    s.grid = dim3((unsigned)ceil_div(groups, kWarps >> s.wpr_log2),
                  (unsigned)ceil_div(tiles_k, 1 << s.wpr_log2));
    return s;
}

}  // namespace

cudaError_t launch_mxfp4_quantize(const void *X, int dtype, int64_t ldx, int64_t R, bool pad,
                                  int64_t K, uint8_t *codes, uint8_t *scales, cudaStream_t s) {
    const int64_t tiles_k = ceil_div(K, kMxCols);
    const Shape sh = shape_for(R, tiles_k);
    auto k = dtype == kF16    ? mxfp4_quantize_kernel<kF16>
             : dtype == kBF16 ? mxfp4_quantize_kernel<kBF16>
                              : mxfp4_quantize_kernel<kF32>;
    const cudaError_t e =
        launch_pdl(k, sh.grid, dim3(kThreads), s, static_cast<const uint8_t *>(X),
                   (uint32_t)(ldx * (dtype == kF32 ? 4 : 2)), (uint32_t)R, pad, (uint32_t)(K / 8),
                   (uint32_t)tiles_k, sh.wpr_log2,
                   reinterpret_cast<uint32_t *>(codes), scales);
    note_launches(1);
    return e;
}

cudaError_t launch_mxfp4_dequant(const uint8_t *codes, const uint8_t *scales, int64_t R,
                                 int64_t K, void *out, int dtype, cudaStream_t s) {
    const int64_t tiles_k = ceil_div(K, kMxCols);
    const Shape sh = shape_for(R, tiles_k);
    auto k = dtype == kF16    ? mxfp4_dequant_kernel<kF16>
             : dtype == kBF16 ? mxfp4_dequant_kernel<kBF16>
                              : mxfp4_dequant_kernel<kF32>;
    const cudaError_t e = launch_pdl(k, sh.grid, dim3(kThreads), s,
                                     reinterpret_cast<const uint32_t *>(codes), scales, (uint32_t)R,
                                     (uint32_t)(K / 8), (uint32_t)tiles_k, sh.wpr_log2,
                                     static_cast<uint8_t *>(out));
    note_launches(1);
    return e;
}

}  // namespace llmint8
