// The MXFP4 format on the device: 32 consecutive elements of a row share one power-of-two scale
// (e8m0) and are e2m1 codes, two to a byte.  Shared by the quantiser and the residual norm.
//
// A chunk is 8 consecutive elements of a row, held by one lane; four neighbouring lanes hold a
// block of 32, and a warp 256 columns of a row, which is one row's share of a scale tile (128
// rows x 256 columns, 1024 bytes: block b of row r at 512 (b / 4) + 16 (r % 32) + 4 (r / 32) +
// b % 4, the order in which a tensor core wants the scales in its memory).
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"

namespace llmint8 {

constexpr int kMxCols = 256;             // columns of a scale tile
constexpr int kMxRows = 128;             // rows of a scale tile
constexpr int kMxTile = 1024;            // its bytes

// Element types of the 16-bit and 32-bit matrices (the values of llmint8_dtype).
constexpr int kF16 = LLMINT8_F16, kBF16 = LLMINT8_BF16, kF32 = LLMINT8_F32;

// The 8 elements of a chunk as loaded.
template <int DT>
struct Chunk {
    static constexpr int kWords = DT == kF32 ? 8 : 4;
    uint32_t w[kWords];
};

template <int DT>
__device__ __forceinline__ Chunk<DT> load_chunk(const void *base, int64_t chunk) {
    Chunk<DT> c;
    const uint4 *p = reinterpret_cast<const uint4 *>(base) + chunk * (Chunk<DT>::kWords / 4);
#pragma unroll
    for (int i = 0; i < Chunk<DT>::kWords / 4; ++i) {
        const uint4 v = p[i];
        c.w[4 * i] = v.x;
        c.w[4 * i + 1] = v.y;
        c.w[4 * i + 2] = v.z;
        c.w[4 * i + 3] = v.w;
    }
    return c;
}

// The same for what is read once: it leaves L1 to the vectors that every row reads.
template <int DT>
__device__ __forceinline__ Chunk<DT> stream_chunk(const void *base, int64_t chunk) {
    static_assert(DT != kF32, "16-bit rows");
    Chunk<DT> c;
    asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(c.w[0]), "=r"(c.w[1]), "=r"(c.w[2]), "=r"(c.w[3])
                 : "l"(reinterpret_cast<const uint4 *>(base) + chunk));
    return c;
}

template <int DT>
__device__ __forceinline__ Chunk<DT> zero_chunk() {
    Chunk<DT> c;
#pragma unroll
    for (int i = 0; i < Chunk<DT>::kWords; ++i) c.w[i] = 0u;
    return c;
}

template <int DT>
__device__ __forceinline__ void store_chunk(void *base, int64_t chunk, const Chunk<DT> &c) {
    uint4 *p = reinterpret_cast<uint4 *>(base) + chunk * (Chunk<DT>::kWords / 4);
#pragma unroll
    for (int i = 0; i < Chunk<DT>::kWords / 4; ++i)
        p[i] = make_uint4(c.w[4 * i], c.w[4 * i + 1], c.w[4 * i + 2], c.w[4 * i + 3]);
}

template <int DT>
__device__ __forceinline__ void unpack_chunk(const Chunk<DT> &c, float (&f)[8]) {
    if constexpr (DT == kF32) {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = __uint_as_float(c.w[e]);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if constexpr (DT == kF16) {
                const float2 t = __half22float2(*reinterpret_cast<const __half2 *>(&c.w[e]));
                f[2 * e] = t.x;
                f[2 * e + 1] = t.y;
            } else {                     // bf16: the upper half of an fp32
                f[2 * e] = __uint_as_float(c.w[e] << 16);
                f[2 * e + 1] = __uint_as_float(c.w[e] & 0xffff0000u);
            }
        }
    }
}

// Two values rounded to the 16-bit type (to nearest, ties to even), the first in the low half.
template <int DT>
__device__ __forceinline__ uint32_t pack_pair(float a, float b) {
    if constexpr (DT == kF16) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
}

template <int DT>
__device__ __forceinline__ Chunk<DT> pack_chunk(const float (&f)[8]) {
    Chunk<DT> c;
    if constexpr (DT == kF32) {
#pragma unroll
        for (int e = 0; e < 8; ++e) c.w[e] = __float_as_uint(f[e]);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) c.w[e] = pack_pair<DT>(f[2 * e], f[2 * e + 1]);
    }
    return c;
}

// The bits of max |x| over the chunk, as an integer of the type's width: non-negative floats
// order as their bits do, an infinity above every finite value and a NaN above that.
template <int DT>
__device__ __forceinline__ uint32_t chunk_absmax_bits(const Chunk<DT> &c) {
    if constexpr (DT == kF32) {
        uint32_t m = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) m = max(m, c.w[e] & 0x7fffffffu);
        return m;
    } else {
        uint32_t m = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) m = __vmaxu2(m, c.w[e] & 0x7fff7fffu);
        return max(m & 0xffffu, m >> 16);
    }
}

// The scale byte of a block whose max |x| has these bits: 2^(floor(log2 max) - 2), that is the
// exponent field less 2, not below the format's least; 255 (NaN) for a NaN or an infinity.
template <int DT>
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax_bits) {
    uint32_t f, top;
    if constexpr (DT == kF16) {
        f = __float_as_uint(__half2float(__ushort_as_half((unsigned short)amax_bits)));
        top = 0x7c00u;
    } else if constexpr (DT == kBF16) {
        f = amax_bits << 16;
        top = 0x7f80u;
    } else {
        f = amax_bits;
        top = 0x7f800000u;
    }
    const int e = (int)(f >> 23) - 2;
    return amax_bits >= top ? 255u : (uint32_t)max(e, 0);
}

// x / scale is exact in fp32 but where it falls below 2^-126, far under half the least code.
__device__ __forceinline__ float inverse_scale(uint32_t s) {
    return __uint_as_float((254u - min(s, 254u)) << 23);
}

// Eight e2m1 codes, element 0 in the lowest four bits; the conversion rounds to nearest, ties
// to the even code, and takes what lies beyond 6 to 6.
__device__ __forceinline__ uint32_t e2m1_codes(const float (&f)[8], float inv) {
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(r)
        : "f"(f[0] * inv), "f"(f[1] * inv), "f"(f[2] * inv), "f"(f[3] * inv), "f"(f[4] * inv),
          "f"(f[5] * inv), "f"(f[6] * inv), "f"(f[7] * inv));
    return r;
}

// Warp-wide: quantises 256 columns of a row whose chunks the lanes hold (zero past K).  Returns
// this lane's eight codes; `word` gets the scale bytes of its half warp's four blocks.
template <int DT>
__device__ __forceinline__ uint32_t quantize_chunk(const Chunk<DT> &c, uint32_t &word, int lane) {
    uint32_t m = chunk_absmax_bits<DT>(c);
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    const uint32_t s = scale_byte<DT>(m);
    word = s << (8 * ((lane >> 2) & 3));
    word |= __shfl_xor_sync(0xffffffffu, word, 4);
    word |= __shfl_xor_sync(0xffffffffu, word, 8);
    float f[8];
    unpack_chunk<DT>(c, f);
    return e2m1_codes(f, inverse_scale(s));
}

}  // namespace llmint8
