// What stands between two blocks of a transformer, in one pass over the rows:
//     h = residual + scale * gate * PostNorm(x)
//     y = Norm(h)
// where a norm is v / sqrt(mean(v^2) + eps) * w + b ("rms") or the same of v - mean(v) ("layer"),
// both norms, the residual and the gate are optional, and y leaves as 16-bit values, as an MXFP4
// operand for the product that follows, or both.
//
// Bound by HBM: x and the residual are read once, h and y written once.  So a row stays in the
// registers of its threads (8 elements to a chunk, up to 4 chunks a thread, 32 to 1024 threads a
// row) from its loads to its stores, and each sum over the row is a shuffle tree and one exchange
// through shared memory.  All arithmetic is fp32; h and y are each rounded once, y from the
// unrounded h, and the MXFP4 form is that of the rounded y, so that it is bit for bit what
// quantising the stored y gives.  A layer norm's variance is the mean of (v - mean)^2, summed
// after the mean is known: the difference of mean squares would cancel.
#include <cfloat>
#include <cmath>

#include "kernels.h"
#include "launch.cuh"
#include "mxfp4.cuh"

namespace llmint8 {

namespace {

constexpr int kMaxWarps = 32;
constexpr int kSms = 148;                // of a B200; nothing but speed depends on it
// A mean square (with eps) from here on has lost nothing to squares below fp32's range: those are under
// 2^-126 each.
constexpr float kLeastSquare = 0x1p-100f;

// Sum over the `tpr` threads of this row (a power of two, 32 to 1024); every thread of the CTA
// takes part.  `red` has one slot per warp, and two calls in turn use two sets of them.
__device__ __forceinline__ float row_sum(float v, float *red, int tpr) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (tpr == 32) return v;
    const int warp = threadIdx.x >> 5, wpr = tpr >> 5;
    if ((threadIdx.x & 31) == 0) red[warp] = v;
    __syncthreads();
    // lane l takes warp l of the row, so that every thread adds in the same order
    const int l = threadIdx.x & 31;
    v = l < wpr ? red[(warp & ~(wpr - 1)) + l] : 0.0f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Norm factors of a row held as NCH chunks of 8 (zero outside the row): mean and 1 / deviation.  False,
// in all threads of the row, where fp32 may not hold the squares (see scaled_row).
template <int NCH>
__device__ __forceinline__ bool row_norm(const float (&v)[NCH][8], const bool (&in)[NCH], int kind,
                                         float inv_k, float eps, float *red, int tpr, float &mean,
                                         float &rstd) {
    mean = 0.0f;
    if (kind == LLMINT8_NORM_LAYER) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < NCH; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) s += v[i][e];
        mean = row_sum(s, red, tpr) * inv_k;
    }
    float q = 0.0f;
    if (kind == LLMINT8_NORM_LAYER) {
#pragma unroll
        for (int i = 0; i < NCH; ++i)
            if (in[i]) {
#pragma unroll
                for (int e = 0; e < 8; ++e) q = fmaf(v[i][e] - mean, v[i][e] - mean, q);
            }
    } else {
#pragma unroll
        for (int i = 0; i < NCH; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) q = fmaf(v[i][e], v[i][e], q);
    }
    const float m = row_sum(q, red + kMaxWarps, tpr) * inv_k + eps;
    rstd = rsqrtf(m);
    return m >= kLeastSquare && m <= FLT_MAX;
}

// v = (v - mean) * rstd * w + b over one chunk, in that order; w and b may be null.
template <int DT>
__device__ __forceinline__ void apply_norm(float (&v)[8], int kind, float mean, float rstd,
                                           const uint8_t *w, const uint8_t *b) {
    if (kind == LLMINT8_NORM_LAYER) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] -= mean;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= rstd;
    float t[8];
    if (w) {
        unpack_chunk<DT>(load_chunk<DT>(w, 0), t);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= t[e];
    }
    if (b) {
        unpack_chunk<DT>(load_chunk<DT>(b, 0), t);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += t[e];
    }
}

// A thread's share of an array with rows: its first chunk of row `row`.
__device__ __forceinline__ const uint8_t *share(const void *base, uint32_t row, uint32_t pitch,
                                                uint32_t off) {
    return base ? static_cast<const uint8_t *>(base) + (uint64_t)row * pitch + off : nullptr;
}
__device__ __forceinline__ uint8_t *share(void *base, uint32_t row, uint32_t pitch, uint32_t off) {
    return const_cast<uint8_t *>(share(static_cast<const void *>(base), row, pitch, off));
}

// The MXFP4 form of a row's chunk that begins `at` bytes into it (`in` the row, else padding), by all
// lanes of a warp.
template <int DT>
__device__ __forceinline__ void store_mx(const NormArgs &a, const Chunk<DT> &y, uint32_t row, uint32_t at,
                                         bool in) {
    const int lane = threadIdx.x & 31;
    uint32_t word;
    const uint32_t q = quantize_chunk<DT>(y, word, lane);
    if (in) *reinterpret_cast<uint32_t *>(share(a.codes, row, a.pitch / 4, at / 4)) = q;
    // a row's share of a scale tile: a word to each half warp (a warp's 32 chunks are 256 columns)
    if ((lane & 15) == 0)
        *reinterpret_cast<uint32_t *>(
            a.scales + ((uint64_t)(row / kMxRows) * a.tiles_k + at / 512) * kMxTile + (lane >> 4) * 512 +
            (row & 31) * 16 + ((row >> 5) & 3) * 4) = word;
}

// ---- Rows whose squares leave fp32's range: from about 1e19 on, and below 1e-19, where values of bf16
// (and scaled ones of either type) need not.  Such a row is scaled by the power of two that brings the
// larger of max |v| and sqrt(eps) near 1, which changes y by nothing:
//     v * 2^-e / sqrt(mean((v * 2^-e)^2) + eps * 2^-2e)
// A row with an infinity or a NaN comes here too, and keeps it.  The kernel leaves these rows to its end, out
// of the way of the others' registers: it writes nothing of a row whose PostNorm comes out so, which then begins
// anew from X, and of one whose Norm does it keeps h, by stores without a branch, in local memory.
// (2048 x 4096 bf16 with norms on both sides, us, to 16 bits and to MXFP4: scaling in place 17.6 and
// 19.0, this 13.9 and 16.1, no such rows at all 13.8 and 15.7.)

// Eight values to a thread's local memory if `on`, and from there.
__device__ __forceinline__ void keep(float *p, const float (&v)[8], bool on = true) {
#pragma unroll
    for (int e = 0; e < 8; e += 4)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.u32 p, %0, 0;\n\t"
            "@p st.v4.f32 [%1], {%2, %3, %4, %5};\n\t}" ::"r"((uint32_t)on),
            "l"(p + e), "f"(v[e]), "f"(v[e + 1]), "f"(v[e + 2]), "f"(v[e + 3]));
}
__device__ __forceinline__ void kept(const float *p, float (&v)[8]) {
#pragma unroll
    for (int e = 0; e < 8; e += 4)
        asm volatile("ld.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(v[e]), "=f"(v[e + 1]), "=f"(v[e + 2]), "=f"(v[e + 3])
                     : "l"(p + e));
}

// Reduction over the threads of this row alone.  Rows of 32 threads need no barrier; there are at most
// four others in a CTA, each with a barrier of its own (by number: with a barrier chosen by a register the
// kernel holds all sixteen, and fewer CTAs fit an SM).
template <typename F>
__device__ __forceinline__ float row_reduce(float v, float *red, int tpr, F op) {
#pragma unroll 1
    for (int o = 16; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
    if (tpr == 32) return v;
    const int warp = threadIdx.x >> 5, wpr = tpr >> 5, l = threadIdx.x & 31;
    if (l == 0) red[warp] = v;
    switch (threadIdx.x / tpr) {
        case 0: asm volatile("bar.sync 1, %0;" ::"r"(tpr) : "memory"); break;
        case 1: asm volatile("bar.sync 2, %0;" ::"r"(tpr) : "memory"); break;
        case 2: asm volatile("bar.sync 3, %0;" ::"r"(tpr) : "memory"); break;
        default: asm volatile("bar.sync 4, %0;" ::"r"(tpr) : "memory");
    }
    v = l < wpr ? red[(warp & ~(wpr - 1)) + l] : 0.0f;       // 0 changes neither sums nor maxima
#pragma unroll 1
    for (int o = 16; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// Scales the row, `n` values of it in this thread, in place and gives its norm factors.  `red` has
// three sets of slots.
__device__ __forceinline__ void scaled_factors(float *h, int n, int kind, float inv_k, float eps,
                                               float *red, int tpr, float &mean, float &rstd) {
    const auto add = [](float a, float b) { return a + b; };
    const auto larger = [](float a, float b) { return fmaxf(a, b); };
    float v[8], top = 0.0f, sum = 0.0f, q = 0.0f;
#pragma unroll 1
    for (int i = 0; i < n; i += 8) {
        kept(h + i, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(v[e]));
    }
    const float root = sqrtf(eps);
    top = fmaxf(row_reduce(top, red, tpr, larger), root);
    // 2^-e for e the exponent of top, held between -126 and 126
    const int field = min(max((int)(__float_as_uint(top) >> 23), 1), 253);
    const float s = __uint_as_float((uint32_t)(254 - field) << 23);
#pragma unroll 1
    for (int i = 0; i < n; i += 8) {
        kept(h + i, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum += v[e] *= s;
        keep(h + i, v);
    }
    mean = kind == LLMINT8_NORM_LAYER ? row_reduce(sum, red + kMaxWarps, tpr, add) * inv_k : 0.0f;
#pragma unroll 1
    for (int i = 0; i < n; i += 8) {
        kept(h + i, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) q = fmaf(v[e] - mean, v[e] - mean, q);
    }
    rstd = rsqrtf(row_reduce(q, red + 2 * kMaxWarps, tpr, add) * inv_k + (root * s) * (root * s));
}

// One row, by all of its threads, each with its chunks in `h`: from PostNorm on (`post`; of X then), or
// from Norm on.
template <int DT>
__device__ __noinline__ void scaled_row(const NormArgs &a, float *h, bool post, int tpr, uint32_t row,
                                        float *red) {
    const uint32_t off = (threadIdx.x & (tpr - 1)) * 16u, step = tpr * 16u;
    const int n = off < a.pitch ? (int)((a.pitch - off + step - 1) / step) * 8 : 0;
    float v[8], u[8];
    if (post) {
#pragma unroll 1
        for (int i = 0; i < n; i += 8) {
            unpack_chunk<DT>(load_chunk<DT>(share(a.X, row, a.x_pitch, off + i / 8 * step), 0), v);
            keep(h + i, v);
        }
    }
#pragma unroll 1
    for (int turn = post ? 0 : 1; turn < 2; ++turn) {
        const int kind = turn ? a.norm : a.post_norm;
        const void *w = turn ? a.weight : a.post_weight, *b = turn ? a.bias : a.post_bias;
        if (kind == LLMINT8_NORM_NONE) break;
        float mean, rstd;
        scaled_factors(h, n, kind, a.inv_k, a.eps, red + 3 * turn * kMaxWarps, tpr, mean, rstd);
#pragma unroll 1
        for (int i = 0; off + i / 8 * step < a.tiles_k * 512; i += 8) {       // uniform over the warp
            const uint32_t at = off + i / 8 * step;
            if (i < n) {
                kept(h + i, v);
                apply_norm<DT>(v, kind, mean, rstd, share(w, 0, 0, at), share(b, 0, 0, at));
            }
            if (turn) {
                const Chunk<DT> y = i < n ? pack_chunk<DT>(v) : zero_chunk<DT>();
                if (i < n && a.Y) store_chunk<DT>(share(a.Y, row, a.pitch, at), 0, y);
                if (a.codes) store_mx<DT>(a, y, row, at, i < n);
            } else if (i < n) {
                if (a.gate) {
                    unpack_chunk<DT>(load_chunk<DT>(share(a.gate, row / a.gate_group, a.pitch, at), 0), u);
                    for (int e = 0; e < 8; ++e) v[e] *= u[e];
                }
                unpack_chunk<DT>(a.residual ? load_chunk<DT>(share(a.residual, row, a.r_pitch, at), 0)
                                            : zero_chunk<DT>(), u);
                for (int e = 0; e < 8; ++e) v[e] = fmaf(v[e], a.scale, u[e]);
                keep(h + i, v);
                if (a.H) store_chunk<DT>(share(a.H, row, a.pitch, at), 0, pack_chunk<DT>(v));
            }
        }
    }
}

// Pitches and offsets are 32-bit bytes, one multiply-add to an address (with 64-bit ones a tenth more
// instructions, which is what bounds the fuller forms: 75 against 71 us for 4096 x 12288 with norms on
// both sides and a gate, 89 against 82 to MXFP4).
// FULL: the row fills its threads' chunks (as K = 1024, 4096 or 12288 does), which leaves out the
// tests of each of them, a tenth of the instructions again (71 against 65 us, 82 against 77).
// WIDE: rows whose squares leave fp32's range are looked for.
template <int DT, int NCH, int THREADS, int CTAS, bool FULL, bool WIDE>
__global__ void __launch_bounds__(THREADS, CTAS)
residual_norm_kernel(const __grid_constant__ NormArgs a, int tpr_log2) {
    pdl_wait_then_release();
    __shared__ float red[(WIDE ? 10 : 4) * kMaxWarps];        // two sets a norm, three of a scaled one
    const int tpr = 1 << tpr_log2;
    const int t = threadIdx.x & (tpr - 1), lane = threadIdx.x & 31;
    const uint32_t rows = blockDim.x >> tpr_log2;             // of a CTA
    const uint32_t row = blockIdx.x * rows + (threadIdx.x >> tpr_log2);
    const bool live = row < a.M;
    const uint32_t rc = live ? row : 0u;
    const uint32_t off = t * 16u, step = 16u << tpr_log2;     // this thread's chunks, in bytes

    const uint8_t *xr = share(a.X, rc, a.x_pitch, off);
    const uint8_t *rr = share(a.residual, rc, a.r_pitch, off);
    // Rows that CTAs half a wave on will load are fetched into L2 meanwhile, so that HBM works
    // through this wave's sums too (4096 x 12288 layer norm: 69.7 us without, 66.3 with).  Not beside
    // the MXFP4 form, whose arithmetic is the bound instead (2048 x 4096: 13.3 and 14.0).
    if (t == 0 && !a.codes) {
        const uint32_t next = row + kSms * CTAS / 2 * rows;
        if (next < a.M) {
            prefetch_l2(share(a.X, next, a.x_pitch, 0), a.pitch);
            if (rr) prefetch_l2(share(a.residual, next, a.r_pitch, 0), a.pitch);
        }
    }
    Chunk<DT> x[NCH], r[NCH];
    bool in[NCH];
#pragma unroll
    for (int i = 0; i < NCH; ++i) {      // issue every load before using any
        in[i] = FULL || off + i * step < a.pitch;
        x[i] = in[i] ? stream_chunk<DT>(xr + i * step, 0) : zero_chunk<DT>();
        r[i] = in[i] && rr ? stream_chunk<DT>(rr + i * step, 0) : zero_chunk<DT>();
    }
    float h[NCH][8];
#pragma unroll
    for (int i = 0; i < NCH; ++i) unpack_chunk<DT>(x[i], h[i]);
    float mean, rstd;
    bool post_ok = true, ok = true;
    __align__(16) float left[WIDE ? NCH * 8 : 4];             // what scaled_row takes up
    if (a.post_norm != LLMINT8_NORM_NONE) {
        post_ok = row_norm<NCH>(h, in, a.post_norm, a.inv_k, a.eps, red, tpr, mean, rstd);
        const uint8_t *w = share(a.post_weight, 0, 0, off), *b = share(a.post_bias, 0, 0, off);
#pragma unroll
        for (int i = 0; i < NCH; ++i)
            if (in[i])
                apply_norm<DT>(h[i], a.post_norm, mean, rstd, w ? w + i * step : nullptr,
                               b ? b + i * step : nullptr);
    }
    const uint8_t *g = a.gate ? share(a.gate, rc / a.gate_group, a.pitch, off) : nullptr;
    uint8_t *hr = share(a.H, rc, a.pitch, off);
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
        if (!in[i]) continue;
        float u[8];
        if (g) {
            unpack_chunk<DT>(load_chunk<DT>(g + i * step, 0), u);
#pragma unroll
            for (int e = 0; e < 8; ++e) h[i][e] *= u[e];
        }
        unpack_chunk<DT>(r[i], u);
#pragma unroll
        for (int e = 0; e < 8; ++e) h[i][e] = fmaf(h[i][e], a.scale, u[e]);
        if (hr && live && (!WIDE || post_ok)) store_chunk<DT>(hr + i * step, 0, pack_chunk<DT>(h[i]));
    }
    if (a.norm != LLMINT8_NORM_NONE) {
        ok = row_norm<NCH>(h, in, a.norm, a.inv_k, a.eps, red + 2 * kMaxWarps, tpr, mean, rstd);
        if constexpr (WIDE) {
#pragma unroll
            for (int i = 0; i < NCH; ++i) keep(left + 8 * i, h[i], !ok);
        }
        const bool put = live && (!WIDE || (post_ok && ok));
        const uint8_t *w = share(a.weight, 0, 0, off), *b = share(a.bias, 0, 0, off);
        uint8_t *yr = share(a.Y, rc, a.pitch, off);
        if (!a.codes) {
#pragma unroll
            for (int i = 0; i < NCH; ++i)
                if (in[i]) {
                    apply_norm<DT>(h[i], a.norm, mean, rstd, w ? w + i * step : nullptr,
                                   b ? b + i * step : nullptr);
                    if (put) store_chunk<DT>(yr + i * step, 0, pack_chunk<DT>(h[i]));
                }
        } else {
            // the grid ends with the last row of scale tiles: a CTA's rows, up to 8, divide 128
            uint8_t *cr = share(a.codes, rc, a.pitch / 4, off / 4);
            // the row's first scale word of this half warp (a warp's 32 chunks are 256 columns)
            uint8_t *sr = a.scales + ((uint64_t)(row / kMxRows) * a.tiles_k + off / 512) * kMxTile +
                          (lane >> 4) * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4;
#pragma unroll
            for (int i = 0; i < NCH; ++i) {
                Chunk<DT> y = zero_chunk<DT>();
                if (in[i]) {
                    apply_norm<DT>(h[i], a.norm, mean, rstd, w ? w + i * step : nullptr,
                                   b ? b + i * step : nullptr);
                    y = pack_chunk<DT>(h[i]);
                    if (yr && put) store_chunk<DT>(yr + i * step, 0, y);
                }
                // rows past M pad the last row of scale tiles with those of zeros
                if (!live) y = zero_chunk<DT>();
                if (FULL || (off + i * step) / 512 < a.tiles_k) {
                    uint32_t word;
                    const uint32_t q = quantize_chunk<DT>(y, word, lane);
                    if (in[i] && live) *reinterpret_cast<uint32_t *>(cr + i * step / 4) = q;
                    if ((lane & 15) == 0) *reinterpret_cast<uint32_t *>(sr + (uint64_t)i * step * 2) = word;
                }
            }
        }
    }
    if constexpr (WIDE) {
        if (live && !(post_ok && ok)) scaled_row<DT>(a, left, !post_ok, tpr, row, red + 4 * kMaxWarps);
    }
}

template <int DT, bool WIDE>
cudaError_t norm_launch(const NormArgs &a, cudaStream_t s) {
    // Threads to a row (a power of two) and chunks to a thread (at most 4): what leaves the fewest
    // idle; of equals, up to 256 threads, else up to 512, and then two chunks, since several rows
    // to an SM, in CTAs of their own, keep its memory busy while one of them waits for its sums
    // (4096 x 16384 layer norm: 84 us with 512 threads, 99 with 1024).  A few rows take one chunk a
    // thread: a lone row's time is its chain of latencies.
    const int64_t chunks = (int64_t)a.tiles_k * 32;
    int best = 10;
    if (a.M <= kSms) {
        best = 5;
        while (best < 10 && ((int64_t)1 << best) < chunks) ++best;
    } else {
        int64_t least = INT64_MAX;
        for (int l = 5; l <= 10; ++l) {
            const int64_t n = ceil_div(chunks, (int64_t)1 << l);
            if (n > 4) continue;
            const int64_t cost = ((n << l) << 4) + (l > 9 ? 8 : l > 8 ? 4 : 0) + (n == 1 ? 2 : 0) + n;
            if (cost < least) {
                least = cost;
                best = l;
            }
        }
    }
    const int per = (int)ceil_div(chunks, (int64_t)1 << best);
    const int threads = std::max(1 << best, 256);
    const int64_t rows = a.codes ? a.rows_out : a.M;
    const dim3 grid((unsigned)ceil_div(rows, threads >> best));
    const bool full = a.pitch == (uint32_t)per * (16u << best);
    const auto go = [&](auto when_full, auto otherwise) {
        return launch_pdl(full ? when_full : otherwise, grid, dim3(threads), s, a, best);
    };
#define LLMINT8_NORM(N, THREADS, CTAS)                           \
    go(residual_norm_kernel<DT, N, THREADS, CTAS, true, WIDE>, \
       residual_norm_kernel<DT, N, THREADS, CTAS, false, WIDE>)
    if (threads == 256)
        return per == 1   ? LLMINT8_NORM(1, 256, 8)
               : per == 2 ? LLMINT8_NORM(2, 256, 6)
               : per == 3 ? LLMINT8_NORM(3, 256, 4)
                          : LLMINT8_NORM(4, 256, 4);
    if (threads == 512)
        return per == 1   ? LLMINT8_NORM(1, 512, 2)
               : per == 3 ? LLMINT8_NORM(3, 512, 2)
                          : LLMINT8_NORM(4, 512, 2);   // two go to 256 threads, with four
    return per == 1   ? LLMINT8_NORM(1, 1024, 1)
           : per == 2 ? LLMINT8_NORM(2, 1024, 1)
           : per == 3 ? LLMINT8_NORM(3, 1024, 1)
                      : LLMINT8_NORM(4, 1024, 1);
#undef LLMINT8_NORM
}

}  // namespace

cudaError_t launch_residual_norm(const NormArgs &a, int dtype, cudaStream_t s) {
    // fp16 rows cannot leave fp32's range unless eps or the scale is out of the ordinary: |h| is at most
    // 2^16 + |scale| 2^40 (a residual; a post norm's sqrt(32768) times a weight, plus a bias, times a
    // gate), and 32768 squares of differences from a mean of such values stay below 2^128.
    const bool wide = dtype == kBF16 || a.eps < kLeastSquare || fabsf(a.scale) > 16384.0f;
    const cudaError_t e = dtype == kBF16 ? norm_launch<kBF16, true>(a, s)
                          : wide         ? norm_launch<kF16, true>(a, s)
                                         : norm_launch<kF16, false>(a, s);
    note_launches(1);
    return e;
}

}  // namespace llmint8
