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
#include "kernels.h"
#include "launch.cuh"
#include "mxfp4.cuh"

namespace llmint8 {

namespace {

constexpr int kMaxWarps = 32;

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

// Norm factors of a row held as NCH chunks of 8 (zero outside the row): mean and 1 / deviation.
template <int NCH>
__device__ __forceinline__ void row_norm(const float (&v)[NCH][8], const bool (&in)[NCH], int kind,
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
    rstd = rsqrtf(row_sum(q, red + kMaxWarps, tpr) * inv_k + eps);
}

// v = (v - mean) * rstd * w + b over one chunk; w and b may be null.
template <int DT>
__device__ __forceinline__ void apply_norm(float (&v)[8], int kind, float mean, float rstd,
                                           const uint8_t *w, const uint8_t *b) {
    if (kind == LLMINT8_NORM_LAYER) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] -= mean;
    }
    float t[8];
    if (w) {
        unpack_chunk<DT>(load_chunk<DT>(w, 0), t);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= rstd * t[e];
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= rstd;
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

// Pitches and offsets are 32-bit bytes, one multiply-add to an address (with 64-bit ones a tenth more
// instructions, which is what bounds the fuller forms: 75 against 71 us for 4096 x 12288 with norms on
// both sides and a gate, 89 against 82 to MXFP4).
// FULL: the row fills its threads' chunks (as K = 1024, 4096 or 12288 does), which leaves out the
// tests of each of them, a tenth of the instructions again (71 against 65 us, 82 against 77).
template <int DT, int NCH, int THREADS, int CTAS, bool FULL>
__global__ void __launch_bounds__(THREADS, CTAS) residual_norm_kernel(const NormArgs a, int tpr_log2) {
    pdl_wait_then_release();
    __shared__ float red[4 * kMaxWarps];
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
        const uint32_t next = row + 148 * CTAS / 2 * rows;
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
    if (a.post_norm != LLMINT8_NORM_NONE) {
        row_norm<NCH>(h, in, a.post_norm, a.inv_k, a.eps, red, tpr, mean, rstd);
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
        if (hr && live) store_chunk<DT>(hr + i * step, 0, pack_chunk<DT>(h[i]));
    }
    if (a.norm == LLMINT8_NORM_NONE) return;   // uniform over the grid
    row_norm<NCH>(h, in, a.norm, a.inv_k, a.eps, red + 2 * kMaxWarps, tpr, mean, rstd);
    const uint8_t *w = share(a.weight, 0, 0, off), *b = share(a.bias, 0, 0, off);
    uint8_t *yr = share(a.Y, rc, a.pitch, off);
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
            if (yr && live) store_chunk<DT>(yr + i * step, 0, y);
        }
        // rows past M pad the last row of scale tiles with those of zeros
        if (!live) y = zero_chunk<DT>();
        if (cr && row < a.rows_out && (off + i * step) / 512 < a.tiles_k) {
            uint32_t word;
            const uint32_t q = quantize_chunk<DT>(y, word, lane);
            if (in[i] && live) *reinterpret_cast<uint32_t *>(cr + i * step / 4) = q;
            if ((lane & 15) == 0) *reinterpret_cast<uint32_t *>(sr + (uint64_t)i * step * 2) = word;
        }
    }
}

template <int DT>
cudaError_t norm_launch(const NormArgs &a, cudaStream_t s) {
    // Threads to a row (a power of two) and chunks to a thread (at most 4): what leaves the fewest
    // idle; of equals, up to 256 threads, else up to 512, and then two chunks, since several rows
    // to an SM, in CTAs of their own, keep its memory busy while one of them waits for its sums
    // (4096 x 16384 layer norm: 84 us with 512 threads, 99 with 1024).  A few rows take one chunk a
    // thread: a lone row's time is its chain of latencies.
    const int64_t chunks = (int64_t)a.tiles_k * 32;
    int best = 10;
    if (a.M <= 148) {
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
#define LLMINT8_NORM(N, THREADS, CTAS)                     \
    go(residual_norm_kernel<DT, N, THREADS, CTAS, true>, \
       residual_norm_kernel<DT, N, THREADS, CTAS, false>)
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
    const cudaError_t e = dtype == kF16 ? norm_launch<kF16>(a, s) : norm_launch<kBF16>(a, s);
    note_launches(1);
    return e;
}

}  // namespace llmint8
