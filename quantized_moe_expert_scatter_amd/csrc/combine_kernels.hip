// combine_kernels.hip -- the MoE combine after the down product: each token's
// output row is the routing-weighted sum of its topk expert rows.
//
// "Strata" PR #3752 names the combine among the prompt-path fusions its port
// leaves out and prints no formula; the reading here is the plain weighted
// sum, one fp32 fused multiply-add per term in slot order from zero:
//   out[t][n] = fmaf(w[t][K-1], dm[t*K+K-1][n], ... fmaf(w[t][0], dm[t*K][n], 0))
// The down product writes dm in (token, slot) order, so a token's K rows are
// consecutive and every read and write is a contiguous float4 run: the kernel
// is bound by HBM (K + 1 rows of H floats per token).  When dm is larger than
// the 256 MB infinity cache it is read and the output written non-temporally
// (10 % faster at 16K tokens); a smaller dm, which the down product has just
// written, is still in that cache and is read normally.
//
// The combine's gradient reads the same rows once more: a token's output
// gradient against each of its K rows (the routing weights' gradient), and
// times each weight (the rows' gradient).  It is bound by HBM too: K + 1 rows
// read per token, K written.  2,048 tokens, top-10 of 2560: 231 MB in 35 us
// (6.5 TB/s); 8,192 with the rows' gradient: 1,762 MB in 315 us (5.6 TB/s;
// torch's copy of 1 GB reaches 5.3).
#include "internal.h"
#include "layer_ops.h"
#include "wave.cuh"

#include <hip/hip_runtime.h>

#include <type_traits>

namespace moe {

namespace {

constexpr int kCombineThreads = 256;   // one float4 of one token per thread, over the flat range
constexpr int kCombineBatch = 16;      // slots whose loads are issued together (all of top-10)

constexpr int kBackwardRows = 8;       // rows of a token that one wave of the gradient takes at most
constexpr int kBackwardFewJobs = 2048; // fewer (token, rows) jobs share their columns over four waves
                                       // (at 4,096 jobs: 38.1 us shared, 34.4 not)

typedef float f32x4 __attribute__((ext_vector_type(4)));

template <bool STREAM>
__device__ __forceinline__ f32x4 load4(const f32x4 *p) {
    if constexpr (STREAM) return __builtin_nontemporal_load(p);
    else return *p;
}

template <bool STREAM>
__global__ __launch_bounds__(kCombineThreads) void combine_kernel(const float *dm, const float *w,
                                                                  float *out, int topk, int h4,
                                                                  long long n4) {
    // one float4 of one token per thread over the flat (token, float4) range
    const long long g = (long long)blockIdx.x * kCombineThreads + threadIdx.x;
    if (g >= n4) return;
    const int t = int(g / h4);
    const int c = int(g - (long long)t * h4);
    const f32x4 *src = reinterpret_cast<const f32x4 *>(dm) + size_t(t) * topk * h4 + c;
    const float *wt = w + size_t(t) * topk;
    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int k0 = 0; k0 < topk; k0 += kCombineBatch) {
        f32x4 d[kCombineBatch];
        float wk[kCombineBatch];
#pragma unroll
        for (int j = 0; j < kCombineBatch; ++j)
            if (k0 + j < topk) {
                d[j] = load4<STREAM>(src + size_t(k0 + j) * h4);
                wk[j] = wt[k0 + j];
            }
#pragma unroll
        for (int j = 0; j < kCombineBatch; ++j)
            if (k0 + j < topk) {
                acc.x = __builtin_fmaf(wk[j], d[j].x, acc.x);
                acc.y = __builtin_fmaf(wk[j], d[j].y, acc.y);
                acc.z = __builtin_fmaf(wk[j], d[j].z, acc.z);
                acc.w = __builtin_fmaf(wk[j], d[j].w, acc.w);
            }
    }
    f32x4 *dst = reinterpret_cast<f32x4 *>(out) + size_t(t) * h4 + c;
    if constexpr (STREAM) __builtin_nontemporal_store(acc, dst);
    else *dst = acc;
}

// NB rows of one token per wave (all of them clamped to the last, so that their
// loads are in flight together): the output gradient's chunk stays in registers
// while the rows' chunks pass; the NB sums are joined over the lanes at the end.
// A lane reads its part of a row before it writes it, so ddm may be dm itself.
// SPLIT: few tokens, the four waves of a workgroup share the columns of the
// same rows and are added through LDS.
template <int NB, bool DW, bool DDM, bool SPLIT, bool STREAM>
__global__ __launch_bounds__(kCombineThreads) void combine_backward_kernel(const float *dm, const float *w,
                                                                           const float *dout, int tokens,
                                                                           int topk, int h4, int groups,
                                                                           float *dw, float *ddm) {
    __shared__ float red[SPLIT ? 4 : 1][NB];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t job = SPLIT ? int64_t(blockIdx.x) : int64_t(blockIdx.x) * 4 + wave;
    if (job >= int64_t(tokens) * groups) return;
    const int64_t t = job / groups;
    const int k0 = int(job % groups) * NB;
    const f32x4 *g4 = reinterpret_cast<const f32x4 *>(dout) + t * h4;
    int64_t row[NB];
    float wk[NB], acc[NB];
#pragma unroll
    for (int j = 0; j < NB; ++j) {
        row[j] = t * topk + min(k0 + j, topk - 1);
        if constexpr (DDM) wk[j] = w[row[j]];
        acc[j] = 0.0f;
    }
    const int step = SPLIT ? 256 : 64;
#pragma unroll 2
    for (int c = SPLIT ? wave * 64 + lane : lane; c < h4; c += step) {
        const f32x4 g = g4[c];
        f32x4 d[NB];
        if constexpr (DW)
#pragma unroll
            for (int j = 0; j < NB; ++j)
                d[j] = load4<STREAM>(reinterpret_cast<const f32x4 *>(dm) + row[j] * h4 + c);
#pragma unroll
        for (int j = 0; j < NB; ++j) {
            if constexpr (DW) {
                acc[j] = __builtin_fmaf(g.x, d[j].x, acc[j]);
                acc[j] = __builtin_fmaf(g.y, d[j].y, acc[j]);
                acc[j] = __builtin_fmaf(g.z, d[j].z, acc[j]);
                acc[j] = __builtin_fmaf(g.w, d[j].w, acc[j]);
            }
            if constexpr (DDM) {
                f32x4 *dst = reinterpret_cast<f32x4 *>(ddm) + row[j] * h4 + c;
                const f32x4 v = {wk[j] * g.x, wk[j] * g.y, wk[j] * g.z, wk[j] * g.w};
                if (k0 + j < topk) {
                    if constexpr (STREAM) __builtin_nontemporal_store(v, dst);
                    else *dst = v;
                }
            }
        }
    }
    if constexpr (DW) {
        float mine = 0.0f;
#pragma unroll
        for (int j = 0; j < NB; ++j) {
            const float s = wave_sum(acc[j]);
            mine = lane == j ? s : mine;
        }
        if constexpr (SPLIT) {
            if (lane < NB) red[wave][lane] = mine;
            __syncthreads();
            if (wave == 0 && lane < NB) mine = (red[0][lane] + red[1][lane]) + (red[2][lane] + red[3][lane]);
        }
        if ((!SPLIT || wave == 0) && lane < NB && k0 + lane < topk) dw[t * topk + k0 + lane] = mine;
    }
}

}  // namespace

hipError_t launch_combine_backward(const float *dm, const float *w, const float *dout, int tokens,
                                   int topk, int hidden, float *dw, float *ddm, hipStream_t stream) {
    const int h4 = hidden / 4;
    // as few groups of at most kBackwardRows rows as there are, of equal size
    const int groups = (topk + kBackwardRows - 1) / kBackwardRows;
    const int nb = (topk + groups - 1) / groups;
    const int64_t jobs = int64_t(tokens) * groups;
    const bool split = jobs < kBackwardFewJobs;
    // rows that do not fit the L2s (8 x 4 MB) pass them by.  Top-10 of 2560, dw
    // alone, normal / past the caches: 26 MB 4.2 / 4.7 us read again at once and
    // 7.1 / 7.2 from memory; 52 MB 10.8 / 9.1 and 12.4 / 11.8; 210 MB 34.4 / 34.5
    // and 41.2 / 35.8.
    const bool big = size_t(tokens) * size_t(topk) * size_t(hidden) * 4u > (size_t(32) << 20);
    const dim3 grid(unsigned(split ? jobs : (jobs + 3) / 4)), block(kCombineThreads);
    auto go = [&](auto NB, auto DW, auto DDM, auto SPLIT, auto STREAM) {
        hipLaunchKernelGGL((combine_backward_kernel<NB.value, DW.value, DDM.value, SPLIT.value, STREAM.value>), grid,
                           block, 0, stream, dm, w, dout, tokens, topk, h4, groups, dw, ddm);
        return hipGetLastError();
    };
    auto flag = [](bool b, auto f) { return b ? f(std::true_type{}) : f(std::false_type{}); };
    auto with = [&](auto NB) {
        return flag(split, [&](auto SPLIT) {
            return flag(big && !split, [&](auto STREAM) {
                if (dw && ddm) return go(NB, std::true_type{}, std::true_type{}, SPLIT, STREAM);
                if (dw) return go(NB, std::true_type{}, std::false_type{}, SPLIT, STREAM);
                return go(NB, std::false_type{}, std::true_type{}, SPLIT, STREAM);
            });
        });
    };
    switch (nb) {
        case 1: return with(std::integral_constant<int, 1>{});
        case 2: return with(std::integral_constant<int, 2>{});
        case 3: return with(std::integral_constant<int, 3>{});
        case 4: return with(std::integral_constant<int, 4>{});
        case 5: return with(std::integral_constant<int, 5>{});
        case 6: return with(std::integral_constant<int, 6>{});
        case 7: return with(std::integral_constant<int, 7>{});
        default: return with(std::integral_constant<int, 8>{});
    }
}

hipError_t launch_combine(const float *dm, const float *w, int tokens, int topk, int hidden,
                          float *out, hipStream_t stream) {
    if (tokens <= 0 || hidden <= 0) return hipSuccess;
    const int h4 = hidden / 4;
    const long long n4 = (long long)tokens * h4;
    const dim3 grid(unsigned((n4 + kCombineThreads - 1) / kCombineThreads)), block(kCombineThreads);
    const size_t dm_bytes = size_t(tokens) * size_t(topk) * size_t(hidden) * 4u;
    if (dm_bytes > (size_t(256) << 20))
        hipLaunchKernelGGL(combine_kernel<true>, grid, block, 0, stream, dm, w, out, topk, h4, n4);
    else
        hipLaunchKernelGGL(combine_kernel<false>, grid, block, 0, stream, dm, w, out, topk, h4, n4);
    return hipGetLastError();
}

}  // namespace moe
