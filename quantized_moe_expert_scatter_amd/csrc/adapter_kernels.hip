// adapter_kernels.hip -- low-rank adapters of many requests beside a shared
// projection: out[t] = base[t] + scale[i] * b[i] * (a[i] * x[t]), i = ids[t].
//
// Two launches: the rows' low-rank values h = a[i] * x[t] (fp32, in the
// workspace), then the update of the output rows.
#include "layer_ops.h"
#include "wave.cuh"

#include <hip/hip_runtime.h>

#include <type_traits>

namespace moe {

namespace {

constexpr int kThreads = 256;

// Eight elements of a row, 16-byte aligned.
template <int DT>
__device__ __forceinline__ void load8(const void *p, int64_t at, float (&f)[8]) {
    using T = typename Elem<DT>::T;
    struct alignas(16) Run { T e[8]; };
    const Run r = *reinterpret_cast<const Run *>(static_cast<const T *>(p) + at);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = to_float<DT>(r.e[j]);
}

__device__ __forceinline__ int adapter_of(const AdapterArgs &g, int64_t t) {
    const int i = g.ids[t];
    return i >= 0 && i < g.n_adapter ? i : -1;
}
__device__ __forceinline__ int rank_of(const AdapterArgs &g, int i) {
    return g.ranks ? min(max(g.ranks[i], 0), g.rank) : g.rank;
}

// One wave per (row, rank row): their dot over n_in.
template <int XT, int WT>
__global__ __launch_bounds__(kThreads) void adapter_down_kernel(AdapterArgs g) {
    const int lane = threadIdx.x & 63;
    const int64_t waves = int64_t(gridDim.x) * (kThreads / 64);
    for (int64_t job = int64_t(blockIdx.x) * (kThreads / 64) + (threadIdx.x >> 6);
         job < int64_t(g.tokens) * g.rank; job += waves) {
        const int64_t t = job / g.rank;
        const int r = int(job % g.rank);
        const int i = adapter_of(g, t);
        if (i < 0 || r >= rank_of(g, i)) continue;
        float sum = 0.0f;
        for (int k = lane * 8; k < g.n_in; k += 512) {
            float x[8], a[8];
            load8<XT>(g.x, t * g.ldx + k, x);
            load8<WT>(g.a, (int64_t(i) * g.rank + r) * g.n_in + k, a);
#pragma unroll
            for (int j = 0; j < 8; ++j) sum = __builtin_fmaf(x[j], a[j], sum);
        }
        sum = wave_sum(sum);
        if (lane == 0) g.ws[job] = sum;
    }
}

// One thread per output element.
template <int XT, int WT>
__global__ __launch_bounds__(kThreads) void adapter_up_kernel(AdapterArgs g) {
    using T = typename Elem<XT>::T;
    const int64_t threads = int64_t(gridDim.x) * kThreads;
    for (int64_t job = int64_t(blockIdx.x) * kThreads + threadIdx.x; job < int64_t(g.tokens) * g.n_out;
         job += threads) {
        const int64_t t = job / g.n_out;
        const int n = int(job % g.n_out);
        const T base = static_cast<const T *>(g.base)[t * g.ldb + n];
        T *out = static_cast<T *>(g.out) + t * g.ldo + n;
        const int i = adapter_of(g, t);
        if (i < 0) {
            if (g.out != g.base) *out = base;
            continue;
        }
        const int rank = rank_of(g, i);
        float sum = 0.0f;
        for (int r = 0; r < rank; r += 8) {
            float b[8];
            load8<WT>(g.b, (int64_t(i) * g.n_out + n) * g.rank + r, b);
            for (int j = 0; j < 8 && r + j < rank; ++j)
                sum = __builtin_fmaf(g.ws[t * g.rank + r + j], b[j], sum);
        }
        *out = from_float<XT>(__builtin_fmaf(g.scale[i], sum, to_float<XT>(base)));
    }
}

template <class F>
hipError_t by_types(const AdapterArgs &g, F f) {
    using F32 = std::integral_constant<int, kF32>;
    using B16 = std::integral_constant<int, kBF16>;
    using H16 = std::integral_constant<int, kF16>;
    if (g.dtype == kF32) return g.wtype == kBF16 ? f(F32{}, B16{}) : f(F32{}, H16{});
    return g.wtype == kBF16 ? f(B16{}, B16{}) : f(H16{}, H16{});
}

}  // namespace

hipError_t launch_adapters(const AdapterArgs &g, hipStream_t stream) {
    return by_types(g, [&](auto XT, auto WT) {
        auto groups = [](int64_t n) { return dim3(unsigned(n < 65536 ? n : 65536)); };
        hipLaunchKernelGGL((adapter_down_kernel<XT.value, WT.value>),
                           groups((int64_t(g.tokens) * g.rank + 3) / 4), dim3(kThreads), 0, stream, g);
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
        hipLaunchKernelGGL((adapter_up_kernel<XT.value, WT.value>),
                           groups((int64_t(g.tokens) * g.n_out + kThreads - 1) / kThreads), dim3(kThreads),
                           0, stream, g);
        return hipGetLastError();
    });
}

}  // namespace moe
