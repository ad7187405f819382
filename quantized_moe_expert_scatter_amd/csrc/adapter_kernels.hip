// adapter_kernels.hip -- low-rank adapters of many requests beside a shared
// projection: out[t] = base[t] + scale[i] * b[i] * (a[i] * x[t]), i = ids[t].
//
// Few rows take one launch: a workgroup has one row and a slice of its
// outputs, and computes the row's low-rank values h = a[i] * x[t] itself.
// More rows take two: the rows' h (fp32, in the workspace), then the update of
// the output rows, by tiles of 16 rows, or of 64 in long batches.
#include "layer_ops.h"
#include "wave.cuh"

#include <hip/hip_runtime.h>

#include <type_traits>

namespace moe {

namespace {

constexpr int kThreads = 256;
// The single launch computes a row's h in each of its output slices, so it is
// taken while tokens * rank * slices is small.  Measured with fp32 rows, one
// launch / two, 2560 -> 2560 (3 slices):
//               one adapter                         48 adapters in any order
//   rank  16    1 row 4.4 / 8.3, 128 7.1 / 9.2      16 rows 4.7 / 22.6, 128 8.4 / 17.3
//   rank  32    1 row 5.8 / 8.6, 128 10.0 / 9.6     16 rows 6.1 / 20.5, 128 14.8 / 18.1
//   rank  64    1 row 10.3 / 9.8, 64 11.3 / 10.8    16 rows 10.7 / 29.0, 64 16.6 / 25.6
//   rank 128    1 row 17.3 / 12.3, 16 17.8 / 13.3   16 rows 24.6 / 41.9
//   rank 256    1 row 28.6 / 16.9, 16 30.2 / 18.1   16 rows 42.0 / 66.0
// and past the rule: rank 16, 256 rows in one and 257 in two 9.3 / 9.2 and 12.4 /
// 20.1, rank 64, 128 rows 20.5 / 10.8 and 29.0 / 23.8.
// The rule does not weigh n_in, and is not the best of both where few rows of
// one adapter meet a high rank or a long contraction (n_in 16384: rank 16 1 row
// 14.1 / 11.8, 16 rows in any order 15.0 / 36.3; rank 256 132 / 22 and 139 / 86).
constexpr int kFewRows = 256;
constexpr int kFewValues = 12288;

// Eight elements of a row, 16-byte aligned.
template <int DT>
__device__ __forceinline__ void load8(const void *p, int64_t at, float (&f)[8]) {
    using T = typename Elem<DT>::T;
    struct alignas(16) Run { T e[8]; };
    const Run r = *reinterpret_cast<const Run *>(static_cast<const T *>(p) + at);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = to_float<DT>(r.e[j]);
}

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// 16 bytes that are used once: past the caches.
template <class R>
__device__ __forceinline__ R stream_load(const void *p) {
    return __builtin_bit_cast(R, __builtin_nontemporal_load(static_cast<const u32x4 *>(p)));
}
template <class R>
__device__ __forceinline__ void stream_store(void *p, const R &r) {
    __builtin_nontemporal_store(__builtin_bit_cast(u32x4, r), static_cast<u32x4 *>(p));
}

__device__ __forceinline__ int adapter_of(const AdapterArgs &g, int64_t t) {
    const int i = g.ids[t];
    return i >= 0 && i < g.n_adapter ? i : -1;
}
__device__ __forceinline__ int rank_of(const AdapterArgs &g, int i) {
    return g.ranks ? min(max(g.ranks[i], 0), g.rank) : g.rank;
}

constexpr int kRowThreads = 1024;
constexpr int kRowWaves = kRowThreads / 64;

// One workgroup per (row, 1024 outputs).  h: each wave takes every 16th rank
// row, RW of them at most, and passes over the row of x once; the outputs:
// one per thread, its row of b (16-byte runs) against h from LDS.  Latency: one
// row of 2560 -> 2560 takes 4.4 us at rank 16, 10.4 at rank 64; 48 rows of 32
// adapters, rank 16, 1280 outputs, 5.1.
template <int XT, int WT, int RW>
__global__ __launch_bounds__(kRowThreads) void adapter_row_kernel(AdapterArgs g, int slices) {
    using T = typename Elem<XT>::T;
    __shared__ float h[RW * kRowWaves];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t t = blockIdx.x / slices;
    const int n = int(blockIdx.x % slices) * kRowThreads + int(threadIdx.x);
    const bool live = n < g.n_out;
    const int i = adapter_of(g, t);
    T *out = static_cast<T *>(g.out) + t * g.ldo + n;
    const T base = live ? static_cast<const T *>(g.base)[t * g.ldb + n] : T(0);
    if (i < 0) {
        if (live && g.out != g.base) *out = base;
        return;
    }
    const int rank = rank_of(g, i);
    // every address is clamped instead of skipped, so that the loads of several
    // rank rows are in flight together; values past the ends are 0 or not used
    constexpr int kGroup = RW < 2 ? RW : 2;
    const int mine = (rank - wave + kRowWaves - 1) / kRowWaves;     // rank rows of this wave
    // the output's row of b, on its way while h is computed
    constexpr int kRuns = RW * kRowWaves / 8 < 8 ? RW * kRowWaves / 8 : 8;
    const uint16_t *b_row = static_cast<const uint16_t *>(g.b) + (int64_t(i) * g.n_out + min(n, g.n_out - 1)) * g.rank;
    u32x4 b_run[kRuns];
#pragma unroll
    for (int q = 0; q < kRuns; ++q)
        b_run[q] = *reinterpret_cast<const u32x4 *>(b_row + min(q * 8, g.rank - 8));
    const uint16_t *mat = static_cast<const uint16_t *>(g.a) + int64_t(i) * g.rank * g.n_in;
    float sum[RW];
#pragma unroll
    for (int q = 0; q < RW; ++q) sum[q] = 0.0f;
#pragma unroll (RW < 4 ? 5 / RW : 2)
    for (int k = lane * 8; k - lane * 8 < g.n_in; k += 512) {
        const int kc = min(k, g.n_in - 8);
        float x[8];
        load8<XT>(g.x, t * g.ldx + kc, x);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = k < g.n_in ? x[j] : 0.0f;
#pragma unroll
        for (int q0 = 0; q0 < RW; q0 += kGroup)
            if (q0 < mine) {
                float a[kGroup][8];
#pragma unroll
                for (int q = 0; q < kGroup; ++q)
                    load8<WT>(mat, int64_t(min((q0 + q) * kRowWaves + wave, rank - 1)) * g.n_in + kc, a[q]);
#pragma unroll
                for (int q = 0; q < kGroup; ++q)
#pragma unroll
                    for (int j = 0; j < 8; ++j) sum[q0 + q] = __builtin_fmaf(x[j], a[q][j], sum[q0 + q]);
            }
    }
#pragma unroll
    for (int q = 0; q < RW; ++q) {
        const float s = wave_sum(sum[q]);
        if (lane == 0) h[q * kRowWaves + wave] = s;
    }
    __syncthreads();
    if (!live) return;
    float acc = 0.0f;
    auto add = [&](u32x4 run, int r) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint16_t e = uint16_t(run[j / 2] >> (j % 2 * 16));
            if (r + j < rank) acc = __builtin_fmaf(h[r + j], to_float<WT>(e), acc);
        }
    };
#pragma unroll
    for (int q = 0; q < kRuns; ++q)
        if (q * 8 < rank) add(b_run[q], q * 8);
    if constexpr (RW * kRowWaves > kRuns * 8)
#pragma unroll 4
        for (int r = kRuns * 8; r < rank; r += 8) add(*reinterpret_cast<const u32x4 *>(b_row + r), r);
    *out = from_float<XT>(__builtin_fmaf(g.scale[i], acc, to_float<XT>(base)));
}

// Eight fp32 values as N bf16 vectors whose sum they are: each takes the next
// eight bits of the mantissa (by truncation, so the rest is exact), three hold
// all 24.  The matrix unit then multiplies fp32 values by bf16 ones with fp32
// accuracy in three passes.  An infinity becomes NaN.
template <int N>
__device__ __forceinline__ void split(const float (&f)[8], u32x4 (&p)[N]) {
    float rest[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) rest[j] = f[j];
#pragma unroll
    for (int q = 0; q < N; ++q) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            p[q][j] = __builtin_amdgcn_perm(__float_as_uint(rest[2 * j + 1]), __float_as_uint(rest[2 * j]),
                                            0x07060302u);
        if (q + 1 < N)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                rest[j] = rest[j] - __uint_as_float(__float_as_uint(rest[j]) & 0xffff0000u);
    }
}

__device__ __forceinline__ f32x4 mfma_bf16(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c,
                                                   0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma_f16(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0,
                                                  0, 0);
}

// A 16-byte run of an adapter matrix as bf16 vectors: itself, or fp16 in two
// (11 bits in 8 + 3).
template <int WT> struct Weight {
    static constexpr int kParts = WT == kBF16 ? 1 : 2;
    u32x4 p[kParts];
    __device__ __forceinline__ void set(u32x4 raw) {
        if constexpr (WT == kBF16) {
            p[0] = raw;
        } else {
            const f16x8 h = __builtin_bit_cast(f16x8, raw);
            float f[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = float(h[j]);
            split<2>(f, p);
        }
    }
};

// c += w * v over all pairs of bf16 parts, the smallest first.  (That of the
// second part of w and the third of v reaches 2^-22.1 of the whole, always with
// its sign; 16,384 fp32 rows at rank 64 with fp16 matrices take 132 us with it and
// 129 without.)
template <int WP, int VP>
__device__ __forceinline__ f32x4 mfma_parts(const u32x4 (&w)[WP], const u32x4 (&v)[VP], f32x4 c) {
#pragma unroll
    for (int s = WP + VP - 2; s >= 0; --s)
#pragma unroll
        for (int i = 0; i < WP; ++i)
            if (s - i >= 0 && s - i < VP) c = mfma_bf16(w[i], v[s - i], c);
    return c;
}

// Which rows a tile has.  Up to kSortRows rows (a batch of new tokens, every
// row its own adapter, where a tile of 16 rows would take up to 16 passes) the
// tiles take the rows by adapter, unless the ids change no more often than
// there are tiles: each workgroup counts the rows per adapter, which gives
// every adapter its places, and for the few adapters that have places in its
// tile a wave walks the ids and numbers their rows in order.  Every workgroup
// comes to the same order, and a row's result does not depend on its tile.
//   fp32 rows of 48 adapters in any order, rank 64 of 2560: 512 rows 37 us
// against 69 in tiles of neighbours, 1,024 rows 44 against 111; rows of one
// adapter, which pay the look at the ids, 13.3 against 13.0 and 16.3 against
// 15.2.
constexpr int kSortRows = 1024;
constexpr int kSortSets = 1024;                   // adapters that are counted, at most
struct TileIds {
    int row[32];                                  // the tile's rows
    int key[kSortRows];                           // adapter by row (n_adapter: none)
    int start[kSortSets];                         // rows of an adapter, then its first place
    int sums[kThreads / 64];
    int found, list[32];                          // adapters with places in the tile
};
__device__ __forceinline__ void tile_rows(const AdapterArgs &g, int64_t first, int rows, int tiles, TileIds &s) {
    constexpr int kEach = 4;                      // rows and adapters of a thread
    static_assert(kSortRows == kEach * kThreads && kSortSets == kEach * kThreads, "one run of ids per thread");
    const int i = int(threadIdx.x), lane = i & 63, wave = i >> 6, t = i * kEach;
    int key[kEach];
    bool sorted = false;
    if (i < rows) s.row[i] = int(min(first + i, int64_t(g.tokens) - 1));
    if (g.tokens <= kSortRows && g.n_adapter < kSortSets) {
        int4 v = {-1, -1, -1, -1};
        if (t + kEach <= g.tokens) {
            v = *reinterpret_cast<const int4 *>(g.ids + t);
        } else {
            if (t < g.tokens) v.x = g.ids[t];
            if (t + 1 < g.tokens) v.y = g.ids[t + 1];
            if (t + 2 < g.tokens) v.z = g.ids[t + 2];
        }
        const int before = t > 0 && t < g.tokens ? g.ids[t - 1] : v.x;
        const int id[kEach] = {v.x, v.y, v.z, v.w};
        int changes = 0;
#pragma unroll
        for (int q = 0; q < kEach; ++q) {
            changes += __popcll(__ballot(t + q < g.tokens && id[q] != (q > 0 ? id[q - 1] : before)));
            key[q] = id[q] >= 0 && id[q] < g.n_adapter ? id[q] : g.n_adapter;
        }
        if (lane == 0) s.sums[wave] = changes;
        __syncthreads();
        changes = 0;
        for (int w = 0; w < kThreads / 64; ++w) changes += s.sums[w];
        sorted = changes > tiles;
    }
    __syncthreads();
    if (!sorted) return;
#pragma unroll
    for (int q = 0; q < kEach; ++q) {
        s.key[t + q] = key[q];
        s.start[t + q] = 0;
    }
    if (i == 0) s.found = 0;
    __syncthreads();
#pragma unroll
    for (int q = 0; q < kEach; ++q)
        if (t + q < g.tokens) atomicAdd(&s.start[key[q]], 1);
    __syncthreads();
    // places: a prefix sum over the adapters, kEach of them per thread
    int count[kEach], sum = 0;
#pragma unroll
    for (int q = 0; q < kEach; ++q) {
        count[q] = s.start[i * kEach + q];
        sum += count[q];
    }
    int scan = sum;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int v = __shfl_up(scan, d);
        scan += lane >= d ? v : 0;
    }
    if (lane == 63) s.sums[wave] = scan;
    __syncthreads();
    int at = scan - sum;
    for (int w = 0; w < wave; ++w) at += s.sums[w];
#pragma unroll
    for (int q = 0; q < kEach; ++q) {
        s.start[i * kEach + q] = at;
        // at most `rows` adapters have places in the tile
        if (count[q] > 0 && at < first + rows && at + count[q] > first) s.list[atomicAdd(&s.found, 1)] = i * kEach + q;
        at += count[q];
    }
    __syncthreads();
    for (int f = wave; f < s.found; f += kThreads / 64) {
        const int a = s.list[f];
        int place = s.start[a] - int(first);
        for (int t0 = 0; t0 < g.tokens && place < rows; t0 += 64) {
            const bool hit = t0 + lane < g.tokens && s.key[t0 + lane] == a;
            const uint64_t hits = __ballot(hit);
            const int mine = place + __popcll(hits & ((uint64_t(1) << lane) - 1));
            if (hit && mine >= 0 && mine < rows) s.row[mine] = t0 + lane;
            place += __popcll(hits);
        }
    }
    __syncthreads();
}

// The adapters of a tile's rows, the same in every wave: lane l has row l.
struct TileRows {
    int id;               // this lane's row's adapter, -1: none (or no such row)
    uint64_t left;        // rows not handled yet
    __device__ __forceinline__ TileRows(const AdapterArgs &g, const TileIds &s, int count, int lane) {
        id = lane < count ? adapter_of(g, s.row[lane]) : -1;
        left = __ballot(id >= 0);
    }
    __device__ __forceinline__ TileRows(const AdapterArgs &g, int64_t first, int count, int lane) {
        id = lane < count ? adapter_of(g, first + lane) : -1;
        left = __ballot(id >= 0);
    }
    // How many adapters the rows have.
    __device__ __forceinline__ int distinct() const {
        TileRows r = *this;
        int n = 0;
        while (r.next() >= 0) ++n;
        return n;
    }
    // The next adapter of the tile, -1 at the end.
    __device__ __forceinline__ int next() {
        if (left == 0) return -1;
        const int a = __builtin_amdgcn_readlane(id, __ffsll((unsigned long long)left) - 1);
        left &= ~__ballot(id == a);
        return a;
    }
};

// h for a tile of 16 * MR rows, 16 * NR rank rows and a slice of n_in: the
// four waves take 32 values in turn and are added through LDS.  A tile with
// rows of several adapters passes over x once for each; gridDim.z workgroups
// share those passes.  The matrix unit's rows are rank rows, its columns rows
// of x, so whatever a row holds stays in its column.
//   a and x are loaded row segment by row segment, neighbouring lanes next to
// each other, and turn through the wave's part of LDS into the matrix unit's
// layout.  (Loaded in that layout, neighbouring lanes are in different rows and
// the address unit takes 64 accesses for a load instead of 16; fp32 x came down
// from 59 to 44 us by this at 16,384 rows of 2560 and rank 64, a from 6.8 to 5.4
// us at 2,047 fp16 rows and rank 24.)  At 16,384 rows it reads x at 4.1 TB/s:
// 30 us with a's loads left out, 33 with x's, of 42; more rows or workgroups in
// flight, deeper prefetch and other shares of the contraction are level.
template <int XT, int WT, int NR, int MR>
__global__ __launch_bounds__(kThreads) void adapter_down_kernel(AdapterArgs g, AdapterSplit s) {
    constexpr int kXP = XT == kF32 ? 3 : 1;
    using T = typename Elem<XT>::T;
    constexpr int kLanes = XT == kF32 ? 8 : 4;           // lanes of a row's 32 values
    constexpr int kLoads = 16 * MR * kLanes / 64;        // 16-byte loads of x per lane and step
    constexpr int kRun = 32 / kLanes;
    // rows of 32 values and 16 bytes: 16 lanes reading 16 bytes of 16 rows meet no bank twice
    struct Turn {
        uint16_t w[16 * NR][32 + 8];
        T x[16 * MR][32 + 16 / sizeof(T)];
    };
    __shared__ union {
        f32x4 red[4][NR][MR][64];
        Turn turn[4];
    } lds;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t first = int64_t(blockIdx.x / s.splits) * (16 * MR);
    const int plane = int(blockIdx.x % s.splits);
    const int r0 = int(blockIdx.y) * 16 * NR;
    const int k0 = plane * s.slice + wave * 32 + (lane & 3) * 8;          // of a, as loaded
    const int k1 = min(g.n_in, (plane + 1) * s.slice);
    __shared__ TileIds ids;
    tile_rows(g, first, 16 * MR, s.tiles, ids);
    const int count = int(min(int64_t(16 * MR), g.tokens - first));      // rows of the tile
    TileRows rows(g, ids, count, lane);
    const int kx = plane * s.slice + wave * 32 + lane % kLanes * kRun;
    const T *x_at[kLoads];
#pragma unroll
    for (int m = 0; m < kLoads; ++m)
        x_at[m] = static_cast<const T *>(g.x) +
                  int64_t(ids.row[min(m * (64 / kLanes) + lane / kLanes, count - 1)]) * g.ldx;
    Turn &turn = lds.turn[wave];
    for (int pass = 0, a; (a = rows.next()) >= 0; ++pass) {
        if (pass % int(gridDim.z) != int(blockIdx.z)) continue;
        if (r0 > 0 && r0 >= rank_of(g, a)) continue;
        const uint16_t *mat = static_cast<const uint16_t *>(g.a) + int64_t(a) * g.rank * g.n_in;
        const uint16_t *a_row[NR];
#pragma unroll
        for (int n = 0; n < NR; ++n)
            a_row[n] = mat + int64_t(min(r0 + n * 16 + (lane >> 2), g.rank - 1)) * g.n_in;
        f32x4 acc[NR][MR];
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
            for (int m = 0; m < MR; ++m) acc[n][m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        // raw loads of one step, in flight while the step before is multiplied
        struct Step {
            u32x4 w[NR], x[kLoads];
        };
        auto load = [&](Step &q, int step) {
            // past the slice: some values, not used
            const int k = k0 + step * kAdapterStep, kc = k < k1 ? k : 0;
            const int kv = kx + step * kAdapterStep, kvc = kv < k1 ? kv : 0;
#pragma unroll
            for (int n = 0; n < NR; ++n) q.w[n] = *reinterpret_cast<const u32x4 *>(a_row[n] + kc);
#pragma unroll
            for (int m = 0; m < kLoads; ++m) q.x[m] = *reinterpret_cast<const u32x4 *>(x_at[m] + kvc);
        };
        auto multiply = [&](const Step &q, int step) {
            const bool in = k0 + step * kAdapterStep < k1, x_in = kx + step * kAdapterStep < k1;
            const u32x4 zero = {0, 0, 0, 0};
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int n = 0; n < NR; ++n)
                *reinterpret_cast<u32x4 *>(&turn.w[n * 16 + (lane >> 2)][(lane & 3) * 8]) = in ? q.w[n] : zero;
#pragma unroll
            for (int m = 0; m < kLoads; ++m)
                *reinterpret_cast<u32x4 *>(&turn.x[m * (64 / kLanes) + lane / kLanes][lane % kLanes * kRun]) =
                    x_in ? q.x[m] : zero;
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
            u32x4 v[MR][kXP];
#pragma unroll
            for (int m = 0; m < MR; ++m) {
                const T *src = &turn.x[m * 16 + (lane & 15)][(lane >> 4) * 8];
                if constexpr (XT == kF32) {
                    float f[8];
                    *reinterpret_cast<f32x4 *>(f) = *reinterpret_cast<const f32x4 *>(src);
                    *reinterpret_cast<f32x4 *>(f + 4) = *reinterpret_cast<const f32x4 *>(src + 4);
                    split<3>(f, v[m]);
                } else {
                    v[m][0] = *reinterpret_cast<const u32x4 *>(src);
                }
            }
#pragma unroll
            for (int n = 0; n < NR; ++n) {
                const u32x4 raw = *reinterpret_cast<const u32x4 *>(&turn.w[n * 16 + (lane & 15)][(lane >> 4) * 8]);
                if constexpr (XT == kF16) {
#pragma unroll
                    for (int m = 0; m < MR; ++m) acc[n][m] = mfma_f16(raw, v[m][0], acc[n][m]);
                } else {
                    Weight<WT> w;
                    w.set(raw);
#pragma unroll
                    for (int m = 0; m < MR; ++m) acc[n][m] = mfma_parts(w.p, v[m], acc[n][m]);
                }
            }
        };
        Step one, two;
        load(one, 0);
        const int steps = (k1 - (k0 - (lane & 3) * 8) + kAdapterStep - 1) / kAdapterStep;
        for (int q = 0; q < steps; q += 2) {
            load(two, q + 1);
            multiply(one, q);
            load(one, q + 2);
            multiply(two, q + 1);
        }
        __syncthreads();            // the union: every wave is done with its values of x
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
            for (int m = 0; m < MR; ++m) lds.red[wave][n][m][lane] = acc[n][m];
        __syncthreads();
        for (int c = threadIdx.x; c < NR * MR * 64; c += kThreads) {
            const int n = c / (MR * 64), m = c / 64 % MR, l = c & 63;
            const f32x4 h = (lds.red[0][n][m][l] + lds.red[1][n][m][l]) +
                            (lds.red[2][n][m][l] + lds.red[3][n][m][l]);
            const int row = m * 16 + (l & 15), r = r0 + n * 16 + (l >> 4) * 4;
            if (r < g.rank && row < count && adapter_of(g, ids.row[row]) == a)
                *reinterpret_cast<f32x4 *>(g.ws + (int64_t(plane) * g.tokens + ids.row[row]) * g.rank + r) = h;
        }
        __syncthreads();
    }
}

// The update of a tile of 16 rows, 256 outputs at a time (64 per wave).  h, its
// planes added, stands in LDS, all rows of the tile at once where the rank fits
// (its loads then wait for nothing else); the matrix unit's rows are outputs,
// its columns rows of the tile, and a pass's results are taken from the columns
// whose rows have its adapter.  The 16 x 64 results pass through LDS so that
// base and out move in whole row segments: 256 bytes of a row per 16 lanes
// reach 6.2 TB/s in a copy of 16,384 fp32 rows of 2560 past the caches, the 64
// that the matrix unit's layout gives 4.6.  KB: blocks of 32 rank values whose part of b is held in registers
// (0: any rank, 64 values at a time).
//   2,047 fp16 rows of 2560 at rank 24: 10.8 us for 21 MB.  Loading the first
// part of b with base and h, or all planes of h at once, was slower, b turned
// through LDS as in the other kernel level (11.6-12.3 and 11.1 where this took
// 10.5, with two parts of h).
constexpr int kUpRank = 64;          // rank values of h in LDS at a time
constexpr int kUpStride = kUpRank + 4;
// Parts of h: all of its fp32, for 16-bit rows too, where the third shows only if
// base takes most of the update away (2,047 bf16 rows at rank 64 24.0 us with two
// parts, 24.9 with three; 2,047 fp16 rows at rank 24 16.9 and 17.1).
constexpr int kHP = 3;

template <int XT, int WT, int KB>
__global__ __launch_bounds__(kThreads) void adapter_up_kernel(AdapterArgs g, AdapterSplit s, int tiles, int slices,
                                                              int per) {
    using T = typename Elem<XT>::T;
    constexpr int kRun = XT == kF32 ? 4 : 8;     // 16 bytes of a row
    constexpr int kLanes = 64 / kRun;            // lanes of a row's 64 outputs
    constexpr int kRows = 64 / kLanes;           // rows of one access
    constexpr int kParts = 16 / kRows;           // accesses of 16 rows
    struct alignas(16) Run { T e[kRun]; };
    __shared__ alignas(16) float h[16][kUpStride];
    __shared__ alignas(16) float turn[4][16][64 + 4];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t first = int64_t(blockIdx.x / slices) * 16;
    const int n_begin = int(blockIdx.x % slices) * per * kThreads;
    const int n_end = min(g.n_out, n_begin + per * kThreads);
    const T *base = static_cast<const T *>(g.base);
    T *out = static_cast<T *>(g.out);
    __shared__ TileIds ids;
    tile_rows(g, first, 16, tiles, ids);
    const int count = int(min(int64_t(16), g.tokens - first));      // rows of the tile
    TileRows rows(g, ids, count, lane);
    if (blockIdx.z > 0 && int(blockIdx.z) >= rows.distinct()) return;      // no pass left for it
    // this lane's share of an access: its rows' adapters and its column
    const int col = wave * 64 + lane % kLanes * kRun;
    int id[kParts];
    int64_t row[kParts];
#pragma unroll
    for (int i = 0; i < kParts; ++i) {
        const int r = i * kRows + lane / kLanes;
        id[i] = __shfl(rows.id, r);
        row[i] = ids.row[min(r, count - 1)];
    }
    Run b_run[kParts];
    auto load_base = [&](int n) {
#pragma unroll
        for (int i = 0; i < kParts; ++i)
            b_run[i] = stream_load<Run>(base + row[i] * g.ldb + min(n, g.n_out - kRun));
    };
    auto stage = [&](int b) {
        for (int c = threadIdx.x; c < 16 * (kUpRank / 4); c += kThreads) {
            const int r0 = c / (kUpRank / 4), r = b + c % (kUpRank / 4) * 4;
            if (r >= g.rank) continue;
            const float *src = g.ws + int64_t(ids.row[min(r0, count - 1)]) * g.rank + r;
            const int64_t plane = int64_t(g.tokens) * g.rank;
            f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
            for (int q = 0; q < s.splits; q += 4) {
                f32x4 p[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    p[i] = *reinterpret_cast<const f32x4 *>(src + min(q + i, s.splits - 1) * plane);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (q + i < s.splits) v += p[i];
            }
            *reinterpret_cast<f32x4 *>(&h[r0][r - b]) = v;
        }
    };
    load_base(n_begin + col);
    if constexpr (KB > 0) {
        stage(0);
        __syncthreads();
    }
    // rows without an adapter
    const bool copied = blockIdx.z == 0 && g.out != g.base &&
                        __popcll(rows.left) < count;
    if (copied)
        for (int n = n_begin + col; n < n_end; n += kThreads) {
            if (n > n_begin + col) load_base(n);
#pragma unroll
            for (int i = 0; i < kParts; ++i)
                if (id[i] < 0 && i * kRows + lane / kLanes < count)
                    stream_store(out + row[i] * g.ldo + n, b_run[i]);
        }
    for (int pass = 0, a; (a = rows.next()) >= 0; ++pass) {
        if (pass % int(gridDim.z) != int(blockIdx.z)) continue;
        const int rank = rank_of(g, a);
        const float scale = g.scale[a];
        const uint16_t *mat = static_cast<const uint16_t *>(g.b) + int64_t(a) * g.n_out * g.rank;
        auto load_b = [&](int n0, int j, int k) {
            const int n = min(n0 + wave * 64 + j * 16 + (lane & 15), g.n_out - 1);
            return *reinterpret_cast<const u32x4 *>(mat + int64_t(n) * g.rank +
                                                    min(k + (lane >> 4) * 8, g.rank - 8));
        };
        u32x4 w_run[KB > 0 ? KB : 1][4];
        auto load_weights = [&](int n0) {
            if constexpr (KB > 0)
#pragma unroll
                for (int q = 0; q < KB; ++q)
#pragma unroll
                    for (int j = 0; j < 4; ++j) w_run[q][j] = load_b(n0, j, q * 32);
        };
        load_weights(n_begin);
        if (pass > 0 || copied) load_base(n_begin + col);
        for (int n0 = n_begin; n0 < n_end; n0 += kThreads) {
            f32x4 acc[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            auto multiply = [&](int b, int k, auto weight) {
                u32x4 v[kHP];
                float f[8];
                const float *src = &h[lane & 15][k - b + (lane >> 4) * 8];
                *reinterpret_cast<f32x4 *>(f) = *reinterpret_cast<const f32x4 *>(src);
                *reinterpret_cast<f32x4 *>(f + 4) = *reinterpret_cast<const f32x4 *>(src + 4);
                // values past the rank may be anything, and 0 times that is not 0
                if (k + 32 > rank)
#pragma unroll
                    for (int i = 0; i < 8; ++i) f[i] = k + (lane >> 4) * 8 + i < rank ? f[i] : 0.0f;
                split<kHP>(f, v);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    u32x4 raw = weight(j);
                    if (k + 32 > rank) {
                        // columns past the adapter's rank are not part of it, whatever they hold
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int c = k + (lane >> 4) * 8 + 2 * i;
                            raw[i] = c + 1 < rank ? raw[i] : (c < rank ? raw[i] & 0xffffu : 0u);
                        }
                    }
                    Weight<WT> w;
                    w.set(raw);
                    acc[j] = mfma_parts(w.p, v, acc[j]);
                }
            };
            if constexpr (KB > 0) {
#pragma unroll
                for (int q = 0; q < KB; ++q)
                    if (q * 32 < rank) multiply(0, q * 32, [&](int j) { return w_run[q][j]; });
                if (n0 + kThreads < n_end) load_weights(n0 + kThreads);
            } else {
                for (int b = 0; b < rank; b += kUpRank) {
                    __syncthreads();
                    stage(b);
                    __syncthreads();
                    for (int k = b; k < min(rank, b + kUpRank); k += 32)
                        multiply(b, k, [&](int j) { return load_b(n0, j, k); });
                }
            }
            // results to rows: the wave's own part of LDS
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int j = 0; j < 4; ++j)
                *reinterpret_cast<f32x4 *>(&turn[wave][lane & 15][j * 16 + (lane >> 4) * 4]) = acc[j];
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int i = 0; i < kParts; ++i) {
                const float *src = &turn[wave][i * kRows + lane / kLanes][lane % kLanes * kRun];
                float u[kRun];
#pragma unroll
                for (int c = 0; c < kRun; c += 4)
                    *reinterpret_cast<f32x4 *>(u + c) = *reinterpret_cast<const f32x4 *>(src + c);
                Run r;
#pragma unroll
                for (int c = 0; c < kRun; ++c)
                    r.e[c] = from_float<XT>(__builtin_fmaf(scale, u[c], to_float<XT>(b_run[i].e[c])));
                if (id[i] == a && n0 + col < n_end) stream_store(out + row[i] * g.ldo + n0 + col, r);
            }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            if (n0 + kThreads < n_end) load_base(n0 + kThreads + col);
        }
    }
}

// The same for many rows and ranks up to 64: a workgroup takes 64 rows, a wave
// 16 of them, and 64 outputs at a time.  The block of b is loaded once for the
// four waves, in row order; h stays in registers, split, for all outputs.
//   Bound by base and out: 16,384 fp32 rows of 2560 at rank 64 take 69 us (336
// MB, 4.9 TB/s; the 16-row kernel 89, 32 rows of it 73).  Short stretches of
// outputs are best, 1,024 / 2,048 / 4,096 / 10,240 workgroups 84 / 71 / 69 / 79
// us.  2,047 fp16 rows at rank 24 take 12.4 us against the 16-row kernel's 10.8.
constexpr int kWideGroups = 4096;

template <int XT, int WT, int KB>
__global__ __launch_bounds__(kThreads) void adapter_up_wide_kernel(AdapterArgs g, AdapterSplit s, int slices, int per) {
    using T = typename Elem<XT>::T;
    constexpr int kRun = XT == kF32 ? 4 : 8;     // 16 bytes of a row
    constexpr int kLanes = 64 / kRun;            // lanes of a row's 64 outputs
    constexpr int kRows = 64 / kLanes;           // rows of one access
    constexpr int kParts = 16 / kRows;           // accesses of 16 rows
    constexpr int kChunks = KB * 4;              // 16-byte runs of a row of b
    struct alignas(16) Run { T e[kRun]; };
    __shared__ alignas(16) uint16_t b_block[64][KB * 32 + 8];
    __shared__ alignas(16) float turns[4][16][64 + 4];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    auto &turn = turns[wave];
    const int64_t first = int64_t(blockIdx.x / slices) * 64;
    const int n_begin = int(blockIdx.x % slices) * per * 64;
    const int n_end = min(g.n_out, n_begin + per * 64);
    const T *base = static_cast<const T *>(g.base);
    T *out = static_cast<T *>(g.out);
    const int count = int(min(int64_t(64), g.tokens - first));
    TileRows rows(g, first, count, lane);
    if (blockIdx.z > 0 && int(blockIdx.z) >= rows.distinct()) return;      // no pass left for it
    // this lane's share of an access: its rows' adapters and its column
    const int col = lane % kLanes * kRun;
    int id[kParts];
    int64_t row[kParts];
#pragma unroll
    for (int i = 0; i < kParts; ++i) {
        const int r = wave * 16 + i * kRows + lane / kLanes;
        id[i] = __shfl(rows.id, r);
        row[i] = first + min(r, count - 1);
    }
    Run b_run[kParts];
    auto load_base = [&](int n) {
#pragma unroll
        for (int i = 0; i < kParts; ++i)
            b_run[i] = stream_load<Run>(base + row[i] * g.ldb + min(n, g.n_out - kRun));
    };
    // h of the wave's rows, in the matrix unit's layout: row lane % 16, values
    // (lane / 16) * 8 of each 32; zeros past the rank of the row's own adapter
    u32x4 v[KB][kHP];
    const int mine = __shfl(rows.id, wave * 16 + (lane & 15));
    {
        const int rank = mine >= 0 ? rank_of(g, mine) : 0;
        const float *src = g.ws + (first + min(wave * 16 + (lane & 15), count - 1)) * g.rank;
        const int64_t plane = int64_t(g.tokens) * g.rank;
#pragma unroll
        for (int q = 0; q < KB; ++q) {
            const int k = q * 32 + (lane >> 4) * 8;
            f32x4 f[2] = {};
            for (int p = 0; p < s.splits; ++p)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    f[i] += *reinterpret_cast<const f32x4 *>(src + p * plane + min(k, g.rank - 8) + i * 4);
            float e[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) e[j] = k + j < rank ? f[j / 4][j % 4] : 0.0f;
            split<kHP>(e, v[q]);
        }
    }
    load_base(n_begin + col);
    // rows without an adapter
    const bool copied = blockIdx.z == 0 && g.out != g.base && __popcll(rows.left) < count;
    if (copied)
        for (int n = n_begin + col; n < n_end; n += 64) {
            if (n > n_begin + col) load_base(n);
#pragma unroll
            for (int i = 0; i < kParts; ++i)
                if (id[i] < 0 && wave * 16 + i * kRows + lane / kLanes < count)
                    stream_store(out + row[i] * g.ldo + n, b_run[i]);
        }
    for (int pass = 0, a; (a = rows.next()) >= 0; ++pass) {
        if (pass % int(gridDim.z) != int(blockIdx.z)) continue;
        const int rank = rank_of(g, a);
        const float scale = g.scale[a];
        const uint16_t *mat = static_cast<const uint16_t *>(g.b) + int64_t(a) * g.n_out * g.rank;
        const bool here = __any(mine == a);      // this wave has rows of it
        u32x4 w_run[KB];
        auto load_block = [&](int n0) {
#pragma unroll
            for (int q = 0; q < KB; ++q) {
                const int i = int(threadIdx.x) + q * kThreads;
                w_run[q] = *reinterpret_cast<const u32x4 *>(mat + int64_t(min(n0 + i / kChunks, g.n_out - 1)) * g.rank +
                                                            min(i % kChunks * 8, g.rank - 8));
            }
        };
        auto store_block = [&] {
#pragma unroll
            for (int q = 0; q < KB; ++q) {
                const int i = int(threadIdx.x) + q * kThreads, k = i % kChunks * 8;
                u32x4 raw = w_run[q];
                // columns past the adapter's rank are not part of it, whatever they hold
                if (KB * 32 > rank)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        raw[j] = k + 2 * j + 1 < rank ? raw[j] : (k + 2 * j < rank ? raw[j] & 0xffffu : 0u);
                *reinterpret_cast<u32x4 *>(&b_block[i / kChunks][k]) = raw;
            }
        };
        load_block(n_begin);
        if (pass > 0 || copied) load_base(n_begin + col);
        store_block();
        __syncthreads();
        for (int n0 = n_begin; n0 < n_end; n0 += 64) {
            const bool more = n0 + 64 < n_end;
            if (more) load_block(n0 + 64);
            if (here) {
                f32x4 acc[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    acc[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int q = 0; q < KB; ++q) {
                        Weight<WT> w;
                        w.set(*reinterpret_cast<const u32x4 *>(
                            &b_block[j * 16 + (lane & 15)][q * 32 + (lane >> 4) * 8]));
                        acc[j] = mfma_parts(w.p, v[q], acc[j]);
                    }
                }
                // results to rows: the wave's own part of LDS
                __builtin_amdgcn_wave_barrier();
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    *reinterpret_cast<f32x4 *>(&turn[lane & 15][j * 16 + (lane >> 4) * 4]) = acc[j];
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                __builtin_amdgcn_wave_barrier();
#pragma unroll
                for (int i = 0; i < kParts; ++i) {
                    const float *src = &turn[i * kRows + lane / kLanes][col];
                    float u[kRun];
#pragma unroll
                    for (int c = 0; c < kRun; c += 4)
                        *reinterpret_cast<f32x4 *>(u + c) = *reinterpret_cast<const f32x4 *>(src + c);
                    Run r;
#pragma unroll
                    for (int c = 0; c < kRun; ++c)
                        r.e[c] = from_float<XT>(__builtin_fmaf(scale, u[c], to_float<XT>(b_run[i].e[c])));
                    if (id[i] == a && n0 + col < n_end) stream_store(out + row[i] * g.ldo + n0 + col, r);
                }
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                if (more) load_base(n0 + 64 + col);
            }
            __syncthreads();
            if (more) {
                store_block();
                __syncthreads();
            }
        }
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
        const int slices = (g.n_out + kRowThreads - 1) / kRowThreads;
        if (g.tokens <= kFewRows && int64_t(g.tokens) * g.rank * slices <= kFewValues) {
            const dim3 grid(unsigned(g.tokens) * unsigned(slices));
            if (g.rank <= 16)
                hipLaunchKernelGGL((adapter_row_kernel<XT.value, WT.value, 1>), grid, dim3(kRowThreads), 0,
                                   stream, g, slices);
            else if (g.rank <= 32)
                hipLaunchKernelGGL((adapter_row_kernel<XT.value, WT.value, 2>), grid, dim3(kRowThreads), 0,
                                   stream, g, slices);
            else if (g.rank <= 64)
                hipLaunchKernelGGL((adapter_row_kernel<XT.value, WT.value, 4>), grid, dim3(kRowThreads), 0,
                                   stream, g, slices);
            else
                hipLaunchKernelGGL((adapter_row_kernel<XT.value, WT.value, 16>), grid, dim3(kRowThreads), 0,
                                   stream, g, slices);
            return hipGetLastError();
        }
        const AdapterSplit s = adapter_split(g.tokens, g.n_in);
        using One = std::integral_constant<int, 1>;
        using Two = std::integral_constant<int, 2>;
        using Four = std::integral_constant<int, 4>;
        // workgroups that share a tile's passes (one for each of its adapters):
        // rows by adapter need few, and each workgroup has to find its rows (1,024
        // rows in any order 44 us with 4, 50 with 16)
        auto passes = [&](int64_t groups) {
            const int64_t most = g.tokens <= kSortRows ? 4 : 16, n = 2048 / groups;
            return unsigned(n < 1 ? 1 : n > most ? most : n);
        };
        auto down = [&](auto NR, auto MR) {
            const unsigned blocks = unsigned((g.rank + 16 * NR.value - 1) / (16 * NR.value));
            const dim3 grid(unsigned(s.tiles) * unsigned(s.splits), blocks, passes(int64_t(s.tiles) * s.splits));
            hipLaunchKernelGGL((adapter_down_kernel<XT.value, WT.value, NR.value, MR.value>), grid, dim3(kThreads),
                               0, stream, g, s);
        };
        auto up_wide = [&](auto KB) {
            const int tiles = (g.tokens + 63) / 64, all = (g.n_out + 63) / 64;
            int slices = (kWideGroups + tiles - 1) / tiles;
            if (slices > all) slices = all;
            const int per = all / slices;               // rounded down: even shares, some more workgroups
            slices = (all + per - 1) / per;
            const dim3 grid(unsigned(tiles) * unsigned(slices), 1, passes(int64_t(tiles) * slices));
            hipLaunchKernelGGL((adapter_up_wide_kernel<XT.value, WT.value, KB.value>), grid, dim3(kThreads), 0, stream,
                               g, s, slices, per);
        };
        auto up = [&](auto KB) {
            const int tiles = (g.tokens + 15) / 16, all = (g.n_out + kThreads - 1) / kThreads;
            int slices = (2048 + tiles - 1) / tiles;
            if (slices > all) slices = all;
            const int per = all / slices;
            slices = (all + per - 1) / per;
            const dim3 grid(unsigned(tiles) * unsigned(slices), 1, passes(int64_t(tiles) * slices));
            hipLaunchKernelGGL((adapter_up_kernel<XT.value, WT.value, KB.value>), grid, dim3(kThreads), 0, stream, g, s,
                               tiles, slices, per);
        };
        auto by_rank = [&](auto MR) {
            if (g.rank <= 16) down(One{}, MR);
            else if (g.rank <= 32) down(Two{}, MR);
            else down(Four{}, MR);
            return hipGetLastError();
        };
        const hipError_t err = s.row_groups == 1 ? by_rank(One{}) : by_rank(Two{});
        if (err != hipSuccess) return err;
        const bool wide = g.tokens > kAdapterLongRows;
        if (g.rank > 64) up(std::integral_constant<int, 0>{});
        else if (g.rank > 32) wide ? up_wide(Two{}) : up(Two{});
        else wide ? up_wide(One{}) : up(One{});
        return hipGetLastError();
    });
}

}  // namespace moe
