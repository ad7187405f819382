// router_kernels.hip -- the router's choice, its balance statistics and its
// gradient.
//
// One wavefront takes one token: lane i holds the J logits of experts
// [i*J, (i+1)*J), J = n_expert / 64 rounded up to a power of two, so a row is
// read once, in wide loads, and every later step is in registers.
//
// The choice: logits become 32-bit keys of the same order, and topk times the
// wave takes its largest key.  Lanes hold ascending experts, so the first
// lane that has the key, and in it the first, is the lowest expert.
#include "layer_ops.h"
#include "wave.cuh"
#include "../../include/moe_layer.h"

#include <hip/hip_runtime.h>

#include <type_traits>

namespace moe {

namespace {

constexpr int kRouteThreads = 256;
constexpr int kRouteWaves = kRouteThreads / 64;
constexpr int kRouteMaxGroups = 16384;      // workgroups; further tokens in a loop
constexpr int kJoinWaves = 16;
constexpr int kJoinMaxGroups = 4096;        // workgroups of the joining kernel; further jobs in a loop

// float -> key: ascending like the number, -0 equal to +0 (a NaN's is to be
// set by the caller: the largest key, above +inf).  No logit's key is 0 (that of -inf is 0x007fffff): 0 marks a place that
// holds no expert, or one already taken.
__device__ __forceinline__ uint32_t order_key(float f) {
    const uint32_t u = __float_as_uint(f + 0.0f);
    return u ^ (uint32_t(int32_t(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float(k == 0xffffffffu ? 0x7fffffffu : k ^ (k >> 31 ? 0x80000000u : 0xffffffffu));
}

// A wave's LDS holds a row by place and lane: expert e = lane * J + j at row j.
// A row of it is 64 / J longer than 64, so that experts in order lie in
// different banks.
template <int J> constexpr int kPlaceStride = 64 + (J > 1 ? 64 / J : 0);
template <int J>
__device__ __forceinline__ int place_of(int e) { return e % J * kPlaceStride<J> + e / J; }

// Experts of a wide access: 16 bytes, or all of a lane's.
template <int J, int SIZE> constexpr int kRunOf = J * SIZE < 16 ? J : 16 / SIZE;

// From expert order, 64 at a time, to the lanes' own experts, through the
// wave's LDS.
template <int J>
__device__ __forceinline__ void turn_in(const float (&x)[J], float (&v)[J], int lane, uint32_t *spare) {
    if constexpr (J == 1) {
        v[0] = x[0];
    } else {
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int j = 0; j < J; ++j) spare[place_of<J>(j * 64 + lane)] = __float_as_uint(x[j]);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int j = 0; j < J; ++j) v[j] = __uint_as_float(spare[j * kPlaceStride<J> + lane]);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
}

// The J logits of lane `from`, in wide accesses or one by one (-inf past the end).
template <int J, int DT, bool VEC>
__device__ __forceinline__ void load_own(const void *logits, int64_t at, int n_expert, int from, bool active,
                                         float (&v)[J]) {
    using T = typename Elem<DT>::T;
    constexpr int kRun = VEC ? kRunOf<J, sizeof(T)> : 1;
    struct alignas(kRun * sizeof(T)) Run { T e[kRun]; };
    const T *row = static_cast<const T *>(logits) + at + from * J;
#pragma unroll
    for (int i = 0; i < J; i += kRun) {
        const bool in = active && from * J + i < n_expert;
        Run r{};
        if (in) r = *reinterpret_cast<const Run *>(row + i);
#pragma unroll
        for (int j = 0; j < kRun; ++j) v[i + j] = in ? to_float<DT>(r.e[j]) : -INFINITY;
    }
}

// A row, every lane its own experts.  Rows that allow no wide access are read
// in expert order and turned (one by one in place, a load's lanes lie J
// elements apart: 47 us instead of 24 for the gradient of 16,384 rows of 509).
template <int J, int DT, bool VEC>
__device__ __forceinline__ void load_row(const void *logits, int64_t at, int n_expert, int lane,
                                         float (&v)[J], uint32_t *spare) {
    if constexpr (VEC) {
        load_own<J, DT, true>(logits, at, n_expert, lane, true, v);
    } else {
        const typename Elem<DT>::T *row = static_cast<const typename Elem<DT>::T *>(logits) + at;
        float x[J];
#pragma unroll
        for (int j = 0; j < J; ++j) x[j] = j * 64 + lane < n_expert ? to_float<DT>(row[j * 64 + lane]) : -INFINITY;
        turn_in<J>(x, v, lane, spare);
    }
}

// c[j] = f * the count of the lane's j-th expert (wide accesses where the
// logits have them: the table's rows are n_expert long, and so as aligned).
template <int J, int DT, bool VEC>
__device__ __forceinline__ void load_counts(const int32_t *row, int n_expert, int lane, float f, float (&c)[J],
                                            uint32_t *spare) {
    if constexpr (VEC) {
        constexpr int kRun = kRunOf<J, 4>;
        struct alignas(kRun * 4) Run { int32_t e[kRun]; };
#pragma unroll
        for (int i = 0; i < J; i += kRun)
            if (lane * J + i < n_expert) {
                const Run r = *reinterpret_cast<const Run *>(row + lane * J + i);
#pragma unroll
                for (int j = 0; j < kRun; ++j) c[i + j] = f * float(r.e[j]);
            }
    } else {
        float x[J];
#pragma unroll
        for (int j = 0; j < J; ++j) x[j] = j * 64 + lane < n_expert ? f * float(row[j * 64 + lane]) : 0.0f;
        turn_in<J>(x, c, lane, spare);
    }
}

// Sorts N = 2^n keys, largest first: Batcher's odd-even merging network, the
// same steps whatever the keys (19 exchanges for 8, 191 for 32).
template <int N>
__device__ __forceinline__ void sort_keys(uint32_t (&k)[N]) {
#pragma unroll
    for (int p = 1; p < N; p *= 2)
#pragma unroll
        for (int d = p; d >= 1; d /= 2)
#pragma unroll
            for (int i = 0; i < N - d; ++i)
                if (i >= d % p && (i - d % p) % (2 * d) < d && i / (2 * p) == (i + d) / (2 * p)) {
                    const uint32_t hi = max(k[i], k[i + d]);
                    k[i + d] = min(k[i], k[i + d]);
                    k[i] = hi;
                }
}

// The topk largest: lane k < topk receives the k-th's expert and logit.
// Returns the row's largest logit (NaN if the row holds one).
//   Each lane sorts its keys and puts the list into the wave's LDS (`lists`,
// place by place, a 0 behind it); it keeps the head and the one behind it.  A
// round takes the largest head (six cross-lane steps), notes it with its lane
// and moves that lane up: 12 vector operations a round, against 45 with the
// keys in registers and their place searched for in each round.  Which of the
// lane's experts it was is found afterwards for all rounds at once, in the row
// itself: the first that equals the round's logit, or the (times+1)-th where
// the `times` rounds just before had the same lane and key (equal keys leave a
// lane one after the other, as the first lane that has the largest key is
// always the one taken).
//   The router is bound by these operations: 16,384 fp32 rows of 512, top-10,
// take 11 us (35 MB, 3.2 TB/s), top-1 7.
template <int J> struct Lists {
    // the last two: the 0, and what a lane taken J times reads
    uint32_t place[J + 2][kPlaceStride<J>];
    uint32_t round[2 * MOE_ROUTE_MAX_TOPK];   // key and lane of each round
};
template <int J, int DT, bool VEC>
__device__ __forceinline__ float choose(const RouteArgs &a, int64_t row, const float (&v)[J], int lane, int &id,
                                        float &logit, Lists<J> &lists) {
    uint32_t key[J];
    bool odd = false;                         // NaN in the row, or infinities of both signs
    {
        float sum = v[0];
#pragma unroll
        for (int j = 1; j < J; ++j) sum += v[j];
        odd = __any(sum != sum);
    }
#pragma unroll
    for (int j = 0; j < J; ++j) key[j] = order_key(v[j]);
    if (odd)
#pragma unroll
        for (int j = 0; j < J; ++j) key[j] = v[j] == v[j] ? key[j] : 0xffffffffu;
    if (a.n_expert < 64 * J) {
        constexpr int kRun = VEC ? kRunOf<J, sizeof(typename Elem<DT>::T)> : 1;      // in or out together
#pragma unroll
        for (int j = 0; j < J; ++j) key[j] = lane * J + j / kRun * kRun < a.n_expert ? key[j] : 0u;
    }
    sort_keys(key);
    uint32_t head = key[0], next = 0;
    __builtin_amdgcn_wave_barrier();
    if constexpr (J > 1) {
        next = key[1];
#pragma unroll
        for (int j = 1; j <= J; ++j) lists.place[j][lane] = j < J ? key[j] : 0u;
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    int at = 1;                               // the place of `next`
    uint32_t first = 0;
    for (int k = 0; k < a.topk; ++k) {
        const uint32_t top = wave_max(head);
        uint64_t owner = __ballot(head == top);
        owner &= -owner;
        const bool taken = __builtin_amdgcn_inverse_ballot_w64(owner);
        first = k == 0 ? top : first;
        if (taken) {
            lists.round[2 * k] = head;
            lists.round[2 * k + 1] = uint32_t(lane);
        }
        head = taken ? next : head;
        if constexpr (J > 1) {
            at += taken;
            next = lists.place[at][lane];
        }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    const int k = min(lane, a.topk - 1);
    const uint32_t mine = lists.round[2 * k];
    const int from = int(lists.round[2 * k + 1]);
    id = from * J;
    logit = key_value(mine);
    if constexpr (J > 1) {
        float u[J];
        load_own<J, DT, VEC>(a.logits, row, a.n_expert, from, lane < a.topk, u);
        int times = 0;
        bool same = lane < a.topk;
        for (int d = 1; d < a.topk; ++d) {
            const int b = max(k - d, 0);
            same = same && k >= d && lists.round[2 * b] == mine && int(lists.round[2 * b + 1]) == from;
            if (!__any(same)) break;
            times += same;
        }
        int place = 0;
        if (!odd && !__any(times > 0)) {
#pragma unroll
            for (int j = J - 1; j >= 0; --j) place = u[j] == logit ? j : place;
        } else {
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const bool hit = u[j] == logit || (u[j] != u[j] && logit != logit);
                place = hit && times == 0 ? j : place;
                times -= hit;
            }
        }
        id += place;
    }
    return key_value(first);
}

// What the exponents are taken against: the row's largest logit, 0 where every
// expert is closed (all exponentials are then 0).
__device__ __forceinline__ float softmax_shift(float top) { return top == -INFINITY ? 0.0f : top; }

// e^x for x <= 0 (0 for -inf, NaN for NaN), within two steps of fp32 and with
// subnormal results: x = (n + f) ln 2, the fraction taken with log2(e) in two
// parts, so that its error does not grow with x.
__device__ __forceinline__ float exp_neg(float x) {
    constexpr float kHi = 1.44269502f, kLo = 1.92596303e-8f;      // log2(e) = kHi + kLo
    const float n = __builtin_rintf(fmaxf(x * kHi, -300.0f));
    const float f = __builtin_fmaf(x, kLo, __builtin_fmaf(x, kHi, -n));
    return __builtin_ldexpf(__builtin_amdgcn_exp2f(f), int(n));
}

// First sequence with seq_off[s+1] > t (n_seq if none), by 64 probes a step.
// Unsigned: 64 steps may pass 2^31, by less than 64.
__device__ __forceinline__ int sequence_of(const int32_t *seq_off, int n_seq, int t, int lane) {
    uint32_t lo = 0, n = n_seq;         // the answer is in [lo, lo + n]
    while (n > 0) {
        const uint32_t step = (n + 63) / 64;
        const uint32_t i = lo + uint32_t(lane + 1) * step - 1;
        const bool past = uint32_t(lane) * step < n && seq_off[1 + min(i, lo + n - 1)] <= t;
        const uint32_t skip = uint32_t(__popcll(__ballot(past))) * step;
        if (skip >= n) return int(lo + n);
        lo += skip;
        n = min(step - 1, n - skip);
    }
    return int(lo);
}

// Routes token t.  With STATS it returns the row's softmax, v * inv, and lane
// k's choice.
template <int J, int DT, bool VEC, bool STATS>
__device__ __forceinline__ void route_token(const RouteArgs &a, int t, int lane, float (&v)[J], float &inv,
                                            int &id, float &logit, Lists<J> &lists) {
    load_row<J, DT, VEC>(a.logits, int64_t(t) * a.ld, a.n_expert, lane, v, &lists.place[0][0]);
    const float top = choose<J, DT, VEC>(a, int64_t(t) * a.ld, v, lane, id, logit, lists);
    const float shift = softmax_shift(top);
    const bool chosen = lane < a.topk;
    const float e = chosen ? exp_neg(logit - shift) : 0.0f;
    inv = 0.0f;
    if (STATS || !a.renorm) {
        float part = 0.0f;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            v[j] = exp_neg(v[j] - shift);
            part += v[j];
        }
        const float sum = wave_sum(part);
        inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    }
    float w = inv;
    if (a.renorm) {
        const float sum = wave_sum(e);
        w = sum == 0.0f ? 0.0f : 1.0f / sum;
    }
    if (chosen) {
        a.ids[int64_t(t) * a.topk + lane] = id;
        a.w[int64_t(t) * a.topk + lane] = a.scale * (e * w);
    }
}

template <int J, int DT, bool VEC>
__global__ __launch_bounds__(kRouteThreads) void route_kernel(RouteArgs a) {
    const int lane = threadIdx.x & 63;
    __shared__ Lists<J> lists[kRouteWaves];
    for (int64_t t = int64_t(blockIdx.x) * kRouteWaves + (threadIdx.x >> 6); t < a.tokens;
         t += int64_t(gridDim.x) * kRouteWaves) {
        float v[J], inv, logit;
        int id;
        route_token<J, DT, VEC, false>(a, int(t), lane, v, inv, id, logit, lists[threadIdx.x >> 6]);
    }
}

// One workgroup per range of tokens: its waves route a token each and then add
// what they have to the sums of the token's sequence, p in registers (over the
// waves through LDS where a sequence ends), the choices in an LDS histogram.
// Several sequences in one round cost their sums only: 12 tokens in 8 sequences
// take 18 us with the joining kernel, 30 with a round for each.
//   16,384 fp32 rows of 512: 15.5 us, the routing's 11 and the exponentials of
// whole rows.  Two workgroups of 1,024 threads share a CU only while a wave
// keeps to 64 vector and about 80 scalar registers; left alone the compiler
// holds a lane mask for each of the J places in the latter (5 us here).
template <int J, int DT, bool VEC>
__global__ __attribute__((amdgpu_waves_per_eu(J <= 8 ? 8 : 1))) __launch_bounds__(64 * balance_waves(J)) void
route_balance_kernel(RouteArgs a, BalanceLayout L) {
    constexpr int kWaves = balance_waves(J), kThreads = 64 * kWaves;
    __shared__ Lists<J> lists[kWaves];        // while routing; then the waves' sums, from place[0] on
    __shared__ int hist[64 * J];
    if (blockIdx.x == 0 && threadIdx.x == 0) *reinterpret_cast<int32_t *>(a.ws + L.done) = 0;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    float *out_p = reinterpret_cast<float *>(a.ws + L.probs);
    int32_t *out_c = reinterpret_cast<int32_t *>(a.ws + L.counts);
    // rows are counted from the range's first: their numbers may reach 2^31 - 1, and a position a
    // round further on would not be one
    const int t0 = int(blockIdx.x) * L.range_tokens;
    const int rows = min(a.tokens - t0, L.range_tokens);
    for (int e = threadIdx.x; e < 64 * J; e += kThreads) hist[e] = 0;
    __syncthreads();
    float acc[J];
#pragma unroll
    for (int j = 0; j < J; ++j) acc[j] = 0.0f;
    int s = 0, end = 0;                        // the sequence at hand ends (or leaves the range) there
    bool inside = false;
    for (int round = 0; round < rows; round += kWaves) {
        const int t = round + wave, round_end = min(rows, round + kWaves);
        float v[J], inv = 0.0f, logit = -INFINITY;
        int id = 0;
        if (t < round_end) route_token<J, DT, VEC, true>(a, t0 + t, lane, v, inv, id, logit, lists[wave]);
        for (int pos = round; pos < round_end;) {
            if (pos >= end) {
                s = sequence_of(a.seq_off, a.n_seq, t0 + pos, lane);
                inside = s < a.n_seq;
                end = rows;
                if (inside) {
                    const int b = a.seq_off[s], e = a.seq_off[s + 1];
                    if (t0 + pos < b) {         // in front of the first sequence
                        inside = false;
                        end = min(b - t0, rows);
                    } else if (e > t0 + pos) {
                        end = min(e - t0, rows);
                    }
                }
            }
            const int stop = min(end, round_end);
            if (inside && t >= pos && t < stop) {
#pragma unroll
                for (int j = 0; j < J; ++j) acc[j] = __builtin_fmaf(v[j], inv, acc[j]);
                if (lane < a.topk && logit != -INFINITY) atomicAdd(hist + id, 1);
            }
            if (inside && stop == end) {
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    lists[wave].place[j][lane] = __float_as_uint(acc[j]);
                    acc[j] = 0.0f;
                }
                __syncthreads();
                const size_t at = (size_t(blockIdx.x) + s) * a.n_expert;
                for (int e = threadIdx.x; e < a.n_expert; e += kThreads) {
                    const int j = e % J, l = e / J;
                    float p = __uint_as_float(lists[0].place[j][l]);
#pragma unroll
                    for (int w = 1; w < kWaves; ++w) p += __uint_as_float(lists[w].place[j][l]);
                    out_p[at + e] = p;
                    out_c[at + e] = hist[e];
                    hist[e] = 0;
                }
                __syncthreads();
            }
            pos = stop;
        }
    }
}

// Joins a sequence's pieces for 16 experts: a quarter wave takes every 64th
// piece (8 of 512, all in flight at once), long sums in 64 bits and a fixed
// order.  The workgroup that is last to write its parts of the loss adds them
// all, in their order.
__global__ __launch_bounds__(64 * kJoinWaves) void balance_join_kernel(RouteArgs a, BalanceLayout L,
                                                                       int cols) {
    constexpr int kParts = 64 / kBalanceCols;        // pieces of a wave's access
    __shared__ double red_p[kJoinWaves * 64];
    __shared__ int red_c[kJoinWaves * 64];
    __shared__ bool last_group;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int col = lane % kBalanceCols;
    const int64_t jobs = int64_t(a.n_seq) * cols;
    float *loss = reinterpret_cast<float *>(a.ws + L.loss);
    for (int64_t job = blockIdx.x; job < jobs; job += gridDim.x) {
        const int s = int(job / cols), e = int(job % cols) * kBalanceCols + col;
        const int b = min(max(a.seq_off[s], 0), a.tokens);
        const int n = min(max(a.seq_off[s + 1], b), a.tokens) - b;
        double p = 0.0;
        int c = 0;
        if (n > 0 && e < a.n_expert) {
            const float *in_p = reinterpret_cast<const float *>(a.ws + L.probs) + size_t(s) * a.n_expert + e;
            const int32_t *in_c = reinterpret_cast<const int32_t *>(a.ws + L.counts) + size_t(s) * a.n_expert + e;
            const int last = (b + n - 1) / L.range_tokens;
#pragma unroll 8
            for (int r = b / L.range_tokens + wave * kParts + lane / kBalanceCols; r <= last;
                 r += kJoinWaves * kParts) {
                p += double(in_p[size_t(r) * a.n_expert]);
                c += in_c[size_t(r) * a.n_expert];
            }
        }
        red_p[threadIdx.x] = p;
        red_c[threadIdx.x] = c;
        __syncthreads();
        if (wave == 0) {
            // lane l adds rows l / 16, l / 16 + 4, ..., then the four are added
            p = 0.0;
            c = 0;
#pragma unroll
            for (int i = 0; i < kJoinWaves; ++i) {
                p += red_p[i * 64 + lane];
                c += red_c[i * 64 + lane];
            }
#pragma unroll
            for (int d = kBalanceCols; d < 64; d *= 2) {
                p += __shfl_xor(p, d);
                c += __shfl_xor(c, d);
            }
            const float mean = n > 0 ? float(p / n) : 0.0f;
            const bool own = lane < kBalanceCols && e < a.n_expert;
            if (own) {
                a.counts[size_t(s) * a.n_expert + e] = c;
                a.probs[size_t(s) * a.n_expert + e] = mean;
            }
            const float part = wave_sum(own ? float(c) * mean : 0.0f);
            if (lane == 0)
                __hip_atomic_store(loss + job,
                                   n > 0 ? part * (float(a.n_expert) / (float(a.topk) * float(n))) : 0.0f,
                                   __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
        __syncthreads();
    }
    if (threadIdx.x == 0)
        last_group = gridDim.x == 1 ||
                     __hip_atomic_fetch_add(reinterpret_cast<int32_t *>(a.ws + L.done), 1, __ATOMIC_ACQ_REL,
                                            __HIP_MEMORY_SCOPE_AGENT) == int(gridDim.x) - 1;
    __syncthreads();
    if (!last_group) return;
    double sum = 0.0;
    for (int64_t i = threadIdx.x; i < jobs; i += 64 * kJoinWaves)
        sum += double(__hip_atomic_load(loss + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
#pragma unroll
    for (int d = 1; d < 64; d *= 2) sum += __shfl_xor(sum, d);
    if (lane == 0) red_p[wave] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        sum = red_p[0];
#pragma unroll
        for (int i = 1; i < kJoinWaves; ++i) sum += red_p[i];
        a.loss[0] = float(double(a.coef) / a.n_seq * sum);
    }
}

// The gradient of one token's row.  The chosen experts' parts are scattered
// through the wave's LDS: each chosen id first writes its lane's number and
// reads it back, and only if an id is named twice (never by moe_route) are the
// parts added one after the other.  16,384 fp32 rows of 512: 17 us (68 MB, 4.0
// TB/s; 30 with a search through the registers for each choice).
template <int J, int DT, bool VEC>
__global__ __launch_bounds__(kRouteThreads) void route_backward_kernel(RouteArgs a) {
    using T = typename Elem<DT>::T;
    __shared__ uint32_t spares[kRouteWaves][J * kPlaceStride<J>];
    const int lane = threadIdx.x & 63;
    uint32_t *spare = spares[threadIdx.x >> 6];       // rows to turn; the chosen experts' parts
    const float dloss = a.seq_off && a.dloss ? a.dloss[0] : 1.0f;
    for (int64_t t = int64_t(blockIdx.x) * kRouteWaves + (threadIdx.x >> 6); t < a.tokens;
         t += int64_t(gridDim.x) * kRouteWaves) {
        float v[J];
        load_row<J, DT, VEC>(a.logits, t * a.ld, a.n_expert, lane, v, spare);
        // the chosen experts: lane k has the k-th
        int id = -1;
        float g = 0.0f, logit = -INFINITY;
        if (lane < a.topk) {
            id = a.ids[t * a.topk + lane];
            if (a.dw) g = a.scale * a.dw[t * a.topk + lane];
            id = id >= 0 && id < a.n_expert ? id : -1;
            if (id >= 0) logit = to_float<DT>(static_cast<const T *>(a.logits)[t * a.ld + id]);
            g = id >= 0 ? g : 0.0f;
        }
        // the loss's part
        float c[J];
#pragma unroll
        for (int j = 0; j < J; ++j) c[j] = 0.0f;
        if (a.seq_off) {
            const int s = sequence_of(a.seq_off, a.n_seq, int(t), lane);
            if (s < a.n_seq && t >= a.seq_off[s]) {
                const float n = float(a.seq_off[s + 1] - a.seq_off[s]);
                const float f = dloss * a.coef * float(a.n_expert) /
                                (float(a.n_seq) * float(a.topk) * n * n);
                load_counts<J, DT, VEC>(a.counts + size_t(s) * a.n_expert, a.n_expert, lane, f, c, spare);
            }
        }
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int j = 0; j < J; ++j) spare[j * kPlaceStride<J> + lane] = 0u;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        uint32_t *spot = spare + (id >= 0 ? place_of<J>(id) : 0);
        if (id >= 0) *spot = uint32_t(lane);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        const bool twice = __any(id >= 0 && *spot != uint32_t(lane));
        float top = v[0];
#pragma unroll
        for (int j = 1; j < J; ++j) top = fmaxf(top, v[j]);          // a NaN stays in v
        const float shift = softmax_shift(key_value(wave_max(order_key(top == top ? top : -INFINITY))));
        float part = 0.0f, pc = 0.0f;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            v[j] = exp_neg(v[j] - shift);
            part += v[j];
            pc = __builtin_fmaf(v[j], c[j], pc);
        }
        const float sum = wave_sum(part);
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        float z = wave_sum(pc) * inv;
        const float e = id >= 0 ? exp_neg(logit - shift) : 0.0f;
        float add;
        if (a.renorm) {
            const float chosen = wave_sum(e);
            const float q = chosen == 0.0f ? 0.0f : e / chosen;
            add = q * (g - wave_sum(q * g));
        } else {
            add = e * inv * g;
            z += wave_sum(add);
        }
        __builtin_amdgcn_wave_barrier();
        if (!twice) {
            if (id >= 0) *spot = __float_as_uint(add);
        } else {
            if (id >= 0) *spot = 0u;
            for (int k = 0; k < a.topk; ++k) {
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                __builtin_amdgcn_wave_barrier();
                if (lane == k && id >= 0) *spot = __float_as_uint(__uint_as_float(*spot) + add);
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int j = 0; j < J; ++j)
            v[j] = __builtin_fmaf(v[j] * inv, c[j] - z, __uint_as_float(spare[j * kPlaceStride<J> + lane]));
        T *row = static_cast<T *>(a.dlogits) + t * a.ldd;
        if constexpr (VEC) {
            constexpr int kRun = kRunOf<J, sizeof(T)>;
            struct alignas(kRun * sizeof(T)) Run { T e[kRun]; };
#pragma unroll
            for (int i = 0; i < J; i += kRun) {
                Run r;
#pragma unroll
                for (int j = 0; j < kRun; ++j) r.e[j] = from_float<DT>(v[i + j]);
                if (lane * J + i < a.n_expert) *reinterpret_cast<Run *>(row + lane * J + i) = r;
            }
        } else {
            // back to expert order
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int j = 0; j < J; ++j) spare[j * kPlaceStride<J> + lane] = __float_as_uint(v[j]);
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int j = 0; j < J; ++j)
                if (j * 64 + lane < a.n_expert)
                    row[j * 64 + lane] = from_float<DT>(__uint_as_float(spare[place_of<J>(j * 64 + lane)]));
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
        }
    }
}

// Wide accesses need whole runs (16 bytes, or a lane's experts) at a multiple
// of their size, at every row.
bool wide_rows(int j, int n_expert, int64_t ld, int dtype) {
    const int size = dtype == kF32 ? 4 : 2;
    const int run = j * size < 16 ? j : 16 / size;
    return n_expert % run == 0 && ld % run == 0;
}

// Calls f(J, DT, VEC) as compile-time constants.
template <class F>
hipError_t by_shape(int j, int dtype, bool vec, F f) {
    auto with_dt = [&](auto J) {
        auto with_vec = [&](auto DT) {
            return vec ? f(J, DT, std::true_type{}) : f(J, DT, std::false_type{});
        };
        if (dtype == kF32) return with_vec(std::integral_constant<int, kF32>{});
        if (dtype == kBF16) return with_vec(std::integral_constant<int, kBF16>{});
        return with_vec(std::integral_constant<int, kF16>{});
    };
    switch (j) {
        case 1: return with_dt(std::integral_constant<int, 1>{});
        case 2: return with_dt(std::integral_constant<int, 2>{});
        case 4: return with_dt(std::integral_constant<int, 4>{});
        case 8: return with_dt(std::integral_constant<int, 8>{});
        case 16: return with_dt(std::integral_constant<int, 16>{});
        default: return with_dt(std::integral_constant<int, 32>{});
    }
}

dim3 token_grid(int tokens) {
    const int64_t groups = (int64_t(tokens) + kRouteWaves - 1) / kRouteWaves;
    return dim3(unsigned(groups < kRouteMaxGroups ? groups : kRouteMaxGroups));
}

}  // namespace

hipError_t launch_route(const RouteArgs &a, hipStream_t stream) {
    const int j = route_lane_experts(a.n_expert);
    return by_shape(j, a.dtype, wide_rows(j, a.n_expert, a.ld, a.dtype), [&](auto J, auto DT, auto V) {
        hipLaunchKernelGGL((route_kernel<J.value, DT.value, V.value>), token_grid(a.tokens),
                           dim3(kRouteThreads), 0, stream, a);
        return hipGetLastError();
    });
}

hipError_t launch_route_balance(const RouteArgs &a, hipStream_t stream) {
    const BalanceLayout L = balance_layout(a.tokens, a.n_expert, a.n_seq);
    const int j = route_lane_experts(a.n_expert);
    hipError_t err = hipSuccess;
    if (a.tokens > 0)
        err = by_shape(j, a.dtype, wide_rows(j, a.n_expert, a.ld, a.dtype), [&](auto J, auto DT, auto V) {
            hipLaunchKernelGGL((route_balance_kernel<J.value, DT.value, V.value>), dim3(L.n_ranges),
                               dim3(64 * balance_waves(J.value)), 0, stream, a, L);
            return hipGetLastError();
        });
    if (err != hipSuccess) return err;
    const int cols = (a.n_expert + kBalanceCols - 1) / kBalanceCols;
    const int64_t jobs = int64_t(cols) * a.n_seq;
    // without tokens nothing has cleared the count of finished workgroups: one does it all
    const int64_t groups = a.tokens == 0 ? 1 : jobs < kJoinMaxGroups ? jobs : kJoinMaxGroups;
    hipLaunchKernelGGL(balance_join_kernel, dim3(unsigned(groups)), dim3(64 * kJoinWaves), 0, stream, a, L, cols);
    return hipGetLastError();
}

hipError_t launch_route_backward(const RouteArgs &a, hipStream_t stream) {
    const int j = route_lane_experts(a.n_expert);
    const bool vec = wide_rows(j, a.n_expert, a.ld, a.dtype) && wide_rows(j, a.n_expert, a.ldd, a.dtype);
    return by_shape(j, a.dtype, vec, [&](auto J, auto DT, auto V) {
        hipLaunchKernelGGL((route_backward_kernel<J.value, DT.value, V.value>), token_grid(a.tokens),
                           dim3(kRouteThreads), 0, stream, a);
        return hipGetLastError();
    });
}

}  // namespace moe
