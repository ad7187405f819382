// layer_ops.h -- launchers of the steps around the expert products
// (moe_layer.cpp checks the arguments, the .hip files hold the kernels).
#pragma once

#include <hip/hip_runtime_api.h>

#include <cstddef>
#include <cstdint>

namespace moe {

// The router's rows: logits and what the router makes of them.
struct RouteArgs {
    const void *logits;
    int64_t ld;
    int dtype;                 // moe_dtype
    int tokens, n_expert, topk;
    bool renorm;
    float scale;
    int32_t *ids;              // forward: out; backward: in
    float *w;                  // forward: out
    // balance statistics
    const int32_t *seq_off;    // NULL: none
    int n_seq;
    float coef;
    int32_t *counts;           // forward: out; backward: in
    float *probs;
    float *loss;
    uint8_t *ws;
    // gradient
    const float *dw;
    const float *dloss;
    void *dlogits;
    int64_t ldd;
};

// The router holds a token's logits in one wave, J per lane.
constexpr int route_lane_experts(int n_expert) {
    int j = 1;
    while (j * 64 < n_expert) j *= 2;
    return j;
}
// Waves of a workgroup of the router with statistics: as many as its LDS (a
// row of fp32 sums per wave) allows.
constexpr int balance_waves(int lane_experts) {
    return lane_experts <= 8 ? 16 : lane_experts == 16 ? 8 : 4;
}

// The balance statistics are summed in pieces: the tokens are cut into ranges
// of range_tokens, one workgroup each, and a range's part of a sequence is a
// piece.  Sequences are in token order, so (range, sequence) -> range +
// sequence numbers the pieces without collisions, and no kernel needs to know
// on the host where sequences begin.  There is room for as many ranges as any
// smaller batch has: the longer ranges of a batch that is just too long for 512
// of the shortest are fewer.
struct BalanceLayout {
    int range_tokens, n_ranges;
    size_t probs;      // fp32 [ranges + n_seq][E]: sums of p over a piece
    size_t counts;     // int32, the same shape
    size_t loss;       // fp32 [n_seq][column blocks]: parts of the loss
    size_t done;       // int32: joining workgroups that have written theirs
    size_t total;
};

constexpr int kBalanceCols = 16;        // columns of one joining workgroup
constexpr int kBalanceMaxRanges = 512;  // two workgroups per CU

inline BalanceLayout balance_layout(int tokens, int n_expert, int n_seq) {
    BalanceLayout L{};
    const int waves = balance_waves(route_lane_experts(n_expert));
    const long long per = ((long long)tokens + kBalanceMaxRanges - 1) / kBalanceMaxRanges;
    L.range_tokens = per > waves ? int((per + waves - 1) / waves * waves) : waves;
    L.n_ranges = int(((long long)tokens + L.range_tokens - 1) / L.range_tokens);
    const long long most = ((long long)tokens + waves - 1) / waves;
    const size_t ranges = size_t(most < kBalanceMaxRanges ? most : kBalanceMaxRanges);
    const size_t cells = (ranges + size_t(n_seq)) * size_t(n_expert);
    auto up = [](size_t x) { return (x + 15) & ~size_t(15); };
    size_t o = 0;
    L.probs = o;  o += up(cells * 4);
    L.counts = o; o += up(cells * 4);
    L.loss = o;   o += up(size_t(n_seq) * size_t((n_expert + kBalanceCols - 1) / kBalanceCols) * 4);
    L.done = o;   o += 16;
    L.total = o;
    return L;
}

hipError_t launch_route(const RouteArgs &a, hipStream_t stream);
hipError_t launch_route_balance(const RouteArgs &a, hipStream_t stream);
hipError_t launch_route_backward(const RouteArgs &a, hipStream_t stream);

// dw[t][k] = dout[t] . dm[t*topk+k], ddm[t*topk+k] = w[t][k] * dout[t] (either may be NULL)
hipError_t launch_combine_backward(const float *dm, const float *w, const float *dout, int tokens,
                                   int topk, int hidden, float *dw, float *ddm, hipStream_t stream);

struct AdapterArgs {
    int wtype, dtype;          // moe_dtype of the matrices and of x, base, out
    int n_adapter, rank, n_in, n_out;
    const void *a, *b;
    const float *scale;
    const int32_t *ranks;
    const int32_t *ids;
    int tokens;
    const void *x;
    int64_t ldx;
    const void *base;
    int64_t ldb;
    void *out;
    int64_t ldo;
    float *ws;
};
// How the rows' low-rank values are computed: tiles of 16 * row_groups rows,
// the contraction in `splits` slices of `slice` (a slice's values are a plane
// of the workspace, fp32 [splits][tokens][rank], added where they are read).
struct AdapterSplit {
    int row_groups, tiles, splits, slice;
};
// More rows than this take 32 of them a tile (half the reads of a) and share b
// over 64: 16,384 fp32 rows of 2560 at rank 64 111 us in 16s, 101 in 32s; 6,000
// rows 55.5 and 58.
constexpr int kAdapterLongRows = 8192;
constexpr int kAdapterStep = 128;        // 4 waves x 32 values: what a slice is a multiple of
// Workgroups a launch should have, one per CU: more slices are more planes to
// add in the update (1,024 / 2,048 fp32 rows at rank 64: 18.1 / 28.4 us with
// two per CU, 15.6 / 25.2 with one).
constexpr int kAdapterGroups = 256;
inline AdapterSplit adapter_split(int tokens, int n_in) {
    AdapterSplit s{};
    s.row_groups = tokens > kAdapterLongRows ? 2 : 1;
    s.tiles = int(((long long)tokens + 16 * s.row_groups - 1) / (16 * s.row_groups));
    const int steps = (n_in + kAdapterStep - 1) / kAdapterStep;
    int want = s.tiles > 0 ? (kAdapterGroups + s.tiles - 1) / s.tiles : 1;
    if (want > 8) want = 8;
    if (want > steps) want = steps;
    const int per = (steps + want - 1) / want;
    s.slice = per * kAdapterStep;
    s.splits = (steps + per - 1) / per;
    return s;
}
// What a call over so many rows uses, and what any call over up to so many does:
// fewer rows are cut into more slices (2,049 of 2560 into 2, 4,096 into 1).
inline size_t adapter_planes(int tokens, int rank, int n_in) {
    const size_t planes = size_t(adapter_split(tokens, n_in).splits);
    return (planes * size_t(tokens) * size_t(rank) * 4 + 15) & ~size_t(15);
}
static_assert(kAdapterLongRows >= 16 * kAdapterGroups, "one slice where tiles have more than 16 rows");
inline size_t adapter_workspace(int tokens, int rank, int n_in) {
    size_t most = adapter_planes(tokens, rank, n_in);
    // the fullest of each number of tiles that has more than one slice
    for (int t = 16; t < tokens && t < 16 * kAdapterGroups; t += 16) {
        const size_t b = adapter_planes(t, rank, n_in);
        if (b > most) most = b;
    }
    return most;
}
hipError_t launch_adapters(const AdapterArgs &a, hipStream_t stream);

}  // namespace moe
