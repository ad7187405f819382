// moe_layer.cpp -- host side of moe_layer.h: argument checks, sizes, launches.
#include "../../include/moe_layer.h"
#include "layer_ops.h"

#include <hip/hip_runtime_api.h>

#include <cmath>

using namespace moe;

namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int hip_status(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_EHIP; }

bool known_dtype(int d) { return d == MOE_F32 || d == MOE_BF16 || d == MOE_F16; }

int check_route(const void *logits, int64_t ld, int dtype, int tokens, int n_expert, int topk,
                int flags, float scale) {
    if (!known_dtype(dtype)) return MOE_EFORMAT;
    if (tokens < 0 || n_expert <= 0 || n_expert > MOE_ROUTE_MAX_EXPERTS) return MOE_EINVAL;
    if (topk <= 0 || topk > n_expert || topk > MOE_ROUTE_MAX_TOPK) return MOE_EINVAL;
    if ((flags & ~MOE_ROUTE_RENORM) != 0 || !std::isfinite(scale)) return MOE_EINVAL;
    if (tokens > 0 && !logits) return MOE_EINVAL;
    if (ld < n_expert || ld > (int64_t(1) << 40)) return MOE_EINVAL;
    if (!aligned16(logits)) return MOE_EALIGN;
    return MOE_OK;
}

RouteArgs route_args(const void *logits, int64_t ld, int dtype, int tokens, int n_expert, int topk,
                     int flags, float scale) {
    RouteArgs a{};
    a.logits = logits; a.ld = ld; a.dtype = dtype;
    a.tokens = tokens; a.n_expert = n_expert; a.topk = topk;
    a.renorm = (flags & MOE_ROUTE_RENORM) != 0;
    a.scale = scale;
    return a;
}

bool valid_set(const moe_adapter_set *s, int *status) {
    *status = MOE_EINVAL;
    if (!s) return false;
    *status = MOE_EFORMAT;
    if (s->dtype != MOE_BF16 && s->dtype != MOE_F16) return false;
    if (s->rank % 8 || s->n_in % 8 || s->n_out % 8) return false;
    *status = MOE_EINVAL;
    if (s->n_adapter <= 0 || s->rank <= 0 || s->rank > MOE_ADAPTER_MAX_RANK) return false;
    if (s->n_in <= 0 || s->n_out <= 0 || s->n_in > (1 << 24) || s->n_out > (1 << 24)) return false;
    *status = MOE_OK;
    return true;
}

}  // namespace

extern "C" {

int moe_route(const void *logits, int64_t ld, int dtype, int tokens, int n_expert, int topk,
              int flags, float scale, int32_t *ids, float *w, void *stream) {
    const int st = check_route(logits, ld, dtype, tokens, n_expert, topk, flags, scale);
    if (st) return st;
    if (tokens == 0) return MOE_OK;
    if (!ids || !w) return MOE_EINVAL;
    if (!aligned16(ids) || !aligned16(w)) return MOE_EALIGN;
    RouteArgs a = route_args(logits, ld, dtype, tokens, n_expert, topk, flags, scale);
    a.ids = ids;
    a.w = w;
    return hip_status(launch_route(a, static_cast<hipStream_t>(stream)));
}

size_t moe_balance_bytes(int tokens, int n_expert, int n_seq) {
    if (tokens < 0 || n_expert <= 0 || n_expert > MOE_ROUTE_MAX_EXPERTS || n_seq <= 0) return 0;
    return balance_layout(tokens, n_expert, n_seq).total;
}

int moe_route_balance(const void *logits, int64_t ld, int dtype, int tokens, int n_expert, int topk,
                      int flags, float scale, const int32_t *seq_off, int n_seq, float coef,
                      int32_t *ids, float *w, int32_t *counts, float *probs, float *loss,
                      void *workspace, size_t workspace_bytes, void *stream) {
    const int st = check_route(logits, ld, dtype, tokens, n_expert, topk, flags, scale);
    if (st) return st;
    if (n_seq <= 0 || !seq_off || !std::isfinite(coef)) return MOE_EINVAL;
    if (tokens > 0 && (!ids || !w)) return MOE_EINVAL;
    if (!counts || !probs || !loss || !workspace) return MOE_EINVAL;
    if (!aligned16(seq_off) || !aligned16(ids) || !aligned16(w) || !aligned16(counts) ||
        !aligned16(probs) || !aligned16(loss) || !aligned16(workspace))
        return MOE_EALIGN;
    if (workspace_bytes < balance_layout(tokens, n_expert, n_seq).total) return MOE_ESIZE;
    RouteArgs a = route_args(logits, ld, dtype, tokens, n_expert, topk, flags, scale);
    a.ids = ids; a.w = w;
    a.seq_off = seq_off; a.n_seq = n_seq; a.coef = coef;
    a.counts = counts; a.probs = probs; a.loss = loss;
    a.ws = static_cast<uint8_t *>(workspace);
    return hip_status(launch_route_balance(a, static_cast<hipStream_t>(stream)));
}

int moe_route_backward(const void *logits, int64_t ld, int dtype, int tokens, int n_expert, int topk,
                       int flags, float scale, const int32_t *ids, const float *dw,
                       const int32_t *seq_off, int n_seq, float coef, const int32_t *counts,
                       const float *dloss, void *dlogits, int64_t ldd, void *stream) {
    const int st = check_route(logits, ld, dtype, tokens, n_expert, topk, flags, scale);
    if (st) return st;
    if (ldd < n_expert || ldd > (int64_t(1) << 40) || !std::isfinite(coef)) return MOE_EINVAL;
    if ((seq_off == nullptr) != (counts == nullptr)) return MOE_EINVAL;
    if (seq_off && n_seq <= 0) return MOE_EINVAL;
    if (tokens == 0) return MOE_OK;
    if (!ids || !dlogits) return MOE_EINVAL;
    if (dlogits == logits && ldd != ld) return MOE_EINVAL;
    if (!aligned16(ids) || !aligned16(dw) || !aligned16(seq_off) || !aligned16(counts) ||
        !aligned16(dloss) || !aligned16(dlogits))
        return MOE_EALIGN;
    RouteArgs a = route_args(logits, ld, dtype, tokens, n_expert, topk, flags, scale);
    a.ids = const_cast<int32_t *>(ids);
    a.dw = dw;
    a.seq_off = seq_off; a.n_seq = n_seq; a.coef = coef;
    a.counts = const_cast<int32_t *>(counts);
    a.dloss = dloss;
    a.dlogits = dlogits; a.ldd = ldd;
    return hip_status(launch_route_backward(a, static_cast<hipStream_t>(stream)));
}

int moe_combine_backward(const float *dm, const float *w, const float *dout, int tokens, int topk,
                         int hidden, float *dw, float *ddm, void *stream) {
    if (tokens < 0 || topk <= 0 || hidden <= 0) return MOE_EINVAL;
    if ((long long)tokens * topk > (1LL << 30)) return MOE_EINVAL;     // as a plan's rows
    // one wave per token and eight of its rows, four to a workgroup: a launch holds 2^32 - 1 threads,
    // so 2^24 - 1 workgroups
    if ((long long)tokens * ((topk + 7) / 8) > (1LL << 26) - 4) return MOE_EINVAL;
    if (hidden % 4) return MOE_EFORMAT;
    if (tokens == 0) return MOE_OK;
    if (!dout || (!dw && !ddm) || (dw && !dm) || (ddm && !w)) return MOE_EINVAL;
    if (!aligned16(dm) || !aligned16(w) || !aligned16(dout) || !aligned16(dw) || !aligned16(ddm))
        return MOE_EALIGN;
    return hip_status(launch_combine_backward(dm, w, dout, tokens, topk, hidden, dw, ddm,
                                              static_cast<hipStream_t>(stream)));
}

size_t moe_adapters_bytes(const moe_adapter_set *set, int tokens) {
    int st;
    if (!valid_set(set, &st) || tokens < 0 || tokens > MOE_ADAPTER_MAX_TOKENS) return 0;
    return adapter_workspace(tokens, set->rank, set->n_in);
}

int moe_adapters(const moe_adapter_set *set, const int32_t *ids, int tokens, int dtype,
                 const void *x, int64_t ldx, const void *base, int64_t ldb, void *out, int64_t ldo,
                 void *workspace, size_t workspace_bytes, void *stream) {
    int st;
    if (!valid_set(set, &st)) return st;
    if (!set->a || !set->b || !set->scale) return MOE_EINVAL;
    if (!aligned16(set->a) || !aligned16(set->b) || !aligned16(set->scale) || !aligned16(set->ranks))
        return MOE_EALIGN;
    if (dtype != MOE_F32 && dtype != set->dtype) return MOE_EFORMAT;
    const int64_t far = int64_t(1) << 40;
    if (tokens < 0 || tokens > MOE_ADAPTER_MAX_TOKENS || ldx < set->n_in || ldb < set->n_out || ldo < set->n_out || ldx > far ||
        ldb > far || ldo > far)
        return MOE_EINVAL;
    if (ldx % 8 || ldb % 8 || ldo % 8) return MOE_EALIGN;
    if (tokens == 0) return MOE_OK;
    if (!ids || !x || !base || !out || !workspace) return MOE_EINVAL;
    if (out == x || (out == base && ldo != ldb)) return MOE_EINVAL;
    if (!aligned16(ids) || !aligned16(x) || !aligned16(base) || !aligned16(out) || !aligned16(workspace))
        return MOE_EALIGN;
    if (workspace_bytes < adapter_planes(tokens, set->rank, set->n_in)) return MOE_ESIZE;
    AdapterArgs a{};
    a.wtype = set->dtype; a.dtype = dtype;
    a.n_adapter = set->n_adapter; a.rank = set->rank; a.n_in = set->n_in; a.n_out = set->n_out;
    a.a = set->a; a.b = set->b; a.scale = set->scale; a.ranks = set->ranks;
    a.ids = ids; a.tokens = tokens;
    a.x = x; a.ldx = ldx; a.base = base; a.ldb = ldb; a.out = out; a.ldo = ldo;
    a.ws = static_cast<float *>(workspace);
    return hip_status(launch_adapters(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
