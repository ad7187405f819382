"""What the operators around the expert products cost: cases, inputs, plain forms and exact values.

Five operators of one MoE layer: the router (logits -> expert ids and weights), the router with its
balance statistics and loss, the router's gradient, the combine's gradient, and the low-rank adapters
of many requests beside a shared projection.  `own` says whether `run` computes their plain form or
calls this repository's kernels.

The sizes are the benchmark layer's (hidden 2560, n_ff 640, 512 experts, top-10) and the ranges around
it; logits carry a lognormal-like expert popularity (a per-expert bias), prompts are ragged and end in
padding rows, adapters differ in rank.
"""
import math

import numpy as np
import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_SIZE = {"f32": 4, "bf16": 2, "f16": 2}


# ---------------------------------------------------------------- cases
def _route(op, tokens, experts, topk, dtype, renorm, seqs=1, pad=0, closed=0, **more):
    return dict(op=op, tokens=tokens, experts=experts, topk=topk, dtype=dtype, renorm=renorm,
                seqs=seqs, pad=pad, closed=closed, **more)


def _adapters(tokens, requests, sets, rank, n_in, n_out, dtype, wdtype):
    return dict(op="adapters", tokens=tokens, requests=requests, sets=sets, rank=rank, n_in=n_in,
                n_out=n_out, dtype=dtype, wdtype=wdtype)


def listed():
    return [
        # one token of one request: latency
        dict(name="route_1", **_route("route", 1, 512, 10, "f32", True)),
        # the benchmark layer's largest prompt chunk
        dict(name="route_16k", **_route("route", 16384, 512, 10, "f32", True)),
        # a ragged batch of eight prompts on a small layer, padded at its end
        dict(name="balance_1531_ragged", **_route("balance", 1531, 60, 6, "bf16", False, seqs=8, pad=41)),
        # the largest chunk as one sequence
        dict(name="balance_16k", **_route("balance", 16384, 512, 10, "f32", True)),
        # router training, 2,048 tokens in four prompts, two experts out of service
        dict(name="route_backward_2k", **_route("route_backward", 2048, 512, 10, "bf16", False, seqs=4,
                                                closed=2)),
        dict(name="route_backward_16k", **_route("route_backward", 16384, 512, 10, "f32", True)),
        # gradients of the routing weights alone (frozen experts)
        dict(name="combine_backward_2k", op="combine_backward", tokens=2048, topk=10, hidden=2560, ddm=False),
        # with the expert rows' gradient
        dict(name="combine_backward_8k", op="combine_backward", tokens=8192, topk=10, hidden=2560, ddm=True),
        # one new token of one request, and of 48 requests with 32 adapters
        dict(name="adapters_decode_1", **_adapters(1, 1, 4, 16, 2560, 2560, "f32", "bf16")),
        dict(name="adapters_decode_48", **_adapters(48, 48, 32, 16, 2560, 1280, "bf16", "bf16")),
        # a ragged prompt batch in half precision, and the largest chunk in fp32
        dict(name="adapters_prefill_2047", **_adapters(2047, 9, 8, 24, 2560, 2560, "f16", "f16")),
        dict(name="adapters_prefill_16k", **_adapters(16384, 6, 8, 64, 2560, 2560, "f32", "bf16")),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "balance", "route_backward", "combine_backward", "adapters", "adapters"])
    if op in ("route", "balance", "route_backward"):
        experts = _log(rng, 8, 2048)
        tokens = _log(rng, 1, min(16384, 16384 * 512 // experts))
        topk = rng.randint(1, min(experts, 12))
        seqs = rng.randint(1, min(tokens, 9))
        return _route(op, tokens, experts, topk, rng.choice(["f32", "bf16", "f16"]), rng.random() < 0.5,
                      seqs=seqs, pad=rng.randint(0, tokens - seqs) // 4, closed=rng.randint(0, experts // 4))
    if op == "combine_backward":
        hidden = 64 * _log(rng, 1, 64)
        topk = rng.randint(1, 12)
        tokens = _log(rng, 1, 8192 * 10 * 2560 // (hidden * topk))
        return dict(op=op, tokens=min(tokens, 16384), topk=topk, hidden=hidden, ddm=rng.random() < 0.5)
    tokens = _log(rng, 1, 16384)
    n_in, n_out = 8 * _log(rng, 8, 320), 8 * _log(rng, 8, 320)
    dtype, wdtype = rng.choice([("f32", "bf16"), ("f32", "f16"), ("bf16", "bf16"), ("f16", "f16")])
    rank = 8 * rng.randint(1, 8)
    # either every request's one new token, or a batch of prompts
    requests = tokens if tokens <= 256 and rng.random() < 0.6 else rng.randint(1, min(tokens, 16))
    return _adapters(tokens, requests, rng.randint(1, 48), rank, n_in, n_out, dtype, wdtype)


# --------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _partition(rng, total, parts):
    """Ragged lengths of `parts` sequences, each at least one, together `total`."""
    cuts = np.sort(rng.choice(np.arange(1, total), parts - 1, replace=False)) if parts > 1 else np.zeros(0, np.int64)
    return np.diff(np.concatenate([[0], cuts, [total]])).astype(np.int64)


def _route_inputs(case, seed):
    g, rng = _gen(seed), np.random.default_rng(seed)
    T, E, K = case["tokens"], case["experts"], case["topk"]
    d = {}
    logits = _randn(g, T, E) + 0.7 * _randn(g, E)
    if case["closed"]:
        # experts out of service, never so many that fewer than topk stay open
        n = min(case["closed"], E - K)
        logits[:, torch.from_numpy(rng.permutation(E)[:n].copy()).cuda()] = -math.inf
    d["logits"] = logits.to(_DT[case["dtype"]])
    lens = _partition(rng, T - case["pad"], case["seqs"])
    off = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    d["seq_off"] = torch.from_numpy(off).cuda()
    d["bounds"] = list(zip(off[:-1].tolist(), off[1:].tolist()))      # the program knows its batch
    d["coef"] = 0.01
    d["dw"] = _randn(g, T, K)
    d["dloss"] = torch.full((1,), 0.5, device="cuda")
    return d


def _choose(d, case):
    """ids of the topk largest logits (ties to the lowest index) and the sequences' counts: what the
    router's forward pass left for its gradient."""
    T, E, K, S = case["tokens"], case["experts"], case["topk"], case["seqs"]
    ids = torch.sort(d["logits"].float(), dim=1, descending=True, stable=True)[1][:, :K].to(torch.int32).contiguous()
    off = d["seq_off"].long()
    inside = int(off[-1])
    seq = torch.bucketize(torch.arange(inside, device="cuda"), off[1:], right=True)
    counts = torch.zeros(S * E, dtype=torch.int64, device="cuda")
    flat = (seq[:, None] * E + ids[:inside].long()).reshape(-1)
    counts.index_add_(0, flat, torch.ones_like(flat))
    return ids, counts.view(S, E).to(torch.int32)


def _combine_inputs(case, seed):
    g = _gen(seed)
    T, K, H = case["tokens"], case["topk"], case["hidden"]
    return {"dm": _randn(g, T * K, H), "w": torch.softmax(_randn(g, T, K), dim=1), "dout": _randn(g, T, H)}


def _adapter_inputs(case, seed):
    g, rng = _gen(seed), np.random.default_rng(seed)
    T, n, R = case["tokens"], case["sets"], case["rank"]
    wt, xt = _DT[case["wdtype"]], _DT[case["dtype"]]
    d = {"a": (_randn(g, n, R, case["n_in"]) / math.sqrt(case["n_in"])).to(wt),
         "b": (0.05 * _randn(g, n, case["n_out"], R)).to(wt),
         "x": _randn(g, T, case["n_in"]).to(xt), "base": _randn(g, T, case["n_out"]).to(xt)}
    # an adapter's rank is at most the set's; a request in ten has no adapter
    ranks = np.array([R if i % 2 == 0 else rng.integers(1, R + 1) for i in range(n)], np.int32)
    d["rank"] = torch.from_numpy(ranks).cuda()
    d["scale"] = torch.from_numpy((2.0 * rng.random(n) + 0.5).astype(np.float32)).cuda()
    of_request = np.where(rng.random(case["requests"]) < 0.1, -1, rng.integers(0, n, case["requests"]))
    if (of_request < 0).all():
        of_request[0] = 0
    ids = np.repeat(of_request, _partition(rng, T, case["requests"])).astype(np.int32)
    d["ids"] = torch.from_numpy(ids).cuda()
    # the program knows its batch: each adapter in it, its rows and its rank
    d["batch"] = [(int(a), torch.from_numpy(np.nonzero(ids == a)[0]).cuda(), int(ranks[a]))
                  for a in sorted(set(ids.tolist())) if a >= 0]
    return d


def _inputs(case, seed):
    op = case["op"]
    if op == "adapters":
        return _adapter_inputs(case, seed)
    if op == "combine_backward":
        return _combine_inputs(case, seed)
    return _route_inputs(case, seed)


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    op = case["op"]
    if op == "route_backward":
        s["ids"], s["counts"] = _choose(s, case)
    if own:
        _own_buffers(s, case)
    return s


def _own_buffers(s, case):
    """The outputs, workspaces and descriptors that a user's program keeps."""
    import quantized_moe_expert_scatter_amd as moe
    op = case["op"]
    f32, i32, cuda = torch.float32, torch.int32, "cuda"
    if op in ("route", "balance"):
        s["o_ids"] = torch.empty(case["tokens"], case["topk"], dtype=i32, device=cuda)
        s["o_w"] = torch.empty(case["tokens"], case["topk"], dtype=f32, device=cuda)
    if op == "balance":
        S, E = case["seqs"], case["experts"]
        s["o_counts"] = torch.empty(S, E, dtype=i32, device=cuda)
        s["o_probs"] = torch.empty(S, E, dtype=f32, device=cuda)
        s["o_loss"] = torch.empty(1, dtype=f32, device=cuda)
        s["ws"] = torch.empty(moe.moe_balance_bytes(case["tokens"], E, S), dtype=torch.uint8, device=cuda)
    if op == "route_backward":
        s["o_dlogits"] = torch.empty_like(s["logits"])
    if op == "combine_backward":
        s["o_dw"] = torch.empty_like(s["w"])
        s["o_ddm"] = torch.empty_like(s["dm"]) if case["ddm"] else None
    if op == "adapters":
        s["set"] = moe.AdapterSet(s["a"], s["b"], s["scale"], rank=s["rank"])
        s["o"] = torch.empty_like(s["base"])
        s["ws"] = torch.empty(moe.moe_adapters_bytes(s["set"], case["tokens"]), dtype=torch.uint8, device=cuda)


# ------------------------------------------------------------ one pass
def run(state):
    return (_run_own if own else _run_plain)(state, state["case"])


def _run_own(s, c):
    import quantized_moe_expert_scatter_amd as moe
    op = c["op"]
    if op == "route":
        moe.moe_route(s["logits"], s["o_ids"], s["o_w"], renorm=c["renorm"])
        return s["o_ids"], s["o_w"]
    if op == "balance":
        moe.moe_route_balance(s["logits"], s["seq_off"], s["coef"], s["o_ids"], s["o_w"], s["o_counts"],
                              s["o_probs"], s["o_loss"], s["ws"], renorm=c["renorm"])
        return s["o_ids"], s["o_w"], s["o_counts"], s["o_probs"], s["o_loss"]
    if op == "route_backward":
        moe.moe_route_backward(s["logits"], s["ids"], s["dw"], s["o_dlogits"], renorm=c["renorm"],
                               seq_off=s["seq_off"], coef=s["coef"], counts=s["counts"], dloss=s["dloss"])
        return s["o_dlogits"]
    if op == "combine_backward":
        moe.moe_combine_backward(s["dm"], s["w"], s["dout"], s["o_dw"], s["o_ddm"])
        return (s["o_dw"], s["o_ddm"]) if c["ddm"] else s["o_dw"]
    moe.moe_adapters(s["set"], s["ids"], s["x"], s["base"], s["o"], s["ws"])
    return s["o"]


def _probs(logits):
    e = torch.exp(logits - logits.max(dim=1, keepdim=True)[0])
    return e / e.sum(dim=1, keepdim=True)


def _seq_of_rows(seq_off, T):
    """Each row's sequence, and whether it lies in one (rows behind the last are padding)."""
    row = torch.arange(T, device=seq_off.device, dtype=torch.int32)
    seq = (row[:, None] >= seq_off[None, 1:]).sum(dim=1)
    inside = seq < seq_off.numel() - 1
    return torch.where(inside, seq, 0), inside


def _plain_route(s, c):
    l = s["logits"].float()
    ids = torch.sort(l, dim=1, descending=True, stable=True)[1][:, :c["topk"]]
    p = _probs(l)
    w = p.gather(1, ids)
    if c["renorm"]:
        w = w / w.sum(dim=1, keepdim=True)
    return l, p, ids, w


def _run_plain(s, c):
    op = c["op"]
    if op == "route":
        _, _, ids, w = _plain_route(s, c)
        return ids.to(torch.int32), w
    if op == "balance":
        l, p, ids, w = _plain_route(s, c)
        S, E = c["seqs"], c["experts"]
        seq, inside = _seq_of_rows(s["seq_off"], c["tokens"])
        taken = ((l.gather(1, ids) > -math.inf) & inside[:, None]).to(torch.int32)
        counts = torch.zeros(S * E, dtype=torch.int32, device=l.device)
        counts.index_add_(0, (seq[:, None] * E + ids).reshape(-1), taken.reshape(-1))
        counts = counts.view(S, E)
        n = (s["seq_off"][1:] - s["seq_off"][:-1]).float()[:, None]
        # the long sums over a sequence's tokens, in 64 bits
        probs = torch.stack([p[b:e].sum(dim=0, dtype=torch.float64) / (e - b) for b, e in s["bounds"]]).float()
        loss = s["coef"] / S * (counts.float() * probs * (E / (c["topk"] * n))).double().sum()
        return ids.to(torch.int32), w, counts, probs, loss.float().reshape(1)
    if op == "route_backward":
        l = s["logits"].float()
        p = _probs(l)
        S, E, K = c["seqs"], c["experts"], c["topk"]
        ids = s["ids"].long()
        seq, inside = _seq_of_rows(s["seq_off"], c["tokens"])
        n = (s["seq_off"][1:] - s["seq_off"][:-1]).float()[:, None]
        g = (s["counts"].float() * (s["dloss"] * (s["coef"] * E / (S * K))) / (n * n))[seq] * inside[:, None]
        if c["renorm"]:
            q = p.gather(1, ids)
            q = q / q.sum(dim=1, keepdim=True)
            d = p * (g - (p * g).sum(dim=1, keepdim=True))
            d.scatter_add_(1, ids, q * (s["dw"] - (q * s["dw"]).sum(dim=1, keepdim=True)))
        else:
            g = g.scatter_add(1, ids, s["dw"])
            d = p * (g - (p * g).sum(dim=1, keepdim=True))
        return d.to(s["logits"].dtype)
    if op == "combine_backward":
        T, K, H = c["tokens"], c["topk"], c["hidden"]
        dw = (s["dm"].view(T, K, H) * s["dout"][:, None, :]).sum(dim=2)
        if not c["ddm"]:
            return dw
        return dw, (s["w"][:, :, None] * s["dout"][:, None, :]).reshape(T * K, H)
    out = s["base"].to(torch.float32, copy=True)
    if c["tokens"] <= 64:
        # few rows: every row's own matrices gathered
        a = s["ids"].clamp(min=0).long()
        on = torch.arange(c["rank"], device=out.device)[None, :] < s["rank"][a][:, None]
        h = (s["a"][a].float() * s["x"].float()[:, None, :]).sum(dim=2) * on
        step = s["scale"][a][:, None] * (s["b"][a].float() * h[:, None, :]).sum(dim=2)
        return torch.where(s["ids"][:, None] >= 0, out + step, out).to(s["base"].dtype)
    for a, rows, r in s["batch"]:
        h = s["x"][rows].float() @ s["a"][a, :r].float().t()
        out.index_add_(0, rows, s["scale"][a] * (h @ s["b"][a, :, :r].float().t()))
    return out.to(s["base"].dtype)


# -------------------------------------------------------- what it costs
def work(case):
    op = case["op"]
    if op in ("route", "balance", "route_backward"):
        T, E, K, S = case["tokens"], case["experts"], case["topk"], case["seqs"]
        z = _SIZE[case["dtype"]]
        if op == "route":
            return {"bytes": T * E * z + T * K * 8, "flops": 4 * T * E}
        if op == "balance":
            return {"bytes": T * E * z + T * K * 8 + S * E * 8 + 4 * S + 8, "flops": 5 * T * E}
        return {"bytes": 2 * T * E * z + T * K * 8 + S * E * 4 + 4 * S + 8, "flops": 8 * T * E}
    if op == "combine_backward":
        T, K, H = case["tokens"], case["topk"], case["hidden"]
        n = T * K * H
        both = case["ddm"]
        # the expert rows' gradient also reads the weights
        return {"bytes": 4 * (n + T * H + T * K) + (4 * n + 4 * T * K if both else 0),
                "flops": 2 * n + (n if both else 0)}
    T, R, z = case["tokens"], case["rank"], _SIZE[case["dtype"]]
    i, o = case["n_in"], case["n_out"]
    used = min(case["sets"], case["requests"])
    return {"bytes": T * (i + 2 * o) * z + T * 4 + used * R * (i + o) * _SIZE[case["wdtype"]],
            "flops": 2 * T * R * (i + o) + 2 * T * o}


# ------------------------------------------------------- in 64 bits
def exact(case, seed):
    d = _inputs(case, seed)
    op = case["op"]
    if op == "adapters":
        x, out = d["x"].double(), d["base"].double()
        scale, rank = d["scale"].tolist(), d["rank"].tolist()
        for a in range(case["sets"]):
            on = (d["ids"] == a).nonzero().reshape(-1)
            if on.numel():
                low = torch.mm(x[on], d["a"][a].double().t().contiguous())
                low[:, rank[a]:] = 0.0
                out[on] += torch.mm(low * scale[a], d["b"][a].double().t().contiguous())
        return out
    if op == "combine_backward":
        T, K = case["tokens"], case["topk"]
        dw = torch.empty(T, K, dtype=torch.float64, device="cuda")
        ddm = torch.empty(T * K, case["hidden"], dtype=torch.float64, device="cuda") if case["ddm"] else None
        do = d["dout"].double()
        for k in range(K):
            dw[:, k] = (d["dm"][k::K].double() * do).sum(dim=1)
            if ddm is not None:
                ddm[k::K] = d["w"][:, k:k + 1].double() * do
        return dw if ddm is None else (dw, ddm)
    # the router: the choice one expert at a time (the first of the largest), in 64 bits
    T, E, K, S = case["tokens"], case["experts"], case["topk"], case["seqs"]
    l = d["logits"].double()
    logz = torch.logsumexp(l, dim=1, keepdim=True)
    p = torch.exp(l - logz)
    rows = torch.arange(T, device="cuda")
    index = torch.arange(E, device="cuda").expand(T, E)
    left = l.clone()
    gone = torch.zeros(T, E, dtype=torch.bool, device="cuda")
    chosen = []
    for _ in range(K):
        top = left.masked_fill(gone, -math.inf).max(dim=1, keepdim=True)[0]
        at = torch.where((left == top) & ~gone, index, E).min(dim=1)[0]
        gone[rows, at] = True
        chosen.append(at)
    ids = torch.stack(chosen, dim=1)
    pick = p[rows[:, None], ids]
    total = pick.sum(dim=1, keepdim=True) if case["renorm"] else torch.ones_like(pick[:, :1])
    w = pick / total
    if op == "route":
        return ids.to(torch.int32), w
    off = d["seq_off"].tolist()
    counts = torch.zeros(S, E, dtype=torch.int64, device="cuda")
    probs = torch.zeros(S, E, dtype=torch.float64, device="cuda")
    for q in range(S):
        at = slice(off[q], off[q + 1])
        counts[q] = (gone[at] & (l[at] > -math.inf)).sum(dim=0)
        probs[q] = p[at].mean(dim=0)
    length = torch.tensor([off[q + 1] - off[q] for q in range(S)], dtype=torch.float64, device="cuda")[:, None]
    share = counts.double() * E / (K * length)
    if op == "balance":
        loss = d["coef"] / S * (share * probs).sum()
        return ids.to(torch.int32), w, counts.to(torch.int32), probs, loss.reshape(1)
    # gradient: the loss's part through p, the weights' part through the choice
    up = torch.zeros(T, E, dtype=torch.float64, device="cuda")
    for q in range(S):
        up[off[q]:off[q + 1]] = float(d["dloss"]) * d["coef"] / S * share[q] / length[q]
    grad = p * up - p * (p * up).sum(dim=1, keepdim=True)
    dw = d["dw"].double()
    for k in range(K):
        # d w_k / d l_e = w_k (delta - w_e over the chosen), or p_k (delta - p_e over all)
        push = dw[:, k:k + 1] * w[:, k:k + 1]
        if case["renorm"]:
            grad[rows[:, None], ids] -= push * w
        else:
            grad -= push * p
        grad[rows, ids[:, k]] += push[:, 0]
    return grad
