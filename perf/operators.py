"""Timed cases of the operators whose sparse matrix the model chooses at run time.

Two operators, both a sparse product whose pattern is new in every call:

* routes: tokens sorted by expert, gathered, and the experts' rows weighted and
  added back per token, with every gradient (a tokens x slots matrix);
* blocks: attention of each query over the key blocks that a cheap score (the
  summed query heads against the mean key of each block) selects for it, with
  its gradient, and its form for single tokens over a cache (a queries x blocks
  matrix).

``own`` False computes the plain forms below in elementary torch operations in
fp32; ``own`` True calls the library.
"""
import math

import torch

own = False

DTYPE = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------- cases
def _blocks(name, kind, batch, queries, keys, heads, kv_heads, dim, block, n, dtype):
    return {"name": name, "op": "blocks", "kind": kind, "batch": batch, "queries": queries,
            "keys": keys, "heads": heads, "kv_heads": kv_heads, "dim": dim, "block": block,
            "n": n, "dtype": dtype}


def _routes(name, kind, tokens, k, experts, hidden, dtype, drop):
    return {"name": name, "op": "routes", "kind": kind, "tokens": tokens, "k": k,
            "experts": experts, "hidden": hidden, "dtype": dtype, "drop": drop}


def listed():
    return [
        # one user's next token over a short cache: latency is all there is
        _blocks("decode_1", "decode", 1, 1, 2000, 16, 4, 64, 64, 8, "fp16"),
        # a full serving batch of ragged caches, some slots free (length 0)
        _blocks("decode_64", "decode", 64, 1, 32768, 32, 4, 128, 64, 16, "bf16"),
        # a prompt's last chunk against the cache of the chunks before it, odd sizes
        _blocks("prefill_odd", "prefill", 3, 333, 1999, 12, 4, 64, 32, 6, "fp16"),
        # a long prompt in one call
        _blocks("prefill_8k", "prefill", 1, 8192, 8192, 32, 4, 128, 64, 16, "bf16"),
        # a fine-tuning step on short documents, every head its own keys
        _blocks("train_odd", "train", 4, 777, 777, 4, 4, 64, 32, 7, "fp16"),
        # a training step on long documents: forward and backward
        _blocks("train_4k", "train", 2, 4096, 4096, 16, 2, 128, 64, 16, "bf16"),
        # one token for each of a few users through the experts
        _routes("route_4", "forward", 4, 8, 64, 2048, "bf16", 0.0),
        # a prompt of odd length, a width that no vector load divides, fp32
        _routes("route_odd", "forward", 1237, 3, 10, 1001, "fp32", 0.05),
        # a large prompt batch
        _routes("route_16k", "forward", 16384, 8, 128, 4096, "bf16", 0.0),
        # a training step: forward and every gradient, some pairs over capacity
        _routes("route_train_1k", "train", 1000, 2, 8, 1024, "fp16", 0.02),
        _routes("route_train_8k", "train", 8192, 8, 64, 2048, "bf16", 0.02),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    if rng.random() < 0.4:
        kind = rng.choice(["forward", "train"])
        experts = _log(rng, 1, 256)
        k = min(experts, rng.choice([1, 2, 3, 4, 6, 8]))
        dtype = rng.choice(["bf16", "fp16", "fp32"])
        hidden = _log(rng, 16, 8192)
        if rng.random() < 0.6:
            hidden = max(16, hidden // 8 * 8)
        most = 16384 * 8 * 4096 // (k * hidden * (2 if dtype == "fp32" else 1)
                                    * (3 if kind == "train" else 1))
        return {"op": "routes", "kind": kind, "tokens": _log(rng, 1, min(16384, most)), "k": k,
                "experts": experts, "hidden": hidden, "dtype": dtype,
                "drop": rng.choice([0.0, 0.0, 0.02, 0.3])}
    kind = rng.choice(["decode", "prefill", "train"])
    dim, block = rng.choice([64, 128]), rng.choice([16, 32, 64, 128])
    kv_heads = rng.choice([1, 2, 4, 8])
    group = rng.choice([g for g in (1, 2, 3, 4, 7, 8, 16) if kv_heads * g <= 32])
    case = {"op": "blocks", "kind": kind, "batch": 1, "queries": 1, "keys": 1,
            "heads": kv_heads * group, "kv_heads": kv_heads, "dim": dim, "block": block,
            "n": _log(rng, 1, 1024 // block), "dtype": rng.choice(["bf16", "fp16"])}
    if kind == "decode":
        case["keys"] = _log(rng, 1, 32768)
        case["batch"] = _log(rng, 1, min(64, 64 * 32768 * 4 // (case["keys"] * kv_heads)))
        case["queries"] = rng.choice([1, 1, 1, 2, 5])
    else:
        top = 8192 if kind == "prefill" else 4096
        case["keys"] = _log(rng, 17, top)
        case["queries"] = case["keys"] if kind == "train" else _log(rng, 1, case["keys"])
        # the listed largest cases bound batch * heads * queries * keys
        room = (32 * 8192 * 8192 if kind == "prefill" else 2 * 16 * 4096 * 4096)
        case["batch"] = _log(rng, 1, max(1, min(8, room // (case["heads"] * case["queries"]
                                                           * case["keys"]))))
        if case["heads"] * case["queries"] * case["keys"] > room:
            case["heads"] = case["kv_heads"] = 4
    return case


def _lengths(case):
    """Valid keys of each sequence. A decode batch is ragged, from 0 (a free
    slot) to the longest; the others are full but for the last sequence."""
    B, Tk = case["batch"], case["keys"]
    if case["kind"] == "decode":
        return [0 if b % 16 == 15 else Tk - (b * 7919) % max(1, Tk - Tk // 8) for b in range(B)]
    return [Tk - (Tk // 3 if b and b == B - 1 else 0) for b in range(B)]


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dev, dt = torch.device("cuda"), DTYPE[case["dtype"]]

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    if case["op"] == "routes":
        T, k, E, H = case["tokens"], case["k"], case["experts"], case["hidden"]
        # experts differ in popularity; a token's experts are distinct, best first
        logits = randn(T, E) + randn(E)
        top = torch.sort(logits, dim=1, descending=True, stable=True)
        ids = top.indices[:, :k].to(torch.int32).contiguous()
        weights = torch.softmax(top.values[:, :k], dim=1).contiguous()
        if case["drop"]:
            ids = torch.where(torch.rand(T, k, generator=g, device=dev) < case["drop"], -1, ids)
            ids = ids.to(torch.int32)
        s = {"case": case, "ids": ids, "weights": weights, "x": randn(T, H).to(dt),
             "y": randn(T * k, H).to(dt)}          # y: what the experts return
        if case["kind"] == "train":
            s["dout"] = randn(T, H).to(dt)
            s["dxs"] = randn(T * k, H).to(dt)      # what the experts' backward returns
        return s

    B, Tq, Tk = case["batch"], case["queries"], case["keys"]
    Hq, Hk, D, blk = case["heads"], case["kv_heads"], case["dim"], case["block"]
    # Blocks have topics and runs of queries ask for one, so neighbouring queries
    # choose alike; every query likes the first block a little. All values are
    # multiples of 1/8 (16-bit types hold them), so block means and scores are
    # exact in fp32 in any order of summation and a choice has one right answer.
    NB = -(-Tk // blk)
    topics = randn(32, D)

    def pick(*shape):
        return topics[torch.randint(32, shape, generator=g, device=dev)]

    def grid(x):
        return (x * 8).round_().mul_(0.125).to(dt)

    k = randn(B, Tk, Hk, D)
    k += 0.5 * pick(B, NB, Hk).repeat_interleave(blk, dim=1)[:, :Tk]
    k[:, :blk] += 0.5 * topics[0]
    q = randn(B, Tq, Hq, D)
    runs = pick(B, -(-Tq // 24), Hk).repeat_interleave(24, dim=1)[:, :Tq]
    q += 0.5 * runs.repeat_interleave(Hq // Hk, dim=2) + 0.25 * topics[0]
    s = {"case": case, "q": grid(q), "k": grid(k), "v": randn(B, Tk, Hk, D).to(dt),
         "lengths": torch.tensor(_lengths(case), dtype=torch.int32, device=dev)}
    if case["kind"] == "decode":
        s["means"] = _means(s["k"], blk, s["lengths"])    # kept beside the cache
    if case["kind"] == "train":
        s["dout"] = randn(B, Tq, Hq, D).to(dt)
    return s


# ------------------------------------------------------------- plain forms
def _means(k, blk, lengths):
    """fp32 mean of each block's valid keys [B, NB, Hk, D]; 0 where there are none."""
    B, Tk, Hk, D = k.shape
    NB = -(-Tk // blk)
    at = torch.arange(NB * blk, device=k.device)
    x = torch.nn.functional.pad(k.float(), (0, 0, 0, 0, 0, NB * blk - Tk))
    x = torch.where((at < lengths[:, None])[:, :, None, None], x, 0.0)
    count = (lengths[:, None] - at[::blk]).clamp(0, blk)
    return x.view(B, NB, blk, Hk, D).sum(2) / count.clamp(min=1)[:, :, None, None]


def _select(q, means, n, blk, lengths):
    """int32 [B, Tq, Hk, n], ascending, -1 behind: the block of the query's own
    position and the n - 1 best-scoring earlier ones, ties to the lowest."""
    B, Tq, Hq, D = q.shape
    NB, Hk = means.shape[1:3]
    qs = q.float().view(B, Tq, Hk, Hq // Hk, D).sum(3)
    score = (qs.transpose(1, 2) @ means.permute(0, 2, 3, 1)).transpose(1, 2)  # [B, Tq, Hk, NB]
    pos = lengths[:, None] - Tq + torch.arange(Tq, device=q.device)
    last = torch.where(pos >= 0, pos // blk, -1)[:, :, None, None]
    at = torch.arange(NB, device=q.device)
    score = torch.where(at < last, score, -math.inf)
    score = torch.where(at == last, math.inf, score)
    order = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :n]
    taken = torch.arange(order.shape[-1], device=q.device) < last + 1
    order = torch.sort(torch.where(taken, order, NB), dim=-1).values
    order = torch.where(order == NB, -1, order)
    return torch.nn.functional.pad(order, (0, n - order.shape[-1]), value=-1).to(torch.int32)


def _attend_gathered(q, k, v, blocks, blk, lengths):
    """Every query's own blocks gathered: the form for few queries."""
    B, Tq, Hq, D = q.shape
    Tk, Hk = k.shape[1:3]
    at = blocks.long()[..., None] * blk + torch.arange(blk, device=q.device)
    pos = (lengths[:, None] - Tq + torch.arange(Tq, device=q.device))[:, :, None, None, None]
    seen = (blocks[..., None] >= 0) & (at <= pos)
    at, seen = at.clamp(0, Tk - 1).flatten(3), seen.flatten(3)[:, :, :, None]
    b = torch.arange(B, device=q.device)[:, None, None, None]
    h = torch.arange(Hk, device=q.device)[:, None]
    kg, vg = k[b, at, h].float(), v[b, at, h].float()               # [B, Tq, Hk, keys, D]
    s = q.float().view(B, Tq, Hk, Hq // Hk, D) @ kg.transpose(-1, -2) / math.sqrt(D)
    s = torch.where(seen, s, -math.inf)
    m = s.amax(-1, keepdim=True).clamp(min=-1e30)
    e = torch.exp(s - m)
    total = e.sum(-1, keepdim=True)
    o = (e @ vg) / torch.where(total > 0, total, 1.0)
    return o.reshape(B, Tq, Hq, D).to(q.dtype), (m + torch.log(total)).reshape(B, Tq, Hq)


def _scores_masked(q, k, blocks, blk, lengths):
    """All scores [B, Hk, G, Tq, Tk], -inf where a key is not selected or not yet seen."""
    B, Tq, Hq, D = q.shape
    Tk, Hk = k.shape[1:3]
    NB = -(-Tk // blk)
    chosen = torch.zeros(B, Tq, Hk, NB + 1, dtype=torch.bool, device=q.device)
    chosen.scatter_(3, torch.where(blocks >= 0, blocks, NB).long(), True)
    chosen = chosen[..., :NB].repeat_interleave(blk, dim=-1)[..., :Tk].transpose(1, 2)
    pos = lengths[:, None] - Tq + torch.arange(Tq, device=q.device)
    seen = torch.arange(Tk, device=q.device) <= pos[:, :, None]       # [B, Tq, Tk]
    seen = (chosen & seen[:, None])[:, :, None]
    s = q.float().view(B, Tq, Hk, Hq // Hk, D).permute(0, 2, 3, 1, 4) @ \
        k.float().permute(0, 2, 3, 1)[:, :, None]
    return torch.where(seen, s / math.sqrt(D), -math.inf)


def _attend_masked(q, k, v, blocks, blk, lengths, dout=None):
    """Dense scores under the selection's mask: the form for many queries."""
    B, Tq, Hq, D = q.shape
    Tk, Hk = k.shape[1:3]

    def back(x):                                     # [B, Hk, G, Tq, D] -> [B, Tq, Hq, D]
        return x.permute(0, 3, 1, 2, 4).reshape(B, Tq, Hq, -1)

    s = _scores_masked(q, k, blocks, blk, lengths)
    m = s.amax(-1, keepdim=True).clamp(min=-1e30)
    lse = m + torch.log(torch.exp(s - m).sum(-1, keepdim=True))
    p = torch.exp(s - torch.where(lse == -math.inf, 0.0, lse))
    del s
    vh = v.float().transpose(1, 2)[:, :, None]       # [B, Hk, 1, Tk, D]
    r = {"out": back(p @ vh).to(q.dtype), "lse": back(lse)[..., 0]}
    if dout is not None:
        do = dout.float().view(B, Tq, Hk, Hq // Hk, D).permute(0, 2, 3, 1, 4)
        qh = q.float().view(B, Tq, Hk, Hq // Hk, D).permute(0, 2, 3, 1, 4)
        r["dv"] = (p.transpose(-1, -2) @ do).sum(2).transpose(1, 2).to(v.dtype)
        dp = do @ vh.transpose(-1, -2)
        ds = p * (dp - (p * dp).sum(-1, keepdim=True)) / math.sqrt(D)
        r["dq"] = back(ds @ k.float().transpose(1, 2)[:, :, None]).to(q.dtype)
        r["dk"] = (ds.transpose(-1, -2) @ qh).sum(2).transpose(1, 2).to(k.dtype)
    return r


def _run_blocks(s):
    case, q, k, v, lengths = s["case"], s["q"], s["k"], s["v"], s["lengths"]
    blk, n = case["block"], case["n"]
    means = s["means"] if case["kind"] == "decode" else _means(k, blk, lengths)
    blocks = _select(q, means, n, blk, lengths)
    if case["kind"] == "decode":
        out, lse = _attend_gathered(q, k, v, blocks, blk, lengths)
        return {"blocks": blocks, "out": out, "lse": lse}
    return {"blocks": blocks, **_attend_masked(q, k, v, blocks, blk, lengths, s.get("dout"))}


def _run_blocks_own(s):
    import sparse_dense_matrix_gb300 as sdm
    case, q, k, v, lengths = s["case"], s["q"], s["k"], s["v"], s["lengths"]
    means = s["means"] if case["kind"] == "decode" else sdm.block_means(k, case["block"], lengths)
    sel = sdm.select_blocks(q, means, case["n"], case["block"], k.shape[1], lengths)
    out, lse = sel.attend(q, k, v)
    r = {"blocks": sel.blocks, "out": out, "lse": lse}
    if case["kind"] == "train":
        r["dq"], r["dk"], r["dv"] = sel.backward(s["dout"], q, k, v, out, lse)
    return r


def _run_routes(s):
    case, ids, x, y, w = s["case"], s["ids"], s["x"], s["y"], s["weights"]
    E, (T, k) = case["experts"], ids.shape
    key = torch.where(ids < 0, E, ids).flatten()
    order = torch.sort(key, stable=True).indices           # slot -> pair
    slot = torch.empty_like(order)
    slot[order] = torch.arange(T * k, device=ids.device)   # pair -> slot
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=ids.device)
    offsets[1:] = (key[:, None] == torch.arange(E, device=ids.device)).sum(0).cumsum(0)
    kept = (ids >= 0)[..., None]
    used = (key < E)[order][:, None]                       # slots that hold a pair
    slot = slot.view(T, k)
    r = {"offsets": offsets.to(torch.int32),
         "slots": torch.where(kept[..., 0], slot, -1).to(torch.int32),
         "xs": torch.where(used, x[order // k], 0)}
    yk = torch.where(kept, y[slot].float(), 0.0)           # [T, k, H]
    r["out"] = (yk * w[..., None]).sum(1).to(x.dtype)
    if case["kind"] == "train":
        do = s["dout"].float()
        wk = torch.where(kept[..., 0], w, 0.0)
        r["dy"] = (do[order // k] * wk.flatten()[order][:, None]).to(y.dtype)
        r["dweights"] = (yk * do[:, None]).sum(-1)
        r["dx"] = torch.where(kept, s["dxs"][slot].float(), 0.0).sum(1).to(x.dtype)
    return r


def _run_routes_own(s):
    import sparse_dense_matrix_gb300 as sdm
    case, y, w = s["case"], s["y"], s["weights"]
    routes = sdm.ExpertRoutes(s["ids"], case["experts"])
    r = {"offsets": routes.offsets, "slots": routes.slots, "xs": routes.dispatch(s["x"]),
         "out": routes.combine(y, w)}
    if case["kind"] == "train":
        r["dy"], r["dweights"] = routes.combine_backward(s["dout"], y, w)
        r["dx"] = routes.dispatch_backward(s["dxs"])
    return r


def run(state):
    if state["case"]["op"] == "routes":
        return _run_routes_own(state) if own else _run_routes(state)
    return _run_blocks_own(state) if own else _run_blocks(state)


# -------------------------------------------------------------------- work
def work(case):
    e = 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "routes":
        T, k, H, E = case["tokens"], case["k"], case["hidden"], case["experts"]
        pairs = T * k * (1 - case["drop"])
        # ids, weights, slots, offsets; x in, all xs rows out, pairs of y in, out out
        b = 12 * T * k + 4 * (E + 1) + e * H * (2 * T + T * k + pairs)
        f = 2 * pairs * H
        if case["kind"] == "train":
            # dout, dxs in; dy (all rows), dx, dweights out
            b += 4 * T * k + e * H * (2 * T + T * k + pairs)
            f += 4 * pairs * H
        return {"bytes": b, "flops": f}
    B, Tq, Tk, Hq, Hk = (case[c] for c in ("batch", "queries", "keys", "heads", "kv_heads"))
    D, blk, n = case["dim"], case["block"], case["n"]
    lens = torch.tensor(_lengths(case))
    pos = lens[:, None] - Tq + torch.arange(Tq)
    last = torch.where(pos >= 0, pos // blk, -1)
    cand = last.clamp(min=0).sum().item()                   # scored blocks, one kv head
    picked = (last + 1).clamp(max=n)
    seen = torch.where(pos >= 0, (picked - 1) * blk + pos % blk + 1, 0).sum().item()
    b = e * 2 * B * Tq * Hq * D + 4 * B * Tq * (Hq + Hk * n)     # q, out, lse, blocks
    f = 2 * D * Hk * cand + 4 * D * Hq * seen
    if case["kind"] == "decode":
        whole = (lens // blk).sum().item()
        b += 4 * D * Hk * min(cand, whole) + e * 2 * D * Hk * min(seen, int(lens.sum()))
    else:
        b += e * 2 * D * Hk * int(lens.sum())
    if case["kind"] == "train":
        b += e * (2 * B * Tq * Hq * D + 2 * B * Tk * Hk * D)    # dout, dq, dk, dv
        f += 10 * D * Hq * seen                                 # five products
    return {"bytes": b, "flops": f}


# ----------------------------------------------------- definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return _exact_routes(s) if case["op"] == "routes" else _exact_blocks(s)


def _exact_routes(s):
    """Through the dense 0/1 tokens x slots matrix's entries, one choice j at a time."""
    case, ids, w = s["case"], s["ids"].long(), s["weights"].double()
    T, k = ids.shape
    kept = ids >= 0
    key = torch.where(kept, ids, case["experts"]) * (T * k) + \
        torch.arange(T * k, device=ids.device).view(T, k)
    slot = torch.searchsorted(key.flatten().sort().values, key)     # rank of each pair
    xs = torch.zeros(T * k, case["hidden"], dtype=torch.float64, device=ids.device)
    out = torch.zeros(T, case["hidden"], dtype=torch.float64, device=ids.device)
    r = {"offsets": None, "slots": None, "xs": xs, "out": out}
    train = case["kind"] == "train"
    if train:
        r["dy"], r["dx"] = torch.zeros_like(xs), torch.zeros_like(out)
        r["dweights"] = torch.zeros_like(w)
    for j in range(k):
        t = kept[:, j].nonzero()[:, 0]
        at = slot[t, j]
        xs[at] = s["x"][t].double()
        out[t] += w[t, j, None] * s["y"][at].double()
        if train:
            do = s["dout"][t].double()
            r["dy"][at] = w[t, j, None] * do
            r["dweights"][t, j] = torch.einsum("th,th->t", do, s["y"][at].double())
            r["dx"][t] += s["dxs"][at].double()
    return r


def _exact_blocks(s):
    """Sequence by sequence, head by head, over whole rows of keys."""
    case, lengths = s["case"], s["lengths"].tolist()
    q, k, v = s["q"], s["k"], s["v"]
    B, Tq, Hq, D = q.shape
    Tk, Hk = k.shape[1:3]
    G, blk, n = Hq // Hk, case["block"], case["n"]
    kw = {"dtype": torch.float64, "device": q.device}
    out, lse = torch.zeros(B, Tq, Hq, D, **kw), torch.full((B, Tq, Hq), -math.inf, **kw)
    dq, dk, dv = torch.zeros_like(out), torch.zeros(B, Tk, Hk, D, **kw), torch.zeros(B, Tk, Hk, D, **kw)
    for b in range(B):
        L = lengths[b]
        if L == 0:
            continue
        pos = L - Tq + torch.arange(Tq, device=q.device)
        nb = -(-L // blk)
        for h in range(Hk):
            kb, vb = k[b, :L, h].double(), v[b, :L, h].double()
            qb = q[b, :, h * G:(h + 1) * G].double()
            key_block = torch.arange(L, device=q.device) // blk
            mean = torch.zeros(nb, D, **kw).index_add_(0, key_block, kb)
            mean /= torch.bincount(key_block, minlength=nb)[:, None]
            score = qb.sum(1) @ mean.T                            # [Tq, nb]
            at = torch.arange(nb, device=q.device)
            mine = torch.div(pos, blk, rounding_mode="floor")[:, None]
            score = score.masked_fill(at == mine, math.inf).masked_fill(at > mine, -math.inf)
            rank = torch.sort(torch.sort(-score, dim=1, stable=True).indices, dim=1).indices
            chosen = (rank < n) & (at <= mine)
            mask = chosen[:, key_block] & (torch.arange(L, device=q.device) <= pos[:, None])
            some = mask.any(1)
            for g in range(G):
                i = h * G + g
                x = (qb[:, g] @ kb.T / math.sqrt(D)).masked_fill(~mask, -math.inf)
                z = torch.logsumexp(x, dim=1)
                lse[b, :, i] = z
                p = torch.where(some[:, None], torch.softmax(x, dim=1), 0.0)
                out[b, :, i] = p @ vb
                if case["kind"] == "train":
                    do = s["dout"][b, :, i].double()
                    dv[b, :L, h] += p.T @ do
                    t = p * (do @ vb.T - (do * out[b, :, i]).sum(1, keepdim=True)) / math.sqrt(D)
                    dq[b, :, i] = t @ kb
                    dk[b, :L, h] += t.T @ qb[:, g]
    r = {"blocks": None, "out": out, "lse": lse}
    if case["kind"] == "train":
        r |= {"dq": dq, "dk": dk, "dv": dv}
    return r
