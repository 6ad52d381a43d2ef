"""Timed cases of the experts' products and of the rotation and norms of heads.

Two operators, each next to one whose sparse matrix the model chooses:

* experts: each expert's rows (between ``dispatch`` and ``combine`` of the
  routes) times that expert's matrix, with the gradients of the rows and of the
  matrices;
* heads: queries and keys turned by their position (pairs of adjacent elements
  or of the two halves, a part of the head, frequencies scaled for long
  contexts), where there are weights after a norm of each head, with every
  gradient, and the form that writes new keys and values into a cache. It comes
  before the selection of key blocks and the attention over them.

``own`` False computes the plain forms below in elementary torch operations in
fp32 (angles in fp64); ``own`` True calls the library.
"""
import math

import torch

own = False

DTYPE = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------- cases
def _experts(name, kind, tokens, k, experts, hidden, inner, dtype, drop, stored):
    return {"name": name, "op": "experts", "kind": kind, "tokens": tokens, "k": k,
            "experts": experts, "hidden": hidden, "inner": inner, "dtype": dtype, "drop": drop,
            "stored": stored}


def _heads(name, kind, batch, tokens, heads, kv_heads, dim, rotary, layout, scaling, norm, dtype,
           cache=0):
    return {"name": name, "op": "heads", "kind": kind, "batch": batch, "tokens": tokens,
            "heads": heads, "kv_heads": kv_heads, "dim": dim, "rotary": rotary, "layout": layout,
            "scaling": scaling, "norm": norm, "dtype": dtype, "cache": cache}


def listed():
    return [
        # one user's next token: eight experts' matrices are read for a row each
        _experts("experts_1", "forward", 1, 8, 64, 2048, 1024, "bf16", 0.0, "in_out"),
        # a serving batch: a few rows for each of many experts
        _experts("experts_64", "forward", 64, 8, 128, 2048, 768, "bf16", 0.0, "out_in"),
        # a prompt of odd length, widths that no tile divides
        _experts("experts_odd", "forward", 1237, 3, 10, 1000, 520, "fp16", 0.05, "in_out"),
        # a large prompt batch
        _experts("experts_16k", "forward", 16384, 8, 128, 2048, 1024, "bf16", 0.0, "in_out"),
        # a training step on few experts: the product and both gradients
        _experts("experts_train_1k", "train", 1000, 2, 8, 1024, 2048, "fp16", 0.02, "in_out"),
        # a training step of ordinary size, matrices stored as outputs x inputs
        _experts("experts_train_8k", "train", 8192, 8, 64, 2048, 1024, "bf16", 0.02, "out_in"),
        # one user's next token into its cache: latency is all there is
        _heads("heads_1", "append", 1, 1, 16, 4, 64, 64, "interleaved", "none", "none", "fp16",
               2000),
        # a full serving batch of ragged caches, some slots free (length 0)
        _heads("heads_64", "append", 64, 1, 32, 4, 128, 128, "half", "linear", "same", "bf16",
               2048),
        # a prompt's last chunk behind the chunks before it, half of each head turned
        _heads("heads_odd", "append", 3, 333, 12, 4, 64, 32, "half", "bands", "fp32", "fp16", 1999),
        # a long prompt in one call
        _heads("heads_8k", "prompt", 1, 8192, 32, 4, 128, 128, "half", "parts", "same", "bf16"),
        # a fine-tuning step on short documents, every head its own keys
        _heads("heads_train_odd", "train", 4, 777, 4, 4, 64, 64, "interleaved", "none", "fp32",
               "fp16"),
        # a training step on long documents
        _heads("heads_train_4k", "train", 2, 4096, 16, 2, 128, 128, "half", "none", "same", "bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    if rng.random() < 0.5:
        kind = rng.choice(["forward", "train"])
        experts = _log(rng, 1, 256)
        k = min(experts, rng.choice([1, 2, 3, 4, 6, 8]))
        hidden, inner = (8 * _log(rng, 4, 512) for _ in range(2))
        # the largest listed case bounds a product's operations and a set of matrices
        experts = max(k, min(experts, 128 * 2048 * 1024 // (hidden * inner)))
        most = 16384 * 8 * 2048 * 1024 // (k * hidden * inner * (3 if kind == "train" else 1))
        return {"op": "experts", "kind": kind, "tokens": _log(rng, 1, max(1, min(16384, most))),
                "k": k, "experts": experts, "hidden": hidden, "inner": inner,
                "dtype": rng.choice(["bf16", "fp16"]), "drop": rng.choice([0.0, 0.0, 0.02, 0.3]),
                "stored": rng.choice(["in_out", "out_in"])}
    kind = rng.choice(["append", "prompt", "train"])
    dim = rng.choice([32, 64, 64, 80, 96, 128, 128, 192, 256])
    kv_heads = rng.choice([1, 2, 4, 8])
    heads = kv_heads * rng.choice([g for g in (1, 2, 3, 4, 7, 8, 16) if kv_heads * g <= 32])
    case = {"op": "heads", "kind": kind, "batch": 1, "tokens": 1, "heads": heads,
            "kv_heads": kv_heads, "dim": dim,
            "rotary": rng.choice([dim, dim, max(16, dim // 32 * 16), 16]),
            "layout": rng.choice(["half", "interleaved"]),
            "scaling": rng.choice(["none", "linear", "base", "parts", "bands"]),
            "norm": rng.choice(["none", "same", "fp32"]),
            "dtype": rng.choice(["bf16", "fp16", "fp32"]), "cache": 0}
    # the longest listed prompt's elements bound a case's
    room = 8192 * 36 * 128 // ((heads + kv_heads) * dim)
    if case["dtype"] == "fp32" or kind == "train":
        room //= 3
    if kind == "append":
        case["tokens"] = rng.choice([1, 1, 1, 2, 5, _log(rng, 1, min(room, 2048))])
        case["batch"] = _log(rng, 1, max(1, min(64, room // case["tokens"])))
        most = 64 * 2048 * 4 * 128 // (case["batch"] * kv_heads * dim)
        case["cache"] = _log(rng, case["tokens"], max(case["tokens"], min(32768, most)))
    else:
        case["tokens"] = _log(rng, 1, min(8192, room))
        case["batch"] = _log(rng, 1, max(1, min(8, room // case["tokens"])))
    return case


# ------------------------------------------------------------------ inputs
SCALING = {"none": None,
           "linear": {"kind": "linear", "factor": 4.0},
           "base": {"kind": "base", "factor": 8.0},
           "parts": {"kind": "parts", "factor": 16.0, "original_length": 4096},
           "bands": {"kind": "bands", "factor": 8.0, "original_length": 8192}}
BASE, EPS = 500000.0, 1e-6


def _lengths(case):
    """Keys of each sequence after the new ones: ragged; in a batch some slots are
    free (length 0), and a sequence may be shorter than what a padded call brings."""
    B, Tk = case["batch"], case["cache"]
    return [0 if b % 16 == 15 else Tk - (b * 7919) % max(1, Tk - Tk // 8) for b in range(B)]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dev, dt = torch.device("cuda"), DTYPE[case["dtype"]]

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    train = case["kind"] == "train"
    if case["op"] == "experts":
        T, k, E = case["tokens"], case["k"], case["experts"]
        H, F = case["hidden"], case["inner"]
        # experts differ in popularity; a token's experts are distinct
        ids = torch.sort(randn(T, E) + randn(E), dim=1, descending=True).indices[:, :k]
        if case["drop"]:
            ids = torch.where(torch.rand(T, k, generator=g, device=dev) < case["drop"], -1, ids)
        ids = ids.to(torch.int32).contiguous()
        counts = torch.bincount(ids[ids >= 0], minlength=E)
        s = {"case": case, "xs": randn(T * k, H).to(dt)}
        s["offsets"] = torch.nn.functional.pad(counts.cumsum(0), (1, 0)).to(torch.int32)
        if case["stored"] == "in_out":
            s["w"] = torch.empty(E, H, F, dtype=dt, device=dev)
        else:                                    # as a linear layer keeps it
            s["w"] = torch.empty(E, F, H, dtype=dt, device=dev).transpose(1, 2)
        for e in range(E):
            s["w"][e] = randn(H, F) * H ** -0.5
        if train:
            s["dys"] = randn(T * k, F).to(dt)
        if own:
            import sparse_dense_matrix_gb300 as sdm
            s["routes"] = sdm.ExpertRoutes(ids, E)
        return s

    B, T, Hq, Hk, D = (case[n] for n in ("batch", "tokens", "heads", "kv_heads", "dim"))
    # one projection's output, of which queries, keys and values are views; keys have
    # a common part, as trained ones do
    qkv = randn(B, T, Hq + 2 * Hk, D)
    qkv[:, :, Hq:Hq + Hk] += 2 * randn(Hk, D)
    s = {"case": case}
    s["q"], s["k"], s["v"] = qkv.to(dt).split([Hq, Hk, Hk], dim=2)
    s["wq"] = s["wk"] = None
    if case["norm"] != "none":
        wt = dt if case["norm"] == "same" else torch.float32
        s["wq"], s["wk"] = ((1 + 0.25 * randn(D)).to(wt) for _ in range(2))
    if case["kind"] == "append":
        s["lengths"] = torch.tensor(_lengths(case), dtype=torch.int32, device=dev)
        s["ck"], s["cv"] = (randn(B, case["cache"], Hk, D).to(dt) for _ in range(2))
    else:
        # documents follow one another in a row: positions begin again, some far out
        start = torch.randint(0, 1 << 17, (B, 1), generator=g, device=dev)
        at = torch.arange(T, device=dev)
        s["positions"] = torch.where(at < T // 3, at, at - T // 3 + start).to(torch.int32)
    if train:
        s["dq"], s["dk"] = randn(B, T, Hq, D).to(dt), randn(B, T, Hk, D).to(dt)
    if own:
        import sparse_dense_matrix_gb300 as sdm
        s["turn"] = sdm.HeadRotation(D, case["rotary"], layout=case["layout"], base=BASE,
                                     scaling=SCALING[case["scaling"]], device=dev)
    else:
        s["freq"], s["magnitude"] = _frequencies(case)
        s["freq"] = s["freq"].to(dev)
    return s


# ------------------------------------------------------------- plain forms
def _run_experts(s):
    case, xs, w = s["case"], s["xs"], s["w"]
    at = s["offsets"].tolist()
    ys = torch.zeros(xs.shape[0], case["inner"], dtype=xs.dtype, device=xs.device)
    train = case["kind"] == "train"
    if train:
        dxs, dw = torch.zeros_like(xs), torch.zeros_like(w)
    for e in range(case["experts"]):
        if at[e] == at[e + 1]:
            continue
        rows = slice(at[e], at[e + 1])
        x, we = xs[rows].float(), w[e].float()
        ys[rows] = (x @ we).to(ys.dtype)
        if train:
            dy = s["dys"][rows].float()
            dxs[rows] = (dy @ we.T).to(xs.dtype)
            dw[e] = (x.T @ dy).to(w.dtype)
    return {"ys": ys, "dxs": dxs, "dw": dw} if train else {"ys": ys}


def _run_experts_own(s):
    routes = s["routes"]
    r = {"ys": routes.product(s["xs"], s["w"])}
    if s["case"]["kind"] == "train":
        r["dxs"], r["dw"] = routes.product_backward(s["dys"], s["xs"], s["w"])
    return r


def _frequencies(case):
    """fp64 [rotary / 2]: radians per position of each pair; and the factor on sines and cosines."""
    R, how = case["rotary"], SCALING[case["scaling"]]
    i = torch.arange(R // 2, dtype=torch.float64)
    if how is None:
        return BASE ** (-2 * i / R), 1.0
    s = how["factor"]
    if how["kind"] == "base":                    # the slowest pair is slowed by s, the first by 1
        return (BASE * s ** (R / (R - 2))) ** (-2 * i / R), 1.0
    f = BASE ** (-2 * i / R)
    if how["kind"] == "linear":
        return f / s, 1.0
    L = how["original_length"]
    if how["kind"] == "parts":                   # between 32 turns and 1 in the original length
        lo, hi = (R * math.log(L / (2 * math.pi * turns)) / (2 * math.log(BASE))
                  for turns in (32, 1))
        lo, hi = max(0, math.floor(lo)), min(R - 1, math.ceil(hi))
        ramp = ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        return f * (1 - ramp) + f / s * ramp, 0.1 * math.log(s) + 1
    turns = L * f / (2 * math.pi)                # bands: 1 turn and 4 in the original length
    mix = ((turns - 1) / (4 - 1)).clamp(0, 1)
    return f * mix + f / s * (1 - mix), 1.0


def _turn(z, angle, case, magnitude):
    """The first `rotary` elements of z [B, T, heads, D] turned by angle [B, T, rotary / 2]."""
    R = case["rotary"]
    c, s = ((magnitude * f(angle)).float()[:, :, None] for f in (torch.cos, torch.sin))
    if case["layout"] == "half":
        a, b = z[..., :R // 2], z[..., R // 2:R]
        y = torch.cat([a * c - b * s, b * c + a * s], -1)
    else:
        a, b = z[..., 0:R:2], z[..., 1:R:2]
        y = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    return torch.cat([y, z[..., R:]], -1)


def _one(x, w, angle, case, magnitude, grad=None):
    """One tensor's result, and with the gradient of it that of x and of w."""
    z = x.float()
    if w is not None:
        r = torch.rsqrt((z * z).mean(-1, keepdim=True) + EPS)
        n = z * r
        z = n * w.float()
    y = _turn(z, angle, case, magnitude).to(x.dtype)
    if grad is None:
        return y
    g = _turn(grad.float(), -angle, case, magnitude)
    if w is None:
        return y, g.to(x.dtype)
    dw = (g * n).double().sum((0, 1, 2)).to(w.dtype)
    u = g * w.float()
    return y, (r * (u - n * (u * n).mean(-1, keepdim=True))).to(x.dtype), dw


def _run_heads(s):
    case, q, k = s["case"], s["q"], s["k"]
    B, T = q.shape[:2]
    if case["kind"] == "append":
        pos = s["lengths"][:, None] - T + torch.arange(T, device=q.device)
    else:
        pos = s["positions"]
    angle = pos[..., None].double() * s["freq"]
    args = angle, case, s["magnitude"]
    if case["kind"] == "train":
        q2 = _one(q, s["wq"], *args, s["dq"])
        k2 = _one(k, s["wk"], *args, s["dk"])
        r = {"q": q2[0], "k": k2[0], "dq": q2[1], "dk": k2[1]}
        if s["wq"] is not None:
            r["dwq"], r["dwk"] = q2[2], k2[2]
        return r
    q, k = _one(q, s["wq"], *args), _one(k, s["wk"], *args)
    if case["kind"] == "prompt":
        return {"q": q, "k": k}
    b, t = torch.nonzero(pos >= 0, as_tuple=True)
    s["ck"][b, pos[b, t].long()] = k[b, t]
    s["cv"][b, pos[b, t].long()] = s["v"][b, t]
    return {"q": q, "cache_k": s["ck"], "cache_v": s["cv"]}


def _run_heads_own(s):
    case, turn = s["case"], s["turn"]
    norm = {"q_weight": s["wq"], "k_weight": s["wk"], "eps": EPS}
    if case["kind"] == "append":
        q = turn.append(s["q"], s["k"], s["v"], s["ck"], s["cv"], s["lengths"], **norm)
        return {"q": q, "cache_k": s["ck"], "cache_v": s["cv"]}
    q, k = turn.rotate(s["q"], s["k"], positions=s["positions"], **norm)
    r = {"q": q, "k": k}
    if case["kind"] == "train":
        r["dq"], r["dk"], dwq, dwk = turn.rotate_backward(
            s["dq"], s["dk"], s["q"], s["k"], positions=s["positions"], **norm)
        if dwq is not None:
            r["dwq"], r["dwk"] = dwq, dwk
    return r


def run(state):
    if state["case"]["op"] == "experts":
        return _run_experts_own(state) if own else _run_experts(state)
    return _run_heads_own(state) if own else _run_heads(state)


# -------------------------------------------------------------------- work
def work(case):
    e = 4 if case["dtype"] == "fp32" else 2
    train = case["kind"] == "train"
    if case["op"] == "experts":
        T, k, E, H, F = (case[n] for n in ("tokens", "k", "experts", "hidden", "inner"))
        pairs = T * k * (1 - case["drop"])
        # matrices of experts that have rows (as many as with experts alike)
        used = E * (1 - (1 - k / E * (1 - case["drop"])) ** T)
        b = 4 * (E + 1) + e * (pairs * H + T * k * F + used * H * F)
        f = 2 * pairs * H * F
        if train:                                # dys in; dxs and dw out
            b += e * (pairs * F + T * k * H + E * H * F)
            f *= 3
        return {"bytes": b, "flops": f}
    B, T, Hq, Hk, D = (case[n] for n in ("batch", "tokens", "heads", "kv_heads", "dim"))
    rows = B * T * (Hq + Hk)
    per = 3 * case["rotary"] + (4 * D if case["norm"] != "none" else 0)
    if case["kind"] == "append":                 # keys of sequences shorter than the call are not
        written = sum(min(T, n) for n in _lengths(case)) * Hk
        b = 4 * B + e * D * (2 * B * T * Hq + 4 * written)
    else:
        b = 4 * B * T + e * D * 2 * rows
    if case["norm"] != "none":
        b += 2 * D * (4 if case["norm"] == "fp32" else e)
    f = per * rows
    if train:                                    # grads and, for a norm's, inputs again; grads out
        b += e * D * 2 * rows
        f += (3 * case["rotary"] + (9 * D if case["norm"] != "none" else 0)) * rows
    return {"bytes": b, "flops": f}


# ----------------------------------------------------- definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return _exact_experts(s) if case["op"] == "experts" else _exact_heads(s)


def _exact_experts(s):
    """Slots one expert at a time, found by their number among the slots; None where a
    64-bit product of this size would take too long."""
    case, xs, w = s["case"], s["xs"], s["w"]
    if work(case)["flops"] > 8e12:
        return None
    P, E = xs.shape[0], case["experts"]
    owner = torch.searchsorted(s["offsets"][1:].long(), torch.arange(P, device=xs.device),
                               right=True)       # E for a slot of no pair
    kw = {"dtype": torch.float64, "device": xs.device}
    r = {"ys": torch.zeros(P, case["inner"], **kw)}
    train = case["kind"] == "train"
    if train:
        r["dxs"], r["dw"] = torch.zeros(P, case["hidden"], **kw), torch.zeros(w.shape, **kw)
    for e in owner.unique().tolist():
        if e == E:
            continue
        at = (owner == e).nonzero()[:, 0]
        we = w[e].double()
        r["ys"][at] = torch.einsum("sh,hf->sf", xs[at].double(), we)
        if train:
            dy = s["dys"][at].double()
            r["dxs"][at] = torch.einsum("sf,hf->sh", dy, we)
            r["dw"][e] = torch.einsum("sh,sf->hf", xs[at].double(), dy)
    return r


def _exact_heads(s):
    """As complex numbers: a pair is turned by a product with magnitude * e^(i p f)."""
    case, q, k = s["case"], s["q"], s["k"]
    B, T, Hq, D = q.shape
    R, how, dev = case["rotary"], SCALING[case["scaling"]] or {"kind": "none"}, q.device
    freq, size = [], 1.0
    for i in range(R // 2):
        f = math.exp(-2 * i / R * math.log(BASE))
        if how["kind"] == "linear":
            f /= how["factor"]
        elif how["kind"] == "base":
            f *= how["factor"] ** (-2 * i / (R - 2))
        elif how["kind"] == "parts":
            size = 1 + math.log(how["factor"]) / 10
            per = R / (2 * math.log(BASE))       # pairs per factor e of the wavelength
            first = max(0, math.floor(per * math.log(how["original_length"] / (64 * math.pi))))
            last = min(R - 1, math.ceil(per * math.log(how["original_length"] / (2 * math.pi))))
            x = min(1.0, max(0.0, (i - first) / max(last - first, 1e-3)))
            f = (1 - x) * f + x * f / how["factor"]
        elif how["kind"] == "bands":
            x = how["original_length"] / (2 * math.pi / f)
            if x < 1:
                f /= how["factor"]
            elif x <= 4:
                x = (x - 1) / 3
                f = x * f + (1 - x) * f / how["factor"]
        freq.append(f)
    if case["kind"] == "append":
        pos = torch.arange(-T, 0, device=dev) + s["lengths"].long()[:, None]
    else:
        pos = s["positions"].long()
    angle = pos.double()[:, :, None, None] * torch.tensor(freq, dtype=torch.float64, device=dev)
    turn = torch.polar(torch.full_like(angle, size), angle)

    def turned(z, by):
        out = z.clone()
        if case["layout"] == "half":
            y = torch.complex(z[..., :R // 2].contiguous(), z[..., R // 2:R].contiguous()) * by
            out[..., :R // 2], out[..., R // 2:R] = y.real, y.imag
        else:
            y = torch.complex(z[..., 0:R:2].contiguous(), z[..., 1:R:2].contiguous()) * by
            out[..., 0:R:2], out[..., 1:R:2] = y.real, y.imag
        return out

    def one(x, w, grad=None):
        x = x.double()
        inv = 1.0 if w is None else (x.square().sum(-1, keepdim=True) / D + EPS) ** -0.5
        y = turned(x if w is None else x * inv * w.double(), turn)
        if grad is None:
            return y, None, None
        g = turned(grad.double(), turn.conj())
        if w is None:
            return y, g, None
        n, u = x * inv, g * w.double()
        dx = inv * u - inv * n * torch.einsum("bthd,bthd->bth", u, n)[..., None] / D
        return y, dx, torch.einsum("bthd,bthd->d", g, n)

    q2, dq, dwq = one(q, s["wq"], s.get("dq"))
    k2, dk, dwk = one(k, s["wk"], s.get("dk"))
    if case["kind"] == "append":
        ck, cv = s["ck"].double(), s["cv"].double()
        for b, length in enumerate(_lengths(case)):
            new = min(T, length)
            ck[b, length - new:length] = k2[b, T - new:]
            cv[b, length - new:length] = s["v"][b, T - new:].double()
        return {"q": q2, "cache_k": ck, "cache_v": cv}
    r = {"q": q2, "k": k2}
    if case["kind"] == "train":
        r.update(dq=dq, dk=dk)
        if dwq is not None:
            r.update(dwq=dwq, dwk=dwk)
    return r
