"""Plain 64-bit forms of the run-time patterns, and the error that a kernel with
fp32 sums and one rounding to its output type may have.

u(T) is the type's unit roundoff (2^-8 bf16, 2^-11 fp16, 2^-24 fp32); fp32 sums
of n products are off by at most about n 2^-24 times the sum of magnitudes."""
import math

import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -126, torch.float16: 2.0 ** -24, torch.float32: 2.0 ** -126}
E32 = 2.0 ** -24


def close(got, want, tol, what=""):
    """|got - want| <= tol elementwise; infinities and NaN in the same places."""
    got, want = got.double(), want.double()
    fin = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN elsewhere"
    assert torch.equal(got[~fin & ~torch.isnan(want)], want[~fin & ~torch.isnan(want)]), what
    if not fin.any():
        return
    tol = tol.expand(want.shape) if isinstance(tol, torch.Tensor) else torch.full_like(want, tol)
    over = ((got - want).abs() - tol)[fin]
    worst = over.max().item()
    assert worst <= 0, f"{what}: {int((over > 0).sum())} of {over.numel()} outside, by up to {worst}"


# ------------------------------------------------------------------- routes
def routes(ids, E):
    """offsets, slots by sorting Python tuples."""
    T, k = ids.shape
    pairs = sorted((e, t, j) for t, row in enumerate(ids.tolist()) for j, e in enumerate(row)
                   if 0 <= e < E)
    slots = torch.full((T, k), -1, dtype=torch.int32)
    counts = [0] * (E + 1)
    for s, (e, t, j) in enumerate(pairs):
        slots[t, j] = s
        counts[e + 1] += 1
    return torch.tensor(counts).cumsum(0).to(torch.int32), slots


def matrix(slots, w):
    """The tokens x slots matrix, dense, fp64."""
    T, k = slots.shape
    R = torch.zeros(T, T * k, dtype=torch.float64, device=slots.device)
    t = torch.arange(T, device=slots.device)[:, None].expand(T, k)
    at = slots >= 0
    R[t[at], slots[at].long()] = w.double()[at]
    return R


# ------------------------------------------------------------------- blocks
def limits(lengths, B, Tq, Tk, causal):
    """Seen keys of each query: [B, Tq]."""
    L = torch.tensor([Tk] * B) if lengths is None else lengths.cpu().clamp(0, Tk)
    if not causal:
        return L[:, None].expand(B, Tq)
    return (L[:, None] - Tq + torch.arange(Tq) + 1).clamp(min=0)


def means(k, block, lengths):
    B, Tk, Hk, D = k.shape
    out = torch.zeros(B, -(-Tk // block), Hk, D, dtype=torch.float64, device=k.device)
    for b in range(B):
        L = Tk if lengths is None else max(0, min(Tk, int(lengths[b])))
        for c in range(-(-L // block)):
            out[b, c] = k[b, c * block:min(L, (c + 1) * block)].double().mean(0)
    return out


def select(q, m, n, block, Tk, lengths, causal):
    """Lists by sorting (-score, block) pairs in fp64, and the scores."""
    B, Tq, Hq, D = q.shape
    Hk = m.shape[2]
    lim = limits(lengths, B, Tq, Tk, causal).tolist()
    qs = q.double().view(B, Tq, Hk, Hq // Hk, D).sum(3)
    score = torch.einsum("bthd,bchd->bthc", qs, m.double()).cpu()
    lists = torch.full((B, Tq, Hk, n), -1, dtype=torch.int32)
    for b in range(B):
        for t in range(Tq):
            if not lim[b][t]:
                continue
            last = (lim[b][t] - 1) // block
            for h in range(Hk):
                row = score[b, t, h].tolist()
                rest = sorted(range(last if causal else last + 1),
                              key=lambda c: (-row[c] if row[c] == row[c] else math.inf, c))
                got = sorted(rest[:n - 1 if causal else n] + ([last] if causal else []))
                lists[b, t, h, :len(got)] = torch.tensor(got, dtype=torch.int32)
    return lists, score


def attend(q, k, v, blocks, block, lengths=None, causal=True, scale=None, grad=None):
    """Attention in fp64 over whole key rows under the selection's mask. Returns
    a dict with each result and, under "tol_" + name, its bound."""
    B, Tq, Hq, D = q.shape
    Tk, Hk = k.shape[1:3]
    G, dev, u = Hq // Hk, q.device, U[q.dtype]
    scale = 1 / math.sqrt(D) if scale is None else scale
    lim = limits(lengths, B, Tq, Tk, causal).to(dev)
    NB = -(-Tk // block)
    f64 = {"dtype": torch.float64, "device": dev}
    r = {"out": torch.zeros(B, Tq, Hq, D, **f64), "lse": torch.full((B, Tq, Hq), -math.inf, **f64)}
    names = ["out", "lse"]
    if grad is not None:
        r |= {"dq": torch.zeros(B, Tq, Hq, D, **f64), "dk": torch.zeros(B, Tk, Hk, D, **f64),
              "dv": torch.zeros(B, Tk, Hk, D, **f64)}
        names += ["dq", "dk", "dv"]
    for x in names:
        r["tol_" + x] = torch.zeros_like(r[x]).fill_(0)
    r["tol_lse"].fill_(0)
    key = torch.arange(Tk, device=dev)
    for b in range(B):
        for h in range(Hk):
            chosen = torch.zeros(Tq, NB + 1, dtype=torch.bool, device=dev)
            list_ = blocks[b, :, h].long()
            chosen.scatter_(1, torch.where(list_ >= 0, list_, NB), True)
            mask = chosen[:, :NB].repeat_interleave(block, 1)[:, :Tk] & (key < lim[b][:, None])
            used = mask.any(0)[:, None]
            # a key that no query sees may hold anything
            kb = torch.where(used, k[b, :, h].double(), 0.0)
            vb = torch.where(used, v[b, :, h].double(), 0.0)
            for g in range(G):
                i = h * G + g
                qb = q[b, :, i].double()
                # rows that see nothing may hold anything too
                some = mask.any(1)[:, None]
                s = (scale * qb @ kb.T).masked_fill(~mask, -math.inf)
                lse = torch.logsumexp(s, 1)
                p = torch.where(some & mask, torch.exp(s - torch.where(some[:, 0], lse, 0.0)[:, None]), 0.0)
                out = p @ vb
                r["out"][b, :, i], r["lse"][b, :, i] = out, lse
                # the score's error, times 2 for p and its normaliser, and exp2's own
                mag = (abs(scale) * (qb.abs() @ kb.abs().T)).masked_fill(~mask, 0.0)
                e = ((D + 8) * 2 * E32 * mag).amax(1, keepdim=True) + 2.0 ** -20
                pv = p @ vb.abs()
                tol_out = u * out.abs() + (u + 2 * e) * pv + TINY[q.dtype]
                r["tol_out"][b, :, i] = tol_out
                fl = torch.where(some[:, 0], lse, 0.0)
                r["tol_lse"][b, :, i] = e[:, 0] + 4 * E32 * (fl.abs() + 1)
                if grad is None:
                    continue
                do = torch.where(some, grad[b, :, i].double(), 0.0)
                qz = torch.where(some, qb, 0.0)
                dp = do @ vb.T
                delta = (do * out).sum(1, keepdim=True)
                ds = scale * p * (dp - delta)
                r["dv"][b, :, h] += p.T @ do
                r["dq"][b, :, i] = ds @ kb
                r["dk"][b, :, h] += ds.T @ qz
                r["tol_dv"][b, :, h] += (p * (u + 2 * e)).T @ do.abs()
                e_dp = 2 * D * E32 * (do.abs() @ vb.abs().T)
                e_delta = (do.abs() * tol_out).sum(1, keepdim=True) \
                    + 2 * D * E32 * (do * out).abs().sum(1, keepdim=True)
                e_ds = abs(scale) * p * ((u + 2 * e) * (dp - delta).abs() + e_dp + e_delta)
                r["tol_dq"][b, :, i] = u * r["dq"][b, :, i].abs() + e_ds @ kb.abs() + TINY[q.dtype]
                r["tol_dk"][b, :, h] += e_ds.T @ qz.abs()
    if grad is not None:
        for x in ("dk", "dv"):
            r["tol_" + x] += u * r[x].abs() + TINY[q.dtype]
    return r
