"""Norm and rotation of heads on the GPU against the formulas in 64 bits.

Bounds (E = 2^-24, D elements): sines and cosines are off by at most 4 E (their
rounding, two units of the function and an angle within 2^-27 of pi), a norm's factor by
(D / 2 + 8) E of itself, and each product and sum by its rounding; a result is rounded to
its type once."""
import math
from decimal import Decimal, getcontext

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

import dynamic_ref as ref  # noqa: E402

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-5


@pytest.fixture(scope="module")
def sdm(cuda_device):
    import sparse_dense_matrix_gb300 as m
    return m


def randn(dev, seed, *shape):
    g = torch.Generator(device=dev).manual_seed(seed)
    return torch.randn(*shape, generator=g, device=dev)


def turned(z, cos, sin, R, layout):
    """The pairs of z [B, T, heads, D] turned by cos, sin [B, T, 1, R / 2]."""
    out = z.clone()
    a, b = ((slice(0, R // 2), slice(R // 2, R)) if layout == "half"
            else (slice(0, R, 2), slice(1, R, 2)))
    out[..., a] = z[..., a] * cos - z[..., b] * sin
    out[..., b] = z[..., b] * cos + z[..., a] * sin
    return out


U, TINY = {**ref.U, torch.float64: 0.0}, {**ref.TINY, torch.float64: 0.0}


def formula(rot, x, w, pos, grad=None):
    """[(y, tolerance)], and with grad those of dx and dw, in 64 bits."""
    D, R, dt = rot.dim, rot.rotary_dim, x.dtype
    angle = pos.double()[..., None, None] * torch.tensor(rot.frequencies, dtype=torch.float64,
                                                         device=x.device)
    cos, sin = rot.magnitude * torch.cos(angle), rot.magnitude * torch.sin(angle)
    ones = torch.full_like(cos, abs(rot.magnitude))
    x = x.double()
    r = 1.0 if w is None else (x.square().mean(-1, keepdim=True) + EPS) ** -0.5
    n = x * r
    z = n if w is None else n * w.double()
    y = turned(z, cos, sin, R, rot.layout)

    def mag(z):                                  # what the terms of a turned element add up to
        return turned(z.abs(), ones, -ones, R, rot.layout).abs().maximum(
            turned(z.abs(), ones, ones, R, rot.layout).abs())

    # angles: the tests' own products p f are off by p 2^-52 of f
    e = (8 + (0 if w is None else D / 2 + 10)) * ref.E32 + \
        (pos.abs().max().item() if pos.numel() else 0) * 2.0 ** -51
    out = [(y, U[dt] * y.abs() + e * mag(z) + TINY[dt])]
    if grad is None:
        return out
    g = turned(grad.double(), cos, -sin, R, rot.layout)
    gm = mag(grad.double())
    if w is None:
        return out + [(g, U[dt] * g.abs() + e * gm + TINY[dt])]
    u, um = g * w.double(), gm * w.double().abs()
    dx = r * (u - n * (u * n).mean(-1, keepdim=True))
    rest = r * (um + n.abs() * (um * n.abs()).mean(-1, keepdim=True))
    out.append((dx, U[dt] * dx.abs() + (2 * e + (2 * D + 8) * ref.E32) * rest + TINY[dt]))
    rows = x[..., 0].numel()
    dw, dwm = ((a * n_).sum((0, 1, 2)) for a, n_ in ((g, n), (gm, n.abs())))
    out.append((dw, U[w.dtype] * dw.abs() + (e + rows * ref.E32) * dwm + TINY[w.dtype]))
    return out


def rotation(sdm, dev, D, R=None, layout="half", **kw):
    return sdm.HeadRotation(D, R, layout=layout, device=dev, **kw)


SHAPES = [  # B, T, Hq, Hk, D, R
    (1, 1, 1, 1, 16, 16), (1, 1, 16, 4, 64, 64), (64, 1, 32, 4, 128, 128), (3, 33, 12, 4, 64, 32),
    (2, 17, 3, 3, 80, 80), (1, 100, 8, 2, 96, 48), (2, 5, 4, 0, 192, 16), (2, 50, 7, 1, 256, 256),
    (1, 700, 16, 2, 128, 64), (5, 3, 2, 6, 48, 0), (1, 9, 33, 17, 32, 32), (4, 777, 4, 4, 64, 64)]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("norm", ["none", "same", "fp32", "one"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("B,T,Hq,Hk,D,R", SHAPES)
def test_rotate_and_gradients(sdm, cuda_device, B, T, Hq, Hk, D, R, layout, norm, dtype):
    dt, dev = DT[dtype], cuda_device
    rot = rotation(sdm, dev, D, R, layout, base=1e4)
    # views of one projection
    qkv = randn(dev, T, B, T, Hq + 2 * Hk, D).to(dt)
    q, k = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hk]
    gq, gk = randn(dev, 2, B, T, Hq, D).to(dt), randn(dev, 3, B, T, Hk, D).to(dt)
    wq = wk = None
    if norm != "none":
        wt = torch.float32 if norm == "fp32" else dt
        wq, wk = ((1 + 0.25 * randn(dev, i, D)).to(wt) for i in (4, 5))
        if norm == "one":
            wq = None
    if not Hk:
        k = gk = wk = None
    pos = torch.randint(-50, 1 << 17, (B, T), generator=torch.Generator().manual_seed(1)).to(
        dev, torch.int32)
    args = dict(positions=pos, q_weight=wq, k_weight=wk, eps=EPS)
    q2, k2 = rot.rotate(q, k, **args)
    dq, dk, dwq, dwk = rot.rotate_backward(gq, gk, q if wq is not None else None,
                                           k if wk is not None else None, **args)
    for x, w, g, got in ((q, wq, gq, (q2, dq, dwq)), (k, wk, gk, (k2, dk, dwk))):
        if x is None:
            assert got[0] is None and got[1] is None
            continue
        want = formula(rot, x, w, pos, g)
        for name, a, (b, tol) in zip(("y", "dx", "dw"), got, want):
            assert a.dtype == (w.dtype if name == "dw" else dt) and a.is_contiguous()
            ref.close(a, b, tol, name)
        assert w is not None or got[2] is None


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("B,T,Tk,Hq,Hk,D,R", [
    (1, 1, 1, 4, 1, 64, 64), (17, 1, 300, 8, 2, 128, 128), (3, 40, 64, 6, 3, 80, 32),
    (2, 5, 3, 2, 2, 16, 16), (4, 260, 300, 3, 1, 256, 64)])
def test_append(sdm, cuda_device, B, T, Tk, Hq, Hk, D, R, dtype, norm, layout):
    dt, dev = DT[dtype], cuda_device
    rot = rotation(sdm, dev, D, R, layout, scaling={"kind": "linear", "factor": 2.0})
    qkv = randn(dev, T, B, T, Hq + 2 * Hk, D).to(dt)
    q, k, v = qkv.split([Hq, Hk, Hk], dim=2)
    w = (1 + 0.25 * randn(dev, 4, D)) if norm else None
    # free slots, sequences shorter than the call's tokens, one past the cache's rows
    lengths = [0, Tk, T // 2, Tk + 2, 1][:B] + [1 + 7919 * b % Tk for b in range(5, B)]
    L = torch.tensor(lengths, dtype=torch.int32, device=dev)
    # the caches are views with rows around them
    room = [randn(dev, 6 + i, B, Tk + 3, Hk + 1, D).to(dt) for i in range(2)]
    before = [r.clone() for r in room]
    ck, cv = (r[:, 1:Tk + 1, :Hk] for r in room)
    q2 = rot.append(q, k, v, ck, cv, L, q_weight=w, k_weight=w, eps=EPS)
    pos = L[:, None] - T + torch.arange(T, device=dev)
    (want, tol), = formula(rot, q, w, pos)
    ref.close(q2, want, tol, "q")
    (want, tol), = formula(rot, k, w, pos)
    for b in range(B):
        for t in range(T):
            p = lengths[b] - T + t
            if 0 <= p < Tk:
                ref.close(room[0][b, 1 + p, :Hk], want[b, t], tol[b, t], "key")
                assert torch.equal(room[1][b, 1 + p, :Hk], v[b, t])
                for r, old in zip(room, before):
                    r[b, 1 + p, :Hk] = old[b, 1 + p, :Hk]
    assert all(torch.equal(r, old) for r, old in zip(room, before)), "another row was written"
    # the same queries as rotate's, which takes lengths too
    assert torch.equal(q2, rot.rotate(q, lengths=L, q_weight=w, eps=EPS)[0])


def test_positions(sdm, cuda_device):
    """No positions, one row of them for all sequences, strided ones, and lengths agree."""
    B, T, D, dev = 3, 20, 64, cuda_device
    rot = rotation(sdm, dev, D)
    q = randn(dev, 1, B, T, 4, D).bfloat16()
    at = torch.arange(T, dtype=torch.int32, device=dev)
    want = rot.rotate(q)[0]
    assert torch.equal(want, rot.rotate(q, positions=at)[0])
    assert torch.equal(want, rot.rotate(q, positions=at.expand(B, T))[0])
    assert torch.equal(want, rot.rotate(q, positions=at[:, None].expand(T, B).contiguous().t())[0])
    assert torch.equal(want, rot.rotate(q, lengths=torch.full((B,), T, dtype=torch.int32,
                                                              device=dev))[0])
    two = torch.stack([at + 1000, at], 1).repeat(B, 1, 1)
    assert torch.equal(want, rot.rotate(q, positions=two[:, :, 1])[0])


@pytest.mark.parametrize("scaling", [
    None, {"kind": "linear", "factor": 8.0}, {"kind": "base", "factor": 4.0},
    {"kind": "parts", "factor": 16.0, "original_length": 4096},
    {"kind": "parts", "factor": 4.0, "original_length": 2048, "fast": 16.0, "slow": 2.0,
     "magnitude": 1.0},
    {"kind": "bands", "factor": 8.0, "original_length": 8192},
    {"kind": "bands", "factor": 8.0, "original_length": 8192, "fast": 8.0, "slow": 2.0}])
def test_far_positions(sdm, cuda_device, scaling):
    """Angles of far positions against 50 digits."""
    getcontext().prec = 50
    pi = Decimal("3.14159265358979323846264338327950288419716939937510")
    D, dev = 32, cuda_device
    rot = rotation(sdm, dev, D, base=5e5, scaling=scaling)
    for p in (1, 4095, 131071, 16777215, -999999):
        q = torch.zeros(1, 1, 2, D, device=dev)
        q[0, 0, 0, :D // 2] = 1                  # gives (cos, sin); the other head (-sin, cos)
        q[0, 0, 1, D // 2:] = 1
        pos = torch.full((1, 1), p, dtype=torch.int32, device=dev)
        got = rot.rotate(q, positions=pos)[0][0, 0].double().cpu()
        for i in range(D // 2):
            angle = Decimal(rot.frequencies[i]) * p
            rest = float(angle - (angle / (2 * pi)).to_integral_value() * 2 * pi)
            c, s = rot.magnitude * math.cos(rest), rot.magnitude * math.sin(rest)
            # the frequency in turns is that of a 64-bit division
            tol = rot.magnitude * (6 * ref.E32 + abs(p) * 2.0 ** -52 * rot.frequencies[i])
            for x, want in ((got[0, i], c), (got[0, D // 2 + i], s), (got[1, i], -s),
                            (got[1, D // 2 + i], c)):
                assert abs(x.item() - want) <= tol, (p, i)


def test_given_frequencies(sdm, cuda_device):
    f = [0.0, 1.0, 2.5, 1e-3, 7.0, 0.25, 100.0, -1.0]
    rot = rotation(sdm, cuda_device, 64, 16, "interleaved", frequencies=f, magnitude=0.5)
    q = randn(cuda_device, 1, 2, 30, 3, 64)
    pos = torch.arange(30, device=cuda_device).expand(2, 30)
    (want, tol), = formula(rot, q, None, pos)
    ref.close(rot.rotate(q)[0], want, tol)


def test_gradients_against_differences(sdm, cuda_device):
    """Central differences of the formula in 64 bits, on values that fp32 holds."""
    B, T, H, D, dev = 2, 3, 2, 32, cuda_device
    rot = rotation(sdm, dev, D, 16, "interleaved", base=100.0)
    q, g = randn(dev, 1, B, T, H, D), randn(dev, 2, B, T, H, D)
    w = 1 + 0.25 * randn(dev, 3, D)
    pos = torch.randint(0, 99, (B, T), generator=torch.Generator().manual_seed(1)).to(
        dev, torch.int32)
    dq, _, dw, _ = rot.rotate_backward(g, None, q, positions=pos, q_weight=w, eps=EPS)

    def loss(q, w):
        return (formula(rot, q, w, pos)[0][0] * g.double()).sum().item()

    h = 2.0 ** -12
    q, w = q.double(), w.double()
    # the third derivatives of a normed row are below 100: h^2 / 6 of them, and fp32's own error
    for t, d in ((q, dq), (w, dw)):
        flat = t.view(-1)
        for i in range(0, t.numel(), 5):
            x = flat[i].item()
            flat[i] = x + h
            up = loss(q, w)
            flat[i] = x - h
            down = loss(q, w)
            flat[i] = x
            assert abs((up - down) / (2 * h) - d.view(-1)[i].item()) <= 100 * h * h + 1e-4


def test_odd_values(sdm, cuda_device):
    """Rows of zeros, huge and tiny rows, and NaN or infinity in one row."""
    rot = rotation(sdm, cuda_device, 64)
    q = randn(cuda_device, 1, 1, 8, 4, 64)
    w = 1 + 0.25 * randn(cuda_device, 2, 64)
    clean = rot.rotate(q, q_weight=w, eps=EPS)[0]
    q[0, 1, 1] = 0
    q[0, 2, 2] *= 1e15
    q[0, 3, 3] *= 1e-25
    q[0, 4, 0, 5] = float("nan")
    q[0, 5, 1, 7] = float("inf")
    got = rot.rotate(q, q_weight=w, eps=EPS)[0]
    assert not got[0, 1, 1].any()
    pos = torch.arange(8, device=cuda_device)[None]
    (want, tol), = formula(rot, q, w, pos)
    ok = torch.ones(8, 4, dtype=torch.bool, device=cuda_device)
    ok[4, 0] = ok[5, 1] = False
    ref.close(got[0][ok], want[0][ok], tol[0][ok])
    assert torch.isnan(got[0, 4, 0]).all()
    assert torch.isnan(got[0, 5, 1]).any() and not torch.isnan(got[0, 5, 2]).any()
    same = torch.ones(8, 4, dtype=torch.bool, device=cuda_device)
    for t, h in ((1, 1), (2, 2), (3, 3), (4, 0), (5, 1)):
        same[t, h] = False
    assert torch.equal(got[0][same], clean[0][same])


def test_past_32_bit_offsets(sdm, cuda_device):
    """A cache and rows of more than 2^31 elements."""
    B, Tk, Hk, D, dt, dev = 3, 1 << 16, 64, 256, torch.bfloat16, cuda_device
    rot = rotation(sdm, dev, D)
    q, k, v = (randn(dev, i, B, 1, Hk, D).to(dt) for i in range(3))
    ck, cv = (torch.zeros(B, Tk, Hk, D, dtype=dt, device=dev) for _ in range(2))
    L = torch.tensor([1, Tk, Tk - 5], dtype=torch.int32, device=dev)
    rot.append(q, k, v, ck, cv, L)
    k2 = rot.rotate(k, lengths=L)[0]
    for b in range(B):
        p = int(L[b]) - 1
        assert torch.equal(ck[b, p], k2[b, 0]) and torch.equal(cv[b, p], v[b, 0])
        ck[b, p] = cv[b, p] = 0
    assert not ck.any() and not cv.any()
    del ck, cv
    q = torch.zeros(1, 1 << 17, 72, 256, dtype=dt, device=dev)     # 2.4e9 elements
    last = randn(dev, 9, 72, 256).to(dt)
    q[0, -1] = last
    got = rot.rotate(q)[0]
    one = rot.rotate(last[None, None], positions=torch.tensor([(1 << 17) - 1], dtype=torch.int32,
                                                              device=dev))[0]
    assert torch.equal(got[0, -1], one[0, 0])
    got[0, -1] = 0
    assert not got.any()


def test_empty(sdm, cuda_device):
    rot = rotation(sdm, cuda_device, 64)
    w = torch.ones(64, device=cuda_device)
    for B, T, H in ((0, 3, 2), (2, 0, 2), (2, 3, 0)):
        q = torch.ones(B, T, H, 64, device=cuda_device)
        q2, k2 = rot.rotate(q, q, q_weight=w)
        assert q2.shape == q.shape and k2.shape == q.shape
        dq, dk, dwq, dwk = rot.rotate_backward(q, q, q, q, q_weight=w, k_weight=w)
        assert dq.shape == q.shape and not dwq.any() and not dwk.any()
    # a cache without rows takes nothing
    q = torch.ones(2, 1, 2, 64, device=cuda_device)
    none = q.new_empty(2, 0, 2, 64)
    L = torch.ones(2, dtype=torch.int32, device=cuda_device)
    assert rot.append(q, q, q, none, none, L).shape == q.shape


def test_reproducible_streams_and_graph(sdm, cuda_device):
    B, T, Hq, Hk, D, dev = 2, 300, 8, 2, 128, cuda_device
    rot = rotation(sdm, dev, D)
    q, k, v, gq, gk = (randn(dev, i, B, T, H, D).bfloat16()
                       for i, H in enumerate((Hq, Hk, Hk, Hq, Hk)))
    wq, wk = (1 + 0.25 * randn(dev, i, D) for i in (7, 8))
    L = torch.tensor([T, T + 40], dtype=torch.int32, device=dev)
    ck, cv = (torch.zeros(B, 400, Hk, D, dtype=q.dtype, device=dev) for _ in range(2))
    norm = dict(lengths=L, q_weight=wq, k_weight=wk)

    def step(**kw):
        ck.zero_()
        out = rot.append(q, k, v, ck, cv, L, wq, wk, **kw)
        return [out, ck.clone(), *rot.rotate(q, k, **norm, **kw),
                *rot.rotate_backward(gq, gk, q, k, **norm, **kw)]

    want = step()
    assert torch.equal(want[1][0, :T], want[3][0])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        got = step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    got = [*rot.rotate(q, k, **norm, stream=side),
           *rot.rotate_backward(gq, gk, q, k, **norm, stream=side)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want[2:], got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    q.mul_(2)
    L.sub_(7)
    graph.replay()
    torch.cuda.synchronize()
    again = step()
    assert all(torch.equal(a, b) for a, b in zip(again, got))


def test_rotated_and_attended(sdm, cuda_device):
    """Rotation before the selection and the attention: a prompt in one call, and its last
    tokens one at a time over a cache, give the same."""
    B, T, Hq, Hk, D, block, n, dev = 2, 70, 4, 2, 64, 16, 3, cuda_device
    rot = rotation(sdm, dev, D)
    qkv = randn(dev, 1, B, T, Hq + 2 * Hk, D).bfloat16()
    q, k, v = qkv.split([Hq, Hk, Hk], dim=2)
    wq, wk = (1 + 0.25 * randn(dev, i, D) for i in (7, 8))
    q2, k2 = rot.rotate(q, k, q_weight=wq, k_weight=wk)
    sel = sdm.select_blocks(q2, sdm.block_means(k2, block), n, block, T)
    out, _ = sel.attend(q2, k2, v)
    ck, cv = (torch.zeros(B, 96, Hk, D, dtype=q.dtype, device=dev) for _ in range(2))
    L = torch.zeros(B, dtype=torch.int32, device=dev)
    means = sdm.block_means(ck, block, L)
    for t0, t1 in ((0, 60), *((t, t + 1) for t in range(60, T))):
        L += t1 - t0
        qt = rot.append(q[:, t0:t1], k[:, t0:t1], v[:, t0:t1], ck, cv, L, wq, wk)
        assert torch.equal(qt, q2[:, t0:t1])
        sdm.block_means(ck, block, L, out=means, new_keys=t1 - t0)
        sel1 = sdm.select_blocks(qt, means, n, block, 96, L)
        assert torch.equal(sel1.blocks, sel.blocks[:, t0:t1])
        one, _ = sel1.attend(qt, ck, cv)
        # the weights are rounded to bf16 in either form: three roundings of values up to v's
        assert (one.float() - out[:, t0:t1].float()).abs().max() <= 3 * 2.0 ** -8 * v.abs().max()
    assert torch.equal(ck[:, :T], k2) and torch.equal(cv[:, :T], v)


def test_refusals(sdm, cuda_device):
    dev = cuda_device
    rot = rotation(sdm, dev, 64)
    q = torch.ones(2, 3, 4, 64, dtype=torch.bfloat16, device=dev)
    k = torch.ones(2, 3, 2, 64, dtype=torch.bfloat16, device=dev)
    pos = torch.zeros(2, 3, dtype=torch.int32, device=dev)
    L = torch.zeros(2, dtype=torch.int32, device=dev)
    w = torch.ones(64, device=dev)
    c = torch.zeros(2, 8, 2, 64, dtype=torch.bfloat16, device=dev)
    for args, kw in (
            ((q.cpu(),), {}), ((q.double(),), {}), ((q[0],), {}), ((q[..., :48],), {}),
            ((q[..., ::2],), {}), ((q, k.half()), {}), ((q, k[:, :2]), {}),
            ((q,), {"positions": pos.long()}), ((q,), {"positions": pos[:, :2]}),
            ((q,), {"positions": pos, "lengths": L}), ((q,), {"lengths": L[:1]}),
            ((q,), {"lengths": L.long()}), ((q,), {"q_weight": w[:32]}),
            ((q,), {"q_weight": w.half()}), ((q,), {"k_weight": w}), ((q,), {"positions": 3}),
            ((q, k), {"q_weight": w, "k_weight": w.bfloat16()}),
            ((q,), {"q_weight": torch.ones(65, device=dev)[1:]})):
        with pytest.raises((ValueError, TypeError)):
            rot.rotate(*args, **kw)
    for args in ((q, None, k, c, c, L), (q, k, k, c, c, None), (q, k, k[:, :2], c, c, L),
                 (q, k, k, c[:1], c, L), (q, k, k, c, c[:, :4], L), (q, k, k, c.half(), c, L),
                 (q, k, k, c[:, :1].expand(2, 8, 2, 64), c, L), (q, k, k, c, c[:1].expand(c.shape), L)):
        with pytest.raises((ValueError, TypeError)):
            rot.append(*args)
    for args, kw in (((q, None), {"q_weight": w}), ((q, k, q), {"k_weight": w}),
                     ((q, k, q[:, :2]), {"q_weight": w})):
        with pytest.raises((ValueError, TypeError)):
            rot.rotate_backward(*args, **kw)
