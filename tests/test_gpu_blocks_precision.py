"""The gradients' dS is used as its rounded value plus what that left out. On inputs whose
sums cancel (keys with a common part, pairs of heads with nearly opposite gradients) one
rounded dS alone is off by several times what rounding the result costs; with both parts
the result's own rounding is nearly all that is left.

Bounds: a part that is off by u of itself costs c u of a result that is 1 / c of its
terms, c = 8 here, so one part gives an error of about c times the result's rounding, and
two parts, off by u^2, of c u times it: 1 + 0.001 or less with it. The limit of 2 lies
between; that one part would not pass is checked on the 64-bit form."""
import math

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def rms(x):
    return x.double().square().mean().sqrt().item()


@pytest.mark.parametrize("dtype,D,block,T", [
    ("bf16", 64, 64, 16), ("bf16", 128, 16, 16), ("fp16", 128, 64, 16),        # by query
    ("bf16", 64, 32, 1000), ("bf16", 128, 16, 1000), ("fp16", 64, 16, 1000),   # by tile
    ("fp16", 128, 64, 1000), ("fp16", 64, 128, 1000),
    ("bf16", 64, 64, 1000), ("bf16", 64, 128, 1000), ("bf16", 128, 64, 1000),  # on tcgen05
    ("bf16", 128, 128, 1000)])
def test_gradients_where_sums_cancel(cuda_device, dtype, D, block, T):
    import sparse_dense_matrix_gb300 as sdm
    B, Tk, Hq, dt = 4, 1000, 2, DT[dtype]
    g = torch.Generator(device=cuda_device).manual_seed(D + block)
    rnd = lambda *s: torch.randn(*s, generator=g, device=cuda_device)  # noqa: E731
    q = rnd(B, T, 1, D).to(dt).expand(B, T, Hq, D).contiguous()
    k = (rnd(B, Tk, 1, D) + 8 * rnd(D).sign()).to(dt)
    v, grad = rnd(B, Tk, 1, D).to(dt), rnd(B, T, Hq, D)
    grad[:, :, 1] = -grad[:, :, 0] + grad[:, :, 1] / 8
    grad = grad.to(dt)
    NB, n = -(-Tk // block), 512 // block
    blocks = torch.rand(B, T, 1, NB, generator=g, device=cuda_device).argsort(-1)[..., :n]
    blocks = blocks.sort(-1).values.to(torch.int32).contiguous()
    sel = sdm.BlockSelection(blocks, block, Tk, causal=False)
    out, lse = sel.attend(q, k, v)
    dq, dk, _ = sel.backward(grad, q, k, v, out, lse)

    # the formula in 64 bits, from the same rounded out and lse
    mask = torch.zeros(B, T, NB, dtype=torch.bool, device=cuda_device)
    mask.scatter_(2, blocks[:, :, 0].long(), True)
    mask = mask.repeat_interleave(block, 2)[:, None, :, :Tk]
    x = {"q": q, "k": k, "v": v, "g": grad, "o": out}
    x = {a: t.double().transpose(1, 2) for a, t in x.items()}           # [B, heads, T, D]
    scale = 1 / math.sqrt(D)
    p = torch.exp(scale * x["q"] @ x["k"].mT - lse.double().transpose(1, 2)[..., None])
    delta = (x["g"] * x["o"]).sum(-1, keepdim=True)
    ds = torch.where(mask, scale * p * (x["g"] @ x["v"].mT - delta), 0.0)

    def products(ds):
        return {"dq": (ds @ x["k"]).transpose(1, 2),
                "dk": (ds.mT @ x["q"]).sum(1, keepdim=True).transpose(1, 2)}

    exact = products(ds)
    unit = 2.0 ** torch.floor(torch.log2(ds.abs().max()))               # fp16's range is not meant
    one_part = products((ds / unit).to(dt).double() * unit)
    for name, got in (("dq", dq), ("dk", dk)):
        floor = rms(exact[name].to(dt).double() - exact[name])
        assert rms(one_part[name] - exact[name]) > 4 * floor, name      # the test can tell
        ratio = rms(got.double() - exact[name]) / floor
        print(f"{name}: {ratio:.3f} times the rounding, one part "
              f"{rms(one_part[name] - exact[name]) / floor:.1f}")
        assert ratio <= 2, name
    sdm.dynamic_sync()
