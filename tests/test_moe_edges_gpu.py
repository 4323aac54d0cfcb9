"""Router and activation where an exponential leaves fp32: sigmoid scores of very negative logits, gates below -87.

Tolerances, from the arithmetic:
* router weights: the argument v - top of the exponential is off by half an ulp (2^-24 of its size), expf is within
  2 ulp, and a sum over the choices, quotients and the scale come to at most 12 more roundings: (|v - top| + 16) * 2^-23
  relative. A sigmoid below 2^-126 is subnormal: off by up to 4 * 2^-149, over a sum of at least e^-18: 4e-37.
* activation: expf within 2 ulp and three roundings, 2^-20 relative (fp32 result); the approximate exponential is
  within 2 + 1.173 |g| ulp (CUDA's documented bound), the quotient 2, two roundings: (6 + 1.2 |g|) * 2^-23, plus 2^-8
  for the rounding to bf16. Below -87.3 the exponential is subnormal, off by up to 4 * 2^-149, and the gate's product
  with it rounds to a multiple of 2^-149: |up| * |g| * 2^-146. A subnormal result: 2^-133 (bf16), 2^-148 (fp32)."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def f64(t):
    return t.detach().double().cpu().numpy()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("E", [16, 64, 512])
def test_sigmoid_of_very_negative_logits(lib, dt, E):
    topk = 8
    tops = [3.0, -10.0, -17.0, -17.9, -18.1, -30.0, -80.0, -87.0, -89.0, -95.0, -103.0, -104.0, -120.0, -1000.0, -3e38]
    g = torch.Generator(device="cuda").manual_seed(E)
    z = torch.empty(2 * len(tops), E, device="cuda")
    for i, t in enumerate(tops):
        for j, spread in enumerate((6.0, 90.0)):
            z[2 * i + j] = t - spread * torch.rand(E, device="cuda", generator=g)
            z[2 * i + j, E // 3] = t
    z = z.to(DT[dt])
    v = f64(z)
    ids = np.argsort(-v, axis=1, kind="stable")[:, :topk]
    v = np.take_along_axis(v, ids, 1)
    ls = np.where(v < 0, v - np.log1p(np.exp(np.minimum(v, 0))), -np.log1p(np.exp(-np.maximum(v, 0))))  # log sigmoid
    for renorm in (True, False):
        got_ids, w = lib.moe_route(z, topk, score="sigmoid", renormalize=renorm, scale=1.0)
        assert np.array_equal(got_ids.cpu().numpy(), ids)
        ref = np.exp(ls - ls[:, :1]) if renorm else np.exp(ls)
        if renorm:
            ref /= ref.sum(1, keepdims=True)
            assert (np.abs(f64(w).sum(1) - 1) <= 1e-5).all()
        rel = (np.minimum(np.abs(v - v[:, :1]), 200) + 16) * 2.0 ** -23
        assert (np.abs(f64(w) - ref) <= rel * ref + 4e-37).all(), (renorm, np.abs(f64(w) - ref).max(1))


@pytest.mark.parametrize("ydt,hdt", [("bf16", "bf16"), ("f32", "bf16"), ("f32", "f32"), ("bf16", "f32")])
def test_gates_below_the_exponentials_range(lib, ydt, hdt):
    ups = torch.tensor([1.0, -2.5, 1e10, 1e30, -3e35], device="cuda")
    inter = 256
    gate = torch.cat([torch.linspace(-110, -80, inter - 64, device="cuda"), torch.linspace(-80, 90, 64, device="cuda")])
    y = torch.cat([gate.expand(5, inter), ups[:, None].expand(5, inter) * torch.linspace(0.5, 1, inter, device="cuda")], 1)
    y = y.to(DT[ydt]).contiguous()
    h = lib.moe_act(y, torch.full((5, inter), float("nan"), dtype=DT[hdt], device="cuda"))
    v = f64(y)
    g, u = v[:, :inter], v[:, inter:]
    ref = g / (1 + np.exp(-g)) * u
    rel = 2.0 ** -8 + (6 + 1.2 * np.abs(g)) * 2.0 ** -23 if hdt == "bf16" else 2.0 ** -20
    tol = rel * np.abs(ref) + np.abs(u * g) * np.where(g < -87, 2.0 ** -146, 0) + (2.0 ** -133 if hdt == "bf16" else 2.0 ** -148)
    fits = np.abs(ref) < 3e38
    bad = (np.abs(f64(h) - ref) > tol) & fits
    assert not bad.any(), f"{int(bad.sum())} off, gates {np.unique(g[bad])[:8]}"
    c, s = lib.moe_act_mx4(y, *lib.mx4_buffers(5, inter))
    rc, rs = lib.mx4_quantize(lib.moe_act(y, torch.empty(5, inter, dtype=torch.bfloat16, device="cuda")))
    assert torch.equal(c, rc) and torch.equal(s[:, :inter // 32], rs[:, :inter // 32])
