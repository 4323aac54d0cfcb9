"""examples/moe_layer.py end to end against the layer's formula in float64: router, experts' products, adapters,
activation and weighted sum together, with and without expert parallelism, adapters and 4-bit weights.

Tolerance on the relative 2-norm. In bf16 the values of y13 are rounded twice (product, delta), h once and y2 twice,
each within 2^-9: 5 * 2^-9 with a gate sensitivity below 2 gives 2e-2. With 4-bit weights h goes through the 4-bit
grid: an h off by 2^-8 lands on the neighbouring code (a step of about a quarter) for about 1.6 % of the elements,
sqrt(0.016) * 0.25 = 3e-2 more, 6e-2 together."""
import importlib.util
import os

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location("moe_layer_example", os.path.join(ROOT, "examples", "moe_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _mx(lib, v):
    """What the 4-bit format keeps of v (float64 in and out; bf16 values)."""
    t = torch.from_numpy(np.ascontiguousarray(v)).cuda().reshape(-1, v.shape[-1]).to(torch.bfloat16)
    c, s = lib.mx4_quantize(t)
    return lib.mx4_dequantize(c, s, torch.empty(t.shape, device="cuda")).double().cpu().numpy().reshape(v.shape)


@pytest.mark.parametrize("mx4", [False, True])
@pytest.mark.parametrize("loras", [0, 2])
@pytest.mark.parametrize("T,E,L,K", [(1, 8, 8, 2), (45, 12, 6, 4), (400, 6, 6, 3)])
def test_layer(lib, T, E, L, K, loras, mx4):
    H, I, R = 256, 160, 16
    g = torch.Generator(device="cuda").manual_seed(T + loras)
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=g).to(torch.bfloat16)  # noqa: E731
    f64 = lambda t: t.double().cpu().numpy()                                          # noqa: E731
    emap = None
    first = E - L                                     # this rank holds the last L experts
    if L < E:
        emap = torch.full((E,), -1, dtype=torch.int32, device="cuda")
        emap[first:] = torch.arange(L, dtype=torch.int32, device="cuda")
    w13, w2 = rnd(L, 2 * I, H) * H ** -0.5, rnd(L, H, I) * I ** -0.5
    layer = _example().MoELayer(w13, w2, E, K, T + 5, emap, loras, R, mx4)
    ads = {}
    for s in range(1, loras + 1):
        for e in range(L):
            ads[s, e] = [rnd(H, R) / 16, rnd(H, R) / 16, rnd(R, I) / 4, rnd(R, I) / 4, rnd(I, R) / 16, rnd(R, H) / 4]
            ag, au, bg, bu, a2, b2 = ads[s, e]
            layer.set_adapter(s, e, R, 0.5, [ag, au], [bg, bu], a2, b2)
    x, z = rnd(T, H), torch.randn(T, E, device="cuda", generator=g)
    slot = torch.randint(0, loras + 1, (T,), dtype=torch.int32, device="cuda", generator=g)
    if loras:
        slot[0] = 1
    out = torch.full((T, H), float("nan"), dtype=torch.bfloat16, device="cuda")
    layer(x, z, out, slot if loras else None)
    torch.cuda.synchronize()
    assert lib.lora_query_status(layer.meta.c) == (lib.LORA_OK, 0)

    xv, zv, sv, w13v, w2v = f64(x), f64(z), slot.cpu().numpy(), f64(w13), f64(w2)
    ids = np.argsort(-zv, axis=1, kind="stable")[:, :K]
    p = np.exp(np.take_along_axis(zv, ids, 1))
    p /= p.sum(1, keepdims=True)
    if mx4:
        w13v, w2v = _mx(lib, w13v), _mx(lib, w2v)
        xq = _mx(lib, xv)
    else:
        xq = xv
    ref = np.zeros((T, H))
    for t in range(T):
        for k in range(K):
            e = ids[t, k] - first
            if e < 0:
                continue
            y = w13v[e] @ xq[t]
            ad = [f64(v) for v in ads[sv[t], e]] if loras and sv[t] else None
            if ad:
                y = y + 0.5 * np.concatenate([xv[t] @ ad[0] @ ad[2], xv[t] @ ad[1] @ ad[3]])
            h = y[:I] / (1 + np.exp(-y[:I])) * y[I:]
            v = w2v[e] @ (_mx(lib, h[None])[0] if mx4 else h)
            if ad:
                v = v + 0.5 * (h @ ad[4] @ ad[5])
            ref[t] += p[t, k] * v
    rel = np.linalg.norm(f64(out) - ref) / np.linalg.norm(ref)
    assert rel <= (6e-2 if mx4 else 2e-2), rel
