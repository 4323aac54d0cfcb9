"""Products launched back to back, so that each one's CTAs take over the SMs and shared memory that its
predecessor's are leaving: every result is bitwise the one the same product gives alone."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

# (weights, pairs, experts, d_in, d_out): narrow and wide tiles, fewer stages than the pipeline has and more,
# grids of one pair and of all of them.
KINDS = [("bf16", 5, 3, 64, 264), ("bf16", 700, 2, 1024, 2056), ("mx4", 9, 4, 256, 136), ("mx4", 900, 2, 2048, 4104),
         ("bf16", 130, 40, 896, 776), ("mx4", 200, 30, 2560, 1032), ("bf16", 2000, 3, 128, 520), ("mx4", 1500, 1, 288, 264)]


def _product(lib, g, dt, P, E, K, N):
    slot = torch.randint(0, E + 1, (P,), dtype=torch.int32, device="cuda", generator=g)
    slot[0] = 1
    meta = lib.TokenMeta(P, E + 1)
    meta.prepare(slot)
    x, W = torch.randn(P, K, device="cuda", generator=g), torch.randn(E, N, K, device="cuda", generator=g)
    if dt == "mx4":
        (xc, xs), (wc, ws) = lib.mx4_quantize(x), lib.mx4_quantize(W.reshape(-1, K))
        return lib.ExpertWeights(wc.view(E, N, -1), ws.view(E, N, -1)), meta, xc, xs, (P, N)
    return lib.ExpertWeights(W.bfloat16()), meta, x.bfloat16(), None, (P, N)


@pytest.mark.parametrize("ydt", [torch.bfloat16, torch.float32])
def test_back_to_back_products_give_what_each_gives_alone(lib, ydt):
    g = torch.Generator(device="cuda").manual_seed(17)
    cases = [_product(lib, g, *k) for k in KINDS]
    alone = []
    for e, meta, x, xs, shape in cases:
        y = torch.zeros(shape, dtype=ydt, device="cuda")
        torch.cuda.synchronize()
        lib.moe_product(e, meta, x, y, x_scale=xs)
        torch.cuda.synchronize()
        assert lib.lora_query_status(meta.c) == (lib.LORA_OK, 0)
        alone.append(y)
    order = np.random.default_rng(3).integers(0, len(cases), 120)
    got = [torch.zeros(cases[i][4], dtype=ydt, device="cuda") for i in order]
    torch.cuda.synchronize()
    for i, y in zip(order, got):
        e, meta, x, xs, _ = cases[i]
        lib.moe_product(e, meta, x, y, x_scale=xs)
    torch.cuda.synchronize()
    for _, meta, *_ in cases:
        assert lib.lora_query_status(meta.c) == (lib.LORA_OK, 0)
    for i, y in zip(order, got):
        assert torch.equal(y, alone[i]), KINDS[i]
