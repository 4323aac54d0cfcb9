"""Products whose CTA pairs take many tiles in turn, each of several pipeline stages: integer operands, so that
every sum is exact in fp32 and the result has to be equal. Then what a row of the result depends on, and how a
bf16 result is rounded."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


def ragged(P, E, seed):
    """Slots of P pairs: experts of very different length, some empty, a twentieth of the pairs elsewhere."""
    rng = np.random.default_rng(seed)
    w = rng.exponential(1, E + 1) + 0.2
    w[0] = w[1:].sum() / 19
    if E > 8:
        w[3] = 0
    return rng.choice(E + 1, P, p=w / w.sum()).astype(np.int32)


def operands(lib, dt, P, E, K, N, g, ints=True):
    """(ExpertWeights, x, x_scale, values of x, values of W) with float64 values."""
    if dt == "bf16":
        draw = (lambda *s: torch.randint(-3, 4, s, device="cuda", generator=g)) if ints else \
            (lambda *s: torch.randn(*s, device="cuda", generator=g))
        x, W = draw(P, K).bfloat16(), draw(E, N, K).bfloat16()
        return lib.ExpertWeights(W), x, None, x.double(), W.double()
    # Codes at random, scales of 1 and 2: values are multiples of 0.5 up to 12, a sum's terms of 0.25 up to 144.
    u8 = dict(dtype=torch.uint8, device="cuda", generator=g)
    xc, xs = lib.mx4_buffers(P, K)
    wc, ws = lib.mx4_buffers(E * N, K)
    for c, s in ((xc, xs), (wc, ws)):
        c.copy_(torch.randint(0, 256, c.shape, **u8))
        s.copy_(torch.randint(127, 129, s.shape, **u8))
    xv, Wv = torch.empty(P, K, device="cuda"), torch.empty(E * N, K, device="cuda")
    lib.mx4_dequantize(xc, xs, xv)
    lib.mx4_dequantize(wc, ws, Wv)
    return lib.ExpertWeights(wc.view(E, N, -1), ws.view(E, N, -1)), xc, xs, xv.double(), Wv.double().view(E, N, K)


def product(lib, ex, slot, x, xs, N, ydt, E):
    P = slot.size
    meta = lib.TokenMeta(P, E + 1)
    meta.prepare(torch.from_numpy(slot).cuda())
    y = torch.full((P, N), float("nan"), dtype=ydt, device="cuda")
    lib.moe_product(ex, meta, x, y, x_scale=xs)
    torch.cuda.synchronize()
    assert lib.lora_query_status(meta.c) == (lib.LORA_OK, 0)
    return y


# 76 CTA pairs. Wide tiles (256 rows in bf16, 192 in 4 bits): 25 blocks of outputs by at least 4 row tiles an
# expert, 5 tiles a pair and more; narrow ones (64 rows): 9 blocks by at least 63 experts, 7 tiles a pair. d_in in
# stages of 64 (bf16: 6 stages wide, 10 narrow) and 256 elements (4-bit: 5 and 9): odd and even counts, below, at
# and above the pipeline's, whole and ragged.
WIDE, NARROW = (4000, 4, 6152), (3000, 64, 2056)
CASES = [("bf16", *WIDE, K) for K in (320, 384, 832, 1856)] + [("mx4", *WIDE, K) for K in (320, 832, 1280, 1344, 1856)] + \
        [("bf16", *NARROW, K) for K in (320, 640, 648, 1208)] + [("mx4", *NARROW, K) for K in (544, 800, 2304, 2336, 2848)]


@pytest.mark.parametrize("ydt", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("dt,P,E,N,K", CASES)
def test_many_tiles_a_pair(lib, dt, P, E, N, K, ydt):
    assert (P <= 48 * E) == (E == NARROW[1])           # the shape takes the tiles it is meant for
    g = torch.Generator(device="cuda").manual_seed(K)
    ex, x, xs, xv, Wv = operands(lib, dt, P, E, K, N, g)
    slot = ragged(P, E, K)
    y = product(lib, ex, slot, x, xs, N, ydt, E)
    s = torch.from_numpy(slot).cuda()
    for e in range(E):
        rows = torch.nonzero(s == e + 1).flatten()
        want = (xv[rows] @ Wv[e].T).float().to(ydt)    # exact in fp32; a bf16 result is that sum rounded once
        assert torch.equal(y[rows], want), f"expert {e}: {int((y[rows] != want).sum())} of {want.numel()} differ"
    assert torch.isnan(y[s == 0]).all(), "a row without an expert was written"


@pytest.mark.parametrize("dt", ["bf16", "mx4"])
@pytest.mark.parametrize("P,E", [(3000, 4), (600, 40)])
def test_a_row_does_not_depend_on_the_others(lib, dt, P, E):
    K, N = 704, 1032
    g = torch.Generator(device="cuda").manual_seed(P)
    ex, x, xs, _, _ = operands(lib, dt, P, E, K, N, g, ints=False)
    slot = ragged(P, E, 5)
    a = product(lib, ex, slot, x, xs, N, torch.float32, E)
    change = torch.rand(P, device="cuda", generator=g) < 0.4
    x2 = x.clone()
    x2[change] = x[change].flip(1)
    b = product(lib, ex, slot, x2, xs, N, torch.float32, E)
    live = torch.from_numpy(slot).cuda() > 0
    assert torch.equal(a[live & ~change], b[live & ~change])
    assert (a[live & change] != b[live & change]).any(1).all()


@pytest.mark.parametrize("dt", ["bf16", "mx4"])
@pytest.mark.parametrize("P,E", [(2000, 4), (300, 32)])
def test_a_bf16_result_is_the_fp32_one_rounded_once(lib, dt, P, E):
    """Random values: the bf16 result is bitwise the rounding of the fp32 one, repeats bitwise, and the fp32 one is
    within d_in * 2^-22 * sum |x||w| of the sum in 64 bits (one rounding or truncation a step)."""
    K, N = 2048, 1032
    g = torch.Generator(device="cuda").manual_seed(P + 1)
    ex, x, xs, xv, Wv = operands(lib, dt, P, E, K, N, g, ints=False)
    slot = ragged(P, E, 7)
    y32 = product(lib, ex, slot, x, xs, N, torch.float32, E)
    live = torch.from_numpy(slot).cuda() > 0
    for _ in range(3):
        y16 = product(lib, ex, slot, x, xs, N, torch.bfloat16, E)
        assert torch.equal(y16[live], y32[live].bfloat16())
        assert torch.equal(product(lib, ex, slot, x, xs, N, torch.float32, E)[live], y32[live])
    for e in np.unique(slot[slot > 0]):
        rows = torch.from_numpy(np.nonzero(slot == e)[0]).cuda()
        ref, mag = xv[rows] @ Wv[e - 1].T, xv[rows].abs() @ Wv[e - 1].abs().T
        assert ((y32[rows].double() - ref).abs() <= K * 2.0 ** -22 * mag).all()
