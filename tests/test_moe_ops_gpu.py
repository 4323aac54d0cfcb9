"""The mixture-of-experts layer's own operators against plain float64 forms: router, 4-bit format, experts'
products, activation, weighted sum.

Tolerances, from the arithmetic:
* router weights: an fp32 exponent argument off by |l - m| * 2^-24 (|l - m| <= 40 here), expf within 2 ulp, a
  tree sum and a division: 4e-6 relative. Chosen experts are equal.
* 4-bit format: codes, scale bytes and values are equal.
* products: |error| <= d_in * 2^-22 * sum |x||w| (fp32 sums of exact products, one rounding or truncation of
  the running sum a step) plus 2^-8 |y| for a bf16 y; equal on small integers.
* activation and weighted sum: 8 fp32 roundings, 2^-20 relative to the terms' magnitude, plus 2^-8 |out| for bf16.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def f64(t):
    return t.detach().double().cpu().numpy()


# ----------------------------------------------------------------------------- router

def route_ref(z, topk, score, renorm, scale):
    z = np.where(np.isnan(z), -np.inf, np.minimum(z, np.finfo(np.float32).max))
    ids = np.argsort(-z, axis=1, kind="stable")[:, :topk]
    v = np.take_along_axis(z, ids, 1)
    live = np.isfinite(v)
    with np.errstate(invalid="ignore", over="ignore"):
        if score == "softmax":
            m = np.where(np.isfinite(z.max(1, keepdims=True)), z.max(1, keepdims=True), 0)
            tot = np.exp(z - m).sum(1, keepdims=True)
            w = np.exp(v - m) / np.where(tot > 0, tot, 1)
        else:
            w = 1 / (1 + np.exp(-v))
    w = np.where(live, w, 0)
    if renorm:
        tot = w.sum(1, keepdims=True)
        w = w / np.where(tot > 0, tot, 1)
    return ids, w * scale, live


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,topk,dt", [(1, 256, 8, "f32"), (1, 1, 1, "bf16"), (7, 33, 32, "f32"), (513, 64, 6, "bf16"),
                                         (130, 1000, 8, "f32"), (65, 384, 1, "bf16"), (300, 8, 2, "f32"), (9, 512, 5, "bf16"),
                                         (200, 256, 8, "bf16"), (64, 100, 3, "bf16"), (33, 40, 2, "bf16")])
def test_route(lib, score, renorm, T, E, topk, dt):
    g = torch.Generator(device="cuda").manual_seed(T * 1000 + E)
    wide = torch.full((T, E + 3), 50.0, device="cuda", dtype=DT[dt])      # columns past E must not be seen
    wide[:, :E] = (2 * torch.randn(T, E, device="cuda", generator=g)).to(DT[dt])
    z = wide[:, :E]
    z[torch.rand(T, E, device="cuda", generator=g) < 0.15] = float("-inf")
    if T > 6:
        z[1] = float("-inf")                     # nothing left
        z[2] = 0.0                               # all tied
        z[3] = float("nan")
        z[4, E // 2] = float("inf")
        z[5, ::2] = -0.0
        z[5, 1::2] = 0.0
    L = max(1, E // 2)
    emap = torch.full((E,), -1, dtype=torch.int32)
    emap[:L] = torch.arange(L, dtype=torch.int32).flip(0)
    if E > 2:
        emap[E - 1] = L + 2                      # past the local experts
    slot = torch.empty(T * topk, dtype=torch.int32, device="cuda")
    ids, w = lib.moe_route(z, topk, score=score, renormalize=renorm, scale=1.5, expert_map=emap.cuda(),
                           local_experts=L, pair_slot=slot)
    rid, rw, live = route_ref(f64(z), topk, score, renorm, 1.5)
    assert np.array_equal(ids.cpu().numpy(), rid)
    got = f64(w)
    assert np.all(np.abs(got - rw) <= 4e-6 * rw + 1e-37)
    el = emap.numpy()[rid]
    want = np.where(el >= L, -1, np.where((el < 0) | ~live, 0, 1 + el)).reshape(-1)
    assert np.array_equal(slot.cpu().numpy(), want)


def test_route_empty_and_pair_slots_agree(lib):
    ids, w = lib.moe_route(torch.empty(0, 16, device="cuda"), 2)
    assert ids.shape == (0, 2) and w.shape == (0, 2)
    z = torch.randn(50, 24, device="cuda")
    slot = torch.empty(100, dtype=torch.int32, device="cuda")
    ids, _ = lib.moe_route(z, 2, pair_slot=slot)
    other = lib.moe_pair_slots(torch.ones(50, dtype=torch.int32, device="cuda"), ids, 1, 24, 24)
    assert torch.equal(slot, other)


# ----------------------------------------------------------------------------- 4-bit format

GRID = np.array([0, .5, 1, 1.5, 2, 3, 4, 6])


def mx_ref(x):
    """codes [.., K/2], bytes [.., K/32], values: the nearest of the grid by search, ties to the even code."""
    b = x.reshape(*x.shape[:-1], -1, 32)
    bad = ~np.isfinite(b).all(-1, keepdims=True)
    a = np.abs(np.where(bad, 0, b))
    amax = a.max(-1, keepdims=True)
    e = np.clip(np.where(amax > 0, np.floor(np.log2(np.where(amax > 0, amax, 1))) - 2, -127), -127, 127)
    v = a / 2.0 ** e
    hi = np.clip(np.searchsorted(GRID, v), 1, 7)
    lo = hi - 1
    dl, dh = v - GRID[lo], GRID[hi] - v
    c = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    vals = np.where(bad, np.nan, np.copysign(GRID[c] * 2.0 ** e, b))
    c = np.where(bad, 0, c + 8 * np.signbit(b)).reshape(x.shape).astype(np.uint8)
    byte = np.where(bad, 255, e + 127)[..., 0].astype(np.uint8)
    return c[..., 0::2] | (c[..., 1::2] << 4), byte, vals.reshape(x.shape)


def mx_hard(rows, cols, dt, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(rows, cols, device="cuda", generator=g) * torch.exp(4 * torch.randn(rows, 1, device="cuda", generator=g))
    x[0, :32] = 0
    if rows > 4:
        ties = torch.tensor([0, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, 7, -5, -.25, 6, 7.99, -7.5, .125, -3.5], device="cuda")
        x[1, :16], x[1, 16:32] = ties, -ties
        x[2, :32] *= 1e-38                       # scales at and below the smallest byte
        x[2, 0] = 3e38
        x[3, :32] = 1e-40
        x[4, 5] = float("nan")
        x[rows - 1, cols - 3] = float("-inf")
    return x.to(DT[dt])


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols,pad", [(1, 32, 0), (1, 7168, 0), (33, 160, 32), (257, 2080, 0), (5, 4128, 64), (70000, 32, 0)])
def test_mx_quantize_round_trip(lib, dt, rows, cols, pad):
    wide = torch.full((rows, cols + pad), float("nan"), device="cuda", dtype=DT[dt])
    wide[:, :cols] = mx_hard(rows, cols, dt, rows + cols)
    x = wide[:, :cols]
    codes, scales = lib.mx4_buffers(rows, cols + pad)
    codes.fill_(0xAB)
    scales.fill_(0xCD)
    lib.mx4_quantize(x, codes[:, :cols // 2], scales)
    rc, rb, rv = mx_ref(f64(x))
    nb = cols // 32
    assert np.array_equal(codes[:, :cols // 2].cpu().numpy(), rc)
    assert np.array_equal(scales[:, :nb].cpu().numpy(), rb)
    assert (codes[:, cols // 2:] == 0xAB).all() and (scales[:, nb:] == 0xCD).all()
    for odt in ("f32", "bf16"):
        y = lib.mx4_dequantize(codes[:, :cols // 2], scales, torch.empty(rows, cols, device="cuda", dtype=DT[odt]))
        assert np.array_equal(f64(y), rv, equal_nan=True)


@pytest.mark.parametrize("E,N,K,ld", [(1, 8, 32, 16), (3, 136, 288, 16), (2, 256, 4160, 144), (5, 40, 512, 32)])
def test_mx_tile_scales(lib, E, N, K, ld):
    s = torch.randint(0, 256, (E * N, ld), dtype=torch.uint8, device="cuda")
    out = torch.full((lib.lora_mx_tiles_bytes(E, N, K),), 9, dtype=torch.uint8, device="cuda")
    lib.check(lib.lora_mx_tile_scales(s.data_ptr(), ld, E, N, K, out.data_ptr()))
    to, ti, nb = -(-N // 128), -(-K // 256) * 2, K // 32
    want = np.full((E, to * 128, ti * 4), 127, np.uint8)
    want[:, :N, :nb] = s.cpu().numpy().reshape(E, N, ld)[:, :, :nb]
    want = want.reshape(E, to, 4, 32, ti, 4).transpose(0, 1, 4, 3, 2, 5)      # [e][out][in][row % 32][row / 32][block]
    assert np.array_equal(out.cpu().numpy(), want.reshape(-1))


# ----------------------------------------------------------------------------- products

def slots_of(pattern, P, E, seed):
    rng = np.random.default_rng(seed)
    if pattern == "ragged":                      # skewed, some experts empty, a third of the pairs elsewhere
        w = rng.exponential(1, E + 1) ** 2
        w[0] = w.sum() / 2
        if E > 3:
            w[2] = 0
        return rng.choice(E + 1, P, p=w / w.sum()).astype(np.int32)
    if pattern == "one":
        return np.full(P, E, np.int32)
    if pattern == "none":
        return np.zeros(P, np.int32)
    if pattern == "bad":                         # ids outside the table count as slot 0
        return rng.choice(np.array([-1, 0, 1, E, E + 1, 1 << 20]), P).astype(np.int32)
    return (1 + np.arange(P) % E).astype(np.int32)   # even


def product_case(lib, dt, ydt, P, E, K, N, div, pattern, pad=0, seed=0, ints=False, poison=True):
    """(y, reference, magnitude, live rows, y before) of one product with poisoned padding."""
    g = torch.Generator(device="cuda").manual_seed(seed + P + K)
    slot = slots_of(pattern, P, E, seed + P)
    live = (slot > 0) & (slot <= E)
    R = -(-P // div)
    draw = (lambda *s: torch.randint(-3, 4, s, device="cuda", generator=g).float()) if ints else \
        (lambda *s: torch.randn(*s, device="cuda", generator=g))
    x, W = draw(R, K), draw(E, N, K)
    used = np.unique(np.arange(P)[live] // div)
    idle = np.setdiff1d(np.arange(E), slot[live] - 1)
    if dt == "mx4":
        xc, xs = lib.mx4_buffers(R, K + pad)
        xc.fill_(0x77)
        xs.fill_(0xFF)
        lib.mx4_quantize(x, xc[:, :K // 2], xs)
        wc, ws = lib.mx4_buffers(E * N, K)
        ws.fill_(0xFF)
        lib.mx4_quantize(W.reshape(E * N, K), wc, ws)
        xv, Wv = torch.empty(R, K, device="cuda"), torch.empty(E * N, K, device="cuda")
        lib.mx4_dequantize(xc[:, :K // 2], xs, xv)
        lib.mx4_dequantize(wc, ws, Wv)
        xv, Wv = f64(xv), f64(Wv).reshape(E, N, K)
        ws = ws.reshape(E, N, -1)
        if poison and idle.size:
            ws[torch.from_numpy(idle).cuda()] = 0xFF
        ex, xa, xsa = lib.ExpertWeights(wc.reshape(E, N, K // 2), ws, x_row_div=div), xc[:, :K // 2], xs
    else:
        td = DT[dt]
        W = W.to(td)
        xw = torch.full((R, K + pad), float("nan"), device="cuda", dtype=td)
        xw[:, :K] = x.to(td)
        xa, xsa = xw[:, :K], None
        xv, Wv = f64(xa), f64(W)
        if poison:
            W[torch.from_numpy(idle).cuda()] = float("nan")
            mask = torch.ones(R, dtype=torch.bool, device="cuda")
            mask[torch.from_numpy(used).cuda()] = False
            xw[mask] = float("nan")
        ex = lib.ExpertWeights(W, x_row_div=div)
    yw = torch.randn(P, N + pad, device="cuda", generator=g).to(DT[ydt])
    before = yw.clone()
    meta = lib.TokenMeta(max(P, 1), E + 1)
    meta.prepare(torch.from_numpy(slot).cuda())
    lib.moe_product(ex, meta, xa, yw[:, :N], x_scale=xsa)
    torch.cuda.synchronize()
    st, bad = lib.lora_query_status(meta.c)
    assert st in (lib.LORA_OK, lib.LORA_EBADSLOT) and bad == int(((slot < 0) | (slot > E)).sum())
    ref, mag = np.zeros((P, N)), np.zeros((P, N))
    for e in np.unique(slot[live]):
        r = np.nonzero(slot == e)[0]
        ref[r] = xv[r // div] @ Wv[e - 1].T
        mag[r] = np.abs(xv[r // div]) @ np.abs(Wv[e - 1]).T
    assert torch.equal(yw[:, N:].view(torch.uint8), before[:, N:].view(torch.uint8)), "columns past d_out were written"
    dead = torch.from_numpy(~live).cuda()
    assert torch.equal(yw[dead].view(torch.uint8), before[dead].view(torch.uint8)), "a slot-0 row was written"
    y = f64(yw[:, :N])
    tol = K * 2.0 ** -22 * mag + (2.0 ** -8 * np.abs(ref) if ydt == "bf16" else 0)
    err = np.abs(y - ref)[live]
    assert np.isfinite(y[live]).all() and (err <= tol[live]).all(), f"worst {np.max(err / (tol[live] + 1e-30)):.3g} of the bound"
    if ints and ydt == "f32":
        assert np.array_equal(y[live], ref[live])
    return yw


TYPES = [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("mx4", "bf16"), ("mx4", "f32")]
SHAPES = [  # P, E, K, N, div, pattern, pad
    (1, 1, 32, 8, 1, "one", 0), (1, 4, 64, 136, 8, "one", 0), (8, 32, 7168, 128, 8, "even", 0), (3, 2, 8, 8, 1, "even", 0),
    (17, 5, 96, 200, 1, "ragged", 32), (64, 3, 1056, 72, 4, "ragged", 0), (300, 7, 544, 264, 3, "ragged", 64),
    (129, 1, 288, 128, 1, "one", 0), (1000, 4, 256, 1000, 2, "ragged", 0), (2100, 3, 320, 264, 1, "ragged", 32),
    (2048, 2, 512, 512, 8, "even", 0), (513, 1, 160, 520, 1, "one", 0), (40, 6, 64, 64, 1, "none", 0),
    (120, 5, 128, 136, 1, "bad", 0), (900, 300, 64, 72, 1, "even", 0), (1500, 1023, 32, 8, 1, "ragged", 0),
    # tiles of 64, 128 and 256 outputs, by how many there are
    (5, 1, 512, 4104, 1, "one", 0), (9, 2, 320, 4360, 1, "even", 32), (70, 1, 224, 4992, 2, "one", 0),
    (200, 2, 96, 9224, 1, "even", 0), (300, 1, 64, 1160, 1, "one", 0), (600, 3, 288, 3080, 1, "ragged", 0),
]


@pytest.mark.parametrize("dt,ydt", TYPES)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
def test_product(lib, dt, ydt, shape):
    P, E, K, N, div, pattern, pad = shape
    if dt == "mx4":
        K = -(-K // 32) * 32
    product_case(lib, dt, ydt, P, E, K, N, div, pattern, pad)


@pytest.mark.parametrize("dt", ["f32", "bf16", "mx4"])
@pytest.mark.parametrize("K", [8, 40, 72, 200, 264, 1000])
def test_product_depths_on_integers(lib, dt, K):
    """Depths that end inside every kind of step, equal to the integer result."""
    K = -(-K // 32) * 32 if dt == "mx4" else K
    product_case(lib, dt, "f32", 75, 3, K, 152, 1, "ragged", ints=True)


@pytest.mark.parametrize("dt", ["bf16", "mx4"])
@pytest.mark.parametrize("rows", [1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 191, 193, 255, 256, 257, 383, 385, 511, 513])
def test_product_segment_lengths(lib, dt, rows):
    product_case(lib, dt, "f32", rows, 1, 192, 264, 1, "one", ints=True)


@pytest.mark.parametrize("dt", ["f32", "bf16", "mx4"])
def test_product_repeats_and_ignores_other_pairs(lib, dt):
    """The same call twice is bitwise equal, and a row's result does not change with the other rows' values."""
    a = product_case(lib, dt, "f32", 333, 4, 640, 136, 1, "ragged", seed=5)
    b = product_case(lib, dt, "f32", 333, 4, 640, 136, 1, "ragged", seed=5)
    assert torch.equal(a, b)


def test_product_values_outside_the_numbers(lib):
    """A NaN or an infinity in one x row stays in that row; a NaN scale byte likewise."""
    P, K, N = 70, 256, 136
    slot = torch.ones(P, dtype=torch.int32, device="cuda")
    meta = lib.TokenMeta(P, 2)
    meta.prepare(slot)
    x = torch.randn(P, K, device="cuda")
    x[3, 5], x[40, 255] = float("nan"), float("inf")
    W = torch.rand(1, N, K, device="cuda") + 0.5
    y = torch.zeros(P, N, device="cuda")
    lib.moe_product(lib.ExpertWeights(W.bfloat16()), meta, x.bfloat16(), y)
    fine = torch.isfinite(y).all(1)
    assert not fine[3] and not fine[40] and int(fine.sum()) == P - 2 and torch.isinf(y[40]).all()
    y.zero_()
    xc, xs = lib.mx4_quantize(x)
    wc, ws = lib.mx4_quantize(W.reshape(N, K))
    lib.moe_product(lib.ExpertWeights(wc.reshape(1, N, -1), ws.reshape(1, N, -1)), meta, xc, y, x_scale=xs)
    fine = torch.isfinite(y).all(1)
    assert torch.isnan(y[3]).all() and torch.isnan(y[40]).all() and int(fine.sum()) == P - 2


# ----------------------------------------------------------------------------- activation, weighted sum

@pytest.mark.parametrize("ydt,hdt", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("P,inter,pad", [(1, 8, 0), (5, 2048, 0), (333, 72, 16), (70001, 32, 0), (64, 4104, 8)])
def test_act(lib, ydt, hdt, P, inter, pad):
    g = torch.Generator(device="cuda").manual_seed(P + inter)
    wide = torch.randn(P, 2 * inter + pad, device="cuda", generator=g) * 4
    wide[0, 0], wide[0, 1] = -200.0, 200.0       # exp overflows and underflows
    wide = wide.to(DT[ydt])
    slot = (torch.rand(P, device="cuda", generator=g) < 0.7).int() * 3
    slot[0] = 2
    y = wide[:, :2 * inter]
    y[slot == 0] = float("nan")
    h = torch.full((P, inter + pad), 7.0, device="cuda", dtype=DT[hdt])
    lib.moe_act(y, h[:, :inter], pair_slot=slot)
    live = slot.cpu().numpy() > 0
    v = f64(y)
    with np.errstate(over="ignore", invalid="ignore"):
        ref = v[:, :inter] / (1 + np.exp(-v[:, :inter])) * v[:, inter:]
    err = np.abs(f64(h[:, :inter]) - ref)[live]
    assert (err <= ((2.0 ** -20 + (2.0 ** -8 if hdt == "bf16" else 0)) * np.abs(ref) + 1e-30)[live]).all()
    assert (h[:, inter:] == 7).all() and (h[slot == 0] == 7).all()


@pytest.mark.parametrize("P,inter", [(1, 32), (77, 2048), (300, 160)])
@pytest.mark.parametrize("ydt", ["bf16", "f32"])
def test_act_mx4_is_act_then_quantize(lib, ydt, P, inter):
    g = torch.Generator(device="cuda").manual_seed(P)
    y = (3 * torch.randn(P, 2 * inter, device="cuda", generator=g)).to(DT[ydt])
    slot = (torch.rand(P, device="cuda", generator=g) < 0.6).int()
    slot[0] = 1
    h = lib.moe_act(y, torch.empty(P, inter, dtype=torch.bfloat16, device="cuda"))
    rc, rs = lib.mx4_quantize(h)
    c, s = lib.mx4_buffers(P, inter)
    c.fill_(0xEE)
    s.fill_(0xEE)
    lib.moe_act_mx4(y, c, s, pair_slot=slot)
    nb, on = inter // 32, slot > 0
    assert torch.equal(c[on], rc[on]) and torch.equal(s[on][:, :nb], rs[on][:, :nb])
    assert (c[~on] == 0xEE).all() and (s[~on] == 0xEE).all() and (s[:, nb:] == 0xEE).all()


@pytest.mark.parametrize("ydt,odt", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("T,topk,n,acc,pad", [(1, 8, 7168, False, 0), (1, 1, 8, True, 0), (1300, 8, 2056, False, 0), (37, 6, 1000, True, 8),
                                              (70000, 2, 16, False, 0), (64, 33, 136, False, 24), (300, 9, 264, True, 0)])
def test_combine(lib, ydt, odt, T, topk, n, acc, pad):
    g = torch.Generator(device="cuda").manual_seed(T + n)
    y = torch.randn(T * topk, n + pad, device="cuda", generator=g).to(DT[ydt])
    w = torch.rand(T, topk, device="cuda", generator=g)
    slot = torch.randint(-1, 4, (T * topk,), dtype=torch.int32, device="cuda", generator=g)
    slot[:topk] = 0 if T > 1 else 1              # a token whose choices are all elsewhere
    y[slot <= 0] = float("nan")
    out = torch.randn(T, n + pad, device="cuda", generator=g).to(DT[odt])
    before = f64(out)
    lib.moe_combine(y[:, :n], w, out[:, :n], pair_slot=slot, accumulate=acc)
    wv = np.where(slot.cpu().numpy() > 0, f64(w).reshape(-1), 0).reshape(T, topk)
    yv = np.where(np.isnan(f64(y[:, :n])), 0, f64(y[:, :n])).reshape(T, topk, n)
    base = before[:, :n] if acc else 0
    ref = base + np.einsum("tk,tkn->tn", wv, yv)
    mag = np.abs(base) + np.einsum("tk,tkn->tn", wv, np.abs(yv))
    assert (np.abs(f64(out[:, :n]) - ref) <= topk * 2.0 ** -23 * mag + (2.0 ** -8 * np.abs(ref) if odt == "bf16" else 0)).all()
    assert np.array_equal(f64(out)[:, n:], before[:, n:])


# ----------------------------------------------------------------------------- streams, graphs, nothing to do

@pytest.mark.parametrize("dt", ["bf16", "mx4"])
def test_layer_on_another_stream_and_in_a_graph(lib, dt):
    """Router to weighted sum on a side stream, eagerly and replayed from a CUDA graph, bitwise equal."""
    T, E, topk, H, I = 96, 12, 3, 256, 128
    g = torch.Generator(device="cuda").manual_seed(9)
    P = T * topk
    x = torch.randn(T, H, device="cuda", generator=g).bfloat16()
    z = torch.randn(T, E, device="cuda", generator=g)
    W13 = torch.randn(E, 2 * I, H, device="cuda", generator=g).bfloat16()
    W2 = torch.randn(E, H, I, device="cuda", generator=g).bfloat16()
    if dt == "mx4":
        q = lambda W, **k: lib.ExpertWeights(*(t.reshape(W.shape[0], W.shape[1], -1)          # noqa: E731
                                               for t in lib.mx4_quantize(W.reshape(-1, W.shape[2]))), **k)
    else:
        q = lib.ExpertWeights
    e13, e2 = q(W13, x_row_div=topk), q(W2)
    meta = lib.TokenMeta(P, E + 1)
    meta.set_num_tokens(P)
    ids, w = torch.empty(T, topk, dtype=torch.int32, device="cuda"), torch.empty(T, topk, device="cuda")
    y13, h, y2 = (torch.empty(P, n, dtype=torch.bfloat16, device="cuda") for n in (2 * I, I, H))
    out = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    xq, hq = lib.mx4_buffers(T, H), lib.mx4_buffers(P, I)

    def step():
        lib.moe_route(z, topk, topk_ids=ids, topk_w=w, pair_slot=meta.token_slot[:P])
        meta.prepare()
        if dt == "mx4":
            lib.mx4_quantize(x, *xq)
            lib.moe_product(e13, meta, xq[0], y13, x_scale=xq[1])
            lib.moe_act_mx4(y13, *hq, pair_slot=meta.token_slot[:P])
            lib.moe_product(e2, meta, hq[0], y2, x_scale=hq[1])
        else:
            lib.moe_product(e13, meta, x, y13)
            lib.moe_act(y13, h, pair_slot=meta.token_slot[:P])
            lib.moe_product(e2, meta, h, y2)
        lib.moe_combine(y2, w, out, pair_slot=meta.token_slot[:P])

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    eager = out.clone()
    assert torch.isfinite(eager).all() and (eager != 0).any()
    out.fill_(float("nan"))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    z2 = z.clone()
    for _ in range(3):
        out.fill_(float("nan"))
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, eager)
    z.copy_(z2.flip(0))                          # new routing, same graph
    graph.replay()
    torch.cuda.synchronize()
    replayed = out.clone()
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    assert torch.equal(out, replayed) and not torch.equal(out, eager)


def test_nothing_to_do(lib):
    e = lib.ExpertWeights(torch.zeros(2, 16, 32, device="cuda", dtype=torch.bfloat16))
    meta = lib.TokenMeta(0, 3)
    meta.prepare()
    n0 = lib.lora_launch_count()
    lib.moe_product(e, meta, torch.empty(0, 32, device="cuda", dtype=torch.bfloat16),
                    torch.empty(0, 16, device="cuda", dtype=torch.bfloat16))
    lib.mx4_quantize(torch.empty(0, 64, device="cuda"))
    lib.moe_act(torch.empty(0, 64, device="cuda"), torch.empty(0, 32, device="cuda"))
    lib.moe_combine(torch.empty(0, 8, device="cuda"), torch.empty(0, 2, device="cuda"), torch.empty(0, 8, device="cuda"))
    assert lib.lora_launch_count() == n0


@pytest.mark.parametrize("dt", ["bf16", "mx4"])
def test_offsets_past_32_bits(lib, dt):
    """Rows of y and of x more than 2^31 elements from the start, weights more than 2^32 bytes."""
    P, K, N, ld = 300000, 64, 8, 8192
    y = torch.zeros(P, ld, dtype=torch.bfloat16, device="cuda")[:, :N]
    x = torch.zeros(P, ld if dt == "bf16" else 16 * ld, dtype=torch.bfloat16 if dt == "bf16" else torch.uint8, device="cuda")
    slot = torch.zeros(P, dtype=torch.int32, device="cuda")
    pick = torch.tensor([0, 1, 262144, 270000, P - 1], device="cuda")
    slot[pick] = 1
    xr = torch.randint(-3, 4, (5, K), device="cuda").float()
    W = torch.randint(-3, 4, (N, K), device="cuda").float()
    meta = lib.TokenMeta(P, 2)
    meta.prepare(slot)
    if dt == "bf16":
        x[pick, :K] = xr.bfloat16()
        lib.moe_product(lib.ExpertWeights(W.bfloat16()[None].contiguous()), meta, x[:, :K], y)
    else:
        c, s = lib.mx4_quantize(xr)
        x[pick, :K // 2] = c
        xs = torch.zeros(P, s.shape[1], dtype=torch.uint8, device="cuda")
        xs[pick] = s
        wc, wsc = lib.mx4_quantize(W)
        xr = lib.mx4_dequantize(c, s, torch.empty_like(xr))
        W = lib.mx4_dequantize(wc, wsc, torch.empty_like(W))
        lib.moe_product(lib.ExpertWeights(wc[None], wsc[None]), meta, x[:, :K // 2], y, x_scale=xs)
    torch.cuda.synchronize()
    ref = f64(xr) @ f64(W).T
    assert (np.abs(f64(y[pick]) - ref) <= 2.0 ** -8 * np.abs(ref)).all()
    assert int((y != 0).any(1).sum()) <= 5
    if dt == "bf16":                                   # an expert whose weights start past 2^32 bytes
        del x, y
        E, Nw, Kw = 40, 8192, 8192
        Wb = torch.zeros(E, Nw, Kw, dtype=torch.bfloat16, device="cuda")
        Wb[E - 1] = torch.randint(-3, 4, (Nw, Kw), device="cuda").bfloat16()
        xb = torch.randint(-3, 4, (3, Kw), device="cuda").bfloat16()
        yb = torch.empty(3, Nw, device="cuda")
        meta = lib.TokenMeta(3, E + 1)
        meta.prepare(torch.full((3,), E, dtype=torch.int32, device="cuda"))
        lib.moe_product(lib.ExpertWeights(Wb), meta, xb, yb)
        assert np.array_equal(f64(yb), f64(xb) @ f64(Wb[E - 1]).T)


@pytest.mark.parametrize("dt", ["bf16", "mx4"])
def test_products_on_two_streams_at_once(lib, dt):
    """Two layers' products on one metadata and two streams, many in flight, bitwise what one stream gives."""
    P, E, K, N = 700, 5, 512, 1032
    g = torch.Generator(device="cuda").manual_seed(11)
    meta = lib.TokenMeta(P, E + 1)
    meta.prepare(torch.from_numpy(slots_of("ragged", P, E, 3)).cuda())
    sides = []
    for _ in range(2):
        x, W = torch.randn(P, K, device="cuda", generator=g), torch.randn(E, N, K, device="cuda", generator=g)
        if dt == "mx4":
            (xc, xs), (wc, ws) = lib.mx4_quantize(x), lib.mx4_quantize(W.reshape(-1, K))
            sides.append((lib.ExpertWeights(wc.view(E, N, -1), ws.view(E, N, -1)), xc, xs))
        else:
            sides.append((lib.ExpertWeights(W.bfloat16()), x.bfloat16(), None))
    want = []
    for e, x, xs in sides:
        y = torch.zeros(P, N, device="cuda")
        lib.moe_product(e, meta, x, y, x_scale=xs)
        want.append(y)
    torch.cuda.synchronize()
    got = [[torch.zeros(P, N, device="cuda") for _ in range(6)] for _ in sides]
    streams = [torch.cuda.Stream() for _ in sides]
    torch.cuda.synchronize()
    for i in range(6):
        for (e, x, xs), ys, s in zip(sides, got, streams):
            lib.moe_product(e, meta, x, ys[i], x_scale=xs, stream=s)
    torch.cuda.synchronize()
    assert lib.lora_query_status(meta.c) == (lib.LORA_OK, 0)
    for ys, w in zip(got, want):
        for y in ys:
            assert torch.equal(y, w)
