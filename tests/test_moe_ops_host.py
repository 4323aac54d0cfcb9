"""The mixture-of-experts operators refuse bad arguments on the host, before any launch (no GPU needed)."""
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 0x10000


@pytest.fixture(scope="module")
def ra():
    import __graft_entry__
    __graft_entry__._load_build_lib().build()
    import rank_adapter_gb300
    return rank_adapter_gb300


def test_constants_match_the_header(ra):
    src = open(os.path.join(ROOT, "include", "lora.h")).read()
    for name in ("LORA_MAX_EXPERTS", "LORA_MAX_ROUTE_TOPK", "LORA_MX_BLOCK"):
        assert int(re.search(rf"#define {name} (\d+)", src).group(1)) == getattr(ra, name)
    assert re.search(r"#define LORA_MAX_EXPERT_DIM \(1 << 24\)", src) and ra.LORA_MAX_EXPERT_DIM == 1 << 24
    assert re.search(rf"LORA_MXFP4 = {ra.LORA_MXFP4}\b", src)
    assert re.search(rf"LORA_SCORE_SOFTMAX = {ra.LORA_SCORE_SOFTMAX}, LORA_SCORE_SIGMOID = {ra.LORA_SCORE_SIGMOID}\b", src)


def test_route(ra):
    def f(logits=P, ld=64, dt=ra.LORA_F32, T=5, E=64, topk=4, score=0, emap=0, local=64, ids=P, w=P, slot=0):
        return ra.lora_moe_route(logits, ld, dt, T, E, topk, score, True, 1.0, emap, local, ids, w, slot, 0)
    assert f(T=0, logits=0, ids=0, w=0) == ra.LORA_OK
    for kw in (dict(dt=ra.LORA_MXFP4), dict(score=2), dict(logits=0), dict(ids=0), dict(w=0), dict(ld=63)):
        assert f(**kw) == ra.LORA_EINVAL, kw
    for kw in (dict(E=0), dict(E=1025, ld=2000), dict(topk=0), dict(topk=33), dict(E=3, topk=4), dict(T=-1),
               dict(T=1 << 24), dict(slot=P, local=0), dict(slot=P, local=65)):
        assert f(**kw) == ra.LORA_ERANGE, kw
    for kw in (dict(logits=P + 2), dict(ids=P + 2), dict(w=P + 1), dict(slot=P + 2), dict(emap=P + 3)):
        assert f(**kw) == ra.LORA_EALIGN, kw


def _meta(ra, T=8, S=5):
    m = ra.Meta()
    m.token_slot, m.num_tokens, m.num_slots = 0x1000, T, S
    m.sorted_rows = m.seg_slot = m.seg_count = m.seg_start = 0x2000
    m.num_segs, m.no_lora, m.status = 0x3000, 0x3004, 0x3008
    m.tiles, m.tiles_bytes = 0x4000, ra.lora_meta_tiles_bytes(S)
    return m


def test_product(ra):
    def f(dt=ra.LORA_BF16, K=64, N=32, E=4, W=P, ws=0, div=1, T=8, S=5, x=P, ldx=64, xs=0, lxs=0, y=P, ldy=32,
          ydt=ra.LORA_BF16, meta=True):
        d = ra.ExpertDesc()
        d.dtype, d.d_in, d.d_out, d.num_experts, d.W, d.W_scale, d.x_row_div = dt, K, N, E, W, ws or None, div
        return ra.lora_moe_product(d, _meta(ra, T, S), x, ldx, xs, lxs, y, ldy, ydt, 0)
    mx = dict(dt=ra.LORA_MXFP4, ws=P, xs=P, lxs=16)
    assert f(T=0, x=0, y=0) == ra.LORA_OK and f(**{**mx, "T": 0}) == ra.LORA_OK
    for kw in (dict(dt=9), dict(K=0), dict(K=12), dict(N=0), dict(N=12), dict(div=-1), dict(W=0), dict(S=6), dict(x=0),
               dict(y=0), dict(ldx=56), dict(ldy=24), dict(ydt=ra.LORA_MXFP4), {**mx, "ws": 0}, {**mx, "xs": 0},
               {**mx, "K": 40, "ldx": 64}, {**mx, "lxs": 0}):
        assert f(**kw) == ra.LORA_EINVAL, kw
    for kw in (dict(E=0, S=1), dict(E=1024, S=1025), dict(T=-1), dict(K=(1 << 24) + 8, ldx=1 << 25),
               dict(N=(1 << 24) + 8, ldy=1 << 25)):
        assert f(**kw) == ra.LORA_ERANGE, kw
    for kw in (dict(W=P + 8), dict(x=P + 8), dict(y=P + 2), dict(ldx=68), dict(ldy=36), {**mx, "ws": P + 8},
               {**mx, "xs": P + 4}, {**mx, "lxs": 20}, {**mx, "ldx": 80}):
        assert f(**kw) == ra.LORA_EALIGN, kw
    assert f(dt=ra.LORA_F32) == ra.LORA_EUNSUPPORTED


def test_mx(ra):
    def f(x=P, ldx=64, dt=ra.LORA_BF16, rows=3, cols=64, c=P, ldc=32, s=P, lds=16):
        a = ra.lora_mx_quantize(x, ldx, dt, rows, cols, c, ldc, s, lds, 0)
        assert a == ra.lora_mx_dequantize(c, ldc, s, lds, rows, cols, x, ldx, dt, 0)
        return a
    assert f(rows=0, x=0, c=0, s=0) == ra.LORA_OK
    for kw in (dict(dt=ra.LORA_MXFP4), dict(cols=0), dict(cols=48), dict(x=0), dict(c=0), dict(s=0), dict(ldx=32),
               dict(ldc=16), dict(lds=0)):
        assert f(**kw) == ra.LORA_EINVAL, kw
    assert f(rows=-1) == ra.LORA_ERANGE
    for kw in (dict(x=P + 2), dict(ldx=68), dict(c=P + 4), dict(ldc=40), dict(s=P + 1), dict(lds=24)):
        assert f(**kw) == ra.LORA_EALIGN, kw


def test_tile_scales(ra):
    def f(s=P, ld=16, E=3, N=40, K=96, t=P):
        return ra.lora_mx_tile_scales(s, ld, E, N, K, t, 0)
    for kw in (dict(E=0), dict(E=1024), dict(N=(1 << 24) + 8), dict(K=(1 << 24) + 32, ld=1 << 20)):
        assert f(**kw) == ra.LORA_ERANGE, kw
    for kw in (dict(N=0), dict(N=12), dict(K=0), dict(K=40), dict(s=0), dict(t=0), dict(ld=0)):
        assert f(**kw) == ra.LORA_EINVAL, kw
    for kw in (dict(s=P + 8), dict(t=P + 4), dict(ld=24)):
        assert f(**kw) == ra.LORA_EALIGN, kw
    assert ra.lora_mx_tiles_bytes(3, 40, 96) == 3 * 1 * 2 * 512
    assert ra.lora_mx_tiles_bytes(2, 129, 257) == 2 * 2 * 4 * 512
    assert ra.lora_mx_tiles_bytes(0, 8, 32) == ra.lora_mx_tiles_bytes(1024, 8, 32) == ra.lora_mx_tiles_bytes(1, 0, 32) == 0


def test_act(ra):
    def f(y=P, ldy=128, ydt=ra.LORA_BF16, slot=P, n=4, inter=64, h=P, ldh=64, hdt=ra.LORA_BF16):
        return ra.lora_moe_act(y, ldy, ydt, slot, n, inter, h, ldh, hdt, 0)
    assert f(n=0, y=0, h=0) == ra.LORA_OK
    for kw in (dict(ydt=5), dict(hdt=ra.LORA_MXFP4), dict(inter=0), dict(inter=12), dict(y=0), dict(h=0), dict(ldy=120),
               dict(ldh=56)):
        assert f(**kw) == ra.LORA_EINVAL, kw
    assert f(n=-1) == ra.LORA_ERANGE and f(n=(1 << 24) + 1) == ra.LORA_ERANGE
    for kw in (dict(y=P + 4), dict(h=P + 8), dict(slot=P + 2), dict(ldy=132), dict(ldh=68)):
        assert f(**kw) == ra.LORA_EALIGN, kw

    def g(y=P, inter=64, n=4, c=P, ldc=32, s=P, lds=16):
        return ra.lora_moe_act_mx(y, 128, ra.LORA_BF16, 0, n, inter, c, ldc, s, lds, 0)
    assert g(n=0, y=0, c=0, s=0) == ra.LORA_OK
    for kw in (dict(inter=40), dict(y=0), dict(c=0), dict(s=0), dict(ldc=16), dict(lds=0)):
        assert g(**kw) == ra.LORA_EINVAL, kw
    for kw in (dict(y=P + 8), dict(c=P + 8), dict(ldc=40), dict(s=P + 2), dict(lds=20)):
        assert g(**kw) == ra.LORA_EALIGN, kw


def test_combine(ra):
    def f(y=P, ldy=64, ydt=ra.LORA_BF16, w=P, slot=P, T=3, topk=2, n=64, out=P, ldo=64, odt=ra.LORA_BF16):
        return ra.lora_moe_combine(y, ldy, ydt, w, slot, T, topk, n, out, ldo, odt, False, 0)
    assert f(T=0, y=0, w=0, out=0) == ra.LORA_OK
    for kw in (dict(ydt=ra.LORA_MXFP4), dict(odt=7), dict(n=0), dict(n=12), dict(y=0), dict(w=0), dict(out=0),
               dict(ldy=56), dict(ldo=56)):
        assert f(**kw) == ra.LORA_EINVAL, kw
    for kw in (dict(topk=0), dict(topk=65), dict(T=-1), dict(T=1 << 23, topk=4)):
        assert f(**kw) == ra.LORA_ERANGE, kw
    for kw in (dict(y=P + 2), dict(out=P + 8), dict(w=P + 2), dict(slot=P + 1), dict(ldy=68), dict(ldo=68)):
        assert f(**kw) == ra.LORA_EALIGN, kw


def test_binding_checks_shapes(ra):
    import torch
    z = torch.zeros
    with pytest.raises(ValueError):
        ra.ExpertWeights(z(2, 16, 32).transpose(1, 2))
    with pytest.raises(ValueError):
        ra.ExpertWeights(z(2, 16, 16, dtype=torch.uint8), z(2, 8, 16, dtype=torch.uint8))
    with pytest.raises(TypeError):
        ra.ExpertWeights(z(2, 16, 32, dtype=torch.float16))
    with pytest.raises(ValueError):
        ra.moe_combine(z(3, 16), z(2, 2), z(2, 16))
    with pytest.raises(ValueError):
        ra.moe_act(z(2, 32), z(3, 16))
    with pytest.raises(ValueError):
        ra.mx4_dequantize(z(3, 16, dtype=torch.uint8), z(3, 16, dtype=torch.uint8), z(4, 32))
    with pytest.raises(ValueError):
        ra.moe_route(z(4, 32).t(), 2)
    for bad in (lambda: ra.moe_act(z(4, 32), z(4, 16), pair_slot=z(4)),                                   # slots not int32
                lambda: ra.moe_act(z(4, 32), z(4, 16), pair_slot=z(3, dtype=torch.int32)),
                lambda: ra.moe_combine(z(4, 16), z(2, 2, dtype=torch.int32), z(2, 16)),                   # weights not fp32
                lambda: ra.moe_route(z(4, 8), 2, expert_map=z(7, dtype=torch.int32), topk_ids=z(4, 2, dtype=torch.int32),
                                     topk_w=z(4, 2)),
                lambda: ra.mx4_quantize(z(64, 2).t())):
        with pytest.raises(ValueError):
            bad()
    u8 = dict(dtype=torch.uint8)
    for bad in (lambda: ra.moe_act(z(4, 32, dtype=torch.float16), z(4, 16)), lambda: ra.moe_act([1], z(4, 16)),
                lambda: ra.mx4_quantize(z(3, 32), z(3, 16), z(3, 16, **u8)),
                lambda: ra.mx4_dequantize(z(3, 16, **u8), z(3, 16, **u8), z(3, 32, dtype=torch.int32)),
                lambda: ra.moe_route(z(4, 8), "two", topk_ids=z(4, 2, dtype=torch.int32), topk_w=z(4, 2))):
        with pytest.raises(TypeError):
            bad()


def test_product_binding_checks(ra):
    import torch
    z, u8 = torch.zeros, dict(dtype=torch.uint8)

    class Meta:                                         # what moe_product reads of a TokenMeta
        c = ra.Meta()
    Meta.c.num_tokens = 6
    w = ra.ExpertWeights(z(2, 16, 32), x_row_div=3)
    for x, y in ((z(1, 32), z(6, 16)), (z(2, 24), z(6, 16)), (z(2, 32), z(5, 16)), (z(2, 32), z(6, 24))):
        with pytest.raises(ValueError):
            ra.moe_product(w, Meta, x, y)
    for x in (z(2, 32).bfloat16(), z(2, 32, **u8), None):
        with pytest.raises(TypeError):
            ra.moe_product(w, Meta, x, z(6, 16))
    w.desc.dtype = ra.LORA_MXFP4                        # as 4-bit weights: codes and scales
    with pytest.raises(TypeError):
        ra.moe_product(w, Meta, z(2, 16, **u8), z(6, 16))
    with pytest.raises(TypeError):
        ra.moe_product(w, Meta, z(2, 16), z(6, 16), x_scale=z(2, 16, **u8))
    with pytest.raises(ValueError):
        ra.moe_product(w, Meta, z(2, 16, **u8), z(6, 16), x_scale=z(1, 16, **u8))
