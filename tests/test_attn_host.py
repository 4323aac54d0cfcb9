"""The attention calls refuse bad arguments on the host, before any launch (no GPU needed)."""
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 0x100000
I32 = dict(dtype=torch.int32)
z = torch.zeros


@pytest.fixture(scope="module")
def ra():
    import __graft_entry__
    __graft_entry__._load_build_lib().build()
    import rank_adapter_gb300
    return rank_adapter_gb300


def test_constants_match_the_header(ra):
    src = open(os.path.join(ROOT, "include", "lora.h")).read()
    for name in ("LORA_MAX_SEQS", "LORA_MAX_HEADS", "LORA_MAX_HEAD_DIM"):
        assert int(re.search(rf"#define {name} (\d+)", src).group(1)) == getattr(ra, name)
    assert re.search(r"#define LORA_MAX_KV_LEN \(1 << 24\)", src) and ra.LORA_MAX_KV_LEN == 1 << 24
    assert re.search(rf"LORA_EBADSEQ = {ra.LORA_EBADSEQ}\b", src)
    assert "unknown" not in ra.lora_strerror(ra.LORA_EBADSEQ)


def seqs(ra, dt=None, H=8, K=2, D=128, causal=1, scale=0.1, S=4, T=40, page=16, pages=10, table=P, ldt=10, q=P, kv=P, plan=P, nb=None):
    d = ra.SeqsDesc()
    d.dtype, d.num_heads, d.num_kv_heads, d.head_dim = ra.LORA_BF16 if dt is None else dt, H, K, D
    d.causal, d.scale, d.q_start, d.kv_len, d.num_seqs, d.num_tokens = causal, scale, q or None, kv or None, S, T
    d.page_size, d.max_pages, d.block_table, d.ld_table, d.plan = page, pages, table or None, ldt, plan or None
    d.plan_bytes = ra.lora_seqs_plan_bytes(d) if nb is None else nb
    return d


GEOMETRY = [(dict(dt=2), "EINVAL"), (dict(H=0), "ERANGE"), (dict(H=1025, K=1), "ERANGE"), (dict(K=0), "ERANGE"), (dict(K=16), "ERANGE"),
            (dict(K=3), "EINVAL"), (dict(D=0), "ERANGE"), (dict(D=264), "ERANGE"), (dict(D=12), "EINVAL"), (dict(scale=0.0), "EINVAL"),
            (dict(scale=-1.0), "EINVAL"), (dict(scale=float("inf")), "EINVAL"), (dict(scale=float("nan")), "EINVAL"),
            (dict(S=-1), "ERANGE"), (dict(S=16385), "ERANGE"), (dict(T=-1), "ERANGE"), (dict(T=(1 << 24) + 1), "ERANGE")]
PLAN = [(dict(page=4), "EINVAL"), (dict(page=24), "EINVAL"), (dict(page=2048), "EINVAL"), (dict(page=-16), "EINVAL"), (dict(pages=0), "ERANGE"),
        (dict(pages=(1 << 20) + 1), "ERANGE"), (dict(plan=0), "EINVAL"), (dict(nb=64), "EINVAL"), (dict(plan=P + 8), "EALIGN")]


def test_prepare(ra):
    assert ra.lora_seqs_plan_bytes(seqs(ra)) > 0 and ra.lora_attn_workspace_bytes(seqs(ra)) > 0
    for kw, st in GEOMETRY + PLAN + [(dict(q=0), "EINVAL"), (dict(q=P + 2), "EALIGN"), (dict(kv=P + 1), "EALIGN")]:
        assert ra.lora_prepare_seqs(seqs(ra, **kw), 0) == getattr(ra, "LORA_" + st), kw
        if (kw, st) in GEOMETRY:
            assert ra.lora_seqs_plan_bytes(seqs(ra, **kw)) == 0 and ra.lora_attn_workspace_bytes(seqs(ra, **kw)) == 0


def cache(ra, k=P, v=2 * P, pages=50, strides=(4096, 256, 128, 4096, 256, 128)):
    c = ra.KVCacheDesc()
    c.k, c.v, c.num_pages = k or None, v or None, pages
    c.k_page, c.k_row, c.k_head, c.v_page, c.v_row, c.v_head = strides
    return c


CACHE = [(dict(k=0), "EINVAL"), (dict(v=0), "EINVAL"), (dict(pages=0), "ERANGE"), (dict(k=P + 8), "EALIGN"), (dict(v=P + 2), "EALIGN"),
         (dict(strides=(4096, 256, 0, 4096, 256, 128)), "EINVAL"), (dict(strides=(4096, 256, 128, 4096, -256, 128)), "EINVAL"),
         (dict(strides=(4096, 260, 128, 4096, 256, 128)), "EALIGN")]


def test_write(ra):
    def f(s={}, c={}, k=3 * P, ldk=256, v=4 * P, ldv=256):
        return ra.lora_kv_write(seqs(ra, **s), cache(ra, **c), k, ldk, v, ldv, 0)
    assert f(dict(S=0, q=0, kv=0)) == ra.LORA_OK and f(dict(T=0), k=0, v=0) == ra.LORA_OK
    for kw, st in GEOMETRY + PLAN + [(dict(page=0), "EINVAL"), (dict(table=0), "EINVAL"), (dict(table=P + 1), "EALIGN"), (dict(ldt=9), "EINVAL")]:
        assert f(kw) == getattr(ra, "LORA_" + st), kw
    for kw, st in CACHE:
        assert f(c=kw) == getattr(ra, "LORA_" + st), kw
    for kw, st in [(dict(k=0), "EINVAL"), (dict(v=0), "EINVAL"), (dict(ldk=248), "EINVAL"), (dict(ldv=0), "EINVAL"), (dict(k=P + 4), "EALIGN"),
                   (dict(ldv=260), "EALIGN")]:
        assert f(**kw) == getattr(ra, "LORA_" + st), kw


ROWS = [(dict(q=0), "EINVAL"), (dict(out=0), "EINVAL"), (dict(ldq=1016), "EINVAL"), (dict(ldo=1000), "EINVAL"), (dict(q=P + 8), "EALIGN"),
        (dict(out=7 * P + 2), "EALIGN"), (dict(ldo=1028), "EALIGN"), (dict(lse=P + 2), "EALIGN"), (dict(ws=0), "EINVAL"), (dict(ws=P + 4), "EALIGN"),
        (dict(nws=100), "EINVAL"), (dict(out=3 * P), "EINVAL"), (dict(out=3 * P + 1024 * 2), "EINVAL"), (dict(out=3 * P + 1024, ldo=1032), "EINVAL")]


def test_prompt(ra):
    def f(s={}, q=3 * P, ldq=1024, k=4 * P, ldk=256, v=5 * P, ldv=256, out=6 * P, ldo=1024, lse=0, ws=P, nws=1 << 40):
        return ra.lora_attn_prompt(seqs(ra, **{**dict(kv=0), **s}), q, ldq, k, ldk, v, ldv, out, ldo, lse, ws, nws, 0)
    assert f(dict(S=0, q=0)) == ra.LORA_OK and f(dict(T=0), q=0, k=0, v=0, out=0, ws=0) == ra.LORA_OK
    for kw, st in GEOMETRY + PLAN + [(dict(kv=P), "EINVAL")]:
        assert f(kw) == getattr(ra, "LORA_" + st), kw
    for kw, st in ROWS + [(dict(k=0), "EINVAL"), (dict(v=0), "EINVAL"), (dict(ldk=0), "EINVAL"), (dict(ldv=252), "EINVAL"), (dict(ldk=260), "EALIGN"),
                          (dict(v=P + 4), "EALIGN"), (dict(out=4 * P), "EINVAL"), (dict(k=5 * P + 512, v=6 * P + 1024), "EINVAL")]:
        assert f(**kw) == getattr(ra, "LORA_" + st), kw


def test_paged(ra):
    def f(s={}, c={}, q=3 * P, ldq=1024, out=6 * P, ldo=1024, lse=0, ws=P, nws=1 << 40):
        return ra.lora_attn_paged(seqs(ra, **s), cache(ra, **c), q, ldq, out, ldo, lse, ws, nws, 0)
    assert f(dict(S=0, q=0, kv=0)) == ra.LORA_OK and f(dict(T=0), q=0, out=0, ws=0) == ra.LORA_OK
    for kw, st in GEOMETRY + PLAN + [(dict(page=0), "EINVAL"), (dict(table=0), "EINVAL"), (dict(ldt=9), "EINVAL")]:
        assert f(kw) == getattr(ra, "LORA_" + st), kw
    for kw, st in CACHE:
        assert f(c=kw) == getattr(ra, "LORA_" + st), kw
    for kw, st in ROWS:
        assert f(**kw) == getattr(ra, "LORA_" + st), kw


def test_columns_of_one_matrix_do_not_overlap(ra):
    """q, k, v and out as column ranges of one matrix: refused only for null scratch, the last check."""
    d = seqs(ra, kv=0)
    assert ra.lora_attn_prompt(d, P, 2576, P + 2048, 2576, P + 2560, 2576, P + 3088, 2576, 0, 0, 0, 0) == ra.LORA_EINVAL
    assert ra.lora_attn_prompt(d, P, 2576, P + 2048, 2576, P + 2560, 2576, P + 3088, 2576, 0, P + 4, 1 << 40, 0) == ra.LORA_EALIGN


def test_query(ra):
    d = seqs(ra, plan=0)
    assert ra.lora_query_seqs(d, 0)[0] == ra.LORA_EINVAL


# ---- the tensor forms

def meta(ra, S=2, T=6, page=16, pages=4, H=4, K=2, D=64, dtype=None):
    att = ra.Attention(H, K, D, dtype=ra.LORA_BF16 if dtype is None else dtype)
    return ra.SeqMeta(att, T, S, page, pages, device="cpu")


def test_geometry_is_refused_at_once(ra):
    for kw in (dict(H=3), dict(D=12), dict(D=512), dict(S=-1), dict(T=-1)):
        with pytest.raises(ValueError, match="invalid geometry"):
            meta(ra, **kw)


def test_prepare_refuses_tensors(ra):
    m = meta(ra)
    q, kv, t = z(3, **I32), z(2, **I32), z(2, 4, **I32)
    for args, what in [((6, z(4, **I32)), "q_start"), ((6, z(0, **I32)), "q_start"), ((7, q), "num_tokens"), ((-1, q), "num_tokens"),
                       ((6, z(3, dtype=torch.int64)), "q_start"), ((6, z(6, **I32)[::2]), "q_start"), ((6, q, z(3, **I32)), "kv_len"),
                       ((6, q, z(2)), "kv_len"), ((6, q, kv, z(1, 4, **I32)), "block_table"), ((6, q, kv, z(2, 3, **I32)), "block_table"),
                       ((6, q, kv, z(2, 4)), "block_table"), ((6, q, kv, z(4, 2, **I32).t()), "block_table"),
                       ((6, q, kv, z(1, 4, **I32).expand(2, 4)), "block_table"), ((6, q, kv, t), "expected a CUDA tensor")]:
        with pytest.raises(ValueError, match=what):
            m.prepare(*args)
    with pytest.raises(ValueError, match="no pages"):
        meta(ra, page=0, pages=0).prepare(6, q, kv, t)
    assert m.c.num_seqs == 0 and m.q_start is None      # a refused call leaves it as it was


def test_cache_refuses_tensors(ra):
    bf = dict(dtype=torch.bfloat16)
    k = z(5, 16, 2, 64, **bf)
    for a, b in [(k, z(4, 16, 2, 64, **bf)), (k, z(5, 16, 2, 64)), (z(5, 16, 128, **bf), z(5, 16, 128, **bf)),
                 (z(5, 16, 64, 2, **bf).transpose(2, 3), k)]:
        with pytest.raises(ValueError, match="KVCache: expected"):
            ra.KVCache(a, b)
    with pytest.raises(ValueError, match="overlap"):
        ra.KVCache(z(1, 16, 2, 64, **bf).expand(5, 16, 2, 64), k)
    with pytest.raises(TypeError, match="bf16 or fp32"):
        ra.KVCache(k.half(), k.half())


def test_calls_refuse_tensors(ra):
    bf = dict(dtype=torch.bfloat16)
    m = meta(ra)
    m.c.num_seqs, m.c.num_tokens, m.block_table = 2, 6, z(2, 4, **I32)
    c = ra.KVCache(z(5, 16, 2, 64, **bf), z(5, 16, 2, 64, **bf))
    q, k, out, ws = z(6, 256, **bf), z(6, 128, **bf), z(6, 256, **bf), z(8, dtype=torch.uint8)
    for call, error, what in [
            (lambda: ra.kv_write(m, c, z(5, 128, **bf), k), ValueError, "k: expected"),
            (lambda: ra.kv_write(m, c, k, z(6, 64, **bf)), ValueError, "v: expected"),
            (lambda: ra.kv_write(m, c, k.float(), k), TypeError, "k: not of"),
            (lambda: ra.kv_write(m, c, k, k), ValueError, "CUDA"),
            (lambda: ra.kv_write(m, ra.KVCache(z(5, 8, 2, 64, **bf), z(5, 8, 2, 64, **bf)), k, k), ValueError, "cache: expected"),
            (lambda: ra.kv_write(m, ra.KVCache(z(5, 16, 2, 64), z(5, 16, 2, 64)), k, k), TypeError, "cache: not of"),
            (lambda: ra.attn_paged(m, c, q[:, :128], out, ws=ws), ValueError, "q: expected"),
            (lambda: ra.attn_paged(m, c, q, out.half(), ws=ws), TypeError, "out: expected"),
            (lambda: ra.attn_paged(m, c, q, out, lse=z(6, 3), ws=ws), ValueError, "lse: expected"),
            (lambda: ra.attn_paged(m, c, q, out, lse=z(6, 4, dtype=torch.float64), ws=ws), ValueError, "lse: expected"),
            (lambda: ra.attn_paged(m, c, q, out, ws=z(8, 2, dtype=torch.uint8).t()), ValueError, "ws: expected"),
            (lambda: ra.attn_paged(m, c, q, out, ws=ws), ValueError, "CUDA"),
            (lambda: ra.attn_prompt(m, q, k, k, z(1, 256, **bf).expand(6, 256), ws=ws), ValueError, "overlap"),
            (lambda: ra.attn_prompt(m, q, k, k[:, ::2], out, ws=ws), ValueError, "v: expected"),
            (lambda: ra.attn_prompt(m, q, k, k, out, ws=ws), ValueError, "CUDA")]:
        with pytest.raises(error, match=what):
            call()
    m.block_table = None
    for call in (lambda: ra.kv_write(m, c, k, k), lambda: ra.attn_paged(m, c, q, out, ws=ws)):
        with pytest.raises(ValueError, match="block_table"):
            call()
    m.c.kv_len = P
    with pytest.raises(ValueError, match="kv_len"):
        ra.attn_prompt(m, q, k, k, out, ws=ws)
