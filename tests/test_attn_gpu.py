"""The attention calls against the 64-bit oracle: types, head layouts, lengths from none to long ones, pages that end
inside a tile, rows without keys, splits along the keys."""
import numpy as np
import pytest
import torch

from attn_harness import Step, f64

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32

# (query heads, key-value heads, head size): groups of 1, 2, 4, 5, 7, 8 and 16, one that fills a tile, one above it
HEADS = [(4, 4, 64), (4, 2, 128), (8, 2, 128), (10, 2, 64), (14, 2, 128), (8, 1, 128), (16, 1, 64), (128, 1, 64), (160, 1, 128)]
OTHER = [(4, 2, 8), (3, 3, 40), (6, 2, 80), (4, 1, 136), (2, 1, 256)]     # sizes without a tensor-core tile
LENGTHS = [[1], [2, 1], [37, 1, 1, 12], [128], [129, 127], [0, 64, 0, 65], [300], [1, 260, 33]]


@pytest.mark.parametrize("heads", HEADS, ids=str)
@pytest.mark.parametrize("causal", [True, False])
def test_prompt_heads(lib, heads, causal):
    s = Step(*heads, [37, 1, 131, 0, 64], causal=causal, seed=1)
    s.prompt()
    s.check()


@pytest.mark.parametrize("new", LENGTHS, ids=str)
@pytest.mark.parametrize("heads", [(4, 2, 128), (3, 3, 64)], ids=str)
def test_prompt_lengths(lib, heads, new):
    s = Step(*heads, new, seed=2, pad_rows=5)
    s.prompt()
    s.check()


@pytest.mark.parametrize("heads", OTHER + [(4, 2, 64), (8, 1, 128), (160, 1, 16)], ids=str)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_other_sizes_and_fp32(lib, heads, dtype):
    s = Step(*heads, [33, 1, 0, 70], dtype=dtype, seed=3)
    s.prompt()
    s.check()
    s = Step(*heads, [3, 1, 40], [130, 7, 0], dtype=dtype, seed=4)
    s.write()
    s.paged()
    s.check()


@pytest.mark.parametrize("heads", HEADS, ids=str)
@pytest.mark.parametrize("page", [8, 16, 128, 256])
def test_decode(lib, heads, page):
    s = Step(*heads, [1] * 7, [0, 1, 15, 16, 127, 128, 500], page=page, seed=5, pad_rows=2)
    s.write()
    s.paged()
    s.check()


@pytest.mark.parametrize("page", [8, 16, 32, 64, 128, 512, 1024])
@pytest.mark.parametrize("heads", [(8, 2, 128), (5, 5, 64)], ids=str)
@pytest.mark.parametrize("causal", [True, False])
def test_chunks(lib, heads, page, causal):
    s = Step(*heads, [5, 70, 1, 0, 129], [300, 61, 0, 40, 3], page=page, causal=causal, seed=6)
    s.write()
    s.paged()
    s.check()


@pytest.mark.parametrize("layout", ["head", "both"])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_cache_layouts(lib, layout, dtype):
    s = Step(8, 2, 64, [5, 33], [100, 0], dtype=dtype, layout=layout, seed=7)
    s.write()
    s.paged()
    s.check()


@pytest.mark.parametrize("heads", [(8, 2, 128), (6, 2, 64), (4, 1, 80)], ids=str)
@pytest.mark.parametrize("new,before", [([1], [3000]), ([9], [2500]), ([1, 1, 2], [4000, 3, 700]), ([90], [1500])], ids=str)
def test_split_keys(lib, heads, new, before):
    """Few rows over many keys: the keys are cut and the parts joined; the same bits each time."""
    s = Step(*heads, new, before, seed=8)
    s.write()
    s.paged()
    s.check()
    first = s.out.clone()
    for _ in range(3):
        s.out.fill_(7.0)
        s.paged()
        assert torch.equal(first, s.out)


@pytest.mark.parametrize("heads", [(8, 8, 128), (8, 8, 64), (16, 4, 128)], ids=str)
def test_long_units(lib, heads):
    """So many sequences that none is split: a CTA walks several units of up to a dozen blocks of keys, odd and even, one and two tiles."""
    r = np.random.default_rng(14)
    s = Step(*heads, [1] * 20 + [2, 3, 40, 1, 100, 1] * 2, [int(x) for x in r.integers(1, 1500, 32)], seed=14)
    s.write()
    s.paged()
    s.check()
    s = Step(heads[0], heads[1], heads[2], [700, 1, 333, 20], seed=15)
    s.prompt()
    s.check()


@pytest.mark.parametrize("dtype,heads", [(BF16, (4, 2, 64)), (BF16, (2, 2, 128)), (F32, (4, 2, 64))])
def test_rows_without_keys(lib, dtype, heads):
    """Fewer keys than rows: the first rows see nothing under a causal mask, and get zeros and -inf."""
    s = Step(*heads, [6, 200, 3], [10, 0, 0], dtype=dtype, seed=9)
    s.write()
    s.kv = np.array([16, 70, 0], np.int32)
    s.kv_len.copy_(torch.from_numpy(s.kv))
    s.seqs.prepare(s.T, s.q_start, s.kv_len, s.table)
    s.paged()
    s.check()
    assert (f64(s.out)[6:6 + 130] == 0).all() and torch.isneginf(s.lse[6:6 + 130]).all() and torch.isneginf(s.lse[206:]).all()


@pytest.mark.parametrize("dtype,heads", [(BF16, (4, 2, 64)), (BF16, (4, 2, 128)), (F32, (4, 2, 64)), (BF16, (4, 2, 80))])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_unseen_values_do_not_reach_a_row(lib, dtype, heads, value):
    """A key or value that a row does not see may be anything: of a later token, of another sequence, of a slot past the keys."""
    new = [50, 20, 140]
    s = Step(*heads, new, dtype=dtype, seed=10)
    s.prompt()
    clean = s.out.clone()
    rows = torch.tensor([40, 69, 70 + 135])          # the last rows of each sequence see them
    s.k[rows] = value
    s.v[rows] = value
    s.prompt()
    for a, first, b in ((0, 40, 50), (50, 69, 70), (70, 205, 210)):
        assert torch.equal(s.out[a:first], clean[a:first])
        assert not torch.isfinite(s.out[first:b]).any()
    s = Step(*heads, new, [100, 0, 30], dtype=dtype, seed=11)
    s.write()
    s.paged()
    s.check()
    clean = s.out.clone()
    s.v[rows] = value                                # values alone: weights stay finite
    s.write()
    s.paged()
    for a, first, b in ((0, 40, 50), (50, 69, 70), (70, 205, 210)):
        assert torch.equal(s.out[a:first], clean[a:first])
        got = s.out[first:b]
        assert torch.isnan(got).all() if value != value else (got == value).all()


@pytest.mark.parametrize("dtype,D", [(BF16, 128), (F32, 64)])
def test_large_scores(lib, dtype, D):
    """Scores of some hundreds: weights fall to nothing beside the largest, sums stay finite."""
    s = Step(4, 2, D, [130, 7], dtype=dtype, spread=60.0, seed=12)
    s.prompt()
    s.check()


def test_write_is_exact_and_leaves_the_rest(lib):
    for dtype in (BF16, F32):
        s = Step(4, 2, 72, [1, 0, 19, 40], [15, 3, 16, 0], dtype=dtype, page=16, seed=13, pad_rows=3)
        kc, vc = s.kc.clone(), s.vc.clone()
        s.write()
        for b, (n, c) in enumerate(zip(s.new, s.before)):
            for i in range(n):
                page, slot = int(s.table[b, (c + i) // 16]), (c + i) % 16
                kc[page, slot] = s.k[s.start[b] + i].view(2, 72)
                vc[page, slot] = s.v[s.start[b] + i].view(2, 72)
        assert torch.equal(kc.nan_to_num(3.0), s.kc.nan_to_num(3.0)) and torch.equal(vc.nan_to_num(3.0), s.vc.nan_to_num(3.0))
