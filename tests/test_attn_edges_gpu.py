"""The attention calls where a serving loop can go wrong: sequences and page ids that do not hold, graphs whose lengths
change between replays, side streams, caches past 2^31 elements, and a layer's calls in a row with its adapters."""
import numpy as np
import pytest
import torch

from attn_harness import Step, f64
from oracle import attn_oracle

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
# The kernels: few rows, tiles of 128 rows, the CUDA cores.
KERNELS = [pytest.param(dict(heads=(8, 2, 128), new=[1, 3, 2, 1]), id="few"),
           pytest.param(dict(heads=(8, 2, 64), new=[70, 3, 150, 1]), id="tiles"),
           pytest.param(dict(heads=(4, 2, 80), new=[20, 3, 2, 1]), id="cores")]


def step(k, before=(100, 40, 0, 500), **kw):
    return Step(*k["heads"], k["new"], before, seed=21, **kw)


def status(lib, s):
    torch.cuda.synchronize()
    return lib.lora_query_seqs(s.seqs.c)


@pytest.mark.parametrize("k", KERNELS)
@pytest.mark.parametrize("what", ["negative keys", "too many keys", "rows past the batch", "falling rows", "negative rows"])
def test_sequences_that_do_not_hold_are_empty(lib, k, what):
    s = step(k)
    s.write()
    s.paged()
    clean = s.out.clone()
    start, kv = s.start.copy(), s.kv.copy()
    bad = [2]
    if what == "negative keys":
        kv[2] = -1
    elif what == "too many keys":
        kv[2] = s.most_pages * s.page + 1
    else:
        start[3] = {"rows past the batch": s.T + 5, "falling rows": start[2] - 1, "negative rows": -7}[what]
        bad = [2] if what == "falling rows" else [2, 3]
    q, L = torch.from_numpy(start).cuda(), torch.from_numpy(kv).cuda()
    s.seqs.prepare(s.T, q, L, s.table)
    s.out.fill_(7.0)
    kc = s.kc.clone()
    s.write()
    s.paged()
    assert status(lib, s) == (lib.LORA_EBADSEQ, len(bad))
    if what != "falling rows":                                         # (there sequence 3 has a row more)
        assert torch.equal(s.kc.nan_to_num(3.0), kc.nan_to_num(3.0))   # the good ones write what is there already
    for b in range(4):
        r0, r1 = int(s.start[b]), int(s.start[b + 1])
        if what == "falling rows":                                     # row r1 - 1 of sequence 1 is sequence 3's first, too
            r1 -= b == 1
        if b not in bad and not (what == "falling rows" and b == 3):
            assert torch.equal(s.out[r0:r1], clean[r0:r1]), b
    if what in ("negative keys", "too many keys"):
        assert (s.out[int(s.start[2]):int(s.start[3])] == 7.0).all()
    s.seqs.prepare(s.T, s.q_start, s.kv_len, s.table)                  # the next plan starts anew
    s.write()
    s.paged()
    assert status(lib, s) == (lib.LORA_OK, 0)
    assert what == "falling rows" or torch.equal(s.out, clean)         # (there a cached key of sequence 3 was written over)


@pytest.mark.parametrize("bad", [[1], [2, 3], [0], [4], [0, 2, 4]])
def test_neighbours_of_sequences_that_do_not_hold_are_written(lib, bad):
    """Their rows belong to nobody; those of the sequences before and behind them go to the cache as ever."""
    s = Step(8, 2, 64, [5, 1, 3, 0, 7], [40, 9, 0, 16, 2], seed=25)
    kv = s.kv.copy()
    kv[bad] = -1
    s.seqs.prepare(s.T, s.q_start, torch.from_numpy(kv).cuda(), s.table)
    kc, vc = s.kc.clone(), s.vc.clone()
    s.write()
    assert status(lib, s) == (lib.LORA_EBADSEQ, len(bad))
    table = s.table.cpu().numpy()
    for b in range(5):
        if b not in bad:
            p = np.arange(s.before[b], s.kv[b])
            rows = slice(int(s.start[b]), int(s.start[b + 1]))
            for new, cache in ((s.k, kc), (s.v, vc)):
                cache[torch.from_numpy(table[b, p // s.page]).long().cuda(), torch.from_numpy(p % s.page).cuda()] = new[rows].reshape(-1, 2, 64)
    assert torch.equal(s.kc.nan_to_num(3.0), kc.nan_to_num(3.0)) and torch.equal(s.vc.nan_to_num(3.0), vc.nan_to_num(3.0))


@pytest.mark.parametrize("heads, new, before", [
    pytest.param((8, 2, 64), [1] * 1500, [i % 37 for i in range(1500)], id="few"),
    pytest.param((4, 2, 64), [1 + 97 * (i % 29 == 0) for i in range(1100)], [i % 150 for i in range(1100)], id="drafts"),
    pytest.param((8, 1, 64), [65 + i % 3 for i in range(1030)], [200 * (i % 100 == 7) for i in range(1030)], id="tiles"),
    pytest.param((2, 2, 40), [i % 3 for i in range(1100)], [5 * (i % 4) for i in range(1100)], id="cores")])
def test_more_sequences_than_a_plan_keeps_at_hand(lib, heads, new, before):
    s = Step(*heads, new, before, page=8, seed=26, pad_rows=3)
    s.write()
    s.paged()
    s.check()


@pytest.mark.parametrize("heads", [(4, 1, 128), (8, 2, 64)], ids=str)
def test_units_of_one_tile_ahead_of_units_of_two(lib, heads):
    """A CTA's first blocks are one stream's alone, its next both streams'. (Beside a long sequence the plan does not tell
    the costs of short ones apart, so that they come in any order.)"""
    r = np.random.default_rng(27)
    new = [64] + [int(r.choice([1, 20, 64, 40])) for _ in range(600)]
    s = Step(*heads, new, [70000] + [int(r.choice([0, 0, 130, 250])) for _ in range(600)], page=64, seed=27)
    s.write()
    s.paged()
    s.check()


@pytest.mark.parametrize("k", KERNELS)
def test_page_ids_outside_the_cache(lib, k):
    """Their keys count as zeros, nothing is written through them, and both are reported."""
    s = step(k, page=16)
    s.write()
    s.table[0, 2], s.table[3, 0], s.table[3, 1] = -1, s.kc.shape[0], (1 << 31) - 1
    last = (s.before[1] + s.new[1] - 1) // 16                          # the page that holds sequence 1's last row
    s.paged()
    s.check(status=lib.LORA_EBADSEQ)
    s.seqs.prepare(s.T, s.q_start, s.kv_len, s.table)
    assert status(lib, s) == (lib.LORA_OK, 0)
    s.table[1, last] = -5
    kc, vc = s.kc.clone(), s.vc.clone()
    s.k.mul_(2), s.v.mul_(2)
    s.write()
    assert status(lib, s)[0] == lib.LORA_EBADSEQ
    for b, (n, c) in enumerate(zip(s.new, s.before)):
        for i in range(n):
            page = int(s.table[b, (c + i) // 16])
            if 0 <= page < kc.shape[0]:
                kc[page, (c + i) % 16] = s.k[s.start[b] + i].view(s.K, s.D)
                vc[page, (c + i) % 16] = s.v[s.start[b] + i].view(s.K, s.D)
    assert torch.equal(kc.nan_to_num(3.0), s.kc.nan_to_num(3.0)) and torch.equal(vc.nan_to_num(3.0), s.vc.nan_to_num(3.0))


@pytest.mark.parametrize("heads", [(8, 2, 128), (4, 4, 64)], ids=str)
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_unseen_values_of_drafts(lib, heads, value):
    """As of prompts: a later draft token's values, in the cache already, do not reach the rows before it."""
    for before in ([100, 30, 0], [3000, 2000, 900]):                   # the latter in pieces along the keys
        s = Step(*heads, [3, 2, 4], before, seed=22, pad_rows=1)
        s.write()
        s.paged()
        s.check()
        clean = s.out.clone()
        last = torch.tensor([2, 4, 8])
        s.v[last] = value
        s.write()
        s.paged()
        for a, b in ((0, 2), (3, 4), (5, 8)):
            assert torch.equal(s.out[a:b], clean[a:b])
        got = s.out[last]
        assert torch.isnan(got).all() if value != value else (got == value).all()


@pytest.mark.parametrize("k", KERNELS + [pytest.param(dict(heads=(32, 8, 128), new=[1] * 4), id="decode")])
@pytest.mark.parametrize("times", [64.0, float("inf"), float("nan")])
def test_other_sequences_do_not_reach_a_result(lib, k, times):
    """Bitwise: neither through the softmax's base, which large scores of others would raise."""
    s = step(k, before=(300, 700, 0, 500))
    s.write()
    s.paged()
    out, lse = s.out.clone(), s.lse.clone()
    for b in (0, 2):
        s.q[int(s.start[b]):int(s.start[b + 1])] *= times
    s.paged()
    torch.cuda.synchronize()
    for b in (1, 3):
        r = slice(int(s.start[b]), int(s.start[b + 1]))
        assert torch.equal(s.out[r], out[r]) and torch.equal(s.lse[r], lse[r])


def test_large_scores_of_few_rows(lib):
    s = Step(8, 2, 128, [1, 2, 1], [900, 300, 5], spread=60.0, seed=23)
    s.write()
    s.paged()
    s.check()


@pytest.mark.parametrize("new", [[1] * 6, [4, 3, 4, 3, 4, 3]], ids=str)
@pytest.mark.parametrize("heads", [(8, 2, 128), (8, 2, 64), (16, 2, 128), (16, 2, 64), (28, 4, 128), (64, 1, 64), (64, 1, 128), (14, 2, 64)], ids=str)
def test_weights_of_few_rows_are_two_bf16(lib, heads, new):
    """Off by half a step of half a step: (2^-8)^2 = 2^-16 of a weight, beside the output's own rounding. With more than 32
    rows of a key-value head a sequence on average they are one bf16."""
    s = Step(*heads, new, [3000, 1, 0, 700, 127, 5000], page=32, seed=28)
    few = s.used * heads[0] // heads[1] <= 32 * len(new)
    s.write()
    s.paged()
    s.check()
    out, lse, spread, reach = s.oracle()
    tol, _ = attn_oracle.tolerance(out, lse, spread, reach, s.D, int(s.kv.max()), 2.0 ** -16 if few else 2.0 ** -8, 2.0 ** -8)
    assert (np.abs(f64(s.out).reshape(out.shape) - out) <= tol).all()


@pytest.mark.parametrize("heads,new", [((4, 2, 128), [3] * 9), ((2, 1, 64), [1, 9, 0, 2]), ((64, 1, 64), [1] * 5), ((8, 8, 128), [2, 31])], ids=str)
def test_short_prompts(lib, heads, new):
    s = Step(*heads, new, seed=24, pad_rows=2)
    s.prompt()
    s.check()


@pytest.mark.parametrize("k", KERNELS)
def test_graph_with_lengths_that_change(lib, k):
    """Plan, write and attention in a graph: replays take the lengths, tables and rows that are there then."""
    s = step(k, page=32)
    ws = lib.attn_workspace(s.seqs)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())

    def run():
        s.seqs.prepare(s.T, s.q_start, s.kv_len, s.table)
        s.write()
        s.paged(ws=ws)
    with torch.cuda.stream(stream):
        run()
    stream.synchronize()
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]          # two of them share the workspace and the plan
    for g in graphs:
        with torch.cuda.graph(g, stream=stream):
            run()
    r = np.random.default_rng(3)
    for i in range(4):
        before = np.array([r.integers(0, c + 1) for c in (100, 40, 0, 500)])
        s.before, s.kv = list(before), (before + np.array(s.new)).astype(np.int32)
        s.kv_len.copy_(torch.from_numpy(s.kv))
        s.table.copy_(s.table[torch.tensor([0, 1, 2, 3])])
        s.q.copy_(torch.randn_like(s.q.float()).to(s.dtype))
        s.k.copy_(torch.randn_like(s.k.float()).to(s.dtype))
        s.out.fill_(7.0)
        s.kc.copy_(torch.randn_like(s.kc.float()).to(s.dtype)), s.vc.copy_(torch.randn_like(s.vc.float()).to(s.dtype))
        graphs[i % 2].replay()
        s.check()


@pytest.mark.parametrize("k", KERNELS)
def test_side_streams(lib, k):
    """Two streams at once, each with its own plan and scratch that the call allocates; tensors dropped at once."""
    steps = [step(k), step(k)]
    for s in steps:
        s.write()
        s.paged()
    torch.cuda.synchronize()
    want = [s.out.clone() for s in steps]
    streams = [torch.cuda.Stream() for _ in steps]
    for s in steps:
        s.out.fill_(7.0)
    torch.cuda.synchronize()
    for _ in range(5):
        for s, st in zip(steps, streams):
            s.seqs.prepare(s.T, s.q_start.clone(), s.kv_len.clone(), s.table, stream=st)
            s.write(stream=st)
            s.paged(stream=st)
            torch.full((1 << 20,), -1, dtype=torch.int32, device="cuda")   # takes freed memory of the current stream
    torch.cuda.synchronize()
    for s, w in zip(steps, want):
        assert torch.equal(s.out, w)


def test_one_plan_on_two_streams(lib):
    """Layers of one plan may run at the same time where each has its own workspace."""
    s = Step(8, 2, 128, [1, 1, 4], [5000, 3000, 40], seed=26)
    s.write()
    s.paged()
    torch.cuda.synchronize()
    want, outs = s.out.clone(), [torch.zeros_like(s.out) for _ in range(2)]
    ws, streams = [lib.attn_workspace(s.seqs) for _ in range(2)], [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for o, w, st in zip(outs, ws, streams):
            lib.attn_paged(s.seqs, s.cache, s.q, o, ws=w, stream=st)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)


def test_a_cache_past_32_bits_of_elements(lib):
    pages = (1 << 31) // (2 * 16 * 128) + 300                          # k and v side by side: more than 2^31 elements
    cache = torch.empty(pages, 2, 16, 1, 128, dtype=BF16, device="cuda")
    for heads, n in ((4, 3), (8, 40)):                                 # few rows; a tile of 128
        s = Step(heads, 1, 128, [n], [50], seed=27)
        used = -(-(50 + n) // 16)
        ids = torch.arange(used, dtype=torch.int32) + (pages - used - 1)
        cache[pages - used - 1:pages - 1, 0] = s.kc[s.table[0, :used].long()]
        cache[pages - used - 1:pages - 1, 1] = s.vc[s.table[0, :used].long()]
        s.table = ids.cuda()[None]
        s.cache = lib.KVCache(cache[:, 0], cache[:, 1])
        s.seqs.prepare(s.T, s.q_start, s.kv_len, s.table)
        s.write()
        s.paged()
        keys = [f64(cache[pages - used - 1:pages - 1, i]).reshape(-1, 1, 128)[:50 + n] for i in range(2)]
        s.check(s.oracle([keys[0]], [keys[1]]))


def test_a_prompt_into_the_cache(lib):
    """One plan for the write and the prompt's attention, which is the attention over the cache afterwards."""
    s = Step(8, 2, 128, [100, 1, 37], [0, 0, 0], seed=28)
    s.seqs.prepare(s.T, s.q_start, None, s.table)
    s.write()
    s.prompt()
    s.check()
    s.out.fill_(7.0)
    s.paged()
    s.check()
    with pytest.raises(ValueError, match="kv_len"):
        s.seqs.prepare(s.T, s.q_start, s.kv_len, s.table)
        s.prompt()


def test_out_must_not_be_the_input(lib):
    s = Step(4, 4, 64, [5], seed=29)
    for out in (s.q, s.k, s.v):
        with pytest.raises(lib.LoraError):
            lib.attn_prompt(s.seqs, s.q, s.k, s.v, out)


@pytest.mark.parametrize("new,before", [([1] * 6, [200, 3, 0, 700, 15, 16]), ([40, 1, 90], [10, 60, 0])], ids=["decode", "prefill"])
def test_layer_with_its_adapters(lib, new, before):
    """qkv adapter -> cache write -> attention -> o adapter, all on packed rows, as a layer runs them."""
    H, K, D, d_in, r = 8, 2, 128, 256, 16
    g = torch.Generator().manual_seed(30)
    rnd = lambda *z: torch.randn(*z, generator=g).to(BF16).cuda()  # noqa: E731
    s = Step(H, K, D, new, before, seed=30)
    qkv, o = lib.SlotTable(d_in, [H * D, K * D, K * D], 3, r), lib.SlotTable(H * D, [d_in], 3, r)
    Bs, Ao, Bo = {}, {}, {}
    for slot in (1, 2):
        A, Bs[slot] = [rnd(d_in, r) / 16 for _ in range(3)], [rnd(r, w) / 4 for w in (H * D, K * D, K * D)]
        Ao[slot], Bo[slot] = rnd(H * D, r) / 32, rnd(r, d_in) / 4
        qkv.set_slot(slot, r, 1.0, A, Bs[slot])
        o.set_slot(slot, r, 2.0, [Ao[slot]], [Bo[slot]])
        Bs[slot] = (A, Bs[slot])
    slots = torch.tensor(np.repeat(np.arange(len(new)) % 3, new), dtype=torch.int32).cuda()
    meta = lib.TokenMeta(s.T, 3)
    meta.prepare(slots)
    x, y = rnd(s.T, d_in), rnd(s.T, d_in)
    base, y0 = s.qkv.clone(), y.clone()
    lib.apply(qkv, meta, x, s.qkv)
    s.write()
    s.paged()
    lib.apply(o, meta, s.out, y)
    s.check()
    want_qkv, want_y = f64(base), f64(y0)
    for t in range(s.T):
        slot = int(slots[t])
        if slot:
            A, B = Bs[slot]
            want_qkv[t] += np.concatenate([f64(x[t]) @ f64(A[i]) @ f64(B[i]) for i in range(3)])
            want_y[t] += 2.0 * (f64(s.out[t]) @ f64(Ao[slot]) @ f64(Bo[slot]))
    for got, want in ((s.qkv, want_qkv), (y, want_y)):
        rms = np.sqrt(np.mean(want ** 2))
        assert np.max(np.abs(f64(got) - want)) <= 1e-2 * rms + 2.0 ** -8 * np.abs(want).max()
