"""A call with ``stream=`` allocates, copies and keeps for that stream: what it returns is not memory that the
current stream may still be using, nor is memory it reads given back before it has been read."""
import pytest
import torch

pytestmark = pytest.mark.gpu
MB = 1 << 20


def _freed(nbytes):
    """Address of a block that has just gone back to the current stream's pool."""
    t = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    p = t.data_ptr()
    del t
    return p


def _outputs(lib):
    """name -> (call giving the tensors that it allocates, bytes of the first)"""
    T, K = 1 << 20, 16
    z = torch.zeros(T, K, device="cuda")
    x = torch.zeros(4096, 32768, dtype=torch.bfloat16, device="cuda")
    ids, slot = torch.zeros(T, K, dtype=torch.int32, device="cuda"), torch.zeros(T, dtype=torch.int32, device="cuda")
    w = torch.zeros(8, 8192, 4096, dtype=torch.uint8, device="cuda")
    sc = torch.zeros(8, 8192, 256, dtype=torch.uint8, device="cuda")
    return {"moe_route": (lambda s: lib.moe_route(z, K, stream=s), T * K * 4),
            "mx4_quantize": (lambda s: lib.mx4_quantize(x, stream=s), 64 * MB),
            "moe_pair_slots": (lambda s: (lib.moe_pair_slots(slot, ids, 1, 1, 1, stream=s),), T * K * 4),
            "ExpertWeights": (lambda s: (lib.ExpertWeights(w, sc, stream=s).scale,), 16 * MB)}


@pytest.mark.parametrize("name", ["moe_route", "mx4_quantize", "moe_pair_slots", "ExpertWeights"])
@pytest.mark.parametrize("raw", [False, True])
def test_outputs_come_from_the_streams_memory(lib, name, raw):
    call, nbytes = _outputs(lib)[name]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    was = _freed(nbytes)
    assert _freed(nbytes) == was                       # the current stream's pool gives that block next
    out = call(s.cuda_stream if raw else s)
    assert out[0].data_ptr() != was
    torch.cuda.synchronize()
    # Read on the current stream, then dropped: not given to the side stream before that.
    torch.cuda._sleep(100_000_000)
    p = out[0].data_ptr()
    del out
    with torch.cuda.stream(s):
        again = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    assert again.data_ptr() != p
    torch.cuda.synchronize()


def test_no_stream_is_the_current_one(lib):
    call, nbytes = _outputs(lib)["mx4_quantize"]
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    for s in (None, torch.cuda.current_stream()):
        was = _freed(nbytes)
        assert call(s)[0].data_ptr() == was
    torch.cuda.synchronize()


def test_expert_weights_scales_outlive_their_layout(lib):
    """The raw scales may be dropped at once: their memory is not reused while the side stream has yet to read it."""
    s = torch.cuda.Stream()
    w = torch.zeros(8, 8192, 4096, dtype=torch.uint8, device="cuda")
    sc = torch.zeros(8, 8192, 256, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(100_000_000)
    p = sc.data_ptr()
    e = lib.ExpertWeights(w, sc, stream=s)
    del sc
    again = torch.empty(16 * MB, dtype=torch.uint8, device="cuda")
    assert again.data_ptr() != p
    torch.cuda.synchronize()
    assert e.scale is not None


def test_metadata_copies_on_the_stream_it_is_prepared_on(lib):
    s = torch.cuda.Stream()
    meta = lib.TokenMeta(300, 4)
    slot = torch.arange(300, dtype=torch.int32, device="cuda") % 4
    meta.prepare(torch.zeros_like(slot), stream=s)     # the kernel is loaded, which waits for the device
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)                     # the current stream is busy with something else
    meta.prepare(slot, stream=s)
    s.synchronize()
    assert meta.seg_count[1:3].tolist() == [75, 75]
    assert torch.equal(meta.sorted_rows.sort().values, torch.arange(300, dtype=torch.int32, device="cuda"))


def test_a_calls_own_workspace_is_the_streams(lib, monkeypatch):
    table = lib.SlotTable(4096, [4096], 5, 64)
    meta = lib.TokenMeta(64, 5)
    meta.prepare(torch.ones(64, dtype=torch.int32, device="cuda"))
    x, y = torch.zeros(64, 4096, dtype=torch.bfloat16, device="cuda"), torch.zeros(64, 4096, device="cuda")
    s, seen = torch.cuda.Stream(), []
    own = lib.workspace

    def spy(*a, **k):
        seen.append(torch.cuda.current_stream().cuda_stream)
        return own(*a, **k)
    monkeypatch.setattr(lib, "workspace", spy)
    torch.cuda.synchronize()
    lib.apply(table, meta, x, y, stream=s)
    torch.cuda.synchronize()
    assert seen == [s.cuda_stream]
