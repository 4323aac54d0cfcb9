"""What the tensor forms of the mixture-of-experts calls refuse before a kernel could use memory that is not
theirs (no GPU needed: each refusal comes before any launch)."""
import pytest
import torch

z = torch.zeros
U8 = dict(dtype=torch.uint8)
I32 = dict(dtype=torch.int32)


@pytest.fixture(scope="module")
def ra():
    import __graft_entry__
    __graft_entry__._load_build_lib().build()
    import rank_adapter_gb300
    return rank_adapter_gb300


class Meta:
    """What moe_product reads of a TokenMeta."""

    def __init__(self, ra, pairs):
        self.c = ra.Meta()
        self.c.num_tokens = pairs


@pytest.mark.parametrize("logits", [z(1, 64).expand(5, 64), z(64 + 4).as_strided((5, 64), (1, 1)), z(400).as_strided((5, 64), (63, 1))],
                         ids=["broadcast", "sliding", "one short"])
def test_route_refuses_overlapping_rows(ra, logits):
    with pytest.raises(ValueError, match="overlap"):
        ra.moe_route(logits, 2, topk_ids=z(5, 2, **I32), topk_w=z(5, 2))


def test_every_matrix_refuses_overlapping_rows(ra):
    for call in (lambda: ra.mx4_quantize(z(1, 64).expand(3, 64), z(3, 32, **U8), z(3, 16, **U8)),
                 lambda: ra.moe_act(z(1, 32).expand(3, 32), z(3, 16)),
                 lambda: ra.moe_act(z(3, 32), z(1, 16).expand(3, 16)),
                 lambda: ra.moe_combine(z(1, 16).expand(6, 16), z(3, 2), z(3, 16)),
                 lambda: ra.moe_product(ra.ExpertWeights(z(2, 16, 32)), Meta(ra, 4), z(1, 32).expand(4, 32), z(4, 16))):
        with pytest.raises(ValueError, match="overlap"):
            call()


# One row of 512 elements has 16 scale bytes; a row of 7168 has 224.
@pytest.mark.parametrize("rows,cols,scales", [(1, 512, z(1, 1, **U8)), (1, 512, z(1, 15, **U8)), (3, 512, z(3, 16, **U8)[:, :1]),
                                              (5, 7168, z(5, 224, **U8)[:, :223]), (1, 7168, z(1, 209, **U8)), (2, 64, z(2, 16, **U8)[:, :1])])
def test_narrow_scales_are_refused(ra, rows, cols, scales):
    codes = z(rows, cols // 2, **U8)
    for call in (lambda: ra.mx4_quantize(z(rows, cols), codes, scales),
                 lambda: ra.mx4_dequantize(codes, scales, z(rows, cols)),
                 lambda: ra.moe_act_mx4(z(rows, 2 * cols), codes, scales)):
        with pytest.raises(ValueError, match="scales: expected at least"):
            call()
    w = ra.ExpertWeights(z(2, 16, cols // 2))
    w.desc.dtype, w.desc.d_in = ra.LORA_MXFP4, cols
    with pytest.raises(ValueError, match="x_scale: expected at least"):
        ra.moe_product(w, Meta(ra, rows), codes, z(rows, 16), x_scale=scales)


def test_x_scale_rows_are_whole_in_memory(ra):
    """A product loads scale bytes 16 at a time: the last row's memory reaches to a multiple of 16."""
    w = ra.ExpertWeights(z(2, 16, 96 // 2))
    w.desc.dtype, w.desc.d_in = ra.LORA_MXFP4, 96
    short = (z(1, 3, **U8), z(16 + 3, **U8).as_strided((2, 3), (16, 1)), z(2, 16, **U8)[1:, 3:])
    for s in short:
        with pytest.raises(ValueError, match="x_scale: expected rows of 16 bytes"):
            ra.moe_product(w, Meta(ra, s.size(0)), z(s.size(0), 48, **U8), z(s.size(0), 16), x_scale=s)


def test_tensors_on_the_cpu_are_refused(ra):
    codes, scales = z(3, 32, **U8), z(3, 16, **U8)
    ids, w, slot = z(3, 2, **I32), z(3, 2), z(6, **I32)
    for call in (lambda: ra.moe_route(z(3, 8), 2, topk_ids=ids, topk_w=w, pair_slot=slot),
                 lambda: ra.mx4_quantize(z(3, 64), codes, scales),
                 lambda: ra.mx4_dequantize(codes, scales, z(3, 64)),
                 lambda: ra.moe_act(z(6, 32), z(6, 16), pair_slot=slot),
                 lambda: ra.moe_act_mx4(z(3, 128), codes, scales),
                 lambda: ra.moe_combine(z(6, 16), w, z(3, 16), pair_slot=slot),
                 lambda: ra.moe_product(ra.ExpertWeights(z(2, 16, 32)), Meta(ra, 4), z(4, 32), z(4, 16)),
                 lambda: ra.ExpertWeights(z(2, 16, 16, **U8), z(2, 16, 16, **U8))):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_shapes_and_types_are_named_before_the_device(ra):
    with pytest.raises(TypeError, match="h: expected bf16 or fp32"):
        ra.moe_act(z(4, 32), z(4, 16, dtype=torch.float16))
    with pytest.raises(ValueError, match="pair_slot: expected 4"):
        ra.moe_act(z(4, 32), z(4, 16), pair_slot=z(3, **I32))
