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
