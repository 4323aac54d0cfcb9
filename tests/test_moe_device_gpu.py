"""One tensor of a call on the CPU among others on the device: refused by name, nothing launched."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_each_tensor_is_checked(lib):
    def z(*s, dtype=torch.float32):
        return torch.zeros(*s, dtype=dtype, device="cuda")
    u8, i32 = torch.uint8, torch.int32
    meta = lib.TokenMeta(6, 3)
    meta.prepare(torch.ones(6, dtype=i32, device="cuda"))
    calls = [  # (call, the names of its tensors, in order)
        (lambda a: lib.moe_route(a[0], 2, expert_map=a[1], topk_ids=a[2], topk_w=a[3], pair_slot=a[4]),
         ["logits", "expert_map", "topk_ids", "topk_w", "pair_slot"],
         [z(3, 8), z(8, dtype=i32), z(3, 2, dtype=i32), z(3, 2), z(6, dtype=i32)]),
        (lambda a: lib.mx4_quantize(*a), ["x", "codes", "scales"], [z(3, 64), z(3, 32, dtype=u8), z(3, 16, dtype=u8)]),
        (lambda a: lib.mx4_dequantize(*a), ["codes", "scales", "y"], [z(3, 32, dtype=u8), z(3, 16, dtype=u8), z(3, 64)]),
        (lambda a: lib.moe_act(*a), ["y13", "h", "pair_slot"], [z(6, 32), z(6, 16), z(6, dtype=i32)]),
        (lambda a: lib.moe_act_mx4(*a), ["y13", "codes", "scales", "pair_slot"],
         [z(6, 64), z(6, 16, dtype=u8), z(6, 16, dtype=u8), z(6, dtype=i32)]),
        (lambda a: lib.moe_combine(*a), ["y", "topk_w", "out", "pair_slot"], [z(6, 16), z(3, 2), z(3, 16), z(6, dtype=i32)]),
        (lambda a: lib.moe_product(lib.ExpertWeights(a[2]), meta, *a[:2]), ["x", "y", "weights"], [z(6, 32), z(6, 16), z(2, 16, 32)]),
    ]
    for call, names, args in calls:
        call(args)
        torch.cuda.synchronize()
        n0 = lib.lora_launch_count()
        for i, name in enumerate(names):
            with pytest.raises(ValueError, match=f"{name}: expected a CUDA tensor"):
                call([t.cpu() if j == i else t for j, t in enumerate(args)])
        assert lib.lora_launch_count() == n0


def test_metadata_on_the_cpu(lib):
    with pytest.raises(ValueError, match="the metadata: expected a CUDA tensor"):
        lib.moe_product(lib.ExpertWeights(torch.zeros(2, 16, 32, device="cuda")), lib.TokenMeta(6, 3, device="cpu"),
                        torch.zeros(0, 32, device="cuda"), torch.zeros(0, 16, device="cuda"))


def test_overlapping_rows_of_logits(lib):
    with pytest.raises(ValueError, match="overlap"):
        lib.moe_route(torch.zeros(1, 64, device="cuda").expand(5, 64), 2)
