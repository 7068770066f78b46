"""CPU tests of the binding's checks of lengths and widths that C takes as 32 bits, on tensors without storage."""
import pytest
import torch


def i32(*shape):
    return torch.empty(*shape, dtype=torch.int32, device="meta")


MORE = 2 ** 32 + 2       # 2 where only the low bits are left


def test_requests(gkr):
    with pytest.raises(ValueError, match="past"):
        gkr.kv_allocate(i32(MORE), i32(MORE), i32(MORE, 1), i32(4), 64, 5)
    with pytest.raises(ValueError, match="lengths"):
        gkr.kv_slots(i32(MORE, 1), i32(MORE), 64, 5)
    with pytest.raises(ValueError, match="lengths"):
        gkr.kv_slots_packed(i32(MORE, 1), i32(MORE), 64, 5)
    q, kv = (torch.empty(*s, 512, dtype=torch.bfloat16, device="meta") for s in ((4, 2), (4,)))
    with pytest.raises(ValueError, match="starts"):
        gkr.prompt_attention(q, kv, i32(MORE), 1.0)


@pytest.mark.parametrize("width", [MORE, 2 ** 31])
def test_table_width(gkr, width):
    with pytest.raises(ValueError, match="block_table"):
        gkr.kv_allocate(i32(2), i32(2), i32(2, width), i32(4), 64, 5)
    with pytest.raises(ValueError, match="block_table"):
        gkr.kv_slots(i32(2, width), i32(2), 64, 5)
    with pytest.raises(ValueError, match="block_table"):
        gkr.kv_slots_packed(i32(2, width), i32(2), 64, 5)
