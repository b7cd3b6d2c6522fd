"""Expert ids of every integer type, in range and outside."""
import pytest
import torch

import linear_ref as ref
from gpu_helpers import DEV, note
from microscaling_fp4_block_fp4q_amd import fp4q as F

pytestmark = pytest.mark.gpu


def check(ids, E):
    r = F.moe_sort(ids.to(DEV), E)
    torch.cuda.synchronize()
    for name, want in zip(("offsets", "rows", "slots"), ref.sort_table(ids.long().clamp(-1, E).numpy(), E)):
        assert torch.equal(r[name].cpu(), torch.from_numpy(want)), name


def test_64_bit_ids_outside_32_bits_belong_to_no_expert():
    note("moe_sort 64-bit ids")
    check(torch.tensor([[1, (1 << 32) + 1], [-(1 << 63), 0], [(1 << 63) - 1, 2], [(1 << 31), -(1 << 31)],
                        [(1 << 32), -1], [3, 4], [-(1 << 32) + 2, 1 << 40]]), 4)
    ids = torch.randint(-2, 7, (3000, 4), generator=torch.Generator().manual_seed(0))
    ids[::7] += 1 << 32
    ids[::11] -= 1 << 32
    check(ids, 5)
    check(ids.t().contiguous().t(), 5)                              # not contiguous


@pytest.mark.parametrize("dtype", [torch.int32, torch.int16, torch.int8, torch.uint8, torch.uint16, torch.uint32,
                                   torch.uint64])
def test_ids_of_other_integer_types(dtype):
    note(f"moe_sort ids {dtype}")
    ids = torch.randint(0, 9, (100, 3), generator=torch.Generator().manual_seed(1)).to(dtype)
    check(ids, 7)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.bool])
def test_ids_that_are_no_integers_are_refused(dtype):
    with pytest.raises(TypeError):
        F.moe_sort(torch.zeros(4, 2, device=DEV).to(dtype), 4)
