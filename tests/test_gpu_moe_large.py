"""The combination and its gradients at sizes whose launches count more than
2^32 threads: 2^24 workgroups of 256 and more."""
import pytest
import torch

from gpu_helpers import DEV, note
from microscaling_fp4_block_fp4q_amd import fp4q as F

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def memory_back():
    yield
    torch.cuda.empty_cache()


def test_combine_gradients_of_many_entries():
    """2^21 tokens of 8 entries: a workgroup per token and row is more than 2^24.
    The last entries of some tokens are dropped, so rows past the entries are zeros."""
    T, k, N = (1 << 21) + 5, 8, 8
    note(f"moe_combine_grad {T} tokens of {k}")
    g = torch.Generator(device=DEV).manual_seed(0)
    live = torch.rand(T, k, generator=g, device=DEV) < 0.9
    place = live.flatten().cumsum(0, dtype=torch.int32).reshape(T, k)
    slots = torch.where(live, place - 1, -1)
    n = int(place[-1, -1])
    off = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    dy = torch.randint(-4, 5, (T, N), generator=g, device=DEV).float()
    h = torch.randint(-4, 5, (T * k, N), generator=g, device=DEV).float()
    w = torch.randint(-4, 5, (T, k), generator=g, device=DEV).float()
    dh, dw = F.moe_combine_grad(dy, h, slots, off, w)
    torch.cuda.synchronize()
    assert bool((dh[n:] == 0).all())
    assert torch.equal(dh[:n], (w[..., None] * dy[:, None])[live])
    want = torch.zeros(T, k, device=DEV)
    want[live] = (h[:n] * dy[:, None].expand(T, k, N)[live]).sum(-1)
    assert torch.equal(dw, want)


def test_combination_of_many_columns_and_tokens():
    """2^23 tokens of 4096 columns: 2^32 pieces of 8 columns, 64 GiB of results."""
    T, N, R = (1 << 23) + 3, 4096, 16
    note(f"moe_combine {T} tokens of {N} columns")
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("needs 80 GiB of device memory")
    g = torch.Generator(device=DEV).manual_seed(1)
    h = torch.randn(R, N, generator=g, device=DEV).bfloat16()
    slots = torch.randint(0, R, (T, 1), generator=g, device=DEV, dtype=torch.int32)
    y = F.moe_combine(h, slots)
    torch.cuda.synchronize()
    for a in range(0, T, 1 << 17):
        assert torch.equal(y[a:a + (1 << 17)], h[slots[a:a + (1 << 17), 0].long()]), a
