"""Products of FP4 weights over row counts up to the documented 2^31 - 1, whose
launches would count more than 2^32 threads: exact on small integers."""
import pytest
import torch

import linear_ref as ref
from gpu_helpers import DEV, note
from microscaling_fp4_block_fp4q_amd import fp4q as F
from test_gpu_linear import gen, integers

pytestmark = pytest.mark.gpu

CHUNK = 1 << 22


@pytest.fixture(autouse=True)
def memory_back():
    yield
    torch.cuda.empty_cache()


def room(gib):
    if torch.cuda.mem_get_info()[0] < gib << 30:
        pytest.skip(f"needs {gib} GiB of device memory")


def many_integers(rows, cols, seed):
    """bf16 [rows, cols] of small integers: a random block, repeated with a
    period that is no multiple of a tile."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    block = torch.randint(-4, 5, (99991, cols), generator=g, device=DEV).bfloat16()
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device=DEV)
    for a in range(0, rows, 99991):
        n = min(99991, rows - a)
        x[a:a + n] = block[:n]
    return x


@pytest.mark.parametrize("fmt,M,N,K,grad,gib", [
    # the few-row kernel (weights too small for the tiles): 2^23 workgroups of 512
    ("mxfp4", (1 << 27) + 37, 1, 32, False, 14),
    # 16-bit rows copied to whole steps: 2^32 pieces of 8 values
    ("mxfp4", (1 << 27) + 19, 8, 32, False, 90),
    # the gradient's largest tiles in several launches
    ("nvfp4", (1 << 27) + 300, 64, 16, True, 30)])
def test_many_rows(fmt, M, N, K, grad, gib):
    note(f"linear many rows {fmt} {M} {N} {K} grad={grad}")
    room(gib)
    cfg = ref.FORMATS[fmt]
    codes, scales = ref.exact_weights(cfg, (N,), K, gen(N))
    w = ref.decode(codes, scales, cfg).float().to(DEV)
    x = many_integers(M, N if grad else K, 1)
    fn = F.linear_grad if grad else F.linear
    y = fn(x, codes.to(DEV), scales.to(DEV), cfg, out_dtype=torch.float32)
    torch.cuda.synchronize()
    for a in range(0, M, CHUNK):
        part = x[a:a + CHUNK].float()
        assert torch.equal(y[a:a + CHUNK], part @ w if grad else part @ w.t()), a


def gathered(E, edges):
    """R = 2^31 - 2 gathered rows of E experts; rows past the last edge are zeros."""
    cfg, dtype = F.mxfp4(), torch.bfloat16
    T, N, K = 1302, 8, 64
    R = (1 << 31) - 2
    room(60)
    k, g = R // T, gen(E)
    assert T * k == R
    codes, scales = ref.exact_weights(cfg, (E, N), K, g)
    x = integers((T, K), g)
    table = (x.double() @ ref.decode(codes, scales, cfg).transpose(1, 2)).to(dtype).to(DEV)     # [E, T, N]
    rows = torch.randint(0, R, (R,), generator=torch.Generator(device=DEV).manual_seed(E), device=DEV,
                         dtype=torch.int32)
    off = torch.tensor([0] + edges, dtype=torch.int32, device=DEV)
    y = F.moe_linear(x.to(dtype).to(DEV), codes.to(DEV), scales.to(DEV), cfg, off, rows=rows)
    torch.cuda.synchronize()
    for e, (lo, hi) in enumerate(zip([0] + edges, edges)):
        for a in range(lo, hi, 1 << 24):
            b = min(a + (1 << 24), hi)
            assert torch.equal(y[a:b], table[e][torch.div(rows[a:b], k, rounding_mode="floor").long()]), (e, a)
    assert bool((y[edges[-1]:] == 0).all())


def test_experts_of_many_rows():
    note("moe_linear 2^31 - 2 rows of 3 experts")
    gathered(3, [700000001, 1500000000, (1 << 31) - 1000])


def test_one_expert_of_almost_all_rows_that_int32_holds():
    """Fewer than a tile below 2^31: the expert's tiles are still counted right."""
    note("moe_linear 2^31 - 2 rows of 1 expert")
    gathered(1, [(1 << 31) - 2])
