"""Products of FP4 weights through kernels and sizes that need a case of their
own to be reached: exact on small integers, whatever the order of the sums."""
import pytest
import torch

import linear_ref as ref
from gpu_helpers import DEV, note
from microscaling_fp4_block_fp4q_amd import fp4q as F
from test_gpu_linear import gen, integers, routed, same, strided

pytestmark = pytest.mark.gpu


def check_dense(fmt, dt, M, N, K, grad):
    cfg, dtype = ref.FORMATS[fmt], ref.DTYPES[dt]
    note(f"linear kernels {fmt} {dt} {M} {N} {K} grad={grad}")
    g = gen(M + N + K)
    codes, scales = ref.exact_weights(cfg, (N,), K, g)
    codes, scales = codes.to(DEV), scales.to(DEV)
    w = ref.decode(codes, scales, cfg)
    x = integers((M, N if grad else K), g).to(DEV)
    got = (F.linear_grad if grad else F.linear)(strided(x, dtype, extra=0), codes, scales, cfg,
                                                out_dtype=torch.float32)
    torch.cuda.synchronize()
    same(got, x.double() @ w if grad else x.double() @ w.t(), f"{M} x {N} x {K}")


def check_experts(fmt, dt, T, k, E, N, K, grad, only=None):
    cfg, dtype = ref.FORMATS[fmt], ref.DTYPES[dt]
    note(f"moe kernels {fmt} {dt} {T} {k} {E} {N} {K} grad={grad}")
    g = gen(T + N + K)
    off, rows, _ = routed(T, k, E, 1, only=only)
    codes, scales = ref.exact_weights(cfg, (E, N), K, g)
    codes, scales, off, rows = (t.to(DEV) for t in (codes, scales, off, rows))
    w = ref.decode(codes, scales, cfg)
    x = integers((T * k if grad else T, N if grad else K), g).to(DEV)
    src = x.double() if grad else x[(rows.clamp_min(0) // k).long()].double()
    src[int(off[-1]):] = 0
    if grad:
        got = F.moe_linear_grad(strided(x, dtype), codes, scales, cfg, off, out_dtype=torch.float32)
    else:
        got = F.moe_linear(strided(x, dtype), codes, scales, cfg, off, rows=rows, out_dtype=torch.float32)
    torch.cuda.synchronize()
    same(got, ref.grouped(src, w, off, transposed=grad))


@pytest.mark.parametrize("fmt,dt,M,N,K", [("nvfp4", "f32", 1030, 4097, 4112), ("mxfp4", "f32", 1030, 4097, 4128),
                                          ("mxfp4", "f16", 1030, 4097, 6176)])
def test_planes_by_turns_over_a_last_tile_of_one_row(fmt, dt, M, N, K):
    """256 x 256 tiles with planes by turns, whose steps go on past K to a whole
    group of four: the last tile holds one row of codes, the last of the array."""
    check_dense(fmt, dt, M, N, K, False)


def test_planes_by_turns_over_a_last_expert_tile_of_one_row():
    check_experts("nvfp4", "f32", 1200, 2, 2, 2049, 4112, False)
