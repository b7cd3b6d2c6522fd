"""Products of FP4 weights through kernels and sizes that need a case of their
own to be reached: exact on small integers, and on one value a row that fills
the planes of its type, whatever the order of the sums."""
import pytest
import torch

import linear_ref as ref
from gpu_helpers import DEV, note
from microscaling_fp4_block_fp4q_amd import fp4q as F
from test_gpu_linear import gen, routed, same

pytestmark = pytest.mark.gpu


# (format, type, M, N, K, gradient)
DENSE = [
    # planes by turns, whose steps go on past K to a whole group of four, over a last tile of one row of codes
    ("nvfp4", "f32", 1030, 4097, 4112, False), ("mxfp4", "f32", 1030, 4097, 4128, False),
    ("mxfp4", "f16", 1030, 4097, 6176, False),
    # fp16 activations as they are in the largest tiles, whole steps and copied rows
    ("nvfp4", "f16", 2100, 4100, 6224, False), ("nvfp4", "f16", 2100, 4100, 6208, False),
    ("nvfp4", "f16", 1300, 8192, 4112, True), ("nvfp4", "f16", 1300, 8200, 4112, True),
    # the gradient's largest tiles with planes by turns
    ("mxfp4", "f16", 1030, 4700, 4128, True), ("mxfp4", "f32", 1030, 3300, 4128, True),
    ("nvfp4", "f32", 1030, 3300, 4112, True)]
# few rows of wide weights: 32 and 64 weight rows a workgroup, sums that end inside a chunk of 128
DENSE += [(fmt, dt, M, N, 2352 if fmt == "nvfp4" else 2336, False) for fmt in ("mxfp4", "nvfp4")
          for dt in ("bf16", "f16", "f32") for M, N in ((1, 7200), (3, 14344), (16, 7200), (16, 14344))]

# (format, type, T, k, E, N, K, gradient, row stride of a gathered x or 0)
EXPERTS = [("nvfp4", "f32", 1200, 2, 2, 2049, 4112, False, 0)]
# x gathered from more than 4 GiB by every tile
FAR = 1 << 21
EXPERTS += [(fmt, dt, 1100, k, E, N, K, False, FAR) for fmt, dt in (("mxfp4", "bf16"), ("nvfp4", "bf16"), ("nvfp4", "f16"))
            for k, E, N, K in ((1, 40, 150, 192), (2, 10, 150, 192), (2, 3, 150, 192), (8, 8, 4100, 1408))]
# planes of 4 GiB and more, beyond the small tiles' offsets
EXPERTS += [("mxfp4", "f32", 1200, 1, 2, 130, 596576, False, 0), ("nvfp4", "f32", 1200, 1, 2, 130, 596592, False, 0),
            ("mxfp4", "f16", 1200, 1, 2, 130, 894816, False, 0),
            ("mxfp4", "f32", 1200, 1, 2, 596600, 160, True, 0), ("nvfp4", "f32", 1200, 1, 2, 596600, 144, True, 0),
            ("mxfp4", "f16", 1200, 1, 2, 894824, 160, True, 0),
            # one plane of 4 GiB: gathered when the planes are made
            ("nvfp4", "f32", 1200, 1, 2, 20, 1789552, False, 0)]


@pytest.fixture(autouse=True)
def memory_back():
    yield
    torch.cuda.empty_cache()


def device_integers(rows, cols, seed, dtype, ld):
    """[rows, cols] of small integers in rows of ld values, NaN between them (not
    filled where rows are far apart)."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    buf = torch.empty(rows, ld, dtype=dtype, device=DEV)
    if ld < 2 * cols + 64:
        buf.fill_(float("nan"))
    buf[:, :cols] = torch.randint(-4, 5, (rows, cols), generator=g, device=DEV, dtype=torch.int8)
    return buf[:, :cols]


# one value of a row in all planes of its type: 18 (11) significant bits in three (two) groups, so that its
# product with a weight of 6 is exact in fp32, whatever the order of the planes
ALL_PLANES = {"f32": 2.0 ** 17 + 2 ** 8 + 1, "f16": 2.0 ** 10 + 1, "bf16": 129.0}


def one_value_a_row(x, dt):
    rows, cols = x.shape
    m = torch.arange(rows, device=DEV)
    x.zero_()
    x[m, m * 7919 % cols] = torch.where(m % 2 == 0, 1.0, -1.0).to(x.dtype) * ALL_PLANES[dt]


@pytest.mark.parametrize("planes", [False, True], ids=["integers", "planes"])
@pytest.mark.parametrize("fmt,dt,M,N,K,grad", DENSE)
def test_dense(fmt, dt, M, N, K, grad, planes):
    cfg, dtype = ref.FORMATS[fmt], ref.DTYPES[dt]
    note(f"linear kernels {fmt} {dt} {M} {N} {K} grad={grad}")
    codes, scales = ref.exact_weights(cfg, (N,), K, gen(M + N + K))
    codes, scales = codes.to(DEV), scales.to(DEV)
    w = ref.decode(codes, scales, cfg)
    C = N if grad else K
    x = device_integers(M, C, M, dtype, (C + 7) // 8 * 8)
    if planes:
        one_value_a_row(x, dt)
    got = (F.linear_grad if grad else F.linear)(x, codes, scales, cfg, out_dtype=torch.float32)
    torch.cuda.synchronize()
    same(got, x.double() @ w if grad else x.double() @ w.t(), f"{M} x {N} x {K}")


@pytest.mark.parametrize("planes", [False, True], ids=["integers", "planes"])
@pytest.mark.parametrize("fmt,dt,T,k,E,N,K,grad,ld", EXPERTS)
def test_experts(fmt, dt, T, k, E, N, K, grad, ld, planes):
    """Long sums stay exact: their terms are multiples of 1/16 below 96, and sums
    of two million of random sign lie far below 2^20."""
    cfg, dtype = ref.FORMATS[fmt], ref.DTYPES[dt]
    note(f"moe kernels {fmt} {dt} {T} {k} {E} {N} {K} grad={grad} ld={ld}")
    off, rows, _ = routed(T, k, E, 1)
    codes, scales = ref.exact_weights(cfg, (E, N), K, gen(T + N + K))
    codes, scales, off, rows = (t.to(DEV) for t in (codes, scales, off, rows))
    C, n = N if grad else K, int(off[-1])
    x = device_integers(T * k if grad else T, C, T, dtype, ld or (C + 7) // 8 * 8)
    if planes:
        one_value_a_row(x, dt)
    if grad:
        got = F.moe_linear_grad(x, codes, scales, cfg, off, out_dtype=torch.float32)
    else:
        got = F.moe_linear(x, codes, scales, cfg, off, rows=rows, out_dtype=torch.float32)
    torch.cuda.synchronize()
    assert bool((got[n:] == 0).all())
    o = off.tolist()
    for e in range(E):
        a, b = o[e], o[e + 1]
        w = ref.decode(codes[e], scales[e], cfg)
        part = (x[a:b] if grad else x[(rows[a:b] // k).long()]).double()
        same(got[a:b], part @ w if grad else part @ w.t(), f"expert {e}")
