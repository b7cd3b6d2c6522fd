"""Every kernel that the products of FP4 weights can choose is run by a case of
the exact-integer GPU tests (host only: the choice is asked, nothing runs)."""
import os

import pytest

import linear_plan as P
import test_gpu_linear as small
import test_gpu_linear_kernels as kernels

pytestmark = pytest.mark.skipif(not os.path.exists(P.PROBE_LIB), reason="libfp4q_probe.so not built")


def cases_of(test):
    """The parameters of a test with one parametrize mark."""
    mark, = [m for m in test.pytestmark if m.name == "parametrize"]
    return mark.args[1]


def plans():
    """(plan, case) of the exact-integer cases."""
    def width(c, extra=8):
        return (c + 7) // 8 * 8 + extra
    for fmt in small.FMT:
        for dt in small.DTS:
            for i, (M, N, K) in enumerate(small.SHAPES):
                K = K + 16 if fmt == "nvfp4" and i % 2 else K
                for grad in (False, True):
                    yield P.plan(fmt, dt, grad, M, N, K), (M, N, K)
            for i, (T, k, E, N, K, _) in enumerate(small.MOE):
                K = K + 16 if fmt == "nvfp4" and i % 2 else K
                yield P.plan(fmt, dt, False, T * k, N, K, E, T, width(K)), (T, k, E, N, K)
                yield P.plan(fmt, dt, True, T * k, N, K, E), (T, k, E, N, K)
    for fmt, dt, M, N, K, grad in cases_of(small.test_exact_on_integers_large) + kernels.DENSE:
        yield P.plan(fmt, dt, grad, M, N, K), (fmt, dt, M, N, K, grad)
    for fmt, dt, T, k, E, N, K, grad in cases_of(small.test_experts_exact_on_integers_large):
        yield P.plan(fmt, dt, grad, T * k, N, K, E, 0 if grad else T, width(K)), (fmt, dt, T, k, E, N, K, grad)
    for fmt, dt, T, k, E, N, K, grad, ld in kernels.EXPERTS:
        yield (P.plan(fmt, dt, grad, T * k, N, K, E, 0 if grad else T, ld or width(K, 0)),
               (fmt, dt, T, k, E, N, K, grad, ld))


def test_every_kernel_is_reached():
    seen = {p.kernel for p, _ in plans()}
    assert seen <= P.every_kernel(), seen - P.every_kernel()
    assert seen == P.every_kernel(), sorted(map(str, P.every_kernel() - seen))


def test_every_way_of_the_activations_and_the_sum_is_reached():
    """Activations as given and copied, gathered by the copy, and sums in parts,
    by every kind of kernel that can."""
    every = [p for p, _ in plans()]
    for grad in (False, True):
        for kind in P.KINDS[1:]:
            mine = [p for p in every if p.kernel.kind == kind and p.kernel.grad is grad]
            if kind == "tile32" and grad:
                assert not mine
                continue
            assert {p.copy for p in mine} == {False, True}, (kind, grad)
            assert any(p.splits > 1 for p in mine) and any(p.splits == 1 for p in mine), (kind, grad)
    assert any(p.gathered for p in every)
