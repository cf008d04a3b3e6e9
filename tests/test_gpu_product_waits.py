"""Waits of the tensor-core products that run out, without a fault (needs a B200).

The self-test makes each step of K wait for 16 bytes more than its copies bring.
The wait gives up after its bound, the kernel records STQ1_DEV_WAIT_LIMIT, frees
what it holds and returns; sums that are not whole are never stored.
"""

import time

import pytest

torch = pytest.importorskip("torch")

if torch.cuda.is_available():
    import sub_bit_sparse_b200 as stq1

# K in eight pieces with more steps than stages, in two, whole; pairs of CTAs with few steps and with more than stages
SIZES = [(40, 256, 16384), (40, 256, 512), (100, 256, 512), (640, 4096, 512), (640, 4100, 2048)]


def _operands(t, n, k):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(t + n + k)
    code = lambda r: torch.randint(-127, 128, (r, k), generator=gen, device="cuda", dtype=torch.int8)  # noqa: E731
    scale = lambda r: torch.rand(r, generator=gen, device="cuda") + 0.5  # noqa: E731
    return code(t), scale(t), code(n), scale(n)


@pytest.mark.gpu
@pytest.mark.parametrize("t,n,k", SIZES)
def test_whole_sums_are_stored(t, n, k):
    ops = _operands(t, n, k)
    y = torch.full((t, n), 77.0, device="cuda")
    assert stq1.selftest_product(*ops, y, True) == 0
    assert torch.equal(y, stq1.i8_matmul(*ops)) and stq1.status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("t,n,k", SIZES)
def test_sums_of_a_wait_that_ran_out_are_not_stored(t, n, k):
    ops = _operands(t, n, k)
    y = torch.full((t, n), 77.0, device="cuda")
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    assert stq1.selftest_product(*ops, y, False) & stq1.DEV_WAIT_LIMIT
    assert time.perf_counter() - t0 < 10.0
    assert bool((y == 77.0).all())
    # the word is cleared by the read, and the next products run normally
    assert stq1.selftest_product(*ops, y, True) == 0
    assert torch.equal(y, stq1.i8_matmul(*ops)) and stq1.status() == 0


def test_refusals_need_no_gpu():
    import sub_bit_sparse_b200 as m
    f, P = m.LIB.stq1_selftest_product, 1 << 20
    for i in range(5):
        a = [P] * 5
        a[i] = None
        assert f(*a, 4, 8, 256, 0, None) == -2
    assert f(P, P, P, P, P, 4, 8, 256, 2, None) == -8
    for t, n, k in ((0, 8, 256), (4, 0, 256), (4, 8, 24), (4, 8, 131072)):
        assert f(P, P, P, P, P, t, n, k, 0, None) == -1
    for i, off in ((0, 8), (1, 2), (2, 8), (3, 2), (4, 8)):
        a = [P] * 5
        a[i] += off
        assert f(*a, 4, 8, 256, 0, None) == -6
