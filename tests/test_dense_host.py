"""The 8-bit integer and gated-block definitions, and the calls' refusals (no GPU)."""

import numpy as np
import pytest

import oracle
from oracle import dense

P = 1 << 20


def test_codes_span_the_row_and_round_to_even():
    v = np.array([[127, -127, 0.5, 1.5, 2.5, -0.5, -1.5, 126.5]], dtype=np.float32)   # inv = 1: ties stay ties
    q, s = dense.quantize_i8(v)
    assert q.tolist() == [[127, -127, 0, 2, 2, 0, -2, 126]] and s[0] == 1.0


def test_codes_never_leave_the_range_and_are_within_half_a_step():
    rng = np.random.default_rng(0)
    v = (rng.standard_normal((64, 512)) * 10.0 ** rng.uniform(-30, 30, (64, 1))).astype(np.float32)
    q, s = dense.quantize_i8(v)
    assert np.abs(q.astype(int)).max() == 127
    # src * (127 / amax) carries two fp32 roundings of values up to 127 on top of the half step, the scale one
    err = np.abs(v.astype(np.float64) - q * s[:, None].astype(np.float64))
    assert np.all(err <= s[:, None] * (0.5 + 127 * 3 * 2.0 ** -24))


def test_zero_tiny_and_non_finite_rows():
    v = np.zeros((5, 16), dtype=np.float32)
    v[1, 3], v[2, 3], v[3, 3], v[4, 3] = 2.0 ** -120, 2.0 ** -119, np.inf, np.nan
    q, s = dense.quantize_i8(v)
    assert not q[[0, 1, 3, 4]].any() and q[2, 3] == 127
    assert s[0] == 0 and s[1] == 0 and s[2] > 0 and np.isinf(s[3]) and np.isnan(s[4])
    y = dense.i8_matmul(q, s, np.ones((2, 16), np.int8), np.ones(2, np.float32))
    assert np.isnan(y[3:]).all() and np.isfinite(y[:3]).all()


def test_gradient_formula_against_differences():
    rng = np.random.default_rng(1)
    x, w = rng.standard_normal((3, 8)), rng.standard_normal((6, 8)) * 0.7
    dact = rng.standard_normal((3, 3))
    dx, dw = dense.glu_backward(dact, dense.glu(x, w)[1], x, w)
    f = lambda x, w: float((dense.glu(x, w)[0] * dact).sum())  # noqa: E731
    h = 1e-5
    # central differences: h^2/6 times a third derivative of order 100, and 2^-52 * |f| / h
    for a, grad, at in ((x, dx, lambda d: f(x + d, w)), (w, dw, lambda d: f(x, w + d))):
        for i in np.ndindex(a.shape):
            d = np.zeros_like(a)
            d[i] = h
            assert abs((at(d) - at(-d)) / (2 * h) - grad[i]) < 1e-7


def test_gradients_at_the_ends_of_the_gate():
    dy = dense.glu_dy(np.ones((1, 3)), np.array([[-200.0, 0.0, 200.0, 2.0, 2.0, 2.0]]))
    assert np.allclose(dy, [[0, 1, 2, 0, 0, 200]], atol=1e-80)


def test_refusals_need_no_gpu():
    import sub_bit_sparse_b200 as m
    L = m.LIB
    q, mm, ffn, glu, back = L.stq1_quantize_i8, L.stq1_i8_matmul, L.stq1_i8_ffn, L.stq1_glu, L.stq1_glu_backward
    big = 1 << 31
    assert q(None, 1, 4, 256, P, P, None) == -2 and q(P, 1, 4, 256, None, P, None) == -2
    assert q(P, 1, 4, 256, P, None, None) == -2
    assert q(P, 2, 4, 256, P, P, None) == -8
    for r, k in ((0, 256), (-1, 256), (4, 0), (4, 8), (4, 250), (big, 16), (4, big), (1 << 30, 1 << 12)):
        assert q(P, 1, r, k, P, P, None) == -1, (r, k)
    assert q(P + 8, 1, 4, 256, P, P, None) == -6 and q(P, 1, 4, 256, P + 8, P, None) == -6
    assert q(P, 1, 4, 256, P, P + 2, None) == -6

    for i in range(5):
        a = [P] * 5
        a[i] = None
        assert mm(*a, 0, 4, 8, 256, None) == -2
    assert mm(P, P, P, P, P, 3, 4, 8, 256, None) == -8
    for t, n, k in ((0, 8, 256), (4, 0, 256), (4, 8, 0), (4, 8, 24), (4, 8, 131072), (big, 8, 256), (1 << 30, 1 << 20, 16)):
        assert mm(P, P, P, P, P, 0, t, n, k, None) == -1, (t, n, k)
    for i, off in ((0, 8), (1, 2), (2, 8), (3, 2), (4, 8)):
        a = [P] * 5
        a[i] += off
        assert mm(*a, 0, 4, 8, 256, None) == -6

    need = L.stq1_i8_ffn_workspace(4, 64, 128)
    assert need > 0 and L.stq1_i8_ffn_workspace(4, 48, 128) == 0 and L.stq1_i8_ffn_workspace(4, 64, 120) == 0
    for i in range(6):
        a = [P] * 6
        a[i] = None
        assert ffn(*a, 4, 64, 128, P, need, None) == -2
    for t, n, h in ((0, 64, 128), (4, 63, 128), (4, 48, 128), (4, 64, 8), (4, 64, 131072), (4, 262144, 16)):
        assert ffn(*[P] * 6, t, n, h, P, 1 << 40, None) == -1, (t, n, h)
    assert ffn(*[P] * 6, 4, 64, 128, None, need, None) == -7 and ffn(*[P] * 6, 4, 64, 128, P, need - 1, None) == -7
    for i, off in ((0, 8), (1, 8), (2, 2), (3, 8), (4, 2), (5, 8)):
        a = [P] * 6
        a[i] += off
        assert ffn(*a, 4, 64, 128, P, need, None) == -6
    assert ffn(*[P] * 6, 4, 64, 128, P + 8, need, None) == -6

    for i in range(3):
        a = [P] * 3
        a[i] = None
        assert glu(*a, None, 4, 64, 128, None) == -2
    for t, n, k in ((0, 64, 128), (4, 63, 128), (4, 24, 128), (4, 64, 4), (4, 64, 100), (4, 64, big)):
        assert glu(P, P, P, P, t, n, k, None) == -1, (t, n, k)
    for i in range(4):
        a = [P] * 4
        a[i] += 8
        assert glu(*a, 4, 64, 128, None) == -6

    need = L.stq1_glu_backward_workspace(4, 64, 128)
    assert need == 4 * 64 * 2 and L.stq1_glu_backward_workspace(4, 24, 128) == 0
    # dact, y, x, W, dx, dW
    assert back(None, P, P, P, P, P, 4, 64, 128, P, need, None) == -2
    assert back(P, None, P, P, P, P, 4, 64, 128, P, need, None) == -2
    assert back(P, P, P, P, None, None, 4, 64, 128, P, need, None) == -2
    assert back(P, P, None, P, P, P, 4, 64, 128, P, need, None) == -2      # dW without x
    assert back(P, P, P, None, P, P, 4, 64, 128, P, need, None) == -2      # dx without W
    for t, n, k in ((0, 64, 128), (4, 63, 128), (4, 24, 128), (4, 64, 4)):
        assert back(P, P, P, P, P, P, t, n, k, P, 1 << 40, None) == -1, (t, n, k)
    assert back(P, P, P, P, P, P, 4, 64, 128, None, need, None) == -7
    assert back(P, P, P, P, P, P, 4, 64, 128, P, need - 1, None) == -7
    for i in range(6):
        a = [P] * 6
        a[i] += 8
        assert back(*a, 4, 64, 128, P, need, None) == -6
    assert back(P, P, P, P, P, P, 4, 64, 128, P + 8, need, None) == -6


def test_binding_refuses_host_tensors_and_wrong_types():
    torch = pytest.importorskip("torch")
    import sub_bit_sparse_b200 as m
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    q, s = torch.zeros((4, 64), dtype=torch.int8), torch.zeros(4)
    for call in (lambda: m.quantize_i8(x), lambda: m.i8_matmul(q, s, q, s), lambda: m.glu(x, x),
                 lambda: m.glu_backward(x, x, x, x), lambda: m.i8_ffn(x, q, s, q, s)):
        with pytest.raises(TypeError):
            call()


def test_activation_is_the_one_swiglu_gives():
    y = np.random.default_rng(2).standard_normal((4, 32)) * 3
    act = oracle.swiglu_bf16(y, 32)
    assert np.array_equal(act, oracle.bf16_bits_from_f64(oracle.silu(y[:, :16]) * y[:, 16:]))
